"""Calls on a stream of their own: what they make must not be memory that the caller's stream still uses, and what
they use or return must not be handed out again early on either stream."""
import math
import types

import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
N = 4096    # activations of 4096 x 4096 fp32: blocks of their own size


class Slow:
    """Keeps a stream busy for some ten milliseconds without allocating."""

    def __init__(self):
        self.a = torch.randn(8192, 8192, device=DEV)
        self.out = torch.empty_like(self.a)

    def __call__(self, times=10):
        for _ in range(times):
            torch.mm(self.a, self.a, out=self.out)


def test_outputs_are_not_memory_that_the_current_stream_still_reads():
    st, slow = torch.cuda.Stream(DEV), Slow()
    x = torch.randn(N, N, device=DEV)
    want = dsa.layer_norm(x).clone()             # (the kernel is loaded; its output's memory is free again)
    late = torch.zeros(N, N, device=DEV)
    held = torch.full((N, N), 3.0, device=DEV)
    torch.cuda.synchronize()
    slow()
    late.copy_(held)
    del held
    y = dsa.layer_norm(x, stream=st)
    torch.cuda.synchronize()
    assert bool((late == 3.0).all())
    assert torch.equal(y, want)


def calls():
    b = workloads.ragged(7, [300, 200], [300, 900], H=64, d=128, k=64, integer=False)
    lay = dsa.Layout.from_batch(b, DEV)
    Q, K, W = b.Q.to(DEV), b.K.to(DEV), b.W.to(DEV)
    idx = dsa.index_topk(lay, Q, K, W, 64)
    ds = torch.randn(idx.shape, generator=torch.Generator().manual_seed(1)).to(DEV)
    teacher = ds.abs()
    pooled = dsa.hisa_pool_keys(lay, K, 64)
    _, cand = dsa.pivot_group_index(lay, Q, K, W, 64, 16, 128, dsa.REUSE, want_cand=True)
    x = torch.randn(500, 128, device=DEV)
    _, mean, rstd = dsa.layer_norm(x, want_stats=True)
    return {
        "layer_norm": lambda **kw: dsa.layer_norm(x, want_stats=True, **kw),
        "layer_norm_backward": lambda **kw: dsa.layer_norm_backward(x, x, None, mean, rstd, **kw),
        "distill_topk": lambda **kw: dsa.distill_topk(ds, teacher, lists=idx, kind=dsa.TEACHER_WEIGHTS, **kw),
        "list_scores": lambda **kw: dsa.list_scores(lay, Q, K, W, idx, **kw),
        "list_scores_backward": lambda **kw: dsa.list_scores_backward(lay, Q, K, W, idx, ds, **kw),
        "index_topk": lambda **kw: dsa.index_topk(lay, Q, K, W, 64, **kw),
        "pivot_group_index": lambda **kw: dsa.pivot_group_index(lay, Q, K, W, 64, 16, 128, dsa.REFINE, **kw),
        "pivot_refine_candidates": lambda **kw: dsa.pivot_refine_candidates(lay, Q, K, W, 64, 16, cand, **kw),
        "hisa_pool_keys": lambda **kw: dsa.hisa_pool_keys(lay, K, 64, **kw),
        "hisa_index": lambda **kw: dsa.hisa_index(lay, Q, K, W, pooled, 64, 64, 3, **kw),
    }


NAMES = ["layer_norm", "layer_norm_backward", "distill_topk", "list_scores", "list_scores_backward", "index_topk",
         "pivot_group_index", "pivot_refine_candidates", "hisa_pool_keys", "hisa_index"]


def tensors(x):
    return [x] if isinstance(x, torch.Tensor) else list(x)


@pytest.mark.parametrize("name", NAMES)
def test_workspaces_are_not_memory_that_the_current_stream_still_writes(name):
    """Memory of every size freed on the current stream, whose last write there is still pending."""
    call, st, slow = calls()[name], torch.cuda.Stream(DEV), Slow()
    want = [t.clone() for t in tensors(call())]
    for _ in range(2):
        junk = [torch.empty(2 ** e, dtype=torch.uint8, device=DEV) for e in range(9, 25) for _ in range(2)]
        torch.cuda.synchronize()
        slow()
        for t in junk:
            t.fill_(255)
        del junk, t
        got = call(stream=st)
        torch.cuda.synchronize()
        for u, v in zip(want, tensors(got)):
            assert torch.equal(u, v)


def test_results_stay_reserved_for_the_callers_stream():
    st, slow = torch.cuda.Stream(DEV), Slow()
    x, other = torch.randn(N, N, device=DEV), torch.randn(N, N, device=DEV)
    want = dsa.layer_norm(x)
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    y = dsa.layer_norm(x, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    slow()
    late.copy_(y)
    del y
    again = [dsa.layer_norm(other, stream=st) for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(late, want)
    del again


def test_arguments_stay_reserved_for_the_calls_stream():
    st, slow = torch.cuda.Stream(DEV), Slow()
    x = torch.randn(N, N, device=DEV)
    want = dsa.layer_norm(x)
    torch.cuda.synchronize()
    held = x.clone()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        slow()
    y = dsa.layer_norm(held, stream=st)
    del held
    junk = [torch.full((N, N), math.nan, device=DEV) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    del junk


def test_a_stream_of_another_device_is_refused():
    elsewhere = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    for name, call in calls().items():
        with pytest.raises(ValueError):
            call(stream=elsewhere)


def test_the_side_stream_of_several_layers_keeps_its_memory():
    """With an event per layer the caller's stream does not wait for the side stream, which still works on the
    inputs, the workspace and the rows when the call has returned."""
    b = workloads.ragged(9, [300, 200], [300, 900], H=64, d=128, k=64, integer=False)
    lay = dsa.Layout.from_batch(b, DEV)
    Q, K, W = b.Q.to(DEV), b.K.to(DEV), b.W.to(DEV)
    want = dsa.index_topk(lay, Q, K, W, 64)
    side, slow = torch.cuda.Stream(DEV), Slow()
    torch.cuda.synchronize()
    for _ in range(2):
        events = [torch.cuda.Event() for _ in range(4)]
        held = [[t.clone() for _ in range(4)] for t in (Q, K, W)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            slow()
        got = dsa.index_layers(lay, *held, 64, retain_every=2, events=events, side_stream=side)
        del held
        junk = [torch.full((2 ** e,), 255, dtype=torch.uint8, device=DEV) for e in range(9, 26) for _ in range(4)]
        torch.cuda.synchronize()
        for t in got:
            assert torch.equal(t, want)
        del junk
