"""The distillation loss where its arithmetic or its indices can go wrong: rows of every kernel form, long ones among
them, with masks of the type's lowest value."""
import math

import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
from train_ref import U, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
LOW = torch.finfo(F32).min


def gen(seed):
    return torch.Generator().manual_seed(seed)


def reference(s, t, lists, weights, tau, g):
    """((loss, ds), bounds) in 64 bits, rows together.

    An exponential's argument has three roundings of a value of magnitude |a| (3 U |a|), the exponential 4 U more; one
    whose |a| is above 104 is zero in fp32, or an error of 2^-126 of the row's largest.  A sum is taken by threads that
    hold k/512 terms at most and joined in 64 steps; where a running sum is rescaled, each batch of 8 terms may add a
    factor (5 U) whose argument is again at most 104, or that is zero.  So q and p are off by
    rel = 2 (3 A + k/512 + 5 k/4096 + 4 A + 116) U of themselves, A = min(max |a|, 104), twice for numerator and
    denominator together; the factors 2^-126 come to less than 2^-100.  The loss adds the cross terms' own roundings."""
    s, t = s.double(), t.double()
    n, k = s.shape
    live = s > -math.inf
    if lists is not None:
        live &= lists >= 0
    gr = torch.ones(n).double() if g is None else g.double()
    ninf = torch.full_like(s, -math.inf)
    a = torch.where(live, s, ninf) / tau
    a = a - a.amax(1, keepdim=True)
    zero = torch.zeros_like(s)
    if weights:
        v = torch.where(live, t, zero)
        p, logp = v / v.sum(1, keepdim=True), torch.log(v) - torch.log(v.sum(1, keepdim=True))
    else:
        v = torch.where(live, t, ninf) / tau
        v = v - v.amax(1, keepdim=True)
        p, logp = v.softmax(1), v.log_softmax(1)
    q, logq = a.softmax(1), a.log_softmax(1)
    ok = live.any(1) & ~p.isnan().any(1) & (p.sum(1) > 0)
    on = live & (p > 0) & ok[:, None]
    cross = torch.where(on, p * (logp - logq), zero)
    loss = torch.where(ok, cross.sum(1), torch.zeros(n).double())
    scale = (gr / tau)[:, None]
    ds = torch.where(live & ok[:, None], scale * (q - p), zero)
    size = torch.where(live & (a.abs() < 104), a.abs(), zero).amax(1)
    rel = 2 * (7 * size + k / 512 + 5 * k / 4096 + 116) * U
    e_ds = torch.where(live & ok[:, None], scale.abs() * ((q + p) * rel[:, None] + 2.0 ** -100), zero)
    mag = torch.where(on, p * (logp.abs() + logq.abs()), zero).sum(1)
    e_loss = torch.where(ok, rel * mag + 2 * rel + 2.0 ** -100, torch.zeros(n).double())
    return (loss, ds), (e_loss, e_ds)


def values(g, n, k, tt, weights, lists):
    """Scores, teacher and lists with dropped places; whatever stands in those does not count."""
    s, t = torch.randn(n, k, generator=g) * 2, torch.randn(n, k, generator=g) * 2
    if weights:
        t = t.exp()
    drop = torch.rand(n, k, generator=g) < 0.3
    drop[:, -1] = False
    l = None
    if lists:
        l = torch.randint(0, 9, (n, k), generator=g, dtype=torch.int32)
        l[drop] = -1
        s[drop] = math.nan
    else:
        s[drop] = -math.inf
    t = t.to(tt)
    t[drop] = math.nan
    return s, t, l


def run(s, t, l, weights, tau, gr=None, off=0, pad=0, into=None):
    """distill_topk on the rows as slices of wider matrices; into: "scores" writes the gradient over them."""
    n, k = s.shape

    def wide(x, fill):
        big = torch.full((n, k + off + pad), fill, dtype=x.dtype, device=DEV)
        big[:, off:off + k] = x.to(DEV)
        return big, big[:, off:off + k]
    _, ss = wide(s, 7)
    _, ts = wide(t, 7)
    ls = None if l is None else wide(l, 5)[1]
    big, ds = wide(torch.zeros(n, k), math.nan)
    if into == "scores":
        ds = ss
    loss, ds = dsa.distill_topk(ss, ts, lists=ls, kind=int(weights), temperature=tau,
                                grad_loss=None if gr is None else gr.to(DEV), dscores=ds)
    torch.cuda.synchronize()
    rest = torch.cat([big[:, :off], big[:, off + k:]], 1)
    assert bool(torch.isnan(rest).all()), "written outside the rows"
    return loss, ds


KINDS = [(F32, False, True), (BF, False, False), (BF, True, True), (F32, True, False)]


@pytest.mark.parametrize("k", [20481, 20484, 40003])
@pytest.mark.parametrize("tt,weights,lists", KINDS)
def test_rows_of_any_length(k, tt, weights, lists):
    """Rows longer than a CTA's registers hold."""
    g = gen(k)
    for n, off, pad, tau in ((3, 0, 0, 1.0), (2, 1, 3, 0.5)):
        s, t, l = values(g, n, k, tt, weights, lists)
        gr = torch.randn(n, generator=g)
        want, bound = reference(s, t, l, weights, tau, gr)
        for into in (None, "scores"):
            got = run(s, t, l, weights, tau, gr, off, pad, into)
            for a, w, e, name in zip(got, want, bound, ("loss", "ds")):
                check(a, w, e, F32, f"{name} n={n}")


@pytest.mark.parametrize("k", [9001, 12285, 12288, 12289, 16381, 16384, 16387, 20477, 20481, 24573, 24576, 24577])
@pytest.mark.parametrize("tt,weights,lists", [(F32, False, True), (BF, True, False), (F32, True, False)])
def test_more_long_rows_than_the_gpu_takes_at_once(k, tt, weights, lists):
    """A CTA's next row is read ahead while it works on one: rows on the 16-byte boundaries, and of odd strides, whose
    end vectors are loaded on their own."""
    n = 160
    g = gen(k + 9)
    s, t, l = values(g, n, k, tt, weights, lists)
    gr = torch.randn(n, generator=g)
    want, bound = reference(s, t, l, weights, 1.0, gr)
    for off, pad, into in ((0, -k % 4, None), (1, 2 + k % 2, "scores"), (2, 0, None)):
        for a, w, e, name in zip(run(s, t, l, weights, 1.0, gr, off, pad, into), want, bound, ("loss", "ds")):
            check(a, w, e, F32, f"{name} off={off}")


@pytest.mark.parametrize("k", [100, 513, 2048, 9001, 20000, 40000])
@pytest.mark.parametrize("tt", [F32, BF])
def test_masks_of_the_lowest_value(k, tt):
    """Teacher logits, or teacher logits and scores, masked with the type's lowest value: at the row's start (past a
    long row's first batches), in all places of some threads, and everywhere but one."""
    g = gen(k + 1)
    s, t, _ = values(g, 6, k, tt, False, False)
    s.nan_to_num_(neginf=0.0)
    t.nan_to_num_(0.0)
    first = max(1, min(8192, k - 1))
    t[0, :first] = torch.finfo(tt).min
    t[1, :first] = torch.finfo(tt).min
    s[1, :first] = LOW
    t[2, :-1] = torch.finfo(tt).min
    s[2, :-1] = LOW
    t[3, 0::2] = torch.finfo(tt).min
    s[3, 0::2] = LOW
    t[4] = torch.finfo(tt).min        # all alike: uniform
    t[5, -first:] = torch.finfo(tt).min
    s[5, -first:] = LOW
    want, bound = reference(s, t, None, False, 1.0, None)
    for a, w, e, name in zip(run(s, t, None, False, 1.0), want, bound, ("loss", "ds")):
        check(a, w, e, F32, name)


@pytest.mark.parametrize("k", [100, 513, 2048, 9001, 20000, 40000])
def test_weights_over_scores_of_the_lowest_value(k):
    """Scores masked with the lowest value where the teacher's weights are zero."""
    g = gen(k + 2)
    s, t, _ = values(g, 3, k, F32, True, False)
    s.nan_to_num_(neginf=0.0)
    t.nan_to_num_(1.0)
    first = max(1, min(8192, k - 1))
    t[0, :first], s[0, :first] = 0.0, LOW
    t[1, 0::2], s[1, 0::2] = 0.0, LOW
    t[2, :-1], s[2, :-1] = 0.0, LOW
    want, bound = reference(s, t, None, True, 1.0, None)
    for a, w, e, name in zip(run(s, t, None, True, 1.0), want, bound, ("loss", "ds")):
        check(a, w, e, F32, name)


@pytest.mark.parametrize("k", [100, 513, 2048, 9001, 20000, 40000])
@pytest.mark.parametrize("tt,weights", [(F32, False), (BF, False), (F32, True), (BF, True)])
def test_scores_of_the_lowest_value_that_the_teacher_weighs(k, tt, weights):
    """The loss is large (up to 1e38) and finite: one such place, half of the places, a few of little weight."""
    g = gen(k + 3)
    s, t, _ = values(g, 4, k, tt, weights, False)
    s.nan_to_num_(neginf=0.0)
    t.nan_to_num_(0.5)
    s[0, 3] = LOW
    s[1, 0::2] = LOW
    s[2, :3] = LOW
    t[2, :3] = 2.0 ** -100 if weights else -60.0
    s[3, -40:] = LOW
    for tau in (1.0, 2.0):
        want, bound = reference(s, t, None, weights, tau, None)
        assert bool((want[0] > 100).all()) and bool((want[0] < 3e38).all())
        for a, w, e, name in zip(run(s, t, None, weights, tau), want, bound, ("loss", "ds")):
            check(a, w, e, F32, f"{name} tau={tau}")


def test_temperatures_the_arithmetic_does_not_hold_are_refused():
    x = torch.zeros(2, 8, device=DEV)
    for tau in (3e-39, 1e-30, 1e30, 3e38):
        with pytest.raises(dsa.DsaError):
            dsa.distill_topk(x, x, temperature=tau)
    for tau in (1e-18, 1e18):
        loss, ds = dsa.distill_topk(x, x, temperature=tau)
        assert not loss.any() and not ds.any()


@pytest.mark.parametrize("k", [5, 300, 2048, 9001, 20000, 40000])
@pytest.mark.parametrize("tt", [F32, BF])
def test_weights_of_any_scale(k, tt):
    """Weights whose sum lies below the normal range of fp32, at its lower end, above its range, and rows whose weights
    span it."""
    g = gen(k + 4)
    scales = [-149 if tt == F32 else -133, -140 if tt == F32 else -130, -126, -100, 0, 100, 119]
    s = torch.randn(len(scales) + 2, k, generator=g) * 2
    m = torch.randint(0, 200, s.shape, generator=g).double()
    m[:, -1] = 200.0
    t = torch.zeros(s.shape, dtype=torch.float64)
    for r, e in enumerate(scales):
        t[r] = m[r] * 2.0 ** e
    span = torch.randint(-120, 120, (k,), generator=g).double()
    t[-2] = 2.0 ** span
    t[-1] = 2.0 ** span.sort().values
    t = t.to(tt)
    assert bool(torch.isfinite(t).all()) and bool((t.double().sum(1) > 0).all())
    gr = torch.randn(s.shape[0], generator=g)
    for into in (None, "scores"):
        want, bound = reference(s, t, None, True, 1.0, gr)
        for a, w, e, name in zip(run(s, t, None, True, 1.0, gr, into=into), want, bound, ("loss", "ds")):
            check(a, w, e, F32, name)


def test_a_row_as_long_as_lengths_go():
    """k = 2^31 - 3, off the 4-place boundaries: one score row of 8.6 GB, the gradient over it.  Scores are equal and
    the teacher's weight lies on the last place: q = 1/k, loss = log k.  A thread's sum counts to 2^22 in ones
    (exact); the joining, the logarithms and the quotient round 20 times at most."""
    k = 2 ** 31 - 3
    s = torch.zeros(1, k, device=DEV)
    t = torch.zeros(1, k, dtype=BF, device=DEV)
    t[0, -1] = 3.0
    loss, ds = dsa.distill_topk(s, t, kind=dsa.TEACHER_WEIGHTS, dscores=s)
    assert abs(float(loss) - math.log(k)) <= 20 * U * math.log(k)
    assert bool((ds[0, :-1] - 1.0 / k).abs().amax() <= 20 * U / k)
    assert abs(float(ds[0, -1]) - (1.0 / k - 1.0)) <= 4 * U


def test_sizes_beyond_32_bits_are_refused():
    """The library counts a row's places in 32 bits: longer ones are refused, not cut."""
    x = torch.empty(1, 2 ** 31, device=DEV)
    y = x.view(BF)[:, :2 ** 31]
    for bad in (lambda: dsa.distill_topk(x, y), lambda: dsa.distill_topk(x.t(), y.t()), lambda: dsa.layer_norm(y)):
        with pytest.raises(ValueError):
            bad()
