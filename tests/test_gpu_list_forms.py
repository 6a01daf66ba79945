"""Scores at listed keys in every form that the sizes choose between, each case asserting the form it took: scores
gathered or picked from those of the whole prefix, dK from dense key blocks or from one row per listed pair."""
import math
import subprocess
import sys

import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
import train_ref as ref
import workloads
from test_gpu_device_checks import ROOT, checked_env
from test_gpu_train import gen, on_gpu, randn, random_lists

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def counted(call):
    """(result, launches by kind)."""
    dsa.profile_enable(True)
    dsa.profile_read()
    try:
        out = call()
        return out, {kind: n for kind, (_, n) in dsa.profile_read().items()}
    finally:
        dsa.profile_enable(False)


def backward(form, launches, lay, Q, K, W, lists, ds):
    """list_scores_backward, which has to take dK's `form`, in so many launches of its rows."""
    got, n = counted(lambda: dsa.list_scores_backward(lay, Q, K, W, lists, ds))
    if form == "rows":
        assert n["setup"] == 1 + 3 * launches and n["list_dk"] == launches and n["list_dq"] == launches, n
    else:
        assert n["setup"] == 1 and n["list_dq"] == 1, n
    return got


def scores(form, lay, Q, K, W, lists, ws=None):
    s, n = counted(lambda: dsa.list_scores(lay, Q, K, W, lists, ws=ws))
    assert ("score_tc" in n) == (form == "picked") and n["list_scores"] == 1, n
    return s


def check_backward(form, launches, b, lists, ds):
    lay, Q, K, W = on_gpu(b)
    got = backward(form, launches, lay, Q, K, W, lists.to(DEV), ds.to(DEV))
    _, want, bound = ref.list_scores(b, lists, ds)
    for a, v, e, t, name in zip(got, want, bound, (BF, BF, F32), ("dQ", "dK", "dW")):
        ref.check(a, v, e, t, name)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("H", [1, 2, 4, 8, 16, 32, 64])
def test_rows_of_dk(H, d):
    """Lists that cover little of long prefixes: places alone in their block of keys, empty lists, lists that end
    inside a tile, a sequence without queries, positions before and behind the sequence."""
    b = workloads.ragged(H * 5 + d, [40, 0, 30], [90000, 300, 60000], H=H, d=d, k=8, integer=False)
    b.q_pos[3], b.q_pos[41] = -1, 70000
    g = gen(H + d)
    lists = random_lists(g, b, 133)
    lists[3] = -1
    lists[5, 1:] = -1
    lists[6, 128:] = -1
    lists[7, 64:] = -1
    check_backward("rows", 1, b, lists, randn(g, b.n_q, 133))


@pytest.mark.parametrize("H,d", [(4, 32), (16, 128), (64, 64)])
def test_rows_of_dk_at_shared_keys(H, d):
    """Neighbouring queries that list the same keys: many rows of one key, in the order of their queries."""
    b = workloads.ragged(H + 3 * d, [300], [150000], H=H, d=d, k=8, integer=False)
    g = gen(H * d)
    shared = torch.randperm(140000, generator=g)[:60].sort().values.int()
    lists = shared.repeat(b.n_q, 1)
    lists[100:, 50:] = -1
    check_backward("rows", 1, b, lists, randn(g, b.n_q, 60))


def exact_dk(Q, K, W, lists, ds, n_k):
    """dQ, dK and dW in 64 bits for queries that all list keys of the first sequence (on the GPU)."""
    Q, K, W, ds = Q.double(), K.double(), W.double(), ds.double()
    dQ, dK, dW = torch.zeros_like(Q), torch.zeros(n_k, K.shape[1], dtype=torch.float64, device=DEV), torch.zeros_like(W)
    for j in range(lists.shape[1]):
        k = K[lists[:, j].long()]
        S = torch.einsum("thd,td->th", Q, k)
        G = torch.where(S > 0, ds[:, j:j + 1] * W, 0.0)
        dQ += G[:, :, None] * k[:, None]
        dW += ds[:, j:j + 1] * S.clamp(min=0)
        dK.index_add_(0, lists[:, j].long(), torch.einsum("th,thd->td", G, Q))
    return dQ, dK, dW


def integer_inputs(g, n, n_k, H, d, k, keys):
    Q = torch.randint(-2, 3, (n, H, d), generator=g).to(BF).to(DEV)
    K = torch.randint(-2, 3, (n_k, d), generator=g).to(BF).to(DEV)
    W = torch.tensor([0.25, 0.5, 1.0])[torch.randint(0, 3, (n, H), generator=g)].to(DEV)
    ds = torch.randint(-1, 2, (n, k), generator=g).float().to(DEV)
    start = torch.randint(0, keys - k + 1, (n, 1), generator=g, dtype=torch.int32)
    return Q, K, W, (start + torch.arange(k, dtype=torch.int32)).to(DEV), ds


def check_exact(got, want):
    dQ, dK, dW = want
    assert torch.equal(got[0], dQ.to(BF)) and torch.equal(got[1], dK.to(BF)) and torch.equal(got[2], dW.float())


@pytest.mark.parametrize("H,d,k,n_k", [(64, 32, 8, 33000), (1, 64, 32, 40000), (16, 128, 8, 33000),
                                         (64, 32, 1, 600)])
def test_rows_of_more_queries_than_a_launch_counts(H, d, k, n_k):
    """Over 32,768 queries, whose places a launch counts in 16 bits; sums carry over.  Integers: exact."""
    n = max(33000, n_k)
    lay = dsa.Layout([0, n], [0, n_k], torch.full((n,), n_k - 1), H, d, DEV)
    keys = max(7, k + 3)     # the listed ones: thousands of rows each
    Q, K, W, lists, ds = integer_inputs(gen(n + H), n, n_k, H, d, k, keys)
    got = backward("rows", 2, lay, Q, K, W, lists, ds)
    check_exact(got, exact_dk(Q, K, W, lists, ds, n_k))


def test_rows_where_partial_sums_would_take_too_much():
    """70,000 queries of one short sequence beside 940,000 keys that no query lists: nine parts of dK's dense form
    would pass 4 GiB, so its rows are summed, some thousand queries a launch."""
    n, n_k, H, d, k = 70000, 256 + 940_000, 1, 128, 200
    lay = dsa.Layout([0, n, n], [0, 256, n_k], torch.full((n,), 255), H, d, DEV)
    Q, K, W, lists, ds = integer_inputs(gen(5), n, n_k, H, d, k, 256)
    chunk = min(32 * (2 ** 30 // (6 * n_k)), n) // 148 * 148
    got = backward("rows", -(-n // chunk), lay, Q, K, W, lists, ds)
    check_exact(got, exact_dk(Q, K, W, lists, ds, n_k))


def test_dense_dk_of_more_queries_than_keys():
    """Many queries of a short prefix, every part of which they list: the dense form in parts."""
    n, n_k, H, d, k = 20000, 512, 4, 64, 200
    lay = dsa.Layout([0, n], [0, n_k], torch.full((n,), n_k - 1), H, d, DEV)
    Q, K, W, lists, ds = integer_inputs(gen(6), n, n_k, H, d, k, n_k)
    got = backward("dense", 0, lay, Q, K, W, lists, ds)
    check_exact(got, exact_dk(Q, K, W, lists, ds, n_k))


# ------------------------------------------------------------------- picked

PICKED = [(4, 64, 601), (16, 64, 1024), (64, 64, 1024), (1, 128, 600), (4, 128, 1024), (32, 128, 601), (64, 128, 602),
          (64, 128, 1000)]


@pytest.mark.parametrize("H,d,k", PICKED)
def test_picked_scores(H, d, k):
    """Lists that cover much of their prefixes, longer than some of them; empty and short ones; positions before and
    behind the sequence; row lengths of four places and odd ones."""
    b = workloads.ragged(H + d + k, [1500, 0, 700, 3], [1500, 40, 700, 0], H=H, d=d, k=8, integer=False)
    b.q_pos[5], b.q_pos[1600], b.q_pos[1499] = -1, 3000, 1499
    g = gen(k + H)
    lists = random_lists(g, b, k)
    lists[9], lists[5] = -1, -1
    lists[10, 1:] = -1
    lay, Q, K, W = on_gpu(b)
    s = scores("picked", lay, Q, K, W, lists.to(DEV))
    want, bound = ref.list_scores(b, lists)
    ref.check(s, want, bound, F32, "scores")


@pytest.mark.parametrize("H,d", [(1, 32), (8, 32)])
def test_picked_scores_of_the_smallest_dimension(H, d):
    b = workloads.ragged(H, [3000], [3000], H=H, d=d, k=8, integer=False, pos_mode="random")
    lists = random_lists(gen(H), b, 1024)
    lay, Q, K, W = on_gpu(b)
    s = scores("picked", lay, Q, K, W, lists.to(DEV))
    want, bound = ref.list_scores(b, lists)
    ref.check(s, want, bound, F32, "scores")


@pytest.mark.parametrize("k", [601, 1024])
def test_bad_lists_are_cut_and_reported_where_scores_are_picked(k):
    b = workloads.ragged(k, [1500, 700], [1500, 700], H=4, d=128, k=8, integer=False)
    g = gen(k)
    lists = random_lists(g, b, k)
    lay, Q, K, W = on_gpu(b)
    ws = torch.zeros(dsa.list_scores_workspace(lay, k), dtype=torch.uint8, device=DEV)
    scores("picked", lay, Q, K, W, lists.to(DEV), ws)
    assert dsa.device_check(ws) == 0

    def full(t, m):     # a list of m ascending keys
        lists[t] = -1
        lists[t, :m] = torch.arange(m, dtype=torch.int32)
    for case in range(7):
        kept = lists.clone()
        t = 1200 + case
        full(t, 590)
        if case == 0:
            lists[t, 300] = 1500                   # outside the sequence
        elif case == 1:
            lists[t, 128] = lists[t, 127]          # the same key twice, across a step of 128 places
        elif case == 2:
            lists[t, 400] = 5                      # not ascending
        elif case == 3:
            lists[t, 31], lists[t, 32] = -1, 40    # a key behind the padding
        elif case == 4:
            lists[t, 0] = 2 ** 31 - 1
        elif case == 5:
            lists[t, 595] = 100                    # behind the end of the list
        else:
            full(1500, 1)                          # the second sequence's first query: its prefix is one key
            lists[1500, 1] = 699                   # in the sequence, behind the prefix: not an error
        s = scores("picked", lay, Q, K, W, lists.to(DEV), ws)
        assert dsa.device_check(ws) == (0 if case == 6 else 2)
        want, bound = ref.list_scores(b, lists)
        ref.check(s, want, bound, F32, f"scores, case {case}")
        lists = kept


def test_both_forms_of_scores_agree():
    """The same queries and lists in a batch that gathers and in one that picks."""
    b = workloads.ragged(3, [1500, 700], [1500, 700], H=64, d=128, k=8, integer=True)
    lists = random_lists(gen(3), b, 1024)
    lay, Q, K, W = on_gpu(b)
    whole = scores("picked", lay, Q, K, W, lists.to(DEV))
    few = dsa.Layout([0, 20], [0, 1500], b.q_pos[1480:1500], 64, 128, DEV)
    part = scores("gathered", few, Q[1480:1500].contiguous(), K[:1500], W[1480:1500].contiguous(),
                  lists[1480:1500].contiguous().to(DEV))
    assert torch.equal(whole[1480:1500], part)


# -------------------------------------------------------------- no numbers

NOT_FINITE = [("gathered", "dense", [300, 200], [400, 300], 4, 32, 200),
              ("gathered", "dense", [300, 200], [300, 200], 64, 64, 150),
              ("gathered", "rows", [60, 30], [200, 300], 4, 32, 40),
              ("gathered", "rows", [60, 30], [9000, 6000], 64, 128, 40),
              ("picked", "dense", [1500, 700], [1500, 700], 4, 128, 601)]


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("forward,form,q_lens,k_lens,H,d,k", NOT_FINITE)
def test_a_key_that_is_not_finite(forward, form, q_lens, k_lens, H, d, k, value):
    """It makes the scores that list it what the formula makes of them (NaN, or infinite), reaches dQ and dW of the
    queries that list it, and nothing else; unlisted ones reach nothing."""
    b = workloads.ragged(H + k, q_lens, k_lens, H=H, d=d, k=8, integer=False)
    g = gen(k)
    lists, ds = random_lists(g, b, k), randn(g, b.n_q, k)
    lay, Q, K, W = on_gpu(b)
    l, e = lists.to(DEV), ds.to(DEV)
    want = dsa.list_scores(lay, Q, K, W, l)
    bwd = dsa.list_scores_backward(lay, Q, K, W, l, e)
    t = q_lens[0] - 2
    bad = int(lists[t, lists[t] >= 0][3])            # a key of the first sequence
    first = torch.zeros(b.n_q, dtype=torch.bool)
    first[:q_lens[0]] = True
    with_bad = ((lists == bad).any(1) & first).to(DEV)
    at = (l == bad) & with_bad[:, None]
    none = torch.ones(k_lens[0], dtype=torch.bool)
    none[lists[:q_lens[0]][lists[:q_lens[0]] >= 0].long().unique()] = False
    K2 = K.clone()
    K2[bad, 1] = value
    K2[:k_lens[0]][none.to(DEV)] = math.nan
    s = scores(forward, lay, Q, K2, W, l)
    assert torch.equal(s[~at], want[~at])
    dot = torch.einsum("thd,d->th", Q.double(), K2[bad].double())
    exact = torch.einsum("th,th->t", torch.relu(dot), W.double())[:, None].expand_as(s)[at]
    assert torch.equal(torch.isnan(s[at]), torch.isnan(exact))
    inf = torch.isinf(exact)
    assert torch.equal(torch.isinf(s[at]), inf) and torch.equal(s[at][inf], exact.float()[inf])
    got = backward(form, 1, lay, Q, K2, W, l, e)
    assert torch.equal(got[0][~with_bad], bwd[0][~with_bad]) and torch.equal(got[2][~with_bad], bwd[2][~with_bad])
    assert not torch.isfinite(got[0][with_bad]).all(2).any()
    reached = (dot > 0) | torch.isnan(dot)
    assert bool((~torch.isfinite(got[2]))[with_bad[:, None] & reached].all())
    others = torch.arange(K.shape[0], device=DEV) != bad
    assert torch.equal(got[1][others], bwd[1][others])


@pytest.mark.parametrize("what", ["Q", "W"])
@pytest.mark.parametrize("forward,form,q_lens,k_lens,H,d,k", NOT_FINITE)
def test_a_query_that_is_not_a_number(forward, form, q_lens, k_lens, H, d, k, what):
    """All its scores are NaN; other queries' scores, dQ and dW stay as they are, and so does dK of other sequences and,
    from rows, of the keys that it does not list."""
    b = workloads.ragged(H + k + 1, q_lens, k_lens, H=H, d=d, k=8, integer=False)
    g = gen(k + 1)
    lists, ds = random_lists(g, b, k), randn(g, b.n_q, k)
    lay, Q, K, W = on_gpu(b)
    l, e = lists.to(DEV), ds.to(DEV)
    want = dsa.list_scores(lay, Q, K, W, l)
    bwd = dsa.list_scores_backward(lay, Q, K, W, l, e)
    t = q_lens[0] - 2
    Q2, W2 = Q.clone(), W.clone()
    if what == "Q":
        Q2[t] = math.nan
    else:
        W2[t] = math.nan
    s = scores(forward, lay, Q2, K, W2, l)
    live = l[t] >= 0
    assert bool(torch.isnan(s[t][live]).all()) and bool((s[t][~live] == -math.inf).all())
    rest = torch.arange(b.n_q, device=DEV) != t
    assert torch.equal(s[rest], want[rest])
    got = backward(form, 1, lay, Q2, K, W2, l, e)
    assert torch.equal(got[0][rest], bwd[0][rest]) and torch.equal(got[2][rest], bwd[2][rest])
    listed = l[t][live].long()
    if what == "Q":
        assert bool(torch.isnan(got[2][t]).all()) and bool(torch.isnan(got[1][listed]).all())
    else:
        assert bool(torch.isnan(got[0][t]).any())
    assert torch.equal(got[1][k_lens[0]:], bwd[1][k_lens[0]:])
    if form == "rows":
        others = torch.ones(K.shape[0], dtype=torch.bool, device=DEV)
        others[listed] = False
        assert torch.equal(got[1][others], bwd[1][others])


def test_every_form_records_no_index_error():
    """These cases in the checked build: every index that the kernels compute lies inside its buffer."""
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_list_forms.py", "-q", "-x", "-m", "gpu", "-k",
                        "not every_form", "-p", "no:cacheprovider"], cwd=ROOT, env=checked_env(),
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout
