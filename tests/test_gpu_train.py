"""The training operators on the GPU against their plain 64-bit forms (train_ref), at the sizes, types, strides and
masks where they can go wrong."""
import math

import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
import train_ref as ref
import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def strided(t, pad, off=0):
    """t's rows on the GPU inside a wider matrix filled with NaN, starting `off` values in."""
    n, d = t.shape
    big = torch.full((n, d + pad + off), math.nan, dtype=t.dtype, device=DEV)
    big[:, off:off + d] = t.to(DEV)
    return big, big[:, off:off + d]


def untouched(big, d, off=0):
    rest = torch.cat([big[:, :off], big[:, off + d:]], 1)
    return bool(torch.isnan(rest).all())


# ------------------------------------------------------------------ layer norm

# every row group of the wide loads and of the single ones, their edges, and rows of one value
WIDTHS = [1, 2, 7, 8, 31, 32, 33, 64, 100, 120, 128, 129, 248, 256, 500, 512, 520, 1000, 1024, 1500, 2048, 2056, 4096,
          5001, 8192, 8200, 9999, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_layer_norm(d, xt, yt):
    g = gen(d)
    for n, pad, off, affine in ((1, 0, 0, True), (67 if d < 4096 else 5, 8, 0, True), (33 if d < 4096 else 3, 3, 1, False)):
        x = (randn(g, n, d) * 1.7 + 1.0).to(xt)
        w, b = (1 + 0.1 * randn(g, d), randn(g, d)) if affine else (None, None)
        big, xs = strided(x, pad, off)
        out, ys = strided(torch.zeros(n, d, dtype=yt), pad, off)
        y, mean, rstd = dsa.layer_norm(xs, None if w is None else w.to(DEV), None if b is None else b.to(DEV),
                                       1e-6, out=ys, want_stats=True)
        torch.cuda.synchronize()
        assert untouched(out, d, off)
        (wy, wm, wr), (ey, em, er) = ref.layer_norm(x, w, b, 1e-6)
        ref.check(y, wy, ey, yt, f"y n={n}")
        ref.check(mean, wm, em, F32, "mean")
        ref.check(rstd, wr, er, F32, "rstd")

        dy = (randn(g, n, d) * 0.1).to(yt)
        dbig, dys = strided(dy, pad, off)
        obig, dxs = strided(torch.zeros(n, d, dtype=xt), pad, off)
        dx, dw, db = dsa.layer_norm_backward(dys, xs, None if w is None else w.to(DEV), mean, rstd, dx=dxs)
        torch.cuda.synchronize()
        assert untouched(obig, d, off)
        want, bound = ref.layer_norm_backward(dy, x, w, mean.cpu(), rstd.cpu())
        for got, a, e, t, name in zip((dx, dw, db), want, bound, (xt, F32, F32), ("dx", "dw", "db")):
            ref.check(got, a, e, t, f"{name} n={n}")


def test_layer_norm_constant_rows_and_large_offset():
    x = torch.cat([torch.full((3, 128), 5.0), torch.zeros(2, 128), 1e4 + randn(gen(1), 4, 128)])
    y, mean, rstd = dsa.layer_norm(x.to(DEV), eps=1e-6, want_stats=True)
    (wy, wm, wr), (ey, em, er) = ref.layer_norm(x, None, None, 1e-6)
    ref.check(y, wy, ey, F32, "y")
    ref.check(rstd, wr, er, F32, "rstd")
    assert torch.equal(y[:5].cpu(), torch.zeros(5, 128))


def test_layer_norm_many_rows_and_same_bits():
    """More rows than one sweep of the grid; the same call twice gives the same bits."""
    n, d = 20011, 128
    g = gen(3)
    x, dy, w = randn(g, n, d).to(BF), (randn(g, n, d) * 1e-2).to(BF), 1 + 0.1 * randn(g, d)
    xs, dys, ws = x.to(DEV), dy.to(DEV), w.to(DEV)
    y, mean, rstd = dsa.layer_norm(xs, ws, want_stats=True)
    (wy, _, _), (ey, _, _) = ref.layer_norm(x, w, None, 1e-6)
    ref.check(y, wy, ey, BF, "y")
    a = dsa.layer_norm_backward(dys, xs, ws, mean, rstd)
    b = dsa.layer_norm_backward(dys, xs, ws, mean, rstd)
    want, bound = ref.layer_norm_backward(dy, x, w, mean.cpu(), rstd.cpu())
    for i, name in enumerate(("dx", "dw", "db")):
        assert torch.equal(a[i], b[i]), name
        ref.check(a[i], want[i], bound[i], (BF, F32, F32)[i], name)


def test_layer_norm_no_rows_and_in_place():
    x = torch.empty(0, 16, device=DEV)
    y, mean, rstd = dsa.layer_norm(x, want_stats=True)
    dx, dw, db = dsa.layer_norm_backward(x, x, None, mean, rstd)
    assert y.shape == (0, 16) and dx.shape == (0, 16)
    assert torch.equal(dw.cpu(), torch.zeros(16)) and torch.equal(db.cpu(), torch.zeros(16))
    x = randn(gen(5), 70, 200).to(DEV)
    want = dsa.layer_norm(x)
    assert torch.equal(dsa.layer_norm(x, out=x), want)


def test_layer_norm_gradient_is_the_difference_quotient():
    """The gradient along a direction against central differences of the 64-bit forward form (h = 1e-5: the
    quotient's own error is of the order h^2, and 1e-16 / h)."""
    g = gen(9)
    x, w, b, c, u = (randn(g, 6, 40), 1 + 0.1 * randn(g, 40), randn(g, 40), randn(g, 6, 40), randn(g, 6, 40))
    _, mean, rstd = dsa.layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), 1e-6, want_stats=True)
    dx, dw, db = dsa.layer_norm_backward(c.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)

    def f(x, w):
        x = x.double()
        m = x.mean(1, keepdim=True)
        return float((((x - m) * ((x - m).square().mean(1, keepdim=True) + 1e-6).rsqrt() * w + b) * c).sum())
    h = 1e-5
    along = (f(x.double() + h * u, w.double()) - f(x.double() - h * u, w.double())) / (2 * h)
    assert abs(float((dx.cpu().double() * u).sum()) - along) < 1e-4 * float((dx.cpu() * u).abs().sum())
    v = randn(g, 40)
    along = (f(x.double(), w + h * v.double()) - f(x.double(), w - h * v.double())) / (2 * h)
    assert abs(float((dw.cpu().double() * v).sum()) - along) < 1e-4 * float((dw.cpu() * v).abs().sum())


# ---------------------------------------------------------------- distillation

def distill_case(g, n, k, tt, weights, lists):
    s, t = randn(g, n, k) * 2, randn(g, n, k) * 2
    if weights:
        t = torch.exp(t)
        t[torch.rand(n, k, generator=g) < 0.2] = 0.0
    else:
        t[torch.rand(n, k, generator=g) < 0.2] = -math.inf
        if k > 3:
            t[0, :2] = torch.finfo(tt).min
    l = torch.randint(0, 9, (n, k), generator=g, dtype=torch.int32) if lists else None
    drop = torch.rand(n, k, generator=g) < 0.3
    if n > 2:
        drop[n // 2] = True      # a row without a counted place
        t[n - 1] = 0.0 if weights else -math.inf     # one without teacher weight
    t = t.to(tt)
    if lists:
        l[drop] = -1
        s[drop] = math.nan       # whatever stands in a place that does not count
        t[drop] = math.nan
        if n > 4:
            s[3, ::2], l[3, ::2] = -math.inf, 1      # a score of -inf does not count either
    else:
        s[drop] = -math.inf
        t[drop] = math.nan
    return s, t, l


@pytest.mark.parametrize("k", [1, 2, 5, 32, 64, 127, 128, 129, 512, 516, 1000, 1024, 2048, 2051, 4096, 8192, 8196,
                               16384, 16385, 20011])
@pytest.mark.parametrize("tt,weights,lists", [(F32, False, True), (BF, False, False), (BF, True, True),
                                              (F32, True, False)])
def test_distill(k, tt, weights, lists):
    g = gen(k)
    for n, pad, off, tau in ((7, 0, 0, 1.0), (9 if k < 4096 else 3, 4, 0, 0.5), (5, 3, 1, 2.0)):
        s, t, l = distill_case(g, n, k, tt, weights, lists)
        gr = None if pad == 4 else randn(g, n)
        sb, ss = strided(s, pad, off)
        tb, ts = strided(t, pad, off)
        ls = None
        if l is not None:
            lb = torch.full((n, k + pad + off), 5, dtype=torch.int32, device=DEV)
            lb[:, off:off + k] = l.to(DEV)
            ls = lb[:, off:off + k]
        ob, ds = strided(torch.zeros(n, k), pad, off)
        loss, ds = dsa.distill_topk(ss, ts, lists=ls,
                                    kind=dsa.TEACHER_WEIGHTS if weights else dsa.TEACHER_LOGITS, temperature=tau,
                                    grad_loss=None if gr is None else gr.to(DEV), dscores=ds)
        torch.cuda.synchronize()
        assert untouched(ob, k, off)
        (wl, wd), (el, ed) = ref.distill(s, t, l, weights, tau, gr)
        ref.check(loss, wl, el, F32, f"loss n={n}")
        ref.check(ds, wd, ed, F32, f"ds n={n}")


@pytest.mark.parametrize("n,k", [(2500, 516), (2380, 1024), (4750, 613), (1250, 1028), (1190, 2048), (600, 2900),
                                 (299, 6000), (300, 8192)])
@pytest.mark.parametrize("tt,weights,lists", [(F32, False, True), (BF, False, False), (BF, True, True)])
def test_distill_many_rows(n, k, tt, weights, lists):
    """More rows than fit the GPU at once: the CTAs take several each, and read ahead where rows are aligned;
    the gradient over its scores gives the same."""
    g = gen(n + k)
    s, t, l = distill_case(g, n, k, tt, weights, lists)
    gr = randn(g, n)
    kind = dsa.TEACHER_WEIGHTS if weights else dsa.TEACHER_LOGITS
    sd, td, ld = s.to(DEV), t.to(DEV), None if l is None else l.to(DEV)
    loss, ds = dsa.distill_topk(sd, td, lists=ld, kind=kind, temperature=0.5, grad_loss=gr.to(DEV))
    (wl, wd), (el, ed) = ref.distill(s, t, l, weights, 0.5, gr)
    ref.check(loss, wl, el, F32, "loss")
    ref.check(ds, wd, ed, F32, "ds")
    loss2, ds2 = dsa.distill_topk(sd, td, lists=ld, kind=kind, temperature=0.5, grad_loss=gr.to(DEV), dscores=sd)
    assert ds2.data_ptr() == sd.data_ptr() and torch.equal(loss, loss2) and torch.equal(ds, ds2)


def test_distill_in_place_alone_and_same_bits():
    g = gen(11)
    for k in (96, 2048, 20000):
        s, t = (randn(g, 37, k) * 2).to(DEV), (randn(g, 37, k) * 2).to(DEV)
        loss, ds = dsa.distill_topk(s, t)
        again, ds2 = dsa.distill_topk(s, t)
        assert torch.equal(loss, again) and torch.equal(ds, ds2)
        own = s.clone()
        loss3, ds3 = dsa.distill_topk(own, t, dscores=own)
        assert ds3.data_ptr() == own.data_ptr() and torch.equal(loss, loss3) and torch.equal(ds, ds3)


def test_distill_extreme_values():
    """One score far above the rest, all equal scores, all-lowest teacher logits (uniform), a NaN score that
    stays in its own row."""
    s = torch.zeros(5, 300)
    t = torch.zeros(5, 300)
    s[0, 7] = 3e4
    t[1] = torch.finfo(F32).min
    t[2, 9] = 1e4
    s[3, 5] = math.nan
    loss, ds = dsa.distill_topk(s.to(DEV), t.to(DEV))
    ok = [0, 1, 2, 4]
    (wl, wd), (el, ed) = ref.distill(s[ok], t[ok], None, False, 1.0, None)
    ref.check(loss[ok], wl, el, F32, "loss")
    ref.check(ds[ok], wd, ed, F32, "ds")
    assert math.isnan(float(loss[3]))


def test_distill_gradient_is_the_difference_quotient():
    g = gen(13)
    s, t, u = randn(g, 3, 50), randn(g, 3, 50), randn(g, 3, 50)
    for weights in (False, True):
        tt = t.exp() if weights else t
        _, ds = dsa.distill_topk(s.to(DEV), tt.to(DEV), kind=int(weights), temperature=0.7)
        h = 1e-5
        f = lambda x: ref.distill(x, tt, None, weights, 0.7, None)[0][0].sum()   # noqa: E731
        along = float(f(s.double() + h * u) - f(s.double() - h * u)) / (2 * h)
        assert abs(float((ds.cpu().double() * u).sum()) - along) < 1e-4 * float((ds.cpu() * u).abs().sum())


# ------------------------------------------------------- scores at listed keys

def random_lists(g, b, k, fill=1.0):
    """Random ascending subsets of each query's prefix, some rows short, some empty."""
    qo, ko = b.q_offsets.tolist(), b.k_offsets.tolist()
    out = torch.full((b.n_q, k), -1, dtype=torch.int32)
    for i in range(len(qo) - 1):
        for t in range(qo[i], qo[i + 1]):
            n = min(int(b.q_pos[t]) + 1, ko[i + 1] - ko[i])
            m = min(k, n)
            if t % 7 == 3:
                m = int(torch.randint(0, m + 1, (1,), generator=g)) if m > 0 else 0
            if m > 0:
                out[t, :m] = torch.randperm(n, generator=g)[:m].sort().values.int()
    return out


def on_gpu(b):
    return dsa.Layout.from_batch(b, DEV), b.Q.to(DEV), b.K.to(DEV), b.W.to(DEV)


def check_lists(b, lists, ds, lay=None):
    lay, Q, K, W = on_gpu(b)
    l, e = lists.to(DEV), ds.to(DEV)
    s = dsa.list_scores(lay, Q, K, W, l)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, l, e)
    torch.cuda.synchronize()
    (ws, es), want, bound = ref.list_scores(b, lists, ds)
    ref.check(s, ws, es, F32, "scores")
    for got, a, d, t, name in zip((dQ, dK, dW), want, bound, (BF, BF, F32), ("dQ", "dK", "dW")):
        ref.check(got, a, d, t, name)
    return s, dQ, dK, dW


SHAPES = [(1, 32), (2, 64), (4, 32), (8, 128), (16, 64), (16, 128), (32, 32), (32, 128), (64, 32), (64, 64), (64, 128)]


@pytest.mark.parametrize("H,d", SHAPES)
def test_list_scores_shapes(H, d):
    """Every head count and dimension, ragged sequences (one without queries, one without keys), positions beyond
    the sequence and before it, lists longer than the prefix."""
    b = workloads.ragged(H + d, [70, 0, 3, 40], [70, 30, 0, 300], H=H, d=d, k=50, integer=False, pos_mode="random")
    b.q_pos[5], b.q_pos[6] = -1, 1000
    g = gen(H * d)
    for k in (1, 50, 130):
        lists = random_lists(g, b, k)
        check_lists(b, lists, randn(g, b.n_q, k))


@pytest.mark.parametrize("k", [127, 128, 129, 255, 1000])
def test_list_scores_tile_edges(k):
    """Lists that end at, before and behind a tile of 128, over key tiles that end inside the cache."""
    b = workloads.ragged(k, [9, 130], [1100, 385], H=64, d=128, k=k, integer=False, pos_mode="random")
    g = gen(k)
    check_lists(b, random_lists(g, b, k), randn(g, b.n_q, k) * 1e-3)


@pytest.mark.parametrize("H,d", [(64, 128), (64, 64), (32, 32), (16, 128), (8, 64), (1, 32)])
def test_list_scores_sparse_lists(H, d):
    """Lists that cover little of their prefix (a few places per block of 256 keys, dK then comes from one row per
    listed pair), empty blocks between them, sequences that begin inside a block of key rows."""
    b = workloads.ragged(H * 3 + d, [37, 0, 90, 3], [5000, 300, 7001, 20], H=H, d=d, k=8, integer=False)
    g = gen(H + d)
    for k in (4, 133):
        check_lists(b, random_lists(g, b, k), randn(g, b.n_q, k))


def test_list_scores_sparse_lists_in_several_launches():
    """More listed pairs than one launch's rows hold (1 GiB): the sums carry over."""
    b = workloads.ragged(5, [1400], [40000], H=64, d=128, k=1500, integer=False)
    g = gen(6)
    check_lists(b, random_lists(g, b, 1500), randn(g, b.n_q, 1500))


def test_list_scores_integers_are_exact():
    """Integer keys and queries, power-of-two weights and gradients: every sum is exact in fp32, zeros of the
    products included, so results are the 64-bit ones rounded once."""
    b = workloads.tiny_integer(seed=3, T=200, H=16, d=64, k=64)
    g = gen(4)
    lists = random_lists(g, b, 64)
    ds = torch.randint(-2, 3, (200, 64), generator=g).float() / 4
    lay, Q, K, W = on_gpu(b)
    (ws, _), (wQ, wK, wW), _ = ref.list_scores(b, lists, ds)
    s = dsa.list_scores(lay, Q, K, W, lists.to(DEV))
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, lists.to(DEV), ds.to(DEV))
    assert torch.equal(s.cpu(), ws.float())
    assert torch.equal(dQ.cpu(), wQ.bfloat16()) and torch.equal(dK.cpu(), wK.bfloat16())
    assert torch.equal(dW.cpu(), wW.float())


def test_list_scores_at_the_selected_keys_are_the_selections_scores():
    b = workloads.ragged(8, [100, 60], [100, 900], H=64, d=128, k=64, integer=False)
    lay, Q, K, W = on_gpu(b)
    idx, top = dsa.index_topk(lay, Q, K, W, 64, want_scores=True)
    s = dsa.list_scores(lay, Q, K, W, idx)
    (_, es) = ref.list_scores(b, idx.cpu())
    live = idx.cpu() >= 0
    assert bool((s.cpu()[~live] == -math.inf).all())
    assert bool(((s.cpu() - top.cpu()).double().abs()[live] <= 2 * es[live] + 1e-30).all())


def test_places_that_do_not_count_are_not_read():
    """NaN in dscores of empty and far places, in keys that no list names and in queries with empty lists."""
    b = workloads.ragged(21, [40, 30], [200, 333], H=64, d=128, k=40, integer=False, pos_mode="random")
    g = gen(22)
    lists = random_lists(g, b, 40)
    lists[4] = -1
    ds = randn(g, b.n_q, 40)
    (ws, es), want, bound = ref.list_scores(b, lists, ds)
    used = torch.zeros(b.K.shape[0], dtype=torch.bool)
    for t in range(b.n_q):
        base = 0 if t < 40 else 200
        used[base + lists[t][lists[t] >= 0].long()] = True
    b.K[~used] = math.nan
    b.Q[4] = math.nan
    b.W[4] = math.nan
    ds[lists < 0] = math.nan
    lay, Q, K, W = on_gpu(b)
    s = dsa.list_scores(lay, Q, K, W, lists.to(DEV))
    got = dsa.list_scores_backward(lay, Q, K, W, lists.to(DEV), ds.to(DEV))
    ref.check(s, ws, es, F32, "scores")
    for a, w, e, t, name in zip(got, want, bound, (BF, BF, F32), ("dQ", "dK", "dW")):
        ref.check(a, w, e, t, name)


def test_bad_lists_are_cut_and_reported():
    b = workloads.ragged(31, [20], [500], H=16, d=64, k=16, integer=False)
    g = gen(32)
    lists = random_lists(g, b, 16)
    lay, Q, K, W = on_gpu(b)
    ws = torch.zeros(dsa.list_scores_backward_workspace(lay, 16), dtype=torch.uint8, device=DEV)
    dsa.list_scores(lay, Q, K, W, lists.to(DEV), ws=ws)
    assert dsa.device_check(ws) == 0
    lists[2, 5] = 500            # outside the sequence
    lists[3, 6] = lists[3, 5]    # the same key twice
    lists[5, 4], lists[5, 5] = -1, 17      # a key behind the padding
    ds = randn(g, 20, 16)
    (wS, eS), want, bound = ref.list_scores(b, lists, ds)
    s = dsa.list_scores(lay, Q, K, W, lists.to(DEV), ws=ws)
    assert dsa.device_check(ws) == 2
    ref.check(s, wS, eS, F32, "scores")
    got = dsa.list_scores_backward(lay, Q, K, W, lists.to(DEV), ds.to(DEV), ws=ws)
    assert dsa.device_check(ws) == 2
    for a, w, e, t, name in zip(got, want, bound, (BF, BF, F32), ("dQ", "dK", "dW")):
        ref.check(a, w, e, t, name)


def test_list_scores_gradients_apart_and_same_bits():
    """Each gradient alone equals the joint call's; the same call twice gives the same bits."""
    b = workloads.ragged(41, [150, 80], [150, 700], H=64, d=128, k=96, integer=False)
    g = gen(42)
    lists, ds = random_lists(g, b, 96).to(DEV), randn(g, b.n_q, 96).to(DEV)
    lay, Q, K, W = on_gpu(b)
    a = dsa.list_scores_backward(lay, Q, K, W, lists, ds)
    again = dsa.list_scores_backward(lay, Q, K, W, lists, ds)
    for i in range(3):
        assert torch.equal(a[i], again[i])
    import ctypes
    ws = torch.empty(dsa.list_scores_backward_workspace(lay, 96), dtype=torch.uint8, device=DEV)
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())   # noqa: E731
    for i in range(3):
        out = [None, None, None]
        out[i] = torch.full_like(a[i], 7)
        st = dsa.library().dsa_list_scores_backward(
            lay.ref(), p(Q), p(K), p(W), 96, p(lists), p(ds), p(out[0]), p(out[1]), p(out[2]), p(ws),
            ctypes.c_size_t(ws.numel()), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert st == 0 and torch.equal(out[i], a[i])


def test_list_scores_long_lists_and_few_queries():
    """The longest lists (16,384 places) of a few queries over a long cache."""
    b = workloads.ragged(51, [2, 1], [17000, 5000], H=8, d=32, k=16384, integer=False)
    g = gen(52)
    check_lists(b, random_lists(g, b, 16384), randn(g, 3, 16384))


@pytest.mark.parametrize("H,d,k", [(64, 128, 1000), (32, 64, 257), (16, 32, 4001), (4, 128, 129), (64, 64, 128)])
def test_list_scores_few_queries_share_the_gpu(H, d, k):
    """A few queries, whose tiles several CTAs take in turn: lists that end in any of them, empty ones, one place."""
    b = workloads.ragged(H + k, [3, 1, 2], [5000, 40, 900], H=H, d=d, k=k, integer=False)
    g = gen(k)
    lists = random_lists(g, b, k)
    lists[1] = -1
    lists[2, 1:] = -1
    check_lists(b, lists, randn(g, b.n_q, k))


def test_list_scores_nothing_to_do():
    b = workloads.ragged(61, [0, 0], [30, 5], H=4, d=32, k=8, integer=False)
    lay, Q, K, W = on_gpu(b)
    none = torch.empty(0, 8, dtype=torch.int32, device=DEV)
    s = dsa.list_scores(lay, Q, K, W, none)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, none, none.float())
    assert s.shape == (0, 8) and dQ.shape == (0, 4, 32) and dW.shape == (0, 4)
    assert torch.equal(dK.cpu(), torch.zeros(35, 32, dtype=BF))
    b = workloads.ragged(62, [5], [0], H=4, d=32, k=8, integer=False)
    lay, Q, K, W = on_gpu(b)
    none = torch.full((5, 8), -1, dtype=torch.int32, device=DEV)
    s = dsa.list_scores(lay, Q, K, W, none)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, none, none.float())
    assert bool((s == -math.inf).all()) and not dQ.any() and not dW.any() and dK.shape == (0, 32)


def test_list_scores_gradient_is_the_difference_quotient():
    """Along a direction of W (the scores are linear in it) and of Q and K, against central differences of the
    64-bit forward form.  h = 1e-6 moves products by less than the distance of nearly all of them from zero;
    2e-2 of the magnitudes covers the bf16 rounding of G and of the gradient (2 B = 2^-7)."""
    b = workloads.ragged(71, [30], [64], H=16, d=64, k=20, integer=False)
    g = gen(72)
    lists = random_lists(g, b, 20)
    c = randn(g, 30, 20)
    lay, Q, K, W = on_gpu(b)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, lists.to(DEV), c.to(DEV))
    live = lists >= 0

    def f(**kw):
        import types
        x = types.SimpleNamespace(**{**vars(b), **kw})
        s = ref.list_scores(x, lists)[0]
        return float((s * c)[live].sum())
    h = 1e-6
    for name, got, tol in (("Q", dQ, 2e-2), ("K", dK, 2e-2), ("W", dW, 1e-5)):
        v = getattr(b, name).double()
        u = randn(g, *v.shape).double()
        along = (f(**{name: v + h * u}) - f(**{name: v - h * u})) / (2 * h)
        have = got.cpu().double() * u
        assert abs(float(have.sum()) - along) <= tol * float(have.abs().sum()), name


# ------------------------------------------------------------ together, as used

def step(lay, x, w, bias, Q, W, teacher, k):
    """One training step of an indexer: keys' norm, selection, scores, loss, gradients."""
    K, mean, rstd = dsa.layer_norm(x, w, bias, want_stats=True)
    idx = dsa.index_topk(lay, Q, K, W, k)
    s = dsa.list_scores(lay, Q, K, W, idx)
    g = torch.full((s.shape[0],), 1.0 / s.shape[0], device=s.device)
    loss, ds = dsa.distill_topk(s, teacher, lists=idx, kind=dsa.TEACHER_WEIGHTS, grad_loss=g)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, idx, ds)
    dx, dw, db = dsa.layer_norm_backward(dK, x, w, mean, rstd)
    return idx, loss, dQ, dK, dW, dx, dw, db


def step_inputs(seed, H=64, d=128, k=48):
    b = workloads.ragged(seed, [90, 40], [90, 300], H=H, d=d, k=k, integer=False)
    g = gen(seed)
    x = randn(g, b.K.shape[0], d + 64).to(BF).to(DEV)[:, :d]      # a slice of a wider projection
    w, bias = (1 + 0.1 * randn(g, d)).to(DEV), (0.1 * randn(g, d)).to(DEV)
    teacher = torch.rand(b.n_q, k, generator=g).to(BF).to(DEV)
    return b, dsa.Layout.from_batch(b, DEV), x, w, bias, b.Q.to(DEV), b.W.to(DEV), teacher


def test_training_step():
    b, lay, x, w, bias, Q, W, teacher = step_inputs(81)
    idx, loss, dQ, dK, dW, dx, dw, db = step(lay, x, w, bias, Q, W, teacher, 48)
    torch.cuda.synchronize()
    (ky, mean, rstd), _ = ref.layer_norm(x.cpu(), w.cpu(), bias.cpu(), 1e-6)
    K = dsa.layer_norm(x, w, bias)
    ref.check(K, ky, torch.zeros_like(ky) + 1e-4, BF, "K")
    b.K = K.cpu()
    lists = idx.cpu()
    s = dsa.list_scores(lay, Q, K, W, idx).cpu()
    (ws, es) = ref.list_scores(b, lists)
    ref.check(s, ws, es, F32, "scores")
    n = b.n_q
    g = torch.full((n,), 1.0 / n)
    (wl, wd), (el, ed) = ref.distill(s, teacher.cpu(), lists, True, 1.0, g)
    ref.check(loss, wl, el, F32, "loss")
    _, ds = dsa.distill_topk(s.to(DEV), teacher, lists=idx, kind=dsa.TEACHER_WEIGHTS, grad_loss=g.to(DEV))
    ref.check(ds, wd, ed, F32, "ds")
    _, want, bound = ref.list_scores(b, lists, ds.cpu())
    for a, v, e, t, name in zip((dQ, dK, dW), want, bound, (BF, BF, F32), ("dQ", "dK", "dW")):
        ref.check(a, v, e, t, name)
    _, m32, r32 = dsa.layer_norm(x, w, bias, want_stats=True)
    want, bound = ref.layer_norm_backward(dK.cpu(), x.cpu(), w.cpu(), m32.cpu(), r32.cpu())
    for a, v, e, t, name in zip((dx, dw, db), want, bound, (BF, F32, F32), ("dx", "dw", "db")):
        ref.check(a, v, e, t, name)


def test_training_step_on_other_streams_and_captured():
    """Two steps at once on two streams, and a captured step replayed on new inputs, give the eager step's bits."""
    one, two = step_inputs(83), step_inputs(84)
    want = [step(*a[1:], 48) for a in (one, two)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    got = []
    for st, a in zip(streams, (one, two)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(step(*a[1:], 48))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        for u, v in zip(x, y):
            assert torch.equal(u, v)
    _, lay, x, w, bias, Q, W, teacher = two
    held = [t.clone() for t in (x, w, bias, Q, W, teacher)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(lay, *held, 48)
    for scale in (1.0, 0.5):
        held[3].copy_(Q * scale)
        graph.replay()
        torch.cuda.synchronize()
        exp = step(lay, x, w, bias, Q * scale, W, teacher, 48)
        for u, v in zip(out, exp):
            assert torch.equal(u, v)


def test_an_explicit_stream_is_used():
    """The call goes to the stream it is given, not to the current one."""
    st = torch.cuda.Stream(DEV)
    x = randn(gen(91), 64, 128).to(DEV)
    want = dsa.layer_norm(x)
    torch.cuda.synchronize()
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        dsa.layer_norm(x, out=y, stream=st)
    assert not y.any()           # captured on st, not run
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_memory_made_for_another_stream_is_not_handed_out_early():
    """A call on a stream of its own makes its workspace and outputs on the current stream; work queued there
    afterwards, which the allocator serves from freed memory, must not reach them while the call still runs."""
    b = workloads.ragged(96, [300, 200], [300, 900], H=64, d=128, k=64, integer=False)
    lay, Q, K, W = on_gpu(b)
    g = gen(96)
    lists, ds = random_lists(g, b, 64).to(DEV), randn(g, b.n_q, 64).to(DEV)
    want = dsa.list_scores_backward(lay, Q, K, W, lists, ds)
    torch.cuda.synchronize()
    st = torch.cuda.Stream(DEV)
    size = dsa.list_scores_backward_workspace(lay, 64)
    busy = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(st):
            for _ in range(4):
                busy @ busy              # keeps the stream behind the host
        got = dsa.list_scores_backward(lay, Q, K, W, lists, ds, stream=st)
        junk = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for u, v in zip(want, got):
            assert torch.equal(u, v)
        del junk


def test_binding_refuses_what_the_library_cannot_read():
    x = torch.zeros(8, 16, device=DEV)
    for bad in (lambda: dsa.layer_norm(x.half()), lambda: dsa.layer_norm(x.t()), lambda: dsa.layer_norm(x[0]),
                lambda: dsa.layer_norm(x, weight=torch.ones(8, device=DEV)),
                lambda: dsa.layer_norm(x, out=torch.empty(8, 15, device=DEV)),
                lambda: dsa.layer_norm(x, weight=torch.ones(16)),
                lambda: dsa.layer_norm(x[:1].expand(8, 16)),
                lambda: dsa.distill_topk(x, x[:, :8]), lambda: dsa.distill_topk(x.bfloat16(), x),
                lambda: dsa.distill_topk(x, x, lists=torch.zeros(8, 16, dtype=torch.int64, device=DEV)),
                lambda: dsa.distill_topk(x, x, grad_loss=torch.ones(7, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    b = workloads.ragged(95, [8], [16], H=4, d=32, k=4, integer=False)
    lay, Q, K, W = on_gpu(b)
    idx = torch.zeros(8, 4, dtype=torch.int32, device=DEV)
    for bad in (lambda: dsa.list_scores(lay, Q[:7], K, W, idx), lambda: dsa.list_scores(lay, Q, K.float(), W, idx),
                lambda: dsa.list_scores(lay, Q, K, W, idx.long()), lambda: dsa.list_scores(lay, Q, K, W, idx[:7]),
                lambda: dsa.list_scores(lay, Q, K, W.bfloat16(), idx),
                lambda: dsa.list_scores_backward(lay, Q, K, W, idx, idx)):
        with pytest.raises(ValueError):
            bad()


def test_many_queries_of_short_lists():
    """More queries than one launch of the rows takes (16-bit counts: 32,768), every one listing the same key: the
    key's gradient is the sum over all of them, and the sums carry over."""
    n = 33000
    g = gen(97)
    b = workloads.ragged(97, [n], [600], H=4, d=32, k=1, integer=True)
    b.q_pos[:] = 599
    lists = torch.full((n, 1), 5, dtype=torch.int32)
    ds = torch.randint(-1, 2, (n, 1), generator=g).float()
    lay, Q, K, W = on_gpu(b)
    dQ, dK, dW = dsa.list_scores_backward(lay, Q, K, W, lists.to(DEV), ds.to(DEV))
    S = torch.einsum("thd,d->th", b.Q.double(), b.K[5].double())
    G = torch.where(S > 0, ds.double() * b.W.double(), 0.0)
    want = torch.zeros(600, 32).double()
    want[5] = torch.einsum("th,thd->d", G, b.Q.double())          # integers and quarters: exact in fp32
    assert torch.equal(dK.cpu(), want.bfloat16())
    assert torch.equal(dQ.cpu(), (G[:, :, None] * b.K[5].double()).bfloat16())
    assert torch.equal(dW.cpu(), (ds.double() * S.clamp(min=0)).float())
