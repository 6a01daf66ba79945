"""Plain 64-bit forms of the training operators, row by row on the CPU, with elementwise bounds of what the
library's roundings may leave.

Units: a rounding to fp32 is off by at most U = 2^-24 of the value, one to bf16 by B = 2^-8.
"""
import math

import torch

U, B = 2.0 ** -24, 2.0 ** -8


def out_round(dtype):
    return B if dtype == torch.bfloat16 else U


# ------------------------------------------------------------------ layer norm

def layer_norm(x, w, b, eps):
    """(y, mean, rstd), and a bound of the error of each before y's own rounding.

    A sum of d fp32 values taken by threads of at most 32 registers, then at most 5 + 32 joining steps, is off
    by at most 72 U of the sum of magnitudes.  The mean is then off by 73 U mean|x|; a centred value by that
    plus U |x - mean|; the variance, being second order in the mean's error, by 76 U var plus the square of
    the mean's error plus twice U-order terms; rstd by half of that, relative, plus 3 U."""
    x, d = x.double(), x.shape[1]
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    wt = torch.ones(d).double() if w is None else w.double()
    bt = torch.zeros(d).double() if b is None else b.double()
    y = c * rstd * wt + bt
    e_mean = 73 * U * x.abs().mean(1, keepdim=True)
    e_c = e_mean + U * c.abs()
    e_rstd = rstd * (40 * U + (0.5 * e_mean ** 2 + e_mean * c.mean(1, keepdim=True).abs()) / (var + eps) + 3 * U)
    e_y = wt.abs() * (e_c * rstd + c.abs() * e_rstd + 2 * U * (c * rstd).abs()) + U * y.abs()
    return (y, mean[:, 0], rstd[:, 0]), (e_y, e_mean[:, 0] + U * mean[:, 0].abs(), e_rstd[:, 0])


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) from the given statistics, and bounds.  xh is off by 2 U |xh| + U |mean| rstd at most (the
    subtraction is one rounding of its result, and both operands are exact); the row sums by 73 U of their
    magnitudes plus what xh's error moves; the column sums by (rows + 40) U of theirs at most."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    n, d = x.shape
    wt = torch.ones(d).double() if w is None else w.double()
    xh = (x - mean) * rstd
    g = dy * wt
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    e_xh = 2 * U * xh.abs()
    e_g = U * g.abs()
    e_m1 = 74 * U * g.abs().mean(1, keepdim=True)
    e_m2 = 76 * U * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e_xh).mean(1, keepdim=True)
    e_dx = rstd * (e_g + e_m1 + e_xh * m2.abs() + xh.abs() * e_m2 + 4 * U * (g.abs() + m1.abs() + (xh * m2).abs()))
    k = (n + 40) * U
    return (dx, (dy * xh).sum(0), dy.sum(0)), (e_dx, k * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0),
                                               k * dy.abs().sum(0))


# ---------------------------------------------------------------- distillation

def distill(s, t, lists, weights, tau, g):
    """(loss, ds) in 64 bits, and bounds.

    exp's argument (three roundings of a value of magnitude a) is off by 3 U a, exp itself by 2 units in the last
    place (4 U), a sum of k terms by threads that hold at most k/1024 + 64 of them by (k/1024 + 64 + 42) U, the
    quotient and products by 6 U more: q and p are off by rel = (3 A + k/1024 + 116) U of themselves, A the
    largest |a|, and twice that covers numerator and denominator together."""
    s, t, n, k = s.double(), t.double(), s.shape[0], s.shape[1]
    loss, ds = torch.zeros(n).double(), torch.zeros(n, k).double()
    e_loss, e_ds = torch.zeros(n).double(), torch.zeros(n, k).double()
    for r in range(n):
        c = s[r] > -math.inf
        if lists is not None:
            c &= lists[r] >= 0
        c = torch.nonzero(c)[:, 0]
        gr = 1.0 if g is None else float(g[r])
        if c.numel() == 0:
            continue
        a, v = s[r, c] / tau, t[r, c]
        if weights:
            if not bool((v > 0).any()):
                continue
            p, logw = v / v.sum(), torch.log(v)
            logy = torch.log(v.sum())
        else:
            v = v / tau
            if bool((v == -math.inf).all()):
                continue
            p, logw = v.softmax(0), v - v.max()
            logy = torch.logsumexp(logw, 0)
        a = a - a.max()
        q, logz = a.softmax(0), torch.logsumexp(a, 0)
        on = p > 0
        cross = (p * (logw - a))[on]
        loss[r] = cross.sum() + logz - logy
        ds[r, c] = gr / tau * (q - p)
        big = max(float(a.abs().max()), float(logw[on].abs().max()))
        rel = 2 * (3 * big + k / 1024 + 116) * U
        e_ds[r, c] = abs(gr) / tau * (q + p) * rel
        e_loss[r] = rel * (p[on] * (logw[on].abs() + a[on].abs())).sum() + 2 * rel + \
            4 * U * (cross.abs().sum() + abs(float(logz)) + abs(float(logy)))
    return (loss, ds), (e_loss, e_ds)


# ------------------------------------------------------- scores at listed keys

def usable(row, pos, L):
    """Usable places of a list row, in words of the header: ascending keys up to the first -1 or bad entry, within
    the prefix."""
    out, prev = 0, -1
    for v in row.tolist():
        if v < 0 or v >= L or v <= prev or v > pos:
            break
        prev = v
        out += 1
    return out


def list_scores(b, lists, ds=None):
    """Scores [n_q, k] with their bound; with ds also ((dQ, dK, dW), bounds) before the outputs' own rounding.

    A dot product of d exact products summed in fp32 is off by at most 2 d U sum|q k| (whatever the order, and
    for adders that truncate).  A score is off by that under |w| plus (H + 2) U sum|w S|.  Backward: G = e w is
    rounded twice, to fp32 and to bf16 (U + B, relative), sums of m terms in fp32 are off by 2 m U of their
    magnitudes, and a product within its own error of zero may fall on either side, which moves a gradient by
    the whole term."""
    Q, K, W = b.Q.double(), b.K.double(), b.W.double()
    n_q, H, d = Q.shape
    k = lists.shape[1]
    qo, ko = b.q_offsets.tolist(), b.k_offsets.tolist()
    s = torch.full((n_q, k), -math.inf, dtype=torch.float64)
    e_s = torch.zeros(n_q, k).double()
    dQ, dW, dK = torch.zeros_like(Q), torch.zeros_like(W), torch.zeros_like(K)
    eQ, eW, eK = torch.zeros_like(Q), torch.zeros_like(W), torch.zeros_like(K)
    cnt = torch.zeros(K.shape[0]).double()
    for i in range(len(qo) - 1):
        for t in range(qo[i], qo[i + 1]):
            m = usable(lists[t], int(b.q_pos[t]), ko[i + 1] - ko[i])
            if m == 0:
                continue
            rows = ko[i] + lists[t, :m].long()
            Kt = K[rows]
            S = Kt @ Q[t].T                                   # [m, H]
            eS = 2 * d * U * (Kt.abs() @ Q[t].abs().T)
            R = S.clamp(min=0)
            s[t, :m] = R @ W[t]
            e_s[t, :m] = eS @ W[t].abs() + (H + 2) * U * (R @ W[t].abs())
            if ds is None:
                continue
            e = ds[t, :m].double()
            dW[t] = e @ R
            eW[t] = e.abs() @ eS + 2 * (m + 2) * U * (e.abs() @ R)
            full = e[:, None] * W[t][None]
            G = torch.where(S > 0, full, 0.0)
            unsure = torch.where(S.abs() <= eS, full.abs(), 0.0)
            eG = G.abs() * (U + B) + unsure * (1 + B)
            dQ[t] = G.T @ Kt
            eQ[t] = eG.T @ Kt.abs() + 2 * (m + 2) * U * (G.abs().T @ Kt.abs())
            dK[rows] += G @ Q[t]
            eK[rows] += eG @ Q[t].abs() + 2 * (H + 2) * U * (G.abs() @ Q[t].abs())
            cnt[rows] += 1
    eK = eK * (1 + (2 * (cnt[:, None] + 2)) * U)
    # sums over the queries that list a key: 2 U of the running magnitude each
    if ds is None:
        return s, e_s
    return (s, e_s), (dQ, dK, dW), (eQ, eK + 2 * cnt[:, None] * U * dK.abs(), eW)


def check(got, want, bound, dtype, what):
    """got (of `dtype`, on any device) within bound + its own rounding of want; infinities equal."""
    got = got.detach().cpu()
    assert got.dtype == dtype, f"{what}: {got.dtype}"
    g = got.double()
    inf = torch.isinf(want)
    assert torch.equal(g[inf], want[inf]), f"{what}: infinities differ"
    g, w, e = g[~inf], want[~inf], bound[~inf]
    assert not torch.isnan(g).any(), f"{what}: NaN"
    lim = e * (1 + out_round(dtype)) + out_round(dtype) * w.abs() + 1e-37
    off = (g - w).abs() - lim
    assert off.numel() == 0 or float(off.max()) <= 0, \
        f"{what}: off by {float((g - w).abs().flatten()[off.argmax()]):.3g}, " \
        f"allowed {float(lim.flatten()[off.argmax()]):.3g}, value {float(w.flatten()[off.argmax()]):.3g}"
