"""The training operators of the indexer as a user's program calls them, case by case, next to their plain forms.

Five calls that one training step of an indexer makes: the keys' layer norm and its backward pass, the indexer's
scores at listed keys and their backward pass, and the distillation loss of those scores against a teacher's top
logits or weights, with its gradient.  The plain forms below are elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False   # True: run() calls the library

EPS = 1e-6


def listed():
    return [
        # the keys of one decode step: 16 sequences, 2 new tokens each (latency)
        dict(name="norm decode 32x128", op="norm", n=32, d=128, pad=0, xt="bf16", yt="bf16"),
        # the keys of a 32K prefill, a column slice of a wider fused projection
        dict(name="norm prefill 32Kx128", op="norm", n=32768, d=128, pad=64, xt="bf16", yt="bf16"),
        # the backward pass over the keys of a training batch of 128K tokens
        dict(name="norm bwd 128Kx128", op="norm_bwd", n=131072, d=128, pad=64, xt="bf16", yt="bf16"),
        # wide rows of an odd width and count, activations kept in 32 bits
        dict(name="norm bwd 4099x5001 fp32", op="norm_bwd", n=4099, d=5001, pad=0, xt="fp32", yt="fp32"),
        # a small step: 512 queries, 64 listed keys each
        dict(name="distill 512x64", op="distill", n=512, k=64, lists=True, kind="logits", tt="fp32", tau=1.0),
        # 8K tokens of sparse training: the attention's weights on the 2048 selected keys, in 16 bits
        dict(name="distill 8Kx2048 weights", op="distill", n=8192, k=2048, lists=True, kind="weights", tt="bf16",
             tau=1.0),
        # whole score rows (dense warm-up): every key of the prefix, odd sizes, more than one block of columns
        dict(name="distill dense 1021x20011", op="distill", n=1021, k=20011, lists=False, kind="logits", tt="fp32",
             tau=2.0),
        # a decode step's 32 queries over 16 caches of 32K keys, scored at another layer's lists
        dict(name="scores decode 16x32K", op="scores", B=16, nq=2, L=32768, H=64, d=128, k=2048, ragged=False),
        # a packed training batch: 8K tokens in sequences of uneven length
        dict(name="scores packed 8K", op="scores", B=3, nq=2731, L=2731, H=64, d=128, k=1024, ragged=True),
        # the smallest training step of the tests
        dict(name="scores bwd 512 H4 d32", op="scores_bwd", B=1, nq=512, L=512, H=4, d=32, k=64, ragged=False),
        # the same packed batch's backward pass
        dict(name="scores bwd packed 8K", op="scores_bwd", B=3, nq=2731, L=2731, H=64, d=128, k=1024, ragged=True),
        # a chunk of 4K queries at the end of a 32K context
        dict(name="scores bwd 4K of 32K", op="scores_bwd", B=1, nq=4096, L=32768, H=64, d=128, k=2048, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "distill", "scores", "scores_bwd"])
    if op in ("norm", "norm_bwd"):
        d = rng.choice([32, 64, 128, 128, _log_int(rng, 8, 8191)])
        n = _log_int(rng, 1, max(2, min(131072, 20_000_000 // d)))
        return dict(op=op, n=n, d=d, pad=rng.choice([0, 0, 1, 8, 64]), xt=rng.choice(["bf16", "fp32"]),
                    yt=rng.choice(["bf16", "fp32"]))
    if op == "distill":
        k = _log_int(rng, 1, 20011)
        n = _log_int(rng, 1, max(2, min(32768, 20_000_000 // k)))
        return dict(op=op, n=n, k=k, lists=rng.random() < 0.7, kind=rng.choice(["logits", "weights"]),
                    tt=rng.choice(["fp32", "bf16"]), tau=rng.choice([1.0, 1.0, 0.5, 2.0]))
    H, d = rng.choice([(64, 128), (64, 128), (64, 64), (32, 128), (16, 64), (8, 128), (4, 32)])
    k = _log_int(rng, 16, 4096)
    B = rng.choice([1, 1, 2, 3, 5])
    most = 8_000_000 // k
    nq = max(1, min(_log_int(rng, 1, 4096), most // B))
    # training batches (every position asks) and chunks at the end of a longer context
    L = nq if rng.random() < 0.5 else _log_int(rng, max(nq, 2), 32768)
    if B * nq * L > 140_000_000:
        L = max(nq, 140_000_000 // (B * nq))
    return dict(op=op, B=B, nq=nq, L=L, H=H, d=d, k=k, ragged=rng.random() < 0.5)


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _lengths(case):
    """(queries, keys) of each sequence: equal, or uneven around the mean; every position asks where nq == L,
    the last nq ones otherwise."""
    out = []
    for b in range(case["B"]):
        f = 1.0 + (0.5 * math.cos(1.0 + 2.4 * b) if case["ragged"] else 0.0)
        nq = max(1, int(case["nq"] * f))
        out.append((nq, max(nq, int(case["L"] * f))))
    return out


def _prepare_scores(case, g):
    lens, H, d, k = _lengths(case), case["H"], case["d"], case["k"]
    q_off = np.concatenate([[0], np.cumsum([a for a, _ in lens])]).tolist()
    k_off = np.concatenate([[0], np.cumsum([b for _, b in lens])]).tolist()
    n_q, n_k = q_off[-1], k_off[-1]
    idx = torch.full((n_q, k), -1, dtype=torch.int32, device="cuda")
    for b, (nq, L) in enumerate(lens):
        # lists as an indexer makes them: neighbouring queries share most of their keys, recent keys are favoured
        for t0 in range(0, nq, 2048):
            t1 = min(nq, t0 + 2048)
            pos = torch.arange(L - nq + t0, L - nq + t1, device="cuda")
            shared = _randn(g, (t1 - t0 + 15) // 16, L).repeat_interleave(16, 0)[: t1 - t0]
            u = 1.5 * shared + _randn(g, t1 - t0, L)
            s = torch.arange(L, device="cuda")
            u += 0.5 * torch.exp((s[None] - pos[:, None]) / (0.1 * L + 1))
            u.masked_fill_(s[None] > pos[:, None], -math.inf)
            m = min(k, L)
            v, i = u.topk(m, dim=1)
            i = torch.where(v > -math.inf, i, L).sort(dim=1).values
            idx[q_off[b] + t0: q_off[b] + t1, :m] = torch.where(i < L, i, -1).int()
    q_pos = np.concatenate([np.arange(L - nq, L) for nq, L in lens])
    # queries with a slowly varying shared part, keys N(0,1), head weights N(0,1)/8
    base = _randn(g, (n_q + 63) // 64, H * d).repeat_interleave(64, 0)[:n_q]
    Q = (0.6 * _randn(g, n_q, H * d) + 0.8 * base).view(n_q, H, d).bfloat16()
    st = dict(Q=Q, K=_randn(g, n_k, d).bfloat16(), W=_randn(g, n_q, H) / 8, idx=idx)
    seq = torch.from_numpy(np.repeat(np.arange(len(lens)), [a for a, _ in lens])).cuda()
    st["k_base"] = torch.tensor(k_off[:-1], device="cuda")[seq]           # [n_q] key row of the sequence's key 0
    if case["op"] == "scores_bwd":
        # the loss's gradient: student less teacher, both softmax over the list, mean over the queries
        a, b = _randn(g, n_q, k) * 1.5, _randn(g, n_q, k) * 1.5
        none = idx < 0
        a.masked_fill_(none, -math.inf)
        b.masked_fill_(none, -math.inf)
        st["ds"] = ((a.softmax(1) - b.softmax(1)) / n_q).nan_to_num_(0.0).contiguous()
    if own:
        import sparse_attention_indexer_04_b200 as dsa
        lay = dsa.Layout(q_off, k_off, q_pos, H, d, "cuda")
        need = dsa.list_scores_backward_workspace(lay, k) if case["op"] == "scores_bwd" else \
            dsa.list_scores_workspace(lay, k)
        st["layout"], st["ws"] = lay, torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(op=op)
    if op in ("norm", "norm_bwd"):
        n, d, pad = case["n"], case["d"], case["pad"]
        xt, yt = _TYPES[case["xt"]], _TYPES[case["yt"]]
        st["x"] = (_randn(g, n, d + pad) * 1.7 + 1.0).to(xt)[:, :d]     # a column slice of a wider projection
        st["w"] = 1.0 + 0.1 * _randn(g, d)
        st["b"] = 0.1 * _randn(g, d)
        st["yt"] = yt
        if op == "norm_bwd":
            st["dy"] = (_randn(g, n, d) * 1e-2).to(yt)
            x = st["x"].double()
            mean = x.mean(1)
            st["mean"] = mean.float()
            st["rstd"] = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        return st
    if op == "distill":
        n, k = case["n"], case["k"]
        s = _randn(g, n, k) * 1.5
        t = 0.7 * s + _randn(g, n, k) * 1.5
        if case["kind"] == "weights":
            t = torch.exp(t - t.amax(1, keepdim=True))
        live = torch.randint(max(1, k // 2), k + 1, (n, 1), generator=g, device="cuda")   # places in use, per row
        none = torch.arange(k, device="cuda") >= live
        st["lists"] = None
        if case["lists"]:   # ascending key indices, -1 behind the last
            step = torch.randint(1, 9, (n, k), generator=g, device="cuda", dtype=torch.int32)
            st["lists"] = step.cumsum(1, dtype=torch.int32).masked_fill_(none, -1)
        s.masked_fill_(none, -math.inf)
        st.update(s=s, t=t.to(_TYPES[case["tt"]]), kind=case["kind"], tau=case["tau"])
        st["g"] = torch.full((n,), 1.0 / n, device="cuda")
        return st
    st.update(_prepare_scores(case, g))
    return st


# ------------------------------------------------------------------------------------------- plain forms

def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    return (c * rstd[:, None] * st["w"] + st["b"]).to(st["yt"]), mean, rstd


def _plain_norm_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    r = st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * r
    gy = dy * st["w"]
    dx = r * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _plain_distill(st):
    s, t = st["s"] / st["tau"], st["t"].float()
    live = s > -math.inf
    if st["lists"] is not None:
        live = live & (st["lists"] >= 0)
    s = torch.where(live, s, -math.inf)
    a = s - s.amax(1, keepdim=True)
    e = torch.exp(a)
    z = e.sum(1, keepdim=True)
    q, logq = e / z, a - torch.log(z)
    if st["kind"] == "logits":
        t = torch.where(live, t / st["tau"], -math.inf)
        c = t - t.amax(1, keepdim=True)
        f = torch.exp(c)
        y = f.sum(1, keepdim=True)
        p, logp = f / y, c - torch.log(y)
    else:
        t = torch.where(live, t, 0.0)
        p = t / t.sum(1, keepdim=True)
        logp = torch.log(p)
    loss = torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    return loss, torch.where(live, (st["g"] / st["tau"])[:, None] * (q - p), 0.0)


def _gathered(st):
    live = st["idx"] >= 0
    rows = st["k_base"][:, None] + st["idx"].clamp(min=0)
    Kg = st["K"].float()[rows]                                     # [n_q, k, d]
    S = torch.bmm(Kg, st["Q"].float().transpose(1, 2))             # [n_q, k, H]
    return live, rows, Kg, S


def _plain_scores(st):
    live, _, _, S = _gathered(st)
    s = torch.bmm(torch.relu_(S), st["W"].unsqueeze(2)).squeeze(2)
    return torch.where(live, s, -math.inf)


def _plain_scores_bwd(st):
    live, rows, Kg, S = _gathered(st)
    ds = torch.where(live, st["ds"], 0.0)
    dW = torch.bmm(ds.unsqueeze(1), torch.relu(S)).squeeze(1)
    G = torch.where(S > 0, ds.unsqueeze(2) * st["W"].unsqueeze(1), 0.0)
    del S
    dQ = torch.bmm(G.transpose(1, 2), Kg)
    dKg = torch.bmm(G, st["Q"].float())
    dK = torch.zeros_like(st["K"], dtype=torch.float32)
    dK.index_add_(0, rows.reshape(-1), dKg.view(-1, dK.shape[1]))
    return dQ.bfloat16(), dK.bfloat16(), dW


def run(state):
    op = state["op"]
    if not own:
        plain = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "distill": _plain_distill,
                 "scores": _plain_scores, "scores_bwd": _plain_scores_bwd}
        return plain[op](state)
    import sparse_attention_indexer_04_b200 as dsa
    if op == "norm":
        return dsa.layer_norm(state["x"], state["w"], state["b"], EPS, out_dtype=state["yt"], want_stats=True)
    if op == "norm_bwd":
        return dsa.layer_norm_backward(state["dy"], state["x"], state["w"], state["mean"], state["rstd"])
    if op == "distill":
        kind = dsa.TEACHER_LOGITS if state["kind"] == "logits" else dsa.TEACHER_WEIGHTS
        return dsa.distill_topk(state["s"], state["t"], lists=state["lists"], kind=kind, temperature=state["tau"],
                                grad_loss=state["g"])
    if op == "scores":
        return dsa.list_scores(state["layout"], state["Q"], state["K"], state["W"], state["idx"], ws=state["ws"])
    return dsa.list_scores_backward(state["layout"], state["Q"], state["K"], state["W"], state["idx"], state["ds"],
                                    ws=state["ws"])


def _pairs(case):
    """Listed (query, key) pairs: a query at position p lists min(k, p + 1) keys."""
    return sum(sum(min(case["k"], p + 1) for p in range(L - nq, L)) for nq, L in _lengths(case))


def work(case):
    op, size = case["op"], {"bf16": 2, "fp32": 4}
    if op == "norm":
        n, d = case["n"], case["d"]
        return {"bytes": n * d * (size[case["xt"]] + size[case["yt"]]) + 8 * d + 8 * n, "flops": 8 * n * d}
    if op == "norm_bwd":
        n, d = case["n"], case["d"]
        return {"bytes": n * d * (2 * size[case["xt"]] + size[case["yt"]]) + 12 * d + 8 * n, "flops": 14 * n * d}
    if op == "distill":
        n, k = case["n"], case["k"]
        return {"bytes": n * k * (8 + size[case["tt"]] + (4 if case["lists"] else 0)) + 8 * n, "flops": 16 * n * k}
    lens, H, d, k = _lengths(case), case["H"], case["d"], case["k"]
    n_q, n_k = sum(a for a, _ in lens), sum(b for _, b in lens)
    pairs = _pairs(case)
    read = n_q * H * d * 2 + min(n_k, pairs) * d * 2 + n_q * H * 4 + n_q * k * 4   # keys: the listed ones at most
    if op == "scores":
        return {"bytes": read + n_q * k * 4, "flops": 2 * pairs * H * d}
    return {"bytes": read + n_q * k * 4 + n_q * H * d * 2 + n_k * d * 2 + n_q * H * 4, "flops": 6 * pairs * H * d}


# ------------------------------------------------------------------------------- the definition in 64 bits

def _exact_scores(st):
    """Query by query over dense masks of the key rows, in blocks of queries of one sequence."""
    K, Q, W = st["K"].double(), st["Q"].double(), st["W"].double()
    n, k = st["idx"].shape
    H, d = Q.shape[1:]
    bwd = st["op"] == "scores_bwd"
    s = torch.full((n, k), -math.inf, dtype=torch.float64, device="cuda")
    dQ, dW, dK = torch.zeros_like(Q), torch.zeros_like(W), torch.zeros_like(K)
    step = max(1, (1 << 28) // (k * max(H, d) * 8))
    for t0 in range(0, n, step):
        r = slice(t0, min(n, t0 + step))
        t, j = torch.nonzero(st["idx"][r] >= 0, as_tuple=True)
        key = st["k_base"][r][t] + st["idx"][r][t, j]
        flat = torch.zeros(st["idx"][r].shape + (d,), dtype=torch.float64, device="cuda")
        flat[t, j] = K[key]
        dot = torch.einsum("thd,tjd->tjh", Q[r], flat)
        if not bwd:
            s[r][t, j] = torch.einsum("tjh,th->tj", dot.clamp(min=0), W[r])[t, j]
            continue
        e = torch.zeros(st["idx"][r].shape, dtype=torch.float64, device="cuda")
        e[t, j] = st["ds"][r].double()[t, j]
        dW[r] = torch.einsum("tj,tjh->th", e, dot.clamp(min=0))
        mask = (dot > 0).double().mul_(e[:, :, None])
        dQ[r] = torch.einsum("tjh,tjd->thd", mask, flat) * W[r][:, :, None]
        part = torch.einsum("tjh,thd->tjd", mask, Q[r] * W[r][:, :, None])
        dK.index_put_((key,), part[t, j], accumulate=True)
    return (dQ, dK, dW) if bwd else s


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op in ("norm", "norm_bwd"):
        x, w = st["x"].double(), st["w"].double()
        d = x.shape[1]
        if op == "norm":
            mean = x.sum(1) / d
            var = (x * x).sum(1) / d - mean * mean
            rstd = 1.0 / torch.sqrt(var.clamp(min=0) + EPS)
            return (x - mean[:, None]) / torch.sqrt(var.clamp(min=0) + EPS)[:, None] * w + st["b"].double(), mean, rstd
        dy, mean, rstd = st["dy"].double(), st["mean"].double(), st["rstd"].double()
        xh = (x - mean[:, None]) * rstd[:, None]
        a = (dy @ w) / d
        b = torch.einsum("nd,nd,d->n", dy, xh, w) / d
        dx = rstd[:, None] * (dy * w - a[:, None] - xh * b[:, None])
        return dx, torch.einsum("nd,nd->d", dy, xh), torch.einsum("nd->d", dy)
    if op == "distill":
        s, t, tau = st["s"].double(), st["t"].double(), st["tau"]
        dead = torch.isneginf(s)
        if st["lists"] is not None:
            dead |= st["lists"] < 0
        logq = (s / tau).masked_fill(dead, -math.inf).log_softmax(1)
        if st["kind"] == "logits":
            p = (t / tau).masked_fill(dead, -math.inf).softmax(1)
        else:
            p = t.masked_fill(dead, 0.0)
            p = p / p.sum(1, keepdim=True)
        loss = torch.special.xlogy(p, p).sum(1) - (p * logq.masked_fill(dead, 0.0)).sum(1)
        return loss, ((logq.exp() - p) * (st["g"].double()[:, None] / tau)).masked_fill(dead, 0.0)
    return _exact_scores(st)
