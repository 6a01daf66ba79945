"""Argument checks of the training operators through the C ABI and the binding (nothing here launches a kernel)."""
import ctypes

import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
from test_abi import host_layout

P, L = ctypes.c_void_p, dsa.library()
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def norm(n=4, d=16, x=0x1000, xt=0, ld_x=16, w=0x2000, b=0x3000, eps=1e-6, y=0x4000, yt=0, ld_y=16, mean=0x5000):
    return L.dsa_layer_norm(n, d, P(x), xt, ld_x, P(w), P(b), eps, P(y), yt, ld_y, P(mean), P(0x6000), None)


def norm_bwd(n=4, d=16, dy=0x1000, dyt=0, x=0x2000, xt=0, mean=0x3000, dx=0x4000, ld=16, dw=0x5000, ws=0x10000,
             ws_bytes=1 << 24):
    return L.dsa_layer_norm_backward(n, d, P(dy), dyt, ld, P(x), xt, ld, None, P(mean), P(0x3100), P(dx), ld, P(dw),
                                     P(0x6000), P(ws), ctypes.c_size_t(ws_bytes), None)


def distill(n=4, k=16, s=0x1000, ld_s=16, lists=0x2000, t=0x3000, tt=1, kind=0, tau=1.0, g=0x4000, loss=0x5000,
            ds=0x6000, ld_t=16, ld_l=16, ld_d=16):
    return L.dsa_distill_topk(n, k, P(s), ld_s, P(lists), ld_l, P(t), tt, ld_t, kind, tau, P(g), P(loss), P(ds), ld_d,
                              None)


def scores(lay, k=4, Q=0x1000, K=0x2000, W=0x3000, lists=0x4000, out=0x5000, ws=0x10000, ws_bytes=1 << 30):
    return L.dsa_list_scores(lay.ref(), P(Q), P(K), P(W), k, P(lists), P(out), P(ws), ctypes.c_size_t(ws_bytes), None)


def scores_bwd(lay, k=4, Q=0x1000, lists=0x4000, ds=0x5000, dQ=0x6000, dK=0x7000, dW=0x8000, ws=0x10000,
               ws_bytes=1 << 30):
    return L.dsa_list_scores_backward(lay.ref(), P(Q), P(0x2000), P(0x3000), k, P(lists), P(ds), P(dQ), P(dK), P(dW),
                                      P(ws), ctypes.c_size_t(ws_bytes), None)


def test_layer_norm_refusals():
    assert norm(n=-1) == INVALID and norm(d=0) == INVALID
    assert norm(eps=-1.0) == INVALID and norm(eps=float("nan")) == INVALID
    assert norm(d=16385, ld_x=16385, ld_y=16385) == UNSUPPORTED
    assert norm(xt=2) == UNSUPPORTED and norm(yt=-1) == UNSUPPORTED
    assert norm(x=0) == INVALID and norm(y=0) == INVALID
    assert norm(ld_x=15) == INVALID and norm(ld_y=8) == INVALID
    assert norm(x=0x1001) == INVALID and norm(y=0x4002, yt=1) == INVALID
    assert norm(w=0x2002) == INVALID and norm(mean=0x5001) == INVALID
    assert norm(n=0, x=0, y=0) == 0


def test_layer_norm_backward_refusals():
    assert norm_bwd(n=-1) == INVALID and norm_bwd(d=0) == INVALID
    assert norm_bwd(d=16385, ld=16385) == UNSUPPORTED
    assert norm_bwd(xt=7) == UNSUPPORTED and norm_bwd(dyt=7) == UNSUPPORTED
    assert norm_bwd(dy=0) == INVALID and norm_bwd(x=0) == INVALID and norm_bwd(mean=0) == INVALID
    assert norm_bwd(ld=15) == INVALID and norm_bwd(dx=0x4001) == INVALID and norm_bwd(dw=0x5001) == INVALID
    assert norm_bwd(ws=0) == WORKSPACE and norm_bwd(ws=0x10010) == WORKSPACE and norm_bwd(ws_bytes=512) == WORKSPACE
    assert dsa.layer_norm_backward_workspace(1 << 20, 128) >= 2 * 128 * 4
    assert dsa.layer_norm_backward_workspace(-1, 128) == 0 and dsa.layer_norm_backward_workspace(4, 16385) == 0


def test_distill_refusals():
    assert distill(n=-1) == INVALID and distill(k=0) == INVALID
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert distill(tau=tau) == INVALID
    assert distill(kind=2) == INVALID and distill(tt=2) == UNSUPPORTED
    assert distill(s=0) == INVALID and distill(t=0) == INVALID
    assert distill(ld_s=15) == INVALID and distill(ld_t=15) == INVALID and distill(ld_l=15) == INVALID
    assert distill(ld_d=15) == INVALID
    assert distill(s=0x1002) == INVALID and distill(lists=0x2001) == INVALID and distill(t=0x3002) == INVALID
    assert distill(g=0x4001) == INVALID and distill(loss=0x5002) == INVALID and distill(ds=0x6002) == INVALID
    assert distill(n=0) == 0 and distill(loss=0, ds=0) == 0


def test_list_scores_refusals():
    lay = host_layout([8], [8])
    assert scores(lay, k=0) == UNSUPPORTED and scores(lay, k=16385) == UNSUPPORTED
    assert scores(lay, Q=0x1008) == INVALID and scores(lay, K=0) == INVALID and scores(lay, W=0x3001) == INVALID
    assert scores(lay, lists=0) == INVALID and scores(lay, out=0) == INVALID and scores(lay, out=0x5002) == INVALID
    assert scores(lay, ws=0) == WORKSPACE and scores(lay, ws=0x10010) == WORKSPACE
    assert scores(lay, ws_bytes=16) == WORKSPACE
    assert scores_bwd(lay, k=0) == UNSUPPORTED and scores_bwd(lay, k=16385) == UNSUPPORTED
    assert scores_bwd(lay, Q=0) == INVALID and scores_bwd(lay, lists=0) == INVALID and scores_bwd(lay, ds=0) == INVALID
    assert scores_bwd(lay, dQ=0x6008) == INVALID and scores_bwd(lay, dK=0x7002) == INVALID
    assert scores_bwd(lay, dW=0x8001) == INVALID and scores_bwd(lay, lists=0x4001) == INVALID
    assert scores_bwd(lay, ws=0) == WORKSPACE and scores_bwd(lay, ws_bytes=16) == WORKSPACE
    for H, d in ((3, 32), (4, 48), (128, 64)):
        bad = host_layout([8], [8], H=H, d=d)
        assert scores(bad) == UNSUPPORTED and scores_bwd(bad) == UNSUPPORTED
        assert dsa.list_scores_workspace(bad, 4) == 0 and dsa.list_scores_backward_workspace(bad, 4) == 0
    assert dsa.list_scores_workspace(lay, 4) > 0 and dsa.list_scores_backward_workspace(lay, 4) > 0
    broken = host_layout([8], [8])
    broken.q_off_host[0] = 1
    assert scores(broken) == INVALID and scores_bwd(broken) == INVALID


def test_binding_takes_cuda_tensors_only():
    x = torch.zeros(4, 16)
    for call in (lambda: dsa.layer_norm(x), lambda: dsa.distill_topk(x, x),
                 lambda: dsa.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
                 lambda: dsa.list_scores(host_layout([4], [4]), x, x, x, x)):
        with pytest.raises(ValueError):
            call()
