"""Layer norm of odd widths around the borders of its kernels."""
import pytest
import torch

import sparse_attention_indexer_04_b200 as dsa
import train_ref as ref
from test_gpu_train import gen, randn, strided, untouched

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d", [4097, 5119, 5120, 5121, 6143, 6144, 6145, 7167, 7168, 7169, 8191, 8193])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
def test_wide_rows(d, xt, yt):
    g = gen(d)
    for n in (1, 7):
        x, dy = (randn(g, n, d) * 1.7 + 1.0).to(xt), (randn(g, n, d) * 0.1).to(yt)
        w, b = 1 + 0.1 * randn(g, d), randn(g, d)
        _, xs = strided(x, 3, 1)
        _, dys = strided(dy, 3, 1)
        y, mean, rstd = dsa.layer_norm(xs, w.to(DEV), b.to(DEV), 1e-6, out_dtype=yt, want_stats=True)
        (wy, wm, wr), (ey, em, er) = ref.layer_norm(x, w, b, 1e-6)
        for got, a, e, t, name in zip((y, mean, rstd), (wy, wm, wr), (ey, em, er), (yt, F32, F32), ("y", "mean", "rstd")):
            ref.check(got, a, e, t, f"{name} n={n}")
        big, dxs = strided(torch.zeros(n, d, dtype=xt), 3, 1)
        got = dsa.layer_norm_backward(dys, xs, w.to(DEV), mean, rstd, dx=dxs)
        torch.cuda.synchronize()
        assert untouched(big, d, 1)
        want, bound = ref.layer_norm_backward(dy, x, w, mean.cpu(), rstd.cpu())
        for a, v, e, t, name in zip(got, want, bound, (xt, F32, F32), ("dx", "dw", "db")):
            ref.check(a, v, e, t, f"{name} n={n}")


@pytest.mark.parametrize("n,d", [(0, 16), (1, 16), (300, 128), (5, 5001)])
def test_the_backward_pass_leaves_a_clear_status(n, d):
    """Its workspace begins with a status word like every other's; what stood there is no error of this call."""
    x = randn(gen(n + d), n, d).to(DEV)
    _, mean, rstd = dsa.layer_norm(x, want_stats=True)
    ws = torch.full((dsa.layer_norm_backward_workspace(n, d),), 255, dtype=torch.uint8, device=DEV)
    dsa.layer_norm_backward(x, x, None, mean, rstd, ws=ws)
    assert dsa.device_check(ws) == 0
