"""GPU tests of the cross entropy's dX where the room for the fp32 sums of its
split reduction bounds the splits: more tiles than fit several times, all rows
counting or few of them, one piece of the vocabulary or several.  Formulas and
tolerances are those of test_gpu_zz_dense_train."""

import pytest
import torch

from test_gpu_zz_dense_train import ACC, U, ce_case, ce_ref, err_word, near

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")


# tiles of 256 x 256: 300 (room for three splits), 1072 (one), with 30 and 80 counting
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,V,ignored", [(5000, 3840, 19000, 0.0), (5000, 3840, 19000, 0.9),
                                           (17000, 4096, 8000, 0.93), (17000, 4096, 1000, 0.0)])
def test_dx_and_dw(T, H, V, ignored, dtype):
    X, W, y, dloss = ce_case(T, H, V, dtype, ignored)
    loss, lse = moe.linear_ce_forward(X, W, y)
    ws = torch.full((moe.linear_ce_backward_workspace_size(T, H, V),), 0xff, dtype=torch.uint8,
                    device="cuda")
    err = err_word()
    dX, dW = moe.linear_ce_backward(dloss, X, W, y, lse, workspace=ws, dev_err=err)
    assert int(err.item()) == 0
    assert (dX[y < 0] == 0).all()
    # the rest on the rows that count
    keep = torch.nonzero(y >= 0)[:, 0]
    Xk, yk, dk, lk = X[keep], y[keep], dloss[keep], lse[keep]
    dl = ce_ref(Xk, W, yk, dk, lk)
    p = (dl / dk.double()[:, None].clamp(min=1e-30)).abs() + \
        (torch.arange(V, device="cuda")[None, :] == yk[:, None])
    lerr = ACC * (Xk.double().abs() @ W.double().abs().t()) + 2.0 ** -20 * (
        1 + lk.double().abs())[:, None]
    under = float(dk.max()) * (2.0 ** -15 * 2.0 ** -25 if dtype == torch.float16 else 1e-38)
    size = dl.abs() + (lerr * p * dk.double()[:, None] + under) / U[dtype]
    near(dX[keep], dl @ W.double(), size @ W.double().abs(), dtype, 1.01, "dX")
    near(dW, dl.t() @ Xk.double(), size.t() @ Xk.double().abs(), dtype, 1.01, "dW")
    again = moe.linear_ce_backward(dloss, X, W, y, lse)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW)
