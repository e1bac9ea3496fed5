"""GPU tests of the dense feed-forward block where a product runs in several
rounds of 128-column tiles: a pair of CTAs then stores tile after tile, each
behind sums of one to a few stages of 64 k, so that a tile's epilogue meets the
stores of the tile before it.  Sizes are chosen by tiles per pair (74 pairs on a
B200) and stages, in brackets; formulas and tolerances are those of
test_gpu_zz_dense_train."""

import pytest
import torch

from test_gpu_zz_dense_train import ACC, DTYPES, TINY, U, err_word, ffn_ref, gen, near, randn

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")


def case(T, H, I, dtype):
    g = gen(T + 7 * H + I)
    return (randn(g, T, H, dtype=dtype), randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5),
            randn(g, H, I, dtype=dtype, sigma=I ** -0.5), randn(g, T, H, dtype=dtype, sigma=0.5))


# tiles of the down product and of dX, with the stages of the first
ROWS = [(4096, 1152, 64), (4096, 1152, 256), (2160, 2472, 256), (2046, 1360, 256),
        (3000, 3000, 256), (4096, 1160, 200)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,I", ROWS)
def test_down_product_and_dx(T, H, I, dtype):
    # tiles: 144 (1 stage), 144 (4), 180 (4), 88 (4), 288 (4), 160 (4)
    X, Wgu, Wd, dY = case(T, H, I, dtype)
    err = err_word()
    Y, gu = moe.gated_ffn_forward(X, Wgu, Wd, save_gu=True, dev_err=err)
    Yr, terms, _, _, _ = ffn_ref(X, Wgu, Wd)
    near(Y, Yr, terms, dtype, 1.5, "Y")
    dX, _, _ = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd, need_dw=False, dev_err=err)
    ga, up = gu.double().chunk(2, 1)
    s = torch.sigmoid(ga)
    dh, dhs = dY.double() @ Wd.double(), dY.double().abs() @ Wd.double().abs()
    ds = s * (1 + ga * (1 - s))
    dgu = torch.cat([dh * up * ds, dh * ga * s], 1)
    size = dgu.abs() + (ACC / U[dtype]) * torch.cat(
        [dhs * (up * ds).abs(), dhs * (ga * s).abs()], 1) + TINY[dtype] / U[dtype]
    near(dX, dgu @ Wgu.double(), size @ Wgu.double().abs(), dtype, 1.5, "dX")
    for _ in range(10):
        assert torch.equal(Y, moe.gated_ffn_forward(X, Wgu, Wd))
        assert torch.equal(dX, moe.gated_ffn_backward(dY, X, gu, Wgu, Wd, need_dw=False)[0])
    assert int(err.item()) == 0


# dW_gu's tiles (dW_d's) and their stages
WEIGHTS = [(60, 312, 6552), (64, 1304, 4000), (128, 1000, 4104), (129, 1304, 4000),
           (200, 1000, 5000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,I", WEIGHTS)
def test_each_weight_gradient_alone(T, H, I, dtype):
    # tiles: 156 (104) of 1 stage, 352 (192) of 1, 264 (132) of 2, 352 (192) of 3, 320 (160) of 4
    X, Wgu, Wd, dY = case(T, H, I, dtype)
    gu = (X.float() @ Wgu.float().t()).to(dtype)
    ga, up = gu.double().chunk(2, 1)
    s = torch.sigmoid(ga)
    dh, dhs = dY.double() @ Wd.double(), dY.double().abs() @ Wd.double().abs()
    ds = s * (1 + ga * (1 - s))
    dgu = torch.cat([dh * up * ds, dh * ga * s], 1)
    size = dgu.abs() + (ACC / U[dtype]) * torch.cat(
        [dhs * (up * ds).abs(), dhs * (ga * s).abs()], 1) + TINY[dtype] / U[dtype]
    h = ga * s * up
    want = [(dgu.t() @ X.double(), size.t() @ X.double().abs()),
            (dY.double().t() @ h, dY.double().t().abs() @ (h.abs() + TINY[dtype] / U[dtype]))]
    ws = torch.empty(moe.gated_ffn_backward_workspace_size(T, H, I), dtype=torch.uint8,
                     device="cuda")
    err = err_word()
    for i, like in enumerate((Wgu, Wd)):
        outs = []
        for _ in range(10):
            out = torch.full_like(like, 7.0)
            st = moe.load().moe_gated_ffn_backward(
                dY.data_ptr(), {torch.bfloat16: 1, torch.float16: 2}[dtype], X.data_ptr(),
                gu.data_ptr(), Wgu.data_ptr(), Wd.data_ptr(), T, H, I, None,
                out.data_ptr() if i == 0 else None, out.data_ptr() if i == 1 else None,
                ws.data_ptr(), ws.numel(), err.data_ptr(),
                torch.cuda.current_stream().cuda_stream)
            assert st == 0
            outs.append(out)
        near(outs[0], *want[i], dtype, 1.5, ("dW_gu", "dW_d")[i])
        assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert int(err.item()) == 0
