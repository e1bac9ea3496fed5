"""GPU tests of the dense training-side operators on matrices of more than 2^31
elements, where an index or an offset of 32 bits would wrap.  What lies at both
ends is compared with 64-bit formulas (as in test_gpu_zz_dense_train)."""

import math

import pytest
import torch

from test_gpu_zz_dense_train import ACC, U, err_word, ffn_ref, gen, near, randn

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")

BF16 = torch.bfloat16


def test_clipping_one_far_tensor():
    n = (1 << 31) + 17
    g = gen(1)
    t = torch.empty(n, dtype=BF16, device="cuda").normal_(0.0, 1e-3, generator=g)
    ends = [slice(0, 4096), slice((1 << 31) - 4096, n)]
    before = [t[s].double() for s in ends]
    total = sum(float(t[a:a + (1 << 28)].double().square().sum()) for a in range(0, n, 1 << 28))
    norm = moe.grad_norm_clip([t], 0.5 * math.sqrt(total))
    assert abs(float(norm) - math.sqrt(total)) <= 6 * 2.0 ** -24 * math.sqrt(total)
    f = 0.5 * math.sqrt(total) / (math.sqrt(total) + 1e-6)
    for s, b in zip(ends, before):
        assert ((t[s].double() - b * f).abs()
                <= (U[BF16] + 8 * 2.0 ** -24) * (b * f).abs() + 2.0 ** -134).all()


@pytest.mark.parametrize("T", [33, 200])
def test_cross_entropy_of_a_far_vocabulary(T):
    H, V = 4104, 530000
    g = gen(T)
    W = torch.empty((V, H), dtype=BF16, device="cuda").normal_(0.0, H ** -0.5, generator=g)
    assert W.numel() > 1 << 31
    X = randn(g, T, H, dtype=BF16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    y[0], y[1], y[2] = V - 1, 0, -100
    dl = torch.rand((T,), generator=g, device="cuda") * 0.01
    keep = y >= 0
    xs = X.double()
    l = torch.cat([xs @ W[a:a + 50000].double().t() for a in range(0, V, 50000)], 1)
    rlse = torch.where(keep, torch.logsumexp(l, 1), 0.0)
    at = y.long().clamp(min=0)[:, None]
    rloss = torch.where(keep, rlse - l.gather(1, at)[:, 0], 0.0)
    terms = torch.stack([(xs.abs() @ W[a:a + 50000].double().abs().t()).amax(1)
                         for a in range(0, V, 50000)], 1).amax(1)
    slack = torch.where(keep, ACC * terms + 2.0 ** -19 * (1 + rlse.abs()), 0.0)
    err = err_word()
    loss, lse = moe.linear_ce_forward(X, W, y, dev_err=err)
    assert ((lse.double() - rlse).abs() <= slack).all()
    assert ((loss.double() - rloss).abs() <= 2 * slack).all()
    dX, dW = moe.linear_ce_backward(dl, X, W, y, lse, dev_err=err)
    assert int(err.item()) == 0
    p = torch.exp(l - lse.double()[:, None])
    del l
    d = p.scatter_add(1, at, torch.full_like(at, -1, dtype=torch.float64))
    scale = torch.where(keep, dl, 0.0).double()[:, None]
    lerr = (ACC * terms + 2.0 ** -20 * (1 + rlse.abs()))[:, None]
    # p itself carries the logit's error, where p - 1 has cancelled too
    size = (d.abs() + lerr * p / U[BF16] + 1e-38) * scale
    d = d * scale
    ref, bound = torch.zeros_like(xs), torch.zeros_like(xs)
    for a in range(0, V, 50000):
        w = W[a:a + 50000].double()
        ref += d[:, a:a + 50000] @ w
        bound += size[:, a:a + 50000] @ w.abs()
    near(dX, ref, bound, BF16, 1.01, "dX")
    assert (dX[2] == 0).all()
    for s in (slice(0, 3000), slice(V // 2, V // 2 + 3000), slice(V - 3000, V)):
        near(dW[s], d[:, s].t() @ xs, size[:, s].t() @ xs.abs(), BF16, 1.01, "dW")


def test_feed_forward_of_far_rows():
    T, H, I = 262200, 64, 4096
    g = gen(2)
    X = randn(g, T, H, dtype=BF16)
    Wgu = randn(g, 2 * I, H, dtype=BF16, sigma=H ** -0.5)
    Wd = randn(g, H, I, dtype=BF16, sigma=I ** -0.5)
    dY = randn(g, T, H, dtype=BF16)
    Y, gu = moe.gated_ffn_forward(X, Wgu, Wd, save_gu=True)
    assert gu.numel() > 1 << 31
    dX, dWgu, dWd = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd)
    refs = [torch.zeros_like(w, dtype=torch.float64) for w in (Wgu, Wgu, Wd, Wd)]
    for a in range(0, T, 32768):
        s = slice(a, min(a + 32768, T))
        x, dy = X[s].double(), dY[s].double()
        if a == 0 or a + 32768 > T:
            near(gu[s], x @ Wgu.double().t(), x.abs() @ Wgu.double().abs().t(), BF16, 0, "gu")
        ga, up = gu[s].double().chunk(2, 1)
        sg = torch.sigmoid(ga)
        h = ga * sg * up
        dh, dhs = dy @ Wd.double(), dy.abs() @ Wd.double().abs()
        ds = sg * (1 + ga * (1 - sg))
        dgu = torch.cat([dh * up * ds, dh * ga * sg], 1)
        size = dgu.abs() + (ACC / U[BF16]) * torch.cat(
            [dhs * (up * ds).abs(), dhs * (ga * sg).abs()], 1)
        if a == 0 or a + 32768 > T:
            Yr, terms, _, _, _ = ffn_ref(X[s], Wgu, Wd)
            near(Y[s], Yr, terms, BF16, 1.5, "Y")
            near(dX[s], dgu @ Wgu.double(), size @ Wgu.double().abs(), BF16, 1.5, "dX")
        refs[0] += dgu.t() @ x
        refs[1] += size.t() @ x.abs()
        refs[2] += dy.t() @ h
        refs[3] += dy.t().abs() @ h.abs()
    near(dWgu, refs[0], refs[1], BF16, 1.5, "dW_gu")
    near(dWd, refs[2], refs[3], BF16, 1.5, "dW_d")
