"""GPU tests of the dense training-side operators against plain 64-bit
statements of the same formulas: the gated feed-forward block, the vocabulary
cross entropy (both with their gradients), the gradient norm and clipping.

Tolerances.  A 16-bit output is one rounding of an fp32 sum over operands that
were rounded once to 16 bits themselves; with u the largest relative error of
one rounding (bf16 2^-8, fp16 2^-11), each term of the sum is off by at most
u of its own size, so element-wise
    |out - ref| <= u |ref| + u sum |terms| + (fp32 sums: 2^-18 sum |terms|)
and ``sum |terms|`` is computed in 64 bits from the absolute operands.  Where a
gradient's operand is itself a product of rounded values the count of u says so.
"""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25}   # half the least subnormal
ACC = 2.0 ** -18                                            # fp32 sums on the tensor cores
DTYPES = [torch.bfloat16, torch.float16]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def near(out, ref, terms, dtype, rounds=1, what=""):
    """Element-wise: ``rounds`` roundings of the summed terms, one of the result."""
    u = U[dtype]
    out, lim = out.double(), u * ref.abs() + (rounds * u + ACC) * terms + TINY[dtype]
    assert torch.isfinite(out).all(), f"{what}: not finite"
    over = (out - ref).abs() - lim
    worst = int(over.argmax())
    assert over.max() <= 0, (f"{what}: element {worst} is {out.flatten()[worst]}, "
                             f"ref {ref.flatten()[worst]}, bound {lim.flatten()[worst]}")


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------- feed-forward block


def ffn_ref(X, Wgu, Wd, residual=None):
    X, Wgu, Wd = X.double(), Wgu.double(), Wd.double()
    g, u = (X @ Wgu.t()).chunk(2, 1)
    h = g * torch.sigmoid(g) * u
    Y, terms = h @ Wd.t(), h.abs() @ Wd.t().abs()
    if residual is not None:
        Y = Y + residual.double()
    return Y, terms, torch.cat([g, u], 1), X.abs() @ Wgu.t().abs(), h


# rows from one to several tiles, widths that fill no tile, splits along k and none
FFN = [(3, 2056, 4096), (11, 2048, 4096), (2, 4096, 8192), (14, 4096, 4096), (33, 256, 8192),
       (5, 464, 7712), (12, 4096, 256), (9, 264, 4200), (400, 640, 1504), (1, 256, 256),
       (64, 8, 8), (90, 264, 1000), (96, 2048, 512), (128, 512, 1096), (129, 264, 72),
       (1, 2048, 1024), (3, 8, 8), (17, 72, 520), (32, 1024, 2048), (40, 136, 264),
       (255, 256, 128), (256, 512, 384), (257, 264, 1032), (300, 1000, 2744), (1024, 512, 256),
       (2049, 384, 640)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,I", FFN)
def test_ffn_forward(T, H, I, dtype):
    g = gen(T + H + I)
    X = randn(g, T, H, dtype=dtype)
    Wgu = randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5)
    Wd = randn(g, H, I, dtype=dtype, sigma=I ** -0.5)
    R = randn(g, T, H)
    err = err_word()
    for res in (None, R):
        Y, gu = moe.gated_ffn_forward(X, Wgu, Wd, residual=res, save_gu=True, dev_err=err)
        Yr, terms, gur, gterms, _ = ffn_ref(X, Wgu, Wd, res)
        near(gu, gur, gterms, dtype, rounds=0, what="gu")
        # h carries its own rounding, and g's and u's fp32 sums through silu'
        # (at most 1.1) and the other factor: within one more u of |h| plus
        # ACC-sized parts, counted as half a rounding more
        near(Y, Yr, terms, dtype, rounds=1.5, what="Y")
        assert torch.equal(Y, moe.gated_ffn_forward(X, Wgu, Wd, residual=res))
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,I", FFN)
def test_ffn_backward(T, H, I, dtype):
    g = gen(T * 3 + H + I)
    X = randn(g, T, H, dtype=dtype)
    Wgu = randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5)
    Wd = randn(g, H, I, dtype=dtype, sigma=I ** -0.5)
    dY = randn(g, T, H, dtype=dtype, sigma=0.5)
    gu = (X.float() @ Wgu.float().t()).to(dtype)
    err = err_word()
    dX, dWgu, dWd = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd, dev_err=err)
    assert int(err.item()) == 0
    ga, up = gu.double().chunk(2, 1)
    s = torch.sigmoid(ga)
    dh = dY.double() @ Wd.double()
    dhs = dY.double().abs() @ Wd.double().abs()  # what dh's fp32 sum can lose: ACC of this
    ds = s * (1 + ga * (1 - s))
    dgu = torch.cat([dh * up * ds, dh * ga * s], 1)
    slack = torch.cat([dhs * (up * ds).abs(), dhs * (ga * s).abs()], 1)
    h = ga * s * up
    size = dgu.abs() + (ACC / U[dtype]) * slack + TINY[dtype] / U[dtype]
    near(dX, dgu @ Wgu.double(), size @ Wgu.double().abs(), dtype, 1.5, "dX")
    near(dWgu, dgu.t() @ X.double(), size.t() @ X.double().abs(), dtype, 1.5, "dW_gu")
    near(dWd, dY.double().t() @ h, dY.double().t().abs() @ (h.abs() + TINY[dtype] / U[dtype]),
         dtype, 1.5, "dW_d")
    a, b, c = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd, need_dw=False)
    assert b is None and c is None and torch.equal(a, dX)
    a, b, c = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd, need_dx=False)
    assert a is None and torch.equal(b, dWgu) and torch.equal(c, dWd)


def test_ffn_gradient_against_differences():
    # the sum of dY * Y along a random direction of X, by central differences
    # of the 64-bit formula; fp16 inputs, a step that keeps them in 64 bits
    T, H, I, dtype = 9, 64, 96, torch.float16
    g = gen(5)
    X, Wgu, Wd = (randn(g, T, H, dtype=dtype), randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5),
                  randn(g, H, I, dtype=dtype, sigma=I ** -0.5))
    dY = randn(g, T, H, dtype=dtype)
    _, gu = moe.gated_ffn_forward(X, Wgu, Wd, save_gu=True)
    grads = moe.gated_ffn_backward(dY, X, gu, Wgu, Wd)
    for i, t in enumerate((X, Wgu, Wd)):
        d = randn(g, *t.shape).double()
        vals = []
        for sgn in (1, -1):
            args = [x.double() for x in (X, Wgu, Wd)]
            args[i] = args[i] + sgn * 1e-4 * d
            vals.append((ffn_ref(*args)[0] * dY.double()).sum())
        diff = (vals[0] - vals[1]) / 2e-4
        got = (grads[i].double() * d).sum()
        # a random sum of n gradients, each within about 4 u of its size
        bound = 4 * U[dtype] * (grads[i].double() * d).norm() * 4 + 1e-6 * abs(diff)
        assert abs(got - diff) <= bound, (i, float(got), float(diff), float(bound))


# ------------------------------------------------------------- cross entropy


def ce_case(T, H, V, dtype, ignored, seed=0):
    g = gen(T + H + V + seed)
    W = randn(g, V, H, dtype=dtype, sigma=H ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    X = (randn(g, T, H) + 6 * torch.rand((T, 1), generator=g, device="cuda") *
         W[y].float()).to(dtype)
    gone = torch.rand((T,), generator=g, device="cuda") < ignored
    y = torch.where(gone, torch.full_like(y, -100), y).int()
    dl = torch.rand((T,), generator=g, device="cuda") * (0.01 if dtype == torch.bfloat16 else 8.0)
    return X, W, y, dl


def ce_ref(X, W, y, dloss=None, lse=None):
    keep = (y >= 0)
    at = y.long().clamp(min=0)
    l = X.double() @ W.double().t()
    rlse = torch.where(keep, torch.logsumexp(l, 1), 0.0)
    loss = torch.where(keep, rlse - l.gather(1, at[:, None])[:, 0], 0.0)
    if dloss is None:
        return loss, rlse
    p = torch.exp(l - lse.double()[:, None])
    p[torch.arange(len(y)), at] -= 1
    return torch.where(keep[:, None], p * dloss.double()[:, None], 0.0)


CE = [(33, 264, 40003, 0.3), (3, 128, 30000, 0.4), (600, 200, 9000, 0.5), (1, 64, 1, 0.0),
      (70, 128, 1000, 0.0), (96, 72, 129, 0.3), (128, 512, 2051, 0.0), (129, 64, 300, 0.2),
      (1, 256, 50304, 0.0), (5, 8, 7, 0.0), (33, 72, 255, 0.0), (40, 1024, 256, 0.3),
      (64, 136, 257, 0.5), (200, 264, 1000, 0.0), (256, 512, 5003, 0.25), (300, 256, 32003, 0.9),
      (513, 128, 700, 0.0), (1030, 320, 4099, 0.4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,V,ignored", CE)
def test_ce_forward(T, H, V, ignored, dtype):
    X, W, y, _ = ce_case(T, H, V, dtype, ignored)
    err = err_word()
    loss, lse = moe.linear_ce_forward(X, W, y, dev_err=err)
    assert int(err.item()) == 0
    rloss, rlse = ce_ref(X, W, y)
    # a logit's fp32 sum is off by at most ACC of its absolute terms; lse moves
    # by at most the largest such error, plus its own fp32 arithmetic
    slack = ACC * (X.double().abs() @ W.double().abs().t()).amax(1) + 2.0 ** -19 * (
        1 + rlse.abs())
    slack = torch.where(y >= 0, slack, 0.0)
    assert ((lse.double() - rlse).abs() <= slack).all()
    assert ((loss.double() - rloss).abs() <= 2 * slack).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,V,ignored", CE)
def test_ce_backward(T, H, V, ignored, dtype):
    X, W, y, dloss = ce_case(T, H, V, dtype, ignored)
    _, rlse = ce_ref(X, W, y)
    lse = rlse.float()
    err = err_word()
    dX, dW = moe.linear_ce_backward(dloss, X, W, y, lse, dev_err=err)
    assert int(err.item()) == 0
    dl = ce_ref(X, W, y, dloss, lse)
    # exp(l - lse) in fp32: the logit's error (ACC of its terms) and that of the
    # scaled argument act on p, where p - 1 has cancelled too
    p = (dl / dloss.double()[:, None].clamp(min=1e-30)).abs() + \
        (torch.arange(V, device="cuda")[None, :] == y[:, None])
    lerr = ACC * (X.double().abs() @ W.double().abs().t()) + 2.0 ** -20 * (1 + rlse.abs())[:, None]
    keep = (y >= 0)[:, None]
    u = U[dtype]
    big = float(dloss[y >= 0].max()) if (y >= 0).any() else 1.0
    under = big * (2.0 ** -15 * 2.0 ** -25 if dtype == torch.float16 else 1e-38)
    size = torch.where(keep, dl.abs() + (lerr * p * dloss.double()[:, None] + under) / u, 0.0)
    near(dX, dl @ W.double(), size @ W.double().abs(), dtype, 1.01, "dX")
    near(dW, dl.t() @ X.double(), size.t() @ X.double().abs(), dtype, 1.01, "dW")
    assert (dX[y < 0] == 0).all()
    a, b = moe.linear_ce_backward(dloss, X, W, y, lse, need_dw=False)
    assert b is None and torch.equal(a, dX)
    a, b = moe.linear_ce_backward(dloss, X, W, y, lse, need_dx=False)
    assert a is None and torch.equal(b, dW)


# ------------------------------------------------------------- gradient norm and clipping


def clip_check(grads, max_norm, outs=None, err=None):
    before = [t.clone() for t in grads]
    norm = moe.grad_norm_clip(moe.grad_list(grads, outs), max_norm, dev_err=err)
    ref = math.sqrt(sum(float(t.double().square().sum()) for t in before))
    # eight squares per fp32 sum: at most 8 roundings of 2^-24 on the sum, half on the root
    # (a norm beyond fp32's 3.4e38 reads as infinity; the clipping still holds)
    if ref > torch.finfo(torch.float32).max:
        assert float(norm) == math.inf
    else:
        assert abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref + 1e-45
    c = min(1.0, max_norm / (ref + 1e-6))
    for b, o, t in zip(before, outs or grads, grads):
        u = {torch.float32: 2.0 ** -24, **U}[t.dtype]
        tiny = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134,
                torch.float16: 2.0 ** -25}[t.dtype]
        lim = (u + 8 * 2.0 ** -24) * (b.double() * c).abs() + tiny
        assert ((o.double() - b.double() * c).abs() <= lim).all()
        if outs is not None:
            assert torch.equal(t, b)


@pytest.mark.parametrize("dtype", [torch.float32] + DTYPES)
@pytest.mark.parametrize("sizes", [[1], [7], [8192], [8193, 0, 1, 16], [100003, 5, 8191, 64] * 3,
                                   [33] * 65, [1000] * 700, [40] * 1100, [9001] * 2100])
def test_clip_sizes_types_and_places(dtype, sizes):
    g = gen(len(sizes) + sizes[0])
    grads = [randn(g, n, dtype=dtype, sigma=0.1) for n in sizes]
    total = sum(sizes)
    clip_check(grads, 0.02 * total ** 0.5)                                  # in place
    clip_check(grads, 10.0 * total ** 0.5)                                  # nothing to clip
    clip_check(grads, 0.01 * total ** 0.5, [torch.empty_like(t) for t in grads])


def test_clip_mixed_types_and_odd_addresses():
    g = gen(3)
    flats = [randn(g, 40000, dtype=d, sigma=0.3) for d in (torch.float32, *DTYPES)]
    outs = [torch.zeros_like(f) for f in flats]
    cuts = [(1, 5000), (5001, 5004), (5007, 21000), (21000, 39999)]
    grads = [f[a:b] for f in flats for a, b in cuts]
    same = [o[a:b] for o in outs for a, b in cuts]
    clip_check(grads, 1.0, same)
    for o in outs:  # what lies between them is left as it was
        assert o[0] == 0 and (o[5004:5007] == 0).all() and o[39999] == 0
    shifted = [o[a + 1:b + 1] for o in outs for a, b in cuts]  # other alignment than the input
    clip_check(grads, 1.0, shifted)


def test_clip_range_zero_and_nonfinite():
    err = err_word()
    for scale in (0.0, 1e-30, 1e-41, 1e19, 3e37):
        clip_check([torch.full((1000,), scale, device="cuda"),
                    torch.full((9,), scale / 2, device="cuda")], max(scale, 1e-3), err=err)
    assert int(err.item()) == 0
    for bad in (math.nan, math.inf):
        t = torch.ones(5000, device="cuda")
        t[4321] = bad
        keep = t.clone()
        norm = moe.grad_norm_clip([t], 0.5, dev_err=err)
        assert not math.isfinite(float(norm)) and int(err.item()) & moe.DEVERR_NONFINITE
        assert torch.equal(t[:4321], keep[:4321])
        err.zero_()
