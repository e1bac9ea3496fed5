"""GPU tests of how the dense training-side operators are used: captured into
graphs and replayed on new inputs, on other streams, two calls at once, a
workspace used again, repeated bits, ignored and bad targets, infinities, rows
that must stay as they were, and a training step of all of them around the
routed layer.  Tolerances: see test_gpu_zz_dense_train."""

import math

import pytest
import torch

from test_gpu_zz_dense_train import (ACC, DTYPES, TINY, U, ce_case, ce_ref, err_word, ffn_ref, gen,
                                     near, randn)

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")

# a size for each way that the operators split their work
FFN = [(1, 256, 256), (5, 464, 7712), (24, 512, 384), (100, 256, 8192), (200, 520, 1032),
       (700, 512, 1024)]
CE = [(2, 64, 300), (33, 264, 40003), (100, 128, 2051), (300, 256, 5003), (2100, 64, 700)]


def ffn_case(T, H, I, dtype=torch.bfloat16, seed=0):
    g = gen(T + H + I + seed)
    return {"X": randn(g, T, H, dtype=dtype),
            "W_gu": randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5),
            "W_d": randn(g, H, I, dtype=dtype, sigma=I ** -0.5), "R": randn(g, T, H),
            "dY": randn(g, T, H, dtype=dtype)}


def ffn_pass(c, ws=None, ws_b=None):
    Y, gu = moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], residual=c["R"], save_gu=True,
                                  workspace=ws)
    return [Y, gu, *moe.gated_ffn_backward(c["dY"], c["X"], gu, c["W_gu"], c["W_d"],
                                           workspace=ws_b)]


def loss_case(T, H, V, seed=0):
    X, W, y, dl = ce_case(T, H, V, torch.bfloat16, 0.3, seed)
    return {"X": X, "W": W, "y": y, "dl": dl}


def loss_pass(c, ws=None, ws_b=None):
    loss, lse = moe.linear_ce_forward(c["X"], c["W"], c["y"], workspace=ws)
    return [loss, lse, *moe.linear_ce_backward(c["dl"], c["X"], c["W"], c["y"], lse,
                                               workspace=ws_b)]


def clip_case(n, m, seed=0):
    g = gen(n + m + seed)
    return {"g": [randn(g, m + 3 * i, dtype=(torch.float32, *DTYPES)[i % 3]) for i in range(n)]}


def clip_pass(c, ws=None, ws_b=None):
    outs = [torch.empty_like(t) for t in c["g"]]
    return [moe.grad_norm_clip(moe.grad_list(c["g"], outs), 0.5, workspace=ws), *outs]


PASSES = [(ffn_case, ffn_pass, s) for s in FFN] + [(loss_case, loss_pass, s) for s in CE] + \
    [(clip_case, clip_pass, s) for s in [(2, 50), (40, 40000), (600, 9)]]
IDS = [f"{p.__name__}-{'-'.join(map(str, s))}" for _, p, s in PASSES]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def tensors(c):
    return [t for v in c.values() for t in (v if isinstance(v, list) else [v])]


@pytest.mark.parametrize("case,run,size", PASSES, ids=IDS)
def test_same_bits_on_every_stream_and_in_a_graph(case, run, size):
    c, other = case(*size), case(*size, seed=7)
    want, want_other = run(c), run(other)
    assert same(run(c), want)                              # again: the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = run(c)
    side.synchronize()
    assert same(on_side, want)
    # captured, then replayed on inputs that were written over the captured ones
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(c)
    for src, expect in ((None, want), (other, want_other), (other, want_other)):
        if src is not None:
            for dst, s in zip(tensors(c), tensors(src), strict=True):
                dst.copy_(s)
        g.replay()
        torch.cuda.synchronize()
        assert same(out, expect)


@pytest.mark.parametrize("case,run,size", PASSES, ids=IDS)
def test_two_calls_at_once(case, run, size):
    cs = [case(*size, seed=s) for s in (1, 2)]
    want = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(run(cs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("size", FFN)
def test_ffn_workspace_given_dirty_and_shared_by_graphs(size):
    T, H, I = size
    cs = [ffn_case(*size, seed=s) for s in (1, 2)]
    want = [ffn_pass(c) for c in cs]
    ws = torch.full((moe.gated_ffn_forward_workspace_size(T, H, I),), 0xff, dtype=torch.uint8,
                    device="cuda")
    wb = torch.full((moe.gated_ffn_backward_workspace_size(T, H, I),), 0xff, dtype=torch.uint8,
                    device="cuda")
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ffn_pass(c, ws, wb))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:  # one stream: one after the other
            g.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("size", CE)
def test_ce_workspace_given_dirty_and_shared_by_graphs(size):
    cs = [loss_case(*size, seed=s) for s in (1, 2)]
    want = [loss_pass(c) for c in cs]
    ws = torch.full((moe.linear_ce_forward_workspace_size(*size),), 0xff, dtype=torch.uint8,
                    device="cuda")
    wb = torch.full((moe.linear_ce_backward_workspace_size(*size),), 0xff, dtype=torch.uint8,
                    device="cuda")
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(loss_pass(c, ws, wb))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))


@pytest.mark.parametrize("size", FFN)
def test_ffn_leaves_the_rows_behind_as_they_were(size):
    T, H, I = size
    c = ffn_case(*size)
    out = torch.full((T + 3, H), 7.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((T + 3, 2 * I), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], out=out[:T], gu=gu[:T])
    assert (out[T:] == 7).all() and (gu[T:] == 7).all()
    want = moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"])
    assert torch.equal(out[:T], want)


def test_no_rows():
    c = ffn_case(0, 64, 48)
    Y, gu = moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], save_gu=True)
    assert Y.shape == (0, 64) and gu.shape == (0, 96)
    dX, dWgu, dWd = moe.gated_ffn_backward(c["dY"], c["X"], gu, c["W_gu"], c["W_d"])
    assert dX.shape == (0, 64) and (dWgu == 0).all() and (dWd == 0).all()
    X, W, y = c["X"], c["W_gu"], torch.zeros(0, dtype=torch.int32, device="cuda")
    loss, lse = moe.linear_ce_forward(X, W, y)
    assert loss.shape == lse.shape == (0,)
    dX, dW = moe.linear_ce_backward(loss, X, W, y, lse)
    assert dX.shape == (0, 64) and (dW == 0).all()


# one size per way of the cross entropy
@pytest.mark.parametrize("T,H,V", CE + [(9000, 64, 300)])
def test_ce_ignored_and_bad_targets(T, H, V):
    X, W, y, dl = ce_case(T, H, V, torch.bfloat16, 0.5, 3)
    # all ignored, by an index that is also a word
    same_y = torch.full_like(y, 5)
    loss, lse = moe.linear_ce_forward(X, W, same_y, ignore_index=5)
    assert (loss == 0).all() and (lse == 0).all()
    dX, dW = moe.linear_ce_backward(dl, X, W, same_y, lse, ignore_index=5)
    assert (dX == 0).all() and (dW == 0).all()
    # NaN and infinities in what is ignored reach nothing
    want = moe.linear_ce_forward(X, W, y)
    grads = moe.linear_ce_backward(dl, X, W, y, want[1])
    gone = y < 0
    dirty, dl2 = X.clone(), dl.clone()
    dirty[gone] = math.nan
    dirty[gone, ::3] = math.inf
    dl2[gone] = math.nan
    lse2 = torch.where(gone, math.nan, want[1])
    assert same(moe.linear_ce_forward(dirty, W, y), want)
    assert same(moe.linear_ce_backward(dl2, dirty, W, y, lse2), grads)
    # a target outside the vocabulary: reported, and as if ignored
    err = err_word()
    bad = y.clone()
    bad[gone] = V
    bad[torch.nonzero(gone)[::2]] = -7
    assert same(moe.linear_ce_forward(X, W, bad, dev_err=err), want)
    assert int(err.item()) == (moe.DEVERR_BAD_INDEX if gone.any() else 0)
    err.zero_()
    assert same(moe.linear_ce_backward(dl, X, W, bad, want[1], dev_err=err), grads)
    assert int(err.item()) == (moe.DEVERR_BAD_INDEX if gone.any() else 0)


@pytest.mark.parametrize("T,H,V", CE)
def test_ce_far_logits_and_confident_rows(T, H, V):
    # logits of hundreds: the target's far above the rest (loss 0, not below) or
    # far below it
    g = gen(11)
    W = randn(g, V, H, dtype=torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    sign = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)
    X = (sign[:, None] * 8 * W[y.long()].float()).bfloat16()
    loss, lse = moe.linear_ce_forward(X, W, y)
    rloss, rlse = ce_ref(X, W, y)
    slack = ACC * (X.double().abs() @ W.double().abs().t()).amax(1) + 2.0 ** -19 * (1 + rlse.abs())
    assert ((lse.double() - rlse).abs() <= slack).all()
    assert ((loss.double() - rloss).abs() <= 2 * slack).all()
    assert (loss >= 0).all()
    # an infinite or NaN input shows in its row only
    if T > 1:
        X[0, 0], X[1, 0] = math.nan, math.inf
        loss2, _ = moe.linear_ce_forward(X, W, y)
        assert not torch.isfinite(loss2[:2]).any() and torch.equal(loss2[2:], loss[2:])


@pytest.mark.parametrize("scale", [0.0, 1e-20, 1e20, -1.0])
def test_ce_backward_upstream_scales(scale):
    for T, H, V in ((40, 64, 300), (300, 64, 300)):
        X, W, y, dl = ce_case(T, H, V, torch.bfloat16, 0.2, 4)
        lse = moe.linear_ce_forward(X, W, y)[1]
        dl = dl * scale
        dX, dW = moe.linear_ce_backward(dl, X, W, y, lse)
        ref = ce_ref(X, W, y, dl, lse)
        # as in test_ce_backward: one rounding of dl, of the sums, and of exp's argument
        p = ce_ref(X, W, y, torch.ones_like(dl), lse).abs() + 1
        lerr = ACC * (X.double().abs() @ W.double().abs().t()) + 2.0 ** -20 * (
            1 + lse.double().abs())[:, None]
        size = ref.abs() + lerr * p * dl.double().abs()[:, None] / U[torch.bfloat16]
        size = torch.where((y >= 0)[:, None], size, 0.0)
        near(dX, ref @ W.double(), size @ W.double().abs(), torch.bfloat16, 1.01, "dX")
        near(dW, ref.t() @ X.double(), size.t() @ X.double().abs(), torch.bfloat16, 1.01, "dW")


@pytest.mark.parametrize("T,H,V", [(2049, 64, 60001), (260, 72, 530000)])
def test_ce_backward_in_pieces_of_the_vocabulary(T, H, V):
    # dl of all rows beyond 256 MB: two pieces and more
    X, W, y, dl = ce_case(T, H, V, torch.bfloat16, 0.4, 5)
    assert (T + 255) // 256 * 256 * V * 2 > 256 << 20
    lse = moe.linear_ce_forward(X, W, y)[1]
    dX, dW = moe.linear_ce_backward(dl, X, W, y, lse)
    u = U[torch.bfloat16]
    lerr = ACC * H * float(X.abs().max()) * float(W.abs().max()) + 2.0 ** -20 * (
        1 + float(lse.abs().max()))
    for sl in (slice(0, 4000), slice(V // 2 - 2000, V // 2 + 2000), slice(V - 4001, V)):
        l = X.double() @ W[sl].double().t()
        hot = (torch.arange(V, device="cuda")[sl][None, :] == y[:, None]).double()
        scale = torch.where(y >= 0, dl, 0.0).double()[:, None]
        d = (torch.exp(l - lse.double()[:, None]) - hot) * scale
        size = d.abs() + lerr * (d.abs() + hot * scale) / u
        near(dW[sl], d.t() @ X.double(), size.t() @ X.double().abs(), torch.bfloat16, 1.01, "dW")
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    terms = torch.zeros_like(ref)
    for v0 in range(0, V, 20000):
        Wi = W[v0:v0 + 20000].double()
        hot = (torch.arange(v0, v0 + len(Wi), device="cuda")[None, :] == y[:, None]).double()
        scale = torch.where(y >= 0, dl, 0.0).double()[:, None]
        d = (torch.exp(X.double() @ Wi.t() - lse.double()[:, None]) - hot) * scale
        ref += d @ Wi
        terms += (d.abs() + lerr * (d.abs() + hot * scale) / u) @ Wi.abs()
    near(dX, ref, terms, torch.bfloat16, 1.01, "dX")
    assert (dX[y < 0] == 0).all()


@pytest.mark.parametrize("T", [3, 40, 200])
def test_ffn_range_and_infinities(T):
    c = ffn_case(T, 64, 72, torch.float16)
    err = err_word()
    moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], dev_err=err)
    assert int(err.item()) == 0
    big = c["X"].clone()
    big[1] *= 6e4 / big[1].abs().max()
    Y = moe.gated_ffn_forward(big, c["W_gu"], c["W_d"], dev_err=err)
    assert int(err.item()) & moe.DEVERR_RANGE        # h beyond fp16
    ok = [i for i in range(T) if i != 1]
    assert torch.equal(Y[ok], moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"])[ok])
    # gates at the type's ends: silu is 0 far below and the gate itself far above
    gu = torch.empty((T, 144), dtype=torch.bfloat16, device="cuda")
    lo = torch.finfo(torch.bfloat16).min
    gu[:, :36], gu[:, 36:72], gu[:, 72:] = lo, 300.0, 0.5
    b = ffn_case(T, 64, 72, torch.bfloat16)
    dX, dWgu, dWd = moe.gated_ffn_backward(b["dY"], b["X"], gu, b["W_gu"], b["W_d"])
    assert all(torch.isfinite(t).all() for t in (dX, dWgu, dWd))
    assert (dWd[:, :36] == 0).all() and (dWgu[:36] == 0).all() and (dWgu[72:108] == 0).all()


@pytest.mark.parametrize("T", [20, 300])
def test_ffn_each_gradient_alone(T):
    # the C call takes any subset; the binding asks for both weights or none
    H, I = 72, 136
    c = ffn_case(T, H, I)
    _, gu = moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], save_gu=True)
    want = moe.gated_ffn_backward(c["dY"], c["X"], gu, c["W_gu"], c["W_d"])
    ws = torch.empty(moe.gated_ffn_backward_workspace_size(T, H, I), dtype=torch.uint8,
                     device="cuda")
    for i in range(3):
        out = [torch.empty_like(w) if i == j else None for j, w in enumerate(want)]
        st = moe.load().moe_gated_ffn_backward(
            c["dY"].data_ptr(), 1, c["X"].data_ptr(), gu.data_ptr(), c["W_gu"].data_ptr(),
            c["W_d"].data_ptr(), T, H, I, *[None if o is None else o.data_ptr() for o in out],
            ws.data_ptr(), ws.numel(), None, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        # alone, a product may be split along k in another way
        close = (out[i].double() - want[i].double()).abs()
        size = want[i].double().abs() + want[i].double().abs().mean()
        assert (close <= 2 * U[torch.bfloat16] * size).all()


@pytest.mark.parametrize("T,H,I", [(70001, 64, 72), (2, 65536, 16), (20, 65536, 16),
                                   (200, 65536, 16), (3, 16, 65536), (130, 16, 65536)])
def test_ffn_long_in_one_dimension(T, H, I):
    dtype = torch.bfloat16
    c = ffn_case(T, H, I)
    Y, gu = moe.gated_ffn_forward(c["X"], c["W_gu"], c["W_d"], residual=c["R"], save_gu=True)
    Yr, terms, gur, gterms, _ = ffn_ref(c["X"], c["W_gu"], c["W_d"], c["R"])
    near(gu, gur, gterms, dtype, 0, "gu")
    near(Y, Yr, terms, dtype, 1.5, "Y")
    dX, dWgu, dWd = moe.gated_ffn_backward(c["dY"], c["X"], gu, c["W_gu"], c["W_d"])
    ga, up = gu.double().chunk(2, 1)
    sg = torch.sigmoid(ga)
    dh = c["dY"].double() @ c["W_d"].double()
    dhs = c["dY"].double().abs() @ c["W_d"].double().abs()
    ds = sg * (1 + ga * (1 - sg))
    dgu = torch.cat([dh * up * ds, dh * ga * sg], 1)
    size = dgu.abs() + (ACC / U[dtype]) * torch.cat(
        [dhs * (up * ds).abs(), dhs * (ga * sg).abs()], 1) + TINY[dtype] / U[dtype]
    X, h = c["X"].double(), ga * sg * up
    near(dX, dgu @ c["W_gu"].double(), size @ c["W_gu"].double().abs(), dtype, 1.5, "dX")
    near(dWgu, dgu.t() @ X, size.t() @ X.abs(), dtype, 1.5, "dW_gu")
    near(dWd, c["dY"].double().t() @ h, c["dY"].double().t().abs() @ h.abs(), dtype, 1.5, "dW_d")


@pytest.mark.parametrize("T,H,V", [(70001, 64, 300), (5, 65536, 40), (200, 32768, 300)])
def test_ce_long_in_one_dimension(T, H, V):
    X, W, y, dl = ce_case(T, H, V, torch.bfloat16, 0.3, 9)
    loss, lse = moe.linear_ce_forward(X, W, y)
    rloss, rlse = ce_ref(X, W, y)
    slack = ACC * (X.double().abs() @ W.double().abs().t()).amax(1) + 2.0 ** -19 * (1 + rlse.abs())
    slack = torch.where(y >= 0, slack, 0.0)
    assert ((lse.double() - rlse).abs() <= slack).all()
    assert ((loss.double() - rloss).abs() <= 2 * slack).all()
    dX, dW = moe.linear_ce_backward(dl, X, W, y, lse)
    ref = ce_ref(X, W, y, dl, lse)
    p = ce_ref(X, W, y, torch.ones_like(dl), lse).abs() + 1
    lerr = ACC * (X.double().abs() @ W.double().abs().t()) + 2.0 ** -20 * (
        1 + lse.double().abs())[:, None]
    size = ref.abs() + lerr * p * dl.double().abs()[:, None] / U[torch.bfloat16]
    size = torch.where((y >= 0)[:, None], size, 0.0)
    near(dX, ref @ W.double(), size @ W.double().abs(), torch.bfloat16, 1.01, "dX")
    near(dW, ref.t() @ X.double(), size.t() @ X.double().abs(), torch.bfloat16, 1.01, "dW")


def test_clip_of_nothing_and_limits():
    empty = torch.empty(0, device="cuda")
    assert float(moe.grad_norm_clip([empty, empty[:0]], 1.0)) == 0.0
    for n in (100, 2_000_000):
        t = torch.ones(n, device="cuda")
        assert float(moe.grad_norm_clip([t], math.inf)) == pytest.approx(math.sqrt(n), rel=1e-6)
        assert (t == 1).all()
        moe.grad_norm_clip([t], 0.0)
        assert (t == 0).all()


def test_clip_uses_what_the_list_holds_each_step():
    g = gen(2)
    grads = [randn(g, 4000), randn(g, 70001, dtype=torch.bfloat16)]
    handle = moe.grad_list(grads)
    for step in range(3):
        for t in grads:
            t.normal_(0, 1.0 + step)
        before = [t.clone() for t in grads]
        norm = moe.grad_norm_clip(handle, 1.0)
        ref = math.sqrt(sum(float(t.double().square().sum()) for t in before))
        assert abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref
        for t, b in zip(grads, before):
            u = {torch.float32: 2.0 ** -24, **U}[t.dtype]
            want = b.double() / (ref + 1e-6)
            assert ((t.double() - want).abs() <= (u + 8 * 2.0 ** -24) * want.abs() + 1e-38).all()


# ------------------------------------------------------------- together


def train_step(s):
    """One step of a layer with routed 4-bit experts and a dense expert beside
    them, a head and its loss: every stage's result, the gradients last."""
    r = moe.route_permute(s["logits"], s["k"], True)
    M = s["X"].shape[0] * s["k"]
    h = moe.nf4_grouped_gemm(s["X"], *s["gu4"], r["expert_offsets"], M, gather=r["sorted_rows"],
                             k=s["k"], epilogue="swiglu", out_dtype=torch.float16)
    Yp = moe.nf4_grouped_gemm(h, *s["d4"], r["expert_offsets"], M, out_dtype=torch.float16)
    routed = moe.unpermute_combine(Yp, r["inv_perm"], r["topk_w"])
    Y, gu = moe.gated_ffn_forward(s["X"], s["W_gu"], s["W_d"], residual=routed, save_gu=True)
    loss, lse = moe.linear_ce_forward(Y, s["W"], s["y"])
    dY, dW = moe.linear_ce_backward(s["dloss"], Y, s["W"], s["y"], lse)
    dX, dWgu, dWd = moe.gated_ffn_backward(dY, s["X"], gu, s["W_gu"], s["W_d"])
    dYp, dw = moe.combine_backward(dY.float(), Yp, r["inv_perm"], r["topk_w"])
    raw = [t.clone() for t in (dW, dWgu, dWd)]
    norm = moe.grad_norm_clip([dW, dWgu, dWd], 0.01)
    return {"routed": routed, "Y": Y, "gu": gu, "loss": loss, "lse": lse, "dY": dY, "dX": dX,
            "dYp": dYp, "dw": dw, "raw": raw, "norm": norm, "grads": [dW, dWgu, dWd]}


@pytest.mark.parametrize("T", [6, 48, 200])
def test_a_training_step(T):
    H, I, V, E, k, dtype = 256, 384, 1003, 8, 2, torch.bfloat16
    g = gen(T)
    s = {"k": k, "X": randn(g, T, H, dtype=dtype), "logits": randn(g, T, E),
         "gu4": moe.nf4_quantize(randn(g, E, 512, H, sigma=0.05)),
         "d4": moe.nf4_quantize(randn(g, E, H, 256, sigma=0.05)),
         "W_gu": randn(g, 2 * I, H, dtype=dtype, sigma=H ** -0.5),
         "W_d": randn(g, H, I, dtype=dtype, sigma=I ** -0.5),
         "W": randn(g, V, H, dtype=dtype, sigma=H ** -0.5)}
    y = torch.randint(0, V, (T,), generator=g, device="cuda").int()
    y[::5] = -100
    s["y"], s["dloss"] = y, (y >= 0).float() / (y >= 0).sum()
    r = train_step(s)
    # each stage against the formulas on what it was given
    Yr, terms, gur, gterms, _ = ffn_ref(s["X"], s["W_gu"], s["W_d"], r["routed"])
    near(r["Y"], Yr, terms, dtype, 1.5, "Y")
    near(r["gu"], gur, gterms, dtype, 0, "gu")
    rloss, rlse = ce_ref(r["Y"], s["W"], y)
    slack = ACC * (r["Y"].double().abs() @ s["W"].double().abs().t()).amax(1) + 2.0 ** -19 * (
        1 + rlse.abs())
    slack = torch.where(y >= 0, slack, 0.0)
    assert ((r["lse"].double() - rlse).abs() <= slack).all()
    assert ((r["loss"].double() - rloss).abs() <= 2 * slack).all()
    dl = ce_ref(r["Y"], s["W"], y, s["dloss"], r["lse"])
    lerr = ACC * (r["Y"].double().abs() @ s["W"].double().abs().t()) + 2.0 ** -20 * (
        1 + rlse.abs())[:, None]
    hot = (torch.arange(V, device="cuda")[None, :] == y[:, None]).double()
    scale = s["dloss"].double()[:, None]
    size = dl.abs() + lerr * (dl.abs() + hot * scale) / U[dtype]
    near(r["dY"], dl @ s["W"].double(), size @ s["W"].double().abs(), dtype, 1.01, "dY")
    near(r["raw"][0], dl.t() @ r["Y"].double(), size.t() @ r["Y"].double().abs(), dtype, 1.01, "dW")
    ga, up = r["gu"].double().chunk(2, 1)
    sg = torch.sigmoid(ga)
    dh = r["dY"].double() @ s["W_d"].double()
    dhs = r["dY"].double().abs() @ s["W_d"].double().abs()
    ds = sg * (1 + ga * (1 - sg))
    dgu = torch.cat([dh * up * ds, dh * ga * sg], 1)
    size = dgu.abs() + (ACC / U[dtype]) * torch.cat([dhs * (up * ds).abs(), dhs * (ga * sg).abs()],
                                                    1) + TINY[dtype] / U[dtype]
    X = s["X"].double()
    near(r["dX"], dgu @ s["W_gu"].double(), size @ s["W_gu"].double().abs(), dtype, 1.5, "dX")
    near(r["raw"][1], dgu.t() @ X, size.t() @ X.abs(), dtype, 1.5, "dW_gu")
    h = ga * sg * up
    near(r["raw"][2], r["dY"].double().t() @ h, r["dY"].double().t().abs() @ h.abs(), dtype, 1.5,
         "dW_d")
    assert (r["dY"][y < 0] == 0).all() and torch.isfinite(r["dYp"]).all()
    ref = math.sqrt(sum(float(t.double().square().sum()) for t in r["raw"]))
    assert abs(float(r["norm"]) - ref) <= 6 * 2.0 ** -24 * ref
    for t, b in zip(r["grads"], r["raw"]):
        want = b.double() * min(1.0, 0.01 / (ref + 1e-6))
        assert ((t.double() - want).abs() <= (U[dtype] + 2.0 ** -20) * want.abs() + 1e-38).all()
    # the same step captured, twice on the same bits
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = train_step(s)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(cap[n], r[n]) for n in ("Y", "loss", "lse", "dY", "dX", "norm"))
        assert same(cap["grads"], r["grads"])
