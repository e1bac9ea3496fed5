"""GPU tests of the dense training-side operators right behind the launch that
writes what they read (no host wait in between, inputs that change from pass to
pass): clipping behind the weight gradients and behind an earlier clipping, and
the feed-forward block on rows that the launch before has gathered.  The results
have to have the bits of the same calls with a wait between them."""

import math

import pytest
import torch

from test_gpu_zz_dense_train import U, gen, randn

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("bit_mixture_experts_route_b200")

BF16 = torch.bfloat16


def backward_into(flat, dY, X, gu, Wgu, Wd, ws):
    """dW_gu and dW_d into one flat buffer (through the C call)."""
    T, H, I = X.shape[0], X.shape[1], Wd.shape[1]
    assert flat.numel() >= 3 * H * I
    st = moe.load().moe_gated_ffn_backward(
        dY.data_ptr(), 1, X.data_ptr(), gu.data_ptr(), Wgu.data_ptr(), Wd.data_ptr(), T, H, I,
        None, flat.data_ptr(), flat.data_ptr() + 2 * 2 * I * H, ws.data_ptr(), ws.numel(), None,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0


def odd_views(flat, n):
    """n packed parts of uneven lengths, starting one element into the buffer."""
    cuts = [1 + (flat.numel() - 2) * i // n + (i * 7 % 5 if 0 < i < n else 0) for i in range(n + 1)]
    return [flat[a:b] for a, b in zip(cuts, cuts[1:])]


# elements 3 H I: one launch of a cluster; two launches; tables for more than 1024 tensors
@pytest.mark.parametrize("T,H,I,parts", [(16, 64, 72, 5), (60, 312, 1024, 9), (200, 512, 1024, 300),
                                         (200, 256, 640, 1100)])
def test_clipping_behind_the_weight_gradients(T, H, I, parts):
    g = gen(T + H + I)
    Wgu = randn(g, 2 * I, H, dtype=BF16, sigma=H ** -0.5)
    Wd = randn(g, H, I, dtype=BF16, sigma=I ** -0.5)
    flat = torch.zeros(3 * H * I + 8, dtype=BF16, device="cuda")
    views = odd_views(flat, parts)
    grads = moe.grad_list(views)
    ws = torch.empty(moe.gated_ffn_backward_workspace_size(T, H, I), dtype=torch.uint8,
                     device="cuda")
    steps = []
    for i in range(8):
        X, dY = randn(g, T, H, dtype=BF16), randn(g, T, H, dtype=BF16, sigma=2.0 ** (i % 3))
        gu = (X.float() @ Wgu.float().t()).to(BF16)
        steps.append((dY, X, gu))
    want = []
    for s in steps:
        backward_into(flat, *s, Wgu, Wd, ws)
        torch.cuda.synchronize()
        raw = flat.clone()
        torch.cuda.synchronize()
        norm = moe.grad_norm_clip(grads, 0.5)
        torch.cuda.synchronize()
        once = flat.clone()
        torch.cuda.synchronize()
        norm2 = moe.grad_norm_clip(grads, 0.25)
        torch.cuda.synchronize()
        want.append((norm, once, norm2, flat.clone()))
        # the clipping itself, in 64 bits
        part = torch.cat([raw[v.storage_offset():v.storage_offset() + v.numel()] for v in views])
        ref = math.sqrt(float(part.double().square().sum()))
        assert ref > 1.0 and abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref
        lo = views[0].storage_offset()
        hi = lo + part.numel()
        scaled = part.double() * (0.5 / (ref + 1e-6))
        assert ((once[lo:hi].double() - scaled).abs()
                <= (U[BF16] + 8 * 2.0 ** -24) * scaled.abs() + 2.0 ** -134).all()
        assert torch.equal(once[:lo], raw[:lo]) and torch.equal(once[hi:], raw[hi:])
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s in steps:
            backward_into(flat, *s, Wgu, Wd, ws)
            norm = moe.grad_norm_clip(grads, 0.5)     # behind the gradients
            norm2 = moe.grad_norm_clip(grads, 0.25)   # behind a clipping
            got.append((norm, norm2, flat.clone()))
        torch.cuda.synchronize()
        for (norm, norm2, end), (wn, _, wn2, wend) in zip(got, want):
            assert torch.equal(norm, wn) and torch.equal(norm2, wn2) and torch.equal(end, wend)


# one size per kernel that the first product may take
@pytest.mark.parametrize("T,H,I", [(3, 256, 520), (12, 256, 520), (40, 256, 520), (300, 256, 520)])
def test_block_behind_the_gathering_of_its_inputs(T, H, I):
    g = gen(T + H + I)
    n = 4
    # rows of several matrices one under another; the launch before gathers one of them
    all_x, all_dy = randn(g, n * T, H, dtype=torch.float16), randn(g, n * T, H, dtype=torch.float16)
    all_gu = randn(g, n * T, 2 * I, dtype=torch.float16)
    all_w = randn(g, n * 2 * I, H, dtype=torch.float16, sigma=H ** -0.5)
    Wd = randn(g, H, I, dtype=torch.float16, sigma=I ** -0.5)
    X, dY = torch.empty_like(all_x[:T]), torch.empty_like(all_dy[:T])
    gu, W = torch.empty_like(all_gu[:T]), torch.empty_like(all_w[:2 * I])

    def rows(i, m):
        return torch.arange(i * m, (i + 1) * m, dtype=torch.int32, device="cuda")

    def one(i, wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        out = []
        moe.permute_rows(all_x, picks[i][0], 1, out=X)
        moe.permute_rows(all_w, picks[i][1], 1, out=W)      # the weights last
        pause()
        out.append(moe.gated_ffn_forward(X, W, Wd))
        moe.permute_rows(all_dy, picks[i][0], 1, out=dY)
        moe.permute_rows(all_gu, picks[i][0], 1, out=gu)    # gate and up last
        pause()
        out += moe.gated_ffn_backward(dY, X, gu, W, Wd)
        pause()
        return out

    picks = [(rows(i, T), rows(i, 2 * I)) for i in range(n)]
    want = [one(i, True) for i in range(n)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [one(i, False) for i in range(n)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("dtype", [torch.float32, BF16, torch.float16])
@pytest.mark.parametrize("n", [777, 50001, 3_000_017])
def test_norm_repeats_at_equal_offsets(n, dtype):
    # the order of the sum follows from the sizes and the offsets modulo 16 bytes
    g = gen(n)
    per = 16 // dtype.itemsize
    values = randn(g, n, dtype=dtype, sigma=0.1)
    ref = math.sqrt(float(values.double().square().sum()))
    for off in (0, 1, per - 1):
        seen = []
        for base in (0, 3 * per, 40 * per):  # other addresses, the same offset
            flat = torch.zeros(n + 50 * per, dtype=dtype, device="cuda")
            t = flat[base + off:base + off + n]
            t.copy_(values)
            norm = moe.grad_norm_clip([t], 0.5 * ref)
            assert abs(float(norm) - ref) <= 6 * 2.0 ** -24 * ref
            seen.append((norm, t.clone()))
        assert all(torch.equal(a, seen[0][0]) and torch.equal(b, seen[0][1]) for a, b in seen)
