"""What the dense training-side operators refuse, on the host: the C entry points'
statuses (all found before anything touches a device) and the binding's checks
(CPU tensors presented as device tensors; the library is a recorder)."""

import ctypes
import math

import pytest
import torch

from bit_mixture_experts_route_b200 import _lib

OK, INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = range(5)
P = 1 << 20          # an aligned address that is never read
BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def c():
    return _lib.load()


def size(c, fn, *args):
    n = ctypes.c_size_t()
    return getattr(c, fn)(*args, ctypes.byref(n)), n.value


SHAPES = ["moe_gated_ffn_forward_workspace_size", "moe_gated_ffn_backward_workspace_size",
          "moe_linear_ce_forward_workspace_size", "moe_linear_ce_backward_workspace_size"]


@pytest.mark.parametrize("fn", SHAPES)
def test_shapes_that_are_refused(c, fn):
    assert size(c, fn, 4, 64, 64)[0] == OK
    assert size(c, fn, -1, 64, 64)[0] == INVALID
    assert size(c, fn, 4, 0, 64)[0] == INVALID
    assert size(c, fn, 4, 64, 0)[0] == INVALID
    assert size(c, fn, 4, 60, 64)[0] == UNSUPPORTED
    assert size(c, fn, (1 << 20) + 1, 64, 64)[0] == UNSUPPORTED
    assert size(c, fn, 4, (1 << 20) + 8, 64)[0] == UNSUPPORTED
    assert getattr(c, fn)(4, 64, 64, None) == INVALID
    if "ffn" in fn:
        assert size(c, fn, 4, 64, 60)[0] == UNSUPPORTED
    else:
        assert size(c, fn, 4, 64, 61)[0] == OK
        assert size(c, fn, 4, 64, (1 << 24) + 1)[0] == UNSUPPORTED


def ffn_fwd(c, X=P, dt=BF16, Wgu=P, Wd=P, T=4, H=64, I=64, res=None, Y=P, gu=None, ws=P,
            n=1 << 30):
    return c.moe_gated_ffn_forward(X, dt, Wgu, Wd, T, H, I, res, Y, gu, ws, n, None, None)


def test_ffn_forward_statuses(c):
    for bad in (dict(X=None), dict(Wgu=None), dict(Wd=None), dict(Y=None), dict(dt=F32),
                dict(dt=3)):
        assert ffn_fwd(c, **bad) == INVALID
    for name in ("X", "Wgu", "Wd", "Y", "gu", "res", "ws"):
        assert ffn_fwd(c, **{name: P + 8}) == MISALIGNED
    assert ffn_fwd(c, ws=None) == WORKSPACE
    need = size(c, "moe_gated_ffn_forward_workspace_size", 4, 64, 64)[1]
    assert ffn_fwd(c, n=need - 1) == WORKSPACE
    assert ffn_fwd(c, T=0, X=None, Y=None, ws=None) == OK


def test_ffn_backward_statuses(c):
    def call(dY=P, dt=BF16, X=P, gu=P, Wgu=P, Wd=P, dX=P, dWgu=P, dWd=P, ws=P, n=1 << 30):
        return c.moe_gated_ffn_backward(dY, dt, X, gu, Wgu, Wd, 4, 64, 64, dX, dWgu, dWd, ws, n,
                                        None, None)
    for bad in (dict(dY=None), dict(X=None), dict(gu=None), dict(Wgu=None), dict(Wd=None),
                dict(dt=F32), dict(dX=None, dWgu=None, dWd=None)):
        assert call(**bad) == INVALID
    for name in ("dY", "X", "gu", "Wgu", "Wd", "dX", "dWgu", "dWd", "ws"):
        assert call(**{name: P + 2}) == MISALIGNED
    need = size(c, "moe_gated_ffn_backward_workspace_size", 4, 64, 64)[1]
    assert call(n=need - 1) == WORKSPACE


def test_linear_ce_statuses(c):
    def fwd(X=P, dt=BF16, W=P, y=P, loss=P, lse=P, ws=P, n=1 << 30, T=4):
        return c.moe_linear_ce_forward(X, dt, W, y, T, 64, 101, -100, loss, lse, ws, n, None, None)

    def bwd(dl=P, X=P, dt=BF16, W=P, y=P, lse=P, dX=P, dW=P, ws=P, n=1 << 30):
        return c.moe_linear_ce_backward(dl, X, dt, W, y, lse, 4, 64, 101, -100, dX, dW, ws, n,
                                        None, None)
    for bad in (dict(X=None), dict(W=None), dict(y=None), dict(loss=None), dict(lse=None),
                dict(dt=F32)):
        assert fwd(**bad) == INVALID
    for bad in (dict(dl=None), dict(X=None), dict(W=None), dict(y=None), dict(lse=None),
                dict(dt=F32), dict(dX=None, dW=None)):
        assert bwd(**bad) == INVALID
    for name in ("X", "W", "y", "loss", "lse", "ws"):
        assert fwd(**{name: P + 4}) == MISALIGNED
    for name in ("dl", "X", "W", "y", "lse", "dX", "dW", "ws"):
        assert bwd(**{name: P + 4}) == MISALIGNED
    for call, fn in ((fwd, SHAPES[2]), (bwd, SHAPES[3])):
        assert call(n=size(c, fn, 4, 64, 101)[1] - 1) == WORKSPACE
    assert fwd(T=0, X=None, y=None, loss=None, lse=None, ws=None) == OK


def test_grad_norm_clip_statuses(c):
    def call(ptrs=(P,), numel=(10,), dts=(F32,), max_norm=1.0, outs=None, norm=P, ws=P,
             nbytes=1 << 30):
        n = len(ptrs)
        arr = (ctypes.c_void_p * n)(*ptrs)
        out = None if outs is None else (ctypes.c_void_p * n)(*outs)
        return c.moe_grad_norm_clip(arr, (ctypes.c_int64 * n)(*numel), (ctypes.c_int * n)(*dts), n,
                                    max_norm, out, norm, ws, nbytes, None, None)
    for bad in (dict(norm=None), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(dts=(7,)),
                dict(numel=(-1,)), dict(ptrs=(None,)), dict(outs=(None,))):
        assert call(**bad) == INVALID
    assert call(ptrs=(P + 2,)) == MISALIGNED           # fp32 at a 2-byte boundary
    assert call(ptrs=(P + 1,), dts=(BF16,)) == MISALIGNED
    assert call(outs=(P + 2,)) == MISALIGNED
    assert call(norm=P + 2) == MISALIGNED and call(ws=P + 8) == MISALIGNED
    assert call(numel=((1 << 42) + 1,)) == UNSUPPORTED
    assert call(ptrs=(P, P), numel=(1 << 42, 1), dts=(F32, F32)) == UNSUPPORTED
    assert call(nbytes=16) == WORKSPACE
    assert c.moe_grad_norm_clip(None, None, None, 1, 1.0, None, P, P, 1 << 30, None,
                                None) == INVALID


# ------------------------------------------------------------- the binding


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args):
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def lib(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    monkeypatch.setattr(_lib, "_lib", rec)
    monkeypatch.setattr(_lib, "_stream", lambda device=None: None)
    monkeypatch.setattr(_lib, "_size", lambda fn, *a: 4096)
    return rec


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_ffn(lib):
    X, Wgu, Wd = b16(4, 64), b16(96, 64), b16(64, 48)
    gu, dY = b16(4, 96), b16(4, 64)
    _lib.gated_ffn_forward(X, Wgu, Wd)
    Y, kept = _lib.gated_ffn_forward(X, Wgu, Wd, save_gu=True)
    assert Y.shape == (4, 64) and kept.shape == (4, 96)
    _lib.gated_ffn_backward(dY, X, gu, Wgu, Wd)
    assert lib.calls == ["moe_gated_ffn_forward"] * 2 + ["moe_gated_ffn_backward"]
    n = len(lib.calls)
    bad = [lambda: _lib.gated_ffn_forward(X.float(), Wgu, Wd),
           lambda: _lib.gated_ffn_forward(X[0], Wgu, Wd),
           lambda: _lib.gated_ffn_forward(X, Wgu.half(), Wd),
           lambda: _lib.gated_ffn_forward(X, Wgu[:-1], Wd),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd.t()),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd.t().contiguous()),
           lambda: _lib.gated_ffn_forward(b16(4, 128)[:, ::2], Wgu, Wd),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, residual=b16(4, 64)),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, residual=torch.zeros(1, 64)),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, out=b16(3, 64)),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, gu=b16(4, 48)),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, workspace=torch.zeros(9, dtype=torch.uint8)),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd, dev_err=torch.zeros(1)),
           lambda: _lib.gated_ffn_forward(None, Wgu, Wd),
           lambda: _lib.gated_ffn_forward(X, None, Wd),
           lambda: _lib.gated_ffn_forward(X, Wgu, None),
           lambda: _lib.gated_ffn_forward(X, Wgu, Wd[0]),
           lambda: _lib.gated_ffn_backward(None, X, gu, Wgu, Wd),
           lambda: _lib.gated_ffn_backward(dY, X, None, Wgu, Wd),
           lambda: _lib.gated_ffn_backward(dY[:3], X, gu, Wgu, Wd),
           lambda: _lib.gated_ffn_backward(dY, X, gu[:, :48], Wgu, Wd),
           lambda: _lib.gated_ffn_backward(dY, X, gu, Wgu, Wd, need_dx=False, need_dw=False)]
    for f in bad:
        with pytest.raises(_lib.MoEError):
            f()
    assert len(lib.calls) == n


def test_binding_linear_ce(lib):
    X, W, y = b16(4, 64), b16(101, 64), torch.zeros(4, dtype=torch.int32)
    f32 = torch.zeros(4)
    loss, lse = _lib.linear_ce_forward(X, W, y)
    assert loss.shape == lse.shape == (4,)
    assert _lib.linear_ce_backward(f32, X, W, y, f32, need_dx=False)[0] is None
    n = len(lib.calls)
    bad = [lambda: _lib.linear_ce_forward(X, W, y.long()),
           lambda: _lib.linear_ce_forward(X, W, y[:3]),
           lambda: _lib.linear_ce_forward(X, W.half(), y),
           lambda: _lib.linear_ce_forward(X, b16(101, 72), y),
           lambda: _lib.linear_ce_forward(X, b16(202, 64)[::2], y),
           lambda: _lib.linear_ce_forward(X, W, None),
           lambda: _lib.linear_ce_forward(X, W, y, ignore_index=1 << 40),
           lambda: _lib.linear_ce_backward(f32, X, W, y, f32, ignore_index=-(1 << 31) - 1),
           lambda: _lib.linear_ce_forward(X, None, y),
           lambda: _lib.linear_ce_backward(None, X, W, y, f32),
           lambda: _lib.linear_ce_backward(f32, X, W, y, None),
           lambda: _lib.linear_ce_backward(f32[:2], X, W, y, f32),
           lambda: _lib.linear_ce_backward(f32, X, W, y, f32.double()),
           lambda: _lib.linear_ce_backward(f32, X, W, y, f32, need_dx=False, need_dw=False)]
    for f in bad:
        with pytest.raises(_lib.MoEError):
            f()
    assert len(lib.calls) == n


def test_binding_grad_list(lib):
    flat, out = torch.zeros(100), torch.zeros(100)
    _lib.grad_norm_clip(_lib.grad_list([flat[:40], flat[40:]]), 1.0)
    _lib.grad_list([flat[:40], flat[20:]], [out[:40], torch.zeros(80)])  # only read: may overlap
    _lib.grad_list([flat[:40], flat[40:]], [flat[:40], out[40:]])        # in place and elsewhere
    _lib.grad_list([flat[:0], flat[:0], flat])
    bad = [lambda: _lib.grad_list([]),
           lambda: _lib.grad_list([flat, flat]),
           lambda: _lib.grad_list([flat[:40], flat[39:]]),
           lambda: _lib.grad_list([flat[:40], flat[40:]], [out[:40], out[30:90]]),
           lambda: _lib.grad_list([flat[:40], flat[40:80]], [flat[1:41], out[:40]]),
           lambda: _lib.grad_list([flat[:40], flat[40:80]], [flat[40:80], out[:40]]),
           lambda: _lib.grad_list([flat], [out, out]),
           lambda: _lib.grad_list([flat], [out[:99]]),
           lambda: _lib.grad_list([flat], [out.half()]),
           lambda: _lib.grad_list([flat.double()]),
           lambda: _lib.grad_list([flat[::2]]),
           lambda: _lib.grad_norm_clip([flat], 1.0, norm=torch.zeros(2))]
    for i, f in enumerate(bad):
        with pytest.raises(_lib.MoEError):
            f()
            print("not refused:", i)
