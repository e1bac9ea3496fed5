"""Workspace sizes of the dense training-side operators, on the host: the
binding asks for them per device."""

import contextlib

import pytest
import torch

from bit_mixture_experts_route_b200 import _lib

SIZES = ["gated_ffn_forward", "gated_ffn_backward", "linear_ce_forward", "linear_ce_backward"]


class _TwoDevices:
    """A library whose sizes depend on the current device, as on GPUs with
    different numbers of SMs."""

    def __init__(self):
        self.current = 0
        self.asked = []

    def __getattr__(self, name):
        def f(T, H, I, out):
            self.asked.append((self.current, name))
            out._obj.value = 1000 * (self.current + 1)
            return 0
        return f


@pytest.fixture
def lib(monkeypatch):
    two = _TwoDevices()

    @contextlib.contextmanager
    def device(d):
        before, two.current = two.current, torch.device(d).index
        yield
        two.current = before

    _lib._size_on.cache_clear()
    monkeypatch.setattr(_lib, "_lib", two)
    monkeypatch.setattr(_lib, "_current_device", lambda: two.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    yield two
    _lib._size_on.cache_clear()


@pytest.mark.parametrize("op", SIZES)
def test_a_size_is_the_current_devices(lib, op):
    size = getattr(_lib, f"{op}_workspace_size")
    assert size(4, 64, 64) == 1000
    lib.current = 1
    assert size(4, 64, 64) == 2000
    lib.current = 0
    assert size(4, 64, 64) == 1000
    assert len(lib.asked) == 2                      # each device was asked once


@pytest.mark.parametrize("op", SIZES)
def test_a_size_for_another_device(lib, op):
    size = getattr(_lib, f"{op}_workspace_size")
    assert size(4, 64, 64, device="cuda:1") == 2000
    assert size(4, 64, 64, device=torch.device("cuda", 0)) == 1000
    assert size(4, 64, 64, "cuda") == 1000 and lib.current == 0


def test_a_size_without_a_device():
    # the library is the built one; no GPU is needed to ask
    assert _lib.linear_ce_backward_workspace_size(4, 64, 64) > 0


@pytest.mark.parametrize("T,H,V", [(4096, 2048, 151936), (5000, 3840, 19000), (17000, 4096, 8000),
                                   (65536, 4096, 151936), (1 << 20, 4096, 32000), (300, 64, 70),
                                   (129, 16384, 1 << 20)])
def test_room_of_the_cross_entropy_backward(T, H, V):
    # the rows once more, a piece of dl, dX's sums, and what there is per row
    rows, wide, mb256 = (T + 255) // 256 * 256, (H + 255) // 256 * 256, 256 << 20
    most = 2 * rows * H + max(mb256, 512 * rows) + max(mb256, 4 * rows * wide) + 64 * rows + 65536
    assert _lib.linear_ce_backward_workspace_size(T, H, V) <= most
