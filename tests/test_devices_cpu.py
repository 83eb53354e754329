"""The norms and the gradient calls take tensors of the current device only: a kernel would fault on another's.  The
tensors, the devices and the library are made up here."""
import types

import pytest
import torch

import serving_router_gate_gb300 as moe

T, H, k, E = 4, 64, 2, 8


class Tensor:
    """What the binding looks at of a tensor, on CUDA device dev."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.dev = dtype, torch.Size(shape), 0

    @property
    def device(self):
        return f"cuda:{self.dev}"

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def numel(self):
        return 1 << 30


def _bf(*s):
    return Tensor(torch.bfloat16, *s)


def _f(*s):
    return Tensor(torch.float32, *s)


def _i(*s):
    return Tensor(torch.int32, *s)


def _ws():
    return Tensor(torch.uint8, 1 << 30)


CALLS = {
    "moe_add_rmsnorm": lambda: [_bf(T, H), _f(T, H), _bf(H), 1e-5, _f(T, H), _bf(T, H), Tensor(torch.uint8, T, H), _f(T)],
    "moe_add_layernorm": lambda: [_bf(T, H), _bf(T, H), _bf(H), _bf(H), 1e-5, _bf(T, H), _bf(T, H),
                                  Tensor(torch.uint8, T, H), _f(T)],
    "moe_add_rmsnorm_bwd": lambda: [_bf(T, H), _f(T, H), _bf(H), 1e-5, _f(T, H), _f(T, H), _bf(T, H), _f(H), _ws()],
    "moe_add_layernorm_bwd": lambda: [_bf(T, H), _bf(T, H), _bf(H), 1e-5, _bf(T, H), _bf(T, H), _bf(T, H), _f(H), _f(H),
                                      _ws()],
    "moe_finalize_bwd": lambda: [_bf(T, H), _bf(T * k, H), _i(T, k), _f(T, k), _bf(T, H), _bf(T, H), _bf(H), _bf(T * k, H),
                                 _f(T, k), _bf(T, H), _f(T), _f(H), _ws()],
    "moe_permute_bwd": lambda: [_bf(T * k, H), _i(T, k), _f(T, k), _bf(T, H), _f(T, H), _f(T), _bf(H), _bf(T, H), _f(T, k),
                                _ws()],
    "moe_route_bwd": lambda: [_i(T, k), _f(T, k), _f(T, k), _f(T, E), False, _f(T, E), _ws()],
}


@pytest.fixture
def made(monkeypatch):
    """The library's calls, by name; the current device is 0."""
    names = []
    lib = types.SimpleNamespace(**{n: (lambda *a, _n=n: names.append(_n) or 0) for n in CALLS})
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return names


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_is_on_the_current_device(made, name):
    getattr(moe, name)(*CALLS[name]())
    assert made == [name]
    del made[:]
    n = 0
    for i, t in enumerate(CALLS[name]()):
        if not isinstance(t, Tensor):
            continue
        args = CALLS[name]()
        args[i].dev = 1
        with pytest.raises(ValueError, match="cuda:1"):
            getattr(moe, name)(*args)
        n += 1
    assert n >= 6 and made == []


@pytest.mark.parametrize("name", CALLS)
def test_all_tensors_on_another_device_are_refused(made, name):
    for stream in (None, types.SimpleNamespace(cuda_stream=5)):
        args = CALLS[name]()
        for t in args:
            if isinstance(t, Tensor):
                t.dev = 1
        with pytest.raises(ValueError, match="current device"):
            getattr(moe, name)(*args, stream=stream)
    assert made == []
