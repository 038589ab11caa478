"""Every tensor of a call of the norm, its gradient and the combine's gradient must lie on the current device: one on
another is refused before a pointer is taken.  Without a GPU: stand-ins for tensors, and a library that is never reached."""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding

BF16, FP32, INT32, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class Tensor:
    def __init__(self, *shape, dtype=BF16, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device

    is_cuda = True
    device = property(lambda self: f"cuda:{self.index}")
    get_device = lambda self: self.index
    is_contiguous = lambda self: True
    numel = lambda self: self.shape.numel()
    element_size = lambda self: self.dtype.itemsize
    data_ptr = lambda self: 1 << 20


class Reached(Exception):
    pass


class Library:
    def __getattr__(self, name):
        def call(*args):
            raise Reached
        return call


@pytest.fixture(autouse=True)
def _no_gpu(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "load_library", Library)
    monkeypatch.setattr(binding, "_stream", lambda stream: 0)


R, C, N, K, E, H, CAP = 4, 256, 6, 2, 8, 64, 40
DESC = binding.LayoutDesc(N, K, E, 1, 4)
CALLS = {
    "rms_norm": (lambda **kw: binding.rms_norm(**kw), dict(
        x=(R, C), weight=(C,), y=(R, C), q=(R, C, E4M3), sf=(R, 2, FP32), residual=(R, C), residual_out=(R, C), rstd=(R, FP32),
        total_rows=(1, INT32))),
    "rms_norm_backward": (lambda **kw: binding.rms_norm_backward(**kw), dict(
        dy=(R, C), z=(R, C), rstd=(R, FP32), weight=(C,), dz=(R, C), dresidual=(R, C), dx=(R, C), dweight=(C, FP32),
        workspace=(4096, torch.uint8), total_rows=(1, INT32))),
    "combine_backward": (lambda **kw: binding.combine_backward(DESC, **kw), dict(
        dout=(N, H), dst_slot=(N * K, INT32), weights=(N, K, FP32), dy=(CAP, H), workspace=(4096, torch.uint8), expert_out=(CAP, H),
        dweights=(N, K, FP32), expert_offset=(E + 1, INT32), expert_count=(E, INT32))),
}


def tensors(spec, elsewhere=None):
    out = {}
    for name, (*shape, last) in spec.items():
        shape, dtype = (shape, last) if isinstance(last, torch.dtype) else (shape + [last], BF16)
        out[name] = Tensor(*shape, dtype=dtype, device=int(name == elsewhere))
    return out


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, spec) in CALLS.items() for n in spec])
def test_one_tensor_elsewhere(call, name):
    run, spec = CALLS[call]
    with pytest.raises(ValueError, match=f"{name} is on cuda:1, the current device is cuda:0"):
        run(**tensors(spec, name))


@pytest.mark.parametrize("call", CALLS)
def test_all_here(call):
    run, spec = CALLS[call]
    with pytest.raises(Reached):
        run(**tensors(spec))


@pytest.mark.parametrize("call", CALLS)
def test_all_elsewhere(call, monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    run, spec = CALLS[call]
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        run(**tensors(spec))
