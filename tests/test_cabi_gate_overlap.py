"""Where the gate's gradient may lie in relation to the logits: the host checks, without a GPU.

A call that passes its checks reaches a launch, which no GPU answers with MOE_ERR_CUDA (2); on a machine with a GPU only the
refusals are tried, since the addresses are not real.  Such calls are made in a thread of their own, which keeps the CUDA
error they leave."""
import concurrent.futures
import ctypes

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

BASE = 1 << 20


@pytest.fixture(scope="module")
def call():
    build.build()
    lib = binding.load_library()
    d = ctypes.byref(binding._CDesc(64, 8, 16, 1, 1))
    n = ctypes.c_size_t(0)
    assert lib.moe_gate_workspace_bytes(d, ctypes.byref(n)) == 0

    def f(logits, stride, dlogits, dstride, bf16=0):
        cfg = ctypes.byref(binding._CGateDesc(bf16, 0, 1, 1.0, 0.0))
        at = ctypes.c_void_p
        return lib.moe_gate_backward(d, cfg, at(logits), stride, at(BASE), at(BASE), at(BASE), None, None, at(dlogits), dstride,
                                     at(BASE), n.value, None)
    return f


@pytest.mark.parametrize("bf16,size", [(0, 4), (1, 2)])
def test_overlapping_rows_are_refused(call, bf16, size):
    at = 1 << 24
    for stride, other, dstride in [(16, at, 20), (20, at, 16),             # same base, other stride
                                   (16, at + size, 16), (16, at - size, 16), (16, at + 63 * 16 * size, 16),
                                   (16, at - 63 * 16 * size - 15 * size, 16),
                                   (40, at + 15 * size, 40), (40, at + 25 * size, 40), (40, at - 15 * size, 40),
                                   (40, at + (40 * 7 + 25) * size, 40),    # from the middle of a row's gap into the next row
                                   (40, at + 16 * size, 41)]:
        assert call(at, stride, other, dstride, bf16) == 1, (stride, other - at, dstride)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
@pytest.mark.parametrize("bf16,size", [(0, 4), (1, 2)])
def test_the_same_rows_and_separate_rows_are_taken(call, bf16, size):
    at = 1 << 24
    for stride, other, dstride in [(16, at, 16), (40, at, 40), (16, at + 64 * 16 * size, 16), (16, at - 64 * 16 * size, 16),
                                   (16, at + 64 * 16 * size, 99), (40, at + 16 * size, 40), (40, at + 24 * size, 40),
                                   (40, at - 16 * size, 40), (32, at + (32 * 9 + 16) * size, 32),
                                   (40, at + (63 * 40 + 16) * size, 41)]:
        with concurrent.futures.ThreadPoolExecutor(1) as thread:
            assert thread.submit(call, at, stride, other, dstride, bf16).result() == 2, (stride, other - at, dstride)
