"""Host-side check of the norm's eps: values beside which the squares that fp32 loses would count are refused.

A row's sum of squares loses what lies below 2^-149, and where it overflows it is taken of scaled values without eps."""
import ctypes

import pytest

from counting_sort_bucketization_gb300 import binding, build

FAKE = [ctypes.c_void_p((i + 1) << 26) for i in range(8)]         # never dereferenced: every call below fails its checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("eps", [1e-45, 1e-40, 2.0 ** -127, 2.0 ** 89, 1e30, 3e38])
def test_eps_out_of_range(lib, eps):
    d = ctypes.byref(binding._CNormDesc(4, 256, eps, 0, 0))
    x, w, y = FAKE[:3]
    assert lib.moe_rms_norm(d, x, None, w, None, None, y, None, None, 0, None, None) == 1
    assert lib.moe_rms_norm_workspace_bytes(d, ctypes.byref(ctypes.c_size_t(0))) == 1


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-6, 2.0 ** 88])
def test_eps_in_range(lib, eps):
    n = ctypes.c_size_t(0)
    assert lib.moe_rms_norm_workspace_bytes(ctypes.byref(binding._CNormDesc(4, 256, eps, 0, 0)), ctypes.byref(n)) == 0
