"""Host-side checks of the combine's gradient that need no GPU: the layout's arrays, where they lie and how."""
import ctypes

import pytest

from counting_sort_bucketization_gb300 import binding, build

FAKE = [ctypes.c_void_p((i + 1) << 26) for i in range(9)]         # apart, never dereferenced: every call below fails its checks
NAMES = ("dout", "slot", "w", "y", "dy", "dw", "off", "cnt", "ws")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def backward(lib, zero_pad=1, **kw):
    d = ctypes.byref(binding._CDesc(64, 8, 16, 4, 128))
    n = ctypes.c_size_t(0)
    assert lib.moe_layout_workspace_bytes(d, ctypes.byref(n)) == 0
    a = dict(zip(NAMES, FAKE), **kw)
    return lib.moe_combine_backward(d, a["dout"], 64, a["slot"], a["w"], a["y"], a["dy"], 1000, a["dw"], a["off"], a["cnt"], zero_pad,
                                    a["ws"], n.value, None)


def at(name, by=0):
    return ctypes.c_void_p(FAKE[NAMES.index(name)].value + by)


@pytest.mark.parametrize("name", ["slot", "off", "cnt"])
def test_words_off_their_boundary(lib, name):
    assert backward(lib, **{name: at(name, 2)}) == 1


@pytest.mark.parametrize("name", ["off", "cnt"])
@pytest.mark.parametrize("over,by", [("dy", 0), ("dy", 128 * 1000 - 4), ("dw", 0), ("dw", 4 * 64 * 8 - 4)])
def test_outputs_over_the_layouts_arrays(lib, name, over, by):
    """The first and the last word of an output."""
    assert backward(lib, **{name: at(over, by)}) == 1
