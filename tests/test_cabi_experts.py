"""Host-side checks of the calls around the layout, without a GPU: bad arguments are refused before any CUDA call."""
import ctypes

import pytest

from counting_sort_bucketization_gb300 import binding, build

FAKE = ctypes.c_void_p(1 << 20)         # never dereferenced: every call below fails its checks
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _desc(N=64, K=8, E=16, R=4, A=128):
    return ctypes.byref(binding._CDesc(N, K, E, R, A))


def _size(fn, d):
    n = ctypes.c_size_t(0)
    assert fn(d, ctypes.byref(n)) == 0
    return n.value


def test_gate_workspace_and_refusals(lib):
    d = _desc()
    n = _size(lib.moe_gate_workspace_bytes, d)
    assert n % 256 == 0 and n >= 256
    assert _size(lib.moe_gate_workspace_bytes, _desc(E=1024)) > n
    bad = ctypes.c_size_t(0)
    assert lib.moe_gate_workspace_bytes(_desc(E=2048), ctypes.byref(bad)) == 6
    assert lib.moe_gate_workspace_bytes(_desc(K=0), ctypes.byref(bad)) == 1
    assert lib.moe_gate_workspace_bytes(d, None) == 1
    cfg = ctypes.byref(binding._CGateDesc(0, 0, 1, 1.0, 0.0))
    fwd = lambda logits=FAKE, ld=16, bias=None, idx=FAKE, w=FAKE, cnt=FAKE, mean=FAKE, rt=FAKE, loss=FAKE, ws=FAKE, nb=n, c=cfg: \
        lib.moe_gate_forward(d, c, logits, ld, bias, idx, w, cnt, mean, rt, loss, ws, nb, None)
    for kw in (dict(logits=None), dict(logits=ODD), dict(ld=15), dict(bias=ODD), dict(idx=None), dict(w=None), dict(cnt=None),
               dict(mean=None), dict(rt=None), dict(loss=None), dict(ws=None), dict(ws=ODD), dict(nb=n - 1), dict(c=None)):
        assert fwd(**kw) == 1, kw
    assert fwd(ld=1 << 29) == 6
    bwd = lambda logits=FAKE, ld=16, idx=FAKE, cnt=FAKE, rt=FAKE, dw=None, dl=None, out=FAKE, old=16: \
        lib.moe_gate_backward(d, cfg, logits, ld, idx, cnt, rt, dw, dl, out, old, FAKE, n, None)
    for kw in (dict(logits=None), dict(ld=4), dict(idx=None), dict(cnt=None), dict(rt=None), dict(dw=ODD), dict(out=None),
               dict(out=ODD), dict(old=15)):
        assert bwd(**kw) == 1, kw


def test_quantiser_refusals(lib):
    rows = lambda x=FAKE, r=8, c=128, q=FAKE, sf=FAKE, ld=0: lib.moe_quantize_rows(x, r, c, None, q, sf, ld, None)
    for kw in (dict(x=None), dict(x=ODD), dict(r=-1), dict(c=0), dict(c=24), dict(q=None), dict(q=ODD), dict(sf=None),
               dict(sf=ODD), dict(ld=4), dict(ld=10)):
        assert rows(**kw) == 1, kw
    assert rows(r=1 << 31) == 6 and rows(c=1 << 29) == 6
    sw = lambda w=128, ld=8, x=FAKE: lib.moe_swiglu_quantize(x, 8, w, None, FAKE, FAKE, ld, None)
    assert sw(w=8) == 1 and sw(ld=0) == 1 and sw(ld=6) == 1 and sw(x=None) == 1
    assert lib.moe_swiglu_backward(FAKE, FAKE, 8, 12, None, FAKE, None) == 1
    assert lib.moe_swiglu_backward(FAKE, None, 8, 16, None, FAKE, None) == 1
    assert lib.moe_swiglu_backward(FAKE, FAKE, 8, 16, None, ODD, None) == 1
    d = _desc()
    n = _size(lib.moe_layout_workspace_bytes, d)
    cols = lambda d=d, cap=1000, c=64, off=FAKE, ld=1024, x=FAKE: \
        lib.moe_quantize_cols(d, x, cap, c, off, FAKE, FAKE, ld, FAKE, FAKE, n, None)
    for kw in (dict(c=12), dict(off=None), dict(ld=1000), dict(ld=896), dict(x=None), dict(cap=-1)):
        assert cols(**kw) == 1, kw
    assert cols(d=_desc(A=64)) == 6


def test_expert_product_refusals(lib):
    d = _desc()
    n = _size(lib.moe_layout_workspace_bytes, d)
    gemm = lambda x=FAKE, xs=FAKE, ld=1000, cap=1000, wi=128, w=FAKE, ws=FAKE, wo=64, off=FAKE, cnt=FAKE, out=FAKE, wk=FAKE, nb=n: \
        lib.moe_expert_gemm_fp8(d, x, xs, ld, cap, wi, w, ws, wo, off, cnt, out, wk, nb, None)
    for kw in (dict(x=None), dict(x=ODD), dict(xs=None), dict(ld=996), dict(ld=1002), dict(cap=-1), dict(wi=24), dict(wi=0),
               dict(w=None), dict(w=ODD), dict(ws=None), dict(wo=12), dict(wo=0), dict(off=None), dict(cnt=None), dict(out=None),
               dict(out=ODD), dict(wk=None), dict(nb=n - 1)):
        assert gemm(**kw) == 1, kw
    assert gemm(cap=0) == 0                     # nothing to do, nothing launched
    assert gemm(cap=1 << 31, ld=1 << 31) == 6
    wgrad = lambda d=d, dy=FAKE, ld=1024, cap=1000, wo=64, wi=64, dw=FAKE, fp32=1, acc=0: \
        lib.moe_expert_wgrad_fp8(d, dy, FAKE, FAKE, FAKE, ld, cap, wo, wi, FAKE, FAKE, dw, fp32, acc, FAKE, n, None)
    for kw in (dict(dy=None), dict(dy=ODD), dict(ld=1000), dict(ld=896), dict(wi=12), dict(wo=0), dict(dw=None), dict(dw=ODD),
               dict(fp32=0, acc=1)):
        assert wgrad(**kw) == 1, kw
    assert wgrad(d=_desc(A=16)) == 6
