"""Host-side checks of the norm, the routing by groups and the combine's gradient, without a GPU: bad arguments are
refused before any CUDA call.  And their plain gradients against differences in 64 bits."""
import ctypes

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

MB = 1 << 20
FAKE = [ctypes.c_void_p((i + 1) * 64 * MB) for i in range(12)]    # apart, never dereferenced: every call below fails its checks


def odd(p, by=2):
    return ctypes.c_void_p(p.value + by)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def norm_desc(rows=64, cols=256, eps=1e-6, fp32=0, wfp32=0):
    return ctypes.byref(binding._CNormDesc(rows, cols, eps, fp32, wfp32))


def test_norm_refusals(lib):
    X, RES, W, TOTAL, ROUT, Y, Q, SF, RSTD = FAKE[:9]

    def fwd(d=None, x=X, res=RES, w=W, total=None, rout=ROUT, y=Y, q=Q, sf=SF, ld=0, rstd=RSTD, **kw):
        return lib.moe_rms_norm(norm_desc(**kw) if d is None else d, x, res, w, total, rout, y, q, sf, ld, rstd, None)

    for kw in (dict(rows=-1), dict(cols=0), dict(cols=24), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(x=None), dict(x=odd(X)), dict(res=None), dict(res=odd(RES)), dict(rout=None),
               dict(rout=odd(ROUT)), dict(res=None, rout=None, fp32=1), dict(w=None), dict(w=odd(W)), dict(y=None, q=None, sf=None),
               dict(y=odd(Y)), dict(q=odd(Q)), dict(q=None), dict(sf=None), dict(sf=odd(SF)), dict(ld=4), dict(ld=66),
               dict(rstd=odd(RSTD)), dict(total=odd(TOTAL))):
        assert fwd(**kw) == 1, kw
    assert fwd(d=ctypes.POINTER(binding._CNormDesc)()) == 1
    assert fwd(rows=1 << 31) == 6 and fwd(cols=32768 + 16) == 6
    # overlaps: only whole, of the same type
    shift = lambda p: odd(p, 64)
    for kw in (dict(y=ROUT), dict(q=X), dict(q=ROUT), dict(y=shift(X)), dict(rout=shift(RES)), dict(rout=X, fp32=1), dict(y=RES, fp32=1),
               dict(y=W), dict(rstd=W), dict(sf=X), dict(rstd=SF), dict(q=shift(Y)), dict(total=Y)):
        assert fwd(**kw) == 1, kw


def test_norm_backward_refusals(lib):
    DY, Z, RSTD, W, DRES, TOTAL, DZ, DX, DW, WS = FAKE[:10]
    n = ctypes.c_size_t(0)
    assert lib.moe_rms_norm_workspace_bytes(norm_desc(), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.moe_rms_norm_workspace_bytes(norm_desc(), None) == 1
    assert lib.moe_rms_norm_workspace_bytes(norm_desc(cols=40), ctypes.byref(ctypes.c_size_t(0))) == 1

    def bwd(dy=DY, z=Z, rstd=RSTD, w=W, dres=DRES, total=None, dz=DZ, dx=None, dw=DW, ws=WS, nb=n.value, **kw):
        return lib.moe_rms_norm_backward(norm_desc(**kw), dy, z, rstd, w, dres, total, dz, dx, dw, 0, ws, nb, None)

    for kw in (dict(dy=None), dict(dy=odd(DY)), dict(z=None), dict(z=odd(Z)), dict(rstd=None), dict(rstd=odd(RSTD)), dict(w=None),
               dict(dres=odd(DRES)), dict(dz=None), dict(dz=odd(DZ)), dict(dx=odd(DX)), dict(dw=odd(DW)), dict(ws=None),
               dict(ws=odd(WS)), dict(nb=n.value - 1), dict(cols=8), dict(total=odd(TOTAL))):
        assert bwd(**kw) == 1, kw
    assert bwd(rows=1 << 31) == 6
    shift = lambda p: odd(p, 64)
    for kw in (dict(dz=shift(DY)), dict(dz=DY, fp32=1), dict(dz=W), dict(dx=DZ), dict(dx=Z, fp32=1), dict(dw=RSTD), dict(ws=Z),
               dict(dw=WS), dict(dz=shift(DRES))):
        assert bwd(**kw) == 1, kw


def layout_desc(N=64, K=8, E=16, A=128):
    return ctypes.byref(binding._CDesc(N, K, E, 4, A))


def size(fn, d):
    n = ctypes.c_size_t(0)
    assert fn(d, ctypes.byref(n)) == 0
    return n.value


def test_grouped_gate_refusals(lib):
    d = layout_desc()
    n = size(lib.moe_gate_workspace_bytes, d)
    cfg = ctypes.byref(binding._CGateDesc(0, 1, 1, 1.0, 0.0))
    L, BIAS, IDX, W, CNT, MEAN, RT, LOSS, WS = FAKE[:9]

    def fwd(g=(4, 2, 2), logits=L, ld=16, bias=None, idx=IDX, w=W, cnt=CNT, mean=MEAN, rt=RT, loss=LOSS, ws=WS, nb=n, c=cfg, d=d):
        g = None if g is None else ctypes.byref(binding._CGateGroups(*g))
        return lib.moe_gate_forward_grouped(d, c, g, logits, ld, bias, idx, w, cnt, mean, rt, loss, ws, nb, None)

    for kw in (dict(g=None), dict(g=(0, 1, 1)), dict(g=(3, 1, 1)), dict(g=(4, 0, 1)), dict(g=(4, 5, 1)), dict(g=(4, 2, 0)),
               dict(g=(4, 2, 3)), dict(logits=None), dict(logits=odd(L)), dict(ld=15), dict(bias=odd(BIAS)), dict(idx=None), dict(w=None),
               dict(cnt=None), dict(mean=None), dict(rt=None), dict(loss=None), dict(ws=None), dict(ws=odd(WS)), dict(nb=n - 1),
               dict(c=None)):
        assert fwd(**kw) == 1, kw
    many = layout_desc(E=64)
    assert fwd(g=(64, 2, 1), d=many, ld=64, nb=1 << 30) == 6


def test_gate_config_of_groups():
    desc = binding.LayoutDesc(4, 2, 8, 1, 1)
    with pytest.raises(ValueError):
        binding.Gate(desc, binding.GateConfig(num_groups=4, topk_groups=2), device="cpu")
    with pytest.raises(ValueError):
        binding.Gate(desc, binding.GateConfig(bias_on="keys"), device="cpu")
    gate = binding.Gate(desc, binding.GateConfig(bias_on="score", num_groups=4, topk_groups=2, group_sum=2), device="cpu")
    g = gate._groups[0]._obj
    assert (g.num_groups, g.topk_groups, g.group_sum) == (4, 2, 2)
    assert binding.Gate(desc, binding.GateConfig(), device="cpu")._groups == ()


def test_combine_backward_refusals(lib):
    d = layout_desc()
    n = size(lib.moe_layout_workspace_bytes, d)
    DOUT, SLOT, W, Y, DY, DW, OFF, CNT, WS = FAKE[:9]

    def bwd(dout=DOUT, h=64, slot=SLOT, w=W, y=Y, dy=DY, cap=1000, dw=DW, off=OFF, cnt=CNT, pad=1, ws=WS, nb=n):
        return lib.moe_combine_backward(d, dout, h, slot, w, y, dy, cap, dw, off, cnt, pad, ws, nb, None)

    shift = lambda p: odd(p, 64)
    for kw in (dict(dout=None), dict(dout=odd(DOUT)), dict(h=0), dict(h=12), dict(slot=None), dict(w=None), dict(w=odd(W)), dict(y=None),
               dict(y=odd(Y)), dict(dy=None), dict(dy=odd(DY)), dict(cap=-1), dict(dw=odd(DW)), dict(off=None), dict(cnt=None),
               dict(ws=None), dict(ws=odd(WS)), dict(nb=n - 1), dict(dy=DOUT), dict(dy=shift(Y)), dict(dy=W), dict(dy=SLOT), dict(dw=W),
               dict(dw=Y), dict(dw=DY), dict(dw=SLOT), dict(dw=DOUT)):
        assert bwd(**kw) == 1, kw
    assert bwd(cap=1 << 31) == 6 and bwd(h=1 << 30) == 6


def test_norm_formula_against_differences():
    """The gradient the GPU tests compare with, against central differences of the definition in 64 bits."""
    g = torch.Generator().manual_seed(0)
    z, w, dy = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, 48), (48,), (4, 48)))
    eps = 1e-5
    y = lambda z, w: z * (z.square().mean(1, keepdim=True) + eps).rsqrt() * w
    r = (z.square().mean(1, keepdim=True) + eps).rsqrt()
    gr, h = dy * w, z * r
    dz, dw = r * (gr - h * (gr * h).mean(1, keepdim=True)), (dy * h).sum(0)
    for arg, grad in ((z, dz), (w, dw)):
        for i in range(arg.numel()):
            keep = float(arg.view(-1)[i])
            sides = []
            for s in (1e-5, -1e-5):
                arg.view(-1)[i] = keep + s
                sides.append(float((y(z, w) * dy).sum()))
            arg.view(-1)[i] = keep
            assert abs((sides[0] - sides[1]) / 2e-5 - float(grad.reshape(-1)[i])) < 1e-7


def test_python_refusals():
    """What the binding refuses by itself, before a pointer is taken: shapes, types, what belongs together."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    x, w = bf(4, 256), bf(256)
    for kw in (dict(residual=x), dict(q=x), dict(sf=x), dict(residual=bf(4, 256).half(), residual_out=x)):
        with pytest.raises(ValueError):
            binding.rms_norm(x, w, y=x, **kw)
    with pytest.raises(ValueError):
        binding.rms_norm(bf(256), w, y=x)
    with pytest.raises(ValueError):
        binding.rms_norm(x, bf(128), y=x)
    with pytest.raises(ValueError):
        binding.rms_norm(x, w.half(), y=x)
    with pytest.raises(ValueError):
        binding.rms_norm_backward(x, x, torch.zeros(4), w, x, dweight=torch.zeros(256))
    desc = binding.LayoutDesc(4, 2, 8, 1, 1)
    with pytest.raises(ValueError):
        binding.combine_backward(desc, x, torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2), bf(8, 256), x, dweights=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        binding.combine_backward(desc, x, torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2), bf(8, 128), x)


def test_a_tensor_elsewhere_is_refused(monkeypatch):
    """Tensors of another device than the current one."""
    class Elsewhere:
        is_cuda, device = True, "cuda:1"
        get_device = staticmethod(lambda: 1)

    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    with pytest.raises(ValueError):
        binding._here(Elsewhere(), "x")
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    binding._here(Elsewhere(), "x")
