"""The norm with the residual's addition, its 8-bit rows and its gradient against plain 64-bit forms.

Tolerances.  The kept z is one fp32 addition rounded once: equal bit for bit.  A sum over a row is at most
8 * 8 additions in a thread and 5 + 16 over threads, all of positive terms or bounded by their magnitudes: 85 * 2^-24
< 2^-17 of the sum of magnitudes.  r = 1 / sqrt(mean) halves that and adds three roundings: 2^-17.  A normed value
has two more roundings, 2^-17 + 2^-23 < 2^-16, then half a step of its type (bf16 2^-8; e4m3 2^-4, or half its
smallest step 2^-10 times the scale).  Scales: 2^-16.
Gradient: mean(g h) errs by 2^-17 of mean|g h|, everything else by a few 2^-24 of the magnitudes that enter (2^-20).
The weight's gradient is a sum over rows of at most 16 a CTA here, then up to 608 / 8 + 8 parts: 2^-17 of the sum of
magnitudes, and h's two roundings: 2^-16.
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def blocks(n):
    return -(-n // 128)


def draw(rows, cols, seed, stream=BF16, weight=BF16, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device=DEV)
    if spread:      # rows of very different sizes, one of zeros
        x = x * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g, device=DEV).float())
        x[5 % rows:: 9] = 0
    res = torch.randn((rows, cols), generator=g, device=DEV) * x.abs().amax(1, keepdim=True)
    w = torch.randn(cols, generator=g, device=DEV) * 0.3 + 1
    return x.to(BF16), res.to(stream), w.to(weight)


def norm(x, w, residual=None, y=True, q=False, col_major=False, total=None, eps=EPS):
    """Outputs with canaries, as a dict."""
    R, C = x.shape
    out = dict(rstd=torch.full((R,), -3.0, device=DEV))
    kw = {}
    if residual is not None:
        out["z"] = kw["residual_out"] = torch.full((R, C), 77.0, dtype=residual.dtype, device=DEV)
    if y:
        out["y"] = torch.full((R, C), 55.0, dtype=BF16, device=DEV)
    if q:
        out["q"] = torch.full((R, C), 0x55, dtype=torch.uint8, device=DEV)
        ld = (R + 3) // 4 * 4 + 4
        out["sf"] = torch.full((blocks(C), ld) if col_major else (R, blocks(C)), -7.0, device=DEV)
    binding.rms_norm(x, w, y=out.get("y"), q=out["q"].view(E4M3) if q else None, sf=out.get("sf"), residual=residual,
                     rstd=out["rstd"], eps=eps, col_major=col_major,
                     total_rows=None if total is None else torch.tensor([total], dtype=torch.int32, device=DEV), **kw)
    if q:
        out["scales"] = out["sf"][:, :R].t() if col_major else out["sf"]
    return out


def check(out, x, w, residual=None, n=None, eps=EPS):
    n = x.shape[0] if n is None else n
    z = x
    if residual is not None:
        z = (x.float() + residual.float()).to(residual.dtype)
        assert torch.equal(out["z"][:n], z[:n])
        assert torch.all(out["z"][n:] == 77.0)
    z = z[:n].double()
    r = (z.square().mean(1) + eps).rsqrt()
    assert torch.all((out["rstd"][:n].double() - r).abs() <= 2.0 ** -17 * r)
    assert torch.all(out["rstd"][n:] == -3.0)
    v = z * r[:, None] * w.double()
    if "y" in out:
        assert torch.all((out["y"][:n].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -16) * v.abs() + 2.0 ** -133)
        assert torch.all(out["y"][n:] == 55.0)
    if "q" in out:
        C, nb = x.shape[1], blocks(x.shape[1])
        pad = torch.nn.functional.pad(v.abs(), (0, nb * 128 - C)).view(n, nb, 128).amax(2).clamp(min=1e-30) / 448.0
        sf = out["scales"][:n].double()
        assert torch.all((sf - pad).abs() <= 2.0 ** -16 * pad)
        wide = sf.repeat_interleave(128, 1)[:, :C]
        got = out["q"].view(E4M3)[:n].double() * wide
        assert torch.all((got - v).abs() <= (2.0 ** -4 + 2.0 ** -16) * v.abs() + 2.0 ** -10 * wide)
        assert torch.all(out["q"][n:] == 0x55)


SHAPES = [(1, 16), (3, 128), (9, 144), (33, 256), (20, 512), (17, 1024), (5, 1040), (40, 2064), (7, 4096), (70, 7168), (3, 8192),
          (2, 8208), (3, 16384), (2, 16400), (2, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream,weight", [(None, BF16), (BF16, FP32), (FP32, BF16)])
def test_forward(rows, cols, stream, weight):
    x, res, w = draw(rows, cols, rows + cols, stream or BF16, weight)
    res = None if stream is None else res
    check(norm(x, w, res, y=True, q=True), x, w, res)
    check(norm(x, w, res, y=False, q=True, col_major=True), x, w, res)
    check(norm(x, w, res), x, w, res)


def test_column_major_scales_leave_the_rest_alone():
    x, res, w = draw(10, 272, 1)
    out = norm(x, w, res, q=True, col_major=True)
    assert torch.all(out["sf"][:, 10:] == -7.0)


@pytest.mark.parametrize("total", [0, 1, 8, 9, 30, 400])
@pytest.mark.parametrize("cols", [272, 2048])
def test_rows_stop_at_the_device_count(cols, total):
    x, res, w = draw(30, cols, 2)
    n = min(total, 30)
    out = norm(x, w, res, q=True, total=total)
    check(out, x, w, res, n)
    assert torch.all(out["sf"][n:] == -7.0)


@pytest.mark.parametrize("stream", [BF16, FP32])
@pytest.mark.parametrize("cols", [528, 2048])
def test_in_place(stream, cols):
    """The stream over itself, and bf16 rows over x."""
    x, res, w = draw(13, cols, 3, stream)
    want = norm(x, w, res)
    x2, res2 = x.clone(), res.clone()
    binding.rms_norm(x2, w, y=x2, residual=res2, residual_out=res2, eps=EPS)
    assert torch.equal(res2, want["z"]) and torch.equal(x2, want["y"])


def test_squares_beyond_fp32():
    """Rows whose squares overflow 32 bits are normed all the same; infinities and NaN stay in their row."""
    x, _, w = draw(6, 1040, 4, spread=False)
    x[0] *= 2.0 ** 100
    x[1] = (x[1].float() * 2.0 ** 126).clamp(-3e38, 3e38).to(BF16)
    check(norm(x, w, q=True), x, w)
    x[2, 7], x[3, 1000] = float("inf"), float("nan")
    out = norm(x, w)
    assert torch.isnan(out["y"][2, 7]) and torch.all(out["y"][2, :7] == 0) and torch.all(torch.isnan(out["y"][3]))
    check({k: v[[0, 1, 4, 5]] for k, v in out.items()}, x[[0, 1, 4, 5]], w)


def grad(dy, z, r, w, dres, n):
    dy, z, r, w = dy[:n].double(), z[:n].double(), r[:n].double()[:, None], w.double()
    g, h = dy * w, z * r
    mean, mag = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    d = torch.zeros_like(z) if dres is None else dres[:n].double()
    dz = r * (g - h * mean) + d
    off = 2.0 ** -17 * r * h.abs() * mag + 2.0 ** -20 * (r * (g.abs() + (h * mean).abs()) + d.abs())
    return dz, off, (dy * h).sum(0), 2.0 ** -16 * (dy * h).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES + [(5000, 256), (2500, 1040), (1500, 4096)])
@pytest.mark.parametrize("stream,weight,with_dres", [(BF16, BF16, True), (FP32, FP32, True), (BF16, FP32, False)])
def test_backward(rows, cols, stream, weight, with_dres):
    x, res, w = draw(rows, cols, rows + cols, stream, weight)
    f = norm(x, w, res)
    g = torch.Generator(device=DEV).manual_seed(8)
    dy = torch.randn((rows, cols), generator=g, device=DEV).to(BF16)
    dres = torch.randn((rows, cols), generator=g, device=DEV).to(stream) if with_dres else None
    dz = torch.full((rows, cols), 9.0, dtype=stream, device=DEV)
    dx = torch.full((rows, cols), 9.0, dtype=BF16, device=DEV) if stream == FP32 else None
    dw = torch.full((cols,), 9.0, device=DEV)
    ws = binding.new_norm_workspace(cols)
    ws.fill_(0xff)          # need not be zeros
    binding.rms_norm_backward(dy, f["z"], f["rstd"], w, dz, dresidual=dres, dx=dx, dweight=dw, workspace=ws)
    want, off, want_w, off_w = grad(dy, f["z"], f["rstd"], w, dres, rows)
    assert torch.all((dz.double() - want).abs() <= off + HALF[stream] * want.abs())
    if dx is not None:
        assert torch.all((dx.double() - want).abs() <= off + HALF[BF16] * want.abs())
    assert torch.all((dw.double() - want_w).abs() <= off_w)
    again = torch.empty_like(dw)
    binding.rms_norm_backward(dy, f["z"], f["rstd"], w, dz, dresidual=dres, dx=dx, dweight=again, workspace=ws)
    assert torch.equal(again, dw)
    binding.rms_norm_backward(dy, f["z"], f["rstd"], w, dz, dresidual=dres, dx=dx, dweight=again, workspace=ws, accumulate=True)
    assert torch.equal(again, dw + dw)


@pytest.mark.parametrize("total", [0, 1, 13, 50, 99])
@pytest.mark.parametrize("cols", [272, 2048])
def test_backward_stops_at_the_device_count(cols, total):
    x, res, w = draw(50, cols, 5)
    f = norm(x, w, res)
    dy = torch.randn((50, cols), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF16)
    dz = torch.full((50, cols), 9.0, dtype=BF16, device=DEV)
    dw = torch.full((cols,), 9.0, device=DEV)
    n = min(total, 50)
    binding.rms_norm_backward(dy, f["z"], f["rstd"], w, dz, dweight=dw, workspace=binding.new_norm_workspace(cols),
                              total_rows=torch.tensor([total], dtype=torch.int32, device=DEV))
    want, off, want_w, off_w = grad(dy, f["z"], f["rstd"], w, None, n)
    assert torch.all((dz[:n].double() - want).abs() <= off + HALF[BF16] * want.abs())
    assert torch.all(dz[n:] == 9.0)
    assert torch.all((dw.double() - want_w).abs() <= off_w)


@pytest.mark.parametrize("cols", [272, 2048])
def test_backward_in_place(cols):
    """dz over dresidual, over z and over dy."""
    x, res, w = draw(21, cols, 6, BF16)
    f = norm(x, w, res)
    g = torch.Generator(device=DEV).manual_seed(9)
    dy, dres = (torch.randn((21, cols), generator=g, device=DEV).to(BF16) for _ in range(2))
    want = torch.empty_like(dy)
    binding.rms_norm_backward(dy, f["z"], f["rstd"], w, want, dresidual=dres)
    for which in ("dy", "z", "dresidual"):
        a = dict(dy=dy.clone(), z=f["z"].clone(), dresidual=dres.clone())
        binding.rms_norm_backward(a["dy"], a["z"], f["rstd"], w, a[which], dresidual=a["dresidual"])
        assert torch.equal(a[which], want), which


def test_no_rows():
    w = torch.ones(256, device=DEV)
    x = torch.empty((0, 256), dtype=BF16, device=DEV)
    r = torch.empty(0, device=DEV)
    binding.rms_norm(x, w, y=torch.empty_like(x))
    dw = torch.full((256,), 5.0, device=DEV)
    ws = binding.new_norm_workspace(256)
    binding.rms_norm_backward(x, x, r, w, torch.empty_like(x), dweight=dw, workspace=ws, accumulate=True)
    assert torch.all(dw == 5.0)
    binding.rms_norm_backward(x, x, r, w, torch.empty_like(x), dweight=dw, workspace=ws)
    assert torch.all(dw == 0.0)


def test_other_stream_and_graph():
    """Both directions on a stream of their own, captured and replayed on other inputs."""
    x, res, w = draw(300, 1040, 7)
    s = torch.cuda.Stream()
    y, z, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(300, device=DEV)
    dz, dw, ws = torch.empty_like(x), torch.empty(1040, device=DEV), binding.new_norm_workspace(1040)

    def step():
        binding.rms_norm(x, w, y=y, residual=res, residual_out=z, rstd=rstd, eps=EPS)
        binding.rms_norm_backward(y, z, rstd, w, dz, dweight=dw, workspace=ws)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(x.flip(0))
    res.copy_(res.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check(dict(z=z, y=y, rstd=rstd), x, w, res)
    want, off, want_w, off_w = grad(y, z, rstd, w, None, 300)
    assert torch.all((dz.double() - want).abs() <= off + HALF[BF16] * want.abs())
    assert torch.all((dw.double() - want_w).abs() <= off_w)


def test_on_a_named_stream():
    """The ``stream`` argument of the norm, its gradient, the routing and the combine's gradient: work that is behind a
    long wait on that stream is not done before it, and is done after."""
    x, res, w = draw(64, 1040, 11)
    s = torch.cuda.Stream()
    y, z, dz = (torch.zeros_like(x) for _ in range(3))
    rstd, dw, ws = torch.zeros(64, device=DEV), torch.zeros(1040, device=DEV), binding.new_norm_workspace(1040)
    desc = binding.LayoutDesc(64, 2, 8, 1, 1)
    gate = binding.Gate(desc, binding.GateConfig("sigmoid", bias_on="score", num_groups=4, topk_groups=2, group_sum=2))
    l = torch.randn((64, 8), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    lay = binding.Layout(desc, 128)
    dy, dwk = torch.zeros((128, 1040), dtype=BF16, device=DEV), torch.zeros((64, 2), device=DEV)

    def run():
        binding.rms_norm(x, w, y=y, residual=res, residual_out=z, rstd=rstd, eps=EPS, stream=s)
        binding.rms_norm_backward(y, z, rstd, w, dz, dweight=dw, workspace=ws, stream=s)
        gate.forward(l, stream=s)
        lay.build(gate.topk_idx, stream=s)
        lay.combine_backward(y, gate.weights, dy, dy, dwk, stream=s)
        return y.clone()                        # on the current stream, which does not wait

    torch.cuda.synchronize()
    run()                                       # a kernel's first launch loads it, which may wait for the device
    torch.cuda.synchronize()
    for t in (y, z, dz, rstd, dw, dy, dwk):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)          # about a tenth of a second
    early = run()
    torch.cuda.current_stream().synchronize()
    assert not early.any()
    s.synchronize()
    check(dict(z=z, y=y, rstd=rstd), x, w, res)
    want, off, want_w, off_w = grad(y, z, rstd, w, None, 64)
    assert torch.all((dz.double() - want).abs() <= off + HALF[BF16] * want.abs())
    assert torch.all((dw.double() - want_w).abs() <= off_w)
    slot = lay.dst_slot[:128].long()
    assert torch.equal(dy[slot], (gate.weights.view(-1, 1) * y.float().repeat_interleave(2, 0)).to(BF16))
    assert gate.error() == 0 and lay.error() == 0
