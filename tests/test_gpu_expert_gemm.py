"""Expert products and weight gradients against 64-bit products.

Tolerances.  Products of e4m3 values are exact in fp32; each of the 128 additions of
a k-block and of the additions over blocks may lose 2^-23 of the running sum, so a
sum errs by at most (128 + blocks + 4) * 2^-23 of the sum of the magnitudes; bf16
results add half a unit, 2^-9 relative.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def blocks(n):
    return -(-n // 128)


def segments(counts, A):
    off = np.zeros(len(counts) + 1, np.int64)
    off[1:] = np.cumsum([(c + A - 1) // A * A for c in counts])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    return i32(list(off)), i32(list(counts)), int(off[-1])


def codes(shape, g):
    """Random e4m3 codes of every magnitude, no NaN."""
    c = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.int32)
    c = torch.where((c & 0x7f) == 0x7f, c - 1, c)
    return c.to(torch.uint8).view(E4M3)


def scales(shape, g):
    return torch.exp2(torch.rand(shape, generator=g, device=DEV) * 8 - 6)


def forward_case(counts, A, wi, wo, seed, slack=0, pairs=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    E = len(counts)
    off, cnt, total = segments(counts, A)
    cap = total + slack
    x = codes((cap, wi), g)
    x_sf = scales((blocks(wi), (cap + 3) // 4 * 4), g)
    w, w_sf = codes((E, wo, wi), g), scales((E, blocks(wo), blocks(wi)), g)
    # what lies outside the real rows may be anything
    real = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for e, c in enumerate(counts):
        real[int(off[e]):int(off[e]) + c] = True
    x.view(torch.uint8)[~real] = 0x7f
    x_sf[:, :cap][:, ~real] = float("nan")
    desc = binding.LayoutDesc(pairs or max(sum(counts), 1), 1, E, 1, A)
    out = torch.full((cap + 1, wo), 3.0, dtype=torch.bfloat16, device=DEV)
    ws = binding.new_workspace(desc)
    return dict(desc=desc, x=x, x_sf=x_sf, w=w, w_sf=w_sf, off=off, cnt=cnt, out=out, ws=ws, cap=cap, total=total)


def run_forward(c):
    binding.expert_gemm(c["desc"], c["x"], c["x_sf"], c["w"], c["w_sf"], c["off"], c["cnt"], c["out"][: c["cap"]], c["ws"])
    return binding.get_error(c["ws"])


def check_forward(c, counts):
    wo, wi = c["w"].shape[1:]
    ib, ob = torch.arange(wi, device=DEV) // 128, torch.arange(wo, device=DEV) // 128
    got = c["out"].double()
    for e, n in enumerate(counts):
        a, z = int(c["off"][e]), int(c["off"][e + 1])
        x = c["x"][a:a + n].double() * c["x_sf"][:, a:a + n].t().double()[:, ib]
        w = c["w"][e].double() * c["w_sf"][e].double()[ob][:, ib]
        want, mag = x @ w.t(), x.abs() @ w.t().abs()
        tol = 2.0 ** -8 * want.abs() + (132 + blocks(wi)) * 2.0 ** -23 * mag
        assert torch.all((got[a:a + n] - want).abs() <= tol), f"expert {e}"
        assert torch.all(got[a + n:z] == 0), f"gap of expert {e}"
    assert torch.all(got[c["total"]:] == 3.0)


FORWARD = [
    # counts, alignment, width_in, width_out, slack
    ([1], 1, 16, 8, 0),
    ([1], 1, 7168, 256, 0),
    ([5, 0, 1], 1, 128, 128, 3),
    ([0, 17, 130, 1], 16, 144, 136, 0),
    ([16, 15, 33], 64, 1040, 520, 9),
    ([127, 128, 129], 128, 256, 384, 0),
    ([40] * 30, 8, 272, 200, 5),
    ([300, 0, 515, 256], 1, 1040, 520, 0),
    ([256, 257], 128, 128, 256, 1),
    ([1000], 128, 2048, 1032, 0),
    ([700, 3, 250], 128, 400, 264, 0),
]


@pytest.mark.parametrize("counts,A,wi,wo,slack", FORWARD)
def test_product(counts, A, wi, wo, slack):
    c = forward_case(counts, A, wi, wo, 3 * wi + wo, slack)
    assert run_forward(c) == 0
    check_forward(c, counts)


@pytest.mark.parametrize("pairs", [1, 100000])
def test_any_tiling_serves_any_segments(pairs):
    """The pair count only chooses the tiling: both give every segment's product."""
    counts = [1, 0, 300, 64, 513]
    c = forward_case(counts, 16, 528, 392, 77, 4, pairs=pairs)
    assert run_forward(c) == 0
    check_forward(c, counts)


@pytest.mark.parametrize("n,wi,wo", [(1, 1024, 128), (3, 1040, 136), (33, 2064, 264), (64, 7168, 128), (65, 1536, 512),
                                     (119, 4096, 200)])
def test_tiles_shared_by_a_cluster(n, wi, wo):
    """Few rows and few tiles: each CTA of a cluster takes a share of K."""
    c = forward_case([n], 16, wi, wo, n + wi)
    assert run_forward(c) == 0
    check_forward(c, [n])


def test_a_shared_tile_for_each_of_too_many_tiles():
    """More tiles than the pair count promised: each cluster takes several, one after the other."""
    counts = [100, 0, 130, 257, 1]
    c = forward_case(counts, 8, 2048, 4096, 5, pairs=1)
    assert run_forward(c) == 0
    check_forward(c, counts)


def test_many_experts():
    g = np.random.default_rng(5)
    counts = [int(v) for v in g.integers(0, 4, 1024)]
    c = forward_case(counts, 1, 256, 136, 8)
    assert run_forward(c) == 0
    check_forward(c, counts)


def test_dense_product_is_one_expert():
    for n in (1, 7, 200, 2000):
        c = forward_case([n], 1, 1024, 768, n)
        assert run_forward(c) == 0
        check_forward(c, [n])


def test_no_rows():
    c = forward_case([0, 0, 0], 128, 256, 128, 1, slack=5)
    assert run_forward(c) == 0
    assert torch.all(c["out"] == 3.0)


def test_repeats_are_equal_and_streams_are_followed():
    counts = [300, 20, 511]
    c = forward_case(counts, 128, 512, 512, 12)
    assert run_forward(c) == 0
    first = c["out"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(5):
            c["out"].fill_(3.0)
            assert run_forward(c) == 0
            assert torch.equal(first, c["out"])


def test_not_a_number_stays_in_its_row():
    c = forward_case([40, 9], 16, 256, 128, 4)
    c["x"].view(torch.uint8)[7, 100] = 0x7f
    assert run_forward(c) == 0
    got = c["out"].float()
    assert torch.isnan(got[7]).all()
    assert torch.isfinite(got[:7]).all() and torch.isfinite(got[8:40]).all() and torch.isfinite(got[48:57]).all()


def test_overflowed_layout_is_left_out_and_reported():
    c = forward_case([20, 30, 40], 16, 128, 128, 6)
    c["cnt"][1] = 5000
    assert run_forward(c) == 4
    a = int(c["off"][1])
    assert torch.all(c["out"][a:int(c["off"][2])] == 3.0)
    c["cnt"][1] = 30
    c["off"][1] = -4
    assert run_forward(c) == 4


def test_rows_past_two_to_the_31_bytes():
    """Offsets into x and out beyond 2^31: the last expert's rows against the same rows alone."""
    wi, wo, n = 8192, 4096, 262144 + 64
    g = torch.Generator(device=DEV).manual_seed(1)
    tail = codes((64, wi), g)
    x = torch.zeros((n, wi), dtype=torch.uint8, device=DEV).view(E4M3)
    x.view(torch.uint8)[n - 64:] = tail.view(torch.uint8)
    x_sf = scales((blocks(wi), n), g)
    w, w_sf = codes((2, wo, wi), g), scales((2, blocks(wo), blocks(wi)), g)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    desc = binding.LayoutDesc(n, 1, 2, 1, 64)
    ws = binding.new_workspace(desc)
    out = torch.full((n, wo), 3.0, dtype=torch.bfloat16, device=DEV)
    binding.expert_gemm(desc, x, x_sf, w, w_sf, i32([0, n - 64, n]), i32([n - 64, 64]), out, ws)
    alone = torch.empty((64, wo), dtype=torch.bfloat16, device=DEV)
    one = binding.LayoutDesc(n, 1, 1, 1, 64)
    binding.expert_gemm(one, tail, x_sf[:, n - 64:].contiguous(), w[1:], w_sf[1:], i32([0, 64]), i32([64]), alone, ws)
    assert binding.get_error(ws) == 0
    assert torch.equal(out[n - 64:], alone)
    assert torch.all(out[: n - 64] == 0)


# ---------------------------------------------------------------- weight gradient
def wgrad_case(counts, A, wo, wi, seed, slack=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    off, cnt, total = segments(counts, A)
    cap = total + slack
    ld = blocks(cap) * 128
    dy, x = codes((wo, ld), g), codes((wi, ld), g)
    dy_sf, x_sf = scales((blocks(cap), wo), g), scales((blocks(cap), wi), g)
    real = torch.zeros(ld, dtype=torch.bool, device=DEV)
    for e, c in enumerate(counts):
        real[int(off[e]):int(off[e]) + c] = True
    dy.view(torch.uint8)[:, ~real] = 0        # gap rows are zeros, as quantize_cols leaves them
    x.view(torch.uint8)[:, ~real] = 0
    desc = binding.LayoutDesc(max(sum(counts), 1), 1, len(counts), 1, A)
    dw = torch.full((len(counts), wo, wi), 5.0, dtype=dtype, device=DEV)
    return dict(desc=desc, dy=dy, dy_sf=dy_sf, x=x, x_sf=x_sf, off=off, cnt=cnt, dw=dw, ws=binding.new_workspace(desc))


def run_wgrad(c, **kw):
    binding.expert_wgrad(c["desc"], c["dy"], c["dy_sf"], c["x"], c["x_sf"], c["off"], c["cnt"], c["dw"], c["ws"], **kw)
    return binding.get_error(c["ws"])


def check_wgrad(c, counts, base=0.0):
    half = 2.0 ** -8 if c["dw"].dtype == torch.bfloat16 else 0.0
    for e, n in enumerate(counts):
        a = int(c["off"][e])
        rb = torch.arange(a, a + n, device=DEV) // 128
        dy = c["dy"][:, a:a + n].double() * c["dy_sf"].double()[rb].t()
        x = c["x"][:, a:a + n].double() * c["x_sf"].double()[rb].t()
        want, mag = dy @ x.t() + base, dy.abs() @ x.abs().t() + abs(base)
        tol = half * want.abs() + (132 + blocks(n) + 1) * 2.0 ** -23 * mag
        assert torch.all((c["dw"][e].double() - want).abs() <= tol), f"expert {e}"


WGRAD = [
    # counts, alignment, width_out, width_in, slack
    ([1], 128, 8, 8, 0),
    ([0, 3], 128, 40, 16, 0),
    ([130, 0, 128, 64], 128, 272, 400, 17),
    ([1000], 256, 264, 520, 0),
    ([64] * 8, 128, 128, 256, 0),
    ([700, 5], 128, 513, 136, 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,A,wo,wi,slack", WGRAD)
def test_weight_gradient(counts, A, wo, wi, slack, dtype):
    c = wgrad_case(counts, A, wo, wi, wo + wi, slack, dtype)
    assert run_wgrad(c) == 0
    check_wgrad(c, counts)


def test_weight_gradient_accumulates():
    counts = [200, 0, 77]
    c = wgrad_case(counts, 128, 136, 264, 5)
    assert run_wgrad(c, accumulate=True) == 0
    check_wgrad(c, counts, base=5.0)


def test_weight_gradient_of_a_segment_off_the_block_grid_is_refused_by_the_kernel():
    counts = [200, 77]
    c = wgrad_case(counts, 128, 136, 264, 5)
    c["off"][1] = 250
    assert run_wgrad(c) == 1
    assert torch.all(c["dw"][1] == 0)
    check_wgrad(c, counts[:1])


def test_quantised_training_products_agree_with_the_bf16_ones():
    """Forward, input gradient and weight gradient from bf16 tensors through the quantisers: each operand carries
    at most 2^-4 relative error of its value, so a product of two at most 2^-3 of the magnitudes."""
    g = torch.Generator(device=DEV).manual_seed(6)
    counts, A, wi, wo = [190, 0, 66], 128, 256, 384
    off, cnt, total = segments(counts, A)
    desc = binding.LayoutDesc(sum(counts), 1, 3, 1, A)
    ws = binding.new_workspace(desc)
    x = torch.randn((total, wi), generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn((total, wo), generator=g, device=DEV).to(torch.bfloat16)
    for e, c in enumerate(counts):
        x[int(off[e]) + c:int(off[e + 1])] = 0
        dy[int(off[e]) + c:int(off[e + 1])] = 0
    w = torch.randn((3, wo, wi), generator=g, device=DEV)
    v = w.view(3, wo // 128, 128, wi // 128, 128)
    w_sf = v.abs().amax((2, 4)) / 448.0
    wq = (v / w_sf[:, :, None, :, None]).view(3, wo, wi).to(E4M3)

    def rows(t):
        q = torch.empty(t.shape, dtype=E4M3, device=DEV)
        sf = binding.new_sf_col_major(t.shape[1] // 128, total)
        binding.quantize_rows(t, q, sf, col_major=True)
        return q, sf

    def cols(t):
        q = torch.empty((t.shape[1], total), dtype=E4M3, device=DEV)
        sf = torch.empty((total // 128, t.shape[1]), device=DEV)
        binding.quantize_cols(desc, t, off, cnt, q, sf, ws)
        return q, sf

    y = torch.empty((total, wo), dtype=torch.bfloat16, device=DEV)
    binding.expert_gemm(desc, *rows(x), wq, w_sf, off, cnt, y, ws)
    dx = torch.empty((total, wi), dtype=torch.bfloat16, device=DEV)
    binding.expert_gemm(desc, *rows(dy), wq.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3),
                        w_sf.transpose(1, 2).contiguous(), off, cnt, dx, ws)
    dw = torch.empty((3, wo, wi), device=DEV)
    binding.expert_wgrad(desc, *cols(dy), *cols(x), off, cnt, dw, ws)
    assert binding.get_error(ws) == 0
    for e, c in enumerate(counts):
        a, z = int(off[e]), int(off[e]) + c
        xe, de, we = x[a:z].double(), dy[a:z].double(), w[e].double()
        for got, want, mag in ((y[a:z], xe @ we.t(), xe.abs() @ we.t().abs()),
                               (dx[a:z], de @ we, de.abs() @ we.abs()),
                               (dw[e], de.t() @ xe, de.t().abs() @ xe.abs())):
            assert torch.all((got.double() - want).abs() <= 2.0 ** -3 * mag + 2.0 ** -8 * want.abs())


# ---------------------------------------------------------------- refusals and waits
def test_refusals():
    c = forward_case([20], 16, 128, 128, 1)
    args = lambda **k: {**dict(desc=c["desc"], x=c["x"], x_sf=c["x_sf"], w=c["w"], w_sf=c["w_sf"], expert_offset=c["off"],
                               expert_count=c["cnt"], out=c["out"][: c["cap"]], workspace=c["ws"]), **k}
    f8 = lambda *s: torch.zeros(s, dtype=E4M3, device=DEV)
    f4 = lambda *s: torch.zeros(s, device=DEV)
    bad = [dict(w=f8(1, 128, 256)), dict(w_sf=f4(1, 1, 2)), dict(out=c["out"]), dict(x_sf=f4(2, 32)), dict(x=c["x"].float()),
           dict(expert_offset=c["off"][:1]), dict(expert_count=c["cnt"].long())]
    for k in bad:
        with pytest.raises(ValueError):
            binding.expert_gemm(**args(**k))
    with pytest.raises(binding.LayoutError) as e:      # width_in not a multiple of 16
        binding.expert_gemm(**args(x=f8(32, 24), w=f8(1, 128, 24), w_sf=f4(1, 1, 1), x_sf=f4(1, 32)))
    assert e.value.status == 1
    with pytest.raises(binding.LayoutError) as e:      # width_out not a multiple of 8
        binding.expert_gemm(**args(w=f8(1, 12, 128), out=torch.zeros((32, 12), dtype=torch.bfloat16, device=DEV)))
    assert e.value.status == 1
    with pytest.raises(binding.LayoutError) as e:      # workspace too small
        binding.expert_gemm(**args(workspace=c["ws"][:128]))
    assert e.value.status == 1
    d = wgrad_case([20], 128, 16, 16, 1)
    with pytest.raises(binding.LayoutError) as e:      # accumulation needs an fp32 gradient
        d["dw"] = d["dw"].to(torch.bfloat16)
        run_wgrad(d, accumulate=True)
    assert e.value.status == 1
    with pytest.raises(binding.LayoutError) as e:      # segments must start on block boundaries
        d["desc"] = binding.LayoutDesc(20, 1, 1, 1, 64)
        run_wgrad(d)
    assert e.value.status == 6


@pytest.mark.parametrize("counts,wi", [([20, 9], 256), ([600, 300], 256), ([20], 2048)], ids=["one_cta", "pair", "shared_tile"])
def test_a_wait_that_runs_out_is_reported(counts, wi):
    c = forward_case(counts, 16, wi, 256, 2)
    try:
        binding.debug_set_waits(limit_ns=2_000_000, extra_tx=16)
        assert run_forward(c) == 5
    finally:
        binding.debug_set_waits()
    assert run_forward(c) == 0
    check_forward(c, counts)
