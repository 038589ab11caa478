"""8-bit rows and columns and the gated activation against plain implementations.

The plain quantiser makes the same three IEEE operations in fp32 (amax / 448,
1 / sf, x * inv) and torch's e4m3 conversion, so codes and scales are equal bit
for bit.  With the activation in front, sigmoid errs by a few 2^-22 relative
(exp, division), so scales agree to 2^-19 and a code can move to its neighbour
where the value lies that close to a rounding boundary: dequantised values agree
to half a code step of each side plus that, 2^-4 + 2^-19 relative to the value
(or half the smallest step, 2^-10 of sf, below the normal range).
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


def plain_rows(x):
    rows, cols = x.shape
    nb = blocks(cols)
    v = torch.nn.functional.pad(x.float(), (0, nb * 128 - cols)).view(rows, nb, 128)
    # a tensor as divisor: torch multiplies by the reciprocal of a scalar one
    sf = v.abs().amax(-1).clamp(min=1e-30) / torch.full((), 448.0, device=DEV)
    q = (v * (torch.ones_like(sf) / sf).unsqueeze(-1)).to(E4M3)
    return q.view(torch.uint8).view(rows, -1)[:, :cols], sf


def values(rows, cols, seed, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device=DEV)
    if spread:      # rows of very different sizes, zero blocks, tiny values
        x = x * torch.exp2(torch.randint(-30, 20, (rows, 1), generator=g, device=DEV).float())
        x[:: 7] = 0
        x[3 % max(rows, 1):: 11] = 1e-39
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (17, 512), (33, 640), (100, 1040), (16, 4096),
                                       (1000, 7168), (5, 2064)])
@pytest.mark.parametrize("col_major", [False, True])
def test_rows(rows, cols, col_major):
    x = values(rows, cols, rows + cols)
    want_q, want_sf = plain_rows(x)
    q = torch.full((rows + 1, cols), 0x55, dtype=torch.uint8, device=DEV)
    nb = blocks(cols)
    ld = (rows + 3) // 4 * 4 + 4
    sf = torch.full((nb, ld) if col_major else (rows, nb), -7.0, device=DEV)
    binding.quantize_rows(x, q[:rows].view(E4M3), sf, col_major=col_major)
    assert torch.equal(q[:rows], want_q)
    assert torch.equal(sf[:, :rows].t() if col_major else sf, want_sf)
    assert torch.all(q[rows:] == 0x55)
    if col_major:
        assert torch.all(sf[:, rows:] == -7.0)


@pytest.mark.parametrize("total", [0, 1, 31, 32, 50, 400])
def test_rows_stop_at_the_device_count(total):
    x = values(50, 272, 4)
    q = torch.full((50, 272), 0x11, dtype=torch.uint8, device=DEV)
    sf = torch.full((50, 3), -1.0, device=DEV)
    binding.quantize_rows(x, q.view(E4M3), sf, total_rows=torch.tensor([total], dtype=torch.int32, device=DEV))
    want_q, want_sf = plain_rows(x)
    n = min(total, 50)
    assert torch.equal(q[:n], want_q[:n]) and torch.equal(sf[:n], want_sf[:n])
    assert torch.all(q[n:] == 0x11) and torch.all(sf[n:] == -1.0)


def test_not_a_number_stays_in_its_block():
    x = values(4, 384, 9, spread=False)
    x[1, 130] = float("nan")
    x[2, 300] = float("inf")
    q = torch.empty((4, 384), dtype=E4M3, device=DEV)
    sf = torch.empty((4, 3), device=DEV)
    binding.quantize_rows(x, q, sf)
    back = q.float() * sf.repeat_interleave(128, 1)
    bad = ~torch.isfinite(back)
    assert bad[1, 128:256].all() and bad[2, 256:].all()
    assert int(bad.sum()) == 256


def test_empty():
    binding.quantize_rows(torch.empty((0, 128), dtype=torch.bfloat16, device=DEV),
                          torch.empty((0, 128), dtype=E4M3, device=DEV), torch.empty((0, 1), device=DEV))


def segments(counts, A):
    off = np.zeros(len(counts) + 1, np.int64)
    off[1:] = np.cumsum([(c + A - 1) // A * A for c in counts])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    return i32(list(off)), i32(list(counts)), int(off[-1])


@pytest.mark.parametrize("counts,cols,A,slack", [([1], 8, 128, 0), ([0, 5, 0, 128], 64, 128, 127), ([300, 1, 129], 200, 128, 40),
                                                 ([513, 0, 7], 72, 256, 0), ([128] * 9, 1040, 128, 3)])
def test_cols(counts, cols, A, slack):
    off, cnt, total = segments(counts, A)
    cap = total + slack
    x = values(cap, cols, cols)
    clean = torch.zeros_like(x)
    for e, c in enumerate(counts):
        a = int(off[e])
        clean[a:a + c] = x[a:a + c]
        x[a + c:int(off[e + 1])] = float("nan")              # gap rows hold anything
    ld = blocks(cap) * 128 + 128
    q = torch.full((cols, ld), 0x33, dtype=torch.uint8, device=DEV)
    sf = torch.full((blocks(cap), cols), -2.0, device=DEV)
    desc = binding.LayoutDesc(max(sum(counts), 1), 1, len(counts), 1, A)
    ws = binding.new_workspace(desc)
    binding.quantize_cols(desc, x, off, cnt, q.view(E4M3), sf, ws)
    assert binding.get_error(ws) == 0
    want_q, want_sf = plain_rows(clean[:total].t().contiguous())
    assert torch.equal(q[:, :total], want_q)
    assert torch.equal(sf[: total // 128], want_sf.t())
    assert torch.all(q[:, total:] == 0x33) and torch.all(sf[total // 128:] == -2.0)


def test_cols_of_a_layout_that_overflowed_write_nothing():
    off, cnt, total = segments([200, 100], 128)
    x = values(total - 128, 64, 3)
    q = torch.full((64, 512), 0x33, dtype=torch.uint8, device=DEV)
    sf = torch.full((2, 64), -2.0, device=DEV)
    desc = binding.LayoutDesc(300, 1, 2, 1, 128)
    ws = binding.new_workspace(desc)
    binding.quantize_cols(desc, x, off, cnt, q.view(E4M3), sf, ws)
    assert binding.get_error(ws) == 4
    assert torch.all(q == 0x33) and torch.all(sf == -2.0)


@pytest.mark.parametrize("rows,width,total", [(1, 16, None), (19, 128, 19), (33, 1040, 20), (200, 2048, None), (64, 1936, 0)])
def test_swiglu_quantize(rows, width, total):
    gu = values(rows, 2 * width, width, spread=False) * 2
    n = rows if total is None else total
    ld = (rows + 3) // 4 * 4
    q = torch.zeros((rows, width), dtype=E4M3, device=DEV)
    sf = torch.full((blocks(width), ld), -3.0, device=DEV)
    binding.swiglu_quantize(gu, q, sf, None if total is None else torch.tensor([total], dtype=torch.int32, device=DEV))
    a, b = gu[:n].double().split(width, 1)
    h = a * torch.sigmoid(a) * b
    v = torch.nn.functional.pad(h, (0, blocks(width) * 128 - width)).view(n, blocks(width), 128)
    want_sf = v.abs().amax(-1).clamp(min=1e-30) / 448.0
    assert torch.all((sf[:, :n].t().double() - want_sf).abs() <= 2.0 ** -19 * want_sf)
    assert torch.all(sf[:, n:] == -3.0)
    wide = want_sf.repeat_interleave(128, 1)[:, :width]
    back = q[:n].double() * sf[:, :n].t().double().repeat_interleave(128, 1)[:, :width]
    assert torch.all((back - h).abs() <= (2.0 ** -4 + 2.0 ** -19) * h.abs() + 2.0 ** -10 * wide)
    assert torch.all(q[n:].view(torch.uint8) == 0)


@pytest.mark.parametrize("rows,width,total", [(1, 8, None), (7, 24, 7), (33, 1048, 20), (129, 2048, None)])
def test_swiglu_backward(rows, width, total):
    """Each result is one bf16 rounding (2^-9) of a product of fp32 factors (2^-19 in all)."""
    g = torch.Generator(device=DEV).manual_seed(width)
    gu = (torch.randn((rows, 2 * width), generator=g, device=DEV) * 3).to(torch.bfloat16)
    dh = torch.randn((rows, width), generator=g, device=DEV).to(torch.bfloat16)
    out = torch.full((rows, 2 * width), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.swiglu_backward(gu, dh, out, None if total is None else torch.tensor([total], dtype=torch.int32, device=DEV))
    n = rows if total is None else total
    x = gu[:n].double().requires_grad_()
    a, b = x.split(width, 1)
    (a * torch.sigmoid(a) * b).backward(dh[:n].double())
    s = torch.sigmoid(a.detach())
    mag = torch.cat([dh[:n].double().abs() * b.detach().abs() * s * (1 + a.detach().abs()), x.grad[:, width:].abs()], 1)
    err = (out[:n].double() - x.grad).abs()
    assert torch.all(err <= 2.0 ** -8 * x.grad.abs() + 2.0 ** -19 * mag)
    assert torch.all(out[n:] == 7.0)


def test_swiglu_gradient_against_differences():
    """Differences of the 64-bit function at bf16 inputs; the step leaves ~1e-9, bf16 outputs 2^-8."""
    gu = torch.tensor([[-3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0, -0.25, 1.0, -2.0, 3.0, 0.5, -1.0, 1.5, 2.5, 0.75]])
    dh = torch.ones((1, 8))
    f = lambda v: float((v[:, :8] * torch.sigmoid(v[:, :8]) * v[:, 8:]).sum())
    num = torch.zeros((1, 16), dtype=torch.float64)
    for j in range(16):
        d = torch.zeros((1, 16), dtype=torch.float64)
        d[0, j] = 1e-5
        num[0, j] = (f(gu.double() + d) - f(gu.double() - d)) / 2e-5
    out = torch.empty((1, 16), dtype=torch.bfloat16, device=DEV)
    binding.swiglu_backward(gu.to(torch.bfloat16).to(DEV), dh.to(torch.bfloat16).to(DEV), out)
    assert torch.all((out.double().cpu() - num).abs() <= 2.0 ** -8 * num.abs() + 1e-6)


def test_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    f8 = lambda *s: torch.zeros(s, dtype=E4M3, device=DEV)
    f4 = lambda *s: torch.zeros(s, device=DEV)
    with pytest.raises(binding.LayoutError):
        binding.quantize_rows(bf(4, 24), f8(4, 24), f4(4, 1))                      # width not a multiple of 16
    with pytest.raises(ValueError):
        binding.quantize_rows(f4(4, 32), f8(4, 32), f4(4, 1))                      # not bf16
    with pytest.raises(ValueError):
        binding.quantize_rows(bf(4, 256), f8(4, 256), f4(4, 1))                    # too few scales
    with pytest.raises(ValueError):
        binding.quantize_rows(bf(4, 256), f8(4, 128), f4(4, 2))
    with pytest.raises(ValueError):
        binding.quantize_rows(bf(8, 256), f8(8, 256), f4(2, 4), col_major=True)    # ld below rows
    with pytest.raises(binding.LayoutError):
        binding.quantize_rows(bf(5, 256), f8(5, 256), f4(2, 5), col_major=True)    # ld not a multiple of 4
    with pytest.raises(ValueError):
        binding.swiglu_quantize(bf(4, 64), f8(4, 64), f4(1, 4))
    with pytest.raises(binding.LayoutError):
        binding.swiglu_backward(bf(4, 24), bf(4, 12), bf(4, 24))                   # width not a multiple of 8
    desc = binding.LayoutDesc(8, 1, 2, 1, 64)
    ws = binding.new_workspace(desc)
    i4 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)
    with pytest.raises(binding.LayoutError) as e:
        binding.quantize_cols(desc, bf(128, 64), i4(3), i4(2), f8(64, 128), f4(1, 64), ws)   # alignment 64
    assert e.value.status == 6
