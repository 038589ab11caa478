"""The norm with the smallest and largest eps, beside rows whose squares overflow or vanish in 32 bits.

Tolerances as for other rows (85 additions of positive terms and a few roundings: 2^-17 of r; a bf16 value 2^-8 and
2^-16): squares that vanish lie below 2^-149, 2^-23 of the smallest eps, which is 2^-24 of r; the largest is 2^-25 of a mean
whose sum overflows, 2^113 at 32768 columns.  A normed value below 2^-126 is rounded to a multiple of 2^-133.
"""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("cols", [64, 1024, 1040, 7168, 16400])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-6, 1.0, 1e20, 2.0 ** 88])
def test_rows_of_every_scale(cols, eps):
    scales = [-120, -90, -76, -74, -70, -64, -60, -50, -49, -40, 0, 40, 60, 63, 64, 70, 120]
    g = torch.Generator(device=DEV).manual_seed(cols)
    x = (torch.randn((len(scales) + 1, cols), generator=g, device=DEV).clamp(-4, 4)
         * torch.tensor([2.0 ** s for s in scales] + [0.0], device=DEV)[:, None]).to(BF16)
    w = (torch.randn(cols, generator=g, device=DEV) * 0.3 + 1).to(BF16)
    y, rstd = torch.empty_like(x), torch.empty(len(x), device=DEV)
    binding.rms_norm(x, w, y=y, rstd=rstd, eps=eps)
    z, e = x.double(), float(torch.tensor(eps))
    r = (z.square().mean(1) + e).rsqrt()
    assert torch.all((rstd.double() - r).abs() <= 2.0 ** -17 * r)
    v = z * r[:, None] * w.double()
    assert torch.all((y.double() - v).abs() <= (2.0 ** -8 + 2.0 ** -16) * v.abs() + 2.0 ** -133)
