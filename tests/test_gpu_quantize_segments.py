"""Columns quantised over segments that a caller laid out: a block of 128 rows belongs to one expert, or the call says so."""
from __future__ import annotations

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


@pytest.mark.parametrize("offsets,counts", [([0, 200, 456], [200, 256]), ([64, 192, 320], [128, 128]),
                                            ([0, 0, 128, 130], [0, 128, 2])])
def test_a_segment_off_the_block_grid_is_reported(offsets, counts):
    """A start that is no multiple of 128 is recorded and nothing is written, as the weight gradient would refuse it."""
    bad = any(o % 128 for o in offsets[:-1])
    cap, cols = 512, 72
    x = torch.randn((cap, cols), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    q = torch.full((cols, cap), 0x33, dtype=torch.uint8, device=DEV)
    sf = torch.full((cap // 128, cols), -2.0, device=DEV)
    desc = binding.LayoutDesc(sum(counts), 1, len(counts), 1, 128)
    ws = binding.new_workspace(desc)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    binding.quantize_cols(desc, x, i32(offsets), i32(counts), q.view(torch.float8_e4m3fn), sf, ws)
    assert binding.get_error(ws) == (1 if bad else 0)
    if bad:
        assert torch.all(q == 0x33) and torch.all(sf == -2.0)
    else:
        assert not torch.any(sf[0] == -2.0)
