"""Expert products and weight gradients of many more tiles than the grid has CTAs, so that each walks several: whatever is
carried from one tile to the next (buffer positions, scales fetched ahead, blocks of results still being stored) counts.
Tolerances as in test_gpu_expert_gemm.py, whose cases and checks these are."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build
from test_gpu_expert_gemm import check_forward, check_wgrad, forward_case, run_forward, run_wgrad, wgrad_case

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def ragged(n, lo, hi, seed):
    return [int(v) for v in np.random.default_rng(seed).integers(lo, hi + 1, n)]


@pytest.mark.parametrize("counts,A,wi,wo", [
    (ragged(24, 130, 700, 1), 16, 400, 2056),              # pairs of CTAs: 4 k-blocks, ~480 tiles, whole and partial quarters
    (ragged(12, 0, 900, 2), 128, 896, 3000),    # 7 k-blocks
    (ragged(40, 100, 300, 3), 1, 128, 2048),               # one k-block a tile
    (ragged(200, 0, 100, 4), 16, 400, 520),                # one CTA a tile: ~1000 tiles
    (ragged(64, 1, 90, 5), 1, 1040, 1032),
], ids=["pair4", "pair7", "pair1", "single4", "single9"])
def test_products_of_many_tiles(counts, A, wi, wo):
    c = forward_case(counts, A, wi, wo, wi + wo, 5)
    assert run_forward(c) == 0
    check_forward(c, counts)
    first = c["out"].clone()
    for _ in range(3):
        c["out"].fill_(3.0)
        assert run_forward(c) == 0
        assert torch.equal(first.view(torch.int16), c["out"].view(torch.int16))


def _some_empty(counts):
    return [0 if i % 5 == 2 else n for i, n in enumerate(counts)]


@pytest.mark.parametrize("kind", ["bf16", "fp32", "added"])
@pytest.mark.parametrize("counts,wo,wi", [
    (_some_empty(ragged(16, 1, 900, 6)), 1040, 1288),      # 480 tiles of 0 to 8 k-blocks
    (_some_empty(ragged(30, 1, 128, 7)), 520, 776),        # at most one k-block a tile
], ids=["k8", "k1"])
def test_weight_gradients_of_many_tiles(counts, wo, wi, kind):
    c = wgrad_case(counts, 128, wo, wi, wo + wi, 3, torch.bfloat16 if kind == "bf16" else torch.float32)
    added = kind == "added"
    assert run_wgrad(c, accumulate=added) == 0
    check_wgrad(c, counts, base=5.0 if added else 0.0)
    first = c["dw"].clone()
    for _ in range(3):
        c["dw"].fill_(5.0)
        assert run_wgrad(c, accumulate=added) == 0
        assert torch.equal(first, c["dw"])


def test_an_added_gradient_leaves_experts_without_rows_alone():
    """Bit for bit: signed zeros, values below the normal range, infinities."""
    counts = [0, 200, 0, 3, 0]
    c = wgrad_case(counts, 128, 264, 520, 8)
    held = torch.randint(-2 ** 31, 2 ** 31 - 1, c["dw"].shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV,
                         dtype=torch.int32)
    held[0] &= -0x7f800001                                 # all below the normal range
    held[2, ::2] = -2 ** 31                                # -0.0
    empty = [0, 2, 4]
    c["dw"].view(torch.int32)[empty] = held[empty]
    assert run_wgrad(c, accumulate=True) == 0
    assert torch.equal(c["dw"].view(torch.int32)[empty], held[empty])
    c["dw"][empty] = 5.0
    check_wgrad(c, counts, base=5.0)
