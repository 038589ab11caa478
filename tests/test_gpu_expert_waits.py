"""Expert products whose first stage never completes (moe_debug_set_waits): every kind gives up, waits for the copies that are
on their way, not for what cannot come, and the next call works.  A wait lasts one limit; the load warp's is followed by one
for the stage that the hook spoils, so the kernel ends within a few limits, however many tiles and stages it has."""
from __future__ import annotations

import time

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build
from test_gpu_expert_gemm import check_forward, check_wgrad, forward_case, run_forward, run_wgrad, wgrad_case

pytestmark = pytest.mark.gpu

TIMEOUT = 5
LIMIT_S = 0.05


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


@pytest.fixture(autouse=True)
def _normal_waits_after():
    yield
    binding.debug_set_waits()


def gives_up(run):
    binding.debug_set_waits(limit_ns=int(LIMIT_S * 1e9), extra_tx=16)
    torch.cuda.synchronize()
    start = time.perf_counter()
    assert run() == TIMEOUT
    took = time.perf_counter() - start
    binding.debug_set_waits()
    return took


@pytest.mark.parametrize("counts,wi,wo", [([20, 9], 2048, 4096), ([100, 128, 7] * 40, 1040, 520), ([600, 300, 513], 2048, 2056),
                                          ([40], 7168, 256)], ids=["single", "single-many", "pair", "shared"])
def test_products_give_up_within_a_few_limits(counts, wi, wo):
    c = forward_case(counts, 16, wi, wo, 2)
    assert run_forward(c) == 0
    assert gives_up(lambda: run_forward(c)) < 4 * LIMIT_S
    c["out"].fill_(3.0)
    assert run_forward(c) == 0
    check_forward(c, counts)


@pytest.mark.parametrize("dtype,added", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True)])
@pytest.mark.parametrize("counts", [[130, 0, 900], [1100]])
def test_weight_gradients_give_up_within_a_few_limits(counts, dtype, added):
    c = wgrad_case(counts, 128, 520, 776, 3, 0, dtype)
    assert run_wgrad(c, accumulate=added) == 0
    assert gives_up(lambda: run_wgrad(c, accumulate=added)) < 4 * LIMIT_S
    c["dw"].fill_(5.0)
    assert run_wgrad(c, accumulate=added) == 0
    check_wgrad(c, counts, base=5.0 if added else 0.0)
