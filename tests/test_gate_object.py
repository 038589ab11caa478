"""What a Gate object keeps between calls stays what its calls use.  No GPU: the buffers are host memory, nothing is launched."""
import types

import pytest
import torch

from counting_sort_bucketization_gb300 import binding, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.load_library()


def _gate(desc=binding.LayoutDesc(4, 2, 8, 1, 1)):
    return binding.Gate(desc, binding.GateConfig("sigmoid", True, 1.5, 0.1), device="cpu")


@pytest.mark.parametrize("name", ["topk_idx", "weights", "expert_count", "prob_mean", "routed_tokens", "loss", "workspace"])
def test_buffers_cannot_be_rebound(name):
    """forward() writes to the addresses taken when the object was made."""
    gate = _gate()
    kept = getattr(gate, name)
    with pytest.raises(AttributeError):
        setattr(gate, name, torch.empty_like(kept))
    assert getattr(gate, name) is kept
