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


@pytest.mark.parametrize("name,value", [("cfg", binding.GateConfig("softmax")), ("desc", binding.LayoutDesc(4, 1, 8, 1, 1))])
def test_settings_cannot_be_replaced(name, value):
    gate = _gate()
    kept = getattr(gate, name)
    with pytest.raises(AttributeError):
        setattr(gate, name, value)
    assert getattr(gate, name) is kept


def test_both_directions_use_the_settings_of_the_object(monkeypatch):
    """A description that its owner changes later changes neither direction."""
    calls = {}
    fake = types.SimpleNamespace(moe_gate_forward=lambda d, c, *a: calls.update(forward=(d, c)) or 0,
                                 moe_gate_backward=lambda d, c, *a: calls.update(backward=(d, c)) or 0)
    desc = types.SimpleNamespace(num_tokens=4, topk=2, num_experts=8, num_ranks=1, alignment=1)
    gate = _gate(desc)
    desc.topk = 1
    monkeypatch.setattr(binding, "load_library", lambda: fake)
    monkeypatch.setattr(binding, "_matrix", lambda t, name, rows, cols, dtypes: (t.data_ptr(), cols))
    monkeypatch.setattr(binding, "_dev", lambda t, *a, **k: None if t is None else t.data_ptr())
    monkeypatch.setattr(binding, "_stream", lambda s: 0)
    logits = torch.zeros((4, 8))
    gate.forward(logits)
    gate.backward(logits, torch.zeros_like(logits))
    values = lambda ref: [getattr(ref._obj, f) for f, _ in ref._obj._fields_]
    for a, b in zip(calls["forward"], calls["backward"]):
        assert values(a) == values(b)
    assert values(calls["backward"][0]) == [4, 2, 8, 1, 1]
    assert values(calls["backward"][1])[:3] == [0, 1, 1]
