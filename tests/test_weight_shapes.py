"""Weights are quantised once their shape is the one that the calls read, on the CPU: the library's
calls only write down what they are given."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L
from tests.test_block_layer_checks import D, E, I, build, calls, weights  # noqa: F401

BF16 = torch.bfloat16


@pytest.mark.parametrize("kind", ["fp8", "mx", "mx4"])
@pytest.mark.parametrize("bad", [dict(W13=torch.zeros(E, 2 * I, D, dtype=BF16)),
                                 dict(W13=torch.zeros(E + 1, I, D, dtype=BF16)),
                                 dict(W2=torch.zeros(E + 1, D, I - 8, dtype=BF16))])
def test_layer(calls, kind, bad):  # noqa: F811
    with pytest.raises(ValueError):
        build(weights(**bad), **{kind: True})
    assert not [c for c in calls if "quantize" in c[0]]
    m = build(**{kind: True})
    m.w.update(bad)
    calls.clear()
    with pytest.raises(ValueError):
        m.quantize_weights()
    assert not calls


def test_projections(calls, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_lib, "moe_fp8_wgrad_workspace_size", lambda *a: 16)
    w = torch.zeros(3, 48, 128, dtype=BF16)
    for p in (L.GroupedLinearMX4(w, 8), L.GroupedLinearFP8(w, 8)):
        calls.clear()
        p.weight = torch.zeros(3, 40, 128, dtype=BF16)
        with pytest.raises(ValueError):
            p.quantize_weights()
        assert not calls
        p.weight = torch.ones(3, 48, 128, dtype=BF16)
        p.quantize_weights()
        assert len(calls) == 1
