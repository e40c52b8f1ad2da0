"""Shapes that the norm or the balance loss's backward do not take are refused when the layer is
built, not at its first call."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

BF16 = torch.bfloat16


def build(T, d, E, k, I, **kw):
    """(No memory behind the tensors: nothing is launched.)"""
    z = lambda *s, t=BF16: torch.empty(*s, dtype=t, device="meta")
    w = dict(W_g=z(E, d), W13=z(E + 1, 2 * I, d), W2=z(E + 1, d, I), norm=z(d, t=torch.float32))
    return L.MoELayer(L.Dims(T, d, E, k, I), w, 2.5, device="meta", **kw)


def test_norm():
    with pytest.raises(ValueError):
        build(8, 65536, 32, 2, 128, norm_eps=1e-6)
    build(8, 32768, 32, 2, 128, norm_eps=1e-6)
    build(8, 65536, 32, 2, 128)


def test_balance_backward():
    T = 1 << 21
    with pytest.raises(ValueError):
        build(T, 128, 8, 2, 128, backward=True, balance=1e-3)
    build(T, 128, 8, 2, 128, balance=1e-3)
    build(T - 1, 128, 8, 2, 128, backward=True, balance=1e-3)
    assert _lib.moe_gate_bwd_workspace_size(T, 128, 8) == 0
