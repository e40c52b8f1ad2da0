"""MoELayer.dispatch(): the codes that move are the ones that it is given, never those of an
earlier call that happened to write the same tensor."""
import pytest
import torch

from moe_expert_layer_04_gb300 import layer as L
from tests.test_block_layer_checks import T, build, calls, names, rows  # noqa: F401

KINDS = ["fp8", "mx", "mx4"]


@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_codes_are_quantised(calls, kind):  # noqa: F811
    m = build(norm_eps=1e-6, **{kind: True})
    xn, _ = m.norm(rows(T))
    xn.mul_(0.5)                       # rows that the norm's codes are not those of
    calls.clear()
    m.dispatch(xn)
    assert names(calls) == ["moe_permute", "moe_fp8_gather" if kind == "fp8" else "moe_mx_gather"]
    calls.clear()
    m.dispatch(xn, codes=(m.xn_q, m.xn_s))
    assert names(calls) == ["moe_permute", "moe_gather_rows", "moe_gather_rows"]
    assert calls[1][1][0] is m.xn_q and calls[2][1][0] is m.xn_s


@pytest.mark.parametrize("kind", KINDS)
def test_codes_of_another_shape(calls, kind):  # noqa: F811
    m = build(norm_eps=1e-6, **{kind: True})
    calls.clear()
    for q, s in ((m.xn_q[:-1], m.xn_s), (m.xn_q, m.xn_s[:, :-1]), (m.xn_q[:, :-16], m.xn_s),
                 (m.xn_q, m.xn_s.to(torch.float64))):
        with pytest.raises(ValueError):
            m.dispatch(rows(T), codes=(q, s))
    assert not calls
    plain = build()
    calls.clear()
    with pytest.raises(ValueError):
        plain.dispatch(rows(T), codes=(m.xn_q, m.xn_s))
    assert not calls


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_rows_changed_behind_the_norm(kind):
    """The steps of forward() one by one, with rows that were changed between norm and dispatch:
    the layer without a norm on those rows."""
    from tests.test_gpu_block import block
    from tests.test_gpu_fp8 import ok
    T, d, E, k, I = 130, 512, 32, 4, 128
    layer, w, bias, x, res = block(T, d, E, k, I, **{kind: True})
    bare = L.MoELayer(L.Dims(T, d, E, k, I), w, 2.5, **{kind: True})
    xn, _ = layer.norm(x, res)
    xn.copy_(xn.roll(1, 0))
    layer.route(xn, bias)
    layer.dispatch(xn)
    layer.experts()
    layer.combine()
    want = bare.forward(xn, bias)
    ok()
    assert torch.equal(layer.y, want)
    layer.norm(x, res)
    layer.route(layer.xn, bias)
    layer.dispatch(layer.xn, codes=(layer.xn_q, layer.xn_s))
    layer.experts()
    layer.combine()
    by_steps = layer.y.clone()
    assert torch.equal(layer.forward(x, bias, residual=res), by_steps)
    ok()
