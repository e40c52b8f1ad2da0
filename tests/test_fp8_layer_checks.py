"""Checks that the layer's classes make before a call, on the CPU: the library's calls
are replaced by ones that write down what they are given."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

BF16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in ("moe_fp8_quantize_weights", "moe_fp8_quantize", "moe_fp8_matmul", "moe_fp8_wgrad",
                 "moe_layer_few"):
        monkeypatch.setattr(_lib, name, lambda *a, _n=name, **k: made.append((_n, a, k)))
    return made


G, N, K, ROWS = 3, 48, 64, 20


def projection(calls):
    p = L.GroupedLinearFP8(torch.zeros(G, N, K, dtype=BF16), ROWS)
    calls.clear()
    return p


def rows(r, c):
    return torch.zeros(r, c, dtype=BF16)


OFFS = torch.zeros(G + 1, dtype=torch.int32)


def test_projection_takes_what_its_buffers_hold(calls):
    p = projection(calls)
    for r in (1, ROWS):
        assert p.forward(rows(r, K), OFFS).shape == (r, N)
        assert p.backward(rows(r, N)).shape == (r, K)
    assert len(calls) == 10


@pytest.mark.parametrize("x,offsets", [
    (rows(ROWS + 1, K), OFFS),                       # more rows than the buffers
    (rows(4, K - 16), OFFS), (rows(4, K + 16), OFFS),
    (torch.zeros(4 * K, dtype=BF16), OFFS),
    (rows(4, K), OFFS[:G]), (rows(4, K), torch.zeros(G + 2, dtype=torch.int32))])
def test_projection_refuses_rows(calls, x, offsets):
    p = projection(calls)
    with pytest.raises(ValueError):
        p.forward(x, offsets)
    assert not calls


@pytest.mark.parametrize("dy", [rows(5, N), rows(3, N), rows(ROWS + 1, N), rows(4, K), rows(0, N),
                                torch.zeros(4 * N, dtype=BF16)])
def test_projection_refuses_gradients_of_other_rows(calls, dy):
    p = projection(calls)
    p.forward(rows(4, K), OFFS)
    calls.clear()
    with pytest.raises(ValueError):
        p.backward(dy)
    assert not calls


def test_projection_refuses_a_gradient_before_a_forward(calls):
    p = projection(calls)
    with pytest.raises(RuntimeError):
        p.backward(rows(4, N))
    # a forward that was refused leaves the one before in place
    p.forward(rows(4, K), OFFS)
    with pytest.raises(ValueError):
        p.forward(rows(ROWS + 1, K), OFFS)
    assert p.backward(rows(4, N)).shape == (4, K)


D, E, KK, I = 128, 8, 2, 64


@pytest.fixture
def decoder(calls):
    """A bf16 layer as far as forward_few needs one."""
    m = L.MoELayer.__new__(L.MoELayer)
    m.dims = L.Dims(16, D, E, KK, I)
    m.mx = m.fp8 = False
    m.scaling, m.clamp = 2.5, 7.0
    m.w = dict(W_g=rows(E, D), W13=None, W2=None)
    m._few_workspace = lambda *a: torch.zeros(8, dtype=torch.uint8)
    return m


def few_args(T=4, vocab=10, **kw):
    a = dict(x=rows(T, D), bias=torch.zeros(2, E), is_vision=torch.zeros(T, dtype=torch.uint8),
             logit_offset=torch.zeros(E), y=rows(T, D))
    a.update(kw)
    return a


HASH = dict(mode=_lib.MOE_ROUTE_HASH, bias=None, input_ids=torch.zeros(4, dtype=torch.int32),
            tid2eid=torch.zeros(10, KK, dtype=torch.int32))


@pytest.mark.parametrize("kw", [{}, HASH, dict(is_vision=None, logit_offset=None, y=None)])
def test_decoding_takes(decoder, calls, kw):
    assert decoder.forward_few(**few_args(**kw)).shape == (4, D)
    assert [c[0] for c in calls] == ["moe_layer_few"]


@pytest.mark.parametrize("kw", [
    dict(x=rows(4, D // 2)), dict(x=rows(4, 2 * D)), dict(x=torch.zeros(D, dtype=BF16)),
    dict(y=rows(3, D)), dict(y=rows(4, D - 1)), dict(bias=torch.zeros(E)), dict(bias=torch.zeros(2, E - 1)),
    dict(is_vision=torch.zeros(3, dtype=torch.uint8)), dict(logit_offset=torch.zeros(E - 1)),
    dict(HASH, input_ids=torch.zeros(3, dtype=torch.int32)),
    dict(HASH, tid2eid=torch.zeros(10, KK + 1, dtype=torch.int32)),
    dict(HASH, tid2eid=torch.zeros(10 * KK, dtype=torch.int32))])
def test_decoding_refuses_other_shapes(decoder, calls, kw):
    with pytest.raises(ValueError):
        decoder.forward_few(**few_args(**kw))
    assert not calls
