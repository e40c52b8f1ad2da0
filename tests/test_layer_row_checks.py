"""MoELayer refuses token rows and results that hold fewer elements than its T, which
the library would read or write past (on the CPU: the calls only write down their
names)."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

BF16 = torch.bfloat16
T, D, E, K, I = 8, 256, 32, 2, 128


@pytest.fixture(params=["bf16", "fp8", "mx"])
def built(request, monkeypatch):
    made = []
    for name in _lib.EXPORTS:
        if name.endswith("_size") or name in ("moe_fp8_scale_cols", "moe_mx_sf_pitch"):
            continue
        if hasattr(_lib, name):
            monkeypatch.setattr(_lib, name, lambda *a, _n=name, **k: made.append(_n))
    w = dict(W_g=torch.zeros(E, D, dtype=BF16), W13=torch.zeros(E + 1, 2 * I, D, dtype=BF16),
             W2=torch.zeros(E + 1, D, I, dtype=BF16))
    kind = request.param
    m = L.MoELayer(L.Dims(T, D, E, K, I), w, 2.5, device="cpu", fp8=kind == "fp8", mx=kind == "mx",
                   backward=kind != "fp8")
    made.clear()
    return m, made


def rows(n):
    return torch.zeros(n, D, dtype=BF16)


BIAS = torch.zeros(2, E)


def test_enough_rows_run(built):
    m, made = built
    for n in (T, T + 3):          # rows past T are not used
        m.forward(rows(n), BIAS, y=rows(T))
    assert len(made) >= 8
    if m.backward_enabled:
        m.backward(rows(T))


@pytest.mark.parametrize("n", [0, 1, T - 1])
def test_too_few_rows_are_refused(built, n):
    m, made = built
    with pytest.raises(ValueError):
        m.forward(rows(n), BIAS)
    with pytest.raises(ValueError):
        m.route(rows(n), BIAS)
    with pytest.raises(ValueError):
        m.dispatch(rows(n))
    with pytest.raises(ValueError):
        m.combine(y=rows(n))
    with pytest.raises(ValueError):
        m.forward(rows(T), BIAS, y=rows(n))
    made.clear()
    if m.backward_enabled:
        m.forward(rows(T), BIAS)
        made.clear()
        with pytest.raises(ValueError):
            m.backward(rows(n))
    assert not made
