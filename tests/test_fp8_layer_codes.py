"""MoELayer(fp8=True) from weights that are FP8 codes and block scales already, as a
checkpoint holds them."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

T, D, E, K, I = 24, 256, 12, 3, 384


def codes(device="cpu"):
    u8, f32 = dict(dtype=torch.uint8, device=device), dict(device=device)
    return dict(W_g=torch.zeros(E, D, dtype=torch.bfloat16, device=device),
                W13_q=torch.zeros(E + 1, 2 * I, D, **u8), W13_s=torch.zeros(E + 1, 2 * I // 128, D // 128, **f32),
                W2_q=torch.zeros(E + 1, D, I, **u8), W2_s=torch.zeros(E + 1, D // 128, I // 128, **f32))


def build(w, device="cpu"):
    return L.MoELayer(L.Dims(T, D, E, K, I), w, scaling=2.5, fp8=True, device=device)


def test_codes_are_taken_as_they_are():
    w = codes()
    m = build(w)
    assert all(getattr(m, n) is w[n] for n in ("W13_q", "W13_s", "W2_q", "W2_s"))
    with pytest.raises(RuntimeError):
        m.quantize_weights()           # from nothing
    w["W2_q"] = w["W2_q"].view(torch.float8_e4m3fn)
    m = build(w)
    assert m.W2_q.dtype == torch.uint8 and m.W2_q.data_ptr() == w["W2_q"].data_ptr()


@pytest.mark.parametrize("change", [
    dict(W13_s=None), dict(W2_q=None), dict(W13=torch.zeros(E + 1, 2 * I, D, dtype=torch.bfloat16)),
    dict(W13_q=torch.zeros(E, 2 * I, D, dtype=torch.uint8)),
    dict(W2_s=torch.zeros(E + 1, D // 128, I // 64)),
    dict(W2_s=torch.zeros(E + 1, D // 128, I // 128, dtype=torch.float64)),
    dict(W13_q=torch.zeros(E + 1, 2 * I, D, dtype=torch.int8))])
def test_other_codes_are_refused(change):
    w = {n: t for n, t in {**codes(), **change}.items() if t is not None}
    with pytest.raises(ValueError):
        build(w)


@pytest.mark.gpu
def test_same_results_as_from_the_weights_they_stand_for():
    from tests.test_gpu_fp8_layer import layer_inputs
    w, bias, x = layer_inputs(T, D, E, K, I)
    a = build(w, "cuda")
    b = build(dict(W_g=w["W_g"], W13_q=a.W13_q.view(torch.float8_e4m3fn), W13_s=a.W13_s,
                   W2_q=a.W2_q, W2_s=a.W2_s), "cuda")
    assert torch.equal(a.forward(x, bias), b.forward(x, bias))
    for n in (1, 5, T):
        assert torch.equal(a.forward_few(x[:n], bias), b.forward_few(x[:n], bias))
    assert _lib.moe_last_device_status() == _lib.MOE_OK
