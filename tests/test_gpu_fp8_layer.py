"""The FP8 operators where a user meets them: MoELayer(fp8=True), its decoding
through forward_few, and GroupedLinearFP8, against plain 64-bit formulas on the
unquantised bf16 tensors.

Relative Frobenius bounds.  A value in [2^e, 2^(e+1)) has E4M3 codes 2^(e-3)
apart, so a rounding error of 2^(e-3) / sqrt(12) on average, and its mean square
is 3 / (2 ln 2) 4^e = 2.16 4^e over evenly spread exponents: q = 0.0361 /
sqrt(2.16) = 0.0245 for each quantised operand, independent of the length of the
sum.  A product of two quantised operands: sqrt(2) q = 0.035, held to 0.045.
h = silu(g) u with errors q' in g and u of unit variance is off by 1.45 q'
(E silu'^2 = 0.40, E silu^2 = 0.36).  Decoding quantises W13 and W2:
sqrt((1.45 q)^2 + q^2) = 0.043, held to 0.06; the prompt also x and h:
sqrt(2 (1.45 q)^2 + 2 q^2) = 0.061, held to 0.085."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from moe_expert_layer_04_gb300.layer import Dims, GroupedLinearFP8, MoELayer
from tests import fp8_ref as R

pytestmark = pytest.mark.gpu


def randn(rng, std, *s):
    return torch.from_numpy(rng.standard_normal(s, dtype=np.float32) * std).to(torch.bfloat16).cuda()


def n64(t):
    return t.detach().double().cpu().numpy()


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def layer_inputs(T, d, E, k, I, seed=0):
    rng = np.random.default_rng(seed)
    w = dict(W_g=randn(rng, 1.28 / d ** 0.5, E, d), W13=randn(rng, d ** -0.5, E + 1, 2 * I, d),
             W2=randn(rng, I ** -0.5, E + 1, d, I))
    bias = torch.from_numpy((rng.random((2, E)).astype(np.float32) - 0.5) * 0.1).cuda()
    return w, bias, randn(rng, 1.0, T, d)


def plain(w, bias, x, k, scaling, clamp):
    return R.few_layer(n64(x), n64(w["W_g"]), lambda e: n64(w["W13"][e]), lambda e: n64(w["W2"][e]),
                       k, scaling, clamp, None, n64(bias), None, None)[0]


@pytest.mark.parametrize("T,d,E,k,I", [(40, 256, 32, 4, 128), (200, 384, 33, 6, 256)])
def test_prompt_then_decode_from_the_same_weights(T, d, E, k, I):
    w, bias, x = layer_inputs(T, d, E, k, I)
    layer = MoELayer(Dims(T, d, E, k, I), w, scaling=2.5, fp8=True)
    y = n64(layer.forward(x, bias))
    want = plain(w, bias, x, k, 2.5, 7.0)
    assert rel(y, want) <= 0.085
    ids = layer.ids.clone()
    for n in (1, 7, 32):
        few = n64(layer.forward_few(x[:n], bias))
        assert rel(few, want[:n]) <= 0.06
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    assert torch.equal(layer.ids, ids)


def test_weights_changed_and_quantised_again():
    w, bias, x = layer_inputs(32, 256, 16, 2, 128)
    layer = MoELayer(Dims(32, 256, 16, 2, 128), w, scaling=2.5, fp8=True)
    a = n64(layer.forward(x, bias))
    w["W2"].mul_(2)
    layer.quantize_weights()
    # a power of two: every scale doubles, no code changes
    assert np.array_equal(n64(layer.forward(x, bias)), 2 * a)


def test_bf16_layer_decodes_and_other_stream():
    w, bias, x = layer_inputs(16, 256, 32, 4, 192)
    layer = MoELayer(Dims(16, 256, 32, 4, 192), w, scaling=2.5)
    y = n64(layer.forward(x, bias))
    s = torch.cuda.Stream()
    out = torch.empty(16, 256, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(s):
        got = layer.forward_few(x, bias, stream=s, y=out)
    s.synchronize()
    assert got is out
    # h and y round to bf16 in both: 1.6e-3 each (see test_gpu_few.py)
    assert rel(n64(out), y) <= 6e-3


@pytest.mark.parametrize("T,d,E,k,I,fp8", [(8, 2176, 24, 3, 64, False), (3, 128, 8, 2, 4160, False),
                                           (16, 640, 64, 6, 256, True)])
def test_decoding_repeats_bit_for_bit(T, d, E, k, I, fp8):
    """Tiles of three and more stages too: who multiplies which of them must not
    show (items go to CTAs as they come)."""
    w, bias, x = layer_inputs(T, d, E, k, I)
    layer = MoELayer(Dims(T, d, E, k, I), w, scaling=2.5, fp8=fp8)
    first = layer.forward_few(x, bias).clone()
    for _ in range(40):
        assert torch.equal(layer.forward_few(x, bias), first)


@pytest.mark.parametrize("G,N,K,cuts", [(1, 128, 256, [0, 300]), (3, 208, 400, [0, 129, 129, 257]),
                                        (4, 512, 128, [0, 1, 130, 130, 131])])
def test_grouped_projection_and_its_gradients(G, N, K, cuts):
    rng = np.random.default_rng(G * 1000 + N)
    weight, rows = randn(rng, K ** -0.5, G, N, K), cuts[-1]
    layer = GroupedLinearFP8(weight, rows + 5)
    x, dy = randn(rng, 1.0, rows, K), randn(rng, 1.0, rows, N)
    offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    y = n64(layer.forward(x, offsets))
    dx = n64(layer.backward(dy))
    dW = n64(layer.dW)
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    W, X, D = n64(weight), n64(x), n64(dy)
    for g, (a, b) in enumerate(zip(cuts, cuts[1:])):
        if a == b:
            assert not dW[g].any()
            continue
        assert rel(y[a:b], X[a:b] @ W[g].T) <= 0.045
        assert rel(dx[a:b], D[a:b] @ W[g]) <= 0.045
        assert rel(dW[g], D[a:b].T @ X[a:b]) <= 0.045
    # the gradient against differences: the loss sum(y D) is linear in the weight,
    # so a step along dW changes it by |dW|^2 up to the same errors
    step = randn(rng, 1.0, G, N, K)
    change = sum(np.sum(D[a:b] * (X[a:b] @ n64(step[g]).T))
                 for g, (a, b) in enumerate(zip(cuts, cuts[1:])))
    # a sum of independent terms: the error is 0.035 of |dW| along a random direction
    assert abs(np.sum(dW * n64(step)) - change) <= 5 * 0.035 * np.linalg.norm(dW)


def test_no_rows():
    layer = GroupedLinearFP8(torch.ones(2, 32, 48, dtype=torch.bfloat16, device="cuda"), 4)
    x = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    assert layer.forward(x, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 32)
    assert layer.backward(torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")).shape == (0, 48)
    assert not layer.dW.any()


def test_example_runs():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "fp8_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_layer_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    gen = torch.Generator(device="cuda").manual_seed(1)
    # two layers that differ by their quantisation (1.3 times unit variance into
    # the SwiGLU) and by the tokens whose routing is the same in both
    first, decoded = ex.serve(gen)
    assert first <= 0.1 and decoded <= 0.075
    # quantised operands leave 0.035 of the outputs' norm, squared; the rest of the
    # loss shrinks by the steps
    a, b = ex.train(gen)
    assert b < 0.5 * a
