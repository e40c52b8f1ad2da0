"""moe_gate_backward against the products of the gradient as it is given, fp32, with what its
rounding to bf16 may cost counted: half a step, 2^-8 of each element.

Of dX's addend: that of each product, 2^-8 sum |dz W|, an fp32 sum of E products (2^-23 of the
magnitudes an addition at most, (1 + 2^-8) of which are there), one rounding to bf16 (2^-8 of the
addend); then of the sum (2^-8 of it).  Of dW_g: the same without the two last, and one fp32 rounding.
The roundings of a sum's terms are independent of one another: the mean square of the error is at
most a third of 2^-16 times that of what is rounded (uniform over a step), with a fifth more for
the sample."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_gpu_block import randn
from tests.test_gpu_fp8 import f64, ok

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8


@pytest.mark.parametrize("T,d,E", [(1, 128, 1), (3, 256, 7), (300, 384, 97), (1000, 256, 384), (129, 128, 1024),
                                   (5000, 512, 130)])
def test_gradient_as_it_is_given(T, d, E):
    rng = np.random.default_rng(7 * T + E)
    dz = (rng.standard_normal((T, E)) * np.exp(2 * rng.standard_normal((T, 1)))).astype(np.float32)
    x, W, dX = randn(rng, 1.0, T, d), randn(rng, 0.05, E, d), randn(rng, 2.0, T, d)
    dW = torch.from_numpy(rng.standard_normal((E, d)).astype(np.float32)).cuda()
    z = dz.astype(np.float64)
    gx, mx, sx = z @ f64(W), np.abs(z) @ np.abs(f64(W)), (z ** 2) @ (f64(W) ** 2)
    gw, mw, sw = z.T @ f64(x), np.abs(z).T @ np.abs(f64(x)), (z ** 2).T @ (f64(x) ** 2)
    ws = torch.empty(_lib.moe_gate_bwd_workspace_size(T, d, E), dtype=torch.uint8, device="cuda").fill_(255)
    a, b = dX.clone(), dW.clone()
    _lib.moe_gate_backward(torch.from_numpy(dz).cuda(), x, W, T, d, E, a, b, ws)
    ok()
    want = f64(dX) + gx
    addend = HALF * mx + (E + 2) * 2.0 ** -23 * (1 + HALF) * mx
    addend += HALF * (np.abs(gx) + addend)
    off = np.abs(f64(a) - want)
    assert (off <= addend + HALF * (np.abs(want) + addend)).all()
    ww = f64(dW) + gw
    part = HALF * mw + (T + 2) * 2.0 ** -23 * (1 + HALF) * mw
    offw = np.abs(f64(b) - ww)
    assert (offw <= part + 2.0 ** -24 * (np.abs(ww) + part)).all()
    if T * d >= 4096:
        most = 1.2 * HALF ** 2 / 3
        assert np.mean(offw ** 2) <= most * np.mean(sw)
        assert np.mean(off ** 2) <= most * (np.mean(sx) + np.mean(gx ** 2) + np.mean(want ** 2))
