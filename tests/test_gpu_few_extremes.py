"""The few-token layer on tokens and weights at the ends of their ranges.  Routing is
pinned (a table, or a zero gate), so that a token's result depends on nothing but
itself: what is not touched stays bit for bit."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_gpu_few import check, make, run

pytestmark = pytest.mark.gpu

SHAPES = [(1, 256, 6, 2, 128), (4, 384, 5, 3, 192), (13, 256, 3, 1, 320), (32, 128, 16, 4, 64)]


def table(E, k):
    return lambda rng, v: np.argsort(rng.random((v, E)), 1)[:, :k]


def result(a):
    a["y"].fill_(3.0)
    run(a)
    return a["y"][:a["T"]].clone()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,I", SHAPES)
@pytest.mark.parametrize("power", [100, 60, -60, -80])
def test_powers_of_two_cancel(T, d, E, k, I, fp8, power):
    """Tokens times 2^p and W13 times 2^-p give the same h: every step is exact."""
    a = make(T, d, E, k, I, fp8)
    a["W_g"].zero_()             # the logits stay what logit_offset says
    want = result(a)
    a["x"] = a["x"] * 2.0 ** power
    if fp8:
        a["W13_s"] = a["W13_s"] * 2.0 ** -power
    else:
        a["W13"] = a["W13"] * 2.0 ** -power
    assert torch.equal(result(a), want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,I", SHAPES)
def test_tiny_tokens(T, d, E, k, I, fp8):
    """2^-110: below what the f16 rows are scaled up to entirely (values under 2^-9 of the
    largest lose bits, at most 2^-17 of it); still within the bounds."""
    a = make(T, d, E, k, I, fp8)
    a["W_g"].zero_()
    a["x"] = a["x"] * 2.0 ** -110
    a["W13_s" if fp8 else "W13"] = a["W13_s" if fp8 else "W13"] * 2.0 ** 110
    run(a)
    check(a)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_token_of_very_different_values(fp8):
    a = make(3, 512, 6, 2, 192, fp8)
    x = a["x"].float()
    x[:, ::3] *= 2.0 ** -30
    x[:, 1::7] *= 2.0 ** -12
    x[1] *= 2.0 ** 20
    a["x"] = x.to(torch.bfloat16)
    a["W_g"].zero_()
    run(a)
    check(a)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,d,E,k,I", SHAPES[1:])
def test_what_is_not_finite_stays_with_its_token(T, d, E, k, I, value, fp8):
    a = make(T, d, E, k, I, fp8, hash_table=table(E, k))
    clean = result(a)
    bad = T // 2
    a["x"][bad, d // 3] = value
    got = result(a)
    assert torch.isnan(got[bad].float()).all()
    keep = [t for t in range(T) if t != bad]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,I", SHAPES[1:])
def test_zero_tokens(T, d, E, k, I, fp8):
    a = make(T, d, E, k, I, fp8, hash_table=table(E, k))
    clean = result(a)
    a["x"][::2] = 0
    got = result(a)
    assert (got[::2] == 0).all() and torch.equal(got[1::2], clean[1::2])


@pytest.mark.parametrize("name", ["W13_s", "W2_s", "W13_q", "W2_q", "W13", "W2"])
def test_nan_weights_reach_their_experts_tokens_only(name):
    T, E, k = 13, 7, 2
    a = make(T, 256, E, k, 192, name[-2:] in ("_s", "_q"), hash_table=table(E, k))
    clean = result(a)
    expert = 3
    a[name][expert].view(-1)[0 if name.startswith("W2") else 5] = 0x7F if name.endswith("_q") else float("nan")
    got = result(a)
    hit = (a["ids"] == expert).any(1)
    assert hit.any() and not hit.all()
    assert torch.equal(got[~hit], clean[~hit])
    assert torch.isnan(got[hit].float()).any(1).all()
    a[name][E].view(-1)[0] = 0x7F if name.endswith("_q") else float("nan")   # the shared one
    assert torch.isnan(result(a).float()).any(1).all()
    # `run` raises no status: numbers that are not finite are no error
    assert _lib.moe_last_device_status() == _lib.MOE_OK
