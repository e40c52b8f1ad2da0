"""Shares of tokens all of whose logits are far below zero: sigmoids that fp32 holds as
subnormals or not at all, whose shares are ordinary numbers all the same.

Roundings: those of tests/test_gpu_balance.py, with z - max z (rounded once, 2^-24 of itself) as an
exponential's argument where the shares are taken so, which its bound of 2^-21 (1 + |argument| / 4)
holds."""
import numpy as np
import pytest

from tests import test_gpu_balance as B
from tests.test_gpu_fp8 import f64, ok

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min
LOW = [-20.0, -45.0, -85.0, -92.0, -95.0, -100.0, -103.0, -104.0, -200.0, -1e4, LOWEST]


def shares(z, score):
    """The shares in 64 bits, of any finite logits: the row's largest sigmoid taken out of them."""
    assert score == B.SIG
    with np.errstate(over="ignore", invalid="ignore"):
        top = z.max(1, keepdims=True)
        s = np.exp(z - np.where(np.isneginf(top), 0.0, top)) / (1 + np.exp(z))
        tot = s.sum(1, keepdims=True)
        return np.where(tot > 0, s / tot, 0.0), 1 / (1 + np.exp(z))


@pytest.fixture(autouse=True)
def _stable(monkeypatch):
    monkeypatch.setattr(B, "shares", shares)


def rows(rng, T, E, k):
    """Rows of one value, of one value and minus infinity, spread around one, and ordinary ones."""
    z, ids = B.inputs(rng, T, E, k)
    for t in range(T):
        low, kind = LOW[t // 4 % len(LOW)], t % 4
        if kind == 0:
            z[t] = low
        elif kind == 1:
            z[t] = low
            z[t, rng.permutation(E)[:E // 3]] = -np.inf
        elif kind == 2:
            z[t] = np.maximum(low + 2 * rng.standard_normal(E), LOWEST)
    z[3] = -np.inf
    return z, ids


# (a CTA for all tokens; many; rows of 4 E bytes that are whole vectors and ones that are not)
@pytest.mark.parametrize("T,E,k", [(44, 16, 2), (88, 40, 4), (120, 97, 3), (500, 16, 2), (700, 384, 6),
                                   (300, 130, 2), (200, 1023, 5)])
def test_shares_of_low_logits(T, E, k):
    rng = np.random.default_rng(T + E)
    z, ids = rows(rng, T, E, k)
    offs = np.array([0, T // 3, T], np.int32)
    a = B.call(z, ids, B.SIG, offs, dloss=np.array([0.6], np.float32))
    ok()
    for n in ("loss", "seq_loss", "dlogits"):
        assert np.isfinite(f64(a[n])).all(), n
    r = B.reference(z.astype(np.float64), ids, B.SIG, offs, dloss=float(np.float32(0.6)))
    assert (f64(a["dlogits"])[3] == 0).all()
    # (the lowest value and -1e4 are no arguments of an exponential: their differences are)
    B.check(a, r, np.where(np.abs(z) > 250, 0.0, z))


@pytest.mark.parametrize("value", LOW)
def test_equal_logits_have_equal_shares(value):
    """Every share 1 / E, so that the sequence's loss is the mean load, 1."""
    T, E = 150, 24
    z = np.full((T, E), value, np.float32)
    ids = (np.arange(2 * T).reshape(T, 2) % E).astype(np.int32)   # 300 slots over 24 experts
    a = B.call(z, ids, B.SIG)
    ok()
    r = B.reference(z.astype(np.float64), ids, B.SIG)
    assert abs(r["seq_loss"][0] - 1) < 1e-12
    B.check(a, r, np.where(np.abs(z) > 250, 0.0, z))


@pytest.mark.parametrize("E", [16, 97, 384])
def test_rows_on_the_border_count_once(E):
    """Scores whose sum is about the one from which shares are taken relative to the largest
    (2^-20), spread over some of fp32's steps around it: every row once."""
    T, k = 1500, 2
    mid = np.float32(np.log(2.0 ** -20 / E))
    z = (mid + np.float32(2.0 ** -19) * np.arange(-T // 2, T - T // 2, dtype=np.float32))[:, None]
    z = np.repeat(z, E, 1) + np.float32(2.0 ** -19) * np.random.default_rng(E).integers(-3, 4, (T, E)).astype(np.float32)
    ids = (np.arange(k * T).reshape(T, k) % E).astype(np.int32)
    a = B.call(z, ids, B.SIG)
    ok()
    B.check(a, B.reference(z.astype(np.float64), ids, B.SIG), z)
