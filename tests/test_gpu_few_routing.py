"""Routing of the few-token layer against the other routing calls' rule: scores are
the sigmoid rounded once to fp32, keys one fp32 addition of the bias, weights one
rounding of scaling s / sum s.  The token rows are zero, so the logits are exactly
logit_offset and nothing but the routing itself is measured.

Bounds: a score is the correctly rounded one, or (the rounding of a value within
2^-33 of the middle between two) its neighbour; a weight follows it by at most 2^-23
and is rounded itself, 2^-24: held to 2^-22.4 = 1.8e-7."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests.test_gpu_few import make, run

pytestmark = pytest.mark.gpu


def scores(z):
    with np.errstate(over="ignore"):
        return (1.0 / (1.0 + np.exp(-z.astype(np.float64)))).astype(np.float32)


def routed(a, z, bias=None):
    """ids and weights of the call for logits z [E] (all tokens)."""
    a["x"].zero_()
    a["logit_offset"] = torch.from_numpy(z.astype(np.float32)).cuda()
    if a["bias"] is not None:
        a["is_vision"] = None
        a["bias"].zero_()
        if bias is not None:
            a["bias"][0] = torch.from_numpy(bias).cuda()
    run(a)
    return a["ids"].cpu().numpy(), a["weights"].cpu().numpy()


def expected(a, z, bias=None, ids=None):
    s = scores(z)
    if ids is None:
        key = s + (np.zeros_like(s) if bias is None else bias)
        ids = np.tile(np.argsort(-key, kind="stable")[:a["k"]], (a["T"], 1))
    sel = s[ids].astype(np.float64)
    return ids, a["scaling"] * sel / sel.sum(1, keepdims=True)


# few tokens (the whole block adds up the logits) and many (a warp a token), by the
# number of experts a lane has
SHAPES = [(1, 384, 6), (5, 384, 8), (32, 60, 4), (32, 128, 8), (7, 300, 6), (32, 384, 6), (3, 1000, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("spread", [0.5, 6.0, 20.0])
def test_weights_are_rounded_once(T, E, k, spread):
    a = make(T, 128, E, k, 64, False)
    rng = np.random.default_rng(E + T)
    for _ in range(8):
        z = (rng.standard_normal(E) * spread).astype(np.float32)
        bias = (rng.standard_normal(E) * 0.3).astype(np.float32)
        ids, w = routed(a, z, bias)
        want_ids, want = expected(a, z, bias)
        assert np.array_equal(ids, want_ids)
        assert np.max(np.abs(w / want - 1)) <= 1.8e-7


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_neighbouring_logits_rank_by_the_rounded_score(T, E, k):
    """Logits one spacing apart: several of them round to one score and tie."""
    a = make(T, 128, E, k, 64, False)
    for base in (-30.0, -3.0, -0.1, 0.1, 0.7, 1.0, 2.0, 5.0):
        z = np.empty(E, np.float32)
        z[0] = base
        for e in range(1, E):
            z[e] = np.nextafter(z[e - 1], np.float32(np.inf))
        ids, _ = routed(a, z)
        assert np.array_equal(ids, expected(a, z)[0])


@pytest.mark.parametrize("T", [1, 20])
def test_table_weights_are_rounded_once(T):
    table = lambda r, v: np.argsort(r.random((v, 12)), 1)[:, :5]
    a = make(T, 128, 12, 5, 64, False, hash_table=table)
    rng = np.random.default_rng(T)
    for _ in range(8):
        z = (rng.standard_normal(12) * 4).astype(np.float32)
        ids, w = routed(a, z)
        want = a["tid2eid"].cpu().numpy()[a["input_ids"].cpu().numpy()]
        assert np.array_equal(ids, want)
        assert np.max(np.abs(w / expected(a, z, ids=want)[1] - 1)) <= 1.8e-7


def test_scores_at_the_ends_of_the_range():
    """Infinite logits, and scores that are subnormal or zero: as in fp64."""
    a = make(2, 128, 8, 4, 64, False)
    z = np.array([-1e4, -100.0, -95.0, -90.0, -88.0, -87.0, -1e30, -103.0], np.float32)
    ids, w = routed(a, z)
    want_ids, want = expected(a, z)
    assert np.array_equal(ids, want_ids)
    assert np.max(np.abs(w / want - 1)) <= 1e-6
    z[:] = -np.inf
    z[3], z[5] = np.inf, 40.0
    ids, w = routed(a, z)
    assert (ids == [3, 5, 0, 1]).all() and (w == [1.25, 1.25, 0, 0]).all()
    z[:] = -np.inf
    ids, w = routed(a, z)
    assert (ids == [0, 1, 2, 3]).all() and (w == 0).all()
