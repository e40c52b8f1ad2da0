"""Biases that mask experts (minus infinity, the lowest fp32 value) or force them
(infinity): the rule is the same for every key, larger first and equal ones by the
lower id, so where a mask leaves fewer than k experts the next ones follow in order.
The token rows are zero: the logits are exactly logit_offset."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min
INF = np.float32(np.inf)


def inputs(T, E, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal(E).astype(np.float32)
    bias = ((rng.random((2, E)) - 0.5) * 0.2).astype(np.float32)
    return rng, z, bias, (rng.random(T) < 0.5).astype(np.uint8)


def expected(z, bias, vision, k, scaling):
    with np.errstate(over="ignore"):
        s = (1.0 / (1.0 + np.exp(-z.astype(np.float64)))).astype(np.float32)
        key = s[None] + bias[vision.astype(int)]
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    sel = s[ids].astype(np.float64)
    return ids, scaling * sel / sel.sum(1, keepdims=True)


def few(z, bias, vision, k):
    T, E, d, I = len(vision), len(z), 128, 64
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    a = dict(T=T, d=d, E=E, k=k, I=I, scaling=2.5, clamp=7.0, mode=_lib.MOE_ROUTE_TOPK, vocab=0,
             x=bf(T, d), W_g=bf(E, d), logit_offset=dev(z), bias=dev(bias), is_vision=dev(vision),
             W13=bf(E + 1, 2 * I, d), W2=bf(E + 1, d, I), y=bf(T, d),
             ids=torch.full((T, k), -1, dtype=torch.int32, device="cuda"),
             weights=torch.zeros(T, k, device="cuda"),
             ws=torch.zeros(_lib.moe_few_workspace_size(T, d, E, k, I), dtype=torch.uint8,
                            device="cuda"))
    _lib.moe_layer_few(a)
    return a["ids"], a["weights"]


def route(z, bias, vision, k, fused):
    T, E, d = len(vision), len(z), 64
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    logits, w, s = (torch.zeros(T, n, device="cuda") for n in (E, k, k))
    args = (bf(T, d), bf(E, d), dev(z), dev(bias), dev(vision), None, None, T, d, E, k, 2.5,
            _lib.MOE_ROUTE_TOPK, logits, ids, w, s)
    if fused:
        _lib.moe_gate_route(*args, None)
    else:
        _lib.moe_route(*args)
    assert torch.equal(logits.cpu(), torch.from_numpy(z).expand(T, E))
    return ids, w


CALLS = dict(few=few, route=lambda *a: route(*a, False), gate_route=lambda *a: route(*a, True))
MASKS = {
    # experts left to the k best, by kind of mask
    "none_left": lambda rng, E, k: np.full(E, -INF),
    "one_left": lambda rng, E, k: np.where(np.arange(E) == E // 2, np.float32(0), -INF),
    "fewer_than_k": lambda rng, E, k: np.where(rng.permutation(E) < k - 1, np.float32(0), -INF),
    "exactly_k": lambda rng, E, k: np.where(rng.permutation(E) < k, np.float32(0), -INF),
    "some": lambda rng, E, k: np.where(rng.random(E) < 0.3, np.float32(0), -INF),
    "lowest_value": lambda rng, E, k: np.where(rng.permutation(E) < k - 1, np.float32(0), LOWEST),
    "both_masks": lambda rng, E, k: rng.choice(np.array([LOWEST, -INF], np.float32), E),
}
FORCED = {
    "one_forced": lambda rng, E, k: np.where(np.arange(E) == E - 1, INF, np.float32(0)),
    "k_forced": lambda rng, E, k: np.where(rng.permutation(E) < k, INF, np.float32(0)),
    "all_forced": lambda rng, E, k: np.full(E, INF),
}


@pytest.mark.parametrize("T,E,k", [(3, 32, 4), (7, 384, 6), (32, 96, 8), (1, 512, 8)])
@pytest.mark.parametrize("call", list(CALLS))
def test_equal_keys_behind_later_winners(call, T, E, k):
    """Many equal keys, then larger ones at higher ids, which push the first down: what
    is left of the equal ones are the lowest ids, in order."""
    for late in (1, 2, k - 1):
        z = np.zeros(E, np.float32)
        z[E - late:] = np.arange(1, late + 1)
        vision = np.zeros(T, np.uint8)
        ids, _ = CALLS[call](z, np.zeros((2, E), np.float32), vision, k)
        assert np.array_equal(ids.cpu().numpy(),
                              expected(z, np.zeros((2, E), np.float32), vision, k, 2.5)[0])


SIZES = [(3, 32, 4), (7, 384, 6), (32, 96, 8), (20, 64, 2), (1, 512, 8)]


def check(call, T, E, k, mask):
    rng, z, bias, vision = inputs(T, E, T * 1000 + E)
    bias = (bias + mask(rng, E, k).astype(np.float32)[None]).astype(np.float32)
    ids, w = CALLS[call](z, bias, vision, k)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    want_ids, want = expected(z, bias, vision, k, 2.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.max(np.abs(w.cpu().numpy() / want - 1)) <= 1e-6


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("call", list(CALLS))
def test_masked_experts(call, T, E, k, mask):
    check(call, T, E, k, MASKS[mask])


@pytest.mark.parametrize("mask", list(FORCED))
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("call", list(CALLS))
def test_forced_experts(call, T, E, k, mask):
    check(call, T, E, k, FORCED[mask])
