"""The few-token layer against the plain 64-bit layer of tests/fp8_ref.py.

Roundings: h and y to bf16 (at most half a spacing, 2^-8 of the value each);
sums in fp32.  With A = sum w |h| |W2| an element is off by at most
(2^-8 + 1e-5) A for h and the sums, and 2^-8 of itself for y; relative
Frobenius: two independent roundings whose errors are uniform in half a spacing
(2^-9 of a value on average, / sqrt(3)): 1.6e-3, held to 4e-3.  Inputs whose
selection hangs on less than 1e-5 of a key are not used (asserted)."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import fp8_ref as R
from tests.helpers import errors

pytestmark = pytest.mark.gpu


def make(T, d, E, k, I, fp8, seed=0, hash_table=None, vocab=64):
    rng = np.random.default_rng(seed + T * 131 + E)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    nrm = lambda std, *s: torch.from_numpy((rng.standard_normal(s, dtype=np.float32) * std)).to(
        torch.bfloat16)
    a = dict(T=T, d=d, E=E, k=k, I=I, scaling=2.5, clamp=1.5, mode=_lib.MOE_ROUTE_TOPK, vocab=0)
    a["x"] = nrm(1.0, T, d).cuda()
    a["W_g"] = nrm(1.28 / d ** 0.5, E, d).cuda()
    a["logit_offset"] = dev(rng.standard_normal(E).astype(np.float32) * 0.1)
    a["bias"] = dev((rng.random((2, E)).astype(np.float32) - 0.5) * 0.1)
    a["is_vision"] = dev((rng.random(T) < 0.4).astype(np.uint8))
    for name, r, c in (("W13", 2 * I, d), ("W2", d, I)):
        if fp8:
            q = torch.from_numpy(R.e4m3_codes(np.clip(
                rng.standard_normal((E + 1, r, c), dtype=np.float32) * 100, -448, 448)))
            a[name + "_q"] = q.cuda()
            a[name + "_s"] = dev(((rng.random((E + 1, R.blocks(r), R.blocks(c))) + 0.5)
                                  * 1.3 / c ** 0.5 / 100).astype(np.float32))
        else:
            a[name] = nrm(1.3 / c ** 0.5, E + 1, r, c).cuda()
    if hash_table is not None:
        table = hash_table(rng, vocab)
        a.update(mode=_lib.MOE_ROUTE_HASH, vocab=vocab, bias=None, is_vision=None,
                 tid2eid=dev(table.astype(np.int32)),
                 input_ids=dev(rng.integers(0, vocab, T).astype(np.int32)))
    a["y"] = torch.full((T + 1, d), 3.0, dtype=torch.bfloat16, device="cuda")
    a["ids"] = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    a["weights"] = torch.zeros(T, k, device="cuda")
    a["ws"] = torch.zeros(_lib.moe_few_workspace_size(T, d, E, k, I), dtype=torch.uint8,
                          device="cuda")
    return a


def n64(t):
    return t.detach().double().cpu().numpy()


def reference(a):
    def weight(name):
        if a.get(name) is not None:
            return lambda e: n64(a[name][e])
        return lambda e: R.weight_values(a[name + "_q"][e].cpu().numpy(), n64(a[name + "_s"][e]))
    ids = None
    if a["mode"] == _lib.MOE_ROUTE_HASH:
        ids = a["tid2eid"].cpu().numpy()[a["input_ids"].cpu().numpy()]
    return R.few_layer(n64(a["x"]), n64(a["W_g"]), weight("W13"), weight("W2"), a["k"],
                       a["scaling"], a["clamp"],
                       None if a["logit_offset"] is None else n64(a["logit_offset"]),
                       None if a["bias"] is None else n64(a["bias"]),
                       None if a["is_vision"] is None else a["is_vision"].cpu().numpy(), ids)


def run(a, stream=None):
    _lib.moe_layer_few(a, stream)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK


def check(a):
    T = a["T"]
    y, ids, w, gap, scale = reference(a)
    assert gap > 1e-5, "pick another seed: the selection is too close"
    assert np.array_equal(a["ids"].cpu().numpy(), ids)
    assert np.max(np.abs(n64(a["weights"]) / w - 1)) <= 2e-5
    got = n64(a["y"][:T])
    assert np.isfinite(got).all()
    lim = (2.0 ** -8 + 1e-5) * scale + 2.0 ** -8 * np.abs(y) * 1.01 + 1e-30
    worst = float(np.max(np.abs(got - y) / lim))
    rel, _ = errors(got, y)
    assert worst <= 1.0 and rel <= 4e-3, (worst, rel)
    assert (a["y"][T:] == 3.0).all()


SHAPES = [(1, 128, 8, 1, 64), (1, 1024, 40, 6, 320), (2, 256, 16, 8, 128), (7, 384, 97, 5, 192),
          (8, 2176, 24, 3, 64), (9, 128, 33, 4, 1088), (16, 256, 12, 6, 256), (17, 640, 64, 8, 192),
          (31, 256, 9, 2, 448), (32, 512, 160, 8, 128), (3, 128, 1024, 8, 64), (5, 128, 1, 1, 64)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,d,E,k,I", SHAPES)
def test_topk(T, d, E, k, I, fp8):
    a = make(T, d, E, k, I, fp8)
    run(a)
    check(a)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 8, 13, 32])
def test_hash_with_repeated_and_crowded_experts(T, fp8):
    """Tables that send every token to the same experts, and one token to the
    same expert more than once: an expert's rows exceed the tokens."""
    for table in (lambda r, v: np.tile([3, 1, 4], (v, 1)), lambda r, v: np.tile([2, 2, 2], (v, 1)),
                  lambda r, v: r.integers(0, 6, (v, 3))):
        a = make(T, 256, 6, 3, 128, fp8, hash_table=table)
        run(a)
        check(a)


def test_ties_go_to_the_lower_expert():
    a = make(4, 128, 50, 6, 64, False)
    a["x"].zero_()
    a["logit_offset"], a["is_vision"] = None, None
    a["bias"].zero_()
    a["bias"][0, 30:] = 0.25
    run(a)
    assert (a["ids"].cpu() == torch.arange(30, 36, dtype=torch.int32)).all()
    assert torch.allclose(a["weights"].cpu(), torch.full((4, 6), 2.5 / 6), rtol=1e-6)
    assert (a["y"][:4] == 0).all()


def test_optional_outputs_and_inputs():
    a = make(6, 256, 20, 4, 128, True)
    run(a)
    y = a["y"].clone()
    a.update(ids=None, weights=None)
    run(a)
    assert torch.equal(a["y"], y)
    a = make(6, 256, 20, 4, 128, True)
    a.update(logit_offset=None, is_vision=None)
    run(a)
    check(a)


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_bit_for_bit_on_one_workspace(fp8):
    """Work is handed out at run time; results must not show it.  The counters
    are zero again after each call, so the workspace serves the next one."""
    a = make(19, 512, 48, 6, 320, fp8)
    run(a)
    y = a["y"].clone()
    for _ in range(20):
        a["y"].fill_(3.0)
        _lib.moe_layer_few(a)
    torch.cuda.synchronize()
    assert torch.equal(a["y"], y)
    check(a)


def test_new_routing_on_a_kept_workspace():
    a = make(8, 256, 32, 4, 192, False)
    run(a)
    check(a)
    a["x"].copy_(a["x"].roll(1, 1) * -1.5)
    run(a)
    check(a)


def test_stream_and_graph():
    a = make(5, 384, 30, 6, 256, True)
    run(a)
    y = a["y"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a["y"].fill_(3.0)
    torch.cuda.synchronize()
    run(a, side)
    assert torch.equal(a["y"], y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _lib.moe_layer_few(a)
    for _ in range(3):
        a["y"].fill_(3.0)
        graph.replay()
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    assert torch.equal(a["y"], y)


def test_nan_stays_with_its_token():
    a = make(6, 256, 16, 2, 128, False)
    run(a)
    clean = a["y"].clone()
    ids = a["ids"].clone()
    a["x"][2, 7] = float("nan")
    run(a)
    assert torch.isnan(a["y"][2].float()).all()
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(a["ids"][keep], ids[keep])
    assert torch.equal(a["y"][keep], clean[keep])


def test_out_of_range_table_entry_is_recorded():
    a = make(3, 128, 6, 3, 64, False, hash_table=lambda r, v: r.integers(0, 6, (v, 3)))
    a["tid2eid"][:, 1] = 77
    _lib.moe_layer_few(a)
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_ERR_INVALID_ARG
    assert (a["ids"][:, 1] == 0).all()
    a["tid2eid"][:, 1] = 0
    run(a)
    check(a)


@pytest.mark.parametrize("T,d,E,k,I,fp8", [(14, 2048, 2, 1, 1024, False), (23, 1152, 33, 4, 704, False),
                                           (14, 2048, 2, 1, 1024, True), (9, 640, 5, 2, 192, True)])
def test_calls_back_to_back_on_one_workspace(T, d, E, k, I, fp8):
    """Two inputs in turn, nothing waited for in between: every call gives what it
    gives alone, bit for bit (a part of the ring rewritten before it is read, a sum
    overtaken by the next or a row of the call before would show)."""
    a = make(T, d, E, k, I, fp8)
    b = dict(a, x=make(T, d, E, k, I, fp8, seed=1)["x"])
    alone = []
    for c in (a, b):
        run(c)
        alone.append(c["y"].clone())
    wrong = []
    for i in range(600):
        w = (i * 7 // 3) % 2
        _lib.moe_layer_few((a, b)[w])
        wrong.append((a["y"] != alone[w]).any())
    assert _lib.moe_last_device_status() == _lib.MOE_OK
    assert not torch.stack(wrong).any()
