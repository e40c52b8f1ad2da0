"""Checks that MoELayer's norm, balance loss and MXFP4 variants and GroupedLinearMX4 make
before a call, on the CPU: the library's calls only write down what they are given."""
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib, layer as L

BF16 = torch.bfloat16
T, D, E, K, I = 8, 256, 32, 2, 128


@pytest.fixture
def calls(monkeypatch):
    made = []
    for name in _lib.EXPORTS:
        if name.endswith("_size") or name in ("moe_fp8_scale_cols", "moe_mx_sf_pitch"):
            continue
        if hasattr(_lib, name):
            monkeypatch.setattr(_lib, name, lambda *a, _n=name, **k: made.append((_n, a, k)))
    return made


def weights(**more):
    w = dict(W_g=torch.zeros(E, D, dtype=BF16), W13=torch.zeros(E + 1, 2 * I, D, dtype=BF16),
             W2=torch.zeros(E + 1, D, I, dtype=BF16), norm=torch.ones(D))
    w.update(more)
    return w


def build(w=None, **kw):
    return L.MoELayer(L.Dims(T, D, E, K, I), weights() if w is None else w, 2.5, device="cpu", **kw)


def rows(n, d=D):
    return torch.zeros(n, d, dtype=BF16)


BIAS = torch.zeros(2, E)
OFFS = torch.zeros(4, dtype=torch.int32)
names = lambda calls: [c[0] for c in calls]


@pytest.mark.parametrize("kind", ["bf16", "fp8", "mx", "mx4"])
def test_order_of_calls(calls, kind):
    train = kind in ("bf16", "mx")
    m = build(norm_eps=1e-6, balance=1e-3, sequences=3, backward=train,
              **({} if kind == "bf16" else {kind: True}))
    calls.clear()
    m.forward(rows(T), BIAS, residual=rows(T), seq_offsets=OFFS)
    got = names(calls)
    moved = [] if kind == "bf16" else ["moe_gather_rows"] * 2
    ffn = dict(bf16="moe_expert_ffn", fp8="moe_expert_ffn_fp8", mx="moe_expert_ffn_mx",
               mx4="moe_expert_ffn_mx4")[kind]
    assert got == (["moe_rmsnorm", "moe_gate_route", "moe_balance_loss", "moe_permute"] + moved
                   + [ffn, "moe_combine"])
    calls.clear()
    if train:
        m.backward(rows(T), d_residual=rows(T), d_balance=torch.ones(1))
        assert names(calls) == ["moe_backward_mx" if kind == "mx" else "moe_backward",
                                "moe_balance_loss_backward", "moe_gate_backward",
                                "moe_rmsnorm_backward"]


def test_plain_layer_makes_the_calls_that_it_made(calls):
    m = build(backward=True)
    m.forward(rows(T), BIAS)
    m.backward(rows(T))
    assert names(calls) == ["moe_gate_route", "moe_permute", "moe_expert_ffn", "moe_combine",
                            "moe_backward"]


@pytest.mark.parametrize("w", [weights(norm=None), weights(norm=torch.ones(D - 1)),
                               weights(norm=torch.ones(D, dtype=BF16))])
def test_norm_weights(calls, w):
    with pytest.raises(ValueError):
        build(w, norm_eps=1e-6)


@pytest.mark.parametrize("kw", [
    dict(x=rows(T + 1)), dict(x=rows(T - 1)), dict(x=rows(T, D - 8)), dict(residual=rows(T - 1)),
    dict(residual=rows(T, 2 * D)), dict(seq_offsets=None), dict(seq_offsets=OFFS[:3]),
    dict(valid=torch.ones(T - 1, dtype=torch.uint8))])
def test_forward_refuses(calls, kw):
    m = build(norm_eps=1e-6, balance=1e-3, sequences=3)
    calls.clear()
    a = dict(x=rows(T), bias=BIAS, residual=rows(T), seq_offsets=OFFS)
    a.update(kw)
    with pytest.raises(ValueError):
        m.forward(**a)
    assert not calls


def test_options_that_the_layer_lacks(calls):
    m = build(backward=True)
    calls.clear()
    for kw in (dict(residual=rows(T)), dict(seq_offsets=OFFS), dict(valid=torch.ones(T, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            m.forward(rows(T), BIAS, **kw)
    for kw in (dict(d_residual=rows(T)), dict(d_balance=torch.ones(1))):
        with pytest.raises(ValueError):
            m.backward(rows(T), **kw)
    with pytest.raises(RuntimeError):
        m.norm(rows(T))
    assert not calls
    n = build(norm_eps=1e-6, balance=1.0, backward=True)
    n.forward(rows(T), BIAS)
    calls.clear()
    for kw in (dict(d_residual=rows(T - 1)), dict(d_balance=torch.ones(2))):
        with pytest.raises(ValueError):
            n.backward(rows(T), **kw)
    assert not calls
    with pytest.raises(RuntimeError):
        n.step_host(rows(T), rows(T))


@pytest.mark.parametrize("kw", [dict(mx=True), dict(fp8=True), dict(backward=True), dict(fused_ffn=True)])
def test_mx4_alone(calls, kw):
    with pytest.raises(ValueError):
        build(mx4=True, **kw)


def test_mx4_weights(calls):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    q = dict(W_g=torch.zeros(E, D, dtype=BF16), W13_q=u8(E + 1, 2 * I, D // 2),
             W13_sf=u8(E + 1, 2 * I, 16), W2_q=u8(E + 1, D, I // 2), W2_sf=u8(E + 1, D, 16))
    m = build(q, mx4=True)
    assert m.W13_q is q["W13_q"] and not calls
    with pytest.raises(RuntimeError):
        m.quantize_weights()
    with pytest.raises(RuntimeError):
        m.forward_few(rows(1), BIAS)
    for bad in (dict(W13_q=u8(E + 1, 2 * I, D)), dict(W2_sf=u8(E + 1, D, 4)),
                dict(W2_q=torch.zeros(E + 1, D, I // 2)), dict(W13=torch.zeros(1))):
        with pytest.raises(ValueError):
            build(dict(q, **bad), mx4=True)
    del q["W2_sf"]
    with pytest.raises(ValueError):
        build(q, mx4=True)


def test_projection(calls):
    for bits, k in ((8, 128), (4, 96)):
        p = L.GroupedLinearMX4(torch.zeros(3, 48, k, dtype=BF16), 20, bits)
        calls.clear()
        assert p.forward(rows(20, k), OFFS).shape == (20, 48)
        assert names(calls) == ["moe_mx_quantize" if bits == 8 else "moe_mx4_quantize", "moe_mx4_matmul"]
        calls.clear()
        assert p.forward(rows(0, k), OFFS).shape == (0, 48) and not calls
        for x, offs, w in ((rows(21, k), OFFS, None), (rows(4, k - 32), OFFS, None), (rows(4, k), OFFS[:3], None),
                           (rows(4, k), OFFS, torch.ones(3))):
            with pytest.raises(ValueError):
                p.forward(x, offs, row_weight=w)
        assert not calls
    for w, bits in ((torch.zeros(3, 48, 96, dtype=BF16), 8), (torch.zeros(3, 48, 40, dtype=BF16), 4),
                    (torch.zeros(3, 44, 128, dtype=BF16), 8), (torch.zeros(3, 48, 128, dtype=BF16), 6), (None, 8)):
        with pytest.raises(ValueError):
            L.GroupedLinearMX4(w, 8, bits)
    c = torch.zeros(3, 48, 64, dtype=torch.uint8), torch.zeros(3, 48, 16, dtype=torch.uint8)
    p = L.GroupedLinearMX4(None, 8, codes=c)
    assert p.K == 128
    with pytest.raises(RuntimeError):
        p.quantize_weights()
    with pytest.raises(ValueError):
        L.GroupedLinearMX4(None, 8, codes=(c[0], c[1][:, :, :8]))
