"""Host side of the FP8 and few-token calls: sizes, argument checks, the
argument struct, and the reference implementation that the GPU tests use."""
import ctypes
import re

import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import fp8_ref as R
from tests.test_abi import HEADER

P, Q = ctypes.c_void_p(256), ctypes.c_void_p(264)   # aligned, and 8-byte aligned only
BAD, UNS, WS, OK = (_lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE,
                    _lib.MOE_OK)


def test_few_args_match_header():
    body = re.search(r"typedef struct \{((?:(?!typedef struct).)*?)\} moe_few_args;", HEADER,
                     flags=re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        names += [re.findall(r"\w+", p)[-1] for p in re.sub(r"^(const\s+)?\w+\s*", "", decl).split(",")]
    assert [f for f, _ in _lib.FewArgs._fields_] == names


def test_sizes():
    lib = _lib.load()
    assert [lib.moe_fp8_scale_cols(K) for K in (-1, 0, 1, 128, 129, 4096)] == [0, 0, 1, 1, 2, 32]
    wg = lib.moe_fp8_wgrad_workspace_size
    assert wg(3, 300, 256, 128) >= (300 // 128 + 3) * (256 + 128) * (128 + 4)
    assert wg(3, 0, 256, 128) > 0
    assert [wg(0, 8, 8, 8), wg(1026, 8, 8, 8), wg(1, 8, 12, 8), wg(1, -1, 8, 8),
            wg(1, 1 << 29, 8, 8)] == [0] * 5
    few = lib.moe_few_workspace_size
    assert few(32, 4096, 384, 6, 2048) >= 32 * 7 * (4096 * 4 + 2048 * 2)
    assert [few(33, 128, 8, 2, 64), few(0, 128, 8, 2, 64), few(1, 192, 8, 2, 64),
            few(1, 128, 8, 2, 96), few(1, 128, 8, 9, 64), few(1, 128, 4, 5, 64),
            few(1, 128, 1025, 2, 64)] == [0] * 7


def test_quantise_refusals():
    lib = _lib.load()
    assert lib.moe_fp8_quantize(P, 4, 24, P, P, None) == BAD
    assert lib.moe_fp8_quantize(P, -1, 32, P, P, None) == BAD
    assert lib.moe_fp8_quantize(Q, 4, 32, P, P, None) == BAD
    assert lib.moe_fp8_quantize(P, 4, 32, None, P, None) == BAD
    assert lib.moe_fp8_quantize(P, 1 << 60, 1 << 20, P, P, None) == UNS
    assert lib.moe_fp8_quantize(None, 0, 32, None, None, None) == OK
    assert lib.moe_fp8_gather(P, P, 4, 24, 2, P, P, None) == BAD
    assert lib.moe_fp8_gather(P, None, 4, 32, 2, P, P, None) == BAD
    assert lib.moe_fp8_gather(P, P, 4, 32, 33, P, P, None) == BAD
    assert lib.moe_fp8_gather(P, P, 1 << 29, 32, 8, P, P, None) == UNS
    w = lib.moe_fp8_quantize_weights
    assert w(P, 1, 24, 32, P, P, None, None, None) == BAD
    assert w(P, 1, 32, 40, P, P, None, None, None) == BAD
    assert w(P, 1, 32, 32, P, P, P, None, None) == BAD
    assert w(P, 1, 32, 32, P, Q, None, None, None) == BAD
    assert w(P, 1, 32, 32, P, P, Q, P, None) == BAD


def test_matmul_refusals():
    lib = _lib.load()

    def mm(a=P, offs=P, G=1, rows=8, w_rows=0, N=64, K=64, out=P):
        return lib.moe_fp8_matmul(a, P, offs, G, rows, P, P, None, w_rows, N, K, out, None)
    assert [mm(a=Q), mm(a=None), mm(offs=None), mm(G=0), mm(G=1026), mm(rows=-1), mm(w_rows=-1),
            mm(N=12), mm(K=24), mm(out=Q)] == [BAD] * 10
    assert mm(G=1025, N=1 << 22) == UNS
    assert mm(rows=0) == OK

    def wg(a=P, G=1, rows=8, M=64, N=64, dW=P, ws=P, n=1 << 30):
        return lib.moe_fp8_wgrad(a, P, P, G, rows, M, N, dW, ws, n, None)
    assert [wg(a=Q), wg(a=None), wg(G=0), wg(M=12), wg(N=4), wg(dW=None)] == [BAD] * 6
    assert wg(rows=1 << 29) == UNS
    assert [wg(ws=None), wg(n=64)] == [WS] * 2

    def ffn(d=128, I=128, clamp=7.0, S=0, hq=P):
        return lib.moe_expert_ffn_fp8(P, P, P, 1, 8, P, P, P, P, None, S, d, I, clamp, hq, P, P, None)
    assert [ffn(d=192), ffn(I=64)] == [UNS] * 2
    assert [ffn(clamp=0.0), ffn(clamp=float("nan")), ffn(S=-1), ffn(hq=Q), ffn(d=0)] == [BAD] * 5


def test_few_refusals():
    lib = _lib.load()

    def few(**kw):
        a = _lib.FewArgs(T=4, d=128, E=8, k=2, I=64, scaling=1.0, clamp=7.0, mode=0, vocab=0)
        for n in ("x", "W_g", "bias", "W13", "W2", "y", "ws"):
            setattr(a, n, 256)
        a.ws_bytes = 1 << 30
        for n, v in kw.items():
            setattr(a, n, v)
        return lib.moe_layer_few(ctypes.byref(a), None)
    assert lib.moe_layer_few(None, None) == BAD
    assert [few(T=33), few(d=192), few(I=96), few(k=9, E=16), few(E=1025)] == [UNS] * 5
    assert [few(T=0), few(mode=2), few(clamp=0.0), few(x=264), few(x=None), few(W_g=None),
            few(y=None), few(bias=None), few(W2=None), few(W13=264)] == [BAD] * 10
    fp8 = dict(W13_q=256, W13_s=256, W2_q=256, W2_s=256)
    assert few(**fp8) == BAD                                    # both sets of weights
    assert few(W13=None, W2=None) == BAD                        # neither
    assert few(W13=None, W2=None, **{**fp8, "W2_s": None}) == BAD
    hashed = dict(mode=1, bias=None, input_ids=256, tid2eid=256, vocab=16)
    assert [few(**{**hashed, n: v}) for n, v in
            (("input_ids", None), ("tid2eid", None), ("vocab", 0))] == [BAD] * 3
    assert [few(ws=None), few(ws_bytes=64), few(ws=264)] == [WS] * 3


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _lib.moe_fp8_quantize(x, 4, 128, x, x)
    with pytest.raises(ValueError):
        _lib.moe_layer_few(dict(x=x))


def test_reference_rounds_as_torch_does():
    """The reference's code table and rounding against torch's E4M3 type."""
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(R.TABLE, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    grid = R.TABLE[:127]
    v = np.concatenate([grid, (grid[:-1] + grid[1:]) / 2, np.linspace(0, 448, 9999), [1e-9, 2.0 ** -10]])
    v = np.concatenate([v, -v]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_codes(v), want)


def test_reference_few_layer_against_dense_sum():
    """The grouped reference equals a token-by-token evaluation."""
    rng = np.random.default_rng(0)
    T, d, E, k, I = 5, 12, 7, 3, 6
    x, W_g = rng.standard_normal((T, d)), rng.standard_normal((E, d))
    W13, W2 = rng.standard_normal((E + 1, 2 * I, d)), rng.standard_normal((E + 1, d, I))
    bias = rng.standard_normal((2, E)) * 0.1
    y, ids, w, _, _ = R.few_layer(x, W_g, lambda e: W13[e], lambda e: W2[e], k, 2.5, 7.0, bias=bias)
    for t in range(T):
        s = 1 / (1 + np.exp(-(W_g @ x[t])))
        best = sorted(range(E), key=lambda e: (-(s[e] + bias[0, e]), e))[:k]
        assert best == ids[t].tolist()
        want = np.zeros(d)
        for e, f in [(E, 1.0)] + [(e, 2.5 * s[e] / s[best].sum()) for e in best]:
            gu = W13[e] @ x[t]
            want += f * (W2[e] @ R.silu_clamped(gu[:I], gu[I:], 7.0))
        assert np.allclose(want, y[t], rtol=1e-12, atol=1e-12)


def test_layer_refusals():
    from moe_expert_layer_04_gb300.layer import Dims, MoELayer
    for kw in (dict(backward=True), dict(mx=True), dict(fused_ffn=True)):
        with pytest.raises(ValueError):
            MoELayer(Dims(8, 256, 32, 2, 128), {}, 1.0, fp8=True, device="cpu", **kw)
    for d, I in ((192, 128), (256, 64)):
        with pytest.raises(ValueError):
            MoELayer(Dims(8, d, 32, 2, I), {}, 1.0, fp8=True, device="cpu")
