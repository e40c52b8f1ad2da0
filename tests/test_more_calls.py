"""Host side of the norm, the balance loss and the MXFP4 calls: argument structs, sizes,
refusals, and the reference implementation that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import mx4_ref as R
from tests.test_abi import test_structs_match_header as structs_match

P, Q = ctypes.c_void_p(256), ctypes.c_void_p(264)     # aligned, and 8-byte aligned only
H = ctypes.c_void_p(272)                              # 16-byte aligned, not 32
BAD, UNS, WS, OK = (_lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE,
                    _lib.MOE_OK)


@pytest.mark.parametrize("struct,mirror", [("moe_norm_args", _lib.NormArgs),
                                           ("moe_norm_bwd_args", _lib.NormBwdArgs),
                                           ("moe_balance_args", _lib.BalanceArgs)])
def test_structs(struct, mirror):
    structs_match(struct, mirror)


def filled(struct, **kw):
    a = struct()
    for n, t in struct._fields_:
        if t is ctypes.c_void_p:
            setattr(a, n, kw.pop(n, P))
        elif n in kw:
            setattr(a, n, kw.pop(n))
    assert not kw
    return a


def test_norm_refusals():
    lib = _lib.load()

    def norm(**kw):
        a = filled(_lib.NormArgs, **dict(dict(T=4, d=128, eps=1e-6, format=_lib.MOE_ROWS_FP8), **kw))
        return lib.moe_rmsnorm(ctypes.byref(a), None)
    none = dict(q=None, scales=None)
    assert [norm(T=-1), norm(d=0), norm(d=12), norm(d=136), norm(eps=0.0), norm(eps=float("nan")),
            norm(eps=float("inf")), norm(format=4), norm(format=-1), norm(q=None), norm(scales=None),
            norm(residual=None), norm(residual_out=None), norm(x=None), norm(x=Q), norm(weight=None),
            norm(y=Q), norm(q=Q), norm(scales=Q), norm(weight=Q)] == [BAD] * 20
    assert norm(d=16, format=_lib.MOE_ROWS_MXFP8) == BAD
    assert norm(d=48, format=_lib.MOE_ROWS_MXFP4) == BAD
    assert norm(format=_lib.MOE_ROWS_NONE) == BAD                 # q without a format
    assert norm(d=32768 + 128) == UNS
    assert norm(T=0) == OK
    assert norm(T=0, format=_lib.MOE_ROWS_NONE, d=8, **none) == OK
    assert lib.moe_rmsnorm(None, None) == BAD


def test_norm_backward_refusals():
    lib = _lib.load()

    def bwd(**kw):
        a = filled(_lib.NormBwdArgs, **dict(dict(T=4, d=128, ws_bytes=1 << 30), **kw))
        return lib.moe_rmsnorm_backward(ctypes.byref(a), None)
    assert [bwd(T=-1), bwd(d=4), bwd(d=12), bwd(x=None), bwd(dy=Q), bwd(dx=None), bwd(weight=None),
            bwd(rstd=None), bwd(d_residual=Q), bwd(d_weight=None), bwd(d_weight=Q)] == [BAD] * 11
    assert bwd(d=32776) == UNS
    assert [bwd(ws=None), bwd(ws=Q), bwd(ws_bytes=64)] == [WS] * 3
    assert lib.moe_rmsnorm_backward(None, None) == BAD
    size = lib.moe_rmsnorm_bwd_workspace_size
    assert size(1, 128) >= 4 * 128 and size(1 << 20, 4096) >= 4 * 4096
    assert [size(-1, 128), size(1, 12), size(1, 32776), size(0, 128)] == [0] * 4


def test_balance_refusals():
    lib = _lib.load()

    def both(**kw):
        a = filled(_lib.BalanceArgs, **dict(dict(T=8, E=16, k=2, n_seq=3, score=0, alpha=1.0,
                                                 ws_bytes=1 << 30), **kw))
        return (lib.moe_balance_loss(ctypes.byref(a), None),
                lib.moe_balance_loss_backward(ctypes.byref(a), None))
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(n_seq=0), dict(score=2), dict(score=-1),
               dict(seq_offsets=None), dict(tokens=None), dict(load=None), dict(load=Q),
               dict(logits=None), dict(logits=Q)):
        assert both(**kw) == (BAD, BAD), kw
    for kw in (dict(E=1025), dict(k=33), dict(n_seq=65536)):
        assert both(**kw) == (UNS, UNS), kw
    assert lib.moe_balance_loss(None, None) == BAD and lib.moe_balance_loss_backward(None, None) == BAD

    def forward(**kw):
        a = filled(_lib.BalanceArgs, **dict(dict(T=8, E=16, k=2, n_seq=1, ws_bytes=1 << 30), **kw))
        return lib.moe_balance_loss(ctypes.byref(a), None)
    assert [forward(counts=None), forward(seq_loss=None), forward(loss=None), forward(ids=None)] == [BAD] * 4
    assert [forward(ws=None), forward(ws=Q), forward(ws_bytes=64)] == [WS] * 3
    a = filled(_lib.BalanceArgs, T=8, E=16, k=2, n_seq=1, dlogits=None)
    assert lib.moe_balance_loss_backward(ctypes.byref(a), None) == BAD
    a = filled(_lib.BalanceArgs, T=0, E=16, k=2, n_seq=1, dlogits=None, logits=None)
    assert lib.moe_balance_loss_backward(ctypes.byref(a), None) == OK
    size = lib.moe_balance_workspace_size
    assert size(65536, 384, 16) >= 16 * 384 * 8 and size(0, 1, 1) > 0
    assert [size(-1, 16, 1), size(8, 1025, 1), size(8, 0, 1), size(8, 16, 0)] == [0] * 4


def test_mx4_refusals():
    lib = _lib.load()
    for f, arrays in ((lib.moe_mx4_quantize, 0), (lib.moe_mx4_dequantize, 1)):
        def call(a=P, b=P, c=P, rows=4, K=64):
            return f(a, rows, K, b, c, None) if not arrays else f(a, b, rows, K, c, None)
        assert [call(rows=-1), call(K=16), call(K=48), call(K=0), call(a=Q), call(b=None),
                call(c=Q)] == [BAD] * 7
        assert call(rows=1 << 40, K=64) == UNS
        assert call(None, None, None, rows=0) == OK
    g = lib.moe_mx4_gather
    assert [g(P, P, 0, 64, 2, P, P, None), g(P, P, 4, 48, 2, P, P, None), g(P, None, 4, 64, 2, P, P, None),
            g(P, P, 4, 64, 33, P, P, None), g(Q, P, 4, 64, 2, P, P, None)] == [BAD] * 5
    assert g(P, P, 1 << 29, 64, 8, P, P, None) == UNS

    def mm(a=P, asf=P, bits=4, offs=P, G=1, rows=8, b=P, w_rows=0, N=64, K=128, out=P):
        return lib.moe_mx4_matmul(a, asf, bits, offs, G, rows, b, P, None, w_rows, N, K, out, None)
    assert [mm(a=Q), mm(a=None), mm(asf=Q), mm(bits=6), mm(offs=None), mm(G=0), mm(G=1026), mm(rows=-1),
            mm(b=None), mm(w_rows=-1), mm(N=12), mm(N=0), mm(K=48), mm(out=Q), mm(bits=8, b=H)] == [BAD] * 15
    assert [mm(G=1025, N=1 << 22), mm(bits=8, K=96)] == [UNS] * 2
    assert [mm(rows=0), mm(rows=0, b=H)] == [OK] * 2

    def ffn(d=128, I=128, clamp=7.0, S=0, w=P, w2=P, hq=P, rows=8, offs=P):
        return lib.moe_expert_ffn_mx4(P, P, offs, 1, rows, w, P, w2, P, None, S, d, I, clamp, hq, P, P, None)
    assert [ffn(clamp=0.0), ffn(clamp=float("nan")), ffn(S=-1), ffn(w=H), ffn(w2=H), ffn(hq=Q), ffn(d=0),
            ffn(offs=None), ffn(rows=-1)] == [BAD] * 9
    assert [ffn(d=192), ffn(I=64)] == [UNS] * 2
    assert ffn(rows=0) == OK


def test_reference_format():
    """Closed forms of the rule, and that no grid value is nearer than the chosen one."""
    assert R.e2m1_codes([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert R.e2m1_codes([-0.25, -0.0, -5.1, 99.0]).tolist() == [8, 8, 15, 7]
    v = np.random.default_rng(0).standard_normal(4000) * 3
    c = R.e2m1_codes(v)
    best = np.abs(np.minimum(np.abs(v), 6)[:, None] - R.GRID).min(1)
    assert np.array_equal(np.abs(np.abs(R.TABLE[c]) - np.minimum(np.abs(v), 6)), best)
    for p in (1.0, 1.5, 1.999, 2.0 ** -100, 3e38):
        x = np.zeros((1, 32))
        x[0, 3] = -p
        q, s = R.quantise4(x)
        assert R.scale(s)[0, 0] == 2.0 ** (np.floor(np.log2(p)) - 2)
        assert abs(R.values4(q, s)[0, 3] + p) <= p / 4
    q, s = R.quantise4(np.zeros((1, 32)))
    assert (s == 0).all() and (q == 0).all()
    c = np.random.default_rng(1).integers(0, 16, (5, 64)).astype(np.uint8)
    assert np.array_equal(R.unpack(R.pack(c)), c)


def test_binding_refuses_other_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        _lib.moe_mx4_quantize(x, 4, 64, x, x)                     # not on the GPU
