"""The norm ahead of the layer and its backward against their formulas in 64 bits.

Roundings (relative, of fp32 unless said): a mean of squares over d elements that a row's
threads sum (at most 32 in order, then in pairs, 15 levels at most): at most 50 2^-24 of
itself; eps, the root and the division 4 2^-24; so rstd is off by at most (25 + 4) 2^-24 <
2^-19 of itself, and u by 3 2^-24 more, E = 2^-18.9.  y is the bf16 rounding of such a
value.  A scale of 128 follows the largest |u|: E and one rounding.  Elements of codes lie
between the roundings of (1 - E') u and (1 + E') u at the scale that came out."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import fp8_ref as F
from tests import mx4_ref as R
from tests.test_gpu_fp8 import bf16, codes, empty, f64, ok

pytestmark = pytest.mark.gpu

EPS = 1e-6
E = 2.0 ** -18


def rows(rng, T, d):
    return bf16(rng.standard_normal((T, d)) * np.exp(rng.standard_normal((T, 1))))


def between(got, ref, lim):
    g = f64(got)
    lo, hi = f64(bf16(ref - lim)), f64(bf16(ref + lim))
    assert np.logical_and(lo <= g, g <= hi).all(), float(np.max(np.abs(g - ref)))


def forward(x, w, residual=None, fmt=_lib.MOE_ROWS_NONE, want_y=True, in_place=False):
    T, d = x.shape
    a = dict(T=T, d=d, eps=EPS, format=fmt, x=x.cuda(), weight=w.cuda(),
             residual=None if residual is None else residual.cuda(),
             rstd=empty(T, dtype=torch.float32))
    if residual is not None:
        a["residual_out"] = a["residual"] if in_place else empty(T, d, dtype=torch.bfloat16)
    if want_y:
        a["y"] = a["x"] if in_place else empty(T, d, dtype=torch.bfloat16)
    if fmt == _lib.MOE_ROWS_FP8:
        a["q"], a["scales"] = empty(T, d), empty(T, F.blocks(d), dtype=torch.float32)
    elif fmt != _lib.MOE_ROWS_NONE:
        a["q"] = empty(T, d if fmt == _lib.MOE_ROWS_MXFP8 else d // 2)
        a["scales"] = empty(T, R.pitch(d), fill=0xA5)
    _lib.moe_rmsnorm(a)
    ok()
    return a


def reference(x, w, residual=None):
    v = f64(x)
    if residual is not None:
        v = f64(bf16(v + f64(residual)))
    r = 1 / np.sqrt((v * v).mean(1) + EPS)
    return v, r, v * r[:, None] * f64(w)


SHAPES = [(1, 8), (1, 4096), (3, 40), (7, 1184), (130, 256), (65, 2056), (5, 8200), (2, 16392),
          (3, 32768), (4099, 128), (300, 7168),
          # more rows than the SMs hold at once
          (1000, 4096), (700, 1184), (311, 256), (5000, 8), (1231, 2056), (613, 4088),
          (913, 3592), (1300, 3584), (310, 7168), (320, 5128), (330, 16384)]


@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("res", [False, True])
def test_forward(T, d, res):
    rng = np.random.default_rng(T * 7 + d)
    x, w = rows(rng, T, d), torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    residual = rows(rng, T, d) if res else None
    for in_place in (False, True):
        a = forward(x, w, residual, in_place=in_place)
        v, r, u = reference(x, w, residual)
        if res:
            assert np.array_equal(f64(a["residual_out"]), v)
        assert (np.abs(f64(a["rstd"]) - r) <= E * r).all()
        between(a["y"], u, E * np.abs(u))


def check_codes(a, u, fmt):
    """Codes and scales of the rows u, which the kernel had within E of themselves."""
    T, d = u.shape
    if fmt == _lib.MOE_ROWS_FP8:
        got, nb = f64(a["scales"]), F.blocks(d)
        block, top = 128, 448.0
        amax = np.zeros((T, nb))
        for b in range(nb):
            amax[:, b] = np.maximum(np.abs(u[:, 128 * b:128 * b + 128]).max(1), F.FLOOR)
        assert (np.abs(got - amax / top) <= (E + 2.0 ** -23) * amax / top).all()
        near = lambda v: F.TABLE[F.e4m3_codes(v)]
        q = F.TABLE[codes(a["q"])]
    else:
        kind = 4 if fmt == _lib.MOE_ROWS_MXFP4 else 8
        block = 32
        sc = codes(a["scales"])
        assert (sc[:, d // 32:] == 0xA5).all()
        s = sc[:, :d // 32]
        quant = R.quantise4 if kind == 4 else R.quantise8
        lo, hi = quant(u * (1 - E))[1], quant(u * (1 + E))[1]
        assert np.logical_and(lo <= s, s <= hi).all()
        got = R.scale(s)
        near = (lambda v: R.TABLE[R.e2m1_codes(v)]) if kind == 4 else \
            (lambda v: F.TABLE[F.e4m3_codes(v)])
        q = R.TABLE[R.unpack(codes(a["q"]))] if kind == 4 else F.TABLE[codes(a["q"])]
    # the factor of FP8 is rounded once more, and so is the product
    m = np.abs(u) / np.repeat(got, block, axis=1)[:, :d]
    lo, hi = near(m * (1 - 3 * E)), near(m * (1 + 3 * E))
    assert np.logical_and(lo <= np.abs(q), np.abs(q) <= hi).all()
    assert np.array_equal(np.signbit(q[q != 0]), (u < 0)[q != 0])


@pytest.mark.parametrize("T,d", [(1, 32), (1, 4096), (5, 1184), (130, 288), (33, 8224), (3, 32768),
                                 (4099, 128), (700, 4096), (1000, 96), (901, 2080),
                                 (1000, 4096), (1300, 3616), (310, 8192), (306, 10016)])
@pytest.mark.parametrize("fmt", [_lib.MOE_ROWS_FP8, _lib.MOE_ROWS_MXFP8, _lib.MOE_ROWS_MXFP4])
def test_forward_codes(T, d, fmt):
    rng = np.random.default_rng(T * 5 + d + fmt)
    x, w = rows(rng, T, d), torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    x[0, :8] = 0.0
    residual = rows(rng, T, d)
    a = forward(x, w, residual, fmt, want_y=T != 5)
    check_codes(a, reference(x, w, residual)[2], fmt)


def test_fp8_short_last_block():
    rng = np.random.default_rng(3)
    for T, d in ((9, 16), (9, 144), (9, 1040), (1000, 3600)):
        x, w = rows(rng, T, d), torch.ones(d)
        check_codes(forward(x, w, None, _lib.MOE_ROWS_FP8), reference(x, w)[2], _lib.MOE_ROWS_FP8)


def test_rows_of_zeros_and_not_finite():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x[1:] = 1.0
    x[2, 5], x[3, 200] = float("nan"), float("inf")
    w = torch.ones(256)
    for fmt in (_lib.MOE_ROWS_FP8, _lib.MOE_ROWS_MXFP8, _lib.MOE_ROWS_MXFP4):
        a = forward(x, w, None, fmt)
        y = f64(a["y"])
        assert (y[0] == 0).all() and np.isfinite(y[1]).all() and np.isnan(y[2]).all()
        assert np.isnan(y[3, 200]) and (np.delete(y[3], 200) == 0).all()
        if fmt == _lib.MOE_ROWS_FP8:
            s = f64(a["scales"])
            assert np.isfinite(s[:2]).all() and np.isnan(s[2]).all() and np.isnan(s[3, 1])
        elif fmt == _lib.MOE_ROWS_MXFP4:
            s = codes(a["scales"])
            assert (s[2, :8] == 255).all() and s[3, 6] == 255 and (s[3, :6] == 0).all()
    assert f64(a["rstd"])[0] == pytest.approx(1e3, rel=1e-6)


# ----------------------------------------------------------------- backward

def backward(x, w, rstd, dy, dres, in_place=False, ws_fill=None):
    T, d = x.shape
    dy, dres = dy.cuda(), None if dres is None else dres.cuda()
    n = _lib.moe_rmsnorm_bwd_workspace_size(T, d)
    ws = empty(n)
    if ws_fill is not None:
        ws.fill_(ws_fill)
    a = dict(T=T, d=d, x=x.cuda(), weight=w.cuda(), rstd=rstd, dy=dy, d_residual=dres,
             dx=(dy if dres is None else dres) if in_place else empty(T, d, dtype=torch.bfloat16),
             d_weight=empty(d, dtype=torch.float32, fill=float("nan")), ws=ws)
    _lib.moe_rmsnorm_backward(a)
    ok()
    return a


@pytest.mark.parametrize("T,d", SHAPES + [(2000, 512), (1500, 32), (200, 16392), (170, 20480),
                                          (90, 32768), (333, 9000)])
@pytest.mark.parametrize("res", [False, True])
def test_backward(T, d, res):
    """dx: the sum of a vh over d rounds like the forward's (at most 50 2^-24 of the sum of
    magnitudes), each of the other products and sums once: 2^-18 of the magnitudes added
    up.  d_weight: T products of three roundings each, summed in at most T + 32 additions."""
    rng = np.random.default_rng(T + 3 * d + res)
    x, w = rows(rng, T, d), torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    dy, dres = rows(rng, T, d), rows(rng, T, d) if res else None
    v = f64(x)
    rstd = torch.from_numpy((1 / np.sqrt((v * v).mean(1) + EPS)).astype(np.float32)).cuda()
    r = f64(rstd)[:, None]
    g, vh = f64(dy), v * r
    a = g * f64(w)
    dx = r * (a - vh * (a * vh).mean(1, keepdims=True))
    mag = r * (np.abs(a) + np.abs(vh) * np.abs(a * vh).mean(1, keepdims=True))
    if res:
        dx, mag = dx + f64(dres), mag + np.abs(f64(dres))
    for in_place in (False, True):
        o = backward(x, w, rstd, dy, dres, in_place, ws_fill=255)
        between(o["dx"], dx, E * mag)
        lim = (T + 36) * 2.0 ** -24 * np.abs(g * vh).sum(0) + 1e-30
        assert (np.abs(f64(o["d_weight"]) - (g * vh).sum(0)) <= lim).all()


def test_backward_is_the_gradient():
    """Against differences of the forward in 64 bits: the slope along random directions."""
    rng = np.random.default_rng(5)
    T, d = 3, 96
    x, dy = rows(rng, T, d), rows(rng, T, d)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    v = f64(x)
    rstd = torch.from_numpy((1 / np.sqrt((v * v).mean(1) + EPS)).astype(np.float32)).cuda()
    o = backward(x, w, rstd, dy, None)

    def loss(v, w):
        r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + EPS)
        return (f64(dy) * v * r * w).sum()
    h = 1e-5
    for i in range(8):
        a, b = rng.standard_normal((T, d)), rng.standard_normal(d)
        num = (loss(v + h * a, f64(w) + h * b) - loss(v - h * a, f64(w) - h * b)) / (2 * h)
        parts = f64(o["dx"]) * a
        # dx is bf16 (2^-8 of each element), differences are off by O(h^2)
        lim = 2.0 ** -8 * np.abs(parts).sum() + 1e-4
        assert abs(parts.sum() + (f64(o["d_weight"]) * b).sum() - num) <= lim


def test_places_behind_32_bits():
    """Elements past 2^31, the last rows of a long list, both directions."""
    T, d, n = 600_000, 4096, 64
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    last, g = rows(rng, n, d), rows(rng, n, d)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[-n:] = last.cuda()
    y, rstd = torch.empty_like(x), torch.empty(T, device="cuda")
    q, s = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, 32, device="cuda")
    _lib.moe_rmsnorm(dict(T=T, d=d, eps=EPS, format=_lib.MOE_ROWS_FP8, x=x, weight=w.cuda(), y=y, rstd=rstd,
                          q=q, scales=s))
    ok()
    v, r, u = reference(last, w)
    between(y[-n:], u, E * np.abs(u))
    check_codes(dict(q=q[-n:], scales=s[-n:]), u, _lib.MOE_ROWS_FP8)
    assert (y[:-n] == 0).all() and (q[:-n] & 127 == 0).all()        # (zeros of either sign)
    y.zero_()
    y[-n:] = g.cuda()
    ws = empty(_lib.moe_rmsnorm_bwd_workspace_size(T, d))
    dw = torch.empty(d, device="cuda")
    _lib.moe_rmsnorm_backward(dict(T=T, d=d, x=x, weight=w.cuda(), rstd=rstd, dy=y, dx=y, d_weight=dw, ws=ws))
    ok()
    r = f64(rstd[-n:])[:, None]
    a, vh = f64(g) * f64(w), v * r
    dot = (a * vh).mean(1, keepdims=True)
    between(y[-n:], r * (a - vh * dot), E * r * (np.abs(a) + np.abs(vh) * np.abs(a * vh).mean(1, keepdims=True)))
    assert (y[:-n] == 0).all()


def test_no_rows():
    w = torch.ones(64)
    x = torch.empty(0, 64, dtype=torch.bfloat16)
    forward(x, w, x)
    o = backward(x, w, empty(0, dtype=torch.float32), x, None)
    assert (f64(o["d_weight"]) == 0).all()


@pytest.mark.parametrize("T,d,fmt", [(1500, 4096, _lib.MOE_ROWS_FP8), (1300, 3616, _lib.MOE_ROWS_MXFP4),
                                     (700, 512, _lib.MOE_ROWS_MXFP8), (5, 2048, _lib.MOE_ROWS_FP8)])
def test_inputs_in_turn(T, d, fmt):
    """Both directions of three inputs in turn, launched behind one another: every result as it
    is alone, bit for bit."""
    rng = np.random.default_rng(d)
    w = torch.from_numpy(rng.standard_normal(d).astype(np.float32))
    calls = []
    for _ in range(3):
        a = forward(rows(rng, T, d), w, rows(rng, T, d), fmt)
        b = backward(a["residual_out"], w, a["rstd"], rows(rng, T, d), rows(rng, T, d))
        calls.append((a, b, [t.clone() for t in (a["y"], a["q"], a["rstd"], b["dx"], b["d_weight"])]))
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(200):
        a, b, want = calls[i % 3]
        got = a["y"], a["q"], a["rstd"], b["dx"], b["d_weight"]
        for t in got:
            t.zero_()
        _lib.moe_rmsnorm(a)
        _lib.moe_rmsnorm_backward(b)
        for x, y in zip(got, want):
            wrong += (x != y).sum()
    ok()
    assert int(wrong) == 0
