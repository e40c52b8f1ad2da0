"""MXFP4 against the plain 64-bit implementation of tests/mx4_ref.py.

Quantisation is a fixed rounding rule: codes and scales match bit for bit.  The products
of the matmuls are exact and only their fp32 sums round.  Bound of an element, with A =
sum |a| |b| over the contraction: K additions one after the other at worst, each off by at
most one fp32 spacing of a partial sum (2^-23 A, truncation allowed), and the row weight's
rounding: (K + 2) 2^-23 A.  A bf16 result has to be the rounding of a value that close: it
lies between the roundings of the interval's two ends (rounding is monotonic)."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import fp8_ref as F
from tests import mx4_ref as R
from tests.test_gpu_fp8 import bf16, codes, counts_offsets, empty, f64, ok

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def padded(s, K, fill):
    """Scale codes with the bytes behind a row set to `fill`."""
    out = np.full((s.shape[0], R.pitch(K)), fill, np.uint8)
    out[:, :s.shape[1]] = s
    return out


def values(rng, rows, K):
    """Values over many magnitudes, with the rule's edge cases at the start."""
    v = rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((rows, 1)))
    v[0, :32] = 0.0
    v[0, :16] = -0.0
    if rows > 4:
        mid = (R.GRID[:7] + R.GRID[1:]) / 2                       # scale 1: every tie, signed
        v[1, :32] = np.resize(np.concatenate([mid, -mid, [4.0, 7.5]]), 32)
        v[2, :32] = np.resize(R.TABLE, 32)                        # on the grid
        v[3, :32] = 2.0 ** -133 * np.resize([1, 3, -5, 0, 60], 32)  # bf16 subnormals
        v[4, :32] = np.resize([3.3e38, -1e38, 1e30, 1.0], 32)
    return v


@pytest.mark.parametrize("rows,K", [(1, 32), (1, 512), (7, 96), (33, 1056), (300, 2048), (5, 4128)])
def test_quantise_bit_exact(rows, K):
    x = bf16(values(np.random.default_rng(rows * 31 + K), rows, K))
    q, sf = empty(rows, K // 2), empty(rows, R.pitch(K), fill=0xA5)
    _lib.moe_mx4_quantize(x.cuda(), rows, K, q, sf)
    out = empty(rows, K, dtype=torch.bfloat16)
    _lib.moe_mx4_dequantize(q, sf, rows, K, out)
    ok()
    c, s = R.quantise4(f64(x))
    assert np.array_equal(codes(q), R.pack(c))
    assert np.array_equal(codes(sf), padded(s, K, 0xA5))          # the padding stays
    assert np.array_equal(f64(out), R.values4(c, s))


def test_quantise_not_finite():
    x = torch.ones(3, 96, dtype=torch.bfloat16)
    x[0, 5], x[1, 40], x[2, 70] = float("nan"), float("inf"), float("-inf")
    q, sf, out = empty(3, 48), empty(3, 16), empty(3, 96, dtype=torch.bfloat16)
    _lib.moe_mx4_quantize(x.cuda(), 3, 96, q, sf)
    _lib.moe_mx4_dequantize(q, sf, 3, 96, out)
    ok()
    assert codes(sf)[:, :3].tolist() == [[255, 125, 125], [125, 255, 125], [125, 125, 255]]
    nan = np.isnan(f64(out)).reshape(3, 3, 32)
    assert np.array_equal(nan.all(2), np.eye(3, dtype=bool)) and nan.sum() == 96


def test_dequantise_every_code_and_scale():
    c = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    s = np.arange(256, dtype=np.uint8)[:, None]
    out = empty(256, 32, dtype=torch.bfloat16)
    _lib.moe_mx4_dequantize(dev(R.pack(c)), dev(padded(s, 32, 0)), 256, 32, out)
    ok()
    with np.errstate(over="ignore"):
        want = R.values4(c, s)
    big = np.abs(want) > 3.3895e38                                # past bf16's range
    want[big] = np.copysign(np.inf, want[big])
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[:255], want[:255])


@pytest.mark.parametrize("T,d,k", [(1, 32, 1), (5, 288, 3), (130, 1152, 8), (64, 4096, 6), (3, 64, 32)])
def test_gather_bit_exact(T, d, k):
    x = bf16(values(np.random.default_rng(T + d + k), T, d))
    slot_row = np.random.default_rng(1).permutation(T * k).astype(np.int32)
    S = T * k
    q, sf = empty(S + T, d // 2, fill=0xAA), empty(S + T, R.pitch(d), fill=0xA5)
    _lib.moe_mx4_gather(x.cuda(), dev(slot_row), T, d, k, q, sf)
    ok()
    tok = np.empty(S + T, int)
    tok[slot_row] = np.repeat(np.arange(T), k)
    tok[S:] = np.arange(T)
    c, s = R.quantise4(f64(x))
    assert np.array_equal(codes(q), R.pack(c)[tok])
    assert np.array_equal(codes(sf), padded(s, d, 0xA5)[tok])


def test_quantise_behind_32_bit_places():
    """Elements and code bytes whose places pass 2^31 and 2^32."""
    K, rows = 8192, 530_000                                        # 4.3e9 elements
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    v = bf16(values(np.random.default_rng(1), 6, K))
    x[-6:] = v.cuda()
    q, sf = empty(rows, K // 2), empty(rows, R.pitch(K))
    _lib.moe_mx4_quantize(x, rows, K, q, sf)
    ok()
    c, s = R.quantise4(f64(v))
    assert np.array_equal(codes(q[-6:]), R.pack(c)) and np.array_equal(codes(sf[-6:]), s)
    x.fill_(1.0)
    _lib.moe_mx4_dequantize(q, sf, rows, K, x)
    ok()
    assert np.array_equal(f64(x[-6:]), R.values4(c, s))


# ------------------------------------------------------------------ matmuls

def between(got, ref, absdot, K, what):
    g = f64(got)
    lim = (K + 2) * 2.0 ** -23 * absdot + 1e-30
    lo, hi = f64(bf16(ref - lim)), f64(bf16(ref + lim))
    assert np.logical_and(lo <= g, g <= hi).all(), f"{what}: {float(np.max(np.abs(g - ref)))}"


def rows_of(rng, rows, K, bits):
    """Codes, scales and values of random rows."""
    v = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1)))
    if bits == 4:
        c, s = R.quantise4(v)
        return R.pack(c), s, R.values4(c, s)
    c, s = R.quantise8(v)
    return c, s, R.values8(c, s)


def weights_of(rng, G, N, K):
    c, s = R.quantise4(rng.standard_normal((G * N, K)) / np.sqrt(K))
    return R.pack(c), s, R.values4(c, s).reshape(G, N, K)


SHAPES = [([1], 8, 32), ([1], 512, 4096), ([3], 136, 416), ([128], 256, 128), ([129, 0, 1, 260], 264, 288),
          ([17, 40, 0, 200, 5], 640, 1152), ([0, 0], 64, 64), ([300], 1000, 2048), ([2] * 40, 72, 160),
          ([32], 384, 512), ([31, 0, 1], 264, 672), ([650, 100, 0, 700], 520, 416), ([513], 264, 1056),
          ([8], 24, 4128), ([9], 264, 544), ([1400, 0, 1201], 1032, 512), ([1], 4096, 128),
          # enough rows for pairs of row tiles: one tile each, many each, a group's last pair
          # with one row tile, one row, or a row of its second tile
          ([2048], 2048, 640), ([700, 1, 0, 900, 300], 4104, 288), ([4000, 129, 257, 127], 2304, 1120),
          ([1, 3333], 8200, 64),
          # as many groups as there can be, and more than wide tiles' tables hold
          ([1] * 1024 + [3], 16, 64), ([40] * 400 + [0, 2] * 200, 264, 64)]
MATMULS = [(c, N, K, 4) for c, N, K in SHAPES]
MATMULS += [(c, N, (K + 127) // 128 * 128, 8) for c, N, K in SHAPES]


@pytest.mark.parametrize("counts,N,K,bits", MATMULS)
@pytest.mark.parametrize("weighted", [False, True])
def test_matmul(counts, N, K, bits, weighted):
    rng = np.random.default_rng(N * 7 + K + len(counts))
    G, rows = len(counts), sum(counts)
    aq, asf, av = rows_of(rng, max(rows, 1) + 1, K, bits)          # one row behind the end
    bq, bsf, bv = weights_of(rng, G, N, K)
    w_rows = rows // 2
    w = F.f32(rng.random(max(w_rows, 1)) + 0.5)
    out = empty(max(rows, 1) + 1, N, dtype=torch.bfloat16, fill=77.0)
    # the bytes behind a row's scales are anything: here the code of a NaN
    _lib.moe_mx4_matmul(dev(aq), dev(padded(asf, K, 255)), bits, counts_offsets(counts), G,
                        max(rows, 1), dev(bq), dev(padded(bsf, K, 255)),
                        dev(w.astype(np.float32)) if weighted else None, w_rows if weighted else 0,
                        N, K, out)
    ok()
    assert (out[rows:] == 77.0).all()
    lo = 0
    for g, n in enumerate(counts):
        f_row = np.ones(n)
        if weighted:
            m = np.arange(lo, lo + n) < w_rows
            f_row[m] = w[np.arange(lo, lo + n)[m]]
        a = av[lo:lo + n]
        between(out[lo:lo + n], (a @ bv[g].T) * f_row[:, None],
                (np.abs(a) @ np.abs(bv[g]).T) * f_row[:, None], K, f"group {g}")
        lo += n


def test_bound_above_rows_and_first_rows():
    """max_rows is an upper bound, and the first group need not begin at row 0."""
    rng = np.random.default_rng(3)
    for rows, N in ((512, 256), (4096, 2048)):
        for bits in (4, 8):
            K, lo, hi = 384, rows // 8, rows // 2 + 5
            aq, asf, av = rows_of(rng, rows, K, bits)
            bq, bsf, bv = weights_of(rng, 2, N, K)
            out = empty(rows, N, dtype=torch.bfloat16, fill=5.0)
            offs = torch.tensor([lo, lo, hi], dtype=torch.int32, device="cuda")
            _lib.moe_mx4_matmul(dev(aq), dev(padded(asf, K, 0)), bits, offs, 2, rows, dev(bq),
                                dev(padded(bsf, K, 0)), None, 0, N, K, out)
            ok()
            a = av[lo:hi]
            between(out[lo:hi], a @ bv[1].T, np.abs(a) @ np.abs(bv[1]).T, K, "rows")
            assert (out[:lo] == 5.0).all() and (out[hi:] == 5.0).all()


def test_not_finite_stays_in_its_rows_and_columns():
    rng = np.random.default_rng(4)
    for rows, N in ((200, 64), (3000, 2048)):
        K = 256
        for bits in (4, 8):
            aq, asf, av = rows_of(rng, rows, K, bits)
            bq, bsf, bv = weights_of(rng, 1, N, K)
            asf[1, 3], bsf[5, 0], bsf[N - 1, 7] = 255, 255, 255
            out = empty(rows, N, dtype=torch.bfloat16)
            _lib.moe_mx4_matmul(dev(aq), dev(padded(asf, K, 0)), bits, counts_offsets([rows]), 1,
                                rows, dev(bq), dev(padded(bsf, K, 0)), None, 0, N, K, out)
            ok()
            nan = np.zeros((rows, N), bool)
            nan[1], nan[:, 5], nan[:, N - 1] = True, True, True
            assert np.array_equal(np.isnan(f64(out)), nan)


def test_scales_at_the_ends_of_their_range():
    """Products of very large and very small scales, exact in fp32's range."""
    K, N, rows = 64, 64, 40
    one4, one8 = np.full((1, 1), 2, np.uint8), np.full((1, 1), 0x38, np.uint8)   # 1.0
    for bits in (4, 8):
        K = 128
        a = R.pack(np.repeat(np.repeat(one4, K, 1), rows, 0)) if bits == 4 else \
            np.repeat(np.repeat(one8, K, 1), rows, 0)
        b = R.pack(np.repeat(np.repeat(one4, K, 1), N, 0))
        for ea, eb in ((0, 254), (254, 0), (127, 0), (10, 110), (1, 140), (200, 127)):
            sa, sb = np.full((rows, K // 32), ea, np.uint8), np.full((N, K // 32), eb, np.uint8)
            out = empty(rows, N, dtype=torch.bfloat16)
            _lib.moe_mx4_matmul(dev(a), dev(padded(sa, K, 0)), bits, counts_offsets([rows]), 1, rows,
                                dev(b), dev(padded(sb, K, 0)), None, 0, N, K, out)
            ok()
            want = K * 2.0 ** (ea - 127) * 2.0 ** (eb - 127)
            if want > 2.0 ** -120:
                assert (f64(out) == want).all(), (bits, ea, eb)


@pytest.mark.parametrize("bits", [4, 8])
def test_places_behind_32_bits(bits):
    """Output and code places past 2^31 and 2^32, in the last rows of a long list."""
    K, N, rows = 256, 8192, 530_000                                # 4.3e9 outputs
    rng = np.random.default_rng(bits)
    aq, asf, av = rows_of(rng, 700, K, bits)
    bq, bsf, bv = weights_of(rng, 1, N, K)
    a = torch.zeros(rows, aq.shape[1], dtype=torch.uint8, device="cuda")
    s = torch.full((rows, R.pitch(K)), 127, dtype=torch.uint8, device="cuda")
    a[-700:], s[-700:] = dev(aq), dev(padded(asf, K, 0))
    out = empty(rows, N, dtype=torch.bfloat16, fill=3.0)
    _lib.moe_mx4_matmul(a, s, bits, counts_offsets([rows]), 1, rows, dev(bq), dev(padded(bsf, K, 0)),
                        None, 0, N, K, out)
    ok()
    between(out[-700:], av @ bv[0].T, np.abs(av) @ np.abs(bv[0]).T, K, "last rows")
    assert (out[:-700] == 0).all()


# ---------------------------------------------------------------------- FFN

FFNS = [([1], 128, 128), ([3, 0, 5], 256, 384), ([40, 200, 0, 129], 512, 256), ([777], 1152, 640),
        ([1500, 1100], 384, 2048), ([2] * 30, 128, 128), ([3000, 257, 1], 256, 1280)]


@pytest.mark.parametrize("counts,d,I", FFNS)
def test_ffn(counts, d, I):
    """h: g and u are sums like the matmul's, (d + 2) 2^-23 of the magnitudes; its scale
    and codes are roundings of such values (the gate's exponential and quotient 2^-20
    more).  y follows from the h that came out, as a matmul of it."""
    rng = np.random.default_rng(d + I)
    G, rows, clamp = len(counts), sum(counts), 2.0
    xq, xsf, xv = rows_of(rng, rows, d, 8)
    w13, s13, v13 = weights_of(rng, G, 2 * I, d)
    w2, s2, v2 = weights_of(rng, G, d, I)
    S = rows // 2
    w = F.f32(rng.random(max(S, 1)) + 0.5)
    hq, hsf = empty(rows + 1, I, fill=7), empty(rows + 1, R.pitch(I), fill=0xA5)
    y = empty(rows + 1, d, dtype=torch.bfloat16, fill=77.0)
    _lib.moe_expert_ffn_mx4(dev(xq), dev(padded(xsf, d, 255)), counts_offsets(counts), G, rows,
                            dev(w13), dev(padded(s13, d, 255)), dev(w2), dev(padded(s2, I, 255)),
                            dev(w.astype(np.float32)), S, d, I, clamp, hq, hsf, y)
    ok()
    assert (y[rows:] == 77.0).all() and (hq[rows:] == 7).all() and (hsf[rows:] == 0xA5).all()
    assert (hsf[:, I // 32:] == 0xA5).all()
    codes_h, scales_h = codes(hq)[:rows], codes(hsf)[:rows, :I // 32]
    lo = 0
    for g, n in enumerate(counts):
        x = xv[lo:lo + n]
        gu, mag = x @ v13[g].T, np.abs(x) @ np.abs(v13[g]).T
        lim = (d + 2) * 2.0 ** -23 * mag + 2.0 ** -20 * np.abs(gu)
        a, u = np.minimum(gu[:, :I], clamp), np.clip(gu[:, I:], -clamp, clamp)
        sig = 1 / (1 + np.exp(-a))
        h = a * sig * u
        # |d silu / dg| <= 1.1, |silu| <= clamp
        e = 1.1 * lim[:, :I] * np.abs(u) + lim[:, I:] * np.abs(a * sig) + 2.0 ** -19 * np.abs(h)
        s = R.scale(scales_h[lo:lo + n])
        for sign, bound in ((-1, np.less_equal), (1, np.greater_equal)):
            _, sc = R.quantise8(np.sign(h) * np.maximum(np.abs(h) + sign * e, 0))
            assert bound(R.scale(sc), s).all()
        m, me = np.abs(h) / np.repeat(s, 32, 1), e / np.repeat(s, 32, 1)
        q = F.TABLE[codes_h[lo:lo + n]]
        near = lambda v: F.TABLE[F.e4m3_codes(np.maximum(v, 0))]
        assert np.logical_and(near(m - me) <= np.abs(q), np.abs(q) <= near(m + me)).all()
        hv = R.values8(codes_h[lo:lo + n], scales_h[lo:lo + n])
        f_row = np.where(np.arange(lo, lo + n) < S, w[np.minimum(np.arange(lo, lo + n), len(w) - 1)], 1.0)
        between(y[lo:lo + n], hv @ v2[g].T * f_row[:, None],
                np.abs(hv) @ np.abs(v2[g]).T * f_row[:, None], I, f"group {g}")
        lo += n


def test_offsets_that_do_not_fit():
    """Cut to the rows and recorded; what lies behind the rows stays."""
    K, N = 256, 264
    rng = np.random.default_rng(1)
    for bits in (4, 8):
        for R_, G, good, bad in ((200, 3, [0, 64, 128, 200], [0, 64, 128, 437]),
                                 (200, 3, [0, 64, 200, 200], [0, 64, 450, 470]),
                                 (200, 3, [0, 0, 128, 200], [-90, 0, 128, 200]),
                                 (7, 1, [0, 7], [0, 120]), (3000, 2, [0, 500, 3000], [0, 500, 3290])):
            aq, asf, _ = rows_of(rng, R_ + 300, K, bits)
            bq, bsf, _ = weights_of(rng, G, N, K)
            got = []
            for offs, status in ((good, _lib.MOE_OK), (bad, _lib.MOE_ERR_INVALID_ARG)):
                out = empty(R_ + 300, N, dtype=torch.bfloat16, fill=3.0)
                _lib.moe_mx4_matmul(dev(aq), dev(padded(asf, K, 0)), bits,
                                    torch.tensor(offs, dtype=torch.int32, device="cuda"), G, R_, dev(bq),
                                    dev(padded(bsf, K, 0)), None, 0, N, K, out)
                torch.cuda.synchronize()
                assert _lib.moe_last_device_status() == status
                assert (out[R_:] == 3.0).all()
                got.append(out)
            assert torch.equal(got[0], got[1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("cuts,R,N,K", [([], 512, 512, 2048), ([700, 701, 1700], 2600, 768, 640),
                                        ([60, 61], 200, 512, 1024), ([], 1, 2048, 4096)])
def test_inputs_in_turn(cuts, R, N, K, bits):
    """Three inputs in turn, launched behind one another: every product as it is alone, bit for
    bit (a stage with another call's codes or scales would show)."""
    G = len(cuts) + 1
    g = torch.Generator(device="cuda").manual_seed(R)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, dtype=torch.uint8, device="cuda")
    offs = torch.tensor([0] + cuts + [R], dtype=torch.int32, device="cuda")
    sets = [(u8(0, 120 if bits == 8 else 256, R, K if bits == 8 else K // 2), u8(117, 132, R, _lib.moe_mx_sf_pitch(K)),
             u8(0, 256, G, N, K // 2), u8(117, 132, G, N, _lib.moe_mx_sf_pitch(K))) for _ in range(3)]
    out = torch.empty(R, N, dtype=torch.bfloat16, device="cuda")

    def run(s):
        _lib.moe_mx4_matmul(s[0], s[1], bits, offs, G, R, s[2], s[3], None, 0, N, K, out)
        return out.view(torch.int16)
    alone = []
    for s in sets:
        torch.cuda.synchronize()
        alone.append(run(s).clone())
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        out.zero_()
        wrong += (run(sets[i % 3]) != alone[i % 3]).sum()
    ok()
    assert int(wrong) == 0
