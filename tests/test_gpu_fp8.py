"""The FP8 operators with a scale for each block of 128 against the plain
64-bit implementation of tests/fp8_ref.py.

Quantisation is a fixed rounding rule: codes and scales must match bit for bit.
The matmuls' products are exact and only their fp32 sums round.  Bound of an
element, with A = sum |a| |b| over the contraction: a block's 128 products and
the K/128 scaled blocks are added one after the other at worst, each addition
off by at most one fp32 spacing (2^-23, truncation allowed), and a scale
product, the scaled block and the row weight round once each: (128 + K/128 +
4) 2^-23 A.  A bf16 result has to be the rounding of a value that close: it lies
between the roundings of the interval's two ends (rounding is monotonic)."""
import numpy as np
import pytest
import torch

from moe_expert_layer_04_gb300 import _lib
from tests import fp8_ref as R

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def codes(t):
    return t.detach().cpu().numpy()


def ok():
    torch.cuda.synchronize()
    assert _lib.moe_last_device_status() == _lib.MOE_OK


def empty(*shape, dtype=torch.uint8, fill=None):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t if fill is None else t.fill_(fill)


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16)


def values(rng, *shape):
    """Values over many magnitudes, with the rule's edge cases at the start."""
    v = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape[:-1] + (1,)))
    flat = v.reshape(-1, shape[-1])
    n = min(shape[-1], 128)
    flat[0, :n] = 0.0
    flat[0, : n // 2] = -0.0
    if flat.shape[0] > 2:
        flat[1, :n] = R.TABLE[np.linspace(0, 126, n).astype(int)]   # scale 1: on the grid
        flat[1, 0] = 448.0
        mid = (R.TABLE[:126] + R.TABLE[1:127]) / 2                  # scale 1: every tie
        flat[2, :n] = -mid[np.linspace(0, 125, n).astype(int)]
        flat[2, 0] = 448.0
    if flat.shape[0] > 5:
        flat[3, :n] = 2.0 ** -120                                   # below the floor
        flat[4, :n] *= 2.0 ** 100
        flat[5, :n] *= 2.0 ** -90
    return v


def counts_offsets(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


# ------------------------------------------------------------- quantisation

@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (7, 144), (33, 1040), (300, 2048)])
def test_quantise_rows_bit_exact(rows, K):
    x = bf16(values(np.random.default_rng(rows * 31 + K), rows, K))
    q, s = empty(rows, K), empty(rows, _lib.moe_fp8_scale_cols(K), dtype=torch.float32)
    _lib.moe_fp8_quantize(x.cuda(), rows, K, q, s)
    ok()
    rq, rs = R.quantise_rows(f64(x))
    assert np.array_equal(f64(s), rs)
    assert np.array_equal(codes(q), rq)


def test_quantise_rows_not_finite():
    x = torch.ones(3, 256, dtype=torch.bfloat16)
    x[0, 5] = float("nan")
    x[1, 130] = float("-inf")
    x[2, 200] = 3e38
    q, s = empty(3, 256), empty(3, 2, dtype=torch.float32)
    _lib.moe_fp8_quantize(x.cuda(), 3, 256, q, s)
    ok()
    s, v = f64(s), R.TABLE[codes(q)]
    assert np.isnan(s[0, 0]) and np.isnan(v[0, :128]).all() and s[0, 1] == R.f32(1 / 448.0)
    assert np.isposinf(s[1, 1]) and np.isnan(v[1, 130]) and (np.delete(v[1, 128:], 2) == 0).all()
    assert np.isfinite(s[2]).all() and v[2, 200] == 448.0


@pytest.mark.parametrize("T,d,k", [(1, 16, 1), (5, 272, 3), (130, 1152, 8), (64, 4096, 6)])
def test_gather_bit_exact(T, d, k):
    x = bf16(values(np.random.default_rng(T + d + k), T, d))
    slot_row = torch.from_numpy(np.random.default_rng(1).permutation(T * k).astype(np.int32))
    S = T * k
    q = empty(S + T, d, fill=0xAA)
    s = empty(S + T, _lib.moe_fp8_scale_cols(d), dtype=torch.float32, fill=-1.0)
    _lib.moe_fp8_gather(x.cuda(), slot_row.cuda(), T, d, k, q, s)
    ok()
    rq, rs = R.quantise_rows(f64(x))
    tok = np.empty(S + T, int)
    tok[slot_row.numpy()] = np.repeat(np.arange(T), k)
    tok[S:] = np.arange(T)
    assert np.array_equal(codes(q), rq[tok])
    assert np.array_equal(f64(s), rs[tok])


@pytest.mark.parametrize("G,N,K,both", [(1, 16, 16, True), (2, 144, 272, True), (3, 256, 128, True),
                                        (1, 128, 4096, False), (2, 400, 656, True)])
def test_quantise_weights_bit_exact(G, N, K, both):
    w = bf16(values(np.random.default_rng(N + K), G, N, K))
    q, s = empty(G, N, K), empty(G, R.blocks(N), R.blocks(K), dtype=torch.float32)
    qt = empty(G, K, N) if both else None
    st = empty(G, R.blocks(K), R.blocks(N), dtype=torch.float32) if both else None
    _lib.moe_fp8_quantize_weights(w.cuda(), G, N, K, q, s, qt, st)
    ok()
    for g in range(G):
        rq, rs = R.quantise_weights(f64(w[g]))
        assert np.array_equal(f64(s[g]), rs)
        assert np.array_equal(codes(q[g]), rq)
        if both:
            assert np.array_equal(f64(st[g]), rs.T)
            assert np.array_equal(codes(qt[g]), rq.T)


# ------------------------------------------------------------------ matmuls

def random_codes(rng, *shape):
    return R.e4m3_codes(np.clip(rng.standard_normal(shape) * 100, -448, 448))


def sum_bound(K):
    return (128 + K / 128 + 4) * 2.0 ** -23


def check(got, ref, absdot, K, bf16_out, what):
    g = f64(got)
    assert np.isfinite(g).all(), what
    lim = sum_bound(K) * absdot + 1e-30
    if bf16_out:
        lo, hi = f64(bf16(ref - lim)), f64(bf16(ref + lim))
        assert np.logical_and(lo <= g, g <= hi).all(), f"{what}: {float(np.max(np.abs(g - ref)))}"
        return
    worst = float(np.max(np.abs(g - ref) / lim)) if g.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} times its bound"


MATMULS = [([1], 8, 16), ([1], 512, 4096), ([3], 136, 400), ([128], 256, 128), ([129, 0, 1, 260], 264, 272),
           ([17, 40, 0, 200, 5], 640, 1152), ([0, 0], 64, 64), ([300], 1000, 2048), ([2] * 40, 72, 144),
           ([32], 384, 512), ([33], 384, 512), ([31, 0, 1], 264, 656),
           ([650, 100, 0, 700], 520, 400), ([513], 264, 1040), ([8], 24, 4112), ([5], 520, 1040),
           ([9], 264, 272)]


@pytest.mark.parametrize("counts,N,K", MATMULS)
@pytest.mark.parametrize("weighted", [False, True])
def test_matmul(counts, N, K, weighted):
    rng = np.random.default_rng(N * 7 + K + len(counts))
    G, rows = len(counts), sum(counts)
    aq, bq = random_codes(rng, rows, K), random_codes(rng, G, N, K)
    a_s = R.f32(rng.random((rows, R.blocks(K))) + 0.01)
    b_s = R.f32((rng.random((G, R.blocks(N), R.blocks(K))) + 0.01) * 2.0 ** -12)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    f = lambda a: dev(a.astype(np.float32))
    w_rows = rows // 2
    w = R.f32(rng.random(max(w_rows, 1)) + 0.5)
    out = empty(max(rows, 1) + 1, N, dtype=torch.bfloat16, fill=77.0)   # one row behind the end
    pad = np.zeros((1, K), np.uint8)
    _lib.moe_fp8_matmul(dev(np.vstack([aq, pad])), f(np.vstack([a_s, a_s[:1] if rows else
                                                               np.zeros((1, R.blocks(K)))])),
                        counts_offsets(counts), G, max(rows, 1), dev(bq), f(b_s),
                        f(w) if weighted else None, w_rows if weighted else 0, N, K, out)
    ok()
    assert (out[rows:] == 77.0).all()
    lo = 0
    for g, n in enumerate(counts):
        a, b = R.rows_values(aq[lo:lo + n], a_s[lo:lo + n]), R.weight_values(bq[g], b_s[g])
        f_row = np.ones(n)
        if weighted:
            m = np.arange(lo, lo + n) < w_rows
            f_row[m] = w[np.arange(lo, lo + n)[m]]
        check(out[lo:lo + n], (a @ b.T) * f_row[:, None], (np.abs(a) @ np.abs(b).T) * f_row[:, None],
              K, 1, f"group {g}")
        lo += n


def test_matmul_bound_above_rows():
    """max_rows is an upper bound: fewer rows than it says."""
    rng = np.random.default_rng(3)
    N, K, n = 256, 384, 40
    aq, bq = random_codes(rng, 512, K), random_codes(rng, 2, N, K)
    one = lambda *s: torch.full(s, 2.0 ** -9, device="cuda")
    dev = lambda a: torch.from_numpy(a).cuda()
    out = empty(512, N, dtype=torch.bfloat16, fill=5.0)
    _lib.moe_fp8_matmul(dev(aq), one(512, 3), counts_offsets([0, n]), 2, 512, dev(bq),
                        one(2, 2, 3), None, 0, N, K, out)
    ok()
    a, b = R.TABLE[aq[:n]] * 2.0 ** -9, R.TABLE[bq[1]] * 2.0 ** -9
    check(out[:n], a @ b.T, np.abs(a) @ np.abs(b).T, K, 1, "rows")
    assert (out[n:] == 5.0).all()


def test_matmul_keeps_non_finite():
    """A row whose scale is NaN or infinite, or a NaN code, gives no number; the
    other rows do not notice."""
    rng = np.random.default_rng(5)
    for rows in (3, 200):
        N, K = 64, 256
        aq, bq = random_codes(rng, rows, K), random_codes(rng, 1, N, K)
        a_s = np.full((rows, 2), 0.01, np.float32)
        a_s[1, 0], aq[2, 5] = np.nan, 0x7F
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        out = empty(rows, N, dtype=torch.bfloat16)
        _lib.moe_fp8_matmul(dev(aq), dev(a_s), counts_offsets([rows]), 1, rows, dev(bq),
                            torch.full((1, 1, 2), 0.01, device="cuda"), None, 0, N, K, out)
        ok()
        fin = torch.isfinite(out)
        assert not fin[1].any() and not fin[2].any()
        assert fin[0].all() and fin[3:].all()


@pytest.mark.parametrize("counts,M,N", [([1], 8, 8), ([128], 128, 256), ([5, 0, 300, 129], 136, 264),
                                        ([0], 64, 64), ([257, 64], 520, 1032), ([1] * 9, 24, 40)])
def test_wgrad(counts, M, N):
    rng = np.random.default_rng(M + N)
    G, rows = len(counts), sum(counts)
    a, b = (bf16(values(rng, max(rows, 1), C) if rows > 6 else rng.standard_normal((max(rows, 1), C)))
            for C in (M, N))
    if rows > 6:   # keep the products of the extreme rows inside fp32
        a[3:6], b[3:6] = 1.0, 0.5
    dW = empty(G, M, N, dtype=torch.float32, fill=9.0)
    ws = empty(_lib.moe_fp8_wgrad_workspace_size(G, rows, M, N))
    _lib.moe_fp8_wgrad(a.cuda(), b.cuda(), counts_offsets(counts), G, rows, M, N, dW, ws)
    ok()
    lo = 0
    for g, n in enumerate(counts):
        va, vb = (R.column_block_values(f64(t[lo:lo + n])) for t in (a, b))
        check(dW[g], va.T @ vb, np.abs(va).T @ np.abs(vb), n, 0, f"group {g}")
        lo += n


def test_linear_and_its_gradients():
    """A linear layer on operands that the format holds exactly (each block has
    448 as its largest value, the others are small whole numbers): forward, data
    and weight gradient against the formulas, and against differences of the
    loss sum(y dy), which is linear in each operand."""
    rng = np.random.default_rng(11)
    n, N, K = 256, 256, 384

    def grid(*s):
        # exact in either direction: one 448 in each 128-block of a row and of a column
        v = rng.integers(-8, 9, s).astype(np.float64)
        for i in range(0, s[0], 128):
            for j in range(0, s[1], 128):
                p = rng.permutation(128)
                v[i + np.arange(128), j + p] = 448.0
        return v
    x, w, dy = grid(n, K), grid(N, K), grid(n, N)
    up = lambda a: bf16(a).cuda()
    offs = counts_offsets([n])
    wq, wqt = empty(1, N, K), empty(1, K, N)
    wsc, wst = empty(1, 2, 3, dtype=torch.float32), empty(1, 3, 2, dtype=torch.float32)
    _lib.moe_fp8_quantize_weights(up(w)[None].contiguous(), 1, N, K, wq, wsc, wqt, wst)

    def rows(a):
        q, s = empty(*a.shape), empty(a.shape[0], R.blocks(a.shape[1]), dtype=torch.float32)
        _lib.moe_fp8_quantize(up(a), a.shape[0], a.shape[1], q, s)
        return q, s
    y, dx = empty(n, N, dtype=torch.bfloat16), empty(n, K, dtype=torch.bfloat16)
    _lib.moe_fp8_matmul(*rows(x), offs, 1, n, wq, wsc, None, 0, N, K, y)
    _lib.moe_fp8_matmul(*rows(dy), offs, 1, n, wqt, wst, None, 0, K, N, dx)
    dW = empty(1, N, K, dtype=torch.float32)
    ws = empty(_lib.moe_fp8_wgrad_workspace_size(1, n, N, K))
    _lib.moe_fp8_wgrad(up(dy), up(x), offs, 1, n, N, K, dW, ws)
    ok()
    check(y, x @ w.T, np.abs(x) @ np.abs(w).T, K, 1, "y")
    check(dx, dy @ w, np.abs(dy) @ np.abs(w), N, 1, "dx")
    check(dW[0], dy.T @ x, np.abs(dy).T @ np.abs(x), n, 0, "dW")
    loss = lambda x, w: np.sum((x @ w.T) * dy)
    for i, j in [(0, 0), (200, 383), (17, 130)]:
        for which, got, tol in (("x", f64(dx)[i, j], 2.0 ** -8), ("w", f64(dW)[0, i, j], 1e-4)):
            a = dict(x=x.copy(), w=w.copy())
            a[which][i, j] += 1.0
            up_loss = loss(a["x"], a["w"])
            a[which][i, j] -= 2.0
            diff = (up_loss - loss(a["x"], a["w"])) / 2.0
            scale = np.abs(dy[i]) @ np.abs(w[:, j]) if which == "x" else np.abs(dy[:, i]) @ np.abs(x[:, j])
            assert abs(got - diff) <= tol * abs(diff) + sum_bound(384) * scale


# ---------------------------------------------------------------------- FFN

@pytest.mark.parametrize("counts,d,I", [([1], 128, 128), ([130, 0, 1, 77], 256, 128),
                                        ([64, 200], 384, 640), ([3, 2, 9], 512, 256), ([520, 129, 385], 256, 384)])
def test_ffn(counts, d, I):
    rng = np.random.default_rng(d + I)
    G, rows, clamp = len(counts), sum(counts), 2.0
    xq, w13, w2 = random_codes(rng, rows, d), random_codes(rng, G, 2 * I, d), random_codes(rng, G, d, I)
    sc = lambda std, *s: R.f32((rng.random(s) + 0.5) * std / 100)
    x_s = sc(1.0, rows, R.blocks(d))
    s13, s2 = sc(1.3 / d ** 0.5, G, 2 * I // 128, d // 128), sc(1.3 / I ** 0.5, G, d // 128, I // 128)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    f = lambda a: dev(a.astype(np.float32))
    w = R.f32(rng.random(rows) + 0.1)
    S = rows - rows // 3
    hq, hs = empty(rows, I), empty(rows, I // 128, dtype=torch.float32)
    y = empty(rows, d, dtype=torch.bfloat16)
    _lib.moe_expert_ffn_fp8(dev(xq), f(x_s), counts_offsets(counts), G, rows, dev(w13), f(s13),
                            dev(w2), f(s2), f(w), S, d, I, clamp, hq, hs, y)
    ok()
    lo = 0
    for g, n in enumerate(counts):
        r = slice(lo, lo + n)
        gu = R.rows_values(xq[r], x_s[r]) @ R.weight_values(w13[g], s13[g]).T
        h = R.silu_clamped(gu[:, :I], gu[:, I:], clamp)
        rq, rs = R.quantise_rows(h)
        if n:
            # scales: the fp32 sums and the fast exponential differ by ~1e-6 of
            # the largest value; codes: a value that close to a rounding boundary
            # (spacing >= 2^-4 of it) may round the other way, ~1e-5 / 2^-4 of them
            assert np.allclose(f64(hs[r]), rs, rtol=1e-4, atol=0)
            mine = R.rows_values(codes(hq[r]), f64(hs[r]))
            step = np.repeat(rs, 128, 1) * np.maximum(2.0 ** -9, np.abs(R.TABLE[rq]) * 2.0 ** -3)
            off = np.abs(mine - R.rows_values(rq, rs))
            assert (off <= 1.01 * step).all()
            assert np.mean(off > 0.25 * step) <= 2e-3
            b = R.weight_values(w2[g], s2[g])
            f_row = np.where(np.arange(lo, lo + n) < S, w[r], 1.0)[:, None]
            check(y[r], (mine @ b.T) * f_row, (np.abs(mine) @ np.abs(b).T) * f_row, I, 1, f"y {g}")
        lo += n


# ------------------------------------------------- streams, graphs, refusals

def test_other_stream_and_graph():
    rng = np.random.default_rng(2)
    n, N, K = 50, 256, 256
    x = bf16(rng.standard_normal((n, K))).cuda()
    bq = torch.from_numpy(random_codes(rng, 1, N, K)).cuda()
    b_s = torch.full((1, 2, 2), 0.01, device="cuda")
    offs = counts_offsets([n])
    q, s = empty(n, K), empty(n, 2, dtype=torch.float32)
    outs = []

    def step(stream):
        out = empty(n, N, dtype=torch.bfloat16, fill=0.0)
        outs.append(out)
        return lambda: (_lib.moe_fp8_quantize(x, n, K, q, s, stream),
                        _lib.moe_fp8_matmul(q, s, offs, 1, n, bq, b_s, None, 0, N, K, out, stream))
    step(None)()
    ok()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)()
    side.synchronize()
    run = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    q.zero_()
    graph.replay()
    ok()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_places_behind_32_bits():
    """Weights of more than 2^32 bytes and codes of more than 2^31: the last
    group's products and the last rows' codes."""
    G, N, K, rows = 520, 2048, 4096, 37
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    assert w.numel() * 2 > 2 ** 32 and w.numel() > 2 ** 31
    last = (torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5).to(torch.bfloat16)
    w[-1] = last
    q, qt = (torch.empty(G, *s, dtype=torch.uint8, device="cuda") for s in ((N, K), (K, N)))
    s = torch.empty(G, N // 128, K // 128, device="cuda")
    st = torch.empty(G, K // 128, N // 128, device="cuda")
    _lib.moe_fp8_quantize_weights(w, G, N, K, q, s, qt, st)
    one = [torch.empty(1, *t.shape[1:], dtype=t.dtype, device="cuda") for t in (q, s, qt, st)]
    _lib.moe_fp8_quantize_weights(last[None].contiguous(), 1, N, K, *one)
    for t, o in zip((q, s, qt, st), one):
        assert torch.equal(t[-1], o[0]) and not (t[-2].float() * (t.dtype == torch.uint8)).any()
    # the same rows as the last group's and as a group of its own
    x = torch.randn(rows, K, generator=gen, device="cuda").to(torch.bfloat16)
    xq, xs = torch.empty(rows, K, dtype=torch.uint8, device="cuda"), torch.empty(rows, K // 128,
                                                                                 device="cuda")
    _lib.moe_fp8_quantize(x, rows, K, xq, xs)
    offsets = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = rows
    a, b = (torch.empty(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _lib.moe_fp8_matmul(xq, xs, offsets, G, rows, q, s, None, 0, N, K, a)
    _lib.moe_fp8_matmul(xq, xs, offsets[-2:].contiguous(), 1, rows, one[0], one[1], None, 0, N, K, b)
    # (each one bf16 rounding of the same sums)
    torch.testing.assert_close(a, b, rtol=2.0 ** -7, atol=1e-4)
    assert float(a.float().std()) > 0.5
    # rows quantised in place: the last of more than 2^31 elements
    flat = w.view(-1, 128)
    _lib.moe_fp8_quantize(flat, flat.shape[0], 128, q.view(-1, 128), torch.empty(
        flat.shape[0], 1, device="cuda"))
    tail = torch.empty(N * K // 128, 128, dtype=torch.uint8, device="cuda")
    _lib.moe_fp8_quantize(last, N * K // 128, 128, tail, torch.empty(N * K // 128, 1, device="cuda"))
    assert torch.equal(q[-1].view(-1, 128), tail)
    ok()
