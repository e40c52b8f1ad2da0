"""Plain 64-bit implementation of the FP8 format with a scale for each block
of 128, of the matmuls on it and of the few-token layer, for the tests.

Only the roundings that the format names are made: a block's scale, its
factor and each scaled value are fp32 numbers; everything else is float64."""
import numpy as np

BLOCK = 128
FLOOR = 2.0 ** -100


def blocks(n):
    return -(-n // BLOCK)


def f32(a):
    return np.asarray(a, dtype=np.float64).astype(np.float32).astype(np.float64)


def e4m3_values():
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else a
        if c & 128:
            v[c] = -v[c]
    return v


TABLE = e4m3_values()


def e4m3_codes(v):
    """Codes of the nearest E4M3 values, ties to the even code, magnitudes above
    448 to 448, the sign kept; NaN to 0x7F."""
    v = np.asarray(v, dtype=np.float64)
    grid = TABLE[:127]
    mag = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(grid, np.nan_to_num(mag)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - grid[lo], grid[hi] - mag
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(v), c | 128, c).astype(np.uint8)
    return np.where(np.isnan(v), np.uint8(0x7F), c).astype(np.uint8)


def scale_factor(amax):
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.where(amax < FLOOR, FLOOR, amax)
        return f32(m / 448.0), f32(448.0 / m)


def _quantise(v, axis):
    """v with one block along `axis` -> codes, scale (axis kept with length 1)."""
    with np.errstate(invalid="ignore"):
        s, r = scale_factor(np.max(np.abs(v), axis=axis, keepdims=True))
        return e4m3_codes(f32(v * r)), s


def quantise_rows(v):
    """[rows, K] float64 -> codes [rows, K], scales [rows, ceil(K/128)]."""
    rows, K = v.shape
    q = np.empty((rows, K), np.uint8)
    s = np.empty((rows, blocks(K)))
    for b in range(blocks(K)):
        c = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        q[:, c], sc = _quantise(v[:, c], 1)
        s[:, b] = sc[:, 0]
    return q, s


def quantise_weights(w):
    """[N, K] -> codes [N, K], scales [ceil(N/128), ceil(K/128)]."""
    N, K = w.shape
    q = np.empty((N, K), np.uint8)
    s = np.empty((blocks(N), blocks(K)))
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            t = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            q[t], sc = _quantise(w[t], (0, 1))
            s[i, j] = sc[0, 0]
    return q, s


def rows_values(q, s):
    return TABLE[q] * np.repeat(np.asarray(s, np.float64), BLOCK, 1)[:, : q.shape[1]]


def weight_values(q, s):
    e = np.repeat(np.repeat(np.asarray(s, np.float64), BLOCK, 0), BLOCK, 1)
    return TABLE[q] * e[: q.shape[0], : q.shape[1]]


def column_block_values(v):
    """[rows, C] of one group, quantised in blocks of 128 rows, every column of a
    block on its own -> the values it stands for."""
    out = np.empty_like(v)
    for r in range(0, v.shape[0], BLOCK):
        q, s = _quantise(v[r:r + BLOCK], 0)
        out[r:r + BLOCK] = TABLE[q] * s
    return out


def silu_clamped(g, u, c):
    a = np.minimum(g, c)
    return a / (1.0 + np.exp(-a)) * np.clip(u, -c, c)


def few_layer(x, W_g, W13, W2, k, scaling, clamp, offset=None, bias=None, vision=None, ids=None):
    """The layer in float64.  W13(e), W2(e): an expert's weights.  ids: the
    table's experts (hash mode).  Returns y, ids, weights, the smallest distance
    between a selected and an unselected key, and sum |h| |W2| weighted."""
    T = x.shape[0]
    E = W_g.shape[0]
    z = x @ W_g.T + (0 if offset is None else offset)
    s = 1.0 / (1.0 + np.exp(-z))
    gap = np.inf
    if ids is None:
        key = s + bias[np.zeros(T, int) if vision is None else vision.astype(int)]
        order = np.argsort(-key, axis=1, kind="stable")
        ids = order[:, :k]
        if k < E:
            sk = np.take_along_axis(key, order, 1)
            gap = float(np.min(sk[:, :k] - sk[:, 1:k + 1]))
    sel = np.take_along_axis(s, ids, 1)
    w = scaling * sel / sel.sum(1, keepdims=True)
    y = np.zeros_like(x)
    scale = np.zeros_like(x)
    I = W2(E).shape[1]
    for e in [E] + sorted(set(ids.ravel().tolist())):
        t, j = (np.arange(T), None) if e == E else np.nonzero(ids == e)
        gu = x[t] @ W13(e).T
        h = silu_clamped(gu[:, :I], gu[:, I:], clamp)
        f = np.ones(T) if e == E else w[t, j]
        np.add.at(y, t, f[:, None] * (h @ W2(e).T))
        np.add.at(scale, t, f[:, None] * (np.abs(h) @ np.abs(W2(e)).T))
    return y, ids, w, gap, scale
