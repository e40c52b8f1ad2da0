"""Plain 64-bit implementation of the MXFP4 format and of the matmuls with MXFP4
weights, for the tests.  E2M1 elements in blocks of 32 with a power of two each."""
import numpy as np

from tests import fp8_ref as F

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TABLE = np.concatenate([GRID, -GRID])     # the value of each of the sixteen codes


def pitch(K):
    return (K // BLOCK + 15) // 16 * 16


def e2m1_codes(v):
    """Codes of the nearest values, ties to the even code, above 6 to 6, the sign kept."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.minimum(np.abs(v), 6.0)
    hi = np.clip(np.searchsorted(GRID, mag), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = mag - GRID[lo], GRID[hi] - mag
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(v), c | 8, c).astype(np.uint8)


def _scale_codes(amax, top):
    """E8M0 codes [...] of blocks whose largest magnitudes are amax."""
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(amax > 0, amax, 1.0)))
    e = np.where(amax >= 2.0 ** (e + 1), e + 1, np.where(amax < 2.0 ** e, e - 1, e))
    return np.where(amax > 0, np.clip(e - top, -127, 127) + 127, 0).astype(np.uint8)


def scale(code):
    c = np.asarray(code).astype(np.float64)
    return np.where(c == 255, np.nan, 2.0 ** (np.minimum(c, 254) - 127))


def quantise4(v):
    """[rows, K] float64 (finite) -> element codes [rows, K], scale codes [rows, K/32]."""
    b = v.reshape(v.shape[0], v.shape[1] // BLOCK, BLOCK)
    s = _scale_codes(np.abs(b).max(2), 2)
    return e2m1_codes(b / scale(s)[:, :, None]).reshape(v.shape), s


def quantise8(v):
    """The same in MXFP8 (E4M3): codes [rows, K], scale codes."""
    b = v.reshape(v.shape[0], v.shape[1] // BLOCK, BLOCK)
    s = _scale_codes(np.abs(b).max(2), 8)
    return F.e4m3_codes(b / scale(s)[:, :, None]).reshape(v.shape), s


def pack(c):
    """Element codes [rows, K] -> bytes [rows, K/2], the even element in the low nibble."""
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    c = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
    return c


def values4(c, s):
    return TABLE[c] * np.repeat(scale(s), BLOCK, axis=1)


def values8(c, s):
    return F.TABLE[c] * np.repeat(scale(s), BLOCK, axis=1)
