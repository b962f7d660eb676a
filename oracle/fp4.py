"""The 4-bit cache: e2m1 codes under an e4m3 scale per 16 head dims, as plain NumPy.

Test infrastructure only (see the package docstring).  The format:

* e2m1: 1 sign bit, 2 exponent bits with bias 1, 1 mantissa bit, no infinity, no NaN: the magnitudes
  0, 0.5, 1, 1.5, 2, 3, 4, 6;
* a row (one position, one kv head, K or V) of 128 head dims is 64 bytes of codes, dim 2i in byte i's low
  nibble, and 8 e4m3 scale bytes, one per 16 dims; value = code * scale * k_scale[g];
* storage row R lies in half-block R // 128: 128 rows' codes, then the 128 rows' scales (9,216 bytes).

The store, every product and quotient rounded to float32: a NaN counts as 0; scale = e4m3(amax / (6 g)),
code = e2m1(x / (scale g)), both to nearest even and saturating; a block whose scale is 0 holds zeros.
"""

import numpy as np

from . import e4m3

HALF_ROWS = 128
CODE_BYTES, SCALE_BYTES = 64, 8
HALF_BYTES = HALF_ROWS * (CODE_BYTES + SCALE_BYTES)
BLOCK = 2 * HALF_BYTES
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes):
    """e2m1 codes (0..15) to float64."""
    c = np.asarray(codes, dtype=np.int64)
    v = MAGNITUDES[c & 7]
    return np.where(c & 8, -v, v)


def encode_f32(x):
    """float32 (no NaN) to e2m1 codes: nearest, ties to the even code, saturating; the sign is kept."""
    x = np.asarray(x, dtype=np.float32)
    a = np.minimum(np.abs(x.astype(np.float64)), 6.0)
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best                                   # one code, or two at a tie
    code = np.argmax(near & (np.arange(8) % 2 == 0) | (near & (near.sum(-1, keepdims=True) == 1)), axis=-1)
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def quantise(x, g):
    """float32 [..., 128] and the kv head's scale: codes uint8 [..., 64], scales uint8 [..., 8]."""
    x = np.asarray(x, dtype=np.float32)
    g = np.float32(g)
    x = np.where(np.isnan(x), np.float32(0), x)
    b = x.reshape(*x.shape[:-1], 8, 16)
    with np.errstate(all="ignore"):
        u = (np.abs(b).max(-1) / np.float32(g * np.float32(6))).astype(np.float32)
        u = np.where(u > 0, u, np.float32(0))
        s = e4m3.encode_f32(u)
        step = (e4m3.decode(s).astype(np.float32) * g).astype(np.float32)[..., None]
        y = np.where(step > 0, (b / step).astype(np.float32), np.float32(0))
    code = encode_f32(y).reshape(x.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), s


def dequantise(codes, scales, g):
    """float64 [..., 128] of codes [..., 64] and scale bytes [..., 8]."""
    codes = np.asarray(codes)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 128)
    s = np.repeat(e4m3.decode(scales), 16, axis=-1)
    return decode(c) * s * np.float64(np.float32(g))


def views(arr):
    """Codes [rows][64] and scales [rows][8] of a pool or slab, as views of its bytes."""
    h = arr.reshape(-1, HALF_BYTES)
    n = HALF_ROWS * CODE_BYTES
    assert h.base is not None or h is arr
    return h[:, :n].reshape(len(h), HALF_ROWS, CODE_BYTES), h[:, n:].reshape(len(h), HALF_ROWS, SCALE_BYTES)


def row_of(seg, hkv, g, pos):
    """Storage row of position(s) pos of kv head g."""
    pos = np.asarray(pos, dtype=np.int64)
    if seg.page_table is not None:
        return (np.asarray(seg.page_table, np.int64)[pos // 256] * hkv + g) * 256 + pos % 256
    return g * (seg.k_slab.shape[1] * 256) + pos


def _arr(cache, seg, which):
    if seg.page_table is not None:
        return cache.k_pool if which == "k" else cache.v_pool
    return seg.k_slab if which == "k" else seg.v_slab


def get_rows(cache, seg, which, g, pos):
    """Stored (codes, scales) of positions pos."""
    r = row_of(seg, cache.hkv, g, pos)
    codes, scales = views(_arr(cache, seg, which))
    return codes[r // HALF_ROWS, r % HALF_ROWS].copy(), scales[r // HALF_ROWS, r % HALF_ROWS].copy()


def set_rows(cache, seg, which, g, pos, codes_new, scales_new):
    r = row_of(seg, cache.hkv, g, pos)
    arr = _arr(cache, seg, which)
    flat = arr.reshape(-1)
    assert np.shares_memory(flat, arr)
    base = (r // HALF_ROWS) * HALF_BYTES
    at = base + (r % HALF_ROWS) * CODE_BYTES
    flat[at[..., None] + np.arange(CODE_BYTES)] = codes_new
    at = base + HALF_ROWS * CODE_BYTES + (r % HALF_ROWS) * SCALE_BYTES
    flat[at[..., None] + np.arange(SCALE_BYTES)] = scales_new


def gather(cache, seg, g, n):
    """K and V of kv head g at positions 0..n-1, float64."""
    pos = np.arange(n)
    return (dequantise(*get_rows(cache, seg, "k", g, pos), cache.k_scale[g]),
            dequantise(*get_rows(cache, seg, "v", g, pos), cache.v_scale[g]))
