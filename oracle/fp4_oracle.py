"""Plain NumPy definition of the 4-bit pool (MLA_FP4_E2M1), for the tests.

Values and rounding in fp64, and the byte layout of a page restated from its description
in the CUDA sources, so that tests can make pools without the library and read what it
wrote.  Nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

D_C, D_R, BLOCK = 512, 64, 16
ROW_BYTES = 400
E_MIN, E_MAX = -8, 6
# bits of a 32-bit word of eight codes: their magnitudes' lowest, and their signs
MAG = np.arange(0, 32, 4, dtype=np.uint64)
SIGN = np.array([7, 15, 23, 31, 3, 11, 19, 27], np.uint64)
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def exponents(x):
    """x [..., 512]: e per block of 16, the smallest in [-8, 6] with max |x| <= 7 2^e (6
    where there is none, for infinities and for NaN)."""
    x = np.asarray(x, np.float64)
    v = np.abs(x.reshape(x.shape[:-1] + (D_C // BLOCK, BLOCK)))
    top = np.where(np.isnan(v), np.inf, v).max(-1)
    e = np.full(top.shape, E_MIN)
    for k in range(E_MIN, E_MAX):
        e = np.where(top > 7.0 * 2.0 ** k, k + 1, e)
    return e


def codes(x, e):
    """E2M1 codes of x in units of 2^e: to nearest, ties to the even code, at most 6."""
    x = np.asarray(x, np.float64)
    v = x.reshape(x.shape[:-1] + (D_C // BLOCK, BLOCK))
    y = np.abs(v) / 2.0 ** e[..., None]
    y = np.where(np.isnan(y), np.inf, y)
    mids = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(y.shape, np.int64)
    for k, mid in enumerate(mids):           # code k below mid, k + 1 above
        code = np.where((y > mid) | ((y == mid) & (k % 2 == 1)), k + 1, code)
    sign = np.signbit(v) & ~np.isnan(v)
    return (code | sign.astype(np.int64) << 3).reshape(x.shape)


def latents(code, e):
    """The values of codes [..., 512] and exponents [..., 32] in fp64."""
    code, e = np.asarray(code), np.minimum(np.asarray(e), E_MAX)
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    shape = v.shape
    return (v.reshape(shape[:-1] + (D_C // BLOCK, BLOCK)) * 2.0 ** e[..., None].astype(np.float64)).reshape(shape)


def rounded(x):
    """Latents as a 4-bit pool holds them."""
    e = exponents(x)
    return latents(codes(x, e), e)


def pack(code, e, key):
    """Pages [n, R] of codes [n, R, 512], exponents [n, R, 32] (-8 .. 7: 7 is no exponent and
    reads as 6) and key bits [n, R, 64] uint16 as the pool's bytes [n, R * 400]."""
    n, R = code.shape[:2]
    w = np.asarray(code, np.uint64).reshape(n, R, D_C // 8, 8)
    word = ((w & np.uint64(7)) << MAG).sum(-1) | ((w >> np.uint64(3)) << SIGN).sum(-1)
    c = word.astype("<u4").view(np.uint8).reshape(n, R, D_C // 2)
    u = (np.asarray(e) + 5) & 15
    x = (u[..., 0::2] | u[..., 1::2] << 4).astype(np.uint8)
    k = np.ascontiguousarray(key).view(np.uint8).reshape(n, R, 8, 16)
    at = np.arange(8)[None, :] ^ (np.arange(R)[:, None] & 7)
    moved = np.empty_like(k)
    np.put_along_axis(moved, np.broadcast_to(at[None, :, :, None], k.shape), k, 2)
    return np.concatenate([np.concatenate([c, x], -1).reshape(n, -1), moved.reshape(n, -1)], 1)


def unpack(pool, page):
    """pack()'s arguments of a pool's bytes."""
    n = pool.size // (page * ROW_BYTES)
    p = np.asarray(pool, np.uint8).reshape(n, page * ROW_BYTES)
    c, k = np.split(p, [page * 272], 1)
    c, k = c.reshape(n, page, 272), k.reshape(n, page, 8, 16)
    c, x = c[..., :256], c[..., 256:]
    w = np.ascontiguousarray(c).view("<u4").astype(np.uint64)[..., None]
    code = ((w >> MAG & np.uint64(7)) | (w >> SIGN & np.uint64(1)) << np.uint64(3)).reshape(n, page, D_C).astype(np.int64)
    e = np.stack([x & 15, x >> 4], -1).reshape(n, page, D_C // BLOCK).astype(np.int64)
    e = ((e + 3) & 15) - 8
    at = np.arange(8)[None, :] ^ (np.arange(page)[:, None] & 7)
    key = np.take_along_axis(k, np.broadcast_to(at[None, :, :, None], k.shape), 2)
    return code, e, np.ascontiguousarray(key).view(np.uint16).reshape(n, page, D_R)
