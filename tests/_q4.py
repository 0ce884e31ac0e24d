"""Inputs of the 4-bit pool's tests, and the error bounds they are held to."""
from __future__ import annotations

import numpy as np
import torch

from _paged import D_C, GARBAGE, ROW, SCALE, attention_bounds, f64, half_step
from oracle import fp4_oracle as F
from oracle import paged_oracle as PO


def bf16_bits(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def from_bf16_bits(u):
    return torch.from_numpy(np.ascontiguousarray(u).view(np.int16)).view(torch.bfloat16).double().numpy()


def values(pool, page):
    """Rows [pages, page, 576] in fp64 of a 4-bit pool's bytes."""
    code, e, key = F.unpack(pool, page)
    return np.concatenate([F.latents(code, e), from_bf16_bits(key)], -1)


def make_pool(rng, lengths, page, extra_pages=3, width=None, gain=None):
    """A 4-bit pool's bytes, its block table and its number of pages, drawn from ``rng``.

    Rows past a sequence's end and the pages nobody holds have random codes, every
    exponent bit set and NaN keys; table entries past a sequence's last page are numbers
    that name no page.
    """
    need = [-(-int(n) // page) for n in lengths]
    pages = sum(need) + extra_pages
    width = width or max(max(need), 1) + 2
    ids = rng.permutation(pages)
    table = np.array([[GARBAGE[(b + j) % len(GARBAGE)] for j in range(width)]
                      for b in range(len(lengths))], np.int64)
    x = rng.randn(pages, page, ROW).astype(np.float32)
    if gain is not None:                       # some rows of large magnitude
        x[rng.rand(pages, page) < 0.02] *= gain
    x[..., :D_C] *= np.exp2(rng.randint(-3, 3, D_C))       # channels of different magnitude
    live = np.zeros((pages, page), bool)
    k = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[k:k + n]
        k += n
        for t in range(int(lengths[b])):
            live[table[b, t // page], t % page] = True
    e = F.exponents(x[..., :D_C])
    code = F.codes(x[..., :D_C], e)
    key = bf16_bits(x[..., D_C:])
    code[~live] = rng.randint(0, 16, ((~live).sum(), D_C))
    e[~live] = 7                               # the bits 15, which no row has
    key[~live] = 0x7FFF
    return (torch.from_numpy(F.pack(code, e, key)), torch.from_numpy(table.astype(np.int32)), pages)


def bounds(q, rows, p, z, io, heads, q_len):
    """Elementwise bounds of |o - exact| and |lse - exact| for one token.

    Every cached value is exact in the tensor cores' operands.  fp32 queries: the E4M3
    cache's bounds (a query within 2^-16 of the head's largest value, weights within 2^-12
    and 2^-18 of the largest one).  bf16 queries: weights are two E4M3 parts (half a step
    is 2^-4 of each: 2^-8, and 2^-19 of the largest weight) or, in SM pairs, a part and its
    E5M2 remainder (2^-7, 2^-19); queries within 2^-17 of the head's largest value.
    """
    one = attention_bounds(q, rows, p, z, "fp8", torch.float32, heads, q_len)
    if io == torch.float32:
        return one
    two = attention_bounds(q, rows, p, z, "fp8", io, max(heads, 48), q_len)
    return np.maximum(one[0], two[0]), np.maximum(one[1], two[1])


def check_attention(got_o, got_lse, q_abs, q_pe, pool, page, table, lengths, q_len, io, tokens=None):
    """Every token's output and lse against the exact ones, element by element."""
    q = np.concatenate([f64(q_abs), f64(q_pe)], 2)
    pool64, tab = values(pool.cpu().numpy(), page), table.cpu().numpy()
    o, lse = f64(got_o), f64(got_lse)
    R, H = q.shape[:2]
    worst = 0.0
    for r in range(R) if tokens is None else tokens:
        b = r // q_len
        n = max(int(lengths[b]) - (q_len - 1 - r % q_len), 0)
        ok = [0 <= t < len(pool64) for t in tab[b, :-(-n // page)]]
        rows = np.concatenate([pool64[t] if good else np.zeros((page, ROW))
                               for t, good in zip(tab[b], ok)] + [np.zeros((0, ROW))])[:n]
        want, want_lse, p, z = PO.attend(q[r], rows, SCALE, D_C)
        if n == 0:
            assert (o[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        do, dl = bounds(q[r], rows, p, z, io, H, q_len)
        do = do + half_step(io) * (np.abs(want) + do) + 1e-30
        assert np.isfinite(o[r]).all() and np.isfinite(lse[r]).all(), f"token {r}"
        worst = max(worst, float((np.abs(o[r] - want) / do).max()),
                    float((np.abs(lse[r] - want_lse) / (dl + 2.0 ** -22 * np.abs(want_lse))).max()))
        assert worst <= 1.0, f"token {r} of {R}: {worst:.3g} of the bound"
    return worst
