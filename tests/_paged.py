"""Inputs of the paged-cache GPU tests, and the error bounds they are held to."""
from __future__ import annotations

import numpy as np
import torch

from oracle import mla_oracle as O
from oracle import paged_oracle as PO

D_C, D_R, ROW = 512, 64, 576
SCALE = 192 ** -0.5
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
GARBAGE = (-1, -7, 1 << 30, -(1 << 31), 123456789)     # table entries that nothing may use


def f64(t):
    """Exact fp64 values of a tensor."""
    t = t.detach().cpu()
    if t.dtype == torch.float8_e4m3fn:
        return O.e4m3_to_float64(t.view(torch.uint8).numpy())
    return t.double().numpy()


def make_pool(rng, lengths, page, dtype, extra_pages=3, width=None, poison=True, gain=None):
    """A pool, its block table and the page order drawn from ``rng``.

    Rows past a sequence's end and the pages nobody holds are NaN; table entries
    past a sequence's last page are numbers that name no page.
    """
    need = [-(-int(n) // page) for n in lengths]
    pages = sum(need) + extra_pages
    width = width or max(max(need), 1) + 2
    ids = rng.permutation(pages)
    table = np.array([[GARBAGE[(b + j) % len(GARBAGE)] for j in range(width)]
                      for b in range(len(lengths))], np.int64)
    pool = rng.randn(pages, page, ROW).astype(np.float32)
    if gain is not None:                       # some rows of large magnitude
        hit = rng.rand(pages, page) < 0.02
        pool[hit] *= gain
    live = np.zeros((pages, page), bool)
    k = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[k:k + n]
        k += n
        for t in range(int(lengths[b])):
            live[table[b, t // page], t % page] = True
    t = torch.from_numpy(pool).to(DT[dtype])
    if poison:
        if dtype == "fp8":
            t.view(torch.uint8)[torch.from_numpy(~live)] = 0x7F
        else:
            t[torch.from_numpy(~live)] = float("nan")
    return t, torch.from_numpy(table.astype(np.int32)), pages


def make_queries(rng, rows, heads, io):
    q_abs = torch.from_numpy((rng.randn(rows, heads, D_C) * 0.3).astype(np.float32)).to(io)
    q_pe = torch.from_numpy(rng.randn(rows, heads, D_R).astype(np.float32)).to(io)
    return q_abs, q_pe


def attention_bounds(q, rows, p, z, dtype, io, heads, q_len):
    """Elementwise bounds of |o - exact| and |lse - exact| for one token.

    q [H, 576], rows [n, 576] exact inputs; p [H, n] exact weights; z [H] exact
    sums of exp(s - max).  Half a step is 2^-8 of a bf16 value and 2^-4 of an E4M3
    one.  Per score: the query's rounding (hi + lo bf16 pairs 2^-16 of each value;
    E4M3 parts in units of the head's largest value: four 2^-16, two of a bf16
    query the last part's smallest step, 2^-17; bf16 and fp32 queries otherwise
    none), products summed in fp32 (600 terms of 2^-23, the tensor core
    truncating), and the softmax's base change and exp2 (2^-21 of the score, 2^-20
    of the weight).  Per weight: hi + lo 2^-16, one part 2^-8, three E4M3 parts
    2^-12 and 2^-18 of the largest weight, an E4M3 part and its E5M2 remainder (half
    a step 2^-3) 2^-7 and 2^-19.  The sums over
    rows add (n + 200) 2^-23 of the sum of magnitudes; the output rounds by half a
    step of its type.
    """
    n = len(rows)
    a = np.abs(q) @ np.abs(rows).T * SCALE                     # [H, n] sums of |q c|
    two = dtype == "fp8" and io == torch.bfloat16 and heads * q_len >= 48   # the SM pairs
    if dtype == "fp8":
        dq = (2.0 ** (-17 if two else -16) * np.abs(q).max(1, keepdims=True)
              * np.abs(rows).sum(1)[None] * SCALE)
        dp, floor = (2.0 ** -7, 2.0 ** -19) if two else (2.0 ** -12, 2.0 ** -18)
    else:
        dq = (2.0 ** -16 if dtype == "bf16" and io == torch.float32 else 0.0) * a
        one = dtype == "bf16" and io == torch.bfloat16 and heads * q_len >= 32   # the SM pairs
        dp = 0.0 if dtype == "f32" else 2.0 ** -8 if one else 2.0 ** -16
        floor = 0.0
    ds = (dq + a * (600 * 2.0 ** -23 + 2.0 ** -21)).max(1)     # [H]
    rel = 2 * ds + dp + 2.0 ** -20 + (n + 200) * 2.0 ** -23
    mag = p @ np.abs(rows[:, :D_C])                            # [H, 512]
    tail = floor / z[:, None] * np.abs(rows[:, :D_C]).sum(0)[None]
    do = 2 * rel[:, None] * mag + 2 * tail
    summed = 2 * dp + n * floor / z if dtype == "fp8" and not two else 0.0   # else unrounded
    dl = ds + summed + 2.0 ** -19 + (n + 200) * 2.0 ** -23
    return do, dl


def half_step(io):
    return torch.finfo(io).eps / 2


def check_attention(got_o, got_lse, q_abs, q_pe, pool, table, lengths, q_len, dtype, io,
                    tokens=None):
    """Every token's output and lse against the exact ones, element by element."""
    q = np.concatenate([f64(q_abs), f64(q_pe)], 2)
    pool64, tab = f64(pool), table.cpu().numpy()
    o, lse = f64(got_o), f64(got_lse)
    R, H = q.shape[:2]
    worst = 0.0
    for r in range(R) if tokens is None else tokens:
        b = r // q_len
        n = max(int(lengths[b]) - (q_len - 1 - r % q_len), 0)
        rows = PO.sequence_rows(pool64, tab[b], n)
        want, want_lse, p, z = PO.attend(q[r], rows, SCALE, D_C)
        if n == 0:
            assert (o[r] == 0).all() and np.isneginf(lse[r]).all()
            continue
        do, dl = attention_bounds(q[r], rows, p, z, dtype, io, H, q_len)
        do = do + half_step(io) * (np.abs(want) + do) + 1e-30   # 0 against 0 where every row has a 0
        assert np.isfinite(o[r]).all() and np.isfinite(lse[r]).all(), f"token {r}"
        worst = max(worst, float((np.abs(o[r] - want) / do).max()),
                    float((np.abs(lse[r] - want_lse) / (dl + 2.0 ** -22 * np.abs(want_lse))).max()))
        assert worst <= 1.0, f"token {r} of {R}: {worst:.3g} of the bound"
    return worst
