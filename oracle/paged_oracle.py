"""Plain NumPy definitions of the paged cache's operators, for the tests.

Integers and fp64 throughout, except where an operator is defined by a chain of
fp32 roundings (the page index and the page score): those chains are spelled out
in fp32, one rounding per line.  Nothing here is shared with the CUDA path.

The cache is a pool of pages ("Transformer and KV Cache Basics": the
preallocated cache buffer whose overflow is an error), a row of a page is the
latent row of "Multi-Head Latent Attention" 3.6.
"""
from __future__ import annotations

import math

import numpy as np

from . import mla_oracle as O

LENGTH, PAGE, EXHAUSTED = 1, 8, 16          # status bits
TINY = np.float32(1e-30)


def extend(cached, new, table, free_list, num_free, page, num_pages, max_tokens):
    """One step's tables and slots; returns a dict, ``table`` copied."""
    B, width = table.shape
    table = table.copy()
    need = [-(-(c + n) // page) - -(-c // page) if c >= 0 and n >= 0 else 0
            for c, n in zip(cached, new)]
    status = 0
    if any(c < 0 or n < 0 or c + n > width * page for c, n in zip(cached, new)):
        status |= LENGTH
    good = [(c, n) for c, n in zip(cached, new) if c >= 0 and n >= 0 and c + n <= width * page]
    if sum(n for _, n in good) > max_tokens:
        status |= LENGTH
    wanted = sum(-(-(c + n) // page) - -(-c // page) for c, n in good)
    if not 0 <= num_free <= num_pages or wanted > num_free:
        status |= EXHAUSTED
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int32)
    starts = np.zeros(B + 1, np.int32)
    if status:
        return dict(table=table, lengths=np.array(cached, np.int32), row_starts=starts,
                    slots=slots, positions=positions, num_free=num_free, status=status)
    t = k = 0
    for b in range(B):
        have = -(-cached[b] // page)
        for j in range(have, have + need[b]):
            p = int(free_list[num_free - 1 - k])
            k += 1
            if not 0 <= p < num_pages:
                status |= PAGE
                p = -1
            table[b, j] = p
        starts[b] = t
        for pos in range(cached[b], cached[b] + new[b]):
            p = int(table[b, pos // page])
            positions[t] = pos
            if 0 <= p < num_pages:
                slots[t] = p * page + pos % page
            else:
                status |= PAGE
            t += 1
    starts[B] = t
    return dict(table=table, lengths=np.array([c + n for c, n in zip(cached, new)], np.int32),
                row_starts=starts, slots=slots, positions=positions, num_free=num_free - k,
                status=status)


def release(finished, lengths, table, free_list, num_free, page, num_pages):
    """Finished requests' pages back on the free stack; copies are returned."""
    lengths, table, free_list = lengths.copy(), table.copy(), free_list.copy()
    bad = 0
    back = []
    for b in np.nonzero(finished)[0]:
        if not 0 <= lengths[b] <= table.shape[1] * page:
            bad |= LENGTH
            continue
        back += [(b, j) for j in range(-(-int(lengths[b]) // page))]
    if not 0 <= num_free <= num_pages or num_free + len(back) > num_pages:
        bad |= EXHAUSTED
    if not bad and any(not 0 <= table[e] < num_pages for e in back):
        bad |= PAGE
    if bad:
        return dict(lengths=lengths, table=table, free_list=free_list, num_free=num_free,
                    status=bad)
    for e in back:
        free_list[num_free] = table[e]
        table[e] = -1
        num_free += 1
    lengths[np.nonzero(finished)[0]] = 0
    return dict(lengths=lengths, table=table, free_list=free_list, num_free=num_free, status=0)


def latent_rows(rows, positions, d_c, base):
    """[c || RoPE(k, position)] in fp64 ("Multi-Head Latent Attention" 3.7)."""
    out = np.asarray(rows, np.float64).copy()
    out[:, d_c:] = O.apply_rope(out[:, d_c:], np.asarray(positions), base)
    return out


def sequence_rows(pool, table_row, n):
    """The first n rows of a sequence; pool [pages, page, width] in fp64."""
    page = pool.shape[1]
    if n == 0:
        return np.zeros((0, pool.shape[2]))
    return np.concatenate([pool[int(p)] for p in table_row[:-(-n // page)]])[:n]


def attend(q, rows, scale, d_c):
    """q [H, width], rows [n, width]: output [H, d_c], lse [H], and for error
    bounds the weights [H, n] and each head's sum of exp(s - max s)."""
    if len(rows) == 0:
        H = q.shape[0]
        return np.zeros((H, d_c)), np.full(H, -np.inf), np.zeros((H, 0)), np.zeros(H)
    s = (q @ rows.T) * scale
    m = s.max(1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(1, keepdims=True)
    p = e / z
    return p @ rows[:, :d_c], (m + np.log(z))[:, 0], p, z[:, 0]


def page_index(rows):
    """Index row of a page from its rows (fp32 values): int8 codes, fp32 scale."""
    x = np.asarray(rows, np.float32)
    zero = np.zeros(x.shape[1], np.int8), np.float32(0)
    top = np.float32(np.abs(x).max()) if len(x) else np.float32(0)
    if not TINY <= top < np.inf:
        return zero
    e = math.frexp(float(top))[1]
    fixed = np.rint(np.ldexp(x.astype(np.float64), 20 - e)).astype(np.int64).sum(0)
    peak = int(np.abs(fixed).max())
    if peak == 0:
        return zero
    inv = np.float32(1) / np.float32(peak)
    inv = inv * np.float32(127)
    codes = np.rint(fixed.astype(np.float32) * inv).astype(np.int8)
    scale = np.float32(peak) * (np.float32(1) / np.float32(127))
    scale = scale / np.float32(len(x))
    return codes, np.float32(np.ldexp(scale, e - 20))


def page_scores(q, codes, scales):
    """q [H, width] fp32 values, codes [P, width] int8, scales [P]: scores [P]."""
    q = np.asarray(q, np.float32)
    top = np.abs(q).max(1)
    live = top >= TINY
    safe = np.where(live, top, np.float32(1))
    inv = (np.float32(1) / safe) * np.float32(127)
    inv = np.where(live, inv, np.float32(0)).astype(np.float32)
    a = np.where(live, safe * (np.float32(1) / np.float32(127)), np.float32(0)).astype(np.float32)
    c = np.rint(q * inv[:, None]).astype(np.int64)
    dot = (c @ codes.astype(np.int64).T).astype(np.float32)
    v = (a[:, None] * dot).max(0)
    return v * scales.astype(np.float32)


def select(scores, P, top, keep_first, keep_last):
    """Positions of the pages kept, ascending."""
    if P <= top:
        return list(range(P))
    mid = list(range(keep_first, P - keep_last))
    best = sorted(mid, key=lambda j: (-scores[j], j))[:top - keep_first - keep_last]
    return list(range(keep_first)) + sorted(best) + list(range(P - keep_last, P))
