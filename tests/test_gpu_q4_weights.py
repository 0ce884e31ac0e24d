"""Softmax weights far below the largest one, over 4-bit pools: many rows that together weigh as
much as the few that outweigh each of them.

A weight enters the output product as a few numbers of few bits.  What that takes from a weight w
may be a share of w, and what it takes from all weights beyond that a share of their sum, which
does not go by the largest weight and hardly grows with the rows:

    |error of w| <= r w + e,   sum of e <= f (sum of weights) + n 2^-40 (largest weight)
    f = d (16 / 2^b + 1/4 + ln(tiles / 16) / 4)

    16 heads a CTA, bf16 queries   two E4M3 parts, 1 and 1/16       r 2^-8,  d 2^-7,  b 5
                    fp32 queries   three, 1, 1/16 and 1/256         r 2^-12, d 2^-11, b 5
    SM pairs                       an E4M3 part, its E5M2 remainder r 2^-7,  d 2^-7,  b 4

Half a step of a part is 2^-4 of its value, or 2^-10 (E4M3) and 2^-17 (E5M2) where that is more; an
E5M2 value's 2^-3 of it.  So e, in units of the softmax's reference, is at most 2^-10 / 16 for two
E4M3 parts, 2^-10 / 256 for three, and for a part and its remainder, which is then at most 2^-10,
2^-14 (half of a step of 2^-13): a tile's 128 rows lose at most d.  How that adds up, L being the sum
of the weights of t tiles, in the same units (a move of the reference scales it and the loss):
  - up to 16 tiles go by after a tile to whose maximum the reference moved, or might have: it added
    2^b or more to L, so they lose at most 16 / 2^b of d times what was added to L;
  - otherwise a sum L bears tiles up to the (L/4)-th.  What was added to L since the last look pays
    for as many as a quarter of it: d / 4 of that.  A move that scales L by 2^c pays for those up to
    t' <= 2^c t, and loses d (t' - t) where L >= 4 t': d / 4 of (1 - 2^-c) <= c ln 2, and the c of
    all such moves, from t >= 16 on, sum to no more than log2(tiles / 16).
No reference lies more than 2^40 below an earlier one.
"""
import numpy as np
import pytest
import torch

import _q4
from _paged import D_C, D_R, SCALE, f64, half_step
from _q4_far import BF16, F32, TILE, Far, shifted
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


def weight_error(io, heads, q_len, n):
    """r and f above."""
    if io == F32:
        r, d, b = 2.0 ** -12, 2.0 ** -11, 5
    else:
        r, d, b = (2.0 ** -7, 2.0 ** -7, 4) if heads * q_len >= 48 else (2.0 ** -8, 2.0 ** -7, 5)
    return r, d * (16 / 2 ** b + 0.25 + max(np.log(n / TILE / 16), 0.0) / 4) + n * 2.0 ** -40


def check(c, tokens=None):
    """Outputs and lse within the bound: scores as tests/_paged.py has them (the query's
    rounding, fp32 sums, the softmax's own), weights as above."""
    q = np.concatenate([f64(c.q_abs), f64(c.q_pe)], 2)
    pool = _q4.values(c.pool.numpy(), c.page)
    o, lse = f64(c.o), f64(c.lse)
    H = q.shape[1]
    worst = [0.0, 0.0]
    for r in range(len(q)) if tokens is None else tokens:
        b = r // c.q_len
        n = int(c.lengths[b]) - (c.q_len - 1 - r % c.q_len)
        rows = pool[c.table[b, :-(-n // c.page)]].reshape(-1, D_C + D_R)[:n]
        want, want_lse, p, z = PO.attend(q[r], rows, SCALE, D_C)
        mag = np.abs(rows[:, :D_C])
        a = np.abs(q[r]) @ np.abs(rows).T * SCALE
        parts = 2.0 ** -17 if c.io == BF16 else 2.0 ** -16
        dq = parts * np.abs(q[r]).max(1, keepdims=True) * np.abs(rows).sum(1)[None] * SCALE
        ds = (dq + a * (600 * 2.0 ** -23 + 2.0 ** -21)).max(1)
        share, beyond = weight_error(c.io, H, c.q_len, n)
        dw = (share + 2 * ds + 2.0 ** -20 + (n + 200) * 2.0 ** -23)[:, None] * p
        lost = dw.sum(1) + beyond                    # of the sum of weights
        do = dw @ mag + beyond * mag.max(0) + np.abs(want) * lost[:, None]
        do = do + half_step(c.io) * (np.abs(want) + do) + 2.0 ** -22
        # (fp32 queries: the sum is that of the rounded weights)
        dl = ds + (lost if c.io == F32 else 0.0) + 2.0 ** -19 + (n + 200) * 2.0 ** -23
        assert np.isfinite(o[r]).all() and np.isfinite(lse[r]).all()
        worst[0] = max(worst[0], float((np.abs(o[r] - want) / do).max()))
        worst[1] = max(worst[1], float((np.abs(lse[r] - want_lse) / (dl + 2.0 ** -22 * np.abs(want_lse))).max()))
    assert max(worst) <= 1.0, f"{worst[0]:.3g} of the output's bound, {worst[1]:.3g} of the lse's"


def sequence(rng, n, at, spread=0.0, tail=None, noise=0.0):
    """Latents and keys of n rows, of which row `at` answers to a query's first key value.  The
    others' scores vary by `spread` nats; their latents have mean 1, that row's -1."""
    lat = (1.0 + noise * rng.randn(n, D_C)).astype(np.float32)
    key = np.zeros((n, D_R), np.float32)
    key[:, 1] = rng.randn(n) * spread / SCALE if tail is None else tail / SCALE
    lat[at], key[at, 0], key[at, 1] = -1.0, 1.0 / SCALE, 0.0
    return lat, key


def queries(tokens, heads, nats):
    """With which that row lies nats[0] .. nats[1] above the others, head by head."""
    q_abs, q_pe = torch.zeros((tokens, heads, D_C)), torch.zeros((tokens, heads, D_R))
    q_pe[:, :, 0] = torch.linspace(nats[0], nats[1], heads)
    q_pe[:, :, 1] = 1.0
    return q_abs, q_pe


def problem(mla, n, at, nats, spread, io, heads, q_len=1, splits=1, page=64, seed=0, tail=None,
            noise=0.0):
    """One such sequence."""
    lat, key = sequence(np.random.RandomState(seed), n, at, spread, tail, noise)
    return Far(mla, [lat], [key], *queries(q_len, heads, nats), page, io, q_len, splits)


FORMS = [(F32, 16), (BF16, 16), (BF16, 48), (BF16, 128)]


@pytest.mark.parametrize("io,heads", FORMS)
@pytest.mark.parametrize("spread", [0.0, 0.5, 1.0, 3.0])
@pytest.mark.parametrize("at", [0, 40001])
def test_one_row_outweighs_65536(cuda_lib, io, heads, spread, at):
    """One row 9 to 14 nats above 65536 others, at the start and far behind it, in one chunk."""
    check(problem(cuda_lib, 65536, at, (9.0, 14.0), spread, io, heads).run())


@pytest.mark.parametrize("io,heads", FORMS + [(F32, 64), (BF16, 32), (BF16, 64)])
@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("splits", [0, 3])
def test_cut_rows(cuda_lib, io, heads, q_len, splits):
    """The same with the rows cut, for one token and two."""
    check(problem(cuda_lib, 20000, 777, (9.0, 14.0), 0.5, io, heads, q_len, splits, page=32,
                  noise=0.3).run())


@pytest.mark.parametrize("io,heads", FORMS)
@pytest.mark.parametrize("nats", [(2.0, 8.0), (15.0, 27.0), (27.0, 40.0), (60.0, 200.0)])
def test_other_distances(cuda_lib, io, heads, nats):
    """From rows that weigh next to nothing at once to ones that weigh nothing."""
    check(problem(cuda_lib, 9000, 300, nats, 0.5, io, heads).run())


@pytest.mark.parametrize("io,heads", FORMS)
def test_tiles_that_climb_and_fall(cuda_lib, io, heads):
    """Every tile lies some nats above or below the one before, up to 30 from one to the next."""
    rng = np.random.RandomState(3)
    steps = np.concatenate([[3, -3, 2, -2, 5, -4, 30, -30], rng.uniform(-6, 6, 40),
                            np.cumsum(np.full(20, -1.5)), np.cumsum(np.full(20, 1.0))])
    tail = steps.repeat(TILE) + rng.randn(len(steps) * TILE) * 0.7
    check(problem(cuda_lib, len(tail), 5 * TILE + 3, (0.0, 10.0), 0.0, io, heads, tail=tail).run())
    check(problem(cuda_lib, len(tail) - 77, 60 * TILE, (0.0, 10.0), 0.0, io, heads, 2, 0,
                  tail=tail[77:]).run())


@pytest.mark.parametrize("io,heads", FORMS + [(F32, 32), (BF16, 32), (BF16, 64)])
@pytest.mark.parametrize("q_len", [1, 2])
def test_ordinary_rows(cuda_lib, io, heads, q_len):
    """Random rows, no row far from the others: each form within its own bound."""
    rng = np.random.RandomState(heads + q_len)
    check(shifted(rng, cuda_lib, [np.zeros(n) for n in (2, 129, 700, 5000)], heads, io, q_len).run())


@pytest.mark.parametrize("io,heads", [(F32, 256), (BF16, 1024)])
def test_long_pieces_of_many_sequences(cuda_lib, io, heads):
    """Equal shares of 43 tiles a CTA or pair: runs that end and begin inside a sequence and look
    at their sums in each of its pieces, with the heavy row in some of them."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1)
    try:
        rng = np.random.RandomState(4)
        lat, key = zip(*(sequence(rng, n, at, 0.5) for n, at in
                         [(4096, 0), (4000, 3999), (4096, 2000), (3900, 700), (130, 3), (4096, 4000),
                          (4096, 100), (4095, 1500), (3000, 2900), (4096, 50), (4096, 3333), (4096, 9)]))
        c = Far(mla, list(lat), list(key), *queries(len(lat), heads, (9.0, 14.0)), 64, io).run()
        check(c, tokens=[0, 1, 2, 3, 4, 8, 11])
        first = c.o.clone()
        assert torch.equal(first, c.run().o)
    finally:
        mla.load().mla_test_set_split_form(0)
