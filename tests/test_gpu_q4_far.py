"""Attention over 4-bit pools whose scores lie far below zero, or far from one another."""
import numpy as np
import pytest
import torch

import _q4
from _paged import D_C, ROW, SCALE, f64
from _q4_far import BF16, F32, i32, shifted
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu
KINDS = [(BF16, 16), (F32, 16), (BF16, 32), (BF16, 48), (BF16, 64), (BF16, 128), (F32, 128)]


def profiles(n):
    """Shifts of a sequence's rows: all alike, the first tile below the others, the others below
    the first, and steps that go down and up again."""
    t = np.arange(n)
    return {"-100": np.full(n, -100.0), "-1000": np.full(n, -1000.0), "+1000": np.full(n, 1000.0),
            "low first": np.where(t < 128, -100.0, 0.0), "very low first": np.where(t < 128, -1000.0, 0.0),
            "low later": np.where(t < 128, 0.0, -100.0), "low last": np.where(t < n - n % 128, -80.0, -180.0),
            "down and up": -100.0 * (t // 128 % 3), "all below": -100.0 - 30.0 * (t // 128 % 3)}


@pytest.mark.parametrize("form", [0, 1, "chunks"])
@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("io,heads", KINDS)
def test_scores_far_below_zero(cuda_lib, io, heads, q_len, form):
    """A softmax does not change with a shift of its scores, and rows far below others take no
    part: whole sequences, first tiles and later ones at -100 and -1000, in one chunk, in chunks
    of two tiles, and in equal shares."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1 if form == 1 else 0)
    try:
        rng = np.random.RandomState(heads + q_len)
        shifts = [p for n in (300, 700) for p in profiles(n).values()] + [np.full(5, -100.0)]
        shifted(rng, mla, shifts, heads, io, q_len, splits=3 if form == "chunks" else 0).run().check()
        shifted(rng, mla, shifts[:9], heads, io, q_len, page=16, splits=1).run().check()
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("q_len", [1, 2, 3])
@pytest.mark.parametrize("shift", [0.0, -100.0, -1000.0])
@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 48), (BF16, 64), (BF16, 128)])
def test_sparse_tokens_and_far_scores(cuda_lib, io, heads, q_len, shift):
    """Attention over chosen pages, one token a sequence and several, with rows far below zero:
    the choice is the definition's over the index that the library made, the rest the exact
    attention over it."""
    mla = cuda_lib
    rng = np.random.RandomState(heads + q_len)
    page, top, kf, kl = 16, 12, 1, 2
    lengths = [5, page * top, page * top + 1, 500, 40 * page + 7]
    c = shifted(rng, mla, [np.full(n, shift) for n in lengths], heads, io, q_len, page=page)
    B, R, x = len(lengths), len(lengths) * q_len, c.dev
    codes = torch.zeros((c.pg.num_pages, ROW), dtype=torch.int8, device="cuda")
    scales = torch.zeros(c.pg.num_pages, device="cuda")
    mla.page_index(c.d, c.pg, x["pool"], x["table"], i32(np.zeros(B)), x["lengths"], c.d.s_max, codes,
                   scales, dev_status=c.status)
    sel = torch.full((R, top), 77, dtype=torch.int32, device="cuda")
    sel_len = torch.full((R,), 77, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.sparse_workspace_bytes(c.d, c.pg, io, top, q_len=q_len), dtype=torch.uint8,
                     device="cuda")

    def run():
        mla.decode_attn_sparse(c.d, c.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"], x["lengths"],
                               codes, scales, sel, sel_len, c.o, ws, SCALE, q_len=q_len, keep_first=kf,
                               keep_last=kl, lse=c.lse, dev_status=c.status)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0

    run()
    q = np.concatenate([f64(c.q_abs), f64(c.q_pe)], 2).astype(np.float32)
    codes_h, scales_h = codes.cpu().numpy(), scales.cpu().numpy()
    want, want_len = np.full((R, top), -1), np.zeros(R, int)
    for r in range(R):
        b, n = r // q_len, lengths[r // q_len] - (q_len - 1 - r % q_len)
        P = -(-n // page)
        ids = c.table[b, :P]
        kept = PO.select(PO.page_scores(q[r], codes_h[ids], scales_h[ids]), P, top, kf, kl)
        want[r, :len(kept)] = ids[kept]
        want_len[r] = n - (P - len(kept)) * page
    assert (sel.cpu().numpy() == want).all() and (sel_len.cpu().numpy() == want_len).all()
    _q4.check_attention(c.o, c.lse, c.q_abs, c.q_pe, c.pool, page, torch.from_numpy(want), want_len, 1, io)
    first = c.o.clone()
    run()
    assert torch.equal(first, c.o)


@pytest.mark.parametrize("form", [0, 1, "one chunk"])
@pytest.mark.parametrize("heads", [16, 48, 128])
def test_infinite_keys(cuda_lib, heads, form):
    """Rows whose score is -infinity weigh nothing, a whole first tile of them and single ones."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1 if form == 1 else 0)
    try:
        rng = np.random.RandomState(heads)
        shifts = [np.zeros(400), np.full(300, -200.0), np.zeros(130)]
        shifts[0][:128] = shifts[0][200] = shifts[0][399] = -np.inf
        shifts[1][:256] = shifts[2][::2] = -np.inf
        c = shifted(rng, mla, shifts, heads, BF16, splits=1 if form == "one chunk" else 0).run()
        for b, s in enumerate(shifts):
            live = np.isfinite(s)
            pages = _q4.values(c.pool.numpy(), c.page)[c.table[b, :-(-len(s) // c.page)]]
            rows = pages.reshape(-1, ROW)[:len(s)][live]
            q = np.concatenate([f64(c.q_abs), f64(c.q_pe)], 2)[b]
            want, want_lse, p, z = PO.attend(q, rows, SCALE, D_C)
            do, dl = _q4.bounds(q, rows, p, z, BF16, heads, 1)
            do = do + 2.0 ** -8 * (np.abs(want) + do)
            assert (np.abs(f64(c.o)[b] - want) <= do).all()
            assert (np.abs(f64(c.lse)[b] - want_lse) <= dl + 2.0 ** -22 * np.abs(want_lse)).all()
    finally:
        mla.load().mla_test_set_split_form(0)
