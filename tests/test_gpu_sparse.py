"""Sparse attention over chosen pages: the choice equals the oracle's exactly, the
attention over it is held to the paged call's bounds, and the paged operators run
together as a serving loop."""
import numpy as np
import pytest
import torch

from _paged import (D_C, DT, ROW, SCALE, check_attention, f64, make_pool, make_queries)
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Sparse:
    def __init__(self, mla, lengths, page, dtype, io, heads, top, q_len=1, kf=1, kl=1, seed=0,
                 s_max=None, index=True):
        rng = np.random.RandomState(seed)
        self.mla, self.lengths, self.q_len, self.top, self.kf, self.kl = mla, np.asarray(lengths), q_len, top, kf, kl
        self.page, self.dtype, self.io = page, dtype, io
        self.pool, self.table, self.pages = make_pool(rng, lengths, page, dtype)
        B, R = len(lengths), len(lengths) * q_len
        self.q_abs, self.q_pe = make_queries(rng, R, heads, io)
        self.d = mla.dims(B, heads, s_max or int(max(lengths)), mla.dtype_code(DT[dtype]))
        self.pg = mla.paging(page, self.pages, self.table.shape[1])
        self.codes = torch.zeros((self.pages, ROW), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros(self.pages, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dev = dict(q_abs=self.q_abs.cuda(), q_pe=self.q_pe.cuda(), pool=self.pool.cuda(),
                        table=self.table.cuda(), lengths=i32(lengths))
        if index:
            mla.page_index(self.d, self.pg, self.dev["pool"], self.dev["table"],
                           i32(np.zeros(B)), self.dev["lengths"], self.d.s_max, self.codes,
                           self.scales, dev_status=self.status)
        self.sel = torch.full((R, top), 77, dtype=torch.int32, device="cuda")
        self.sel_len = torch.full((R,), 77, dtype=torch.int32, device="cuda")
        n = mla.sparse_workspace_bytes(self.d, self.pg, io, top, q_len)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.o = torch.full((R, heads, D_C), 7.0, dtype=io, device="cuda")
        self.lse = torch.full((R, heads), 7.0, device="cuda")

    def run(self):
        x = self.dev
        self.mla.decode_attn_sparse(self.d, self.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"],
                                    x["lengths"], self.codes, self.scales, self.sel, self.sel_len,
                                    self.o, self.ws, SCALE, q_len=self.q_len, keep_first=self.kf,
                                    keep_last=self.kl, lse=self.lse, dev_status=self.status)
        return self

    def select(self):
        x = self.dev
        self.mla.select_pages(self.d, self.pg, x["q_abs"], x["q_pe"], x["table"], x["lengths"],
                              self.codes, self.scales, self.sel, self.sel_len, self.ws,
                              q_len=self.q_len, keep_first=self.kf, keep_last=self.kl,
                              dev_status=self.status)
        return self

    def choice(self):
        """The oracle's choice from the device's index and queries."""
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        q = np.concatenate([f64(self.q_abs), f64(self.q_pe)], 2).astype(np.float32)
        R, tab = len(q), self.table.numpy()
        sel, lens = np.full((R, self.top), -1), np.zeros(R, int)
        for r in range(R):
            b = r // self.q_len
            n = max(int(self.lengths[b]) - (self.q_len - 1 - r % self.q_len), 0)
            P = -(-n // self.page)
            ids = tab[b, :P]
            kept = PO.select(PO.page_scores(q[r], codes[ids], scales[ids]) if P else [], P,
                             self.top, self.kf, self.kl)
            sel[r, :len(kept)] = ids[kept]
            lens[r] = n - (P - len(kept)) * self.page
        return sel, lens

    def check_choice(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        sel, lens = self.choice()
        assert (self.sel.cpu().numpy() == sel).all()
        assert (self.sel_len.cpu().numpy() == lens).all()
        return sel, lens

    def check(self, status=0, tokens=None):
        sel, lens = self.check_choice(status)
        return check_attention(self.o, self.lse, self.q_abs, self.q_pe, self.pool,
                               torch.from_numpy(sel), lens, 1, self.dtype, self.io, tokens)


@pytest.mark.parametrize("dtype,io,heads", [("f32", F32, 1), ("f32", F32, 5), ("bf16", BF16, 16),
                                            ("bf16", F32, 32), ("bf16", BF16, 48), ("bf16", BF16, 64),
                                            ("fp8", BF16, 128), ("fp8", F32, 80), ("bf16", BF16, 128)])
@pytest.mark.parametrize("page,top,kf,kl", [(16, 4, 1, 1), (16, 9, 0, 2), (32, 2, 1, 1), (64, 3, 1, 1)])
def test_sparse_matches_the_oracle(cuda_lib, dtype, io, heads, page, top, kf, kl):
    lengths = [1, page, top * page, top * page + 1, 20 * page + 5, 33 * page]
    Sparse(cuda_lib, lengths, page, dtype, io, heads, top, kf=kf, kl=kl, seed=heads + page).run().check()


@pytest.mark.parametrize("q_len", [2, 4])
def test_sparse_several_tokens(cuda_lib, q_len):
    """Each token chooses for itself; tokens on both sides of a page border."""
    lengths = [16 * 20 + q_len - 1, 16 * 20 + 1, q_len, 16 * 11]
    Sparse(cuda_lib, lengths, 16, "bf16", BF16, 16, 5, q_len=q_len, kl=2, seed=q_len).run().check()


def test_select_many_pages(cuda_lib):
    """Pages by the thousand: several score tiles, a choice of many, and more scores
    than the selection keeps in shared memory."""
    Sparse(cuda_lib, [16 * 9001 + 3, 16 * 1025], 16, "bf16", BF16, 16, 700, seed=1).select().check_choice()
    Sparse(cuda_lib, [16 * 2500 + 3, 16 * 129, 5], 16, "bf16", F32, 16, 128, seed=2).select().check_choice()


def test_select_ties_go_to_the_lowest(cuda_lib):
    """Equal index rows, and queries of zeros: every score ties."""
    mla = cuda_lib
    s = Sparse(mla, [16 * 40 + 1, 16 * 30], 16, "bf16", BF16, 16, 7, seed=3)
    s.codes.copy_(s.codes[:1].expand_as(s.codes).clone())
    s.scales.fill_(0.25)
    s.select().check_choice()
    want = [0, 1, 2, 3, 4, 5, 40]
    assert s.sel[0].cpu().tolist() == s.table[0][want].tolist()
    s = Sparse(mla, [16 * 40 + 1, 16 * 30], 16, "bf16", BF16, 16, 7, seed=4)
    s.dev["q_abs"].zero_(), s.dev["q_pe"].zero_(), s.q_abs.zero_(), s.q_pe.zero_()
    s.select().check_choice()
    assert s.sel[0].cpu().tolist() == s.table[0][want].tolist()


def test_select_scores_of_both_signs(cuda_lib):
    """Scores below zero, zero scales among them (-0 and +0 tie)."""
    mla = cuda_lib
    s = Sparse(mla, [16 * 60], 16, "bf16", BF16, 16, 20, seed=5)
    s.codes.copy_(-s.codes.abs())
    s.q_abs.abs_(), s.q_pe.abs_()
    s.dev["q_abs"].abs_(), s.dev["q_pe"].abs_()
    s.scales[::3] = 0
    s.select().check_choice()


def test_select_is_the_same_in_any_batch(cuda_lib):
    """A sequence's choice does not depend on its neighbours."""
    mla = cuda_lib
    many = Sparse(mla, [16 * 300 + 7] * 9, 16, "bf16", BF16, 64, 16, seed=6).select()
    torch.cuda.synchronize()
    one = Sparse(mla, [16 * 300 + 7] * 9, 16, "bf16", BF16, 64, 16, seed=6)
    d1 = mla.dims(1, 64, one.d.s_max, mla.MLA_BF16)
    for b in (0, 4, 8):
        mla.select_pages(d1, one.pg, one.dev["q_abs"][b:b + 1].clone(),
                         one.dev["q_pe"][b:b + 1].clone(), one.dev["table"][b:b + 1].clone(),
                         one.dev["lengths"][b:b + 1].clone(), one.codes, one.scales,
                         one.sel[b:b + 1], one.sel_len[b:b + 1], one.ws)
        torch.cuda.synchronize()
        assert torch.equal(one.sel[b], many.sel[b])


def test_empty_long_and_bad(cuda_lib):
    mla = cuda_lib
    s = Sparse(mla, [0, 100], 16, "bf16", BF16, 16, 4, seed=7).run()
    s.check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    assert (s.sel[0] == -1).all() and int(s.sel_len[0]) == 0
    # a page outside the pool is never chosen while others are left
    s = Sparse(mla, [16 * 30, 100], 16, "bf16", BF16, 16, 4, seed=8)
    s.dev["table"][0, 5] = s.pages
    s.select()
    torch.cuda.synchronize()
    assert int(s.status.item()) == mla.MLA_DEV_PAGE_OUT_OF_RANGE
    assert s.pages not in s.sel[0].cpu().tolist()


def test_every_page_kept_is_the_paged_call(cuda_lib):
    """top_pages that cover the table: the bits of decode_attn_paged."""
    mla = cuda_lib
    s = Sparse(mla, [500, 129], 32, "bf16", BF16, 16, 16, seed=9, s_max=512).run()
    n = mla.paged_workspace_bytes(s.d, s.pg, BF16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(s.o), torch.empty_like(s.lse)
    mla.decode_attn_paged(s.d, s.pg, s.dev["q_abs"], s.dev["q_pe"], s.dev["pool"], s.dev["table"],
                          s.dev["lengths"], o, ws, SCALE, lse=lse)
    s.check()
    assert torch.equal(o, s.o) and torch.equal(lse, s.lse)


@pytest.mark.parametrize("io", [F32, BF16])
def test_same_bits_each_time_and_from_a_graph(cuda_lib, io):
    s = Sparse(cuda_lib, [16 * 200 + 1, 16 * 150, 40], 16, "bf16", io, 16, 20, seed=10).run()
    torch.cuda.synchronize()
    first = [t.clone() for t in (s.o, s.lse, s.sel, s.sel_len)]

    def same():
        torch.cuda.synchronize()
        for t, w in zip((s.o, s.lse, s.sel, s.sel_len), first):
            assert torch.equal(t, w)
            t.fill_(3)
        s.ws.fill_(0xFF)
        torch.cuda.synchronize()

    same()
    for _ in range(3):      # back to back: a call may not begin before the last one's readers end
        s.run()
    same()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
            s.run()
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
        same()


def test_serving_loop(cuda_lib):
    """Pages, rows, index, sparse and full attention and release together: three
    requests admitted with prompts, ten steps decoded, one request finished and its
    pages given to a new one.  Every step's outputs against the oracle on the rows
    that were appended."""
    mla = cuda_lib
    rng = np.random.RandomState(11)
    page, pages, width, B, H, top = 16, 60, 24, 4, 16, 6
    pg, d = mla.paging(page, pages, width), mla.dims(B, H, width * page, mla.MLA_BF16)
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    table, free, nf = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), i32(rng.permutation(pages)), i32([pages])
    cache = torch.full((pages, page, ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    codes, scales, status = z(pages, ROW, dt=torch.int8), z(pages, dt=torch.float32), z(1)
    lengths, old, starts = z(B), z(B), z(B + 1)
    o, lse, o_full = z(B, H, D_C, dt=F32), z(B, H, dt=F32), z(B, H, D_C, dt=F32)
    sel, sel_len = z(B, top), z(B)
    ws = z(max(mla.sparse_workspace_bytes(d, pg, F32, top), mla.paged_workspace_bytes(d, pg, F32)),
           dt=torch.uint8)
    history = [np.zeros((0, ROW)) for _ in range(B)]

    def step(new):
        T = max(sum(new), 1) + 2
        slots, pos = z(T, dt=torch.int64), z(T)
        old.copy_(lengths)
        mla.pages_extend(pg, lengths, i32(new), table, free, nf, lengths, starts, slots, pos,
                         dev_status=status)
        rows = torch.from_numpy(rng.randn(T, ROW).astype(np.float32)).bfloat16()
        mla.cache_append_paged(d, pg, rows.cuda(), pos, slots, cache, dev_status=status)
        mla.page_index(d, pg, cache, table, old, lengths, max(max(new), 1), codes, scales,
                       dev_status=status)
        exact = PO.latent_rows(f64(rows), pos.cpu().numpy(), D_C, 1e4)
        k = 0
        for b, n in enumerate(new):
            history[b] = np.concatenate([history[b], exact[k:k + n]])
            k += n
        live = [b for b in range(B) if len(history[b])]
        if len(live) < B:                       # empty rows of the batch set the length bit
            return
        qa, qp = make_queries(rng, B, H, F32)
        mla.decode_attn_paged(d, pg, qa.cuda(), qp.cuda(), cache, table, lengths, o_full, ws, SCALE,
                              dev_status=status)
        mla.decode_attn_sparse(d, pg, qa.cuda(), qp.cuda(), cache, table, lengths, codes, scales,
                               sel, sel_len, o, ws, SCALE, lse=lse, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert lengths.cpu().tolist() == [len(h) for h in history]
        q = np.concatenate([f64(qa), f64(qp)], 2)
        pool = f64(cache)
        for b in range(B):
            rows_b = PO.sequence_rows(pool, table[b].cpu().numpy(), len(history[b]))
            # the cached rows: the exact ones rounded to bf16
            assert (np.abs(rows_b - history[b]) <= 2.0 ** -8 * np.abs(history[b]) + 1e-5).all()
            want = PO.attend(q[b], rows_b, SCALE, D_C)[0]
            assert np.abs(f64(o_full[b]) - want).max() <= 1e-4 * np.abs(rows_b).max()
        check_attention(o, lse, qa, qp, cache, sel, sel_len.cpu().numpy(), 1, "bf16", F32)

    step([40, 100, 17, 5])
    for _ in range(10):
        step([1, 1, 1, 1])
    step([0, 1, 3, 1])
    mla.pages_release(pg, i32([0, 1, 0, 0]), lengths, table, free, nf, dev_status=status)
    history[1] = np.zeros((0, ROW))
    step([1, 200, 1, 1])
    step([1, 1, 1, 1])
    held = sum(-(-len(h) // page) for h in history)
    assert int(nf.item()) == pages - held
    mla.pages_release(pg, i32([1, 1, 1, 1]), lengths, table, free, nf, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert int(nf.item()) == pages and sorted(free.cpu().tolist()) == list(range(pages))


@pytest.mark.parametrize("pages,top", [(8, 7), (33, 3), (1025, 64), (9001, 700)])
def test_all_scores_equal_again_and_again(cuda_lib, pages, top):
    """Zero queries, as in a warm-up: every score ties in every token of many, and the
    lowest positions are kept each time, without a synchronisation in between."""
    mla, R = cuda_lib, 40
    s = Sparse(mla, [16 * pages], 16, "bf16", BF16, 16, top, seed=pages)
    s.d = mla.dims(R, 16, 16 * pages, mla.MLA_BF16)
    table = s.dev["table"].expand(R, -1).contiguous()
    q_abs = torch.zeros((R, 16, D_C), dtype=BF16, device="cuda")
    q_pe = torch.zeros((R, 16, 64), dtype=BF16, device="cuda")
    lengths = torch.full((R,), 16 * pages, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.select_workspace_bytes(s.d, s.pg), dtype=torch.uint8, device="cuda")
    want = table[0].cpu()[list(range(top - 1)) + [pages - 1]].tolist()
    sels = [torch.full((R, top), 77, dtype=torch.int32, device="cuda") for _ in range(25)]
    lens = torch.full((R,), 77, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for sel in sels:
        mla.select_pages(s.d, s.pg, q_abs, q_pe, table, lengths, s.codes, s.scales, sel, lens, ws,
                         dev_status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    for sel in sels:
        assert sel.cpu().tolist() == [want] * R
    assert lens.cpu().tolist() == [16 * top] * R


@pytest.mark.parametrize("s_max", [16 * 4, 16 * 40])
@pytest.mark.parametrize("bad", [-1, 60, 1 << 30, -(1 << 31)])
def test_select_reports_pages_it_keeps_unscored(cuda_lib, s_max, bad):
    """A token that keeps all its pages: a number that names no page is reported there too,
    whether other tokens are scored or none can be."""
    mla = cuda_lib
    s = Sparse(mla, [60, 40, 17], 16, "bf16", BF16, 16, 4, seed=12)
    assert s.pages <= 60
    table = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    table[:, :4] = s.dev["table"][:, :4]
    s.dev["table"], s.pg = table, mla.paging(16, s.pages, 40)
    s.d = mla.dims(3, 16, s_max, mla.MLA_BF16)
    s.ws = torch.empty(mla.select_workspace_bytes(s.d, s.pg), dtype=torch.uint8, device="cuda")
    s.select()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0        # entries past a token's pages may hold anything
    table[1, 2] = bad
    s.select()
    torch.cuda.synchronize()
    assert int(s.status.item()) == mla.MLA_DEV_PAGE_OUT_OF_RANGE
    assert s.sel[1].cpu().tolist() == [int(table[1, 0]), int(table[1, 1]), bad, -1]
    assert s.sel_len.cpu().tolist() == [60, 40, 17]
