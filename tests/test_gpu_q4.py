"""4-bit pools on the GPU: rows quantised into their slots and read back, the page index,
decode and sparse attention, each against the oracle, and a run of them together."""
import numpy as np
import pytest
import torch

import _q4
from _paged import D_C, DT, GARBAGE, ROW, SCALE, f64, half_step, make_queries
from _paged import make_pool as make_plain_pool
from oracle import fp4_oracle as F
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
PAGES = [16, 32, 64, 128, 256]


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rows in
def append(mla, rows, positions, slots, page, pages, pool=None, base=1e4):
    d, pg = mla.dims(1, 16, 1, mla.MLA_FP4_E2M1), mla.paging(page, pages, 1)
    if pool is None:
        pool = torch.full((mla.pool_bytes(d, pg),), 0xA5, dtype=torch.uint8, device="cuda")
    status = status_word()
    mla.cache_append_paged(d, pg, rows, i32(positions),
                           torch.as_tensor(np.asarray(slots), dtype=torch.int64).cuda(), pool,
                           rope_base=base, dev_status=status)
    torch.cuda.synchronize()
    return pool.cpu().numpy(), int(status.item())


def check_rows(before, after, rows, positions, slots, page, base=1e4):
    """Latents bit for bit, keys within half a step of the rotation in 64 bits (and the
    rotation's own error in fp32: 4 2^-24 of the pair's length), other rows untouched."""
    code0, e0, key0 = F.unpack(before, page)
    code, e, key = F.unpack(after, page)
    code, e, key = code.reshape(-1, D_C), e.reshape(-1, 32), key.reshape(-1, 64)
    x = f64(rows)
    live = [t for t, s in enumerate(slots) if s >= 0]
    at = np.asarray(slots)[live]
    want_e = F.exponents(x[live, :D_C])
    assert (e[at] == want_e).all()
    want = F.latents(F.codes(x[live, :D_C], want_e), want_e)
    assert (F.latents(code[at], e[at]) == want).all()
    turned = PO.latent_rows(x[live], np.asarray(positions)[live], D_C, base)[:, D_C:]
    size = np.hypot(x[live, D_C::2], x[live, D_C + 1::2]).repeat(2, 1)
    err = np.abs(_q4.from_bf16_bits(key[at]) - turned)
    assert (err <= half_step(BF16) * np.abs(turned) * 1.01 + 4 * 2.0 ** -24 * size + 2.0 ** -133).all()
    rest = np.ones(len(code), bool)
    rest[at] = False
    assert (code[rest] == code0.reshape(-1, D_C)[rest]).all()
    assert (e[rest] == e0.reshape(-1, 32)[rest]).all()
    assert (key[rest] == key0.reshape(-1, 64)[rest]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("n", [1, 3, 33, 200])
def test_append(cuda_lib, dtype, page, n):
    """Rows of every magnitude into scattered slots; a slot of -1 writes nothing."""
    rng = np.random.RandomState(n + page)
    pages = -(-n // page) + 3
    x = rng.randn(n, ROW) * np.exp2(rng.randint(-13, 10, (n, 36))).repeat(16, 1)
    rows = torch.from_numpy(x.astype(np.float32)).to(dtype)
    slots = rng.permutation(pages * page)[:n]
    slots[rng.rand(n) < 0.1] = -1
    pos = rng.randint(0, 100000, n)
    before = np.full(pages * page * 400, 0xA5, np.uint8)
    after, status = append(cuda_lib, rows.cuda(), pos, slots, page, pages)
    assert status == 0
    check_rows(before, after, rows, pos, slots, page)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_append_borders(cuda_lib, dtype):
    """Values on and next to the borders between codes and between exponents, zeros of both
    signs, numbers too small and too large, infinities and NaN."""
    top = [6.0, 7.0, 7.03125, 4.0, 3.5, 448.0, 1e30, np.inf, -np.inf, np.nan, 2.0 ** -9, 7 / 256, 0.0,
           -0.0, 1e-42]
    y = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, .2490234375, .2509765625, 4.96875, 5.03125, -.25,
                  -2.5, -5, 0.0])
    rows = np.zeros((len(top), ROW), np.float32)
    for r, t in enumerate(top):
        for b in range(32):
            unit = 2.0 ** (F.exponents(np.full((1, 512), t))[0, 0] if b % 2 else b // 2 - 8)
            rows[r, 16 * b:16 * b + 15] = np.roll(y, b) * unit
            rows[r, 16 * b + 15] = t
    rows[:, D_C:] = np.random.RandomState(0).randn(len(top), 64)
    t = torch.from_numpy(rows).to(dtype)
    slots, pos = np.arange(len(top))[::-1].copy(), np.arange(len(top)) * 7919
    before = np.full(16 * 400, 0xA5, np.uint8)
    after, status = append(cuda_lib, t.cuda(), pos, slots, 16, 1)
    assert status == 0
    check_rows(before, after, t, pos, slots, 16)


def test_append_reports_bad_slots_and_positions(cuda_lib):
    mla = cuda_lib
    rows = torch.randn(5, ROW)
    before = np.full(2 * 16 * 400, 0xA5, np.uint8)
    for slot, pos, bit in [(32, 0, mla.MLA_DEV_PAGE_OUT_OF_RANGE), (-2, 0, mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                           (1 << 40, 0, mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                           (3, -1, mla.MLA_DEV_LENGTH_OUT_OF_RANGE), (-1, -1, 0)]:
        slots, positions = np.array([5, slot, 31, -1, 0]), np.array([1, pos, 3, 4, 2 ** 31 - 1])
        after, status = append(mla, rows.cuda(), positions, slots, 16, 2)
        assert status == bit
        slots[1] = -1
        check_rows(before, after, rows, positions, slots, 16)


def test_append_past_2_to_32_bytes(cuda_lib):
    """Rows of pages that lie beyond 2^32 bytes of the pool's start, there and back."""
    mla = cuda_lib
    page, pages = 256, (1 << 32) // (256 * 400) + 9
    d, pg = mla.dims(1, 16, 300, mla.MLA_FP4_E2M1), mla.paging(page, pages, 2)
    pool = torch.empty(mla.pool_bytes(d, pg), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    pool[-4 * page * 400:] = 0xA5
    rows = torch.randn(300, ROW)
    table = np.array([[pages - 1, pages - 3]])
    pos = np.arange(300)
    slots = table[0, pos // page] * page + pos % page
    mla.cache_append_paged(d, pg, rows.cuda(), i32(pos), torch.from_numpy(slots).cuda(), pool)
    out = torch.empty((300, ROW), device="cuda")
    status = status_word()
    mla.cache_read_paged(d, pg, pool, i32(table), i32([300]), i32([0, 300]), out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    tail = pool[-4 * page * 400:].cpu().numpy()
    check_rows(np.full(4 * page * 400, 0xA5, np.uint8), tail, rows, pos, slots - (pages - 4) * page, page)
    assert (f64(out)[:, :D_C] == F.rounded(f64(rows)[:, :D_C])).all()


# ------------------------------------------------------------------ rows out
def pool_of(rng, lengths, page, dtype):
    if dtype == "fp4":
        pool, table, pages = _q4.make_pool(rng, lengths, page)
        return pool, table, pages, _q4.values(pool.numpy(), page)
    pool, table, pages = make_plain_pool(rng, lengths, page, dtype)
    return pool, table, pages, f64(pool)


@pytest.mark.parametrize("out", [F32, BF16])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", PAGES)
def test_read(cuda_lib, dtype, out, page):
    """Ragged sequences, empty ones among them, from the start and from a later row; rows
    behind the last one stay as they were."""
    mla = cuda_lib
    rng = np.random.RandomState(page)
    lengths = np.array([0, 1, 17, 0, 0, 300, page, page + 1, 5, 0])
    pool, table, pages, val = pool_of(rng, lengths, page, dtype)
    code = mla.MLA_FP4_E2M1 if dtype == "fp4" else mla.dtype_code(DT[dtype])
    d, pg = mla.dims(len(lengths), 16, 300, code), mla.paging(page, pages, table.shape[1])
    for first in (None, np.minimum([0, 0, 16, 0, 0, 129, page - 1, 2, 5, 0], lengths)):
        count = lengths - (0 if first is None else first)
        starts = np.concatenate([[0], np.cumsum(count)])
        rows = torch.full((starts[-1] + 5, ROW), 3.0, dtype=out, device="cuda")
        status = status_word()
        mla.cache_read_paged(d, pg, pool.cuda(), table.cuda(), i32(lengths), i32(starts), rows,
                             first_rows=None if first is None else i32(first), dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        want = np.concatenate([PO.sequence_rows(val, table[b].numpy(), int(n))[0 if first is None else first[b]:]
                               for b, n in enumerate(lengths)])
        want = torch.from_numpy(want).to(F32).to(out)     # fp32 holds every pool's values
        assert torch.equal(rows[:starts[-1]].cpu(), want)
        assert (rows[starts[-1]:] == 3).all()


def test_read_many_sequences(cuda_lib):
    """More sequences than one round of the search sees, most of them empty or of one row;
    a captured call follows new starts."""
    mla = cuda_lib
    rng = np.random.RandomState(1)
    B = 5000
    lengths = rng.randint(0, 2, B)
    lengths[[0, 1700, B - 1]] = [40, 100, 33]
    pool, table, pages, val = pool_of(rng, lengths, 16, "fp4")
    d, pg = mla.dims(B, 16, 112, mla.MLA_FP4_E2M1), mla.paging(16, pages, table.shape[1])
    starts = i32(np.concatenate([[0], np.cumsum(lengths)]))
    first = i32(np.zeros(B))
    n = int(lengths.sum())
    rows = torch.zeros((n, ROW), device="cuda")
    status = status_word()
    args = (d, pg, pool.cuda(), table.cuda(), i32(lengths), starts, rows, first, status)
    mla.cache_read_paged(*args)
    want = np.concatenate([PO.sequence_rows(val, table[b].numpy(), int(k)) for b, k in enumerate(lengths)])
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and (f64(rows) == want).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.cache_read_paged(*args)
    new = lengths.copy()
    new[1700], new[0] = 60, 0
    starts.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
    first.copy_(i32(lengths - new))
    rows.fill_(9)
    g.replay()
    torch.cuda.synchronize()
    want = np.concatenate([PO.sequence_rows(val, table[b].numpy(), int(k))[k - m:]
                           for b, (k, m) in enumerate(zip(lengths, new))])
    assert int(status.item()) == 0 and (f64(rows)[:len(want)] == want).all()
    assert (rows[len(want):] == 9).all()


def test_read_reports_rows_and_pages_that_are_not_there(cuda_lib):
    mla = cuda_lib
    rng = np.random.RandomState(2)
    pool, table, pages, val = pool_of(rng, [40, 20], 16, "fp4")
    d, pg = mla.dims(2, 16, 40, mla.MLA_FP4_E2M1), mla.paging(16, pages, table.shape[1])

    def read(lengths, starts, first, tab, n=70):
        rows = torch.full((n, ROW), 3.0, device="cuda")
        status = status_word()
        mla.cache_read_paged(d, pg, pool.cuda(), i32(tab), i32(lengths), i32(starts), rows,
                             first_rows=i32(first), dev_status=status)
        torch.cuda.synchronize()
        return f64(rows), int(status.item())

    seq = [PO.sequence_rows(val, table[b].numpy(), n) for b, n in enumerate([40, 20])]
    L, G = mla.MLA_DEV_LENGTH_OUT_OF_RANGE, mla.MLA_DEV_PAGE_OUT_OF_RANGE
    rows, status = read([40, 20], [0, 45, 65], [0, 0], table)        # five rows too many
    assert status == L and (rows[:40] == seq[0]).all() and (rows[40:45] == 0).all()
    assert (rows[45:65] == seq[1]).all() and (rows[65:] == 3).all()
    rows, status = read([40, 20], [0, 42, 62], [-2, 0], table)       # before the first row
    assert status == L and (rows[:2] == 0).all() and (rows[2:42] == seq[0]).all()
    rows, status = read([1 << 30, 20], [0, 1, 21], [1 << 29, 0], table)   # past the table's row
    assert status == L and (rows[0] == 0).all() and (rows[1:21] == seq[1]).all()
    for bad in GARBAGE:
        tab = table.numpy().copy()
        tab[0, 1] = bad
        rows, status = read([40, 20], [0, 40, 60], [0, 0], tab)
        assert status == G and (rows[:16] == seq[0][:16]).all() and (rows[16:32] == 0).all()
        assert (rows[32:40] == seq[0][32:]).all() and (rows[40:60] == seq[1]).all()
    rows, status = read([40, 20], [0, 40, 60], [0, 0], table, n=50)  # room for fewer rows
    assert status == 0 and (rows[40:] == seq[1][:10]).all()


def test_read_refuses_wrong_tensors(cuda_lib):
    mla = cuda_lib
    pool, table, pages, _ = pool_of(np.random.RandomState(2), [40, 20], 16, "fp4")
    d, pg = mla.dims(2, 16, 40, mla.MLA_FP4_E2M1), mla.paging(16, pages, table.shape[1])
    good = dict(cache=pool.cuda(), block_table=table.cuda(), lengths=i32([40, 20]),
                row_starts=i32([0, 40, 60]), rows=torch.empty((60, ROW), device="cuda"))
    for name, t in [("cache", good["cache"].cpu()), ("cache", good["cache"].view(torch.int8)),
                    ("cache", good["cache"].flatten()[400:]), ("block_table", table.cuda().long()),
                    ("lengths", i32([40])), ("row_starts", i32([0, 40])),
                    ("rows", good["rows"].half()), ("rows", good["rows"].cpu()),
                    ("rows", good["rows"][:, :575].contiguous()), ("rows", good["rows"][:, ::2]),
                    ("first_rows", i32([0]))]:
        with pytest.raises(ValueError):
            mla.cache_read_paged(d, pg, **{**good, name: t})


# ------------------------------------------------------------------ the page index
@pytest.mark.parametrize("page", PAGES)
def test_index(cuda_lib, page):
    mla = cuda_lib
    rng = np.random.RandomState(page)
    lengths = np.array([1, page, page + 1, 5 * page - 3, 700, 0])
    pool, table, pages = _q4.make_pool(rng, lengths, page)
    val = _q4.values(pool.numpy(), page)
    d, pg = mla.dims(6, 16, 5 * 256, mla.MLA_FP4_E2M1), mla.paging(page, pages, table.shape[1])
    first = np.array([0, page - 1, 0, page + 2, 690, 0])
    codes = torch.full((pages, ROW), 77, dtype=torch.int8, device="cuda")
    scales = torch.full((pages,), 7.0, device="cuda")
    status = status_word()
    mla.page_index(d, pg, pool.cuda(), table.cuda(), i32(first), i32(lengths), 5 * 256, codes, scales,
                   dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_c, want_s = np.full((pages, ROW), 77, np.int8), np.full(pages, 7.0, np.float32)
    for b, n in enumerate(lengths):
        for j in range(first[b] // page, -(-int(n) // page)):
            i = int(table[b, j])
            want_c[i], want_s[i] = PO.page_index(val[i][:min(page, n - j * page)])
    assert (codes.cpu().numpy() == want_c).all() and (scales.cpu().numpy() == want_s).all()


def test_index_of_every_value(cuda_lib):
    """A page's unit comes from its largest value: each that a pool can hold, alone and beside
    smaller ones, under smaller and larger keys, and a page with an infinite key (zeros)."""
    mla = cuda_lib
    rng = np.random.RandomState(3)
    page, each = 16, [(c, e) for c in [*range(1, 8), *range(9, 16)] for e in range(-8, 7)]
    pages = 4 * len(each) + 2
    code = np.zeros((pages, page, D_C), np.int64)
    exp = rng.randint(-8, 7, (pages, page, 32))
    key = np.zeros((pages, page, 64), np.float32)
    for i, (c, e) in enumerate(each):
        for k in range(4):
            p, r, col = 4 * i + k, rng.randint(page), rng.randint(D_C)
            if k == 1:                           # smaller ones beside it
                code[p], exp[p] = rng.randint(0, 2, (page, D_C)), -8
            code[p, r, col], exp[p, r, col // 16] = c, e
            if k >= 2:
                key[p, rng.randint(page), rng.randint(64)] = 2.0 ** (-20 if k == 2 else 12) * 1.5
    key[-1, 3, 5] = np.inf
    code[-1] = rng.randint(0, 16, (page, D_C))
    pool = F.pack(code, exp, _q4.bf16_bits(key))
    val = _q4.values(pool, page)
    d, pg = mla.dims(1, 16, pages * page, mla.MLA_FP4_E2M1), mla.paging(page, pages, pages)
    codes = torch.full((pages, ROW), 77, dtype=torch.int8, device="cuda")
    scales, status = torch.full((pages,), 7.0, device="cuda"), status_word()
    mla.page_index(d, pg, torch.from_numpy(pool).cuda(), i32([np.arange(pages)]), i32([0]),
                   i32([pages * page]), pages * page, codes, scales, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    for p in range(pages - 1):
        want_c, want_s = PO.page_index(val[p])
        assert got_s[p] == want_s and (got_c[p] == want_c).all(), p
    assert got_s[-1] == 0 and (got_c[-1] == 0).all()


def test_index_of_many_requests(cuda_lib):
    """More pages that could be touched than the kernel looks up at once, few that are."""
    mla = cuda_lib
    rng = np.random.RandomState(5)
    B, page, width = 700, 16, 34
    lengths = rng.randint(0, 60, B)
    pool, table, pages = _q4.make_pool(rng, lengths, page, width=width)
    val = _q4.values(pool.numpy(), page)
    first = np.maximum(lengths - rng.randint(0, 3, B), 0)
    d, pg = mla.dims(B, 16, width * page, mla.MLA_FP4_E2M1), mla.paging(page, pages, width)
    codes = torch.full((pages, ROW), 77, dtype=torch.int8, device="cuda")
    scales, status = torch.full((pages,), 7.0, device="cuda"), status_word()
    mla.page_index(d, pg, pool.cuda(), table.cuda(), i32(first), i32(lengths), width * page, codes, scales,
                   dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_c, want_s = np.full((pages, ROW), 77, np.int8), np.full(pages, 7.0, np.float32)
    for b, n in enumerate(lengths):
        for j in range(first[b] // page, -(-int(n) // page)) if first[b] < n else ():
            i = int(table[b, j])
            want_c[i], want_s[i] = PO.page_index(val[i][:min(page, n - j * page)])
    assert (codes.cpu().numpy() == want_c).all() and (scales.cpu().numpy() == want_s).all()


def test_index_reports(cuda_lib):
    mla = cuda_lib
    pool, table, pages = _q4.make_pool(np.random.RandomState(0), [40, 20], 16)
    d, pg = mla.dims(2, 16, 64, mla.MLA_FP4_E2M1), mla.paging(16, pages, table.shape[1])
    for lengths, first, tab, bit in [([40, 20], [0, 0], -1, mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                                     ([40, -1], [39, 0], None, mla.MLA_DEV_LENGTH_OUT_OF_RANGE),
                                     ([1 << 20, 20], [39, 19], None, mla.MLA_DEV_LENGTH_OUT_OF_RANGE),
                                     ([40, 20], [0, 19], None, mla.MLA_DEV_LENGTH_OUT_OF_RANGE)]:
        t = table.clone()
        if tab is not None:
            t[0, 1] = tab
        codes = torch.zeros((pages, ROW), dtype=torch.int8, device="cuda")
        scales, status = torch.zeros(pages, device="cuda"), status_word()
        mla.page_index(d, pg, pool.cuda(), t.cuda(), i32(first), i32(lengths),
                       40 if tab is not None else 5, codes, scales, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == bit


# ------------------------------------------------------------------ attention
class Call:
    """One decode_attn_paged problem over a 4-bit pool."""

    def __init__(self, mla, lengths, page, io, heads, q_len=1, splits=0, seed=0, s_max=None, **kw):
        rng = np.random.RandomState(seed)
        self.mla, self.q_len, self.io, self.splits, self.page = mla, q_len, io, splits, page
        self.lengths = np.asarray(lengths)
        self.pool, self.table, self.pages = _q4.make_pool(rng, self.lengths, page, **kw)
        B = len(lengths)
        self.q_abs, self.q_pe = make_queries(rng, B * q_len, heads, io)
        s_max = s_max or max(int(self.lengths.max()), 1)
        self.d = mla.dims(B, heads, s_max, mla.MLA_FP4_E2M1)
        self.pg = mla.paging(page, self.pages, self.table.shape[1])
        n = mla.paged_workspace_bytes(self.d, self.pg, io, q_len, splits)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.o = torch.full((B * q_len, heads, D_C), 7.0, dtype=io, device="cuda")
        self.lse = torch.full((B * q_len, heads), 7.0, device="cuda")
        self.status = status_word()
        self.dev = dict(q_abs=self.q_abs.cuda(), q_pe=self.q_pe.cuda(), pool=self.pool.cuda(),
                        table=self.table.cuda(), lengths=i32(self.lengths))

    def run(self):
        x = self.dev
        self.mla.decode_attn_paged(self.d, self.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"],
                                   x["lengths"], self.o, self.ws, SCALE, q_len=self.q_len,
                                   num_splits_requested=self.splits, lse=self.lse,
                                   dev_status=self.status)
        return self

    def check(self, status=0, tokens=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        return _q4.check_attention(self.o, self.lse, self.q_abs, self.q_pe, self.pool, self.page,
                                   self.table, self.lengths, self.q_len, self.io, tokens)


EDGES = [1, 15, 16, 17, 127, 128, 129, 300]
KINDS = [(F32, 16), (BF16, 16), (F32, 32), (BF16, 32), (BF16, 48), (BF16, 64), (F32, 64), (BF16, 128),
         (F32, 128), (BF16, 256)]


@pytest.mark.parametrize("io,heads", KINDS)
@pytest.mark.parametrize("page", PAGES)
def test_lengths_and_pages(cuda_lib, io, heads, page):
    """Ragged lengths around every tile and page edge, garbage past each end, table entries
    past a sequence's pages that name nothing."""
    Call(cuda_lib, EDGES, page, io, heads, seed=page + heads).run().check()


@pytest.mark.parametrize("io,heads", KINDS)
@pytest.mark.parametrize("splits", [1, 2, 3])
def test_chunks(cuda_lib, io, heads, splits):
    """The rows cut into one, two and three chunks, the last ones of short sequences empty."""
    Call(cuda_lib, [700, 129, 1, 513], 64, io, heads, splits=splits, seed=splits, gain=4.0).run().check()


@pytest.mark.parametrize("io,heads", KINDS)
@pytest.mark.parametrize("q_len", [2, 3, 4])
def test_several_tokens(cuda_lib, io, heads, q_len):
    """q_len tokens per sequence, causal among themselves; lengths q_len and up."""
    Call(cuda_lib, [q_len, 128 + q_len, 131, 400], 32, io, heads, q_len=q_len, seed=q_len).run().check()


@pytest.mark.parametrize("io,heads", KINDS)
def test_long_and_ragged(cuda_lib, io, heads):
    """Enough rows for every plan: one sequence over all CTAs, and many of different lengths."""
    Call(cuda_lib, [20001, 3], 64, io, heads, seed=6).run().check()
    n = np.random.RandomState(heads).randint(1, 4000, 60)
    n[:4] = [1, 128, 129, 3999]
    Call(cuda_lib, n, 64, io, heads, seed=7).run().check(tokens=[0, 1, 2, 3, 17, 59])


def share_lengths(kind, B):
    rng = np.random.RandomState(B)
    if kind == "ragged":
        n = rng.randint(0, 900, B)
        n[:5] = [0, 1, 128, 129, 899]
    elif kind == "one long":              # all but one sequence short or empty
        n = rng.randint(0, 3, B)
        n[B // 2] = 6000
    else:                                 # "edges": multiples of a tile, and one more row
        n = 128 * rng.randint(0, 6, B) + rng.randint(0, 2, B)
    return n


@pytest.mark.parametrize("kind", ["ragged", "one long", "edges"])
@pytest.mark.parametrize("io,heads,q_len,page", [(F32, 16, 1, 16), (BF16, 16, 1, 64), (BF16, 32, 1, 256),
                                                 (F32, 128, 1, 64), (F32, 16, 3, 32), (BF16, 16, 2, 128),
                                                 (BF16, 48, 1, 16), (BF16, 128, 1, 64),
                                                 (BF16, 256, 1, 128), (BF16, 64, 2, 32)])
@pytest.mark.parametrize("B", [7, 70])
def test_equal_shares(cuda_lib, kind, io, heads, q_len, page, B):
    """Tiles cut into equal runs: runs that start and end inside a sequence, hold several,
    one tile each, and fewer tiles than CTAs; a call repeated gives the same bits."""
    mla = cuda_lib
    lengths = share_lengths(kind, B)
    if q_len > 1:
        lengths = np.maximum(lengths, q_len)
    mla.load().mla_test_set_split_form(1)
    try:
        c = Call(mla, lengths, page, io, heads, q_len=q_len, seed=B + heads)
        c.ws = torch.empty(c.ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]
        c.run()
        first = c.o.clone()
        c.check(tokens=range(0, B * q_len, max(1, B * q_len // 12)),
                status=0 if lengths.min() else mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
        c.o.fill_(7)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(first, c.o)
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 64), (BF16, 128)])
def test_back_to_back_captured_and_on_a_stream(cuda_lib, io, heads, form):
    """Calls that follow one another on one workspace, unsynchronised, with lengths that
    change between them, from a side stream and from two graphs: each gives what it gives
    alone."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(form)
    try:
        calls = [Call(mla, lengths, 64, io, heads, seed=seed, s_max=7000, width=110)
                 for seed, lengths in enumerate((share_lengths("ragged", 24) + 1,
                                                 share_lengths("one long", 24) + 1, np.full(24, 640)))]
        alone = []
        for c in calls:
            c.ws = calls[0].ws
            c.run()
            torch.cuda.synchronize()
            alone.append((c.o.clone(), c.lse.clone()))
            c.check(tokens=[0, 11, 12, 23])

        def same():
            torch.cuda.synchronize()
            for (o, lse), c in zip(alone, calls):
                assert torch.equal(o, c.o) and torch.equal(lse, c.lse)
                c.o.fill_(3)
                c.lse.fill_(3)
            calls[0].ws.fill_(0xFF)
            torch.cuda.synchronize()

        same()
        for _ in range(10):
            for c in calls:
                c.run()
        same()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for c in calls:
                c.run()
        same()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for c in calls:
                    c.run()
            graphs.append(g)
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
            same()
        c = calls[0]
        c.lengths = np.asarray(share_lengths("edges", 24)) % np.maximum(c.lengths, 1) + 1
        c.lengths = np.minimum(c.lengths, calls[0].dev["lengths"].cpu().numpy())
        c.dev["lengths"].copy_(i32(c.lengths))
        graphs[0].replay()
        c.check(tokens=[0, 1, 11, 12, 23])
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("io,heads", KINDS)
def test_empty_and_bad_lengths(cuda_lib, io, heads):
    """No rows: zeros and -inf, with the status bit; a length above s_max is cut there."""
    mla = cuda_lib
    bit = mla.MLA_DEV_LENGTH_OUT_OF_RANGE
    Call(mla, [0, 5, 0, 140], 16, io, heads, seed=1).run().check(status=bit)
    Call(mla, [0, 5, 0, 140], 16, io, heads, seed=1, splits=1).run().check(status=bit)
    c = Call(mla, [200, 130], 16, io, heads, seed=2, s_max=150).run()
    c.lengths = np.array([150, 130])
    c.check(status=bit)
    c = Call(mla, [-3, 130], 16, io, heads, seed=2).run()
    c.lengths = np.array([0, 130])
    c.check(status=bit)


@pytest.mark.parametrize("io,heads", KINDS)
@pytest.mark.parametrize("bad", [-1, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("page,form", [(32, 0), (256, 0), (64, 1)])
def test_pages_outside_the_pool_read_as_zeros(cuda_lib, io, heads, bad, page, form):
    mla = cuda_lib
    mla.load().mla_test_set_split_form(form)
    try:
        c = Call(mla, [600, 430, 90], page, io, heads, seed=3)
        c.table[0, 1] = bad
        c.table[2, 0] = bad
        c.dev["table"].copy_(c.table)
        c.run().check(status=mla.MLA_DEV_PAGE_OUT_OF_RANGE)
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("io,heads", KINDS)
@pytest.mark.parametrize("size", [0.0, 1e-42, 1e-37, 1e-30])
def test_tiny_queries(cuda_lib, io, heads, size):
    """Queries of zeros, and of hardly anything with zeros among it: every row weighs the same."""
    c = Call(cuda_lib, [300, 17], 32, io, heads, seed=11)
    c.q_abs, c.q_pe = (c.q_abs.float() * size).to(io), (c.q_pe.float() * size).to(io)
    c.q_abs[:, :, ::3] = 0
    c.dev["q_abs"], c.dev["q_pe"] = c.q_abs.cuda(), c.q_pe.cuda()
    c.run().check()


@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 64), (BF16, 128)])
def test_one_row_outweighs_many(cuda_lib, io, heads):
    """A row whose weight is 2^10 to 2^16 times that of each of the others, which together
    weigh as much: nothing of the small weights may be lost, nor of a maximum that comes late."""
    for at in (0, 130, 2999):
        c = Call(cuda_lib, [3000], 64, io, heads, seed=12)
        code, e, key = F.unpack(c.pool.numpy(), 64)
        for t in range(3000):
            i, r = int(c.table[0, t // 64]), t % 64
            key[i, r] = _q4.bf16_bits(np.full(64, 1.0 if t == at else 0.0))
            e[i, r] = -8
        c.pool = torch.from_numpy(F.pack(code, e, key))
        c.dev["pool"] = c.pool.cuda()
        c.q_pe = torch.zeros_like(c.q_pe)
        c.q_pe[:, :, 0] = torch.linspace(96, 154, heads).to(io)      # scores of 6.9 to 11.1
        c.dev["q_pe"] = c.q_pe.cuda()
        c.run().check()


def test_rows_of_other_sequences_are_left_alone(cuda_lib):
    """Outputs behind the last token keep what they held."""
    c = Call(cuda_lib, [100, 30], 16, BF16, 16, seed=6)
    o = torch.full((5, 16, D_C), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((5, 16), 3.0, device="cuda")
    c.o, c.lse = o[:2], lse[:2]
    c.run().check()
    assert (o[2:] == 3).all() and (lse[2:] == 3).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_shared_pages_and_no_lse(cuda_lib, heads):
    """Two sequences with a common prefix in the same pages; lse not asked for."""
    c = Call(cuda_lib, [100, 100], 16, BF16, heads, seed=7)
    c.table[1, :4] = c.table[0, :4]
    c.dev["table"].copy_(c.table)
    c.run().check()
    o, c.lse = c.o.clone(), None
    c.o.fill_(7)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.o, o)


@pytest.mark.parametrize("heads", [16, 128])
def test_pool_past_2_to_32_bytes(cuda_lib, heads):
    mla = cuda_lib
    page, pages = 256, (1 << 32) // (256 * 400) + 40
    c = Call(mla, [300, 129], page, BF16, heads, seed=8)
    big = torch.zeros((pages, page * 400), dtype=torch.uint8, device="cuda")
    top = pages - c.pages
    big[top:].copy_(c.dev["pool"])
    live = (c.table >= 0) & (c.table < c.pages)
    c.dev["table"] = torch.where(live, c.table + top, c.table).cuda()
    c.dev["pool"], c.pg = big, mla.paging(page, pages, c.table.shape[1])
    c.run().check()


def test_refuses_wrong_tensors(cuda_lib):
    mla = cuda_lib
    c = Call(mla, [100, 30], 16, BF16, 16, seed=6)

    def with_(**kw):
        saved = dict(c.dev)
        c.dev.update(kw)
        try:
            with pytest.raises(ValueError):
                c.run()
        finally:
            c.dev = saved

    with_(pool=c.dev["pool"].cpu())
    with_(pool=c.dev["pool"].view(torch.float8_e4m3fn))
    with_(pool=c.dev["pool"].flatten()[400:])
    with_(q_abs=c.dev["q_abs"].float())
    with_(q_abs=c.dev["q_abs"].half())
    c.ws = c.ws[:100]
    with pytest.raises(mla.MlaError):
        c.run()


# ------------------------------------------------------------------ sparse attention, and all together
@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 32), (BF16, 48), (BF16, 64), (BF16, 128), (F32, 80)])
@pytest.mark.parametrize("page,top,kf,kl", [(16, 4, 1, 1), (16, 9, 0, 2), (64, 3, 1, 1), (256, 2, 1, 1)])
def test_sparse(cuda_lib, io, heads, page, top, kf, kl, q_len=1):
    mla = cuda_lib
    lengths = np.array([1, page, top * page, top * page + 1, 7 * page + 5, 15 * page])
    c = Call(mla, lengths, page, io, heads, seed=heads + page, q_len=q_len)
    B = len(lengths)
    codes = torch.zeros((c.pages, ROW), dtype=torch.int8, device="cuda")
    scales = torch.zeros(c.pages, device="cuda")
    x = c.dev
    mla.page_index(c.d, c.pg, x["pool"], x["table"], i32(np.zeros(B)), x["lengths"], c.d.s_max, codes,
                   scales, dev_status=c.status)
    sel = torch.full((B, top), 77, dtype=torch.int32, device="cuda")
    sel_len = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    ws = torch.empty(mla.sparse_workspace_bytes(c.d, c.pg, io, top), dtype=torch.uint8, device="cuda")

    def run():
        mla.decode_attn_sparse(c.d, c.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"], x["lengths"],
                               codes, scales, sel, sel_len, c.o, ws, SCALE, keep_first=kf, keep_last=kl,
                               lse=c.lse, dev_status=c.status)

    run()
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    q = np.concatenate([f64(c.q_abs), f64(c.q_pe)], 2).astype(np.float32)
    codes_h, scales_h = codes.cpu().numpy(), scales.cpu().numpy()
    want, want_len = np.full((B, top), -1), np.zeros(B, int)
    for b, n in enumerate(lengths):
        P = -(-int(n) // page)
        ids = c.table[b].numpy()[:P]
        kept = PO.select(PO.page_scores(q[b], codes_h[ids], scales_h[ids]), P, top, kf, kl)
        want[b, :len(kept)] = ids[kept]
        want_len[b] = n - (P - len(kept)) * page
    assert (sel.cpu().numpy() == want).all() and (sel_len.cpu().numpy() == want_len).all()
    _q4.check_attention(c.o, c.lse, c.q_abs, c.q_pe, c.pool, page, torch.from_numpy(want), want_len, 1, io)
    first = c.o.clone()
    for _ in range(5):
        run()
    torch.cuda.synchronize()
    assert torch.equal(first, c.o)


def test_serving_loop(cuda_lib):
    """Requests admitted, decoded for some steps and released, over a 4-bit pool: tables, rows,
    index, attention over all pages and over chosen ones, and the prefix read back, step for
    step against the oracle's copy of the cache."""
    mla = cuda_lib
    rng = np.random.RandomState(9)
    B, page, pages, width, heads, top = 5, 16, 90, 20, 16, 4
    pg = mla.paging(page, pages, width)
    d = mla.dims(B, heads, width * page, mla.MLA_FP4_E2M1)
    pool = torch.full((mla.pool_bytes(d, pg),), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, num_free = i32(rng.permutation(pages)), i32([pages])
    lengths, starts = i32(np.zeros(B)), i32(np.zeros(B + 1))
    slots = torch.zeros(400, dtype=torch.int64, device="cuda")
    positions, status = i32(np.zeros(400)), status_word()
    codes = torch.zeros((pages, ROW), dtype=torch.int8, device="cuda")
    scales = torch.zeros(pages, device="cuda")
    ws = torch.empty(max(mla.paged_workspace_bytes(d, pg, BF16), mla.sparse_workspace_bytes(d, pg, BF16, top)),
                     dtype=torch.uint8, device="cuda")
    o, lse = torch.empty((B, heads, D_C), dtype=BF16, device="cuda"), torch.empty((B, heads), device="cuda")
    sel, sel_len = torch.empty((B, top), dtype=torch.int32, device="cuda"), i32(np.zeros(B))
    cached = [np.zeros((0, ROW)) for _ in range(B)]
    for step in range(6):
        new = rng.randint(30, 80, B) if step == 0 else np.ones(B, int)
        if step == 3:                               # one request ends and another takes its place
            done = i32(np.arange(B) == 2)
            mla.pages_release(pg, done, lengths, table, free, num_free, dev_status=status)
            cached[2] = np.zeros((0, ROW))
            new[2] = 70
        first = lengths.clone()
        mla.pages_extend(pg, lengths, i32(new), table, free, num_free, lengths, starts, slots, positions,
                         dev_status=status)
        T = int(new.sum())
        rows = torch.from_numpy(rng.randn(T, ROW).astype(np.float32)).to(BF16)
        mla.cache_append_paged(d, pg, rows.cuda(), positions[:T], slots[:T], pool, dev_status=status)
        mla.page_index(d, pg, pool, table, first, lengths, int(new.max()), codes, scales, dev_status=status)
        q_abs, q_pe = make_queries(rng, B, heads, BF16)
        mla.decode_attn_paged(d, pg, q_abs.cuda(), q_pe.cuda(), pool, table, lengths, o, ws, SCALE, lse=lse,
                              dev_status=status)
        back = torch.empty((T, ROW), dtype=BF16, device="cuda")
        mla.cache_read_paged(d, pg, pool, table, lengths, starts, back, first_rows=first, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        x, pos, at = f64(rows), positions.cpu().numpy(), starts.cpu().numpy()
        turned = PO.latent_rows(x, pos[:T], D_C, 1e4)
        got = f64(back)
        assert (got[:, :D_C] == F.rounded(x[:, :D_C])).all()
        # half a step of the value, and the rotation's own error in fp32
        assert (np.abs(got - turned)[:, D_C:] <= 2.0 ** -8 * 1.01 * np.abs(turned[:, D_C:]) + 2.0 ** -20).all()
        for b in range(B):
            cached[b] = np.concatenate([cached[b], got[at[b]:at[b + 1]]])
        n = lengths.cpu().numpy()
        assert [len(c) for c in cached] == n.tolist()
        host = pool.cpu()
        val, tab = _q4.values(host.numpy(), page), table.cpu()
        for b in range(B):
            assert (PO.sequence_rows(val, tab[b].numpy(), int(n[b])) == cached[b]).all()
        _q4.check_attention(o, lse, q_abs, q_pe, host, page, tab, n, 1, BF16)
        mla.decode_attn_sparse(d, pg, q_abs.cuda(), q_pe.cuda(), pool, table, lengths, codes, scales, sel,
                               sel_len, o, ws, SCALE, lse=lse, dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        _q4.check_attention(o, lse, q_abs, q_pe, host, page, sel.cpu(), sel_len.cpu().numpy(), 1, BF16)


@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 32), (BF16, 128)])
def test_calls_at_once(cuda_lib, io, heads, form):
    """Two calls on two streams, of one pool and each its own workspace, while a third stream
    writes and reads other pages of the pool: each gives what it gives alone."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(form)
    try:
        calls = [Call(mla, np.minimum(share_lengths("ragged", 20), 900) + 1, 64, io, heads, seed=9,
                      s_max=7000, extra_pages=40, width=110) for _ in range(2)]
        calls[1].q_abs = calls[1].q_abs.flip(0).contiguous()
        calls[1].dev.update(pool=calls[0].dev["pool"], q_abs=calls[1].q_abs.cuda())
        alone = []
        for c in calls:
            c.run().check(tokens=[0, 7, 19])
            alone.append((c.o.clone(), c.lse.clone()))
        free = sorted(set(range(calls[0].pages)) - set(calls[0].table[calls[0].table >= 0].tolist()))[:40]
        rng = np.random.RandomState(10)
        rows = torch.from_numpy(rng.randn(64 * len(free), ROW).astype(np.float32)).cuda()
        slots = (torch.tensor(free).repeat_interleave(64) * 64 + torch.arange(64).repeat(len(free))).cuda()
        table, zero = i32([free]), torch.zeros(len(slots), dtype=torch.int32, device="cuda")
        d = mla.dims(1, 16, len(slots), mla.MLA_FP4_E2M1)
        pg = mla.paging(64, calls[0].pages, len(free))
        out = torch.empty_like(rows)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        for _ in range(20):
            for c, s in zip(calls, streams):
                with torch.cuda.stream(s):
                    c.run()
            with torch.cuda.stream(streams[2]):
                mla.cache_append_paged(d, pg, rows, zero, slots, calls[0].dev["pool"])
                mla.cache_read_paged(d, pg, calls[0].dev["pool"], table, i32_at(len(slots)),
                                     i32_at(0, len(slots)), out)
        torch.cuda.synchronize()
        for c, (o, lse) in zip(calls, alone):
            assert int(c.status.item()) == 0
            assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
        x = f64(rows)
        e = F.exponents(x[:, :D_C])
        assert (f64(out)[:, :D_C] == F.latents(F.codes(x[:, :D_C], e), e)).all()
    finally:
        mla.load().mla_test_set_split_form(0)


_KEPT = {}


def i32_at(*x):
    """Small constants on the GPU, made once: streams that run at once do not wait for copies."""
    if x not in _KEPT:
        _KEPT[x] = i32(list(x))
    return _KEPT[x]


@pytest.mark.parametrize("io,heads,q_len", [(BF16, 16, 1), (F32, 16, 3), (BF16, 64, 2)])
def test_many_short_sequences(cuda_lib, io, heads, q_len):
    """More sequences than are ever cut into shares, most of a page or less, some of none."""
    B = 1500
    c = Call(cuda_lib, np.arange(B) * 7 % 41, 16, io, heads, q_len, seed=11)
    c.run().check(status=cuda_lib.MLA_DEV_LENGTH_OUT_OF_RANGE,       # those of none are reported
                  tokens=[0, 1, 5 * q_len, 41 * q_len - 1, 700 * q_len, B * q_len - 1])
    empty = torch.from_numpy(np.arange(B) * 7 % 41 == 0).cuda().repeat_interleave(q_len)
    assert (c.o[empty] == 0).all() and torch.isneginf(c.lse[empty]).all()
    assert torch.isfinite(c.o.float()).all()


def test_read_with_starts_in_no_order(cuda_lib):
    """Row starts that do not ascend: rows that belong to nobody may be anything, but nothing
    behind the last start, or the block's end, is written."""
    mla = cuda_lib
    rng = np.random.RandomState(12)
    pool, t, pages = _q4.make_pool(rng, [40, 25, 60], 16)
    d, pg = mla.dims(3, 16, 64, mla.MLA_FP4_E2M1), mla.paging(16, pages, t.shape[1])
    for starts, end in (([0, 90, 20, 70], 70), ([50, 10, 3, 0], 0), ([0, -5, 1 << 30, 100], 80),
                        ([-(1 << 31), (1 << 31) - 1, 5, -3], 0)):
        out = torch.full((100, ROW), 3.0, device="cuda")
        mla.cache_read_paged(d, pg, pool.cuda(), t.cuda(), i32([40, 25, 60]),
                             torch.tensor(starts, dtype=torch.int32, device="cuda"), out[:80],
                             dev_status=status_word())
        torch.cuda.synchronize()
        assert (out[end:] == 3).all()


@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 128)])
def test_plain_launches_and_the_other_form(cuda_lib, io, heads):
    """Launches without overlap give the same bits; SM pairs asked for two parts run as CTAs of
    16 heads, within the same bounds."""
    mla = cuda_lib
    c = Call(mla, [1, 640, 257, 2000], 64, io, heads, seed=13, s_max=2100, width=40)
    c.run().check()
    o, lse = c.o.clone(), c.lse.clone()
    mla.set_launch_overlap(False)
    try:
        c.o.fill_(7)
        c.run()
        torch.cuda.synchronize()
    finally:
        mla.set_launch_overlap(True)
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    mla.set_split_parts(2)
    try:
        n = mla.paged_workspace_bytes(c.d, c.pg, io)
        c.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        c.o.fill_(7)
        c.run().check()
    finally:
        mla.set_split_parts(0)
