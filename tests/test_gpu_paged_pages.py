"""The paged cache's bookkeeping on the GPU against the oracle: block tables and
slot maps, released pages, rows appended to their slots, and the page index.
Whole numbers are compared exactly."""
import numpy as np
import pytest
import torch

from _paged import D_C, DT, ROW, f64, half_step, make_pool
from oracle import mla_oracle as O
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Tables:
    """Device state of one pool's tables."""

    def __init__(self, cached, table, free, num_free, page, pages, max_tokens):
        B = len(cached)
        self.page, self.pages = page, pages
        self.cached, self.table = i32(cached), i32(table)
        self.free, self.num_free = i32(free), i32([num_free])
        self.lengths = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        self.starts = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
        self.slots = torch.full((max_tokens,), -9, dtype=torch.int64, device="cuda")
        self.pos = torch.full((max_tokens,), -9, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def extend(self, mla, new, **kw):
        pg = mla.paging(self.page, self.pages, self.table.shape[1])
        mla.pages_extend(pg, kw.pop("cached", self.cached), new, self.table, self.free,
                         self.num_free, kw.pop("lengths", self.lengths), self.starts, self.slots,
                         self.pos, dev_status=self.status, **kw)

    def check(self, want, lengths=None):
        n = lambda t: t.cpu().numpy()
        assert int(self.status.item()) == want["status"]
        assert (n(self.table) == want["table"]).all()
        assert (n(self.lengths if lengths is None else lengths) == want["lengths"]).all()
        assert (n(self.starts) == want["row_starts"]).all()
        assert (n(self.slots) == want["slots"]).all()
        assert (n(self.pos) == want["positions"]).all()
        assert int(self.num_free.item()) == want["num_free"]


def draw_tables(rng, B, page, width, most_new):
    cached = rng.randint(0, width * page + 1, B)
    new = np.minimum(rng.randint(0, most_new + 1, B), width * page - cached)
    have = -(-cached // page)
    pages = int(have.sum() + (-(-(cached + new) // page) - have).sum()) + 4
    ids = rng.permutation(pages)
    table = np.full((B, width), -1)
    k = 0
    for b in range(B):
        table[b, :have[b]] = ids[k:k + have[b]]
        k += have[b]
    free = np.full(pages, -3)                 # entries above the stack's top are never read
    free[:pages - k] = ids[k:]
    return cached, new, table, free, pages - k, pages


@pytest.mark.parametrize("B,page,width,most,room", [
    (1, 16, 4, 40, 0), (1, 64, 2, 0, 1), (7, 32, 9, 100, 3), (64, 64, 130, 1, 0),
    (300, 16, 20, 200, 5), (1025, 128, 3, 2, 0), (2050, 16, 3, 17, 11), (16384, 256, 2, 1, 0),
    (40, 64, 60, 3000, 1),
    (3, 16, 900, 14000, 2), (5000, 16, 9, 5, 0)])
def test_extend_matches_the_oracle(cuda_lib, B, page, width, most, room):
    rng = np.random.RandomState(B + page)
    cached, new, table, free, nf, pages = draw_tables(rng, B, page, width, most)
    T = max(int(new.sum()) + room, 1)
    t = Tables(cached, table, free, nf, page, pages, T)
    t.extend(cuda_lib, i32(new))
    torch.cuda.synchronize()
    t.check(PO.extend(list(map(int, cached)), list(map(int, new)), table, free, nf, page, pages, T))


def test_extend_in_place_and_replayed(cuda_lib):
    """lengths over cached_lens, num_free in place: one captured step replayed is a
    decode loop; padding tokens keep slot -1."""
    rng = np.random.RandomState(5)
    B, page, width = 9, 16, 6
    cached, _, table, free, nf, pages = draw_tables(rng, B, page, 3, 0)
    table = np.concatenate([table, np.full((B, 3), -1)], 1)
    pages += 40
    free = np.concatenate([free[:nf], np.arange(pages - 40, pages)])
    free = np.concatenate([free, np.full(pages - len(free), -3)])
    nf += 40
    new = (np.arange(B) % 3 != 0).astype(int)
    t = Tables(cached, table, free, nf, page, pages, B)
    g = torch.cuda.CUDAGraph()
    dev_new = i32(new)
    t.extend(cuda_lib, i32(np.zeros(B)), cached=i32(np.zeros(B)), lengths=t.lengths)   # loads the module
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        t.extend(cuda_lib, dev_new, lengths=t.cached)
    want = dict(table=table, lengths=cached, num_free=nf)
    for _ in range(20):
        g.replay()
        want = PO.extend(list(map(int, want["lengths"])), list(map(int, new)), want["table"], free,
                         want["num_free"], page, pages, B)
    torch.cuda.synchronize()
    assert want["status"] == 0
    t.check(want, lengths=t.cached)


@pytest.mark.parametrize("what", ["exhausted", "table", "tokens", "negative", "stack", "huge"])
def test_extend_all_or_nothing(cuda_lib, what):
    rng = np.random.RandomState(6)
    B, page, width = 5, 16, 4
    cached, table, pages = [0, 5, 16, 30, 2], np.full((B, width), 3), 30
    new = [1, 20, 30, 2, 0]
    free, nf, T = rng.permutation(pages), 6, 60
    if what == "exhausted":
        nf = 3
    elif what == "table":
        new = [1, 20, 30, 35, 0]
    elif what == "tokens":
        T = 52
    elif what == "negative":
        new = [1, -1, 0, 0, 0]
    elif what == "stack":
        nf = pages + 1
    else:
        cached, new = [0, 2 ** 31 - 1, 16, 30, 2], [1, 2 ** 31 - 1, 0, 0, 0]
    t = Tables(cached, table, free, nf, page, pages, T)
    t.extend(cuda_lib, i32(new))
    torch.cuda.synchronize()
    want = PO.extend(cached, new, table, free, nf, page, pages, T)
    assert want["status"] != 0
    t.check(want)


def test_extend_reports_pages_outside_the_pool(cuda_lib):
    """A free-list or table entry that names no page: status, slots -1, no write elsewhere."""
    page, pages = 16, 8
    table = np.array([[1, -1, -1], [9, -1, -1], [-5, 2, -1]])
    free = np.array([4, 8, 5, -1, 6, 0, 0, 0])
    cached, new = [10, 10, 20], [30, 2, 3]
    t = Tables(cached, table, free, 5, page, pages, 40)
    t.extend(cuda_lib, i32(new))
    torch.cuda.synchronize()
    want = PO.extend(cached, new, table, free, 5, page, pages, 40)
    assert want["status"] == PO.PAGE
    t.check(want)


@pytest.mark.parametrize("what", ["some", "none", "all", "bad page", "bad length", "double"])
def test_release(cuda_lib, what):
    mla = cuda_lib
    rng = np.random.RandomState(7)
    B, page, width = 1500 if what == "some" else 6, 16, 5
    lengths, _, table, free, nf, pages = draw_tables(rng, B, page, width, 0)
    done = (rng.rand(B) < 0.4).astype(int)
    done[2] = 1
    lengths[2] = max(lengths[2], 1)
    if what == "none":
        done[:] = 0
    elif what == "all":
        done[:] = -1                                  # any nonzero value
    elif what == "bad page":
        table[2, 0] = pages
    elif what == "bad length":
        lengths[2] = width * page + 1
    elif what == "double":
        nf = pages
    if what in ("some", "all", "none"):               # entries of row 2 made valid above
        table[2, 0] = table[2, 0] if table[2, 0] >= 0 else 0
    pg = mla.paging(page, pages, width)
    dev = dict(lengths=i32(lengths), table=i32(table), free=i32(free), nf=i32([nf]))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.pages_release(pg, i32(done), dev["lengths"], dev["table"], dev["free"], dev["nf"],
                      dev_status=status)
    torch.cuda.synchronize()
    want = PO.release(done, np.asarray(lengths), table, free, nf, page, pages)
    assert int(status.item()) == want["status"]
    assert (want["status"] != 0) == (what in ("bad page", "bad length", "double"))
    assert (dev["lengths"].cpu().numpy() == want["lengths"]).all()
    assert (dev["table"].cpu().numpy() == want["table"]).all()
    assert (dev["free"].cpu().numpy() == want["free_list"]).all()
    assert int(dev["nf"].item()) == want["num_free"]


@pytest.mark.parametrize("dtype,rows", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                        ("fp8", "bf16"), ("fp8", "f32")])
@pytest.mark.parametrize("n", [1, 5, 1027])
def test_append_paged(cuda_lib, dtype, rows, n):
    """Values rounded once to the cache's type: within half a step of the exact row
    (and fp32's own error of the rotation); every other row stays bit for bit."""
    mla = cuda_lib
    rng = np.random.RandomState(n)
    page, pages = 32, 50
    x = torch.from_numpy((rng.randn(n, ROW) * 3).astype(np.float32)).to(DT[rows])
    x[0, 3] = 1000.0                                   # saturates an E4M3 cache
    pos = rng.randint(0, 1 << 20, n)
    pos[0] = 0
    slots = rng.permutation(page * pages)[:n].astype(np.int64)
    skip = np.arange(n) % 7 == 3
    slots[skip] = -1
    pool0 = torch.from_numpy(rng.randn(pages, page, ROW).astype(np.float32)).to(DT[dtype])
    cache = pool0.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d, pg = mla.dims(1, 16, 64, mla.dtype_code(DT[dtype])), mla.paging(page, pages, 2)
    mla.cache_append_paged(d, pg, x.cuda(), i32(pos), torch.from_numpy(slots).cuda(), cache, 1e4,
                           dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = PO.latent_rows(f64(x), pos, D_C, 1e4)
    got = f64(cache).reshape(-1, ROW)
    live = slots[~skip]
    if dtype == "fp8":
        want = np.clip(want, -448, 448)
        step = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10)
    else:
        step = half_step(DT[dtype]) * np.abs(want)
    # the rotation: sine, cosine and angle to 2^-22 each, three fp32 roundings
    pair = np.repeat(np.abs(f64(x)[:, D_C:]).reshape(n, 32, 2).sum(2), 2, 1)
    extra = np.concatenate([np.zeros((n, D_C)), pair * 2.0 ** -20], 1)
    assert (np.abs(got[live] - want[~skip]) <= (step + 1.1 * extra)[~skip]).all()
    rest = np.ones(page * pages, bool)
    rest[live] = False
    raw = lambda t: t.cpu().view(torch.uint8).reshape(page * pages, -1).numpy()
    assert (raw(cache)[rest] == raw(pool0)[rest]).all()


def test_append_paged_reports_bad_rows(cuda_lib):
    mla = cuda_lib
    page, pages = 16, 3
    d, pg = mla.dims(1, 16, 16, mla.MLA_BF16), mla.paging(page, pages, 1)
    rows = torch.ones((4, ROW), dtype=torch.bfloat16, device="cuda")
    for slots, pos, bit in [([5, 48, 7, 8], [0, 0, 0, 0], mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                            ([5, -2, 7, 8], [0, 0, 0, 0], mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                            ([5, 1 << 40, 7, 8], [0, 0, 0, 0], mla.MLA_DEV_PAGE_OUT_OF_RANGE),
                            ([5, 6, 7, 8], [0, -1, 0, 0], mla.MLA_DEV_LENGTH_OUT_OF_RANGE)]:
        cache = torch.zeros((pages, page, ROW), dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mla.cache_append_paged(d, pg, rows, i32(pos), torch.tensor(slots, device="cuda"), cache,
                               dev_status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == bit
        written = torch.nonzero(cache.view(-1, ROW).abs().sum(1)).flatten().cpu().tolist()
        assert written == [5, 7, 8]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_index_matches_the_oracle(cuda_lib, dtype, page):
    """Codes and scales equal the oracle's exactly, for the touched pages only."""
    mla = cuda_lib
    rng = np.random.RandomState(page)
    lengths = np.array([1, page, page + 1, 3 * page - 1, 0, 2 * page, 5 * page + 7])
    first = np.array([0, page - 1, 0, page + 3, 0, 2 * page, 0])
    pool, table, pages = make_pool(rng, lengths, page, dtype, gain=20.0)
    zero = int(table[6, 1])
    pool.view(torch.uint8)[zero] = 0                       # a page of zeros
    codes = torch.full((pages, ROW), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((pages,), -5.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = mla.dims(len(lengths), 16, int(lengths.max()), mla.dtype_code(DT[dtype]))
    pg = mla.paging(page, pages, table.shape[1])
    mla.page_index(d, pg, pool.cuda(), table.cuda(), i32(first), i32(lengths),
                   int((lengths - first).max()), codes, scales, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want_c, want_s = np.full((pages, ROW), 99), np.full(pages, -5.0, np.float32)
    rows64, tab = f64(pool), table.numpy()
    for b, n in enumerate(lengths):
        if first[b] >= n:
            continue
        for j in range(first[b] // page, -(-n // page)):
            c, s = PO.page_index(rows64[tab[b, j]][:min(page, n - j * page)].astype(np.float32))
            want_c[tab[b, j]], want_s[tab[b, j]] = c, s
    assert (codes.cpu().numpy() == want_c).all()
    assert (scales.cpu().numpy() == want_s).all()
    assert want_s[zero] == 0 and (want_c[zero] == 0).all()


def test_page_index_reports(cuda_lib):
    mla = cuda_lib
    rng = np.random.RandomState(9)
    lengths, page = np.array([40, 40, 40]), 16
    pool, table, pages = make_pool(rng, lengths, page, "bf16")
    d, pg = mla.dims(3, 16, 64, mla.MLA_BF16), mla.paging(page, pages, table.shape[1])
    run = lambda tab, first, lens, most: _index(mla, d, pg, pool, tab, first, lens, most, pages)
    assert run(table, [0, 0, 0], [40, 40, 40], 40)[0] == 0
    bad = table.clone()
    bad[1, 1] = pages
    st, codes = run(bad, [0, 0, 0], [40, 40, 40], 40)
    assert st == mla.MLA_DEV_PAGE_OUT_OF_RANGE
    assert (codes[table[1, 1]] == 0).all() and (codes[table[1, 2]] != 0).any()
    assert run(table, [0, 0, 0], [40, 41, 40], 40)[0] == mla.MLA_DEV_LENGTH_OUT_OF_RANGE
    for first, lens in [([0, -1, 0], [40] * 3), ([0] * 3, [40, 16 * table.shape[1] + 1, 40])]:
        st, codes = run(table, first, lens, 40)
        assert st == mla.MLA_DEV_LENGTH_OUT_OF_RANGE
        assert (codes[table[1, 0]] == 0).all() and (codes[table[2, 0]] != 0).any()


def _index(mla, d, pg, pool, table, first, lens, most, pages):
    codes = torch.zeros((pages, ROW), dtype=torch.int8, device="cuda")
    scales = torch.zeros(pages, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.page_index(d, pg, pool.cuda(), table.cuda(), i32(first), i32(lens), most, codes, scales,
                   dev_status=status)
    torch.cuda.synchronize()
    return int(status.item()), codes.cpu()
