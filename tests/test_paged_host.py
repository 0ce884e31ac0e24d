"""The paged cache's operators without a GPU: the oracle's definitions against
facts that do not depend on them, and the argument checks of the C ABI."""
import ctypes

import numpy as np
import pytest

from oracle import mla_oracle as O
from oracle import paged_oracle as PO


@pytest.fixture(scope="module")
def lib():
    from head_latent_attention_absorbed_gb300 import build as b
    path = b.build()
    import head_latent_attention_absorbed_gb300 as mla
    return mla, mla.load(path)


# ------------------------------------------------------------------ the oracle
def test_extend_then_release_restores_the_pool():
    rng = np.random.RandomState(1)
    page, pages, B, width = 16, 40, 5, 8
    free = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    cached, new = [0] * B, [0, 1, 16, 17, 100]
    r = PO.extend(cached, new, table, free, pages, page, pages, 200)
    assert r["status"] == 0 and r["num_free"] == pages - (0 + 1 + 1 + 2 + 7)
    used = r["table"][r["table"] >= 0]
    assert len(set(used)) == len(used) == 11                     # no page twice
    live = r["slots"][:134]
    assert len(set(live)) == 134 and (r["slots"][134:] == -1).all()
    assert list(r["row_starts"]) == [0, 0, 1, 17, 34, 134]
    # growing by nothing changes nothing; growing inside a page takes none
    again = PO.extend(list(r["lengths"]), [1, 0, 0, 15, 12], r["table"], free, r["num_free"], page,
                      pages, 64)
    assert again["num_free"] == r["num_free"] - 1 - 0
    back = PO.release(np.ones(B, np.int32), again["lengths"], again["table"], free,
                      again["num_free"], page, pages)
    assert back["status"] == 0 and back["num_free"] == pages
    assert sorted(back["free_list"]) == list(range(pages)) and (back["lengths"] == 0).all()


def test_extend_is_all_or_nothing():
    free = np.arange(4, dtype=np.int32)
    table = np.full((2, 3), -1, np.int32)
    for cached, new, nf, most, bit in [([0, 0], [16, 49], 4, 99, PO.LENGTH),   # longer than the table
                                       ([0, 0], [48, 48], 4, 99, PO.EXHAUSTED),
                                       ([0, 0], [30, 30], 4, 59, PO.LENGTH),   # too many tokens
                                       ([0, -1], [1, 1], 4, 99, PO.LENGTH)]:
        r = PO.extend(cached, new, table, free, nf, 16, 4, most)
        assert r["status"] == bit and r["num_free"] == nf and (r["slots"] == -1).all()
        assert (r["table"] == -1).all() and list(r["lengths"]) == cached


def test_attend_over_pages_is_the_dense_oracle():
    """Pages in any order hold the same sequence as a dense cache."""
    rng = np.random.RandomState(2)
    H, n, page = 3, 37, 16
    q_nope, q_rope = rng.randn(1, H, 128), rng.randn(1, H, 64)
    w_uk, w_uv = rng.randn(H, 128, 512) * 0.02, rng.randn(H, 128, 512) * 0.02
    dense = rng.randn(1, n, 576)
    r = O.decode_absorbed(q_nope, q_rope, w_uk, w_uv, dense, np.array([n]), np.array([n - 1]),
                          192 ** -0.5, 1e4)
    pool = np.full((5, page, 576), np.nan)
    table = np.array([4, 0, 2])
    for t in range(n):
        pool[table[t // page], t % page] = dense[0, t]
    q = np.concatenate([r["q_abs"][0], r["q_pe"][0]], 1)
    o, lse, p, z = PO.attend(q, PO.sequence_rows(pool, table, n), 192 ** -0.5, 512)
    assert np.abs(o - r["o_c"][0]).max() < 1e-12 and np.abs(lse - r["lse"][0]).max() < 1e-12
    assert np.allclose(p.sum(1), 1)


def test_page_index_is_the_mean_row():
    rng = np.random.RandomState(3)
    for n in (1, 5, 64):
        x = rng.randn(n, 576).astype(np.float32)
        codes, scale = PO.page_index(x)
        mean = x.astype(np.float64).mean(0)
        # half a code step, and 2^-21 of the power of two above the largest value
        bound = scale / 2 + 2.0 ** -20 * np.abs(x).max()
        assert np.abs(codes * float(scale) - mean).max() <= bound * (1 + 1e-6)
        assert np.abs(codes).max() == 127
        perm = PO.page_index(x[rng.permutation(n)])
        assert (perm[0] == codes).all() and perm[1] == scale     # order does not matter
    assert PO.page_index(np.zeros((4, 576), np.float32))[1] == 0
    inf = np.zeros((4, 576), np.float32)
    inf[0, 0] = np.inf
    assert PO.page_index(inf)[1] == 0


def test_page_score_finds_the_planted_page():
    rng = np.random.RandomState(4)
    q = rng.randn(4, 576).astype(np.float32)
    pages = [rng.randn(16, 576).astype(np.float32) for _ in range(12)]
    pages[7] += 2 * q[1]                                          # one head's rows of interest
    idx = [PO.page_index(x) for x in pages]
    s = PO.page_scores(q, np.stack([c for c, _ in idx]), np.array([z for _, z in idx]))
    assert np.argmax(s) == 7
    exact = np.max([(q.astype(np.float64) @ x.astype(np.float64).mean(0)) for x in pages], axis=1)
    # each code is off by half a step: relative to the largest |q| and |mean| 2 x 1/254 at most
    for j, x in enumerate(pages):
        m = x.astype(np.float64).mean(0)
        slack = np.max(np.abs(q).max(1) / 254 * np.abs(m).sum() +
                       (np.abs(q).sum(1) + 576 * np.abs(q).max(1) / 254) * np.abs(m).max() / 254)
        assert abs(s[j] - exact[j]) <= slack * 1.01


def test_select_keeps_ends_best_and_lowest_of_ties():
    s = np.array([9, 1, 5, 5, 7, 5, 0, 9], np.float32)
    assert PO.select(s, 8, 8, 1, 1) == list(range(8))
    assert PO.select(s, 8, 5, 1, 1) == [0, 2, 3, 4, 7]
    assert PO.select(s, 8, 4, 1, 2) == [0, 4, 6, 7]
    assert PO.select(s, 8, 2, 1, 1) == [0, 7]
    assert PO.select(s, 8, 3, 0, 1) == [0, 4, 7]


# ------------------------------------------------------------------ the C ABI's refusals
GOOD = 0x10000


def P(x=GOOD):
    return ctypes.c_void_p(x)


def test_paging_is_checked(lib):
    mla, so = lib
    d = mla.dims(2, 16, 100, mla.MLA_BF16)

    def splits(pg, dd=d, io=mla.MLA_BF16, q_len=1):
        return so.mla_paged_num_splits(ctypes.byref(dd), ctypes.byref(pg), io, q_len, 0)

    assert splits(mla.paging(64, 10, 2)) >= 1
    for pg in (mla.paging(8, 10, 20), mla.paging(48, 10, 20), mla.paging(512, 10, 20),
               mla.paging(64, 0, 2), mla.paging(64, 10, 0), mla.paging(64, 1 << 26, 2),
               mla.paging(64, 10, 1)):                         # s_max = 100 rows need two pages
        assert splits(pg) == 0, (pg.page_size, pg.num_pages, pg.table_stride)
        assert so.mla_last_error_message()
    pg = mla.paging(64, 10, 2)
    assert splits(pg, q_len=0) == 0 and splits(pg, q_len=40000) == 0
    assert splits(pg, io=7) == 0
    assert splits(pg, mla.dims(2, 16, 100, mla.MLA_F32), mla.MLA_BF16) == 0    # fp32 cache: fp32 queries
    assert splits(pg, mla.dims(2, 16, 100, mla.MLA_F32), mla.MLA_F32) >= 1
    # chunks are whole tiles
    assert splits(pg) == 1


def test_paged_plan_goes_by_the_query_type(lib):
    """bf16 queries take 64 heads per CTA at multiples of 64 heads, fp32 ones 32:
    twice the CTAs per chunk, so the planner takes about half the chunks."""
    mla, so = lib
    d, pg = mla.dims(4, 128, 16384, mla.MLA_BF16), mla.paging(64, 2000, 256)
    import torch
    b = mla.paged_num_splits(d, pg, torch.bfloat16)
    f = mla.paged_num_splits(d, pg, torch.float32)
    assert b > f >= 1
    assert mla.paged_workspace_bytes(d, pg, torch.bfloat16) >= 4 * 128 * b * 513 * 4
    with pytest.raises(ValueError):
        mla.paged_workspace_bytes(d, mla.paging(63, 2000, 300), torch.bfloat16)
    with pytest.raises(ValueError):
        mla.paged_num_splits(d, pg, torch.float16)


def test_refusals_before_any_launch(lib):
    mla, so = lib
    d, pg = mla.dims(2, 16, 100, mla.MLA_BF16), mla.paging(64, 10, 2)
    D, G = ctypes.byref(d), ctypes.byref(pg)
    big = 1 << 30

    def attn(q=P(), cache=P(), table=P(), lengths=P(), scale=0.1, splits=0, ws=P(), n=big, o=P(),
             io=1, q_len=1):
        return so.mla_decode_attn_paged(D, G, io, q_len, q, P(), cache, table, lengths, scale,
                                        splits, ws, n, o, None, None, None)

    assert attn(q=None) == 1 and attn(table=None) == 1 and attn(lengths=None) == 1
    assert attn(o=P(GOOD + 8)) == 1 and attn(cache=P(GOOD + 4)) == 1 and attn(ws=None) == 1
    assert attn(scale=0.0) == 1 and attn(scale=float("nan")) == 1 and attn(splits=-1) == 1
    assert attn(n=16) == 3 and attn(io=2) == 2 and attn(q_len=0) == 1

    def extend(batch=2, most=8, **kw):
        a = dict(cached=P(), new=P(), table=P(), free=P(), nf=P(), nfo=P(), lens=P(), starts=P(),
                 slots=P(), pos=P())
        a.update(kw)
        return so.mla_pages_extend(batch, G, a["cached"], a["new"], most, a["table"], a["free"],
                                   a["nf"], a["nfo"], a["lens"], a["starts"], a["slots"],
                                   a["pos"], None, None)

    assert extend(batch=0) == 1 and extend(batch=16385) == 2 and extend(most=0) == 1
    for k in ("cached", "new", "table", "free", "nf", "nfo", "lens", "starts", "slots", "pos"):
        assert extend(**{k: None}) == 1, k
    assert so.mla_pages_release(0, G, P(), P(), P(), P(), P(), None, None) == 1
    assert so.mla_pages_release(2, G, None, P(), P(), P(), P(), None, None) == 1

    def append(n=4, dt=1, rows=P(), pos=P(), slots=P(), cache=P(), base=1e4, dd=d):
        return so.mla_cache_append_paged(ctypes.byref(dd), G, n, dt, rows, pos, slots, base, cache,
                                         None, None)

    assert append(n=-1) == 1 and append(base=0.0) == 1 and append(rows=None) == 1
    assert append(rows=P(GOOD + 8)) == 1 and append(cache=P(GOOD + 2)) == 1
    assert append(dt=2) == 2 and append(dd=mla.dims(2, 16, 100, mla.MLA_F32)) == 2
    assert append(n=0, rows=None) == 0                          # nothing to write

    def index(most=4, **kw):
        a = dict(cache=P(), table=P(), first=P(), lens=P(), codes=P(), scales=P())
        a.update(kw)
        return so.mla_page_index(D, G, most, a["cache"], a["table"], a["first"], a["lens"],
                                 a["codes"], a["scales"], None, None)

    assert index(most=0) == 1 and index(codes=P(GOOD + 1)) == 1
    for k in ("cache", "table", "first", "lens", "codes", "scales"):
        assert index(**{k: None}) == 1, k

    def select(top=2, kf=1, kl=1, n=big, io=1, **kw):
        a = dict(q=P(), table=P(), lens=P(), codes=P(), scales=P(), ws=P(), sel=P(), sl=P())
        a.update(kw)
        return so.mla_select_pages(D, G, io, 1, a["q"], P(), a["table"], a["lens"], a["codes"],
                                   a["scales"], top, kf, kl, a["ws"], n, a["sel"], a["sl"], None,
                                   None)

    assert select(top=0) == 1 and select(kf=-1) == 1 and select(kl=0) == 1
    assert select(top=2, kf=2, kl=1) == 1 and select(n=16) == 3 and select(io=5) == 2
    for k in ("q", "table", "lens", "codes", "scales", "ws", "sel", "sl"):
        assert select(**{k: None}) == 1, k

    def sparse(n=big, scale=0.1, o=P(), top=2):
        return so.mla_decode_attn_sparse(D, G, 1, 1, P(), P(), P(), P(), P(), P(), P(), scale, top,
                                         1, 1, 0, P(), n, P(), P(), o, None, None, None)

    need = so.mla_sparse_workspace_bytes(D, G, 1, 1, 2, 0)
    assert need > so.mla_select_workspace_bytes(D, G, 1) > 0
    assert sparse(n=need - 1) == 3 and sparse(scale=-1.0) == 1 and sparse(o=None) == 1
    assert sparse(top=1) == 1
    assert so.mla_sparse_workspace_bytes(D, G, 1, 1, 0, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    """Every paged wrapper names what is wrong before it calls the library (on a
    machine without a GPU every tensor is one on the wrong device)."""
    mla, _ = lib
    import torch
    from head_latent_attention_absorbed_gb300 import _binding as b
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)
    pg = mla.paging(64, 10, 2)
    b._paged_lib()

    class Fake:
        """A tensor that says it is on device 0."""

        def __init__(self, t):
            self.t, self.dtype, self.is_cuda = t, t.dtype, True

        def __getattr__(self, name):
            return getattr(self.t, name)

        def get_device(self):
            return 0

    good = Fake(z(3))
    assert b._is(good, 0, torch.int32, 3)
    assert not b._is(good, 1, torch.int32, 3) and not b._is(good, 0, torch.int64, 3)
    assert not b._is(good, 0, torch.int32, 4) and not b._is(Fake(z(3, 2)[:, 0]), 0, torch.int32, 3)
    for t, dt, n, word in [(z(3), torch.int32, 3, "device"), (good, torch.int64, 3, "int64"),
                           (good, torch.int32, 4, "4 values"),
                           (Fake(z(3, 2)[:, 0]), torch.int32, 3, "contiguous")]:
        with pytest.raises(ValueError, match=word):
            b._explain(0, lengths=(t, dt, n))
    with pytest.raises(ValueError, match="fp32 or bf16"):
        b._io_code(torch.float16)
    assert b._io_code(torch.bfloat16) == mla.MLA_BF16 and b._io_code(torch.float32) == mla.MLA_F32
