"""The 4-bit pool without a GPU: the oracle's definition against facts that do not depend
on it, and the argument checks of the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest

from oracle import fp4_oracle as F


@pytest.fixture(scope="module")
def lib():
    from head_latent_attention_absorbed_gb300 import build as b
    path = b.build()
    import head_latent_attention_absorbed_gb300 as mla
    return mla, mla.load(path)


# ------------------------------------------------------------------ the oracle
def test_rounding_is_to_the_nearest_value_of_the_block():
    rng = np.random.RandomState(0)
    x = rng.randn(50, 512) * np.exp2(rng.randint(-12, 9, (50, 32))).repeat(16, 1)
    e = F.exponents(x)
    got = F.latents(F.codes(x, e), e)
    grid = np.concatenate([-F.GRID[::-1], F.GRID])
    unit = 2.0 ** e.repeat(16, 1)
    best = np.abs(x[..., None] - grid * unit[..., None]).min(-1)
    assert (np.abs(x - got) == best).all()
    near = np.abs(x) <= 448                      # what lies further saturates
    assert (np.abs(x - got)[near] <= unit[near]).all()


def test_exponent_is_the_smallest_that_holds_the_block():
    x = np.zeros((1, 512))
    for top, e in [(0, -8), (2.0 ** -9, -8), (7 / 256, -8), (7.0001 / 256, -7), (6, 0), (7, 0),
                   (7.01, 1), (384, 6), (448, 6), (1e30, 6), (np.inf, 6), (np.nan, 6)]:
        x[0, 21] = -top
        got = F.exponents(x)
        assert got[0, 1] == e and (np.delete(got[0], 1) == -8).all(), top
    assert F.rounded(np.array([[np.nan] + [0.0] * 511]))[0, 0] == 384
    assert F.rounded(np.array([[-np.inf] + [31.0] * 511]))[0, :2].tolist() == [-384, 32]


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 512))
    x[0, :9] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25]
    assert F.rounded(x)[0, :9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0]


def test_every_value_is_an_e4m3_number():
    import torch
    code = np.tile(np.arange(16), 32)[None].repeat(15, 0)
    e = np.arange(-8, 7)[:, None].repeat(32, 1)
    v = torch.from_numpy(F.latents(code, e))
    assert torch.equal(v.to(torch.float8_e4m3fn).double(), v)


@pytest.mark.parametrize("page", [16, 256])
def test_pack_and_unpack(page):
    rng = np.random.RandomState(page)
    code, e = rng.randint(0, 16, (3, page, 512)), rng.randint(-8, 8, (3, page, 32))
    key = rng.randint(0, 1 << 16, (3, page, 64)).astype(np.uint16)
    pool = F.pack(code, e, key)
    assert pool.shape == (3, page * 400)
    for a, b in zip(F.unpack(pool, page), (code, e, key)):
        assert (a == b).all()
    # rows by their own bytes: codes and exponents, then keys
    flat = pool[1]
    word = int(flat[5 * 272 + 12:][:4].view("<u4")[0])
    bits = [7, 15, 23, 31, 3, 11, 19, 27]
    assert [(word >> 4 * k & 7) | (word >> bits[k] & 1) << 3 for k in range(8)] == code[1, 5, 24:32].tolist()
    assert flat[5 * 272 + 256 + 3] == ((e[1, 5, 6] + 5) & 15) | ((e[1, 5, 7] + 5) & 15) << 4
    piece = flat[page * 272 + 5 * 128:][:128].reshape(8, 16)[2 ^ 5]
    assert (piece.view(np.uint16) == key[1, 5, 16:24]).all()


# ------------------------------------------------------------------ the calls' checks
GOOD = 1 << 20


def P(x=GOOD):
    return ctypes.c_void_p(x)


def test_pool_bytes(lib):
    mla, _ = lib
    for dtype, row in [(mla.MLA_F32, 2304), (mla.MLA_BF16, 1152), (mla.MLA_FP8_E4M3, 576),
                       (mla.MLA_FP4_E2M1, 400)]:
        assert mla.pool_bytes(mla.dims(2, 16, 100, dtype), mla.paging(64, 7, 2)) == 7 * 64 * row
    big = mla.paging(256, 8000000, 2)              # past 2^31 bytes
    assert mla.pool_bytes(mla.dims(2, 16, 100, mla.MLA_FP4_E2M1), big) == 8000000 * 256 * 400
    with pytest.raises(ValueError):
        mla.pool_bytes(mla.dims(2, 16, 100, 7), mla.paging(64, 7, 2))
    with pytest.raises(ValueError):
        mla.pool_bytes(mla.dims(2, 16, 100, mla.MLA_FP4_E2M1), mla.paging(48, 7, 2))


def test_dense_calls_refuse_the_type(lib):
    mla, so = lib
    d = mla.dims(2, 16, 100, mla.MLA_FP4_E2M1)
    D = ctypes.byref(d)
    assert so.mla_decode_num_splits(D, 0) == 0 and so.mla_decode_workspace_bytes(D, 0) == 0
    assert so.mla_decode_multi_num_splits(D, 2, 0) == 0 and so.mla_decode_heads_per_cta(D) == 0
    assert so.mla_decode_plan(D, 0, None, None, None) == 2
    assert so.mla_decode_attn(D, P(), P(), P(), P(), 0.1, 0, P(), 1 << 30, P(), None, None, None) == 2
    assert so.mla_decode_attn_multi(D, 2, P(), P(), P(), P(), 0.1, 0, P(), 1 << 30, P(), None, None,
                                    None) == 2
    assert so.mla_absorb_q(D, P(), P(), P(), P(), 1e4, P(), P(), None) == 2
    assert so.mla_out_proj(D, P(), P(), P(), None) == 2
    assert so.mla_cache_append(D, 2048, P(), P(), P(), 1e4, P(), None, None) == 2
    assert so.mla_wo_proj(D, 2048, P(), P(), P(), None) == 2
    assert b"paged" in so.mla_last_error_message()


def test_heads_are_multiples_of_16(lib):
    mla, so = lib
    pg = mla.paging(64, 10, 2)
    import torch
    for h, ok in [(16, True), (48, True), (8, False), (130, False)]:
        d = mla.dims(2, h, 100, mla.MLA_FP4_E2M1)
        n = so.mla_paged_workspace_bytes(ctypes.byref(d), ctypes.byref(pg), 1, 1, 0)
        assert (n > 0) == ok


def test_read_refusals(lib):
    mla, so = lib
    G = ctypes.byref(mla.paging(64, 10, 2))

    def read(dtype=mla.MLA_FP4_E2M1, n=4, kind=1, g=G, **kw):
        a = dict(cache=P(), table=P(), lens=P(), starts=P(), rows=P())
        a.update(kw)
        return so.mla_cache_read_paged(ctypes.byref(mla.dims(2, 16, 100, dtype)), g, a["cache"],
                                       a["table"], a["lens"], a["starts"], None, n, kind, a["rows"],
                                       None, None)

    for k in ("cache", "table", "lens", "starts", "rows"):
        assert read(**{k: None}) == 1, k
    assert read(cache=P(GOOD + 8)) == 1 and read(rows=P(GOOD + 8)) == 1 and read(n=-1) == 1
    assert read(kind=2) == 2 and read(kind=3) == 2 and read(dtype=9) == 2
    assert read(g=ctypes.byref(mla.paging(24, 10, 2))) == 2 and read(g=None) == 1
    assert read(n=0, rows=None) == 0


def test_append_and_attention_refusals(lib):
    mla, so = lib
    d, pg = mla.dims(2, 16, 100, mla.MLA_FP4_E2M1), mla.paging(64, 10, 2)
    D, G = ctypes.byref(d), ctypes.byref(pg)

    def append(n=4, dt=1, rows=P(), cache=P()):
        return so.mla_cache_append_paged(D, G, n, dt, rows, P(), P(), 1e4, cache, None, None)

    assert append(dt=2) == 2 and append(dt=3) == 2 and append(rows=P(GOOD + 8)) == 1
    assert append(cache=P(GOOD + 4)) == 1 and append(n=0, rows=None) == 0

    def attn(cache=P(), n=1 << 30, io=1):
        return so.mla_decode_attn_paged(D, G, io, 1, P(), P(), cache, P(), P(), 0.1, 0, P(), n, P(),
                                        None, None, None)

    assert attn(cache=P(GOOD + 8)) == 1 and attn(cache=None) == 1 and attn(n=16) == 3
    assert attn(io=2) == 2 and attn(io=3) == 2
    need = so.mla_sparse_workspace_bytes(D, G, 1, 1, 2, 0)
    assert need > so.mla_select_workspace_bytes(D, G, 1) > 0
    assert so.mla_decode_attn_sparse(D, G, 1, 1, P(), P(), P(), P(), P(), P(), P(), 0.1, 2, 1, 1, 0,
                                     P(), need - 1, P(), P(), P(), None, None, None) == 3


def test_binding_knows_the_pool(lib):
    mla, _ = lib
    from head_latent_attention_absorbed_gb300 import _binding as b
    pg = mla.paging(64, 10, 2)
    for dtype in (mla.MLA_F32, mla.MLA_BF16, mla.MLA_FP8_E4M3):
        assert b._pool_numel(mla.dims(2, 16, 100, dtype), pg) == 10 * 64 * 576
    d = mla.dims(2, 16, 100, mla.MLA_FP4_E2M1)
    assert b._pool_numel(d, pg) == mla.pool_bytes(d, pg)
