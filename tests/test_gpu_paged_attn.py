"""Decode attention over a paged cache against the oracle, element by element
within bounds derived from the roundings the kernels make (see _paged)."""
import numpy as np
import pytest
import torch

from _paged import D_C, DT, SCALE, check_attention, f64, make_pool, make_queries

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Call:
    """One decode_attn_paged problem on the GPU."""

    def __init__(self, mla, lengths, page, dtype, io, heads, q_len=1, splits=0, seed=0, s_max=None,
                 **kw):
        rng = np.random.RandomState(seed)
        self.mla, self.q_len, self.dtype, self.io, self.splits = mla, q_len, dtype, io, splits
        self.lengths = np.asarray(lengths)
        self.pool, self.table, self.pages = make_pool(rng, self.lengths, page, dtype, **kw)
        B = len(lengths)
        self.q_abs, self.q_pe = make_queries(rng, B * q_len, heads, io)
        s_max = s_max or max(int(self.lengths.max()), 1)
        self.d = mla.dims(B, heads, s_max, mla.dtype_code(DT[dtype]))
        self.pg = mla.paging(page, self.pages, self.table.shape[1])
        n = mla.paged_workspace_bytes(self.d, self.pg, io, q_len, splits)
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.o = torch.full((B * q_len, heads, D_C), 7.0, dtype=io, device="cuda")
        self.lse = torch.full((B * q_len, heads), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
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
        return check_attention(self.o, self.lse, self.q_abs, self.q_pe, self.pool, self.table,
                               self.lengths, self.q_len, self.dtype, self.io, tokens)


F32, BF16 = torch.float32, torch.bfloat16
EDGES = [1, 15, 16, 17, 127, 128, 129, 300]
KINDS = [("f32", F32, 5), ("f32", F32, 16), ("bf16", F32, 16), ("bf16", BF16, 16), ("bf16", F32, 32),
         ("bf16", BF16, 48), ("bf16", BF16, 64), ("bf16", F32, 64), ("fp8", F32, 16),
         ("fp8", BF16, 32), ("bf16", BF16, 128), ("fp8", BF16, 128), ("bf16", BF16, 256),
         ("bf16", F32, 128), ("fp8", F32, 128)]


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_lengths_and_pages(cuda_lib, dtype, io, heads, page):
    """Ragged lengths around every tile and page edge, NaN past each end, table
    entries past a sequence's pages that name nothing."""
    Call(cuda_lib, EDGES, page, dtype, io, heads, seed=page + heads).run().check()


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("splits", [1, 2, 3])
def test_chunks(cuda_lib, dtype, io, heads, splits):
    """The rows cut into one, two and three chunks, the last ones of short sequences empty."""
    Call(cuda_lib, [700, 129, 1, 513], 64, dtype, io, heads, splits=splits, seed=splits,
         gain=8.0 if dtype != "fp8" else None).run().check()


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("q_len", [2, 3, 4])
def test_several_tokens(cuda_lib, dtype, io, heads, q_len):
    """q_len tokens per sequence, causal among themselves; lengths q_len and up."""
    Call(cuda_lib, [q_len, 128 + q_len, 131, 400], 32, dtype, io, heads, q_len=q_len,
         seed=q_len).run().check()


@pytest.mark.parametrize("io,page", [(F32, 16), (BF16, 64), (BF16, 256)])
def test_persistent_grid(cuda_lib, io, page):
    """Enough work for the persistent grid of the 16-head kernel: items of many
    sequences in one CTA, sequences that end inside a tile in the middle of a
    CTA's stream."""
    mla = cuda_lib
    rng = np.random.RandomState(3)
    lengths = rng.randint(1, 1500, 60)
    lengths[:4] = [1, 128, 1499, 129]
    mla.load().mla_test_set_split_form(1)
    try:
        Call(mla, lengths, page, "bf16", io, 16, seed=8).run().check(tokens=range(0, 60, 3))
        Call(mla, lengths, page, "bf16", io, 48, seed=9).run().check(tokens=range(0, 60, 7))
    finally:
        mla.load().mla_test_set_split_form(0)
    c = Call(mla, rng.randint(3000, 6000, 40), page, "bf16", io, 16, seed=10).run()
    c.check(tokens=[0, 17, 39])


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
@pytest.mark.parametrize("io,heads,q_len,page", [(F32, 16, 1, 16), (BF16, 16, 1, 64),
                                                 (BF16, 32, 1, 256), (F32, 128, 1, 64),
                                                 (F32, 16, 3, 32), (BF16, 16, 2, 128)])
@pytest.mark.parametrize("B", [7, 70])
def test_equal_shares(cuda_lib, kind, io, heads, q_len, page, B):
    """The FP8 cache's tiles in equal runs: runs that start and end inside a sequence,
    hold several, one tile each, and fewer tiles than CTAs."""
    mla = cuda_lib
    lengths = share_lengths(kind, B)
    if q_len > 1:
        lengths = np.maximum(lengths, q_len)
    mla.load().mla_test_set_split_form(1)
    try:
        c = Call(mla, lengths, page, "fp8", io, heads, q_len=q_len, seed=B + heads)
        c.run()
        first = c.o.clone()
        c.check(tokens=range(0, B * q_len, max(1, B * q_len // 12)),
                status=0 if lengths.min() else mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
        c.o.fill_(7)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(first, c.o)   # no order of arrival changes a bit
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("kind", ["ragged", "one long", "edges"])
@pytest.mark.parametrize("dtype,heads,q_len,page", [("bf16", 32, 1, 16), ("bf16", 128, 1, 64),
                                                    ("bf16", 160, 1, 256), ("bf16", 16, 3, 32),
                                                    ("fp8", 48, 1, 16), ("fp8", 128, 1, 64),
                                                    ("fp8", 256, 1, 128), ("fp8", 64, 2, 32)])
@pytest.mark.parametrize("B", [7, 70])
def test_equal_shares_of_pairs(cuda_lib, kind, dtype, heads, q_len, page, B):
    """The same with SM pairs, in a workspace that is 16-byte aligned and no more."""
    mla = cuda_lib
    lengths = share_lengths(kind, B)
    if q_len > 1:
        lengths = np.maximum(lengths, q_len)
    mla.load().mla_test_set_split_form(1)
    try:
        c = Call(mla, lengths, page, dtype, BF16, heads, q_len=q_len, seed=B + heads)
        c.ws = torch.empty(c.ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]
        c.run()
        first = c.o.clone()
        c.check(tokens=range(0, B * q_len, max(1, B * q_len // 8)),
                status=0 if lengths.min() else mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
        c.o.fill_(7)
        c.run()
        torch.cuda.synchronize()
        assert torch.equal(first, c.o)
    finally:
        mla.load().mla_test_set_split_form(0)


SHARED = [("fp8", BF16, 16), ("fp8", F32, 32), ("bf16", BF16, 64), ("fp8", BF16, 128)]


@pytest.mark.parametrize("dtype,io,heads", SHARED)
def test_equal_shares_back_to_back(cuda_lib, dtype, io, heads):
    """Calls that follow one another on one workspace, unsynchronised, with lengths that
    change between them: each gives what it gives alone.  The counts of one call's partials
    may not reach the combine of another."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1)
    try:
        calls = []
        for seed, lengths in enumerate((share_lengths("ragged", 24) + 1,
                                        share_lengths("one long", 24) + 1, np.full(24, 640))):
            calls.append(Call(mla, lengths, 64, dtype, io, heads, seed=seed, s_max=7000,
                              width=110))
        for c in calls:
            c.ws = calls[0].ws
        alone = []
        for c in calls:
            c.run()
            torch.cuda.synchronize()
            alone.append((c.o.clone(), c.lse.clone()))
            c.check(tokens=[0, 11, 12, 23])
        outs = [[torch.full_like(c.o, 7) for _ in range(12)] for c in calls]
        torch.cuda.synchronize()
        for k in range(12):
            for c, o in zip(calls, outs):
                c.o = o[k]
                c.run()
        torch.cuda.synchronize()
        for (o, lse), c, got in zip(alone, calls, outs):
            assert all(torch.equal(o, g) for g in got)
            assert torch.equal(lse, c.lse)
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("dtype,io,heads", SHARED)
def test_equal_shares_captured(cuda_lib, dtype, io, heads):
    """A captured call cuts its shares anew from the lengths of each replay; without lse."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1)
    try:
        c = Call(mla, [1500] * 20, 64, dtype, io, heads, seed=5)
        c.lse = None
        c.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        c.lse = torch.empty((20, heads), device="cuda")
        for lengths in (share_lengths("ragged", 20), [1] * 20, [1500] * 20, [0] * 19 + [1500]):
            c.dev["lengths"].copy_(i32(lengths))
            graph.replay()
            got = c.o.clone()
            c.o.fill_(7)
            c.run()
            torch.cuda.synchronize()
            assert torch.equal(got, c.o)
            c.lengths = np.asarray(lengths)
            # rows between the length and the page's end are finite here; so are the pages
            c.check(tokens=[0, 1, 10, 19],
                    status=int(c.status.item()))
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("dtype,io,heads", SHARED)
def test_equal_shares_of_one_long_sequence(cuda_lib, dtype, io, heads):
    """One sequence over all CTAs: over a hundred partials."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1)
    try:
        Call(mla, [40001], 64, dtype, io, heads, seed=6).run().check()
    finally:
        mla.load().mla_test_set_split_form(0)


def test_equal_shares_by_size(cuda_lib):
    """Enough tiles that the planner takes equal shares itself; 512 query groups are the
    most it takes them for, and a length past s_max is cut and reported there too."""
    mla = cuda_lib
    rng = np.random.RandomState(4)
    lengths = rng.randint(1, 4000, 60)
    c = Call(mla, lengths, 64, "fp8", BF16, 16, seed=3).run()
    c.check(tokens=[0, 11, 31, 32, 59])
    lengths = rng.randint(0, 1200, 512)
    lengths[511] = 1200
    c = Call(mla, lengths, 64, "fp8", BF16, 16, seed=5).run()
    c.check(tokens=[0, 255, 256, 510, 511], status=0 if lengths.min() else
            mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    lengths = np.concatenate([lengths, [1000]])
    c = Call(mla, lengths, 64, "fp8", BF16, 16, seed=5).run()
    c.check(tokens=[0, 511, 512], status=0 if lengths.min() else mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    lengths = np.full(40, 3000)
    c = Call(mla, lengths, 64, "fp8", F32, 16, seed=6, s_max=2900).run()
    c.lengths = np.full(40, 2900)
    c.check(tokens=[0, 39], status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)


@pytest.mark.parametrize("dtype,io,heads", KINDS)
def test_empty_and_bad_lengths(cuda_lib, dtype, io, heads):
    """No rows: zeros and -inf, with the status bit; a length above s_max is cut there."""
    mla = cuda_lib
    c = Call(mla, [0, 5, 0, 140], 16, dtype, io, heads, seed=1).run()
    c.check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    c = Call(mla, [200, 130], 16, dtype, io, heads, seed=2, s_max=150).run()
    c.lengths = np.array([150, 130])
    c.check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    c = Call(mla, [-3, 130], 16, dtype, io, heads, seed=2).run()
    c.lengths = np.array([0, 130])
    c.check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("bad", [-1, 1 << 30, -(1 << 31)])
def test_pages_outside_the_pool_read_as_zeros(cuda_lib, dtype, io, heads, bad):
    mla = cuda_lib
    page = 32
    c = Call(mla, [200, 130], page, dtype, io, heads, seed=3)
    c.dev["table"][0, 2] = bad
    # the oracle reads a page of zeros there
    zero = torch.zeros((1,) + tuple(c.pool.shape[1:])).to(c.pool.dtype)
    c.pool = torch.cat([c.pool, zero])
    c.table[0, 2] = c.pool.shape[0] - 1
    c.run().check(status=mla.MLA_DEV_PAGE_OUT_OF_RANGE)


@pytest.mark.parametrize("dtype,io,heads", [("bf16", F32, 16), ("bf16", F32, 32), ("fp8", F32, 16)])
def test_paged_equals_dense(cuda_lib, dtype, io, heads):
    """With fp32 queries the paged call gives the dense call's bits when the chunks are
    the same."""
    mla = cuda_lib
    page, S, B = 64, 512, 3
    c = Call(mla, [512, 300, 77], page, dtype, io, heads, splits=2, seed=4, s_max=S).run()
    flat = c.pool.view(torch.uint8).reshape(c.pages, page, -1)
    dense = torch.zeros((B, S, flat.shape[2]), dtype=torch.uint8)
    for b, n in enumerate(c.lengths):
        for j in range(-(-int(n) // page)):
            dense[b, j * page:(j + 1) * page] = flat[int(c.table[b, j])]
    cache = dense.view(DT[dtype]).view(B, S, 576).cuda()
    d = mla.dims(B, heads, S, mla.dtype_code(DT[dtype]))
    ws = torch.empty(mla.workspace_bytes(d, 2), dtype=torch.uint8, device="cuda")
    o = torch.empty((B, heads, D_C), device="cuda")
    lse = torch.empty((B, heads), device="cuda")
    mla.decode_attn(d, c.dev["q_abs"].float(), c.dev["q_pe"].float(), cache, c.dev["lengths"], o,
                    ws, SCALE, 2, lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(c.lse, lse)
    assert torch.equal(c.o, o.to(io))


@pytest.mark.parametrize("dtype,io,heads", [("bf16", BF16, 16), ("bf16", BF16, 64), ("fp8", BF16, 16),
                                            ("f32", F32, 3), ("bf16", BF16, 128), ("fp8", BF16, 128)])
def test_same_bits_each_time_and_from_a_graph(cuda_lib, dtype, io, heads):
    """Two runs, a side stream and two graphs that share a workspace give the same bits."""
    c = Call(cuda_lib, [1000, 257, 40], 16, dtype, io, heads, seed=5).run()
    torch.cuda.synchronize()
    first, lse = c.o.clone(), c.lse.clone()

    def same():
        torch.cuda.synchronize()
        assert torch.equal(c.o, first) and torch.equal(c.lse, lse)
        c.o.fill_(3)
        c.lse.fill_(3)
        c.ws.fill_(0xFF)
        torch.cuda.synchronize()

    same()
    c.run()
    same()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run()
    same()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
        same()
    # new lengths in place: the captured call reads them
    c.dev["lengths"].copy_(i32([900, 20, 40]))
    c.lengths = np.array([900, 20, 40])
    graphs[0].replay()
    c.check()


def test_rows_of_other_sequences_are_left_alone(cuda_lib):
    """Outputs behind the last token keep what they held."""
    mla = cuda_lib
    c = Call(mla, [100, 30], 16, "bf16", BF16, 16, seed=6)
    o = torch.full((5, 16, D_C), 3.0, dtype=BF16, device="cuda")
    lse = torch.full((5, 16), 3.0, device="cuda")
    c.o, c.lse = o[:2], lse[:2]
    c.run().check()
    assert (o[2:] == 3).all() and (lse[2:] == 3).all()


def test_shared_pages(cuda_lib):
    """Two sequences with a common prefix in the same pages."""
    c = Call(cuda_lib, [100, 100], 16, "bf16", F32, 16, seed=7)
    c.table[1, :4] = c.table[0, :4]
    c.dev["table"].copy_(c.table)
    c.run().check()


def test_pool_past_2_to_31_elements(cuda_lib):
    """Pages whose values lie beyond 2^31 elements of the pool's start."""
    mla = cuda_lib
    page, pages = 256, (1 << 31) // (256 * 576) + 40
    c = Call(mla, [300, 129], page, "bf16", BF16, 16, seed=8)
    big = torch.full((pages, page, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    top = pages - c.pages
    big[top:].copy_(c.dev["pool"])
    live = (c.table >= 0) & (c.table < c.pages)
    c.dev["table"] = torch.where(live, c.table + top, c.table).cuda()
    c.dev["pool"], c.pg = big, mla.paging(page, pages, c.table.shape[1])
    c.run().check()


def test_refuses_wrong_tensors(cuda_lib):
    mla = cuda_lib
    c = Call(mla, [100, 30], 16, "bf16", BF16, 16, seed=6)

    def with_(**kw):
        saved = dict(c.dev)
        c.dev.update(kw)
        try:
            with pytest.raises(ValueError):
                c.run()
        finally:
            c.dev = saved

    with_(pool=c.dev["pool"].cpu())
    with_(pool=c.dev["pool"].float())
    with_(pool=c.dev["pool"][1:])
    with_(q_abs=c.dev["q_abs"].float())
    with_(q_abs=c.dev["q_abs"][:, ::2])
    with_(table=c.dev["table"].long())
    with_(table=c.dev["table"][:, 1:])
    with_(lengths=c.dev["lengths"][:1])
    with_(lengths=c.dev["lengths"].repeat(2)[::2])
    c.ws = c.ws[:100]
    with pytest.raises(mla.MlaError):
        c.run()


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("size", [0.0, 1e-42, 1e-37, 1e-30])
def test_tiny_queries(cuda_lib, dtype, io, heads, size):
    """Queries of zeros, and of hardly anything with zeros among it: every row weighs the same."""
    c = Call(cuda_lib, [300, 17], 32, dtype, io, heads, seed=11)
    c.q_abs, c.q_pe = (c.q_abs.float() * size).to(io), (c.q_pe.float() * size).to(io)
    c.q_abs[:, :, ::3] = 0
    c.dev["q_abs"], c.dev["q_pe"] = c.q_abs.cuda(), c.q_pe.cuda()
    c.run().check()
