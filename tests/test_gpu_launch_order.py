"""Paged calls that follow one another without a synchronisation: each gives the bits it
gives alone, whatever the calls before it still have in flight."""
import numpy as np
import pytest
import torch

from _paged import D_C, D_R, DT, SCALE
from test_gpu_paged_attn import BF16, F32, KINDS, Call, i32
from test_gpu_sparse import Sparse

pytestmark = pytest.mark.gpu
ROUNDS = 12


def alone_and_together(calls, chain):
    """chain(k, round) queues call k and returns its outputs; each is held to what it gave
    alone."""
    alone = []
    for k in range(len(calls)):
        got = chain(k, ROUNDS)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in got])
    torch.cuda.synchronize()
    outs = [[chain(k, r) for k in range(len(calls))] for r in range(ROUNDS)]
    torch.cuda.synchronize()
    for row in outs:
        for got, want in zip(row, alone):
            assert all(torch.equal(g, w) for g, w in zip(got, want))


def absorb_inputs(seed, rows, heads):
    g = torch.Generator().manual_seed(seed)
    x = dict(q_nope=torch.randn((rows, heads, 128), generator=g).bfloat16().cuda(),
             q_rope=torch.randn((rows, heads, D_R), generator=g).bfloat16().cuda(),
             w_uk=(torch.randn((heads, 128, D_C), generator=g) * 0.02).bfloat16().cuda())
    return x, i32(np.arange(rows))


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_f32_calls_on_one_workspace(cuda_lib, splits):
    """fp32 caches, lengths that change from call to call, one chunk and several: partials
    and results of one call are not overwritten under the combine of another."""
    calls = [Call(cuda_lib, lengths, 16, "f32", F32, 16, splits=splits, seed=k, s_max=1000,
                  width=70)
             for k, lengths in enumerate(([1000, 7, 400, 33], [64, 900, 1, 512], [250] * 4))]
    for c in calls:
        c.ws = calls[0].ws
        c.outs = [(torch.full_like(c.o, 7), torch.full_like(c.lse, 7)) for _ in range(ROUNDS + 1)]

    def chain(k, r):
        calls[k].o, calls[k].lse = calls[k].outs[r]
        calls[k].run()
        return calls[k].outs[r]

    alone_and_together(calls, chain)
    for c in calls:
        c.o, c.lse = c.outs[0]
        c.check()
    # one output as well: the last call's result stands
    for _ in range(ROUNDS):
        for c in calls:
            c.o, c.lse = calls[0].outs[0]
            c.run()
    torch.cuda.synchronize()
    for got, want in zip(calls[0].outs[0], calls[-1].outs[ROUNDS]):
        assert torch.equal(got, want)


@pytest.mark.parametrize("splits", [1, 3])
def test_f32_call_behind_the_absorb(cuda_lib, splits):
    """The queries come from mla_absorb_q, which lets its successor start at once."""
    mla = cuda_lib
    B, H = 24, 16
    calls = [Call(mla, np.random.RandomState(k).randint(1, 300, B), 16, "f32", F32, H, splits=splits,
                  seed=k, s_max=300, width=30) for k in range(3)]
    d = mla.dims(B, H, 300, mla.MLA_BF16)
    x = [absorb_inputs(k, B, H) for k in range(3)]

    def chain(k, r):
        c = calls[k]
        ins, pos = x[k]
        c.ws = calls[0].ws
        c.dev["q_abs"], c.dev["q_pe"] = calls[0].dev["q_abs"], calls[0].dev["q_pe"]
        c.o, c.lse = torch.full_like(c.o, 7), torch.full_like(c.lse, 7)
        mla.absorb_q(d, ins["q_nope"], ins["q_rope"], ins["w_uk"], pos, c.dev["q_abs"],
                     c.dev["q_pe"])
        c.run()
        return c.o, c.lse

    alone_and_together(calls, chain)


SHORT = [("bf16", F32, 16), ("bf16", F32, 64), ("bf16", BF16, 16), ("bf16", BF16, 64),
         ("fp8", F32, 16), ("fp8", BF16, 32), ("fp8", BF16, 128), ("f32", F32, 4)]


def short_sparse(mla, k, dtype, io, heads, long, B=20, page=16, top=6):
    """A sparse call whose s_max spans 40 pages, over sequences of at most `top` pages
    (`long`: all but one)."""
    c = Sparse(mla, [40 * page] * B, page, dtype, io, heads, top, seed=k)
    c.lengths = np.random.RandomState(k).randint(1, page * top + 1, B)
    if long:
        c.lengths[k] = 39 * page + 3
    c.dev["lengths"].copy_(i32(c.lengths))
    c.outs = [(torch.full_like(c.o, 7), torch.full_like(c.lse, 7)) for _ in range(ROUNDS + 1)]
    return c


@pytest.mark.parametrize("dtype,io,heads", SHORT)
@pytest.mark.parametrize("long", [False, True])
def test_sparse_calls_on_short_sequences(cuda_lib, dtype, io, heads, long):
    """No sequence holds more pages than are kept (or one alone does), so that the score
    kernel has nothing to do: calls with other queries and lengths on one workspace and one
    selection."""
    calls = [short_sparse(cuda_lib, k, dtype, io, heads, long) for k in range(3)]
    for c in calls:
        c.ws, c.sel, c.sel_len = calls[0].ws, calls[0].sel, calls[0].sel_len

    def chain(k, r):
        c = calls[k]
        c.o, c.lse = c.outs[r]
        c.run()
        return c.outs[r]

    alone_and_together(calls, chain)
    for c in calls:
        c.o, c.lse = c.outs[0]
        c.run().check()


@pytest.mark.parametrize("dtype,heads", [("bf16", 16), ("bf16", 64), ("fp8", 16)])
@pytest.mark.parametrize("long", [False, True])
def test_absorb_sparse_out_proj(cuda_lib, dtype, heads, long):
    """The library's own chain: queries of mla_absorb_q, which lets its successor start at
    once, a sparse call on short sequences, and mla_out_proj."""
    mla, B = cuda_lib, 40
    calls = [short_sparse(mla, k, dtype, F32, heads, long, B) for k in range(3)]
    x = [absorb_inputs(k, B, heads) for k in range(3)]
    w_uv = (torch.randn((heads, 128, D_C), generator=torch.Generator().manual_seed(9)) * 0.04
            ).bfloat16().cuda()
    outs = [[torch.full((B, heads, 128), 7.0, device="cuda") for _ in range(ROUNDS + 1)]
            for _ in calls]
    one = calls[0]

    def chain(k, r):
        c, (ins, pos) = calls[k], x[k]
        c.ws, c.sel, c.sel_len, c.o, c.lse = one.ws, one.sel, one.sel_len, one.o, one.lse
        c.dev["q_abs"], c.dev["q_pe"] = one.dev["q_abs"], one.dev["q_pe"]
        mla.absorb_q(c.d, ins["q_nope"], ins["q_rope"], ins["w_uk"], pos, c.dev["q_abs"],
                     c.dev["q_pe"])
        c.run()
        mla.out_proj(c.d, c.o, w_uv, outs[k][r])
        return (outs[k][r],)

    alone_and_together(calls, chain)
    for k, c in enumerate(calls):
        chain(k, 0)
        torch.cuda.synchronize()
        c.q_abs, c.q_pe = c.dev["q_abs"].cpu(), c.dev["q_pe"].cpu()
        c.check()


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("form,splits", [(0, 1), (0, 3), (1, 0)])
def test_a_call_without_any_row(cuda_lib, dtype, io, heads, form, splits):
    """Every sequence empty, as in a batch of nothing but padding, between two calls with rows
    on the same workspace and outputs: it gives zeros and -inf, and the others what they give
    alone."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(form)
    try:
        calls = [Call(mla, [600, 40, 300], 16, dtype, io, heads, splits=splits, seed=k, s_max=600,
                      width=40) for k in range(2)]
        none = Call(mla, [0, 0, 0], 16, dtype, io, heads, splits=splits, seed=2, s_max=600, width=40)
        alone = []
        for c in calls + [none]:
            c.ws, c.o, c.lse = calls[0].ws, calls[0].o, calls[0].lse
            c.run()
            torch.cuda.synchronize()
            alone.append((c.o.clone(), c.lse.clone()))
        assert (alone[2][0] == 0).all() and torch.isneginf(alone[2][1]).all()
        kept = []
        for _ in range(ROUNDS):
            for c in (calls[0], none, calls[1]):
                c.run()
            kept.append((calls[0].o.clone(), calls[0].lse.clone()))
            none.run()
        torch.cuda.synchronize()
        for o, lse in kept:
            assert torch.equal(o, alone[1][0]) and torch.equal(lse, alone[1][1])
        assert (none.o == 0).all() and torch.isneginf(none.lse).all()
        assert int(none.status.item()) == mla.MLA_DEV_LENGTH_OUT_OF_RANGE
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("dtype,heads", [("bf16", 16), ("bf16", 32), ("fp8", 16)])
def test_decode_steps_over_pages(cuda_lib, dtype, heads):
    """Decode steps as a server runs them, none synchronised: pages, the new rows, queries of
    mla_absorb_q, attention over the pages, mla_out_proj.  The same bits as the dense calls
    over the rows that the pages hold."""
    mla, B, page, S, steps = cuda_lib, 6, 16, 512, 5
    rng = np.random.RandomState(heads)
    start = rng.randint(1, S - steps, B)
    start[:2] = [page * 3, S - steps]
    pages, width = B * (S // page) + 3, S // page
    pg, d = mla.paging(page, pages, width), mla.dims(B, heads, S, mla.dtype_code(DT[dtype]))
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, nf, lengths, starts, status = i32(rng.permutation(pages)), i32([pages]), z(B), z(B + 1), z(1)
    pool = torch.full((pages, page, 576), float("nan")).to(DT[dtype]).cuda()
    T = int(start.sum())
    slots, pos = z(T, dt=torch.int64), z(T)
    mla.pages_extend(pg, lengths, i32(start), table, free, nf, lengths, starts, slots, pos,
                     dev_status=status)
    mla.cache_append_paged(d, pg, torch.from_numpy(rng.randn(T, 576)).bfloat16().cuda(), pos, slots,
                           pool, dev_status=status)
    ws = z(max(mla.paged_workspace_bytes(d, pg, F32, 1, 2), mla.workspace_bytes(d, 2)), dt=torch.uint8)
    q_abs, q_pe, o = z(B, heads, D_C, dt=F32), z(B, heads, D_R, dt=F32), z(B, heads, D_C, dt=F32)
    w_uv = torch.from_numpy(rng.randn(heads, 128, D_C) * 0.04).bfloat16().cuda()
    x = [absorb_inputs(k, B, heads)[0] for k in range(steps)]
    rows = [torch.from_numpy(rng.randn(B, 576)).bfloat16().cuda() for _ in range(steps)]
    one, slot, at = torch.ones(B, dtype=torch.int32, device="cuda"), z(B, dt=torch.int64), z(B)
    outs, kept = [z(B, heads, 128, dt=F32) for _ in range(2 * steps)], []
    torch.cuda.synchronize()
    for k in range(steps):
        mla.pages_extend(pg, lengths, one, table, free, nf, lengths, starts, slot, at,
                         dev_status=status)
        mla.cache_append_paged(d, pg, rows[k], at, slot, pool, dev_status=status)
        mla.absorb_q(d, x[k]["q_nope"], x[k]["q_rope"], x[k]["w_uk"], at, q_abs, q_pe)
        mla.decode_attn_paged(d, pg, q_abs, q_pe, pool, table, lengths, o, ws, SCALE,
                              num_splits_requested=2, dev_status=status)
        mla.out_proj(d, o, w_uv, outs[k])
        kept.append((table.clone(), lengths.clone(), at.clone()))
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lengths.cpu().tolist() == (start + steps).tolist()
    flat = pool.view(torch.uint8).view(pages, -1)
    for k, (tab, n, p) in enumerate(kept):
        cache = torch.zeros((B, width, flat.shape[1]), dtype=torch.uint8, device="cuda")
        live = tab >= 0
        cache[live] = flat[tab[live].long()]
        mla.absorb_q(d, x[k]["q_nope"], x[k]["q_rope"], x[k]["w_uk"], p, q_abs, q_pe)
        mla.decode_attn(d, q_abs, q_pe, cache.view(DT[dtype]).view(B, S, 576), n, o, ws, SCALE, 2)
        mla.out_proj(d, o, w_uv, outs[steps + k])
        torch.cuda.synchronize()
        assert torch.isfinite(outs[k]).all() and torch.equal(outs[k], outs[steps + k])


def test_calls_at_once_on_two_streams(cuda_lib):
    """Different calls on two streams, each with its own workspace and outputs, at the same
    time: the bits they give alone."""
    left = [Call(cuda_lib, [900, 300, 41] * 8, 16, dtype, io, heads, seed=k)
            for k, (dtype, io, heads) in enumerate([("fp8", BF16, 128), ("bf16", BF16, 16),
                                                    ("bf16", BF16, 64), ("f32", F32, 5)])]
    right = [short_sparse(cuda_lib, k, dtype, io, heads, True)
             for k, (dtype, io, heads) in enumerate([("bf16", BF16, 16), ("fp8", BF16, 128),
                                                     ("fp8", F32, 16), ("bf16", F32, 32)])]
    alone = []
    for c in left + right:
        c.run()
        torch.cuda.synchronize()
        alone.append((c.o.clone(), c.lse.clone()))
        c.o.fill_(7), c.lse.fill_(7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for pair in zip(left, right):
            for stream, c in zip(streams, pair):
                with torch.cuda.stream(stream):
                    c.run()
    torch.cuda.synchronize()
    for c, (o, lse) in zip(left + right, alone):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse) and int(c.status.item()) == 0
