"""Corners of the paged calls: lengths below the tokens of a step, more chunks than tiles,
large batches, every kind with several tokens in the sparse call."""
import numpy as np
import pytest
import torch

from _paged import D_C, DT, SCALE
from test_gpu_paged_attn import BF16, F32, KINDS, Call
from test_gpu_sparse import Sparse

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("form,splits,q_len", [(0, 0, 2), (0, 3, 4), (1, 0, 3), (1, 0, 4)])
def test_lengths_below_the_tokens(cuda_lib, dtype, io, heads, form, splits, q_len):
    """A sequence with fewer rows than new tokens: its first tokens see nothing, and the
    status says so."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(form)
    try:
        c = Call(mla, [1, 300, 0, q_len - 1, q_len], 16, dtype, io, heads, q_len=q_len,
                 splits=splits, seed=q_len)
        c.run().check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("dtype,io,heads", KINDS)
def test_more_chunks_than_tiles(cuda_lib, dtype, io, heads):
    Call(cuda_lib, [700, 129, 1, 513], 64, dtype, io, heads, splits=1000, seed=1).run().check()


@pytest.mark.parametrize("dtype,io,heads", [("f32", F32, 1), ("bf16", F32, 16), ("bf16", BF16, 16),
                                            ("bf16", BF16, 32), ("fp8", BF16, 16),
                                            ("fp8", BF16, 48)])
def test_large_batch(cuda_lib, dtype, io, heads):
    """Thousands of short sequences."""
    rng = np.random.RandomState(1)
    c = Call(cuda_lib, rng.randint(1, 40, 5003), 16, dtype, io, heads, seed=2)
    c.run().check(tokens=list(range(0, 5003, 419)) + [5002])


@pytest.mark.parametrize("dtype,io,heads", [("f32", F32, 5), ("bf16", F32, 16), ("bf16", BF16, 64),
                                            ("bf16", F32, 64), ("fp8", F32, 16), ("fp8", BF16, 32),
                                            ("fp8", BF16, 128)])
@pytest.mark.parametrize("q_len", [2, 3])
def test_sparse_tokens_of_every_kind(cuda_lib, dtype, io, heads, q_len):
    """Several tokens, some of a sequence that keep every page and some that choose, also
    with lengths below the tokens."""
    mla, page, top = cuda_lib, 16, 5
    lengths = [page * top + 1, page * 33, q_len, page * top + q_len]
    Sparse(mla, lengths, page, dtype, io, heads, top, q_len=q_len, seed=q_len).run().check()
    s = Sparse(mla, [1, page * 20, q_len - 1], page, dtype, io, heads, top, q_len=q_len, seed=q_len)
    s.run().check(status=mla.MLA_DEV_LENGTH_OUT_OF_RANGE)


@pytest.mark.parametrize("dtype,io,heads", [("bf16", BF16, 16), ("fp8", BF16, 128), ("f32", F32, 3)])
def test_sparse_in_a_barely_aligned_workspace(cuda_lib, dtype, io, heads):
    s = Sparse(cuda_lib, [16 * 30 + 1, 16 * 9], 16, dtype, io, heads, 4, seed=3)
    s.ws = torch.empty(s.ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:]
    o = torch.full((4, heads, D_C), 3.0, dtype=io, device="cuda")
    s.o = o[:2]
    s.run().check()
    assert (o[2:] == 3).all()


def poison_row(call, b, t, value):
    """Row t of sequence b of a call's pool on the GPU becomes `value` (E4M3: NaN) in every
    third column, the RoPE key's among them."""
    pool, page = call.dev["pool"], call.pg.page_size
    at = int(call.table[b, t // page])
    if call.dtype == "fp8":
        pool.view(torch.uint8)[at, t % page, ::3] = 0x7F
    else:
        pool[at, t % page, ::3] = value


@pytest.mark.parametrize("dtype,io,heads", KINDS)
@pytest.mark.parametrize("form,q_len", [(0, 2), (1, 2), (0, 3), (1, 4)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_later_tokens_row_is_not_seen(cuda_lib, dtype, io, heads, form, q_len, value):
    """Rows that the last token of a step attends and the tokens before it do not: NaN and
    infinities there do not reach the earlier tokens, wherever in a tile the rows lie."""
    mla = cuda_lib
    lengths = [127, 128, 129, 130, 256, 300, 257 + q_len, q_len, 5]
    mla.load().mla_test_set_split_form(form)
    try:
        c = Call(mla, lengths, 16, dtype, io, heads, q_len=q_len, seed=q_len)
        for b, n in enumerate(lengths):
            poison_row(c, b, n - 1, value)
        c.run().check(tokens=[r for r in range(len(lengths) * q_len) if r % q_len < q_len - 1])
        last = c.o.view(len(lengths), q_len, heads, D_C)[:, -1].float()
        assert not torch.isfinite(last).any()
        # every row of the step but the first token's
        c = Call(mla, lengths, 16, dtype, io, heads, q_len=q_len, seed=q_len)
        for b, n in enumerate(lengths):
            for t in range(n - q_len + 1, n):
                poison_row(c, b, t, value)
        c.run().check(tokens=range(0, len(lengths) * q_len, q_len))
    finally:
        mla.load().mla_test_set_split_form(0)


@pytest.mark.parametrize("dtype,heads", [("f32", 5), ("bf16", 16), ("bf16", 32), ("bf16", 48),
                                         ("bf16", 64), ("fp8", 16)])
@pytest.mark.parametrize("q_len,splits", [(2, 0), (2, 3), (3, 0), (4, 0)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_later_tokens_row_is_not_seen_dense(cuda_lib, dtype, heads, q_len, splits, value):
    """The same over a dense cache: the earlier tokens' bits are those over finite rows."""
    mla, S = cuda_lib, 600
    lengths = [127, 128, 129, 130, 256, 300, 600, q_len]
    B = len(lengths)
    g = torch.Generator().manual_seed(q_len)
    cache = torch.randn((B, S, 576), generator=g).to(DT[dtype]).cuda()
    q_abs = (torch.randn((B * q_len, heads, D_C), generator=g) * 0.3).cuda()
    q_pe = torch.randn((B * q_len, heads, 64), generator=g).cuda()
    d = mla.dims(B, heads, S, mla.dtype_code(DT[dtype]))
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    ws = torch.empty(int(mla.load().mla_decode_multi_workspace_bytes(d, q_len, splits)),
                     dtype=torch.uint8, device="cuda")

    def run():
        o, lse = torch.empty_like(q_abs), torch.empty((B * q_len, heads), device="cuda")
        mla.decode_attn_multi(d, q_len, q_abs, q_pe, cache, n, o, ws, SCALE, splits, lse=lse)
        torch.cuda.synchronize()
        return o.view(B, q_len, heads, D_C), lse.view(B, q_len, heads)

    want, want_lse = run()
    for b, k in enumerate(lengths):
        if dtype == "fp8":
            cache.view(torch.uint8)[b, k - 1, ::3] = 0x7F
        else:
            cache[b, k - 1, ::3] = value
    got, lse = run()
    assert torch.equal(got[:, :-1], want[:, :-1]) and torch.equal(lse[:, :-1], want_lse[:, :-1])
    assert not torch.isfinite(got[:, -1]).any()
