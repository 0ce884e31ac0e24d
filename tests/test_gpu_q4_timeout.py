"""The 4-bit split kernels' bounded waits, made to run out on purpose without a fault.

As for the bf16 kernel (test_gpu_timeout.py): a test hook shortens every bounded wait to a few
milliseconds and stops the copies of codes after a CTA's first tile, so that its decoding, score,
softmax and output warps wait for rows that are never asked for.  The kernels must return on their
own, report MLA_DEV_PIPELINE_TIMEOUT, write no result, and leave the context usable: the next call
with the hooks reset is right.
"""
import numpy as np
import pytest
import torch

from _q4_far import BF16, F32, shifted

pytestmark = pytest.mark.gpu


def run_out(mla, c, tiles=1):
    lib, x = mla.load(), c.dev
    torch.cuda.synchronize()
    try:
        lib.mla_test_set_split_hooks(5_000_000, tiles)      # 5 ms waits
        mla.decode_attn_paged(c.d, c.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"], x["lengths"],
                              c.o, c.ws, 192 ** -0.5, q_len=c.q_len, num_splits_requested=c.splits,
                              lse=c.lse, dev_status=c.status)
    finally:
        lib.mla_test_set_split_hooks(0, 0)
    torch.cuda.synchronize()                                # the kernels returned by themselves
    assert int(c.status.item()) & mla.MLA_DEV_PIPELINE_TIMEOUT
    c.status.zero_()


@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 48), (BF16, 128)])
@pytest.mark.parametrize("q_len", [1, 2])
@pytest.mark.parametrize("tiles", [1, 3])
def test_waits_run_out_in_chunks(cuda_lib, io, heads, q_len, tiles):
    """One chunk of five tiles a sequence, whose result the kernel writes itself: it writes none."""
    rng = np.random.RandomState(heads)
    c = shifted(rng, cuda_lib, [np.zeros(640), np.zeros(600)], heads, io, q_len, splits=1)
    run_out(cuda_lib, c, tiles)
    assert bool((c.o == 7).all()) and bool((c.lse == 7).all())
    c.run().check()


@pytest.mark.parametrize("io,heads", [(BF16, 16), (F32, 16), (BF16, 64), (BF16, 128)])
def test_waits_run_out_in_shares(cuda_lib, io, heads):
    """Equal shares of several tiles and sequences a CTA, then the same call as it should be."""
    mla = cuda_lib
    mla.load().mla_test_set_split_form(1)
    try:
        rng = np.random.RandomState(heads)
        c = shifted(rng, mla, [np.zeros(n) for n in rng.randint(1, 1300, 80)], heads, io)
        run_out(mla, c)
        c.run().check(tokens=[0, 1, 40, 79])
    finally:
        mla.load().mla_test_set_split_form(0)
