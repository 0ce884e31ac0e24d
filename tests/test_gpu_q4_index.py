"""The page index over 4-bit pools where a call could touch very many pages."""
import numpy as np
import pytest
import torch

import _q4
from _paged import ROW
from _q4_far import i32
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


def test_more_pages_than_2_to_31(cuda_lib):
    """Requests times pages of a request's row of the table pass 2^31 (the table itself 8 GB)."""
    mla = cuda_lib
    rng = np.random.RandomState(0)
    page, B, width = 16, 65536, 32769
    assert B * width > 1 << 31
    pool, _, pages = _q4.make_pool(rng, [64], page, extra_pages=0)
    val = _q4.values(pool.numpy(), page)
    d, pg = mla.dims(B, 16, 1, mla.MLA_FP4_E2M1), mla.paging(page, pages, width)
    table = torch.full((B, width), -7, dtype=torch.int32, device="cuda")
    lengths, first = np.zeros(B, np.int64), np.zeros(B, np.int64)
    want = {}
    for b, j, rows, i in ((0, 0, 5, 2), (40001, width - 1, 16, 0), (B - 1, 7, 9, 3), (B - 1, 8, 1, 1)):
        table[b, j] = i
        first[b] = min(j * page, first[b] or 1 << 60)
        lengths[b] = j * page + rows
        want[i] = rows
    want[3] = page                                  # a page with another behind it is whole
    codes = torch.full((pages, ROW), 77, dtype=torch.int8, device="cuda")
    scales, status = torch.full((pages,), 7.0, device="cuda"), i32([0])
    mla.page_index(d, pg, pool.cuda(), table, i32(first), i32(lengths), width * page, codes, scales,
                   dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for i, rows in want.items():
        c, s = PO.page_index(val[i][:rows])
        assert (codes[i].cpu().numpy() == c).all() and float(scales[i]) == s
