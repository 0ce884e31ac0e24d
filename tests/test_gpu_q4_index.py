"""The page index over 4-bit pools where a call could touch very many pages."""
import numpy as np
import pytest
import torch

import _q4
from _paged import ROW
from _q4_far import i32
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width", [(5, 8), (150, 8), (152, 8), (153, 8), (300, 40), (1, 3000)])
def test_items_for_one_cta_each_and_walked(cuda_lib, B, width):
    """Few and many pages that could be touched, around the number from which CTAs walk them, some
    touched from a later row on and some not at all."""
    mla = cuda_lib
    rng = np.random.RandomState(B + width)
    page = 16
    lengths = rng.randint(0, width * page + 1, B) if B < 300 else rng.randint(0, 3 * page, B)
    first = np.minimum(lengths, rng.randint(0, width * page, B))
    first[::3] = np.maximum(lengths[::3] - 1, 0)
    pool, table, pages = _q4.make_pool(rng, lengths, page, width=width)
    val = _q4.values(pool.numpy(), page)
    d, pg = mla.dims(B, 16, width * page, mla.MLA_FP4_E2M1), mla.paging(page, pages, width)
    codes = torch.full((pages, ROW), 77, dtype=torch.int8, device="cuda")
    scales, status = torch.full((pages,), 7.0, device="cuda"), i32([0])
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
