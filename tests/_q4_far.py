"""4-bit pools whose scores are chosen, for tests of scores that lie far apart."""
from __future__ import annotations

import numpy as np
import torch

import _q4
from _paged import D_C, D_R, ROW, SCALE
from oracle import fp4_oracle as F

F32, BF16 = torch.float32, torch.bfloat16
TILE = 128                                     # rows that the kernels take together


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def shift_unit(q0):
    """What a key's first value of 1 adds to a score where the query's is q0."""
    return SCALE * q0


class Far:
    """One decode_attn_paged problem over a 4-bit pool whose rows are given: sequence after
    sequence, latents [n, 512] (as the pool will round them) and keys [n, 64]."""

    def __init__(self, mla, latents, keys, q_abs, q_pe, page, io, q_len=1, splits=0, s_max=None):
        rng = np.random.RandomState(len(latents))
        self.mla, self.page, self.io, self.q_len, self.splits = mla, page, io, q_len, splits
        self.lengths = np.array([len(x) for x in latents])
        need = -(-self.lengths // page)
        pages = int(need.sum()) + 1
        ids = rng.permutation(pages)
        self.table = np.full((len(latents), int(need.max()) + 1), -1)
        x = np.zeros((pages, page, ROW), np.float32)
        k = 0
        for b, n in enumerate(need):
            mine = ids[k:k + n]
            self.table[b, :n] = mine
            k += n
            rows = np.zeros((n * page, ROW), np.float32)
            rows[:self.lengths[b], :D_C], rows[:self.lengths[b], D_C:] = latents[b], keys[b]
            x[mine] = rows.reshape(n, page, ROW)
        e = F.exponents(x[..., :D_C])
        self.pool = torch.from_numpy(F.pack(F.codes(x[..., :D_C], e), e, _q4.bf16_bits(x[..., D_C:])))
        self.q_abs, self.q_pe = q_abs.to(io), q_pe.to(io)
        heads = q_abs.shape[1]
        self.d = mla.dims(len(latents), heads, s_max or int(self.lengths.max()), mla.MLA_FP4_E2M1)
        self.pg = mla.paging(page, pages, self.table.shape[1])
        self.ws = torch.empty(mla.paged_workspace_bytes(self.d, self.pg, io, q_len, splits),
                              dtype=torch.uint8, device="cuda")
        self.o = torch.full((len(latents) * q_len, heads, D_C), 7.0, dtype=io, device="cuda")
        self.lse = torch.full((len(latents) * q_len, heads), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dev = dict(q_abs=self.q_abs.cuda(), q_pe=self.q_pe.cuda(), pool=self.pool.cuda(),
                        table=i32(self.table), lengths=i32(self.lengths))

    def run(self):
        x = self.dev
        self.mla.decode_attn_paged(self.d, self.pg, x["q_abs"], x["q_pe"], x["pool"], x["table"],
                                   x["lengths"], self.o, self.ws, SCALE, q_len=self.q_len,
                                   num_splits_requested=self.splits, lse=self.lse,
                                   dev_status=self.status)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        return self

    def check(self, tokens=None):
        return _q4.check_attention(self.o, self.lse, self.q_abs, self.q_pe, self.pool, self.page,
                                   torch.from_numpy(self.table), self.lengths, self.q_len, self.io,
                                   tokens)


def shifted(rng, mla, shifts, heads, io, q_len=1, page=64, splits=0, **kw):
    """Random rows and queries, row t of sequence b with shifts[b][t] added to every score (and
    what bf16 rounds off it: the key holds it)."""
    q0 = 16.0
    latents, keys = [], []
    for s in shifts:
        latents.append(rng.randn(len(s), D_C).astype(np.float32))
        key = rng.randn(len(s), D_R).astype(np.float32)
        key[:, 0] = np.asarray(s) / shift_unit(q0)
        keys.append(key)
    rows = len(shifts) * q_len
    q_abs = torch.from_numpy((rng.randn(rows, heads, D_C) * 0.3).astype(np.float32))
    q_pe = torch.from_numpy(rng.randn(rows, heads, D_R).astype(np.float32))
    q_pe[:, :, 0] = q0
    return Far(mla, latents, keys, q_abs, q_pe, page, io, q_len, splits, **kw)
