"""The paged latent cache's operators as a serving program calls them: what is measured.

Each case is one call (``op``) at one size:

- ``extend``: block tables and slot maps of one step, from the requests' lengths;
- ``append``: new latent rows written into their pages, the RoPE key rotated;
- ``attn``:   decode attention over the paged cache;
- ``index``:  the per-page index (int8 mean row and scale) of the pages a step touched;
- ``sparse``: pages chosen by the index's score, then attention over the chosen pages.

With ``own`` false, ``run`` computes the operator in its plain form with elementary
torch operations; with ``own`` true it makes the library's call.  Lengths are spread
evenly over [lo, hi] and dealt to the sequences by the seed, so that the work of a
case is known from its sizes alone.
"""
import math

import numpy as np
import torch

own = False

D_C, D_R = 512, 64
ROW = D_C + D_R
SCALE = (128 + 64) ** -0.5
BASE = 10000.0
TINY = 1e-30                     # below this largest magnitude an index row or a query counts as zero
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


def listed():
    return [
        # one decode step's tables: 64 requests, one token each
        dict(name="extend_decode_b64", op="extend", batch=64, lo=512, hi=8192, new_lo=1, new_hi=1,
             page=64),
        # prompts of many requests admitted at once, some of them continuing a cached prefix
        dict(name="extend_prefill_b256", op="extend", batch=256, lo=0, hi=8192, new_lo=0,
             new_hi=2047, page=64),
        # one decode step's new rows
        dict(name="append_decode_b8_bf16", op="append", batch=8, lo=4000, hi=4095, new=1, page=64,
             dtype="bf16"),
        # prompts' rows, rounded into an E4M3 cache (61 x 1021 tokens: odd on purpose)
        dict(name="append_prefill_b61_fp8", op="append", batch=61, lo=0, hi=3000, new=1021, page=64,
             dtype="fp8"),
        # the smallest decode call: one short sequence, everything fp32
        dict(name="attn_f32_b1_s64", op="attn", batch=1, heads=16, lo=64, hi=64, page=16,
             dtype="f32", q_len=1),
        # an ordinary decode step of a small server
        dict(name="attn_bf16_b8_s4096", op="attn", batch=8, heads=16, lo=4096, hi=4096, page=64,
             dtype="bf16", q_len=1),
        # many requests of very different lengths over an E4M3 cache
        dict(name="attn_fp8_b64_ragged", op="attn", batch=64, heads=16, lo=512, hi=8192, page=64,
             dtype="fp8", q_len=1),
        # a large model's decode step: 128 heads share every cached row
        dict(name="attn_bf16_h128_b32_s16384", op="attn", batch=32, heads=128, lo=16384, hi=16384,
             page=64, dtype="bf16", q_len=1),
        # a decode step's index update: the one page each request wrote to
        dict(name="index_decode_b64_bf16", op="index", batch=64, lo=512, hi=8192, new=1, page=64,
             dtype="bf16"),
        # the index of long prompts
        dict(name="index_prefill_b4_s65536", op="index", batch=4, lo=65536, hi=65536, new=65536,
             page=64, dtype="bf16"),
        # long contexts decoded over 2048 chosen rows each
        dict(name="sparse_bf16_b4_s65536", op="sparse", batch=4, heads=16, lo=65536, hi=65536,
             page=64, dtype="bf16", q_len=1, top=32),
        # a large model's decode step over 2048 chosen rows of an E4M3 cache
        dict(name="sparse_fp8_h128_b32", op="sparse", batch=32, heads=128, lo=9000, hi=16384,
             page=64, dtype="fp8", q_len=1, top=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "append", "attn", "attn", "attn", "index", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 64, 128])
    if op == "extend":
        new_hi = rng.choice([1, _log(rng, 2, 2047)])
        return dict(op=op, batch=_log(rng, 1, 256), lo=0, hi=_log(rng, 1, 8192),
                    new_lo=1 if new_hi == 1 else 0, new_hi=new_hi, page=page)
    dtype = rng.choice(["f32", "bf16", "bf16", "fp8"])
    if op in ("append", "index"):
        new = _log(rng, 1, 1024)
        return dict(op=op, batch=_log(rng, 1, 60), lo=new if op == "index" else 0,
                    hi=new + _log(rng, 1, 3000), new=new, page=page, dtype=dtype)
    q_len = rng.choice([1, 1, 1, 2, 3, 4])
    if dtype == "f32":                                  # the small exact path
        batch, heads, hi = _log(rng, 1, 8), rng.choice([1, 5, 16]), _log(rng, 64, 2000)
    else:
        heads = rng.choice([16, 16, 32, 48, 64, 128])
        batch = _log(rng, 1, 64 if heads <= 32 else 16)
        hi = _log(rng, 100, min(65536, 400000 // (batch * q_len)))
    lo = rng.randint(q_len, hi)
    c = dict(op=op, batch=batch, heads=heads, lo=lo, hi=hi, page=page, dtype=dtype, q_len=q_len)
    if op == "sparse":
        c["top"] = rng.choice([4, 9, 16, 32])
    return c


# --------------------------------------------------------------------------- inputs

def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], both ends among them."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64) if n > 1 else np.array([hi])


def _lengths(case):
    return _spread(case["lo"], case["hi"], case["batch"])


def _pages(n, page):
    return -(-n // page)


def _pool(g, num_pages, page, dtype):
    """Latent rows; rows of one page resemble one another, as neighbouring tokens do."""
    x = torch.randn((num_pages, page, ROW), generator=g, device="cuda").mul_(0.8)
    x.add_(torch.randn((num_pages, 1, ROW), generator=g, device="cuda"), alpha=0.6)
    return x.to(DTYPES[dtype])


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    B, page, op = case["batch"], case["page"], case["op"]
    s = {"case": case, "op": op, "page": page}
    order = r.permutation(B)
    if op == "extend":
        cached = _lengths(case)[order]
        new = _spread(case["new_lo"], case["new_hi"], B)[r.permutation(B)]
        have = _pages(cached, page)
        width = int(_pages(case["hi"] + case["new_hi"], page))
        num_pages = int(_pages(_lengths(case), page).sum()) + B * (_pages(case["new_hi"], page) + 1) + 5
        ids = r.permutation(num_pages)
        table = np.full((B, width), -1)
        n = 0
        for b in range(B):
            table[b, :have[b]] = ids[n:n + have[b]]
            n += have[b]
        free = np.zeros(num_pages, np.int64)
        free[:num_pages - n] = ids[n:]
        T = int(_spread(case["new_lo"], case["new_hi"], B).sum()) + 3      # room for a few more
        dev = torch.device("cuda")
        s.update(cached=_i32(cached), new=_i32(new), table=_i32(table), free=_i32(free),
                 num_free=_i32([num_pages - n]), num_pages=num_pages,
                 num_free_out=torch.zeros(1, dtype=torch.int32, device=dev),
                 lengths=torch.zeros(B, dtype=torch.int32, device=dev),
                 row_starts=torch.zeros(B + 1, dtype=torch.int32, device=dev),
                 slots=torch.zeros(T, dtype=torch.int64, device=dev),
                 positions=torch.zeros(T, dtype=torch.int32, device=dev))
    else:
        grown = case.get("new", 0) if op == "append" else 0
        total = _lengths(case)[order] + grown
        n_pages = _pages(total, page)
        width = int(n_pages.max())
        num_pages = int(n_pages.sum()) + 7
        ids = r.permutation(num_pages)[:int(n_pages.sum())]
        table = np.full((B, width), -1)
        n = 0
        for b in range(B):
            table[b, :n_pages[b]] = ids[n:n + n_pages[b]]
            n += n_pages[b]
        s.update(cache=_pool(g, num_pages, page, case["dtype"]), table=_i32(table),
                 lengths=_i32(total), num_pages=num_pages)
    if op == "append":
        first = total - case["new"]
        pos = (first[:, None] + np.arange(case["new"])[None, :])
        slots = np.take_along_axis(table, pos // page, 1) * page + pos % page
        rows = torch.randn((pos.size, ROW), generator=g, device="cuda")
        s.update(rows=rows if case["dtype"] == "f32" else rows.bfloat16(),
                 positions=_i32(pos.reshape(-1)), slots=torch.as_tensor(slots.reshape(-1)).cuda())
    if op == "index":
        s.update(first=_i32(total - case["new"]), new=case["new"])
    if op in ("index", "sparse"):
        s.update(codes=torch.zeros((num_pages, ROW), dtype=torch.int8, device="cuda"),
                 scales=torch.zeros(num_pages, device="cuda"))
    if op in ("attn", "sparse"):
        H, R = case["heads"], B * case["q_len"]
        io = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        # the absorbed query of N(0, 1) queries and N(0, 0.02^2) weights, and a rotated query
        s.update(q_abs=(torch.randn((R, H, D_C), generator=g, device="cuda") * 0.226).to(io),
                 q_pe=torch.randn((R, H, D_R), generator=g, device="cuda").to(io),
                 o=torch.empty((R, H, D_C), dtype=io, device="cuda"),
                 lse=torch.empty((R, H), device="cuda"), q_len=case["q_len"])
    if op == "sparse":
        s["codes"], s["scales"] = _index(s["cache"], s["table"], torch.zeros_like(s["lengths"]),
                                         s["lengths"], s["codes"], s["scales"], page)
        s.update(sel=torch.empty((R, case["top"]), dtype=torch.int32, device="cuda"),
                 sel_len=torch.empty(R, dtype=torch.int32, device="cuda"), top=case["top"])
    if own:
        import head_latent_attention_absorbed_gb300 as mla
        s["pg"] = mla.paging(page, s["num_pages"], int(s["table"].shape[1]))
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op != "extend":
            s["d"] = mla.dims(B, case.get("heads", 16), int(total.max()),
                              mla.dtype_code(DTYPES[case["dtype"]]))
        if op == "attn":
            n = mla.paged_workspace_bytes(s["d"], s["pg"], s["q_abs"].dtype, case["q_len"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        if op == "sparse":
            n = mla.sparse_workspace_bytes(s["d"], s["pg"], s["q_abs"].dtype, case["top"],
                                           case["q_len"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms

def _extend(s):
    cached, new, p, table = s["cached"].long(), s["new"].long(), s["page"], s["table"]
    B, W = table.shape
    T, nf = s["slots"].shape[0], s["num_free"].long()
    have, want = (cached + p - 1) // p, (cached + new + p - 1) // p
    need_end, row_end = (want - have).cumsum(0), new.cumsum(0)
    ok = (need_end[-1] <= nf) & (want.max() <= W) & (row_end[-1] <= T)
    j = torch.arange(W, device=table.device)[None, :]
    take = ok & (j >= have[:, None]) & (j < want[:, None])
    at = nf - 1 - ((need_end - (want - have))[:, None] + j - have[:, None])
    table = torch.where(take, s["free"][at.clamp(0, s["free"].shape[0] - 1)], table)
    starts = torch.where(ok, torch.cat([row_end.new_zeros(1), row_end]), row_end.new_zeros(1))
    t = torch.arange(T, device=table.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(0, B - 1)
    pos = cached[b] + t - starts[b]
    live = t < starts[-1]
    page = table[b, (pos // p).clamp(0, W - 1)].long()
    slots = torch.where(live, page * p + pos % p, -1)
    pos = torch.where(live, pos, 0)
    lengths = torch.where(ok, cached + new, cached)
    left = torch.where(ok, nf - need_end[-1], nf)
    return [table, lengths.int(), starts.int(), slots, pos.int(), left.int()]


def _append(s):
    x = s["rows"].float()
    inv = BASE ** (-torch.arange(0, D_R, 2, device=x.device, dtype=torch.float64) / D_R)
    a = s["positions"].double()[:, None] * inv[None, :]
    c, n = a.cos().float(), a.sin().float()
    k = x[:, D_C:].unflatten(1, (D_R // 2, 2))
    k = torch.stack([k[..., 0] * c - k[..., 1] * n, k[..., 0] * n + k[..., 1] * c], -1)
    y = torch.cat([x[:, :D_C], k.flatten(1)], 1)
    cache = s["cache"]
    if cache.dtype == torch.float8_e4m3fn:
        y = y.clamp(-448.0, 448.0)
        # one-byte rows are placed as bytes
        cache.view(torch.uint8).view(-1, ROW)[s["slots"]] = y.to(cache.dtype).view(torch.uint8)
    else:
        cache.view(-1, ROW)[s["slots"]] = y.to(cache.dtype)
    return [cache]


def _gather(cache, table, rows):
    """The first `rows` rows of each sequence [B, rows, 576] in fp32."""
    page = cache.shape[1]
    t = torch.arange(rows, device=cache.device)
    slot = table[:, t // page].long().clamp(min=0) * page + t % page
    flat = cache.view(-1, ROW)
    if cache.dtype == torch.float8_e4m3fn:
        return flat.view(torch.uint8)[slot].view(cache.dtype).float()
    return flat[slot].float()


def _attend(q_abs, q_pe, cache, table, lengths, q_len):
    """Attention of q_len tokens per table row; q [R, H, .], R = table rows x q_len."""
    B, (R, H, _) = table.shape[0], q_abs.shape
    rows = table.shape[1] * cache.shape[1]
    c = _gather(cache, table, rows)
    q = torch.cat([q_abs.float(), q_pe.float()], 2).view(B, q_len * H, ROW)
    sc = torch.matmul(q, c.transpose(1, 2)).view(B, q_len, H, rows) * SCALE
    back = torch.arange(q_len - 1, -1, -1, device=c.device)
    live = lengths.long()[:, None] - back[None, :]
    dead = torch.arange(rows, device=c.device)[None, None, :] >= live[:, :, None]
    sc = sc.masked_fill(dead[:, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = (sc - m).exp()
    z = e.sum(-1, keepdim=True)
    o = torch.matmul((e / z).view(B, q_len * H, rows), c[:, :, :D_C])
    return [o.view(R, H, D_C).to(q_abs.dtype), (m + z.log()).view(R, H)]


def _index(cache, table, first, lengths, codes, scales, page):
    """Index rows of the pages that hold rows [first, length) of each sequence."""
    B, W = table.shape
    j = torch.arange(W, device=cache.device)[None, :]
    hit = (j >= first.long()[:, None] // page) & (j * page < lengths.long()[:, None])
    hit = hit & (first < lengths)[:, None]
    ids = table[hit].long()
    n = (lengths.long()[:, None] - j * page).clamp(0, page)[hit]
    x = (cache.view(torch.uint8).view(cache.shape[0], -1)[ids].view(cache.dtype)
         if cache.dtype == torch.float8_e4m3fn else cache[ids])
    x = x.view(-1, page, ROW).float()
    live = torch.arange(page, device=x.device)[None, :, None] < n[:, None, None]
    x = torch.where(live, x, 0.0)
    top = x.abs().amax((1, 2))
    unit = torch.frexp(top)[0] / top                       # 2^-e, top = mantissa 2^e: exact
    fixed = (x * (unit * 2.0 ** 20)[:, None, None]).round().long().sum(1)     # whole numbers
    peak = fixed.abs().amax(1)
    good = (top >= TINY) & (peak > 0)
    pf = peak.clamp(min=1).float()
    code = (fixed.float() * (127.0 / pf)[:, None]).round()
    scale = pf / 127.0 / n.float() * (2.0 ** -20 / unit)
    codes[ids] = torch.where(good[:, None], code, 0.0).to(torch.int8)
    scales[ids] = torch.where(good, scale, 0.0)
    return [codes, scales]


def _choose(q, codes, scales, table, lengths, page, top, q_len):
    """Chosen pages [R, top] (positions ascending, as page ids) and the rows they hold."""
    B, W = table.shape
    R, H = q.shape[:2]
    back = torch.arange(q_len - 1, -1, -1, device=q.device)
    live = (lengths.long()[:, None] - back[None, :]).clamp(min=0).view(R)
    P = (live + page - 1) // page
    big = q.abs().amax(2)
    ok = big >= TINY
    qc = (q * torch.where(ok, 127.0 / big, 0.0)[:, :, None]).round().double()
    a = torch.where(ok, big / 127.0, 0.0)
    ids = table.long().clamp(min=0)
    key = codes[ids].double()                                                  # [B, W, 576]
    dot = torch.matmul(qc.view(B, q_len * H, ROW), key.transpose(1, 2)).view(B, q_len, H, W)
    v = a.view(B, q_len, H, 1) * dot.float()
    score = (v.amax(2) * scales[ids][:, None, :]).view(R, W)
    j = torch.arange(W, device=q.device)[None, :]
    forced = (j < 1) | (j >= P[:, None] - 1)                                   # first and last page
    score = torch.where(forced, math.inf, score)
    score = torch.where(j < P[:, None], score, -math.inf)
    rank = torch.argsort(torch.argsort(score, dim=1, descending=True, stable=True), dim=1)
    pick = (rank < top) & (j < P[:, None])
    pos = torch.sort(torch.where(pick, j, W), 1)[0][:, :top]
    pos = torch.nn.functional.pad(pos, (0, top - pos.shape[1]), value=W)
    rowid = torch.arange(R, device=q.device) // q_len
    sel = torch.where(pos < W, table[rowid[:, None], pos.clamp(max=W - 1)], -1).int()
    kept = torch.minimum(P, torch.full_like(P, top))
    return sel, (live - (P - kept) * page).int()


def _sparse(s):
    q = torch.cat([s["q_abs"].float(), s["q_pe"].float()], 2)
    sel, sel_len = _choose(q, s["codes"], s["scales"], s["table"], s["lengths"], s["page"],
                           s["top"], s["q_len"])
    return _attend(s["q_abs"], s["q_pe"], s["cache"], sel, sel_len, 1) + [sel, sel_len]


def run(s):
    if own:
        import head_latent_attention_absorbed_gb300 as mla
        if s["op"] == "extend":
            mla.pages_extend(s["pg"], s["cached"], s["new"], s["table"], s["free"], s["num_free"],
                             s["lengths"], s["row_starts"], s["slots"], s["positions"],
                             num_free_out=s["num_free_out"], dev_status=s["status"])
            return [s["table"], s["lengths"], s["row_starts"], s["slots"], s["positions"],
                    s["num_free_out"]]
        if s["op"] == "append":
            mla.cache_append_paged(s["d"], s["pg"], s["rows"], s["positions"], s["slots"],
                                   s["cache"], rope_base=BASE, dev_status=s["status"])
            return [s["cache"]]
        if s["op"] == "attn":
            mla.decode_attn_paged(s["d"], s["pg"], s["q_abs"], s["q_pe"], s["cache"], s["table"],
                                  s["lengths"], s["o"], s["ws"], SCALE, q_len=s["q_len"],
                                  lse=s["lse"], dev_status=s["status"])
            return [s["o"], s["lse"]]
        if s["op"] == "index":
            mla.page_index(s["d"], s["pg"], s["cache"], s["table"], s["first"], s["lengths"],
                           s["new"], s["codes"], s["scales"], dev_status=s["status"])
            return [s["codes"], s["scales"]]
        mla.decode_attn_sparse(s["d"], s["pg"], s["q_abs"], s["q_pe"], s["cache"], s["table"],
                               s["lengths"], s["codes"], s["scales"], s["sel"], s["sel_len"],
                               s["o"], s["ws"], SCALE, q_len=s["q_len"], keep_first=1, keep_last=1,
                               lse=s["lse"], dev_status=s["status"])
        return [s["o"], s["lse"], s["sel"], s["sel_len"]]
    if s["op"] == "extend":
        return _extend(s)
    if s["op"] == "append":
        return _append(s)
    if s["op"] == "attn":
        return _attend(s["q_abs"], s["q_pe"], s["cache"], s["table"], s["lengths"], s["q_len"])
    if s["op"] == "index":
        return _index(s["cache"], s["table"], s["first"], s["lengths"], s["codes"], s["scales"],
                      s["page"])
    return _sparse(s)


# --------------------------------------------------------------------------- what a pass needs

def work(case):
    B, page, op = case["batch"], case["page"], case["op"]
    lens = _lengths(case)
    if op == "extend":
        T = int(_spread(case["new_lo"], case["new_hi"], B).sum())
        pages = T / page                     # taken from the free list, written to the table
        return {"bytes": 16.0 * B + 8 * pages + 12.0 * T, "flops": 0}
    elt = BYTES[case["dtype"]]
    if op == "append":
        T = B * case["new"]
        return {"bytes": T * (ROW * (elt + (4 if elt == 4 else 2)) + 12.0), "flops": 6.0 * T * D_R}
    if op == "index":
        n = int((lens - (lens - case["new"]) // page * page).sum())      # rows of the touched pages
        return {"bytes": n * ROW * elt + (n / page) * (ROW + 8.0), "flops": 2.0 * n * ROW}
    H, R, io = case["heads"], B * case["q_len"], 4 if elt == 4 else 2
    qo = R * H * ((ROW + D_C) * io + 4.0)
    if op == "attn":
        n = float(lens.sum())
        return {"bytes": n * ROW * elt + qo + 4 * n / page,
                "flops": 2.0 * n * case["q_len"] * H * (ROW + D_C)}
    pages = float(_pages(lens, page).sum())
    n = float(np.minimum(lens, case["top"] * page).sum()) * case["q_len"]
    return {"bytes": pages * (ROW + 8.0) + n * ROW * elt + qo + 4.0 * R * (case["top"] + 1),
            "flops": 2.0 * pages * case["q_len"] * H * ROW + 2.0 * n * H * (ROW + D_C)}


# --------------------------------------------------------------------------- in 64 bits

def _softmax64(q, c):
    """q [H, 576], c [n, 576] in 64 bits: the attention output and its log-sum-exp."""
    x = (q @ c.T) * SCALE
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ c[:, :D_C], lse


def exact(case, seed):
    op = case["op"]
    if op == "extend":
        return None                         # whole numbers only
    s = prepare(case, seed)
    page, B = case["page"], case["batch"]
    cache = s["cache"]
    table, lengths = s["table"].cpu().numpy(), s["lengths"].cpu().numpy()
    if op == "append":
        y = cache.double().view(-1, ROW).clone()
        x = s["rows"].double()
        i = torch.arange(D_R // 2, device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                           s["positions"].double()[:, None] * torch.exp(-math.log(BASE) * i / 32))
        k = torch.view_as_real(torch.view_as_complex(x[:, D_C:].reshape(-1, 32, 2).contiguous()) * turn)
        y[s["slots"]] = torch.cat([x[:, :D_C], k.reshape(-1, D_R)], 1)
        return [y.view(cache.shape)]
    if op == "index":
        scales = s["scales"].double().clone()
        first = s["first"].cpu().numpy()
        for b in range(B):
            for j in range(int(first[b]) // page, int(_pages(lengths[b], page))):
                p = int(table[b, j])
                mean = cache[p, :min(page, int(lengths[b]) - j * page)].double().mean(0)
                scales[p] = mean.abs().max() / 127
        return [None, scales]
    H, q_len = case["heads"], case["q_len"]
    q = torch.cat([s["q_abs"].double(), s["q_pe"].double()], 2)
    o, lse = [], []
    sel = sel_len = None
    if op == "sparse":
        q32 = torch.cat([s["q_abs"].float(), s["q_pe"].float()], 2).cpu().numpy()
        codes, scales = s["codes"].cpu().numpy(), s["scales"].cpu().numpy()
        sel = np.full((B * q_len, case["top"]), -1, np.int32)
        sel_len = np.zeros(B * q_len, np.int32)
    for r in range(B * q_len):
        b = r // q_len
        n = int(lengths[b]) - (q_len - 1 - r % q_len)
        pages = table[b, :_pages(n, page)]
        if op == "sparse":
            if len(pages) > case["top"]:
                big = np.abs(q32[r]).max(1)
                qc = np.rint(q32[r] * (np.float32(127) / big)[:, None]).astype(np.int64)
                v = (big / np.float32(127))[:, None] * (qc @ codes[pages].astype(np.int64).T).astype(np.float32)
                score = v.max(0) * scales[pages]
                inner = np.argsort(-score[1:-1], kind="stable")[:case["top"] - 2] + 1
                keep = np.sort(np.concatenate([[0], inner, [len(pages) - 1]]))
                n -= (len(pages) - len(keep)) * page
                pages = pages[keep]
            sel[r, :len(pages)] = pages
            sel_len[r] = n
        c = cache.view(torch.uint8).view(cache.shape[0], -1)[torch.as_tensor(pages).cuda().long()].view(cache.dtype)
        y, z = _softmax64(q[r], c.view(-1, ROW)[:n].double())
        o.append(y)
        lse.append(z)
    out = [torch.stack(o), torch.stack(lse)]
    return out if sel is None else out + [sel, sel_len]
