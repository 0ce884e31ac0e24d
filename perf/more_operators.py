"""The 4-bit latent cache's operators as a serving program calls them: what is measured.

A 4-bit pool keeps each row's 512 latent values as E2M1 numbers (0, 1/2, 1, 3/2, 2, 3, 4,
6 with a sign) times a power of two 2^e, -8 <= e <= 6, per 16 values -- the smallest with
which the block's largest magnitude is at most 7 2^e, so that no value is further than 2^e
from its code -- and the 64 rotated key values as bf16.  Each case is one pass:

- ``append``: new rows rotated, quantised and written into their pages, then read back;
- ``read``:   cached rows of a pool read back as one packed block of rows;
- ``attn``:   decode attention over the 4-bit pages;
- ``sparse``: the index of the pages that a step touched, the pages chosen by its score, and
  attention over the chosen ones.

With ``own`` false, ``run`` computes the operator in its plain form with elementary torch
operations; with ``own`` true it makes the library's calls.  Lengths are spread evenly over
[lo, hi] and dealt to the sequences by the seed, so that the work of a case is known from
its sizes alone.
"""
import math

import numpy as np
import torch

own = False

D_C, D_R, BLOCK = 512, 64, 16
ROW = D_C + D_R
E_MIN, E_MAX = -8, 6
SCALE = (128 + 64) ** -0.5
BASE = 10000.0
TINY = 1e-30                     # below this largest magnitude an index row or a query counts as zero
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BYTES = {"f32": ROW * 4, "bf16": ROW * 2, "fp8": ROW, "fp4": D_C // 2 + D_C // BLOCK // 2 + 2 * D_R}


def listed():
    return [
        # one decode step's new rows, and what the cache made of them
        dict(name="append_decode_b8", op="append", batch=8, lo=4000, hi=4095, new=1, page=64,
             rows="bf16", out="bf16"),
        # prompts' rows (61 x 1021 tokens: odd on purpose), read back for the chunk that follows
        dict(name="append_prefill_b61", op="append", batch=61, lo=0, hi=3000, new=1021, page=64,
             rows="bf16", out="bf16"),
        # a cached prefix handed to a chunk of prefill: four long ones
        dict(name="read_fp4_b4_s16384", op="read", batch=4, lo=16384, hi=16384, page=64, dtype="fp4",
             out="bf16"),
        # many short prefixes of an E4M3 pool, some of them shorter than a page
        dict(name="read_fp8_b61_ragged", op="read", batch=61, lo=1, hi=1500, page=64, dtype="fp8",
             out="bf16"),
        # the smallest decode call: one short sequence
        dict(name="attn_b1_s64", op="attn", batch=1, heads=16, lo=64, hi=64, page=16, q_len=1),
        # an ordinary decode step of a small server
        dict(name="attn_b8_s4096", op="attn", batch=8, heads=16, lo=4096, hi=4096, page=64, q_len=1),
        # many requests of very different lengths
        dict(name="attn_b64_ragged", op="attn", batch=64, heads=16, lo=512, hi=8192, page=64, q_len=1),
        # a few very long contexts
        dict(name="attn_b4_s65536", op="attn", batch=4, heads=16, lo=65536, hi=65536, page=64, q_len=1),
        # two tokens a sequence (speculative decoding), odd lengths
        dict(name="attn_h64_b16_q2", op="attn", batch=16, heads=64, lo=333, hi=8191, page=128, q_len=2),
        # a large model's decode step: 128 heads share every cached row
        dict(name="attn_h128_b32_s16384", op="attn", batch=32, heads=128, lo=16384, hi=16384, page=64,
             q_len=1),
        # long contexts decoded over 2048 chosen rows each
        dict(name="sparse_b4_s65536", op="sparse", batch=4, heads=16, lo=65536, hi=65536, page=64,
             q_len=1, top=32),
        # a large model's decode step over 2048 chosen rows
        dict(name="sparse_h128_b32", op="sparse", batch=32, heads=128, lo=9000, hi=16384, page=64,
             q_len=1, top=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "attn", "attn", "sparse", "sparse"])
    page = rng.choice([16, 32, 64, 64, 128, 256])
    if op == "append":
        new = _log(rng, 1, 1024)
        return dict(op=op, batch=_log(rng, 1, 60), lo=0, hi=_log(rng, 1, 3000), new=new, page=page,
                    rows=rng.choice(["f32", "bf16"]), out="bf16")
    if op == "read":
        batch = _log(rng, 1, 60)
        hi = _log(rng, 1, 60000 // batch)
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, page=page,
                    dtype=rng.choice(["f32", "bf16", "fp8", "fp4", "fp4", "fp4"]),
                    out=rng.choice(["f32", "bf16", "bf16"]))
    q_len = rng.choice([1, 1, 1, 2, 3, 4])
    heads = rng.choice([16, 16, 32, 48, 64, 128])
    batch = _log(rng, 1, 64 if heads <= 32 else 16)
    hi = _log(rng, 100, min(65536, 400000 // (batch * q_len)))
    c = dict(op=op, batch=batch, heads=heads, lo=rng.randint(q_len, hi), hi=hi, page=page, q_len=q_len)
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


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _latents(g, shape):
    """Latent rows and keys in bf16; rows of one page (the last but one axis) resemble one
    another, as neighbouring tokens do, and the channels differ in magnitude."""
    gain = torch.rand((ROW,), generator=g, device="cuda").mul_(2.0).sub_(1.0).exp2_()
    gain[D_C:] = 1.0
    x = torch.randn(shape + (ROW,), generator=g, device="cuda").mul_(0.8)
    x.add_(torch.randn(shape[:-1] + (1, ROW), generator=g, device="cuda"), alpha=0.6)
    return x.mul_(gain).bfloat16()


def _inputs(case, seed):
    """What both forms start from: rows, tables, lengths and queries."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    B, page, op = case["batch"], case["page"], case["op"]
    order = r.permutation(B)
    total = _lengths(case)[order] + (case["new"] if op == "append" else 0)
    n_pages = _pages(total, page)
    width = max(int(n_pages.max()), 1)
    num_pages = int(n_pages.sum()) + 7
    ids = r.permutation(num_pages)[:int(n_pages.sum())]
    table = np.full((B, width), -1)
    n = 0
    for b in range(B):
        table[b, :n_pages[b]] = ids[n:n + n_pages[b]]
        n += n_pages[b]
    s = {"op": op, "page": page, "num_pages": num_pages, "total": total, "table64": table,
         "table": _i32(table), "lengths": _i32(total)}
    if op == "append":
        new = case["new"]
        first = total - new
        pos = first[:, None] + np.arange(new)[None, :]
        slots = np.take_along_axis(table, pos // page, 1) * page + pos % page
        s.update(rows=_latents(g, (B, new)).view(-1, ROW).to(OUT[case["rows"]]), new=new,
                 positions=_i32(pos.reshape(-1)), slots=torch.as_tensor(slots.reshape(-1)).cuda(),
                 first=_i32(first), starts=_i32(np.arange(B + 1) * new))
        return s
    if op == "read":
        pool = _latents(g, (num_pages, page))
        s.update(pool=pool if case["dtype"] == "fp4" else pool.to(DTYPES[case["dtype"]]),
                 starts=_i32(np.concatenate([[0], np.cumsum(total)])))
        return s
    H, R = case["heads"], B * case["q_len"]
    s["pool"] = _latents(g, (num_pages, page))
    # the absorbed query of N(0, 1) queries and N(0, 0.02^2) weights, and a rotated query
    s.update(q_abs=(torch.randn((R, H, D_C), generator=g, device="cuda") * 0.226).bfloat16(),
             q_pe=torch.randn((R, H, D_R), generator=g, device="cuda").bfloat16(),
             q_len=case["q_len"])
    if op == "sparse":
        s.update(first=_i32(total - case["q_len"]), new=case["q_len"], top=case["top"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, page, n, dev = s["op"], s["page"], s["num_pages"], torch.device("cuda")
    out_rows = int(s["total"].sum()) if op == "read" else case["batch"] * case.get("new", 0)
    dtype = case.get("dtype", "fp4")
    pool = s.pop("pool", None)
    lut = _lut()
    if op == "sparse":                       # the index of every page
        s["codes"], s["scales"] = _index(
            lut, _held(pool, lut), s["table"], torch.zeros_like(s["lengths"]), s["lengths"],
            torch.zeros((n, ROW), dtype=torch.int8, device=dev), torch.zeros(n, device=dev), page)
    if op in ("append", "read"):
        s["out"] = torch.empty((max(out_rows, 1), ROW), dtype=OUT[case["out"]], device=dev)
    if not own:
        s["lut"] = lut
        if op == "append":
            s["held"] = _held(torch.zeros((n, page, ROW), dtype=torch.bfloat16, device=dev), lut)
        elif dtype == "fp4":
            s["held"] = _held(pool, lut)
        else:
            s["cache"] = pool
        return s
    import head_latent_attention_absorbed_gb300 as mla
    code = mla.MLA_FP4_E2M1 if dtype == "fp4" else mla.dtype_code(DTYPES[dtype])
    pg = mla.paging(page, n, int(s["table"].shape[1]))
    d = mla.dims(case["batch"], case.get("heads", 16), max(int(s["total"].max()), 1), code)
    s.update(pg=pg, d=d, status=torch.zeros(1, dtype=torch.int32, device=dev))
    if dtype != "fp4":
        s["cache"] = pool
        return s
    s["cache"] = torch.zeros(mla.pool_bytes(d, pg), dtype=torch.uint8, device=dev)
    if pool is not None:                     # its keys are rotated already
        every = torch.arange(n * page, device=dev)
        mla.cache_append_paged(d, pg, pool.view(-1, ROW), torch.zeros_like(every, dtype=torch.int32),
                               every, s["cache"], rope_base=BASE)
    if op in ("attn", "sparse"):
        R, H = s["q_abs"].shape[:2]
        s.update(o=torch.empty((R, H, D_C), dtype=torch.bfloat16, device=dev),
                 lse=torch.empty((R, H), device=dev))
        size = (mla.paged_workspace_bytes(d, pg, torch.bfloat16, s["q_len"]) if op == "attn" else
                mla.sparse_workspace_bytes(d, pg, torch.bfloat16, s["top"], s["q_len"]))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=dev)
    if op == "sparse":
        s.update(sel=torch.empty((R, s["top"]), dtype=torch.int32, device=dev),
                 sel_len=torch.empty(R, dtype=torch.int32, device=dev))
    return s


# --------------------------------------------------------------------------- plain forms

def _lut():
    """The two values of each code byte, and 2^e by e - E_MIN."""
    half = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
    pairs = torch.stack([half.repeat(16), half.repeat_interleave(16)], 1)
    return pairs.cuda(), torch.tensor([2.0 ** e for e in range(E_MIN, E_MAX + 1)]).cuda()


def _quantise(x, lut):
    """x [..., 512] fp32 as codes (two a byte, the even value low) and e - E_MIN."""
    v = x.unflatten(-1, (D_C // BLOCK, BLOCK))
    m, k = torch.frexp(v.abs().amax(-1))
    e = (torch.where(m <= 0.875, k - 3, k - 2)).clamp(E_MIN, E_MAX)     # the largest <= 7 2^e
    e = torch.where(m == 0, E_MIN, e) - E_MIN
    y = v.abs() / lut[1][e][..., None]
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = ((y / step).round() * step).clamp(max=6.0)
    code = torch.where(y <= 2, 2 * y, torch.where(y < 6, y + 2, 7.0)).to(torch.uint8)
    code = (code | (v < 0).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, e.to(torch.uint8)


def _held(pool, lut):
    """A pool [pages, page, 576] as a 4-bit cache holds it: codes, exponents, keys."""
    code, e = _quantise(pool[..., :D_C].float(), lut)
    return [code, e, pool[..., D_C:].contiguous()]


def _values(lut, code, e, key):
    """Rows in fp32 from their codes, exponents and keys."""
    v = lut[0][code.int()].flatten(-2).unflatten(-1, (D_C // BLOCK, BLOCK))
    return torch.cat([(v * lut[1][e.int()][..., None]).flatten(-2), key.float()], -1)


def _rotated(x, positions):
    """x [n, 576] fp32 with its key rotated."""
    inv = BASE ** (-torch.arange(0, D_R, 2, device=x.device, dtype=torch.float64) / D_R)
    a = positions.double()[:, None] * inv[None, :]
    c, n = a.cos().float(), a.sin().float()
    k = x[:, D_C:].unflatten(1, (D_R // 2, 2))
    return torch.stack([k[..., 0] * c - k[..., 1] * n, k[..., 0] * n + k[..., 1] * c], -1).flatten(1)


def _append(s):
    x = s["rows"].float()
    code, e = _quantise(x[:, :D_C], s["lut"])
    held = [t.flatten(0, 1) for t in s["held"]]
    held[0][s["slots"]] = code
    held[1][s["slots"]] = e
    held[2][s["slots"]] = _rotated(x, s["positions"]).bfloat16()
    # the rows just written lie at their slots
    return [_values(s["lut"], *[t[s["slots"]] for t in held]).to(s["out"].dtype)]


def _flat(s, slot):
    """The rows at these slots in fp32."""
    if "held" in s:
        return _values(s["lut"], *[t.flatten(0, 1)[slot] for t in s["held"]])
    flat = s["cache"].view(-1, ROW)
    if flat.dtype == torch.float8_e4m3fn:    # one-byte rows are gathered as bytes
        return flat.view(torch.uint8)[slot].view(flat.dtype).float()
    return flat[slot].float()


def _read(s):
    page, starts = s["page"], s["starts"].long()
    t = torch.arange(s["out"].shape[0], device=starts.device)
    b = (torch.searchsorted(starts, t, right=True) - 1).clamp(0, s["table"].shape[0] - 1)
    pos = t - starts[b]
    return [_flat(s, s["table"][b, pos // page].long() * page + pos % page).to(s["out"].dtype)]


def _attend(s, table, lengths, q_len):
    """Attention of q_len tokens per table row; q [R, H, .], R = table rows x q_len."""
    B, (R, H, _) = table.shape[0], s["q_abs"].shape
    page = s["page"]
    rows = table.shape[1] * page
    t = torch.arange(rows, device=table.device)
    c = _flat(s, table[:, t // page].long().clamp(min=0) * page + t % page)
    q = torch.cat([s["q_abs"].float(), s["q_pe"].float()], 2).view(B, q_len * H, ROW)
    sc = torch.matmul(q, c.transpose(1, 2)).view(B, q_len, H, rows) * SCALE
    back = torch.arange(q_len - 1, -1, -1, device=c.device)
    live = lengths.long()[:, None] - back[None, :]
    dead = t[None, None, :] >= live[:, :, None]
    sc = sc.masked_fill(dead[:, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = (sc - m).exp()
    z = e.sum(-1, keepdim=True)
    o = torch.matmul((e / z).view(B, q_len * H, rows), c[:, :, :D_C])
    return [o.view(R, H, D_C).bfloat16(), (m + z.log()).view(R, H)]


def _index(lut, held, table, first, lengths, codes, scales, page):
    """Index rows of the pages that hold rows [first, length) of each sequence."""
    B, W = table.shape
    j = torch.arange(W, device=table.device)[None, :]
    hit = (j >= first.long()[:, None] // page) & (j * page < lengths.long()[:, None])
    hit = hit & (first < lengths)[:, None]
    ids = table[hit].long()
    n = (lengths.long()[:, None] - j * page).clamp(0, page)[hit]
    x = _values(lut, *[t[ids] for t in held])
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
    codes, scales = codes.clone(), scales.clone()
    codes[ids] = torch.where(good[:, None], code, 0.0).to(torch.int8)
    scales[ids] = torch.where(good, scale, 0.0)
    return codes, scales


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
    codes, scales = _index(s["lut"], s["held"], s["table"], s["first"], s["lengths"], s["codes"],
                           s["scales"], s["page"])
    q = torch.cat([s["q_abs"].float(), s["q_pe"].float()], 2)
    sel, sel_len = _choose(q, codes, scales, s["table"], s["lengths"], s["page"], s["top"], s["q_len"])
    return _attend(s, sel, sel_len, 1) + [sel, sel_len, codes, scales]


def run(s):
    op = s["op"]
    if own:
        import head_latent_attention_absorbed_gb300 as mla
        if op == "append":
            mla.cache_append_paged(s["d"], s["pg"], s["rows"], s["positions"], s["slots"], s["cache"],
                                   rope_base=BASE, dev_status=s["status"])
            mla.cache_read_paged(s["d"], s["pg"], s["cache"], s["table"], s["lengths"], s["starts"],
                                 s["out"], first_rows=s["first"], dev_status=s["status"])
            return [s["out"]]
        if op == "read":
            mla.cache_read_paged(s["d"], s["pg"], s["cache"], s["table"], s["lengths"], s["starts"],
                                 s["out"], dev_status=s["status"])
            return [s["out"]]
        if op == "attn":
            mla.decode_attn_paged(s["d"], s["pg"], s["q_abs"], s["q_pe"], s["cache"], s["table"],
                                  s["lengths"], s["o"], s["ws"], SCALE, q_len=s["q_len"],
                                  lse=s["lse"], dev_status=s["status"])
            return [s["o"], s["lse"]]
        mla.page_index(s["d"], s["pg"], s["cache"], s["table"], s["first"], s["lengths"], s["new"],
                       s["codes"], s["scales"], dev_status=s["status"])
        mla.decode_attn_sparse(s["d"], s["pg"], s["q_abs"], s["q_pe"], s["cache"], s["table"],
                               s["lengths"], s["codes"], s["scales"], s["sel"], s["sel_len"],
                               s["o"], s["ws"], SCALE, q_len=s["q_len"], keep_first=1, keep_last=1,
                               lse=s["lse"], dev_status=s["status"])
        return [s["o"], s["lse"], s["sel"], s["sel_len"], s["codes"], s["scales"]]
    if op == "append":
        return _append(s)
    if op == "read":
        return _read(s)
    if op == "attn":
        return _attend(s, s["table"], s["lengths"], s["q_len"])
    return _sparse(s)


# --------------------------------------------------------------------------- what a pass needs

def work(case):
    B, page, op = case["batch"], case["page"], case["op"]
    lens, elt = _lengths(case), {"f32": 4, "bf16": 2}
    if op == "append":                       # rows in, the cache written, rows out
        T = B * case["new"]
        return {"bytes": T * (ROW * (elt[case["rows"]] + elt[case["out"]]) + BYTES["fp4"] + 12.0),
                "flops": T * (6.0 * D_R + 4.0 * D_C)}
    if op == "read":
        n = float(lens.sum())
        return {"bytes": n * (BYTES[case["dtype"]] + ROW * elt[case["out"]]) + 4 * n / page,
                "flops": n * ROW}
    H, R = case["heads"], B * case["q_len"]
    qo = R * H * ((ROW + D_C) * 2 + 4.0)
    if op == "attn":
        n = float(lens.sum())
        return {"bytes": n * BYTES["fp4"] + qo + 4 * n / page,
                "flops": 2.0 * n * case["q_len"] * H * (ROW + D_C)}
    pages = float(_pages(lens, page).sum())
    n = float(np.minimum(lens, case["top"] * page).sum()) * case["q_len"]
    touched = float((lens - (lens - case["q_len"]) // page * page).sum())      # rows of those pages
    return {"bytes": pages * (ROW + 8.0) + (n + touched) * BYTES["fp4"] + qo + 4.0 * R * (case["top"] + 1),
            "flops": 2.0 * pages * case["q_len"] * H * ROW + 2.0 * n * H * (ROW + D_C)}


# --------------------------------------------------------------------------- in 64 bits

def _rounded64(x):
    """x [..., 512] in 64 bits to the values that a 4-bit cache has for them."""
    v = x.reshape(x.shape[:-1] + (D_C // BLOCK, BLOCK))
    top = v.abs().max(-1, keepdim=True)[0]
    unit = torch.full_like(top, 2.0 ** E_MIN)
    for e in range(E_MIN, E_MAX):
        unit = torch.where(top > 7 * 2.0 ** e, 2.0 ** (e + 1), unit)
    y = v.abs() / unit
    out = torch.zeros_like(y)
    # borders between neighbours; the even code has the tie
    for border, even_above, above in ((.25, 0, .5), (.75, 1, 1.), (1.25, 0, 1.5), (1.75, 1, 2.),
                                      (2.5, 0, 3.), (3.5, 1, 4.), (5., 0, 6.)):
        out = torch.where((y > border) | ((y == border) if even_above else (y < 0)), above, out)
    return torch.copysign(out * unit, v).reshape(x.shape)


def _cached64(pool, dtype):
    x = pool.double()
    return torch.cat([_rounded64(x[..., :D_C]), x[..., D_C:]], -1) if dtype == "fp4" else x


def _softmax64(q, c):
    """q [H, 576], c [n, 576] in 64 bits: the attention output and its log-sum-exp."""
    x = (q @ c.T) * SCALE
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ c[:, :D_C], lse


def exact(case, seed):
    op, page = case["op"], case["page"]
    s = _inputs(case, seed)
    lengths, table = s["total"], s["table64"]
    if op == "append":
        x = s["rows"].double()
        i = torch.arange(D_R // 2, device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                           s["positions"].double()[:, None] * torch.exp(-math.log(BASE) * i / 32))
        k = torch.view_as_real(torch.view_as_complex(x[:, D_C:].reshape(-1, 32, 2).contiguous()) * turn)
        return [torch.cat([_rounded64(x[:, :D_C]), k.reshape(-1, D_R)], 1)]

    def rows_of(pages, n):
        at = torch.as_tensor(np.ascontiguousarray(pages)).cuda().long()
        pool = s["pool"]
        c = (pool.view(torch.uint8).view(pool.shape[0], -1)[at].view(pool.dtype)
             if pool.dtype == torch.float8_e4m3fn else pool[at])
        return _cached64(c.reshape(-1, ROW)[:n], case.get("dtype", "fp4"))

    if op == "read":
        out = torch.cat([rows_of(t[:_pages(int(n), page)], int(n)) for t, n in zip(table, lengths)])
        return [out if len(out) else torch.zeros((1, ROW), dtype=torch.float64, device="cuda")]
    q_len, B = case["q_len"], case["batch"]
    q = torch.cat([s["q_abs"].double(), s["q_pe"].double()], 2)
    o, lse, sel, sel_len = [], [], None, None
    if op == "sparse":
        codes = np.zeros((s["num_pages"], ROW), np.int8)
        scales, exact_scales = np.zeros(s["num_pages"], np.float32), np.zeros(s["num_pages"])
        for b in range(B):
            n, P = int(lengths[b]), int(_pages(lengths[b], page))
            c = torch.zeros((P * page, ROW), dtype=torch.float64, device="cuda")
            c[:n] = rows_of(table[b, :P], n)
            c = c.view(P, page, ROW)
            held = np.minimum(page, n - page * np.arange(P))
            e = np.frexp(c.abs().amax((1, 2)).cpu().numpy())[1]
            fine = torch.as_tensor(2.0 ** (20 - e)).cuda()
            sums = (c * fine[:, None, None]).round().sum(1).cpu().numpy()
            peak = np.abs(sums).max(1)
            f = peak.astype(np.float32)
            inv = (np.float32(127) * (np.float32(1) / f)).astype(np.float32)
            codes[table[b, :P]] = np.rint(sums.astype(np.float32) * inv[:, None]).astype(np.int8)
            scales[table[b, :P]] = (f * (np.float32(1) / np.float32(127)) / held.astype(np.float32)
                                    * (2.0 ** (e - 20)).astype(np.float32))
            exact_scales[table[b, :P]] = (np.abs(c.sum(1).cpu().numpy()).max(1) / held) / 127
        q32 = torch.cat([s["q_abs"].float(), s["q_pe"].float()], 2).cpu().numpy()
        sel = np.full((B * q_len, case["top"]), -1, np.int32)
        sel_len = np.zeros(B * q_len, np.int32)
    for r in range(B * q_len):
        b = r // q_len
        n = int(lengths[b]) - (q_len - 1 - r % q_len)
        pages = table[b, :_pages(n, page)]
        if op == "sparse":
            if len(pages) > case["top"]:
                big = np.abs(q32[r]).max(1)
                qc = np.rint(q32[r] * (np.float32(127) * (np.float32(1) / big))[:, None]).astype(np.int64)
                v = (big * (np.float32(1) / np.float32(127)))[:, None] * (
                    qc @ codes[pages].astype(np.int64).T).astype(np.float32)
                score = v.max(0) * scales[pages]
                inner = np.argsort(-score[1:-1], kind="stable")[:case["top"] - 2] + 1
                keep = np.sort(np.concatenate([[0], inner, [len(pages) - 1]]))
                n -= (len(pages) - len(keep)) * page
                pages = pages[keep]
            sel[r, :len(pages)] = pages
            sel_len[r] = n
        y, z = _softmax64(q[r], rows_of(pages, n))
        o.append(y)
        lse.append(z)
    out = [torch.stack(o), torch.stack(lse)]
    return out if sel is None else out + [sel, sel_len, codes, exact_scales]
