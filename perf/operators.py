"""The operators of a decode step over a 4-bit paged KV cache, and the cases they are measured at.

Three operators, in the order in which a serving step calls them:

  tables  page tables and slot maps of the step, built on the GPU from the requests' lengths
  append  the step's new K/V rows quantised into the cache: e2m1 codes in blocks of 16 with an e4m3 scale
  attend  attention of the step's query rows over that cache, through the device tables

Each has its plain form here (elementary torch operations in 32 bits) and, with `own`, the framework's call.
"""
import math

import torch

own = False  # False: run() computes the plain forms; True: it calls the framework

GROUP = 16  # values that share a scale, along head_dim
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
NEVER_WRITTEN = 0x7F  # the scale byte that memory of unused cache slots holds here: NaN as e4m3
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # a small server's decode step: every request appends one token, few of them start a page
        {"name": "tables decode 64", "op": "tables", "batch": 64, "qo_lo": 1, "qo_hi": 1, "kv_lo": 500, "kv_hi": 8191,
         "page": 16, "prompts": 0, "pad": 0},
        # continuous batching at its largest: 2000 requests, some of them new prompts, 200 padded rows
        {"name": "tables mixed 2000", "op": "tables", "batch": 2000, "qo_lo": 1, "qo_hi": 200, "kv_lo": 0,
         "kv_hi": 4000, "page": 16, "prompts": 300, "pad": 200},
        # one layer's rows of a decode step (64 requests), as slices of the fused projection's output
        {"name": "append decode 64", "op": "append", "rows": 64, "pad": 0, "heads": 8, "group": 8, "dim": 128,
         "page": 16, "pages": 4096, "layout": "NHD", "dtype": "bf16"},
        # one layer's rows of a long prompt chunk beside some padding
        {"name": "append prompt 16000", "op": "append", "rows": 16000, "pad": 384, "heads": 8, "group": 8,
         "dim": 128, "page": 16, "pages": 4096, "layout": "HND", "dtype": "bf16"},
        # the smallest call: one request that has just started to decode
        {"name": "attend 1x77", "op": "attend", "batch": 1, "qo_lo": 1, "qo_hi": 1, "kv_lo": 77, "kv_hi": 77, "heads": 8,
         "kv_heads": 1, "dim": 128, "page": 16, "layout": "NHD", "dtype": "fp16"},
        # the decode timing script's batch: 128 requests of 1024 keys
        {"name": "attend decode script", "op": "attend", "batch": 128, "qo_lo": 1, "qo_hi": 1, "kv_lo": 1024,
         "kv_hi": 1024, "heads": 8, "kv_heads": 1, "dim": 128, "page": 16, "layout": "NHD", "dtype": "fp16"},
        # the mixed benchmark's decodes: 256 requests of 512 to 8192 keys
        {"name": "attend decode 256", "op": "attend", "batch": 256, "qo_lo": 1, "qo_hi": 1, "kv_lo": 512, "kv_hi": 8192,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "layout": "NHD", "dtype": "bf16"},
        # few requests of very long context: the keys of one have to be split over the card
        {"name": "attend long 3", "op": "attend", "batch": 3, "qo_lo": 1, "qo_hi": 1, "kv_lo": 60001, "kv_hi": 131071,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "layout": "HND", "dtype": "bf16"},
        # speculative decoding: four drafted tokens of each request
        {"name": "attend drafts 64x4", "op": "attend", "batch": 64, "qo_lo": 4, "qo_hi": 4, "kv_lo": 512, "kv_hi": 8192,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "layout": "NHD", "dtype": "bf16"},
        # head dimension 64, three query heads a kv head, small pages, short and odd lengths
        {"name": "attend odd heads", "op": "attend", "batch": 33, "qo_lo": 1, "qo_hi": 2, "kv_lo": 2, "kv_hi": 2999,
         "heads": 12, "kv_heads": 4, "dim": 64, "page": 8, "layout": "HND", "dtype": "fp16"},
        # ragged short prompts, each attending to itself
        {"name": "attend prompts 32", "op": "attend", "batch": 32, "qo_lo": 16, "qo_hi": 200, "kv_lo": 0, "kv_hi": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "layout": "NHD", "dtype": "bf16"},
        # a prompt's chunk of 2000 tokens behind 6000 cached ones
        {"name": "attend chunk 2000", "op": "attend", "batch": 1, "qo_lo": 2000, "qo_hi": 2000, "kv_lo": 8000,
         "kv_hi": 8000, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "layout": "NHD", "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "attend", "attend", "attend", "attend"))
    page = rng.choice((1, 4, 8, 16, 16, 32, 64, 128))
    if op == "tables":
        batch, hi = _spread(rng, 1, 2000), _spread(rng, 16, 8000)
        return {"op": op, "batch": batch, "qo_lo": rng.choice((0, 1)), "qo_hi": rng.randint(1, 8),
                "kv_lo": rng.randint(0, hi // 2), "kv_hi": min(hi, 8_000_000 // batch), "page": max(page, 8),
                "prompts": 0, "pad": rng.randint(0, 300)}
    layout, dtype, dim = rng.choice(("NHD", "HND")), rng.choice(("fp16", "bf16")), rng.choice((64, 128, 128, 256))
    if op == "append":
        return {"op": op, "rows": _spread(rng, 1, 8000), "pad": rng.randint(0, 100), "heads": rng.randint(1, 8),
                "group": rng.randint(1, 8), "dim": dim, "page": page, "pages": 65536 // page, "layout": layout,
                "dtype": dtype}
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16))
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "layout": layout,
            "dtype": dtype}
    kind = rng.choice(("decode", "decode", "drafts", "prompts", "chunk"))
    if kind in ("decode", "drafts"):
        hi = _spread(rng, 16, 100_000)
        batch = _spread(rng, 1, max(1, min(256, 1_000_000_000 // (hi * kv_heads * dim))))
        qo = 1 if kind == "decode" else rng.randint(2, 8)
        return {**case, "batch": batch, "qo_lo": 1, "qo_hi": qo, "kv_lo": max(qo, hi // rng.randint(1, 16)),
                "kv_hi": hi}
    if kind == "prompts":
        return {**case, "batch": rng.randint(1, 40), "qo_lo": 1, "qo_hi": _spread(rng, 16, 500), "kv_lo": 0, "kv_hi": 0}
    qo = _spread(rng, 33, 1500)
    kv = qo + _spread(rng, 1, 4000)
    return {**case, "batch": rng.randint(1, 2), "qo_lo": max(1, qo // 2), "qo_hi": qo, "kv_lo": qo, "kv_hi": kv}


# ------------------------------------------------------------------------------------------------- lengths and inputs


def _generators(seed, device="cuda"):
    return torch.Generator().manual_seed(int(seed)), torch.Generator(device=device).manual_seed(int(seed))


def _whole(g, lo, hi, n):
    return torch.randint(int(lo), int(hi) + 1, (int(n),), generator=g)


def _lengths(case):
    """(query lengths, kv lengths with the new tokens) of the attended batch: by the case alone, so that work() knows
    them.  A prompt (kv_hi 0) has no keys but its own."""
    g = torch.Generator().manual_seed(int(case["batch"]) * 1009 + int(case["kv_hi"]))
    qo = _whole(g, case["qo_lo"], case["qo_hi"], case["batch"])
    kv = qo if case["kv_hi"] == 0 else torch.maximum(_whole(g, case["kv_lo"], case["kv_hi"], case["batch"]), qo)
    return qo, kv


def _table_lengths(case):
    """(new tokens, cached tokens) of the batch that tables are built for: `prompts` of them start from nothing."""
    g = torch.Generator().manual_seed(int(case["batch"]) * 1013 + int(case["kv_hi"]))
    B, n = int(case["batch"]), int(case["prompts"])
    kv = _whole(g, min(case["kv_lo"], case["kv_hi"]), case["kv_hi"], B)
    qo = _whole(g, case["qo_lo"], case["qo_hi"] if not n else case["qo_lo"], B)
    if n:
        first = torch.randperm(B, generator=g)[:n]
        kv[first] = 0
        qo[first] = _whole(g, 1, case["qo_hi"], n)
    return qo, kv


def _indptr(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)])


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    g, _ = _generators(seed)
    qo, kv = _table_lengths(case)
    # which request has which length is the seed's; how many tokens and pages there are in all is the case's
    order = torch.randperm(case["batch"], generator=g)
    qo, kv, page = qo[order], kv[order], case["page"]
    old, new = (kv + page - 1) // page, (kv + qo + page - 1) // page
    total, T = int(new.sum()), int(qo.sum())
    width = int(new.max()) + 3
    num_pages = total + 64
    ids = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32)
    held = torch.arange(width)[None, :] < old[:, None]
    table[held] = ids[: int(old.sum())]
    free = ids[int(old.sum()):]
    s = {"op": "tables", "page": page, "num_pages": num_pages, "max_tokens": T + case["pad"], "max_pages": total + 32,
         "qo_lens": qo.to(torch.int32).cuda(), "kv_lens": kv.to(torch.int32).cuda(), "block_table": table.cuda(),
         "free_pages": free.cuda(), "free_count": torch.tensor([len(free)], dtype=torch.int32).cuda()}
    if own:
        import attention_paged_kv_gb300 as pa

        s["tables"] = pa.BatchTables(case["batch"], s["max_tokens"], s["max_pages"], page, num_pages)
    return s


def _prepare_append(case, seed):
    g, gc = _generators(seed)
    n, h, d = case["rows"] + case["pad"], case["heads"], case["dim"]
    # K and V are slices of the fused projection's output, behind the query heads
    qkv = torch.randn((n, h * (case["group"] + 2) * d), generator=gc, device="cuda").to(DTYPES[case["dtype"]])
    at = h * case["group"] * d
    k, v = qkv[:, at: at + h * d].view(n, h, d), qkv[:, at + h * d:].view(n, h, d)
    slots = torch.full((n,), -1, dtype=torch.int64)  # the rows behind the last sequence have no slot
    slots[: case["rows"]] = torch.randperm(case["pages"] * case["page"], generator=g)[: case["rows"]]
    s = {"op": "append", "page": case["page"], "k": k, "v": v, "slots": slots.cuda(), "layout": case["layout"],
         "k_scale": 0.5, "v_scale": 1.0, **_empty_cache(case["pages"], case["page"], h, d, case["layout"]),
         "k_values": torch.zeros(k.shape, dtype=k.dtype, device="cuda"),
         "v_values": torch.zeros(v.shape, dtype=v.dtype, device="cuda")}
    if own:
        import attention_paged_kv_gb300 as pa

        s["cache"] = pa.Kv4Cache(case["pages"], case["page"], h, d, kv_layout=case["layout"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], codes=s["codes"], scales=s["scales"])
    return s


def _empty_cache(pages, page, heads, dim, layout):
    mid = (page, heads) if layout == "NHD" else (heads, page)
    return {"codes": torch.zeros((pages, 2, *mid, dim // 2), dtype=torch.uint8, device="cuda"),
            "scales": torch.full((pages, 2, *mid, dim // GROUP), NEVER_WRITTEN, dtype=torch.uint8, device="cuda")}


def _prepare_attend(case, seed):
    g, gc = _generators(seed)
    qo, kv = _lengths(case)
    page, h, d, B = case["page"], case["kv_heads"], case["dim"], case["batch"]
    pages = (kv + page - 1) // page
    qo_indptr, page_indptr = _indptr(qo), _indptr(pages)
    n, T = int(page_indptr[-1]), int(qo_indptr[-1])
    num_pages = n + 7
    ids = torch.randperm(num_pages, generator=g)[:n]
    last = kv - (pages - 1) * page
    s = {"op": "attend", "page": page, "layout": case["layout"], "k_scale": 0.5, "v_scale": 2.0,
         "max_qo": int(qo.max()), "max_kv": int(kv.max()),
         **_empty_cache(num_pages, page, h, d, case["layout"]),
         "q": torch.randn((T, case["heads"], d), generator=gc, device="cuda").to(DTYPES[case["dtype"]]),
         "qo_indptr": qo_indptr.to(torch.int32).cuda(), "kv_page_indptr": page_indptr.to(torch.int32).cuda(),
         "kv_page_indices": ids.to(torch.int32).cuda(), "kv_last_page_len": last.to(torch.int32).cuda()}
    # every page in use holds quantised rows; slots behind a request's last key stay as never written
    filled = torch.full((num_pages,), 0, dtype=torch.int64)
    filled[ids] = page
    filled[ids[page_indptr[1:] - 1]] = last
    filled = filled.cuda()
    step = max(1, (1 << 26) // (2 * page * h * d))
    for at in range(0, num_pages, step):
        codes, scales = s["codes"][at: at + step], s["scales"][at: at + step]
        x = torch.randn((*codes.shape[:-1], d), generator=gc, device="cuda")
        c, sc = _quantise(x, 1.0)
        slot = torch.arange(page, device="cuda").view((1, 1, page, 1, 1) if case["layout"] == "NHD" else (1, 1, 1, page, 1))
        there = slot < filled[at: at + step].view(-1, 1, 1, 1, 1)
        codes.copy_(c)
        scales.copy_(torch.where(there, sc, NEVER_WRITTEN))
    if own:
        import attention_paged_kv_gb300 as pa

        s["cache"] = pa.Kv4Cache(num_pages, page, h, d, kv_layout=case["layout"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], codes=s["codes"], scales=s["scales"])
        s["attention"] = pa.Kv4Attention(B, T, case["heads"], h, d, page, DTYPES[case["dtype"]],
                                         max_qo_len=s["max_qo"])
    return s


# -------------------------------------------------------------------------------------------------------- one pass


def run(state):
    return {"tables": _run_tables, "append": _run_append, "attend": _run_attend}[state["op"]](state)


def _run_tables(s):
    if own:
        t = s["tables"]
        t.build(s["qo_lens"], s["kv_lens"], s["block_table"], s["free_pages"], s["free_count"])
        return {"block_table": s["block_table"], "qo_indptr": t.qo_indptr, "kv_page_indptr": t.kv_page_indptr,
                "kv_page_indices": t.kv_page_indices, "kv_last_page_len": t.kv_last_page_len, "kv_lens": t.kv_lens,
                "slot_mapping": t.slot_mapping, "positions": t.positions, "free_count": t.free_count}
    page = s["page"]
    qo, kv, free = s["qo_lens"].long(), s["kv_lens"].long(), s["free_count"].long()
    old, new = (kv + page - 1) // page, (kv + qo + page - 1) // page
    add = new - old
    first = torch.cumsum(add, 0) - add
    col = torch.arange(s["block_table"].shape[1], device=qo.device)
    taken = free - 1 - (first[:, None] + col - old[:, None])
    fresh = (col >= old[:, None]) & (col < new[:, None])
    page_of = s["free_pages"][taken.clamp(0, s["free_pages"].shape[0] - 1)]
    s["block_table"].copy_(torch.where(fresh, page_of, s["block_table"]))
    zero = torch.zeros(1, dtype=torch.int64, device=qo.device)
    qo_indptr, page_indptr = torch.cat([zero, torch.cumsum(qo, 0)]), torch.cat([zero, torch.cumsum(new, 0)])

    def spread(indptr, n):
        at = torch.arange(n, device=qo.device)
        req = torch.searchsorted(indptr[1:], at, right=True).clamp(max=qo.shape[0] - 1)
        return req, at - indptr[req], at < indptr[-1]

    req, nth, there = spread(page_indptr, s["max_pages"])
    indices = torch.where(there, s["block_table"][req, torch.where(there, nth, 0)], -1)
    req, nth, there = spread(qo_indptr, s["max_tokens"])
    pos = torch.where(there, kv[req] + nth, 0)
    slots = torch.where(there, s["block_table"][req, pos // page].long() * page + pos % page, -1)
    as32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"block_table": s["block_table"], "qo_indptr": as32(qo_indptr), "kv_page_indptr": as32(page_indptr),
            "kv_page_indices": as32(indices), "kv_last_page_len": as32(torch.where(new > 0, kv + qo - (new - 1) * page, 0)),
            "kv_lens": as32(kv + qo), "slot_mapping": slots, "positions": as32(pos), "free_count": as32(free - add.sum())}


def _quantise(x, g):
    """Codes (two to a byte, the even element low) and e4m3 scale bytes of x in blocks of 16, every step in 32 bits."""
    x = x.float().unflatten(-1, (-1, GROUP))
    amax = x.abs().amax(-1)
    s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    per = (s.float() * g)[..., None]
    y = torch.where(per > 0, x / per, 0.0)
    a = y.abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, halfway values to the even code, beyond 6 to 6
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _values(codes, scales):
    """What codes and scale bytes stand for, in 32 bits (without the cache's scales of K and V)."""
    pairs = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], dtype=torch.float32).to(codes.device, non_blocking=True)
    x = pairs[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _rows(cache, half, page, slot, layout):
    """The rows [..., heads, bytes] of the given pages and slots of one half of the cache."""
    return cache[page, half, slot] if layout == "NHD" else cache[page, half, :, slot]


def _run_append(s):
    if own:
        s["cache"].append(s["k"], s["v"], s["slots"], k_values=s["k_values"], v_values=s["v_values"])
        return {"k_values": s["k_values"], "v_values": s["v_values"], "codes": s["codes"],
                "scales": s["scales"].view(torch.float8_e4m3fn)}
    codes, scales, ok = s["codes"], s["scales"], s["slots"] >= 0
    at = torch.where(ok, s["slots"], s["slots"][0])  # a row without a slot repeats the first row
    page, slot = at // s["page"], at % s["page"]
    out = {}
    for half, name in enumerate("kv"):
        g = s[name + "_scale"]
        x = torch.where(ok[:, None, None], s[name], s[name][:1])
        c, sc = _quantise(x, g)
        if s["layout"] == "NHD":
            codes[page, half, slot], scales[page, half, slot] = c, sc
        else:
            codes[page, half, :, slot], scales[page, half, :, slot] = c, sc
        out[name + "_values"] = torch.where(ok[:, None, None], (_values(c, sc) * g).to(x.dtype), s[name + "_values"])
    return {**out, "codes": codes, "scales": scales.view(torch.float8_e4m3fn)}


def _run_attend(s):
    if own:
        out, lse = s["attention"].run(s["q"], s["cache"], (s["qo_indptr"], s["kv_page_indptr"], s["kv_page_indices"],
                                                           s["kv_last_page_len"]))
        return {"out": out, "lse": lse}
    q, page, dev = s["q"], s["page"], s["q"].device
    T, Hq, D = q.shape
    qo = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    pages = (s["kv_page_indptr"][1:] - s["kv_page_indptr"][:-1]).long()
    kv = (pages - 1) * page + s["kv_last_page_len"]
    t = torch.arange(s["max_kv"], device=dev)
    there = t < kv[:, None]  # [B, keys]
    nth = torch.where(there, s["kv_page_indptr"][:-1, None] + t // page, 0)
    at, slot = s["kv_page_indices"][nth].long(), (t % page).expand(there.shape)
    k, v = (_values(_rows(s["codes"], half, at, slot, s["layout"]), _rows(s["scales"], half, at, slot, s["layout"]))
            for half in (0, 1))  # [B, keys, Hkv, D]
    v = torch.where(there[..., None, None], v, 0.0)
    Hkv = k.shape[2]
    i = torch.arange(s["max_qo"], device=dev)
    row = torch.where(i < qo[:, None], s["qo_indptr"][:-1, None] + i, 0)
    qp = q.float()[row.long()].unflatten(2, (Hkv, Hq // Hkv))  # [B, qo, Hkv, G, D]
    seen = (t <= (kv - qo)[:, None, None] + i[None, :, None]) & there[:, None, :]  # [B, qo, keys]
    z = torch.matmul(qp.permute(0, 2, 1, 3, 4).flatten(2, 3), k.permute(0, 2, 3, 1))  # [B, Hkv, qo * G, keys]
    z = z.mul_(s["k_scale"] / math.sqrt(D)).unflatten(2, (-1, Hq // Hkv))
    z = z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(m > -math.inf, m, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (-1, Hq // Hkv))
    o = o * (s["v_scale"] / torch.where(total > 0, total, 1.0))
    lse = (m + total.log())[..., 0]
    # back from [B, Hkv, qo, G, ...] to the packed rows
    req = torch.searchsorted(s["qo_indptr"][1:].long(), torch.arange(T, device=dev), right=True)
    nth = torch.arange(T, device=dev) - s["qo_indptr"][req]
    return {"out": o[req, :, nth].flatten(1, 2).to(q.dtype), "lse": lse[req, :, nth].flatten(1, 2)}


# ------------------------------------------------------------------------------------------- what a pass cannot avoid


def work(case):
    if case["op"] == "tables":
        qo, kv = _table_lengths(case)
        page = case["page"]
        old, new = (kv + page - 1) // page, (kv + qo + page - 1) // page
        pages, T = int(new.sum()), int(qo.sum()) + case["pad"]
        fresh = pages - int(old.sum())
        # lengths and held pages read, free pages read and entered; packed pages, slots, positions and lengths written
        return {"bytes": 8 * len(qo) + 4 * (pages - fresh) + 8 * fresh + 4 * pages + 12 * T + 16 * len(qo),
                "flops": 10 * (pages + T)}
    if case["op"] == "append":
        n = case["rows"] * 2 * case["heads"] * case["dim"]
        return {"bytes": 2 * n + n // 2 + n // GROUP + 2 * n + 8 * (case["rows"] + case["pad"]), "flops": 6 * n}
    qo, kv = (x.double() for x in _lengths(case))
    D, T = case["dim"], float(qo.sum())
    pairs = float((qo * kv - qo * (qo - 1) / 2).sum()) * case["heads"]
    cache = float(kv.sum()) * case["kv_heads"] * 2 * (D // 2 + D // GROUP)
    return {"bytes": cache + T * case["heads"] * (4 * D + 4) + 4 * float(kv.sum()) / case["page"], "flops": 4 * D * pairs}


# ------------------------------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s)


def _exact_append(s):
    out = {"codes": None, "scales": None}
    # the e4m3 values of finite scales, from the format's definition: 4 exponent bits of bias 7, 3 of mantissa
    scale_of = torch.tensor([(b % 8) / 8 * 2.0 ** -6 if b < 8 else (1 + b % 8 / 8) * 2.0 ** (b // 8 - 7) for b in range(127)],
                            dtype=torch.float64, device="cuda")
    code_of = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")

    def nearest(a, grid):  # the nearest of the grid's values, halfway to the even index, beyond the last to it
        i = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
        lo, hi = a - grid[i - 1], grid[i] - a
        return torch.where((hi < lo) | ((hi == lo) & (i % 2 == 0)), i, i - 1)

    for name in "kv":
        x, g = s[name].double().unflatten(-1, (-1, GROUP)), float(s[name + "_scale"])
        sc = scale_of[nearest(x.abs().amax(-1) / 6 / g, scale_of)][..., None]
        q = code_of[nearest(torch.where(sc > 0, x.abs() / g / sc, 0.0), code_of)]
        value = (torch.sign(x) * q * sc * g).flatten(-2)
        out[name + "_values"] = torch.where((s["slots"] >= 0)[:, None, None], value, s[name + "_values"].double())
    return out


def _exact_attend(s):
    q = s["q"].double()
    T, Hq, D = q.shape
    code = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out, lse = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda"), torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    qo_indptr, page_indptr, last = (s[n].tolist() for n in ("qo_indptr", "kv_page_indptr", "kv_last_page_len"))
    codes, scales = s["codes"], s["scales"].view(torch.float8_e4m3fn)
    if s["layout"] == "HND":
        codes, scales = codes.transpose(2, 3), scales.view(torch.uint8).transpose(2, 3).contiguous().view(torch.float8_e4m3fn)
    for b in range(len(last)):
        r0, r1 = qo_indptr[b], qo_indptr[b + 1]
        ids = s["kv_page_indices"][page_indptr[b]: page_indptr[b + 1]].long()
        n = (len(ids) - 1) * s["page"] + last[b]
        if r1 == r0:
            continue
        c, sc = codes[ids].transpose(0, 1).flatten(1, 2)[:, :n], scales[ids].double().transpose(0, 1).flatten(1, 2)[:, :n]
        x = torch.stack([code[(c & 15).int()], code[(c >> 4).int()]], -1).flatten(-2) * sc.repeat_interleave(GROUP, -1)
        k, v = x[0] * s["k_scale"], x[1] * s["v_scale"]  # [n, Hkv, D]
        Hkv = k.shape[1]
        for a in range(r0, r1, 256):
            e = min(a + 256, r1)
            z = torch.einsum("ihgd,thd->hgit", q[a:e].unflatten(1, (Hkv, -1)), k) / math.sqrt(D)
            limit = n - (r1 - r0) + torch.arange(a - r0, e - r0, device="cuda")
            z.masked_fill_(torch.arange(n, device="cuda") > limit[:, None], -math.inf)
            lse[a:e] = torch.logsumexp(z, -1).permute(2, 0, 1).flatten(1)
            out[a:e] = torch.einsum("hgit,thd->ihgd", torch.softmax(z, -1), v).flatten(1, 2)
    return {"out": out, "lse": lse}
