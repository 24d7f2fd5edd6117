"""The operators of a serving step with block-sparse attention over a 16-bit paged KV cache, and the cases they are measured at.

Five operators, in the order in which such a step calls them:

  rope    rotary positions of q and k, one position a token or one for each axis (time, height, width); with `inverse` the
          rotation back, which is its gradient
  append  the step's new K and V rows into the paged cache, k rotated on the way and q beside it
  bounds  the largest and smallest value of each of a page's key channels, in 8 bits, for the pages that the step wrote to
  select  the pages that a query attends to: first and last ones, and those whose bounds allow the largest scores
  attend  attention of each query over the pages selected for it

Each has its plain form here (elementary torch operations in 32 bits, angles in 64) and, with `own`, the framework's call.
"""
import math

import torch

own = False  # False: run() computes the plain forms; True: it calls the framework

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
BASE = 500000.0  # of the rotary frequencies: long contexts


# --------------------------------------------------------------------------------------------------------- the cases


def listed():
    return [
        # a decode step's rows where another cache takes them: 64 requests, 64 / 8 heads
        {"name": "rope decode 64", "op": "rope", "tokens": 64, "heads": 64, "kv_heads": 8, "dim": 128, "rotary": 128,
         "interleaved": False, "axes": 1, "far": 131072, "inverse": False, "dtype": "bf16"},
        # the gradient of q and k of a video: three axes, pairs side by side
        {"name": "rope video 12001 back", "op": "rope", "tokens": 12001, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": True, "axes": 3, "far": 4096, "inverse": True, "dtype": "bf16"},
        # one layer's rows of a decode step, as slices of the fused projection's output
        {"name": "append decode 64", "op": "append", "rows": 64, "pad": 0, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "axes": 1, "far": 131072, "page": 16, "pages": 4096, "layout": "NHD",
         "dtype": "bf16"},
        # one layer's rows of a long prompt with images, half of each head rotated, beside some padding
        {"name": "append prompt 16000", "op": "append", "rows": 16000, "pad": 384, "heads": 64, "kv_heads": 8, "dim": 128,
         "rotary": 64, "interleaved": False, "axes": 3, "far": 16384, "page": 64, "pages": 1024, "layout": "HND",
         "dtype": "bf16"},
        # a decode step of 256 requests: each of their last pages anew
        {"name": "bounds decode 256", "op": "bounds", "batch": 256, "qo_lo": 1, "qo_hi": 1, "kv_lo": 512, "kv_hi": 1024,
         "kv_heads": 8, "dim": 128, "page": 16, "layout": "NHD", "dtype": "bf16"},
        # prompts of up to 4000 tokens behind cached ones that end inside a page
        {"name": "bounds prompts 8", "op": "bounds", "batch": 8, "qo_lo": 1001, "qo_hi": 4000, "kv_lo": 1, "kv_hi": 500,
         "kv_heads": 8, "dim": 128, "page": 32, "layout": "HND", "dtype": "fp16"},
        # the smallest server: one request of some length
        {"name": "select 1x5000", "op": "select", "batch": 1, "qo_lo": 1, "qo_hi": 1, "kv_lo": 5000, "kv_hi": 5000,
         "heads": 8, "kv_heads": 1, "dim": 128, "page": 16, "blocks": 64, "first": 1, "last": 2, "dtype": "fp16"},
        # 64 requests of 512 to 8192 keys
        {"name": "select decode 64", "op": "select", "batch": 64, "qo_lo": 1, "qo_hi": 1, "kv_lo": 512, "kv_hi": 8192,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "blocks": 128, "first": 1, "last": 4, "dtype": "bf16"},
        # a prompt's chunk of 2000 tokens behind 6000 cached ones: each token selects for itself
        {"name": "select chunk 2000", "op": "select", "batch": 1, "qo_lo": 2000, "qo_hi": 2000, "kv_lo": 8000,
         "kv_hi": 8000, "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "blocks": 128, "first": 1, "last": 4,
         "dtype": "bf16"},
        # few requests of very long context: 4096 keys of up to 131071
        {"name": "attend long 3", "op": "attend", "batch": 3, "qo_lo": 1, "qo_hi": 1, "kv_lo": 60001, "kv_hi": 131071,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "blocks": 64, "layout": "HND", "dtype": "bf16"},
        # the decode step of 64 requests: 2048 keys each, where they have as many
        {"name": "attend decode 64", "op": "attend", "batch": 64, "qo_lo": 1, "qo_hi": 1, "kv_lo": 512, "kv_hi": 8192,
         "heads": 64, "kv_heads": 8, "dim": 128, "page": 16, "blocks": 128, "layout": "NHD", "dtype": "bf16"},
        # a prompt's chunk: each of its tokens with pages of its own
        {"name": "attend chunk 1000", "op": "attend", "batch": 1, "qo_lo": 1000, "qo_hi": 1000, "kv_lo": 8000,
         "kv_hi": 8000, "heads": 64, "kv_heads": 8, "dim": 128, "page": 32, "blocks": 64, "layout": "NHD",
         "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "bounds", "select", "select", "attend", "attend", "attend"))
    dim, dtype, layout = rng.choice((64, 128, 128, 256)), rng.choice(("fp16", "bf16")), rng.choice(("NHD", "HND"))
    kv_heads, group = rng.choice((1, 2, 3, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16))
    page = rng.choice((8, 16, 16, 32, 64, 128))
    turn = {"rotary": rng.choice((dim, dim, dim // 2, dim // 4)), "interleaved": rng.random() < 0.4,
            "axes": rng.choice((1, 1, 2, 3)), "far": _spread(rng, 64, 1_000_000)}
    if op == "rope":
        return {"op": op, "tokens": _spread(rng, 1, 8000), "heads": kv_heads * group, "kv_heads": kv_heads,
                "dim": rng.choice((dim, 96)) if turn["rotary"] < 96 else dim, **turn, "inverse": rng.random() < 0.5,
                "dtype": dtype}
    if op == "append":
        return {"op": op, "rows": _spread(rng, 1, 8000), "pad": rng.randint(0, 100), "heads": kv_heads * group,
                "kv_heads": kv_heads, "dim": dim, **turn, "page": page, "pages": 65536 // page, "layout": layout,
                "dtype": dtype}
    if op == "bounds":
        hi = _spread(rng, 1, 2000)
        return {"op": op, "batch": _spread(rng, 1, max(1, min(256, 16000 // hi))), "qo_lo": 1, "qo_hi": hi, "kv_lo": 0,
                "kv_hi": _spread(rng, 1, 1000), "kv_heads": kv_heads, "dim": dim, "page": min(page, 64),
                "layout": layout, "dtype": dtype}
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}
    keys = _spread(rng, 256, 4096)  # to attend to
    if rng.random() < 0.65:  # a decode step, or drafts
        hi = _spread(rng, 32 * page if op == "select" else 16, 100_000)
        qo = rng.choice((1, 1, 1, 4))
        most = min(1_000_000_000 // (hi * kv_heads * dim), 500_000_000 // (keys * kv_heads * dim * qo))
        batch = _spread(rng, 1, max(1, min(128, most)))
        case.update(batch=batch, qo_lo=1, qo_hi=qo, kv_lo=max(qo, hi // rng.randint(1, 3 if op == "select" else 16)), kv_hi=hi)
    else:  # chunks of prompts
        qo = _spread(rng, 33, 1500)
        qo = min(qo, max(33, 2_000_000_000 // (2 * max(keys, 4 * page) * kv_heads * dim)))
        hi = qo + _spread(rng, 32 * page if op == "select" else 1, 8000)
        case.update(batch=rng.randint(1, 2), qo_lo=max(1, qo // 2), qo_hi=qo, kv_lo=max(qo, hi // 2), kv_hi=hi)
    if op == "attend":
        return {**case, "blocks": max(4, keys // page), "layout": layout}
    blocks = max(4, min(keys, hi // 4) // page)  # of a quarter of the longest request's pages at most
    first = rng.randint(0, 1)
    return {**case, "blocks": blocks, "first": first, "last": rng.randint(1, min(8, blocks - first - 1))}


# ------------------------------------------------------------------------------------------------- lengths and inputs


def _generators(seed, device="cuda"):
    return torch.Generator().manual_seed(int(seed)), torch.Generator(device=device).manual_seed(int(seed))


def _whole(g, lo, hi, n):
    return torch.randint(int(lo), int(hi) + 1, (int(n),), generator=g)


def _lengths(case):
    """(query lengths, kv lengths with the new tokens): by the case alone, so that work() knows them."""
    g = torch.Generator().manual_seed(int(case["batch"]) * 1009 + int(case["kv_hi"]))
    qo, kv = _whole(g, case["qo_lo"], case["qo_hi"], case["batch"]), _whole(g, case["kv_lo"], case["kv_hi"], case["batch"])
    return (qo, kv + qo) if case["op"] == "bounds" else (qo, torch.maximum(kv, qo))


def _indptr(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n, 0)])


def _frequencies(case):
    """Radians a position of each pair, and the axis whose position turns it."""
    pairs = case["rotary"] // 2
    inv_freq = BASE ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    cut = [0, pairs // 4, pairs // 4 + 3 * pairs // 8] if case["axes"] == 3 else [0, pairs // 2][: case["axes"]]
    axes = sum((torch.arange(pairs) >= c).long() for c in cut) - 1
    return inv_freq, axes


def prepare(case, seed):
    made = {"rope": _prepare_rope, "append": _prepare_append, "bounds": _prepare_bounds, "select": _prepare_select,
            "attend": _prepare_attend}[case["op"]](case, seed)
    return {"op": case["op"], **made}


def _turned(case, n, g, gc):
    """q, k and v as slices of one projection's output, their positions and the frequencies."""
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    qkv = torch.randn((n, (h + 2 * hk) * d), generator=gc, device="cuda").to(DTYPES[case["dtype"]])
    s = {"q": qkv[:, : h * d].view(n, h, d), "k": qkv[:, h * d: (h + hk) * d].view(n, hk, d),
         "v": qkv[:, (h + hk) * d:].view(n, hk, d)}
    positions = torch.randint(0, case["far"], (case["axes"], n), generator=g, dtype=torch.int32)
    inv_freq, axes = _frequencies(case)
    s.update(positions=positions.cuda() if case["axes"] > 1 else positions[0].cuda(), inv_freq=inv_freq.cuda(),
             axes=axes.cuda(), interleaved=case["interleaved"])
    if own:
        import attention_paged_kv_gb300 as pa

        s["rope"] = pa.Rope(inv_freq, interleaved=case["interleaved"], axes=axes.tolist() if case["axes"] > 1 else None)
    return s


def _prepare_rope(case, seed):
    g, gc = _generators(seed)
    return {**_turned(case, case["tokens"], g, gc), "inverse": case["inverse"]}


def _prepare_append(case, seed):
    g, gc = _generators(seed)
    n, page = case["rows"] + case["pad"], case["page"]
    slots = torch.full((n,), -1, dtype=torch.int64)  # the rows behind the last sequence have no slot
    slots[: case["rows"]] = torch.randperm(case["pages"] * page, generator=g)[: case["rows"]]
    s = {**_turned(case, n, g, gc), "page": page, "layout": case["layout"], "slots": slots.cuda(),
         "data": torch.zeros(_cache_shape(case, case["pages"]), dtype=DTYPES[case["dtype"]], device="cuda")}
    if own:
        import attention_paged_kv_gb300 as pa

        s["cache"] = pa.KvCache(case["pages"], page, case["kv_heads"], case["dim"], DTYPES[case["dtype"]],
                                kv_layout=case["layout"], data=s["data"])
    return s


def _cache_shape(case, num_pages):
    mid = (case["page"], case["kv_heads"]) if case.get("layout", "NHD") == "NHD" else (case["kv_heads"], case["page"])
    return (num_pages, 2, *mid, case["dim"])


def _tables(case, g):
    """The batch's tables as BatchTables builds them, over permuted pages."""
    qo, kv = _lengths(case)
    page = case["page"]
    pages = (kv + page - 1) // page
    qo_indptr, page_indptr = _indptr(qo), _indptr(pages)
    n = int(page_indptr[-1])
    ids = torch.randperm(n + 7, generator=g)[:n]
    last = kv - (pages - 1) * page
    filled = torch.zeros(n + 7, dtype=torch.int64)  # slots in use of each page
    filled[ids] = page
    filled[ids[page_indptr[1:] - 1]] = last
    # the request of each token, its position, and the slot that it has
    req = torch.repeat_interleave(torch.arange(len(qo)), qo)
    pos = (kv - qo)[req] + torch.arange(len(req)) - qo_indptr[req]
    slots = ids[page_indptr[req] + pos // page] * page + pos % page
    as32 = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    tables = {"qo_indptr": as32(qo_indptr), "kv_page_indptr": as32(page_indptr), "kv_page_indices": as32(ids),
              "kv_last_page_len": as32(last)}
    return {"page": page, "layout": case.get("layout", "NHD"), "max_qo": int(qo.max()), "max_kv": int(kv.max()),
            **tables}, n + 7, filled.cuda(), req, pos, slots


def _fill(case, data, filled, gc):
    """Keys and values in the slots in use, NaN in the others, as memory never written may hold."""
    page, hnd = case["page"], case["layout"] == "HND"
    slot = torch.arange(page, device="cuda").view((1, 1, 1, page, 1) if hnd else (1, 1, page, 1, 1))
    step = max(1, (1 << 27) // (2 * page * case["kv_heads"] * case["dim"]))
    for at in range(0, data.shape[0], step):
        x = data[at: at + step]
        x.normal_(generator=gc)
        x.masked_fill_(slot >= filled[at: at + step].view(-1, 1, 1, 1, 1), math.nan)


def _prepare_bounds(case, seed):
    g, gc = _generators(seed)
    s, num_pages, filled, _, _, slots = _tables(case, g)
    h, d = case["kv_heads"], case["dim"]
    s.update(slots=slots.cuda(), data=torch.empty(_cache_shape(case, num_pages), dtype=DTYPES[case["dtype"]], device="cuda"),
             bounds=torch.zeros((num_pages, h, 2, d), dtype=torch.int8, device="cuda"),
             bound_scales=torch.zeros((num_pages, h), dtype=torch.float32, device="cuda"))
    _fill(case, s["data"], filled, gc)
    if own:
        s["cache"] = _own_cache(case, s)
    return s


def _own_cache(case, s):
    import attention_paged_kv_gb300 as pa

    return pa.KvCache(s["data"].shape[0], case["page"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]],
                      kv_layout=s["layout"], data=s["data"], bounds=s.get("bounds", False),
                      bound_scales=s.get("bound_scales"))


def _own_attention(case, s):
    import attention_paged_kv_gb300 as pa

    return pa.BlockAttention(case["batch"], s["q"].shape[0], case["heads"], case["kv_heads"], case["dim"], case["page"],
                             DTYPES[case["dtype"]], case["blocks"], s["max_kv"], first=case.get("first", 1),
                             last=case.get("last", 1))


def _prepare_select(case, seed):
    g, gc = _generators(seed)
    s, num_pages, _, req, _, _ = _tables(case, g)
    h, d, dtype = case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    s.update(q=torch.randn((len(req), case["heads"], d), generator=gc, device="cuda").to(dtype), blocks=case["blocks"],
             first=case["first"], last=case["last"],
             data=torch.empty(_cache_shape(case, num_pages), dtype=dtype, device="cuda"),
             bounds=torch.empty((num_pages, h, 2, d), dtype=torch.int8, device="cuda"),
             bound_scales=torch.empty((num_pages, h), dtype=torch.float32, device="cuda"))
    # the bounds of keys that lie around a centre of their page's own
    step = max(1, (1 << 26) // (h * d))
    for at in range(0, num_pages, step):
        n = min(step, num_pages - at)
        centre, reach = torch.randn((2, n, h, d), generator=gc, device="cuda")
        reach = (1.8 + 0.4 * reach).clamp_min_(0.1)  # of about `page` rows of a normal distribution
        codes, scales = _codes((centre + reach).to(dtype).float(), (centre - reach).to(dtype).float())
        s["bounds"][at: at + n], s["bound_scales"][at: at + n] = codes, scales
    if own:
        s["cache"], s["attention"] = _own_cache(case, s), _own_attention(case, s)
    return s


def _prepare_attend(case, seed):
    g, gc = _generators(seed)
    s, num_pages, filled, req, pos, _ = _tables(case, g)
    dtype, n = DTYPES[case["dtype"]], case["blocks"]
    s.update(q=torch.randn((len(req), case["heads"], case["dim"]), generator=gc, device="cuda").to(dtype),
             data=torch.empty(_cache_shape(case, num_pages), dtype=dtype, device="cuda"))
    _fill(case, s["data"], filled, gc)
    # the first block, the query's own, and others by chance; in ascending order, -1 behind them
    own_block = (pos // case["page"]).cuda()[:, None, None]
    most = int(own_block.max()) + 1
    col = torch.arange(most, device="cuda")
    lists = torch.full((len(req), case["kv_heads"], n), -1, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // (most * case["kv_heads"]))
    for at in range(0, len(req), step):
        b = own_block[at: at + step]
        luck = torch.rand((len(b), case["kv_heads"], most), generator=gc, device="cuda")
        luck = torch.where((col == 0) | (col == b), 2.0, torch.where(col > b, -1.0, luck))
        top, idx = luck.topk(min(n, most), dim=-1)
        idx = torch.where(top < 0, most, idx).sort(-1).values
        lists[at: at + step, :, : idx.shape[-1]] = torch.where(idx < most, idx, -1).to(torch.int32)
    s["lists"] = lists
    if own:
        s["cache"], s["attention"] = _own_cache(case, s), _own_attention(case, s)
    return s


# -------------------------------------------------------------------------------------------------------- one pass


def run(state):
    return {"rope": _run_rope, "append": _run_append, "bounds": _run_bounds, "select": _run_select,
            "attend": _run_attend}[state["op"]](state)


def _turn(s, x, inverse=False):
    positions = s["positions"] if s["positions"].dim() == 2 else s["positions"][None]
    angle = positions[s["axes"]].t().double() * s["inv_freq"]  # [n, pairs]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sin = -sin
    r = 2 * s["axes"].shape[0]
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["interleaved"] else (y[..., : r // 2], y[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _run_rope(s):
    if own:
        q, k = s["rope"].apply(s["q"], s["k"], s["positions"], inverse=s["inverse"])
        return {"q": q, "k": k}
    return {"q": _turn(s, s["q"], s["inverse"]), "k": _turn(s, s["k"], s["inverse"])}


def _run_append(s):
    if own:
        q = s["cache"].append(s["k"], s["v"], s["slots"], rope=s["rope"], positions=s["positions"], q=s["q"])
        return {"q": q, "data": s["data"]}
    ok = s["slots"] >= 0
    at = torch.where(ok, s["slots"], s["slots"][0])  # a row without a slot repeats the first row
    page, slot = at // s["page"], at % s["page"]
    k = _turn(s, s["k"])
    for half, x in ((0, k), (1, s["v"])):
        x = torch.where(ok[:, None, None], x, x[:1])
        if s["layout"] == "NHD":
            s["data"][page, half, slot] = x
        else:
            s["data"][page, half, :, slot] = x
    return {"q": _turn(s, s["q"]), "data": s["data"]}


def _codes(top, low):
    """8-bit codes [..., 2, dim] that enclose the largest and smallest values [..., dim], and their scale."""
    most = torch.maximum(top.abs(), low.abs()).amax(-1)
    per = torch.where(most > 0, 127.0 / most, 0.0)[..., None]
    codes = torch.stack([(top * per).ceil().clamp(max=127.0), (low * per).floor().clamp(min=-127.0)], -2)
    return codes.to(torch.int8), most / 127.0


def _run_bounds(s):
    if own:
        s["cache"].update_bounds(s["slots"])
        return {"bounds": s["bounds"], "bound_scales": s["bound_scales"]}
    page = s["slots"] // s["page"]
    end = torch.zeros(s["data"].shape[0], dtype=torch.int64, device=page.device)
    end = end.scatter_reduce(0, page, s["slots"] % s["page"] + 1, "amax")  # the slots up to the last one written
    keys = s["data"][page, 0]  # each new token's page; tokens of one page find the same
    keys = (keys.transpose(1, 2) if s["layout"] == "NHD" else keys).float()  # [n, heads, slots, dim]
    there = (torch.arange(s["page"], device=page.device) < end[page][:, None])[:, None, :, None]
    top, low = torch.where(there, keys, -math.inf).amax(2), torch.where(there, keys, math.inf).amin(2)
    s["bounds"][page], s["bound_scales"][page] = _codes(top, low)
    return {"bounds": s["bounds"], "bound_scales": s["bound_scales"]}


def _batch(s):
    """Of the padded batch [B, max_qo]: the packed rows, and the queries' positions (below 0: no query there)."""
    qo = (s["qo_indptr"][1:] - s["qo_indptr"][:-1]).long()
    pages = (s["kv_page_indptr"][1:] - s["kv_page_indptr"][:-1]).long()
    kv = (pages - 1) * s["page"] + s["kv_last_page_len"]
    i = torch.arange(s["max_qo"], device=qo.device)
    row = torch.where(i < qo[:, None], s["qo_indptr"][:-1, None] + i, 0).long()
    return row, torch.where(i < qo[:, None], (kv - qo)[:, None] + i, -1)


def _packed(s, x, T):
    """Rows [T, ...] of the padded batch's [B, max_qo, ...]."""
    t = torch.arange(T, device=x.device)
    req = torch.searchsorted(s["qo_indptr"][1:].long(), t, right=True)
    return x[req, t - s["qo_indptr"][req]]


def _tables_of(s):
    return s["qo_indptr"], s["kv_page_indptr"], s["kv_page_indices"], s["kv_last_page_len"]


def _run_select(s):
    if own:
        return {"blocks": s["attention"].select(s["q"], s["cache"], _tables_of(s))}
    page, q = s["page"], s["q"]
    T, Hkv = q.shape[0], s["bounds"].shape[1]
    # a group's heads as whole numbers of one power of two, their positive and negative parts summed, then in 8 bits
    x = q.float().unflatten(1, (Hkv, -1))
    x = torch.ldexp(x, 15 - torch.frexp(x.abs().amax((2, 3), keepdim=True)).exponent).round()
    parts = torch.stack([x.clamp(min=0.0).sum(2), x.clamp(max=0.0).sum(2)], 2).flatten(2)  # [T, Hkv, 2 * dim]
    most = parts.abs().amax(-1, keepdim=True)
    codes = (parts * torch.where(most > 0, 127.0 / most, 0.0)).round()
    row, pos = _batch(s)
    width = (s["max_kv"] + page - 1) // page
    col = torch.arange(width, device=q.device)
    own_block = torch.where(pos >= 0, pos // page, 0)[:, :, None, None]  # [B, qo, 1, 1]
    at = s["kv_page_indptr"][:-1, None] + col
    ids = s["kv_page_indices"][at.clamp(max=s["kv_page_indices"].shape[0] - 1).long()].long()  # [B, width]
    bounds = s["bounds"][ids].flatten(3).float().permute(0, 2, 3, 1)  # [B, Hkv, 2 * dim, width]
    z = torch.matmul(codes[row].transpose(1, 2), bounds).transpose(1, 2)  # whole numbers below 2^24: exact
    z = z * s["bound_scales"][ids].transpose(1, 2)[:, None]
    z = torch.where((col < s["first"]) | (col > own_block - s["last"]), math.inf, z)
    z = torch.where(col > own_block, -math.inf, z)
    take = min(s["blocks"], width)
    got = z.sort(dim=-1, descending=True, stable=True).indices[..., :take]
    got = torch.where(got <= own_block, got, width).sort(-1).values
    got = torch.nn.functional.pad(torch.where(got < width, got, -1), (0, s["blocks"] - take), value=-1)
    return {"blocks": _packed(s, got.to(torch.int32), T)}


def _run_attend(s):
    if own:
        out, lse = s["attention"].run(s["q"], s["cache"], _tables_of(s), s["lists"])
        return {"out": out, "lse": lse}
    q, page, lists = s["q"], s["page"], s["lists"].long()
    T, Hq, D = q.shape
    Hkv, n = lists.shape[1:]
    t = torch.arange(T, device=q.device)
    req = torch.searchsorted(s["qo_indptr"][1:].long(), t, right=True)
    _, pos = _batch(s)
    pos = pos[req, t - s["qo_indptr"][req]][:, None, None, None]
    ids = s["kv_page_indices"][(s["kv_page_indptr"][req][:, None, None] + lists).clamp(min=0).long()].long()
    head = torch.arange(Hkv, device=q.device)[None, :, None].expand_as(ids)
    seen = (lists[..., None] * page + torch.arange(page, device=q.device) <= pos) & (lists[..., None] >= 0)
    k, v = (s["data"][ids, half, :, head] if s["layout"] == "NHD" else s["data"][ids, half, head] for half in (0, 1))
    k, v, seen = k.flatten(2, 3).float(), v.flatten(2, 3).float(), seen.flatten(2)  # [T, Hkv, keys(, D)]
    v = torch.where(seen[..., None], v, 0.0)
    z = torch.matmul(q.float().unflatten(1, (Hkv, -1)), k.transpose(2, 3)) / math.sqrt(D)
    z = torch.where(seen[:, :, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = (z - m).exp()
    total = p.sum(-1, keepdim=True)
    return {"out": (torch.matmul(p, v) / total).flatten(1, 2).to(q.dtype), "lse": (m + total.log())[..., 0].flatten(1)}


# ------------------------------------------------------------------------------------------- what a pass cannot avoid


def work(case):
    D, op = case["dim"], case["op"]
    if op in ("rope", "append"):
        n = case["tokens"] if op == "rope" else case["rows"]
        values = n * (case["heads"] + case["kv_heads"]) * D
        copied = n * case["kv_heads"] * D if op == "append" else 0
        # each row read and written, one position for each axis, a slot; two products and a sum a rotated value
        return {"bytes": 4 * (values + copied) + n * 4 * case["axes"] + (8 * n if copied else 0),
                "flops": 3 * n * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    qo, kv = (x.double() for x in _lengths(case))
    page, Hkv = case["page"], case["kv_heads"]
    if op == "bounds":
        # the keys of the pages written to, up to the last new one; codes and scales of those pages
        first = ((kv - qo) // page).floor()
        keys, pages = float((kv - first * page).sum()), float((((kv - 1) // page).floor() - first + 1).sum())
        return {"bytes": keys * Hkv * D * 2 + pages * Hkv * (2 * D + 4) + 8 * float(qo.sum()), "flops": 2 * keys * Hkv * D}
    # of each query: the blocks it sees, and how many of them it attends to
    seen = [torch.div(torch.arange(int(k - q), int(k), dtype=torch.float64), page, rounding_mode="floor") + 1 for q, k in zip(qo, kv)]
    T = float(qo.sum())
    if op == "select":
        pages = sum(float(x[-1]) for x in seen)
        return {"bytes": pages * Hkv * (2 * D + 4) + 4 * pages + T * (case["heads"] * D * 2 + Hkv * case["blocks"] * 4),
                "flops": 4 * D * Hkv * sum(float(x.sum()) for x in seen)}
    keys, read = 0.0, 0.0
    for x, k, q in zip(seen, kv, qo):
        own_keys = torch.arange(int(k - q), int(k), dtype=torch.float64) - (x - 1) * page + 1  # of the query's own block
        mine = float(((x.clamp(max=case["blocks"]) - 1) * page + own_keys).sum())
        keys, read = keys + mine, read + min(mine, float(k))
    return {"bytes": read * Hkv * D * 4 + T * case["heads"] * (4 * D + 4) + T * Hkv * case["blocks"] * 4,
            "flops": 4 * D * keys * case["heads"]}


# ------------------------------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "bounds": _exact_bounds, "attend": _exact_attend}[case["op"]](s)


def _exact_turn(s, x, sign=1.0):
    """Each pair as a complex number, times e^(i angle)."""
    positions = s["positions"].reshape(-1, x.shape[0]).double()
    angle = torch.stack([positions[a] * w for a, w in zip(s["axes"].tolist(), s["inv_freq"].tolist())], 1)
    pairs = angle.shape[1]
    y = x.double().clone()
    real = torch.arange(pairs, device=x.device) * (2 if s["interleaved"] else 1)
    imag = real + (1 if s["interleaved"] else pairs)
    z = torch.complex(y[..., real], y[..., imag]) * torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    y[..., real], y[..., imag] = z.real, z.imag
    return y


def _exact_rope(s):
    sign = -1.0 if s["inverse"] else 1.0
    return {"q": _exact_turn(s, s["q"], sign), "k": _exact_turn(s, s["k"], sign)}


def _exact_append(s):
    data, there = s["data"].double(), s["slots"] >= 0
    at = s["slots"][there]
    flat = data if s["layout"] == "NHD" else data.transpose(2, 3)
    for half, x in ((0, _exact_turn(s, s["k"])), (1, s["v"].double())):
        flat[at // s["page"], half, at % s["page"]] = x[there]
    return {"q": _exact_turn(s, s["q"]), "data": data}


def _exact_bounds(s):
    """The scales: the largest magnitude of a page's keys over 127.  (The codes are whole numbers.)"""
    scales = s["bound_scales"].double()
    keys = s["data"][:, 0] if s["layout"] == "HND" else s["data"][:, 0].transpose(1, 2)
    page, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    end = torch.full((scales.shape[0],), -1, device=page.device).scatter_reduce(0, page, slot, "amax")
    for at in range(s["page"]):
        there = end >= at
        scales[there] = torch.maximum(scales[there], keys[there, :, at].double().abs().amax(-1) / 127)
    return {"bounds": None, "bound_scales": scales}


def _exact_attend(s):
    q = s["q"].double()
    T, Hq, D = q.shape
    Hkv, page = s["lists"].shape[1], s["page"]
    out, lse = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda"), torch.zeros((T, Hq), dtype=torch.float64, device="cuda")
    qo_indptr, page_indptr, last = (s[n].tolist() for n in ("qo_indptr", "kv_page_indptr", "kv_last_page_len"))
    data = s["data"] if s["layout"] == "HND" else s["data"].transpose(2, 3)  # [pages, 2, heads, slots, dim]
    for b in range(len(last)):
        r0, r1 = qo_indptr[b], qo_indptr[b + 1]
        ids = s["kv_page_indices"][page_indptr[b]: page_indptr[b + 1]].long()
        n = (len(ids) - 1) * page + last[b]
        for h in range(Hkv):
            k, v = (data[ids, half, h].flatten(0, 1)[:n].double() for half in (0, 1))
            mine = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for a in range(r0, r1, 256):
                e = min(a + 256, r1)
                # a dense attention whose mask says which pages are on the query's list
                on = torch.zeros((e - a, len(ids) + 1), dtype=torch.bool, device="cuda")
                on.scatter_(1, torch.where(s["lists"][a:e, h] >= 0, s["lists"][a:e, h].long(), len(ids)), True)
                see = on[:, :-1].repeat_interleave(page, 1)[:, :n]
                see &= torch.arange(n, device="cuda") <= (n - r1 + torch.arange(a, e, device="cuda"))[:, None]
                z = torch.einsum("igd,td->git", q[a:e, mine], k) / math.sqrt(D)
                z.masked_fill_(~see, -math.inf)
                lse[a:e, mine] = torch.logsumexp(z, -1).t()
                out[a:e, mine] = torch.einsum("git,td->igd", torch.softmax(z, -1), v)
    return {"out": out, "lse": lse}
