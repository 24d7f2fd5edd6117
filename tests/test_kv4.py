"""Device-built tables, the 4-bit cache and the attention over it, against the fp64 restatement in oracle/kv4.py."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4

pa = pytest.importorskip("attention_paged_kv_gb300")
from attention_paged_kv_gb300 import _binding as raw  # noqa: E402

gpu = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    import os
    if not os.path.exists(pa.LIB_PATH):
        from attention_paged_kv_gb300 import build
        build.build()


# ---------------------------------------------------------------- refusals (no kernel runs)

FAKE = 1 << 20  # an aligned address that no refused call reads


def refused(call, status, text):
    with pytest.raises(pa.PagedAttnError) as e:
        raw.check(call())
    assert e.value.status == status and text in str(e.value), str(e.value)


def tables_args(**kw):
    d = dict(qo_lens=FAKE, kv_lens=FAKE, block_table=FAKE, free_pages=FAKE, free_count=FAKE, block_table_stride=8,
             block_table_width=8, free_capacity=4, batch_size=2, page_size=16, num_pages=9)
    o = dict(qo_indptr=FAKE, kv_page_indptr=FAKE, new_page_indptr=FAKE, kv_page_indices=FAKE, kv_last_page_len=FAKE,
             kv_lens=FAKE, slot_mapping=FAKE, positions=FAKE, free_count=FAKE, status=FAKE, max_tokens=4, max_pages=4)
    for k, v in kw.items():
        (o if k.startswith("out_") else d)[k.removeprefix("out_")] = v
    return raw.TablesIn(**d), raw.TablesOut(**o)


@pytest.mark.parametrize("kw, status, text", [
    (dict(page_size=24), raw.PA_ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=256), raw.PA_ERR_UNSUPPORTED, "page_size"),
    (dict(batch_size=-1), raw.PA_ERR_INVALID_ARG, "negative"),
    (dict(block_table_stride=7), raw.PA_ERR_INVALID_ARG, "block_table_stride"),
    (dict(num_pages=0), raw.PA_ERR_INVALID_ARG, "num_pages"),
    (dict(qo_lens=None), raw.PA_ERR_INVALID_ARG, "NULL"),
    (dict(free_count=None), raw.PA_ERR_INVALID_ARG, "NULL"),
    (dict(out_status=None), raw.PA_ERR_INVALID_ARG, "NULL"),
    (dict(out_slot_mapping=FAKE + 4), raw.PA_ERR_INVALID_ARG, "8-byte"),
])
def test_tables_refusals(kw, status, text):
    i, o = tables_args(**kw)
    refused(lambda: pa.load().pagedattn_build_tables(ctypes.byref(i), ctypes.byref(o), None), status, text)


def cache_args(**kw):
    d = dict(codes=FAKE, scales=FAKE, num_pages=4, page_size=16, num_kv_heads=2, head_dim=128, kv_layout=0, k_scale=1.0,
             v_scale=1.0)
    return raw.Kv4CacheArgs(**{**d, **kw})


BAD_CACHE = [
    (dict(codes=None), raw.PA_ERR_INVALID_ARG, "codes"),
    (dict(scales=FAKE + 8), raw.PA_ERR_INVALID_ARG, "aligned"),
    (dict(head_dim=96), raw.PA_ERR_UNSUPPORTED, "head_dim"),
    (dict(page_size=12), raw.PA_ERR_UNSUPPORTED, "page_size"),
    (dict(num_kv_heads=0), raw.PA_ERR_INVALID_ARG, "num_kv_heads"),
    (dict(num_pages=0), raw.PA_ERR_INVALID_ARG, "num_pages"),
    (dict(kv_layout=2), raw.PA_ERR_UNSUPPORTED, "kv_layout"),
    (dict(k_scale=0.0), raw.PA_ERR_INVALID_ARG, "k_scale"),
    (dict(v_scale=float("nan")), raw.PA_ERR_INVALID_ARG, "k_scale"),
    (dict(v_scale=float("inf")), raw.PA_ERR_INVALID_ARG, "k_scale"),
]


@pytest.mark.parametrize("cache, rows, status, text", [(c, {}, s, t) for c, s, t in BAD_CACHE] + [
    ({}, dict(num_tokens=-1), raw.PA_ERR_INVALID_ARG, "num_tokens"),
    ({}, dict(dtype=7), raw.PA_ERR_UNSUPPORTED, "dtype"),
    ({}, dict(k=None), raw.PA_ERR_INVALID_ARG, "required"),
    ({}, dict(v=FAKE + 2), raw.PA_ERR_INVALID_ARG, "aligned"),
    ({}, dict(k_values=FAKE + 2), raw.PA_ERR_INVALID_ARG, "aligned"),
    ({}, dict(k_stride=255), raw.PA_ERR_INVALID_ARG, "strides"),
    ({}, dict(v_stride=260), raw.PA_ERR_INVALID_ARG, "strides"),
    ({}, dict(status=None), raw.PA_ERR_INVALID_ARG, "required"),
])
def test_append_refusals(cache, rows, status, text):
    c = cache_args(**cache)
    d = dict(k=FAKE, v=FAKE, k_stride=256, v_stride=256, k_values=None, v_values=None, slot_mapping=FAKE, status=FAKE,
             num_tokens=3, dtype=raw.PA_BF16)
    r = raw.Kv4Rows(**{**d, **rows})
    refused(lambda: pa.load().pagedattn_kv4_append(ctypes.byref(c), ctypes.byref(r), None), status, text)


@pytest.mark.parametrize("cache, batch, more, status, text", [(c, {}, {}, s, t) for c, s, t in BAD_CACHE] + [
    ({}, dict(num_qo_heads=3), {}, raw.PA_ERR_INVALID_ARG, "num_qo_heads"),
    ({}, dict(num_qo_heads=2 * 129), {}, raw.PA_ERR_UNSUPPORTED, "128"),
    ({}, dict(dtype=2), {}, raw.PA_ERR_UNSUPPORTED, "dtype"),
    ({}, dict(batch_size=-1), {}, raw.PA_ERR_INVALID_ARG, "negative"),
    ({}, dict(num_tokens=1 << 29), {}, raw.PA_ERR_UNSUPPORTED, "2^30"),
    ({}, {}, dict(workspace=None), raw.PA_ERR_INVALID_ARG, "workspace"),
    ({}, {}, dict(workspace=FAKE + 128), raw.PA_ERR_INVALID_ARG, "workspace"),
])
def test_attention_refusals(cache, batch, more, status, text):
    c = cache_args(**cache)
    d = dict(qo_indptr=FAKE, kv_page_indptr=FAKE, kv_page_indices=FAKE, kv_last_page_len=FAKE, batch_size=2,
             num_page_indices=8, num_tokens=2, max_qo_len=1, num_qo_heads=8, causal=1, dtype=raw.PA_FP16)
    b = raw.Kv4Batch(**{**d, **batch})
    m = {**dict(q=FAKE, out=FAKE, workspace=FAKE), **more}
    refused(lambda: pa.load().pagedattn_kv4_run(ctypes.byref(c), ctypes.byref(b), m["q"], 1024, m["out"], None,
                                                m["workspace"], 1 << 40, None), status, text)


# ---------------------------------------------------------------- tables


def make_tables(rng, B, page, qo, kv, slack=5):
    """Lengths, table, free stack of a batch whose held pages are permuted."""
    old, new = -(-kv // page), -(-(kv + qo) // page)
    width = max(1, int(new.max()) + 2) if B else 1
    ids = rng.permutation(int(new.sum()) + slack).astype(np.int32)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, : old[b]] = ids[at: at + old[b]]
        at += old[b]
    return table, ids[at:], len(ids)


def lens(rng, B, kind):
    if kind == "decode":
        return np.ones(B, np.int32), rng.integers(0, 300, B).astype(np.int32)
    if kind == "mixed":  # idle requests, new prompts, drafts
        qo = rng.choice([0, 1, 1, 4, 150], B).astype(np.int32)
        return qo, np.where(rng.random(B) < 0.3, 0, rng.integers(0, 500, B)).astype(np.int32)
    return np.zeros(B, np.int32), np.zeros(B, np.int32)


def check_tables(t, want, table, table_t, pad_pages):
    got = {n: getattr(t, n).cpu().numpy() for n in want}
    nnz, T = int(want["kv_page_indptr"][-1]), int(want["qo_indptr"][-1])
    for n in ("qo_indptr", "kv_page_indptr", "new_page_indptr", "kv_last_page_len", "kv_lens", "free_count"):
        np.testing.assert_array_equal(got[n].reshape(-1), np.atleast_1d(want[n]), err_msg=n)
    np.testing.assert_array_equal(got["kv_page_indices"][:nnz], want["kv_page_indices"])
    assert (got["kv_page_indices"][nnz:] == pad_pages).all()
    np.testing.assert_array_equal(got["slot_mapping"][:T], want["slot_mapping"])
    np.testing.assert_array_equal(got["positions"][:T], want["positions"])
    assert (got["slot_mapping"][T:] == -1).all() and (got["positions"][T:] == 0).all()
    np.testing.assert_array_equal(table_t.cpu().numpy(), table)


@gpu
@pytest.mark.parametrize("B, page, kind", [(0, 16, "none"), (1, 1, "mixed"), (1, 128, "decode"), (7, 16, "none"),
                                           (33, 4, "mixed"), (64, 16, "decode"), (257, 16, "mixed"), (1024, 2, "mixed"),
                                           (1025, 16, "mixed"), (2500, 64, "mixed"), (3000, 1, "decode")])
def test_tables_equal_restated(B, page, kind):
    rng = np.random.default_rng(B * 7 + page)
    qo, kv = lens(rng, B, kind)
    table, free, num_pages = make_tables(rng, B, page, qo, kv)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    wide = dev(np.concatenate([table, np.full((B, 3), -9, np.int32)], 1))  # rows of a wider table
    table_t = wide[:, : table.shape[1]]
    count = torch.tensor([len(free)], dtype=I32).cuda()
    need = int((-(-(kv + qo) // page)).sum())
    t = pa.BatchTables(B, int(qo.sum()) + 13, need + 4, page, num_pages)
    t.build(dev(qo), dev(kv), table_t, dev(free), count)
    want = kv4.tables(qo, kv, table, free, len(free), page)
    check_tables(t, want, table, table_t, -1)
    assert (wide[:, table.shape[1]:] == -9).all() and t.device_status() == 0 and int(count) == len(free)


@gpu
def test_tables_advance_in_place_over_replays():
    """A captured build whose lengths and free count are its own outputs: each replay is the next step."""
    rng = np.random.default_rng(5)
    B, page, steps = 40, 16, 40
    qo, kv = np.ones(B, np.int32), rng.integers(0, 60, B).astype(np.int32)
    table, free, num_pages = make_tables(rng, B, page, np.full(B, steps + 2, np.int32), kv)
    qo_t, table_t, free_t = (torch.from_numpy(a).cuda() for a in (qo, table.copy(), free))
    t = pa.BatchTables(B, B, num_pages, page, num_pages)
    t.kv_lens.copy_(torch.from_numpy(kv))
    t.free_count.fill_(len(free))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.build(qo_t, t.kv_lens, table_t, free_t, t.free_count)
    count = len(free)
    for _ in range(steps):
        t.kv_page_indices.fill_(-1)
        g.replay()
        want = kv4.tables(qo, kv, table, free, count, page)
        kv, count = want["kv_lens"].astype(np.int32), want["free_count"]
        check_tables(t, want, table, table_t, -1)
    assert t.device_status() == 0


@gpu
@pytest.mark.parametrize("B", [2000, 3500])  # several blocks of one launch, and two launches
def test_tables_in_place_with_many_blocks(B):
    rng = np.random.default_rng(B)
    page = 16
    qo, kv = rng.choice([0, 1, 30], B).astype(np.int32), rng.integers(0, 200, B).astype(np.int32)
    table, free, num_pages = make_tables(rng, B, page, 3 * qo, kv)
    t = pa.BatchTables(B, int(qo.sum()) + 100, num_pages, page, num_pages)
    t.kv_lens.copy_(torch.from_numpy(kv))
    t.free_count.fill_(len(free))
    qo_t, table_t, free_t = (torch.from_numpy(a).cuda() for a in (qo, table.copy(), free))
    count = len(free)
    for _ in range(3):
        t.kv_page_indices.fill_(-1)
        t.build(qo_t, t.kv_lens, table_t, free_t, t.free_count)
        want = kv4.tables(qo, kv, table, free, count, page)
        kv, count = want["kv_lens"].astype(np.int32), want["free_count"]
        check_tables(t, want, table, table_t, -1)
    assert t.device_status() == 0


@gpu
@pytest.mark.parametrize("B", [6, 1500, 3500])
@pytest.mark.parametrize("fault, flag", [("pages", 4), ("tokens", 8), ("lists", 8), ("width", 8), ("qo", 2), ("kv", 2),
                                         ("sum", 2), ("count", 2)])
def test_tables_all_or_nothing(B, fault, flag):
    rng = np.random.default_rng(3)
    page = 16
    qo, kv = rng.integers(1, 40, B).astype(np.int32), rng.integers(0, 90, B).astype(np.int32)
    table, free, num_pages = make_tables(rng, B, page, qo, kv)
    need = int((-(-(kv + qo) // page)).sum())
    T, nnz, count, width = int(qo.sum()), need, len(free), table.shape[1]
    if fault == "pages":
        count = int(need - (-(-kv // page)).sum()) - 1
    elif fault == "tokens":
        T -= 1
    elif fault == "lists":
        nnz -= 1
    elif fault == "width":
        width = int((-(-(kv + qo) // page)).max()) - 1
    elif fault == "qo":
        qo[B // 2] = -1
    elif fault == "kv":
        kv[B - 1] = -5
    elif fault == "sum":
        kv[0] = 2 ** 31 - 10
    elif fault == "count":
        count = len(free) + 1
    table_t = torch.from_numpy(table.copy()).cuda()
    t = pa.BatchTables(B, T, nnz, page, num_pages)
    t.kv_lens.copy_(torch.from_numpy(kv))
    t.free_count.fill_(count)
    t.build(torch.from_numpy(qo).cuda(), t.kv_lens, table_t[:, :width], torch.from_numpy(free).cuda(), t.free_count)
    assert t.device_status() == flag
    for n in ("qo_indptr", "kv_page_indptr", "new_page_indptr", "kv_last_page_len", "positions"):
        assert not getattr(t, n).any(), n
    assert (t.slot_mapping == -1).all() and (t.kv_page_indices == -1).all()
    np.testing.assert_array_equal(t.kv_lens.cpu().numpy(), kv)
    np.testing.assert_array_equal(table_t.cpu().numpy(), table)
    assert int(t.free_count) == count and t.device_status() == 0


@gpu
@pytest.mark.parametrize("B", [6, 3500])
def test_tables_without_room_for_anything(B):
    """Requests of no tokens and no pages need no lists; one with a token then fails the whole build."""
    z = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    t = pa.BatchTables(B, 0, 0, 16, 4)
    qo = z(B)
    t.build(qo, z(B), z(B, 1), z(0), z(1))
    assert t.device_status() == 0 and not t.qo_indptr.any() and not t.kv_lens.any()
    qo[3] = 1
    t.build(qo, z(B), z(B, 1), z(0), z(1))
    assert t.device_status() == raw.PA_DEV_NO_PAGES | raw.PA_DEV_NO_ROOM and not t.qo_indptr.any()


@gpu
def test_tables_bad_page_id():
    t = pa.BatchTables(2, 4, 8, 16, 10)
    dev = lambda *a: torch.tensor(a, dtype=I32).cuda()  # noqa: E731
    table = torch.tensor([[3, 10], [4, -1]], dtype=I32).cuda()
    t.build(dev(1, 1), dev(20, 3), table, dev(5, 6), dev(2))
    assert t.device_status() == pa.PA_DEV_BAD_INDEX
    assert t.slot_mapping.tolist() == [-1, 4 * 16 + 3, -1, -1] and t.positions.tolist() == [20, 3, 0, 0]


@gpu
def test_tables_python_refusals():
    t = pa.BatchTables(2, 4, 8, 16, 10)
    z = lambda *s: torch.zeros(s, dtype=I32).cuda()  # noqa: E731
    good = dict(qo_lens=z(2), kv_lens=z(2), block_table=z(2, 3), free_pages=z(4), free_count=z(1))
    t.build(**good)
    for name, bad in [("qo_lens", z(3)), ("kv_lens", z(2).long()), ("kv_lens", torch.zeros(2, dtype=I32)),
                      ("block_table", z(3, 2).t()), ("block_table", z(3, 3)), ("free_pages", z(8)[::2]),
                      ("free_count", z(2))]:
        with pytest.raises(pa.PagedAttnError):
            t.build(**{**good, name: bad})


# ---------------------------------------------------------------- append


def special_rows(rng, n, h, d, dtype):
    """Rows of ordinary values and of every case of the format, rounded to dtype."""
    x = rng.standard_normal((n, h, d))
    kind = rng.integers(0, 12, (n, h, d // 16))
    x = x.reshape(n, h, d // 16, 16)
    x[kind == 1] = 0.0
    x[kind == 2] = -0.0
    x[kind == 3] *= 1e-4                                   # the scale is a subnormal of e4m3, or 0
    x[kind == 4] *= 3000.0                                 # beyond 448 * 6: the scale saturates
    x[kind == 5] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -2.5, -5.0], x[kind == 5].shape)
    x[kind == 5, 0] = 6.0                                  # scale 1: every other value lies halfway
    x[kind == 6] = x[kind == 6].round() * 6 * 1.0625       # amax / 6 halfway between two scales
    x = x.reshape(n, h, d)
    t = torch.from_numpy(x).to(dtype)
    for value, at in ((float("nan"), 0), (float("inf"), 1), (-float("inf"), 2)):
        if n > at + 3:
            t[at + 3, h - 1, 16 + at] = value
    return t


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n, h, d, page, layout, scales", [
    (1, 1, 64, 1, "NHD", (1.0, 1.0)), (77, 3, 64, 16, "HND", (0.5, 2.0)), (130, 8, 128, 16, "NHD", (1.0, 0.25)),
    (9, 2, 256, 128, "HND", (1.0, 1.0)), (300, 1, 128, 4, "HND", (0.013, 0.77)), (65, 5, 256, 8, "NHD", (1e-3, 300.0))])
def test_append_equals_restated(dtype, n, h, d, page, layout, scales):
    rng = np.random.default_rng(n + d)
    pages = -(-n // page) + 3
    cache = pa.Kv4Cache(pages, page, h, d, layout, *scales)
    cache.codes.fill_(0xA5)
    cache.scales.fill_(0x5A)
    want = {"codes": cache.codes.cpu().numpy().copy(), "scales": cache.scales.cpu().numpy().copy()}
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[rng.random(n) < 0.2] = -1
    # slices of a wider buffer, with the token stride of a fused projection
    rows = [special_rows(rng, n, h, d, dtype) for _ in range(2)]
    fused = torch.cat([torch.randn(n, 8).to(dtype), rows[0].flatten(1), rows[1].flatten(1)], 1).cuda()
    k, v = fused[:, 8: 8 + h * d].view(n, h, d), fused[:, 8 + h * d:].view(n, h, d)
    out = [torch.full((n, h, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    cache.append(k, v, torch.from_numpy(slots).cuda(), k_values=out[0], v_values=out[1])
    assert cache.device_status() == 0
    live = slots >= 0
    for half in range(2):
        codes, sb, values = kv4.quantise(rows[half].double().numpy(), scales[half])
        for i in np.flatnonzero(live):
            p, s = divmod(int(slots[i]), page)
            at = (p, half, slice(None), s) if layout == "HND" else (p, half, s)
            want["codes"][at], want["scales"][at] = codes[i], sb[i]
        got = out[half].double().cpu().numpy()
        # a value is code * scale (exact) times g, rounded to fp32 and then to the type: bit-equal to numpy's
        ref = torch.from_numpy(np.float32(values)).to(dtype).double().numpy()
        np.testing.assert_array_equal(got[live], ref[live])
        assert (got[~live] == 7.0).all()
    np.testing.assert_array_equal(cache.scales.cpu().numpy(), want["scales"])
    np.testing.assert_array_equal(cache.codes.cpu().numpy(), want["codes"])


@gpu
@pytest.mark.parametrize("g", [1.0, 0.37, 1.7e-4, 913.0, 1.1e-15, 0.9e15])
def test_append_divides_as_the_device_does(g):
    """Millions of values of every size against the definition with the device's own fp32 divisions."""
    n, h, d = 4096, 4, 128
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((n, h, d), generator=gen, device="cuda") * torch.exp2(
        torch.randint(-14, 14, (n, h, d // 16, 1), generator=gen, device="cuda").float()).expand(-1, -1, -1, 16).reshape(n, h, d)
    x = x.bfloat16() * g if g < 1e-6 or g > 1e6 else x.bfloat16()  # values in the cache's range
    x = x.bfloat16()
    cache = pa.Kv4Cache(n // 16, 16, h, d, "NHD", g, 1.0)
    cache.append(x, x, torch.arange(n, device="cuda"))
    b = x.float().unflatten(-1, (-1, 16))
    six = torch.tensor(6.0, device="cuda") * torch.tensor(g, device="cuda", dtype=torch.float32)
    s = (b.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = (s.float() * torch.tensor(g, device="cuda", dtype=torch.float32))[..., None]
    y = torch.where(unit > 0, b / unit, 0.0)
    a = y.abs()
    code = sum(m.int() for m in (a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0))
    code = (code + 8 * torch.signbit(y).int()).flatten(-2)
    want = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    assert torch.equal(cache.scales[:, 0].reshape(n, h, -1), s.view(torch.uint8))
    assert torch.equal(cache.codes[:, 0].reshape(n, h, -1), want)


@gpu
def test_append_slots_out_of_range_and_empty():
    cache = pa.Kv4Cache(2, 16, 1, 64)
    k = torch.ones(3, 1, 64, dtype=torch.float16, device="cuda")
    cache.append(k, k, torch.tensor([32, 5, 1 << 40]).cuda())
    assert cache.device_status() == pa.PA_DEV_BAD_INDEX and cache.device_status() == 0
    written = (cache.codes != 0).any(-1).nonzero().tolist()
    assert written == [[0, 0, 5, 0], [0, 1, 5, 0]]
    cache.append(k[:0], k[:0], torch.zeros(0, dtype=torch.int64).cuda())
    good = torch.tensor([1, 2, 3]).cuda()
    for bad in [dict(k=k.float(), v=k.float()), dict(v=k.bfloat16()), dict(slot_mapping=good.int()),
                dict(k=k[:2]), dict(k=k.expand(3, 1, 64)[:, :, ::2]), dict(k_values=k.bfloat16()),
                dict(slot_mapping=good.cpu())]:
        with pytest.raises(pa.PagedAttnError):
            cache.append(**{**dict(k=k, v=k, slot_mapping=good), **bad})


@gpu
def test_append_rows_beyond_32_bit_offsets():
    """A cache of over 2^32 code bytes: rows at its ends."""
    pages, page, h, d = 530_000, 128, 1, 128  # 8.7 GB of codes
    cache = pa.Kv4Cache(pages, page, h, d)
    k = torch.randn(4, h, d, device="cuda").half()
    slots = torch.tensor([0, pages * page - 1, pages * page // 2, 1 << 26]).cuda()
    cache.append(k, -k, slots)
    codes, sb, _ = kv4.quantise(k.double().cpu().numpy(), 1.0)
    for i, s in enumerate(slots.tolist()):
        assert (cache.codes[s // page, 0, s % page].cpu().numpy() == codes[i]).all()
        assert (cache.scales[s // page, 1, s % page].cpu().numpy() == sb[i]).all()


# ---------------------------------------------------------------- attention


class Batch:
    """A batch over a 4-bit cache of quantised normal values; slots that no request uses hold NaN scales."""

    def __init__(self, qo, kv, Hq, Hkv, D, page, layout, dtype, seed=0, k_scale=0.5, v_scale=2.0, pad=0, q_gain=1.0):
        rng = np.random.default_rng(seed)
        qo, kv = np.asarray(qo), np.asarray(kv)
        self.hnd, self.page, self.D, self.Hkv = layout == "HND", page, D, Hkv
        pages = -(-kv // page)
        self.qo_indptr = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
        self.page_indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.where(pages > 0, kv - (pages - 1) * page, 0).astype(np.int32)
        num_pages = int(pages.sum()) + 3
        self.pages = rng.permutation(num_pages)[: int(pages.sum())].astype(np.int32)
        self.T = int(qo.sum()) + pad
        self.pad = pad
        mid = (Hkv, page) if self.hnd else (page, Hkv)
        codes = rng.integers(0, 256, (num_pages, 2, *mid, D // 2), dtype=np.uint8)
        scales = np.full((num_pages, 2, *mid, D // 16), 0x7F, np.uint8)
        for b in range(len(kv)):
            t = np.arange(kv[b])
            ids = self.pages[self.page_indptr[b] + t // page]
            for half in range(2):
                c, s, _ = kv4.quantise(rng.standard_normal((kv[b], Hkv, D)), 1.0)
                if self.hnd:
                    codes[ids, half, :, t % page], scales[ids, half, :, t % page] = c, s
                else:
                    codes[ids, half, t % page], scales[ids, half, t % page] = c, s
        self.codes, self.scales = codes, scales
        self.cache = pa.Kv4Cache(num_pages, page, Hkv, D, layout, k_scale, v_scale,
                                 codes=torch.from_numpy(codes).cuda(), scales=torch.from_numpy(scales).cuda())
        self.q = (torch.from_numpy(rng.standard_normal((self.T, Hq, D))) * q_gain).to(dtype).cuda()
        self.dtype, self.Hq, self.max_qo = dtype, Hq, int(qo.max()) if len(qo) else 0

    def tables(self):
        return tuple(torch.from_numpy(a).cuda() for a in (self.qo_indptr, self.page_indptr, self.pages, self.last))

    def attention(self, causal=True, max_qo=None, **kw):
        return pa.Kv4Attention(len(self.last), self.T, self.Hq, self.Hkv, self.D, self.page, self.dtype, causal,
                               self.max_qo if max_qo is None else max_qo, **kw)

    def want(self, causal=True):
        n = self.T - self.pad
        return kv4.attention(self.q[:n].double().cpu().numpy(), self.codes, self.scales, self.cache.k_scale,
                             self.cache.v_scale, self.qo_indptr, self.page_indptr, self.pages, self.last, self.page,
                             self.hnd, causal)

    def check(self, out, lse, want):
        """Error bounds of the kernels' arithmetic, from fp64 sums over each row's keys.

        logits  fp32 sums of exact products in D/16 steps, truncated at worst:
                ds = 2^-22 (D/16 + 2) sum |q k| scale
        p       exp2 and its argument: 2^-21, and ds; both in numerator and
                normaliser, hence twice
        P       rounded to fp16: 2^-11 of each p, and 2^-25 (of the largest
                p, 1 or more) where p is a subnormal of fp16
        out     half a step of its type
        lse     ds, 2^-21, the fp32 sum of n terms and the last roundings
        """
        n = self.T - self.pad
        ref, ref_lse, sp = want
        eps = torch.finfo(self.dtype).eps / 2
        ds = 2.0 ** -22 * (self.D / 16 + 2) * sp["s"]
        rel = 2 * (ds + 2.0 ** -21) + 2.0 ** -11
        bound = (rel[..., None] * sp["av"] + 2.0 ** -25 * sp["v"]) * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25
        err = np.abs(out[:n].double().cpu().numpy() - ref)
        assert (err <= bound).all(), (err / bound).max()
        got = lse[:n].double().cpu().numpy()
        none = np.isneginf(ref_lse)
        assert (np.isneginf(got) == none).all() and (err[none] == 0).all()
        bound = ds + 2.0 ** -20 + 2.0 ** -24 * (sp["n"] / 16 + 64) + 2.0 ** -22 * np.abs(np.where(none, 0, ref_lse))
        lerr = np.abs(np.where(none, 0, got) - np.where(none, 0, ref_lse))
        assert (lerr <= bound).all(), (lerr / bound).max()


SHAPES = [
    # qo, kv, Hq, Hkv, D, page, layout
    ([1], [1], 1, 1, 64, 16, "NHD"),
    ([1], [77], 8, 1, 128, 16, "NHD"),
    ([1, 1, 1], [16, 17, 15], 4, 4, 128, 16, "HND"),
    ([1] * 5, [1, 63, 64, 65, 1000], 8, 2, 64, 32, "HND"),
    ([1, 1], [2049, 300], 16, 2, 128, 64, "NHD"),
    ([1, 1, 1], [130, 5, 700], 4, 1, 256, 16, "NHD"),
    ([1, 1, 1], [130, 5, 700], 6, 2, 256, 128, "HND"),
    ([1] * 4, [33, 100, 7, 258], 6, 2, 128, 1, "NHD"),
    ([1] * 4, [33, 100, 7, 258], 10, 2, 64, 4, "HND"),
    ([1, 2, 3], [40, 41, 300], 7, 1, 128, 8, "NHD"),
    ([4, 4, 4], [4, 130, 1025], 8, 1, 128, 16, "HND"),     # 32 packed rows
    ([3, 1, 2], [3, 515, 64], 32, 2, 64, 16, "NHD"),
    ([0, 1, 0, 2, 0], [50, 60, 0, 70, 16], 4, 2, 128, 16, "NHD"),  # idle requests
    ([2, 1, 5], [0, 0, 3], 4, 2, 128, 16, "HND"),          # rows that see no key
    ([33, 5], [33, 700], 4, 4, 128, 16, "NHD"),
    ([40, 1], [200, 300], 8, 1, 64, 16, "HND"),
    ([17, 66], [90, 66], 8, 2, 256, 32, "NHD"),
    ([129, 300, 64], [129, 400, 1000], 8, 1, 128, 16, "NHD"),
    ([150, 1, 20], [777, 50, 20], 6, 2, 128, 4, "HND"),
    ([256, 9], [256, 256], 5, 1, 64, 128, "HND"),
]


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-%s-%d.%d.%d-p%d%s" % (
    "_".join(map(str, s[0])), "_".join(map(str, s[1])), *s[2:]))
def test_attention_equals_restated(shape, causal, dtype):
    b = Batch(*shape, dtype, seed=len(shape[0]) + shape[4], pad=3)
    out = torch.full((b.T, b.Hq, b.D), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((b.T, b.Hq), 9.0, device="cuda")
    a = b.attention(causal)
    a.run(b.q, b.cache, b.tables(), out=out, lse=lse)
    assert a.device_status() == 0
    b.check(out, lse, b.want(causal))
    assert (out[-3:] == 9.0).all() and (lse[-3:] == 9.0).all()  # rows behind the last sequence


@gpu
def test_attention_splits_of_long_requests():
    """One request over many slices, beside ones within a slice, at 1 and 2 kv heads."""
    for kv, Hkv in (([20_000], 1), ([9000, 3, 5000], 2), ([64 * 4 * 3, 64 * 4], 2)):
        b = Batch([1] * len(kv), kv, 8 * Hkv, Hkv, 128, 16, "NHD", torch.bfloat16, seed=3)
        a = b.attention()
        out, lse = a.run(b.q, b.cache, b.tables())
        b.check(out, lse, b.want())


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", [
    ([8], [5000], 8, 1, 128, 16, "NHD"),           # one row tile, cut along the keys, two states a part
    ([5, 33], [1100, 2900], 8, 2, 128, 64, "HND"),
    ([300], [2600], 4, 1, 128, 16, "NHD"),         # a pair of row tiles and an odd one
    ([40], [4100], 2, 1, 64, 16, "HND"),
    ([50], [3000], 3, 1, 256, 16, "NHD"),
    ([64, 1, 40], [64, 4000, 1300], 8, 2, 128, 16, "HND"),
], ids=str)
def test_attention_items_cut_along_the_keys(shape, dtype):
    """Few items of many keys: the prefill kernel cuts them and joins the parts, run after run in one workspace."""
    b = Batch(*shape, dtype, seed=31, pad=1)
    for causal in (True, False):
        a, want = b.attention(causal), b.want(causal)
        first = None
        for _ in range(3):
            out, lse = a.run(b.q, b.cache, b.tables())
            first = first or (out, lse)
            assert torch.equal(out[:-1], first[0][:-1]) and torch.equal(lse[:-1], first[1][:-1])
        b.check(out, lse, want)
        assert a.device_status() == 0


@gpu
def test_attention_one_workspace_for_several_shapes():
    """Runs of other shapes take turns in one workspace: each leaves its counters as it found them."""
    bs = [Batch([1, 1], [3000, 900], 8, 1, 128, 16, "NHD", torch.float16, seed=1),
          Batch([1] * 3, [2000, 100, 1500], 28, 7, 64, 16, "HND", torch.bfloat16, seed=2),
          Batch([40, 1], [2100, 1900], 16, 2, 128, 16, "NHD", torch.float16, seed=3),
          Batch([2], [1700], 6, 2, 256, 16, "NHD", torch.bfloat16, seed=4)]
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    objs = [b.attention(workspace=ws) for b in bs]
    want = [b.want() for b in bs]
    for _ in range(3):
        for b, a, w in zip(bs, objs, want):
            out, lse = a.run(b.q, b.cache, b.tables())
            b.check(out, lse, w)


@gpu
def test_attention_many_short_requests():
    rng = np.random.default_rng(1)
    kv = rng.integers(1, 90, 1300)
    b = Batch([1] * 1300, kv, 2, 1, 64, 16, "HND", torch.float16, seed=4)
    out, lse = b.attention().run(b.q, b.cache, b.tables())
    b.check(out, lse, b.want())


@gpu
@pytest.mark.parametrize("kv_hi, D", [(40, 64), (2500, 64), (60, 256)])
def test_attention_prompts_in_a_large_batch(kv_hi, D):
    """More requests than a block has threads, long chunks and single tokens among them (both kernels' longer scans)."""
    rng = np.random.default_rng(kv_hi)
    B = 700
    qo = np.where(rng.random(B) < 0.03, rng.integers(20, 40, B), rng.integers(0, 2, B))
    kv = qo + np.where(rng.random(B) < 0.02, kv_hi, rng.integers(0, 30, B))
    b = Batch(qo, kv, 4, 1, D, 16, "NHD", torch.bfloat16, seed=5)
    a = b.attention()
    out, lse = a.run(b.q, b.cache, b.tables())
    assert a.device_status() == 0
    b.check(out, lse, b.want())


@gpu
@pytest.mark.parametrize("qo, kv, Hq, Hkv, D", [([1, 1], [300, 40], 128, 1, 64), ([2], [90], 320, 320, 64),
                                                ([1], [700], 400, 400, 64), ([1, 3], [200, 33], 26, 13, 128),
                                                ([1, 1, 1], [1500, 9, 100], 12, 12, 128)], ids=str)
def test_attention_of_many_heads(qo, kv, Hq, Hkv, D):
    """Groups of 128, more kv heads than CTAs fit the card, odd numbers of kv heads."""
    b = Batch(qo, kv, Hq, Hkv, D, 16, "HND", torch.float16, seed=6)
    out, lse = b.attention().run(b.q, b.cache, b.tables())
    b.check(out, lse, b.want())


@gpu
def test_empty_calls():
    """No requests, no rows, requests without rows: nothing is written and nothing raised."""
    cache = pa.Kv4Cache(4, 16, 2, 64)
    z = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    for B, T in ((0, 0), (3, 0), (0, 4), (3, 4)):
        a = pa.Kv4Attention(B, T, 4, 2, 64, 16, torch.float16)
        out = torch.full((T, 4, 64), 5.0, dtype=torch.float16, device="cuda")
        got, lse = a.run(torch.zeros_like(out), cache, (z(B + 1), z(B + 1), z(0), z(B)), out=out)
        assert (got == 5.0).all() and a.device_status() == 0
    t = pa.BatchTables(3, 0, 0, 16, 4)
    t.build(z(3), z(3), z(3, 1), z(0), z(1))
    assert t.device_status() == 0 and not t.qo_indptr.any()


@gpu
@pytest.mark.parametrize("gain", [1e-30, 1e-5, 300.0, 1e4])
def test_attention_bf16_queries_of_any_size(gain):
    """Queries that fp16 cannot hold as they are: rows are scaled by powers of two."""
    b = Batch([1, 40], [200, 333], 8, 2, 128, 16, "NHD", torch.bfloat16, seed=8, q_gain=gain)
    out, lse = b.attention().run(b.q, b.cache, b.tables())
    b.check(out, lse, b.want())


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B, qo, kv, G, D", [(160, 1, 900, 1, 128), (160, 2, 900, 1, 64), (40, 4, 900, 8, 128),
                                             (4, 40, 700, 4, 128), (4, 70, 700, 4, 64), (2, 20, 90, 4, 256)])
def test_attention_keeps_a_long_tail(B, qo, kv, G, D, dtype):
    """One key of 2^26 times the others' weight and values of zero: the outputs are the others' sum.

    Their P is 2^7 * 2^-26 or more, which fp16 rounds by at most 2^-25: 2^-6
    of it.  The same P stands for every key of a row's slice, so the errors
    do not cancel; logits and weights add less than 2^-10, the output rounds
    by half a step (v_scale keeps it a normal number of fp16).  A logit has one
    product that is not zero, so it is off by four roundings, 2^-22 of its 18;
    lse by three more of 2^-20: less than 2^-17 in all.
    """
    H = 8
    cache = pa.Kv4Cache(B * kv, 1, H, D, v_scale=4096.0)
    k = torch.zeros(B, kv, H, D, dtype=dtype, device="cuda")
    v = torch.full((B, kv, H, D), 6.0 * 4096, dtype=dtype, device="cuda")
    k[:, kv // 5, :, 0] = 6.0
    v[:, kv // 5] = 0.0
    cache.append(k.view(B * kv, H, D), v.view(B * kv, H, D), torch.arange(B * kv, device="cuda"))
    q = torch.zeros(B * qo, H * G, D, dtype=dtype, device="cuda")
    q[..., 0] = 26 * np.log(2) * D ** 0.5 / 6
    dev = lambda a: torch.as_tensor(a, dtype=I32).cuda()  # noqa: E731
    tables = (dev(range(0, B * qo + 1, qo)), dev(range(0, B * kv + 1, kv)), dev(range(B * kv)), dev([1] * B))
    a = pa.Kv4Attention(B, B * qo, H * G, H, D, 1, dtype, False, qo)
    out, lse = a.run(q, cache, tables)
    logit = float(q[0, 0, 0]) * 6 / D ** 0.5
    w = (kv - 1) * np.exp(-logit)
    want, want_lse = 6 * 4096 * w / (1 + w), logit + np.log1p(w)
    assert a.device_status() == 0
    rel = (out.double() / want - 1).abs().max().item()
    assert rel <= 2.0 ** -6 + 2.0 ** -10 + torch.finfo(dtype).eps / 2, rel
    assert (lse.double() - want_lse).abs().max().item() <= 2.0 ** -17


@gpu
def test_attention_max_qo_len_is_a_hint():
    """A bound below the longest request costs time, not results."""
    b = Batch([40, 1, 3], [500, 77, 20], 8, 2, 128, 16, "NHD", torch.bfloat16, seed=9)
    want = b.want()
    for bound in (0, 1, 3, 40, 1000):
        a = b.attention(max_qo=bound)
        out, lse = a.run(b.q, b.cache, b.tables())
        assert a.device_status() == 0
        b.check(out, lse, want)


@gpu
def test_attention_nan_rows_stay_their_own():
    """A NaN in q or in one request's cache reaches that row or request alone."""
    b = Batch([1, 1, 1], [100, 100, 100], 8, 2, 128, 16, "NHD", torch.float16, seed=2)
    clean, _ = b.attention().run(b.q, b.cache, b.tables())
    b.q[0, 3, 5] = float("nan")
    b.cache.scales[int(b.pages[b.page_indptr[1]]), 1, 4, 1, :] = 0x7F
    out, lse = b.attention().run(b.q, b.cache, b.tables())
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    assert torch.isnan(out[1, 4:]).all() and not torch.isnan(lse[1]).any()
    clean_of = lambda x: torch.cat([x[0, :3].flatten(), x[0, 4:].flatten(), x[1, :4].flatten(), x[2].flatten()])  # noqa: E731
    assert torch.equal(clean_of(out), clean_of(clean))


@gpu
@pytest.mark.parametrize("qo, kv, G, D", [([4, 1], [40, 200], 2, 128), ([3], [1000], 8, 64), ([3], [70], 8, 128),
                                          ([2], [33], 4, 256), ([60], [300], 4, 128), ([300], [333], 2, 64),
                                          ([70], [1500], 2, 128), ([50], [90], 4, 256)], ids=str)
def test_attention_nan_behind_the_mask(qo, kv, G, D):
    """A NaN of K or V at a key reaches the rows that see it, and no others, in the dims of its block."""
    b = Batch(qo, kv, 2 * G, 2, D, 16, "NHD", torch.bfloat16, seed=17)
    a = b.attention()
    clean, clean_lse = a.run(b.q, b.cache, b.tables())
    n, q = kv[0], qo[0]
    for back in (0, 1, q - 1):  # the last key, and the one that all but the first rows see
        key = n - 1 - back
        page, slot = int(b.pages[key // 16]), key % 16
        first_row = max(0, key - (n - q))  # rows from here on see it
        for half in (0, 1):
            at = (page, half, slot, 1, D // 16 - 1)
            old = b.cache.scales[at].item()
            b.cache.scales[at] = 0x7F
            out, lse = a.run(b.q, b.cache, b.tables())
            b.cache.scales[at] = old
            hit = torch.zeros_like(clean, dtype=torch.bool)
            hit[first_row:q, G:, (0 if half == 0 else D - 16):] = True
            assert torch.equal(torch.isnan(out), hit), (back, half)
            assert torch.equal(out[~hit], clean[~hit])
            assert torch.equal(torch.isnan(lse), hit.any(-1) if half == 0 else torch.zeros_like(lse, dtype=torch.bool))


@gpu
def test_attention_same_for_any_page_placement_and_layout():
    ref = None
    for layout in ("NHD", "HND"):
        for page in (16, 64):
            b = Batch([1, 4, 50], [700, 300, 444], 8, 2, 128, page, layout, torch.bfloat16, seed=6)
            q = torch.from_numpy(np.random.default_rng(0).standard_normal((55, 8, 128))).to(torch.bfloat16).cuda()
            # the same logical rows in every placement
            rng = np.random.default_rng(11)
            for r, n in enumerate((700, 300, 444)):
                t = np.arange(n)
                ids = b.pages[b.page_indptr[r] + t // page]
                for half in range(2):
                    c, s, _ = kv4.quantise(rng.standard_normal((n, 2, 128)), 1.0)
                    at = (ids, half, slice(None), t % page) if b.hnd else (ids, half, t % page)
                    b.codes[at], b.scales[at] = c, s
            b.cache.codes.copy_(torch.from_numpy(b.codes))
            b.cache.scales.copy_(torch.from_numpy(b.scales))
            got = b.attention().run(q, b.cache, b.tables())
            ref = ref or got
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@gpu
def test_attention_strided_q_and_no_lse():
    b = Batch([1, 5], [100, 30], 8, 2, 64, 16, "NHD", torch.float16, seed=12)
    fused = torch.zeros(b.T, 8 * 64 + 24, dtype=torch.float16, device="cuda")
    fused[:, 8: 8 + 512] = b.q.flatten(1)
    want, _ = b.attention().run(b.q, b.cache, b.tables())
    out, lse = b.attention().run(fused[:, 8: 520].view(b.T, 8, 64), b.cache, b.tables(), return_lse=False)
    assert lse is None and torch.equal(out, want)


@gpu
def test_attention_bad_tables_are_contained():
    b = Batch([1, 1, 1], [100, 60, 40], 8, 2, 128, 16, "NHD", torch.float16, seed=13)
    want = b.attention().run(b.q, b.cache, b.tables())
    for which, at, value in (("last", 1, 17), ("last", 1, 0), ("pages", int(b.page_indptr[1]), 1 << 20),
                             ("pages", int(b.page_indptr[1]), -1)):
        good = getattr(b, which).copy()
        getattr(b, which)[at] = value
        a = b.attention()
        out, lse = a.run(b.q, b.cache, b.tables())
        assert a.device_status() == pa.PA_DEV_BAD_INDEX and a.device_status() == 0
        for r in (0, 2):
            assert torch.equal(out[r], want[0][r]) and torch.equal(lse[r], want[1][r])
        setattr(b, which, good)


@gpu
@pytest.mark.parametrize("pairs", [1, 3, 5, 11])
def test_attention_overlapping_requests_leave_the_workspace_usable(pairs):
    """Tables whose valid requests overlap (between bad ones): flagged, and the next run joins its parts as ever."""
    good = Batch([300], [40000], 32, 4, 64, 16, "NHD", torch.bfloat16, seed=9)
    fresh, used = good.attention(), good.attention()
    want = fresh.run(good.q, good.cache, good.tables())
    qo = torch.tensor([0] + [300, 0] * pairs, dtype=I32).cuda()
    n = int(good.page_indptr[1])
    tables = (qo, torch.tensor([0] + [n, 0] * pairs, dtype=I32).cuda(), good.tables()[2],
              torch.full((2 * pairs,), int(good.last[0]), dtype=I32).cuda())
    bad = pa.Kv4Attention(2 * pairs, 300, 32, 4, 64, 16, torch.bfloat16, True, 300, workspace=used.workspace)
    used.workspace.zero_()
    bad.run(good.q, good.cache, tables)
    assert bad.device_status() == raw.PA_DEV_BAD_INDEX
    for _ in range(2):
        out, lse = used.run(good.q, good.cache, good.tables())
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert used.device_status() == 0


@gpu
@pytest.mark.parametrize("qo, kv", [([1, 1], [3000, 77]), ([4, 1], [500, 300]), ([40, 9], [900, 60]), ([300], [300])])
def test_attention_beyond_32_bit_offsets(qo, kv):
    """Pages in the upper part of a cache of 8.7 GB of codes give what the same pages of a small one do."""
    pages, page, H, D = 530_000, 128, 1, 128
    rows = int(sum(-(-k // page) * page for k in kv))
    k, v = (torch.randn(rows, H, D, device="cuda").half() for _ in range(2))
    slots = torch.arange(rows, device="cuda")
    first, got = torch.tensor(qo).cumsum(0), []
    indptr = torch.tensor([0] + first.tolist(), dtype=I32).cuda()
    counts = torch.tensor([-(-n // page) for n in kv])
    page_indptr = torch.tensor([0] + counts.cumsum(0).tolist(), dtype=I32).cuda()
    last = torch.tensor([(n - 1) % page + 1 for n in kv], dtype=I32).cuda()
    q = torch.randn(sum(qo), 8, D, device="cuda").half()
    for num, base in ((pages, pages - rows // page), (rows // page, 0)):
        cache = pa.Kv4Cache(num, page, H, D)
        cache.append(k, v, slots + base * page)
        ids = torch.arange(base, base + rows // page, dtype=I32, device="cuda")
        a = pa.Kv4Attention(len(qo), sum(qo), 8, H, D, page, torch.float16, True, max(qo))
        got.append(a.run(q, cache, (indptr, page_indptr, ids, last)))
        assert a.device_status() == 0 and cache.device_status() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@gpu
def test_attention_python_refusals():
    b = Batch([1, 1], [20, 30], 8, 2, 128, 16, "NHD", torch.float16)
    a, t = b.attention(), b.tables()
    a.run(b.q, b.cache, t)
    other = pa.Kv4Cache(4, 16, 2, 64)
    for args, kw in [((b.q.bfloat16(), b.cache, t), {}), ((b.q[:1], b.cache, t), {}), ((b.q, other, t), {}),
                     ((b.q.cpu(), b.cache, t), {}), ((b.q, b.cache, (t[0].long(), *t[1:])), {}),
                     ((b.q, b.cache, (t[0][:2], *t[1:])), {}), ((b.q, b.cache, t), dict(out=b.q.float())),
                     ((b.q, b.cache, t), dict(lse=torch.zeros(2, 8, dtype=torch.float64, device="cuda"))),
                     ((b.q, b.cache, pa.BatchTables(3, 4, 8, 16, 9)), {})]:
        with pytest.raises(pa.PagedAttnError):
            a.run(*args, **kw)
    with pytest.raises(pa.PagedAttnError):
        b.attention(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- the step


@gpu
def test_captured_step_grows_requests():
    """tables, append and attention in one graph, replayed: after each replay the attention's result is that of the
    rows appended so far, on a side stream and with padding behind the last request."""
    B, Hq, Hkv, D, page, steps = 5, 8, 2, 128, 16, 12
    rng = np.random.default_rng(21)
    kv = np.array([0, 15, 16, 40, 7], np.int32)
    table, free, num_pages = make_tables(rng, B, page, np.full(B, steps + 1, np.int32), kv)
    t = pa.BatchTables(B, B + 2, num_pages, page, num_pages)
    cache = pa.Kv4Cache(num_pages, page, Hkv, D, k_scale=0.5)
    cache.scales.fill_(0x7F)
    attn = pa.Kv4Attention(B, B + 2, Hq, Hkv, D, page, torch.bfloat16, max_qo_len=1)
    table_t, free_t = torch.from_numpy(table.copy()).cuda(), torch.from_numpy(free).cuda()
    t.kv_lens.zero_()
    t.free_count.fill_(len(free) + int((-(-kv // page)).sum()))
    stack = torch.from_numpy(np.concatenate([free, table[table >= 0]])).cuda()
    # the prompts: a build, an append and nothing attended
    prompt = pa.BatchTables(B, int(kv.sum()), num_pages, page, num_pages)
    new = lambda n: torch.randn(n, Hkv, D, device="cuda").bfloat16()  # noqa: E731
    seen = [[np.zeros((0, Hkv, D))] * 2 for _ in range(B)]

    def keep(rows, counts):
        at = 0
        for b, n in enumerate(counts):
            seen[b] = [np.concatenate([seen[b][h], kv4.quantise(rows[h][at: at + n].double().cpu().numpy(), s)[2]])
                       for h, s in enumerate((0.5, 1.0))]
            at += n

    k, v = new(int(kv.sum())), new(int(kv.sum()))
    table_t.fill_(-1)
    prompt.build(torch.from_numpy(kv).cuda(), torch.zeros(B, dtype=I32).cuda(), table_t, stack, t.free_count)
    cache.append(k, v, prompt.slot_mapping)
    keep((k, v), kv)
    t.kv_lens.copy_(prompt.kv_lens)
    t.free_count.copy_(prompt.free_count)
    qo = torch.ones(B, dtype=I32).cuda()
    q = torch.zeros(B + 2, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(new(B + 2)), torch.zeros_like(new(B + 2))
    out, lse = torch.full_like(q, 3.0), torch.zeros(B + 2, Hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t.build(qo, t.kv_lens, table_t, stack, t.free_count)
        cache.append(k, v, t.slot_mapping)
        attn.run(q, cache, t, out=out, lse=lse)
    for _ in range(steps):
        q.copy_(torch.randn(B + 2, Hq, D).bfloat16())
        k.copy_(torch.randn(B + 2, Hkv, D).bfloat16())
        v.copy_(torch.randn(B + 2, Hkv, D).bfloat16())
        g.replay()
        keep((k, v), [1] * B)
        qd = q.double().cpu().numpy()
        for b in range(B):
            for h in range(Hq):
                kk, vv = seen[b][0][:, h // 4], seen[b][1][:, h // 4]
                z = kk @ qd[b, h] / np.sqrt(D)
                p = np.exp(z - z.max())
                ref, av = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
                # as in Batch.check, for at most 60 keys: P's and the output's half steps, and logits to 2^-14
                err = np.abs(out[b, h].double().cpu().numpy() - ref)
                assert (err <= (2.0 ** -11 + 2.0 ** -13) * av + 2.0 ** -8 * np.abs(ref) + 1e-6).all()
                assert abs(float(lse[b, h]) - (z.max() + np.log(p.sum()))) < 2.0 ** -13
        assert (out[B:] == 3.0).all()
    assert t.device_status() == cache.device_status() == attn.device_status() == 0
    assert t.kv_lens.tolist() == (kv + steps).tolist()


@gpu
def test_memory_outlives_calls_on_another_stream():
    """What a call on a given stream uses is not given away while the stream has not passed it, nor what objects hold."""
    z = lambda *s, t=I32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    B, T, side = 3, 1000, torch.cuda.Stream()
    tables, cache = pa.BatchTables(B, T, 100, 16, 100), pa.Kv4Cache(100, 16, 2, 64)
    attention = pa.Kv4Attention(B, T, 4, 2, 64, 16, torch.float16)
    rows = z(T, 2, 64, t=torch.float16)
    args = (z(B), z(B), z(B, 1), z(1), z(1))
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    q = z(T, 4, 64, t=torch.float16)
    held = {tables: "qo_indptr kv_page_indices slot_mapping positions kv_lens status free_count", cache:
            "codes scales status", attention: "workspace"}
    ptrs = {getattr(o, n).data_ptr(): getattr(o, n).numel() * getattr(o, n).element_size()
            for o, names in held.items() for n in names.split()}
    torch.cuda.synchronize()
    for cycles in (0, 400_000_000):  # (first calls load kernels and may wait); then a fifth of a second
        with torch.cuda.stream(side):
            torch.cuda._sleep(cycles)
        tables.build(*args, stream=side)
        cache.append(rows, rows, slots, stream=side)
        attention.run(q, cache, tables, stream=side)
        if not cycles:
            torch.cuda.synchronize()
    del tables, cache, attention, held
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in ptrs.values() for _ in range(2)]
    assert not side.query()  # (else the allocator may rightly give it away)
    assert not ptrs.keys() & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@gpu
def test_two_objects_on_two_streams():
    """Runs that overlap, each with its own workspace, and a stream given by hand."""
    bs = [Batch([1] * 6, [3000, 100, 50, 700, 900, 11], 8, 2, 128, 16, "NHD", torch.bfloat16, seed=s) for s in (1, 2)]
    objs = [b.attention() for b in bs]
    want = [a.run(b.q, b.cache, b.tables()) for a, b in zip(objs, bs)]
    streams = [torch.cuda.Stream() for _ in bs]
    tabs = [b.tables() for b in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [a.run(b.q, b.cache, t, stream=s) for a, b, t, s in zip(objs, bs, tabs, streams)]
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


# ---------------------------------------------------------------- logit factors at the ends of fp32's range


@gpu
@pytest.mark.parametrize("k_scale, gain", [(1e-15, 1e-30), (1e-7, 2e-38), (1e-15, 1e-38)])
@pytest.mark.parametrize("qo, kv, G, D", [([1, 40], [200, 333], 4, 128), ([300], [2600], 4, 128), ([40], [4100], 2, 64),
                                          ([300, 33], [1500, 1500], 4, 128), ([17, 66], [90, 66], 4, 256)], ids=str)
def test_attention_of_tiny_bf16_queries_and_scales(qo, kv, G, D, k_scale, gain):
    """Factors below fp32's range stand for logits of zero: every key a row sees has the same weight, the others none."""
    b = Batch(qo, kv, 2 * G, 2, D, 16, "NHD", torch.bfloat16, seed=8, k_scale=k_scale, q_gain=gain)
    for causal in (True, False):
        a = b.attention(causal)
        out, lse = a.run(b.q, b.cache, b.tables())
        b.check(out, lse, b.want(causal))
        assert a.device_status() == 0


@gpu
@pytest.mark.parametrize("qo, kv, G, D", [([1, 2], [200, 33], 4, 128), ([40], [333], 4, 128), ([300], [2600], 2, 64),
                                          ([17, 66], [90, 66], 4, 256)], ids=str)
def test_attention_of_huge_bf16_queries_and_scales_over_zero_keys(qo, kv, G, D):
    """Factors above fp32's range over keys of zero: the logits are zero."""
    b = Batch(qo, kv, 2 * G, 2, D, 16, "NHD", torch.bfloat16, seed=8, k_scale=1e15, q_gain=1e30)
    b.codes[:, 0] = 0
    b.cache.codes[:, 0] = 0
    for causal in (True, False):
        a = b.attention(causal)
        out, lse = a.run(b.q, b.cache, b.tables())
        b.check(out, lse, b.want(causal))
        assert a.device_status() == 0


# ---------------------------------------------------------------- objects made on one stream and used on another


def garbage_for(*sizes):
    """The allocator's next blocks of these sizes hold 0x5A."""
    junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    del junk


@gpu
@pytest.mark.parametrize("by_hand", [True, False])
def test_first_calls_on_another_stream_wait_for_the_objects_memory(by_hand):
    """Objects are made while their stream is busy, so that their zeroing is still queued when another stream calls."""
    b = Batch([1], [20_000], 8, 1, 128, 16, "NHD", torch.bfloat16, seed=3)
    want, want_lse = b.attention().run(b.q, b.cache, b.tables())
    rng, B, page, n = np.random.default_rng(4), 40, 16, 500
    qo, kv = np.ones(B, np.int32), rng.integers(0, 300, B).astype(np.int32)
    table, free, num_pages = make_tables(rng, B, page, qo, kv)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    qo_t, kv_t, table_t, free_t, count = dev(qo), dev(kv), dev(table.copy()), dev(free), dev(np.int32([len(free)]))
    k, slots, tables = torch.randn(n, 2, 64, device="cuda").half(), torch.arange(n, device="cuda"), b.tables()
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    ref = pa.Kv4Cache(64, page, 2, 64)
    ref.append(k, k, slots)
    lists = pa.BatchTables(B, B + 7, num_pages, page, num_pages)
    lists.build(qo_t, kv_t, table_t, free_t, count)
    side = torch.cuda.Stream()
    garbage_for(b.attention().workspace.numel(), ref.codes.numel(), ref.scales.numel(), 512)
    del ref.status
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # a fifth of a second
    a, cache = b.attention(), pa.Kv4Cache(64, page, 2, 64)
    t = pa.BatchTables(B, B + 7, num_pages, page, num_pages)
    kw = dict(stream=side) if by_hand else {}
    with torch.cuda.stream(torch.cuda.current_stream() if by_hand else side):
        for _ in range(2):
            a.run(b.q, b.cache, tables, out=out, lse=lse, **kw)
            cache.append(k, k, slots, **kw)
            t.build(qo_t, kv_t, table_t, free_t, count, **kw)
    assert a.device_status(side) == cache.device_status(side) == t.device_status(side) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert torch.equal(cache.codes, ref.codes) and torch.equal(cache.scales, ref.scales)
    for name in ("qo_indptr", "kv_page_indptr", "new_page_indptr", "kv_page_indices", "kv_last_page_len", "kv_lens",
                 "slot_mapping", "positions", "free_count", "status"):
        assert torch.equal(getattr(t, name), getattr(lists, name)), name


@gpu
def test_memory_outlives_calls_under_another_current_stream():
    """As test_memory_outlives_calls_on_another_stream, for the objects' own memory under torch.cuda.stream."""
    z = lambda *s, t=I32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    B, T, side = 3, 1000, torch.cuda.Stream()
    tables, cache = pa.BatchTables(B, T, 100, 16, 100), pa.Kv4Cache(100, 16, 2, 64)
    attention = pa.Kv4Attention(B, T, 4, 2, 64, 16, torch.float16)
    rows, args = z(T, 2, 64, t=torch.float16), (z(B), z(B), z(B, 1), z(1), z(1))
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    q = z(T, 4, 64, t=torch.float16)
    held = {tables: "qo_indptr kv_page_indices slot_mapping positions kv_lens status free_count", cache:
            "codes scales status", attention: "workspace"}
    ptrs = {getattr(o, n).data_ptr(): getattr(o, n).numel() * getattr(o, n).element_size()
            for o, names in held.items() for n in names.split()}
    torch.cuda.synchronize()
    for cycles in (0, 400_000_000):  # (first calls load kernels and may wait); then a fifth of a second
        with torch.cuda.stream(side):
            torch.cuda._sleep(cycles)
            tables.build(*args)
            cache.append(rows, rows, slots)
            attention.run(q, cache, tables)
        if not cycles:
            torch.cuda.synchronize()
    del tables, cache, attention, held
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in ptrs.values() for _ in range(2)]
    assert not side.query()  # (else the allocator may rightly give it away)
    assert not ptrs.keys() & {t.data_ptr() for t in again}
    torch.cuda.synchronize()


@gpu
def test_a_given_workspace_is_cleared_behind_the_runs_in_it():
    """A run is queued on another stream when an object is made over its workspace: the clearing comes after it, and
    before that stream's next run."""
    b = Batch([1], [20_000], 8, 1, 128, 16, "NHD", torch.bfloat16, seed=3)
    a, side = b.attention(), torch.cuda.Stream()
    want, want_lse = a.run(b.q, b.cache, b.tables())
    tables, got = b.tables(), []
    a.run(b.q, b.cache, tables, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got.append(a.run(b.q, b.cache, tables, stream=side))
    other = b.attention(workspace=a.workspace)
    assert side.query()  # the constructor waited
    got.append(a.run(b.q, b.cache, tables, stream=side))
    torch.cuda.synchronize()
    got.append(other.run(b.q, b.cache, tables))
    for out, lse in got:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@gpu
def test_objects_that_share_a_workspace():
    """An object in place of a workspace: its memory, its status word and its counts are taken as they are."""
    bs = [Batch([1, 1], [3000, 900], 8, 1, 128, 16, "NHD", torch.float16, seed=1),
          Batch([40, 1], [2100, 1900], 16, 2, 128, 16, "NHD", torch.float16, seed=3),
          Batch([2], [1700], 6, 2, 256, 16, "NHD", torch.bfloat16, seed=4)]
    want, tables = [b.want() for b in bs], [b.tables() for b in bs]
    first = bs[0].attention(workspace=torch.empty(256 << 20, dtype=torch.uint8, device="cuda"))
    bad = tables[0][:3] + (torch.tensor([17, 1], dtype=I32).cuda(),)
    first.run(bs[0].q, bs[0].cache, bad)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1_000_000_000)
    objs = [first] + [b.attention(workspace=first) for b in bs[1:]]
    assert not side.query()  # nothing was waited for
    assert all(o.workspace is first.workspace for o in objs)
    assert objs[1].device_status() == pa.PA_DEV_BAD_INDEX and first.device_status() == 0
    for _ in range(3):
        for b, a, w, t in zip(bs, objs, want, tables):
            out, lse = a.run(b.q, b.cache, t)
            b.check(out, lse, w)
    small = bs[0].attention()
    with pytest.raises(pa.PagedAttnError) as e:
        pa.Kv4Attention(1, 64, 128, 1, 128, 16, torch.float16, workspace=pa.Kv4Attention(1, 1, 1, 1, 64, 16, torch.float16))
    assert e.value.status == raw.PA_ERR_WORKSPACE_TOO_SMALL and small.device_status() == 0


# ---------------------------------------------------------------- a NaN of V at head_dim 64


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("qo, kv, G", [(4, 70, 2), (3, 33, 1), (5, 97, 3), (8, 64, 4)], ids=str)
def test_attention_nan_of_v_reaches_its_whole_block_at_head_dim_64(qo, kv, G, dtype):
    """Two lanes share a scale byte there: both halves of the block's 16 dims get the NaN, whichever key and block."""
    b = Batch([qo], [kv], 2 * G, 2, 64, 16, "HND", dtype, seed=23)
    a = b.attention()
    clean, clean_lse = a.run(b.q, b.cache, b.tables())
    for key in [kv - 1 - i for i in range(qo + 1)] + [kv - 32, 0]:
        at = (int(b.pages[key // 16]), 1, slice(None), key % 16)
        for block in range(4):
            old = b.cache.scales[at][:, block].clone()
            b.cache.scales[at][:, block] = 0xFF if block % 2 else 0x7F
            out, lse = a.run(b.q, b.cache, b.tables())
            b.cache.scales[at][:, block] = old
            hit = torch.zeros_like(clean, dtype=torch.bool)
            hit[max(0, key - (kv - qo)):, :, 16 * block: 16 * block + 16] = True
            assert torch.equal(torch.isnan(out), hit), (key, block)
            assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, clean_lse)


@gpu
@pytest.mark.parametrize("B", [3, 3500])
def test_tables_of_width_zero(B):
    """A block table without columns holds requests without pages, and no token."""
    z = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    t, qo = pa.BatchTables(B, 4, 8, 16, 10), z(B)
    t.build(qo, z(B), z(B, 0), z(2), z(1))
    assert t.device_status() == 0 and not t.kv_page_indptr.any() and (t.slot_mapping == -1).all()
    qo[1] = 1
    t.build(qo, z(B), z(B, 0), z(2), z(1) + 2)
    assert t.device_status() == raw.PA_DEV_NO_ROOM and not t.qo_indptr.any()


# ---------------------------------------------------------------- the structures' two descriptions


@pytest.mark.parametrize("packed, struct, values", [
    ("_TABLES_IN", "TablesIn", [11, 12, 13, 14, 15, 1 << 40, 7, 6, 5, 16, 9]),
    ("_KV4_ROWS", "Kv4Rows", [11, 12, 1 << 40, 1 << 41, 13, 14, 15, 16, 3, 1]),
    ("_KV4_BATCH", "Kv4Batch", [11, 12, 13, 14, 2, 8, 5, 4, 64, 1, 1])])
def test_packed_arguments_are_the_structures(packed, struct, values):
    """The calls pack their arguments' bytes; the binding's structures, which the refusals are tested with, hold the same."""
    from attention_paged_kv_gb300 import _kv4
    cls = getattr(raw, struct)
    assert len(values) == len(cls._fields_) and getattr(_kv4, packed).size == ctypes.sizeof(cls)
    assert getattr(_kv4, packed).pack(*values) == bytes(cls(*values))


@pytest.mark.parametrize("struct, name", [("TablesIn", "tables_in"), ("TablesOut", "tables_out"), ("Kv4Rows", "kv4_rows"),
                                          ("Kv4CacheArgs", "kv4_cache"), ("Kv4Batch", "kv4_batch")])
def test_structures_are_the_headers(struct, name):
    """Field by field, in order, with the header's types."""
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(pa.LIB_PATH)), "include", "pagedattn.h")
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} pagedattn_%s;" % name, text).group(1)
    want = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = re.match(r"(?:const )?(\w+)\s*(.*)", line, re.S).groups()
        for n in (x.strip() for x in names.split(",")):
            ctype = ctypes.c_void_p if n.startswith("*") else {
                "int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float,
                "pagedattn_dtype": ctypes.c_int}[kind]
            want.append((n.lstrip("* "), ctype))
    assert getattr(raw, struct)._fields_ == want


def test_built_prefill_kernels_have_the_registers_they_hand_over():
    """The warps' shares after the hand-over add up to what the launch gives (two row tiles 128 a thread, one 80)."""
    import os
    import re
    log = os.path.join(os.path.dirname(pa.LIB_PATH), "_build", "kv4_prefill.cu.o.log")
    if not os.path.exists(log):
        pytest.skip("the build's log is not there")
    name, seen = None, {}
    for line in open(log):
        name = (re.search(r"Compiling entry function '(\S+)'", line) or [None, name])[1]
        used = re.search(r"Used (\d+) registers", line)
        if used and "kv4_prefill_kernel" in name:
            D, NT = map(int, re.search(r"Li(\d+)ELi(\d)EE", name).groups())
            seen.setdefault((D, NT), set()).add(int(used[1]))
    assert seen.keys() == {(64, 1), (64, 2), (128, 1), (128, 2), (256, 1)}
    for (D, NT), regs in seen.items():
        if D < 256:
            assert regs == {128 if NT == 2 else 80}, (D, NT)
