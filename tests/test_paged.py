"""Rotary positions, the 16-bit cache's append and bounds, the selection of pages and the attention over them, against
the fp64 restatement in oracle/paged.py."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import paged

pa = pytest.importorskip("attention_paged_kv_gb300")
from attention_paged_kv_gb300 import _binding as raw  # noqa: E402

gpu = pytest.mark.gpu
I32 = torch.int32
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(pa.LIB_PATH):
        from attention_paged_kv_gb300 import build
        build.build()


def dev(a, dtype=I32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ---------------------------------------------------------------- refusals (no kernel runs)

FAKE = 1 << 20  # an aligned address that no refused call reads


def refused(call, status, text):
    with pytest.raises(pa.PagedAttnError) as e:
        raw.check(call())
    assert e.value.status == status and text in str(e.value), str(e.value)


INVALID, UNSUPPORTED = raw.PA_ERR_INVALID_ARG, raw.PA_ERR_UNSUPPORTED
ROTATION = dict(turns=FAKE, axes=None, num_axes=1, rotary_dim=128, interleaved=0, scale=1.0)
CACHE = dict(data=FAKE, bounds=FAKE, bound_scales=FAKE, num_pages=4, page_size=16, num_kv_heads=2, head_dim=128,
             kv_layout=0, dtype=1)
BAD_ROTATION = [
    (dict(turns=None), INVALID, "turns"), (dict(turns=FAKE + 4), INVALID, "turns"),
    (dict(rotary_dim=24), UNSUPPORTED, "rotary_dim"), (dict(rotary_dim=0), UNSUPPORTED, "rotary_dim"),
    (dict(rotary_dim=144), UNSUPPORTED, "rotary_dim"), (dict(num_axes=0), INVALID, "num_axes"),
    (dict(scale=float("nan")), INVALID, "scale"), (dict(scale=float("inf")), INVALID, "scale")]
BAD_CACHE = [
    (dict(data=None), INVALID, "data"), (dict(data=FAKE + 8), INVALID, "aligned"),
    (dict(bounds=FAKE + 8), INVALID, "aligned"), (dict(bound_scales=None), INVALID, "together"),
    (dict(bounds=None), INVALID, "together"), (dict(head_dim=96), UNSUPPORTED, "head_dim"),
    (dict(page_size=12), UNSUPPORTED, "page_size"), (dict(page_size=256), UNSUPPORTED, "page_size"),
    (dict(num_kv_heads=0), INVALID, "num_kv_heads"), (dict(num_pages=0), INVALID, "num_pages"),
    (dict(kv_layout=2), UNSUPPORTED, "kv_layout"), (dict(dtype=2), UNSUPPORTED, "dtype")]


@pytest.mark.parametrize("rotation, rows, status, text", [(r, {}, s, t) for r, s, t in BAD_ROTATION] + [
    ({}, dict(num_tokens=-1), INVALID, "negative"), ({}, dict(num_tokens=(1 << 31) - 1), UNSUPPORTED, "num_tokens"),
    ({}, dict(head_dim=100), UNSUPPORTED, "head_dim"), ({}, dict(head_dim=272), UNSUPPORTED, "head_dim"),
    ({}, dict(dtype=3), UNSUPPORTED, "dtype"), ({}, dict(q=None), INVALID, "q and its output"),
    ({}, dict(k_out=None), INVALID, "k and its output"), ({}, dict(q=FAKE + 8), INVALID, "aligned"),
    ({}, dict(q_stride=1000), INVALID, "stride"), ({}, dict(k_out_stride=260), INVALID, "stride"),
    ({}, dict(q_out=FAKE), INVALID, "in place"), ({}, dict(positions=None), INVALID, "positions"),
    ({}, dict(position_stride=-1), INVALID, "position_stride"), ({}, dict(num_q_heads=70000), UNSUPPORTED, "65535")])
def test_rope_refusals(rotation, rows, status, text):
    r = raw.Rotation(**{**ROTATION, **rotation})
    d = dict(q=FAKE, k=FAKE, q_out=2 * FAKE, k_out=2 * FAKE, q_stride=1024, k_stride=256, q_out_stride=2048,
             k_out_stride=256, positions=FAKE, position_stride=3, num_tokens=3, num_q_heads=8, num_k_heads=2,
             head_dim=128, inverse=0, dtype=0)
    w = raw.RopeRows(**{**d, **rows})
    refused(lambda: pa.load().pagedattn_rope(ctypes.byref(r), ctypes.byref(w), None), status, text)


@pytest.mark.parametrize("cache, rotation, rows, status, text", [(c, {}, {}, s, t) for c, s, t in BAD_CACHE] +
                         [({}, r, {}, s, t) for r, s, t in BAD_ROTATION] + [
    ({}, {}, dict(num_tokens=-1), INVALID, "negative"), ({}, {}, dict(k=None), INVALID, "required"),
    ({}, {}, dict(v=FAKE + 2), INVALID, "aligned"), ({}, {}, dict(status=None), INVALID, "required"),
    ({}, {}, dict(slot_mapping=FAKE + 4), INVALID, "8-byte"), ({}, {}, dict(k_stride=255), INVALID, "k_stride"),
    ({}, {}, dict(v_stride=260), INVALID, "v_stride"), ({}, {}, dict(q_out=None), INVALID, "q_out"),
    ({}, {}, dict(q_stride=8), INVALID, "q_stride"), ({}, None, {}, INVALID, "rotation"),
    ({}, {}, dict(q_out=FAKE, q_out_stride=2048), INVALID, "in place")])
def test_append_refusals(cache, rotation, rows, status, text):
    c = raw.KvCacheArgs(**{**CACHE, **cache})
    r = None if rotation is None else raw.Rotation(**{**ROTATION, **rotation})
    d = dict(k=FAKE, v=FAKE, q=FAKE, q_out=2 * FAKE, k_stride=256, v_stride=256, q_stride=1024, q_out_stride=1024,
             slot_mapping=FAKE, positions=FAKE, position_stride=3, status=FAKE, num_tokens=3, num_qo_heads=8)
    w = raw.KvRows(**{**d, **rows})
    refused(lambda: pa.load().pagedattn_kv_append(ctypes.byref(c), None if r is None else ctypes.byref(r),
                                                  ctypes.byref(w), None), status, text)


@pytest.mark.parametrize("cache, n, slots, status, text", [(c, 3, FAKE, s, t) for c, s, t in BAD_CACHE] + [
    (dict(bounds=None, bound_scales=None), 3, FAKE, INVALID, "no bounds"), ({}, -1, FAKE, INVALID, "negative"),
    ({}, 3, None, INVALID, "required"), ({}, 3, FAKE + 4, INVALID, "8-byte")])
def test_bounds_refusals(cache, n, slots, status, text):
    c = raw.KvCacheArgs(**{**CACHE, **cache})
    refused(lambda: pa.load().pagedattn_kv_bounds(ctypes.byref(c), slots, n, FAKE, None), status, text)


BAD_BATCH = [
    (dict(num_qo_heads=3), {}, INVALID, "num_qo_heads"), (dict(num_qo_heads=2 * 129), {}, UNSUPPORTED, "128"),
    (dict(batch_size=-1), {}, INVALID, "negative"), (dict(max_pages=-1), {}, INVALID, "negative"),
    (dict(max_qo_len=-1), {}, INVALID, "negative"),
    (dict(num_tokens=1 << 29), {}, UNSUPPORTED, "2^30"), (dict(num_blocks=0), {}, UNSUPPORTED, "num_blocks"),
    (dict(num_blocks=4097), {}, UNSUPPORTED, "num_blocks"), ({}, dict(workspace=None), INVALID, "workspace"),
    ({}, dict(workspace=FAKE + 128), INVALID, "workspace")]


@pytest.mark.parametrize("cache, batch, more, status, text", [(c, {}, {}, s, t) for c, s, t in BAD_CACHE] +
                         [({}, b, m, s, t) for b, m, s, t in BAD_BATCH])
@pytest.mark.parametrize("which", ["select", "run"])
def test_block_refusals(which, cache, batch, more, status, text):
    c = raw.KvCacheArgs(**{**CACHE, **cache})
    d = dict(qo_indptr=FAKE, kv_page_indptr=FAKE, kv_page_indices=FAKE, kv_last_page_len=FAKE, batch_size=2,
             num_page_indices=8, num_tokens=2, num_qo_heads=8, num_blocks=4, first=1, last=1, max_pages=100, max_qo_len=1)
    b = raw.BlockBatch(**{**d, **batch})
    m = {**dict(q=FAKE, blocks=FAKE, out=FAKE, workspace=FAKE), **more}
    lib = pa.load()
    if which == "select":
        call = lambda: lib.pagedattn_select_blocks(ctypes.byref(c), ctypes.byref(b), m["q"], 1024, m["blocks"],  # noqa: E731
                                                   m["workspace"], 1 << 40, None)
    else:
        call = lambda: lib.pagedattn_blocks_run(ctypes.byref(c), ctypes.byref(b), m["blocks"], m["q"], 1024, m["out"],  # noqa: E731
                                                None, m["workspace"], 1 << 40, None)
    refused(call, status, text)


@pytest.mark.parametrize("packed, struct, values", [
    ("_ROPE_ROWS", "RopeRows", [11, 12, 13, 14, 1 << 40, 1 << 41, 15, 16, 17, 1 << 42, 3, 4, 5, 6, 1, 1]),
    ("_KV_ROWS", "KvRows", [11, 12, 13, 14, 1 << 40, 1 << 41, 15, 16, 17, 18, 1 << 42, 19, 3, 4]),
    ("_BLOCK_BATCH", "BlockBatch", [11, 12, 13, 14, 1, 2, 3, 4, 5, 6, 7, 8, 9])])
def test_packed_arguments_are_the_structures(packed, struct, values):
    from attention_paged_kv_gb300 import _paged
    cls = getattr(raw, struct)
    assert len(values) == len(cls._fields_) and getattr(_paged, packed).size == ctypes.sizeof(cls)
    assert getattr(_paged, packed).pack(*values) == bytes(cls(*values))


@pytest.mark.parametrize("struct, name", [("Rotation", "rotation"), ("RopeRows", "rope_rows"), ("KvCacheArgs", "kv_cache"),
                                          ("KvRows", "kv_rows"), ("BlockBatch", "block_batch")])
def test_structures_are_the_headers(struct, name):
    path = os.path.join(os.path.dirname(os.path.dirname(pa.LIB_PATH)), "include", "pagedattn.h")
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} pagedattn_%s;" % name, text).group(1)
    want = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = re.match(r"(?:const )?(\w+)\s*(.*)", line, re.S).groups()
        for n in (x.strip() for x in names.split(",")):
            want.append((n.lstrip("* "), ctypes.c_void_p if n.startswith("*") else {
                "int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float,
                "pagedattn_dtype": ctypes.c_int}[kind]))
    assert getattr(raw, struct)._fields_ == want


# ---------------------------------------------------------------- rotation


def frequencies(pairs, base=10000.0):
    return base ** (-np.arange(pairs) / pairs)


def check_rotated(got, want, size, dtype):
    """The angle is off by its last bits before the cosine (2^-24 half turns, 2 pi 2^-33 by truncation: below 2^-22 rad), cosine
    and sine by two units of 2^-24, products and sum by three roundings of 2^-24: below 2^-20 of |a| + |b| in all; the
    result by half a step of its type (2^-25 or less where it is subnormal in fp16)."""
    eps = torch.finfo(dtype).eps / 2
    err = np.abs(host(got) - want)
    bound = size * 2.0 ** -20 * (1 + eps) + eps * np.abs(want) + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert (err <= bound).all(), (err / np.maximum(bound, 1e-300)).max()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n, heads, k_heads, dim, rotary, axes", [
    (1, 1, 1, 64, 64, 1), (3, 8, 2, 128, 128, 1), (77, 5, 3, 96, 32, 2), (33, 4, 4, 16, 16, 1), (130, 64, 8, 128, 64, 3),
    (65, 3, 1, 256, 256, 3), (1000, 20, 4, 128, 128, 1), (2, 1, 0, 80, 80, 1), (9, 17, 1, 256, 128, 1)])
def test_rope_equals_restated(n, heads, k_heads, dim, rotary, axes, interleaved, dtype):
    rng = np.random.default_rng(n + dim)
    w = frequencies(rotary // 2)
    on = rng.integers(0, axes, rotary // 2) if axes > 1 else None
    if on is not None:
        on[:axes] = np.arange(axes)
    r = pa.Rope(w, interleaved=interleaved, axes=on, scale=1.25)
    positions = rng.integers(-50, 1_000_000, (axes, n))
    positions[:, 0] = 0
    fused = torch.from_numpy(rng.standard_normal((n, (heads + k_heads) * dim + 8))).to(dtype).cuda()
    q = fused[:, 8: 8 + heads * dim].view(n, heads, dim)
    k = fused[:, 8 + heads * dim:].view(n, k_heads, dim) if k_heads else None
    pos = dev(positions) if axes > 1 else dev(positions[0])
    before = fused.clone()
    for inverse in (False, True):
        got = r.apply(q, k, pos, inverse=inverse)
        for x, y in zip((q, k), got):
            if x is not None:
                want, size = paged.rope(host(x), positions, w, on, interleaved, 1.25, inverse)
                check_rotated(y, want, size, dtype)
                assert torch.equal(y[..., rotary:], x[..., rotary:])
        assert torch.equal(fused, before)
    out = r.apply(q, k, pos, q_out=q, k_out=k, inverse=True)  # in place
    assert out[0] is q and torch.equal(q, got[0]) and (k is None or torch.equal(k, got[1]))
    assert torch.equal(fused[:, :8], before[:, :8])


@gpu
def test_rope_of_far_positions():
    """Angles at the ends of int32 are as good as near ones; fp64 has them to 2^31 * 2^-53 of a turn."""
    w = frequencies(64)
    positions = np.array([[2 ** 31 - 1, -2 ** 31, 2 ** 30 + 7, 123456789, -1]])
    x = torch.ones(5, 1, 128, dtype=torch.float16, device="cuda")
    got, _ = pa.Rope(w).apply(x, None, dev(positions[0]))
    want, size = paged.rope(host(x), positions, w)
    check_rotated(got, want, size, torch.float16)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_inverse_is_the_gradient(interleaved):
    """sum(y * rope(x)) has the gradient inverse(y) in x, up to the roundings of the three results: n half steps of fp16
    each, of values whose size is theirs (a pair's rotation keeps its length), and 2^-20 of the pairs as above."""
    rng = np.random.default_rng(3)
    n, h, d = 50, 6, 128
    r = pa.Rope(frequencies(48), interleaved=interleaved, axes=[0] * 16 + [1] * 16 + [2] * 16)
    pos = dev(rng.integers(0, 5000, (3, n)))
    x, y, e = (torch.from_numpy(rng.standard_normal((n, h, d))).half().cuda() for _ in range(3))
    grad, _ = r.apply(y, None, pos, inverse=True)
    # the rotation is linear: the difference along e is y . rope(e)
    moved, _ = r.apply(e, None, pos)
    left, right = (host(y) * host(moved)).sum(), (host(grad) * host(e)).sum()
    size = lambda a, b: (np.abs(host(a)) * np.abs(host(b))).sum()  # noqa: E731
    bound = 2.0 ** -11 * (size(y, moved) + size(grad, e)) + 2.0 ** -18 * (size(y, y) + size(e, e))
    assert abs(left - right) <= bound
    back, _ = r.apply(r.apply(x, None, pos)[0], None, pos, inverse=True)
    assert (np.abs(host(back) - host(x)) <= 2.0 ** -11 * (2 * np.abs(host(x)) + np.abs(host(x)).max()) + 2.0 ** -10).all()


@gpu
def test_rope_one_row_for_all_axes_and_no_tokens():
    r = pa.Rope(frequencies(32), axes=[0] * 10 + [1] * 22)
    x = torch.randn(40, 4, 64, device="cuda").half()
    pos = torch.arange(40, dtype=I32, device="cuda")
    same, _ = r.apply(x, None, pos.expand(2, 40))
    plain, _ = pa.Rope(frequencies(32)).apply(x, None, pos)
    assert torch.equal(same, plain)
    q, k = r.apply(x[:0], x[:0], pos[:0].expand(2, 0))
    assert q.shape == (0, 4, 64) and k.shape == (0, 4, 64)


@gpu
def test_rope_python_refusals():
    for bad in ([1.0] * 7, [1.0] * 12, [1.0] * 136, [float("nan")] * 8):
        with pytest.raises(pa.PagedAttnError):
            pa.Rope(bad)
    for bad in ([0] * 7, [0] * 7 + [-1]):
        with pytest.raises(pa.PagedAttnError):
            pa.Rope([1.0] * 8, axes=bad)
    r = pa.Rope([1.0] * 8, axes=[0, 1] * 4)
    x, pos = torch.zeros(5, 2, 64, dtype=torch.float16, device="cuda"), torch.zeros(2, 5, dtype=I32, device="cuda")
    r.apply(x, x, pos)
    for kw in (dict(q=x.float()), dict(q=x[0]), dict(k=x.bfloat16()), dict(k=x[:4]), dict(k=x[..., :32]), dict(q=x.cpu()),
               dict(positions=pos.long()), dict(positions=pos[0]), dict(positions=pos[:, :4]), dict(k_out=x[:4]),
               dict(positions=torch.zeros(5, 2, dtype=I32, device="cuda").t()), dict(k=None, k_out=x),
               dict(q=x.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(pa.PagedAttnError):
            r.apply(**{**dict(q=x, k=x, positions=pos), **kw})


# ---------------------------------------------------------------- append


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, heads, h, d, page, layout, rotary, axes, interleaved", [
    (1, 1, 1, 64, 1, "NHD", 64, 1, False), (77, 6, 3, 64, 16, "HND", 32, 1, True), (130, 64, 8, 128, 16, "NHD", 128, 3, False),
    (9, 4, 2, 256, 128, "HND", 256, 1, False), (300, 1, 1, 128, 4, "HND", 64, 2, True), (65, 0, 5, 256, 8, "NHD", 0, 1, False),
    (1500, 24, 8, 128, 16, "NHD", 128, 1, False)])
def test_append_equals_restated(n, heads, h, d, page, layout, rotary, axes, interleaved, dtype):
    rng = np.random.default_rng(n)
    pages = -(-n // page) + 3
    cache = pa.KvCache(pages, page, h, d, dtype, layout)
    cache.data.fill_(9.0)
    slots = rng.permutation(pages * page)[:n].astype(np.int64)
    slots[rng.random(n) < 0.1] = -1
    wide = torch.from_numpy(rng.standard_normal((n, (heads + 2 * h) * d + 24))).to(dtype).cuda()
    part = lambda a, m: wide[:, 8 + a * d: 8 + (a + m) * d].view(n, m, d)  # noqa: E731
    q, k, v = part(0, heads), part(heads, h), part(heads + h, h)
    positions = rng.integers(0, 200_000, (axes, n))
    w = frequencies(rotary // 2) if rotary else None
    on = rng.integers(0, axes, rotary // 2) if axes > 1 else None
    if on is not None:
        on[:axes] = np.arange(axes)
    if rotary:
        rope = pa.Rope(w, interleaved=interleaved, axes=on)
        got = cache.append(k, v, dev(slots, torch.int64), rope=rope, positions=dev(positions if axes > 1 else positions[0]),
                           q=q if heads else None)
        want_k, size_k = paged.rope(host(k), positions, w, on, interleaved)
        if heads:
            check_rotated(got, *paged.rope(host(q), positions, w, on, interleaved), dtype)
        else:
            assert got is None
    else:
        assert cache.append(k, v, dev(slots, torch.int64)) is None
        want_k, size_k = host(k), np.zeros(k.shape)
    assert cache.device_status() == 0
    at = slots >= 0
    data = cache.data if layout == "NHD" else cache.data.transpose(2, 3)
    rows = data[torch.from_numpy(slots[at] // page).cuda(), :, torch.from_numpy(slots[at] % page).cuda()]
    check_rotated(rows[:, 0], want_k[at], size_k[at], dtype)
    assert torch.equal(rows[:, 1], v[torch.from_numpy(at).cuda()])
    left = torch.ones(pages, page, dtype=torch.bool, device="cuda")
    left.view(-1)[dev(slots[at], torch.int64)] = False
    assert (data.transpose(1, 2)[left] == 9.0).all()  # other slots


@gpu
def test_append_bad_slots_and_other_memory():
    """Slots beyond the cache are skipped and raise; data and bounds may be the caller's."""
    data = torch.zeros(4, 2, 16, 2, 64, dtype=torch.float16, device="cuda")
    codes, scales = torch.full((4, 2, 2, 64), 3, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, device="cuda")
    cache = pa.KvCache(4, 16, 2, 64, torch.float16, data=data, bounds=codes, bound_scales=scales)
    k = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    cache.append(k, 2 * k, torch.tensor([64, 5, 1 << 40], device="cuda"))
    assert cache.device_status() == pa.PA_DEV_BAD_INDEX and cache.device_status() == 0
    assert (data[0, 0, 5] == 1).all() and (data[0, 1, 5] == 2).all() and data.float().sum() == 3 * 128
    assert (codes[1:] == 3).all() and (codes[0, :, 0] == 127).all() and (codes[0, :, 1] == 0).all()
    assert torch.equal(scales, torch.tensor([[1, 1], [0, 0], [0, 0], [0, 0]], device="cuda") * np.float32(1 / 127))


@gpu
def test_append_is_what_plan_run_reads():
    """A cache filled by append serves the planned attention."""
    n, page = 100, 16
    cache = pa.KvCache(7, page, 2, 64, torch.float16)
    rope = pa.Rope(frequencies(32))
    q, k, v = (torch.randn(n, m, 64, device="cuda").half() for m in (4, 2, 2))
    pos = torch.arange(n, dtype=I32, device="cuda")
    turned = cache.append(k, v, torch.arange(n, device="cuda"), rope=rope, positions=pos, q=q)
    plan = pa.Plan([0, n], [0, 7], list(range(7)), [n - 6 * page], 4, 2, 64, page, 7, torch.float16)
    out, lse = plan.run(turned, cache.data)
    lists = torch.arange(7, dtype=I32, device="cuda").expand(n, 2, 7).contiguous()
    a = pa.BlockAttention(1, n, 4, 2, 64, page, torch.float16, 7, n)
    tables = tuple(dev(x) for x in ([0, n], [0, 7], range(7), [n - 6 * page]))
    got, got_lse = a.run(turned, cache, tables, lists)
    assert (out.float() - got.float()).abs().max() <= 4e-3 and (lse - got_lse).abs().max() <= 1e-4


# ---------------------------------------------------------------- bounds


def check_bounds(cache, pages, filled, untouched):
    data = cache.data.float().cpu().numpy()
    hnd = cache.kv_layout == raw.PA_LAYOUT_HND
    codes, scales = cache.bounds.cpu().numpy(), cache.bound_scales.cpu().numpy()
    for page, n in zip(pages, filled):
        for h in range(cache.num_kv_heads):
            c, s = paged.bounds(paged.rows_of(data, [page], 0, h, hnd)[:n])
            assert np.array_equal(codes[page, h], c) and scales[page, h] == s, (page, h)
    assert (codes[untouched] == 77).all() and (scales[untouched] == 77).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("runs, page, h, d, layout", [
    ([(0, 1)], 16, 1, 64, "NHD"), ([(5, 1), (0, 16), (3, 9), (15, 1)], 16, 3, 128, "HND"),
    ([(0, 300), (2, 61), (127, 2)], 128, 2, 256, "NHD"), ([(i % 8, 1) for i in range(200)], 8, 8, 128, "NHD"),
    ([(0, 5), (0, 1)], 1, 2, 64, "HND"), ([(7, 3000)], 16, 2, 64, "NHD"), ([(1, 40), (31, 33)], 32, 5, 128, "HND")])
def test_bounds_equal_restated(runs, page, h, d, layout, dtype):
    """Runs of (first slot in its page, tokens): pages partly filled before, written anew, ended inside."""
    rng = np.random.default_rng(d + len(runs))
    slots, pages, filled = [], [], []
    need = sum(-(-(a + n) // page) for a, n in runs)
    ids = rng.permutation(need + 5)
    at = 0
    for a, n in runs:
        used = -(-(a + n) // page)
        t = np.arange(a, a + n)
        slots += list(ids[at + t // page] * page + t % page) + [-1]
        pages += list(ids[at: at + used])
        filled += [page] * (used - 1) + [(a + n - 1) % page + 1]
        at += used
    cache = pa.KvCache(need + 5, page, h, d, dtype, layout, bounds=True)
    cache.data.copy_(torch.randn(cache.data.shape, device="cuda"))
    mid = cache.data[:, 0] if layout == "NHD" else cache.data[:, 0].transpose(1, 2)  # [pages, slots, heads, d]
    mid *= torch.from_numpy(np.exp(rng.normal(0, 2, (need + 5, 1, h, 1)))).cuda()
    mid[int(pages[0]), :filled[0]] = 0.0
    if len(pages) > 3:
        mid[int(pages[1]), 0, 0, 5] = float("nan")
        mid[int(pages[2]), filled[2] - 1, h - 1, d - 1] = -float("inf")
        mid[int(pages[3]), :filled[3], 0] = 2.0 ** -20 if dtype == torch.float16 else 2.0 ** -110
    for p, n in zip(pages, filled):
        mid[int(p), n:] = float("nan")  # slots behind the last one written
    cache.bounds.fill_(77)
    cache.bound_scales.fill_(77)
    cache.update_bounds(dev(np.array(slots), torch.int64))
    assert cache.device_status() == 0
    check_bounds(cache, pages, filled, ids[need:])


@gpu
def test_bounds_follow_appends():
    """A page filled over several steps, given back and filled again: its bounds are always those of its keys."""
    cache = pa.KvCache(3, 16, 2, 64, torch.bfloat16, "HND", bounds=True)
    cache.bounds.fill_(77)
    cache.bound_scales.fill_(77)
    rope = pa.Rope(frequencies(32))
    for first, n, gain in ((0, 5, 30.0), (5, 1, 1.0), (6, 10, 1.0), (0, 3, 0.1)):
        k = gain * torch.randn(n, 2, 64, device="cuda")
        slots = 16 + torch.arange(first, first + n, device="cuda")
        cache.append(k.bfloat16(), k.bfloat16(), slots, rope=rope, positions=slots.int())
        check_bounds(cache, [1], [first + n], [0, 2])
    assert cache.device_status() == 0


@gpu
def test_cache_python_refusals():
    z = lambda *s, t=torch.float16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    plain = pa.KvCache(4, 16, 2, 64, torch.float16)
    assert plain.bounds is None
    slots, k = z(3, t=torch.int64), z(3, 2, 64)
    with pytest.raises(pa.PagedAttnError):
        plain.update_bounds(slots)
    for kw in (dict(head_dim=96), dict(num_pages=0), dict(data=z(4, 2, 2, 16, 64)), dict(data=z(4, 2, 16, 2, 64).bfloat16()),
               dict(bounds=z(4, 2, 2, 64, t=torch.int8)), dict(bound_scales=z(4, 2, t=torch.float32)), dict(dtype=torch.float32)):
        with pytest.raises(pa.PagedAttnError):
            pa.KvCache(**{**dict(num_pages=4, page_size=16, num_kv_heads=2, head_dim=64, dtype=torch.float16), **kw})
    rope, pos, q = pa.Rope([1.0] * 8), z(3, t=I32), z(3, 4, 64)
    good = dict(k=k, v=k, slot_mapping=slots - 1, rope=rope, positions=pos, q=q)
    plain.append(**good)
    for kw in (dict(k=z(3, 2, 128)), dict(v=z(2, 2, 64)), dict(slot_mapping=pos), dict(rope=None), dict(positions=None),
               dict(rope=None, positions=None), dict(q=z(3, 4, 128)), dict(q=None, q_out=q), dict(q=q.bfloat16()),
               dict(k=k.bfloat16()), dict(q_out=z(3, 5, 64)), dict(positions=z(4, t=I32))):
        with pytest.raises(pa.PagedAttnError):
            plain.append(**{**good, **kw})


# ---------------------------------------------------------------- selection and attention


class Batch:
    """Requests of the given lengths over permuted pages; unused slots hold NaN, and the bounds are the pages'."""

    def __init__(self, qo, kv, Hq, Hkv, D, page, layout, dtype, seed=0, pad=0, q_gain=1.0):
        rng = np.random.default_rng(seed)
        self.qo, self.kv, self.page, self.Hq, self.Hkv, self.D, self.dtype = qo, kv, page, Hq, Hkv, D, dtype
        n = [-(-k // page) for k in kv]
        self.qo_indptr = np.concatenate([[0], np.cumsum(qo)]).astype(np.int32)
        self.page_indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.pages = rng.permutation(int(self.page_indptr[-1]) + 3)[: int(self.page_indptr[-1])].astype(np.int32)
        self.last = np.array([k - (m - 1) * page if m else 0 for k, m in zip(kv, n)], np.int32)
        self.T, self.pad, self.hnd = int(self.qo_indptr[-1]) + pad, pad, layout == "HND"
        num_pages = len(self.pages) + 3
        self.cache = pa.KvCache(num_pages, page, Hkv, D, dtype, layout, bounds=True)
        g = torch.Generator(device="cuda").manual_seed(seed)
        centre = torch.randn((num_pages, 1, 1, 1, D), generator=g, device="cuda")
        self.cache.data.copy_(0.7 * torch.randn(self.cache.data.shape, generator=g, device="cuda") + 0.7 * centre)
        slots = np.concatenate([[]] + [self.pages[self.page_indptr[b] + np.arange(k) // page].astype(np.int64) * page + np.arange(k) % page
                                       for b, k in enumerate(kv)]).astype(np.int64)
        used = torch.zeros(num_pages * page, dtype=torch.bool, device="cuda")
        used[dev(slots, torch.int64)] = True
        used = used.view((num_pages, 1, 1, page, 1) if self.hnd else (num_pages, 1, page, 1, 1))
        self.cache.data.masked_fill_(~used, float("nan"))
        self.cache.update_bounds(dev(slots, torch.int64))
        self.q = (q_gain * torch.randn((self.T, Hq, D), generator=g, device="cuda")).to(dtype)

    def tables(self):
        return tuple(dev(a) for a in (self.qo_indptr, self.page_indptr, self.pages, self.last))

    def attention(self, num_blocks, first=0, last=1, max_kv=None, **kw):
        return pa.BlockAttention(len(self.kv), self.T, self.Hq, self.Hkv, self.D, self.page, self.dtype, num_blocks,
                                 max([*self.kv, 0]) if max_kv is None else max_kv, first, last, **kw)

    def lists(self, num_blocks, first=0, last=1):
        """The selection restated."""
        q, G = host(self.q), self.Hq // self.Hkv
        codes, scales = self.cache.bounds.cpu().numpy(), self.cache.bound_scales.cpu().numpy()
        out = np.full((self.T, self.Hkv, num_blocks), -5, np.int32)
        for i, (_, start, _, pos) in enumerate(paged.queries(self.qo_indptr, self.page_indptr, self.last, self.page)):
            ids = self.pages[start: start + (pos // self.page + 1 if pos >= 0 else 0)]
            for h in range(self.Hkv):
                c = paged.query_codes(q[i, h * G: (h + 1) * G])
                out[i, h] = paged.select(paged.scores(c, codes[ids, h], scales[ids, h]), num_blocks, first, last)
        return out

    def want(self, lists):
        n = self.T - self.pad
        return paged.attention(host(self.q[:n]), self.cache.data.float().cpu().numpy(), lists, self.qo_indptr,
                               self.page_indptr, self.pages, self.last, self.page, self.hnd)

    def check(self, out, lse, want):
        """Error bounds of the kernel's arithmetic, from fp64 sums over each row's keys.

        logits  fp32 sums of exact products in D/16 steps, truncated at worst: ds = 2^-22 (D/16 + 2) sum |q k| scale
        p       exp2 and its argument: 2^-21, and ds; both in numerator and normaliser, hence twice
        P       fp16: 2^-11 of each p, and 2^-25 of the largest where p is a subnormal; bf16: two terms, 2^-16; in
                requests of more than 32 packed rows half a step of either type
        sums    fp32 products of P V over n / 16 steps: 2^-23 (n / 16 + 8) of sum p |v|
        out     half a step of its type
        lse     ds, 2^-20, the fp32 sum of n terms and the last roundings
        """
        n = self.T - self.pad
        ref, ref_lse, sp = want
        eps = torch.finfo(self.dtype).eps / 2
        ds = 2.0 ** -22 * (self.D / 16 + 2) * sp["s"]
        long = np.repeat([q * (self.Hq // self.Hkv) > 32 and q > 1 and self.page >= 8 for q in self.qo], self.qo)[:, None]
        rel = 2 * (ds + 2.0 ** -21) + np.where(long, eps, 2.0 ** -11 if self.dtype == torch.float16 else 2.0 ** -16) + \
            2.0 ** -23 * (sp["n"] / 16 + 8)
        bound = (rel[..., None] * sp["av"] + 2.0 ** -25 * sp["v"]) * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25
        err = np.abs(host(out[:n]) - ref)
        assert (err <= bound).all(), (err / bound).max()
        got = host(lse[:n])
        none = np.isneginf(ref_lse)
        assert (np.isneginf(got) == none).all() and (err[none] == 0).all()
        bound = ds + 2.0 ** -20 + 2.0 ** -24 * (sp["n"] / 16 + 64) + 2.0 ** -22 * np.abs(np.where(none, 0, ref_lse))
        lerr = np.abs(np.where(none, 0, got) - np.where(none, 0, ref_lse))
        assert (lerr <= bound).all(), (lerr / bound).max()


SHAPES = [
    # qo, kv, Hq, Hkv, D, page, layout, blocks, first, last
    ([1], [1], 1, 1, 64, 16, "NHD", 4, 0, 1),
    ([1], [77], 8, 1, 128, 16, "NHD", 3, 1, 1),
    ([1] * 5, [1, 63, 64, 65, 1000], 8, 2, 64, 32, "HND", 5, 1, 2),
    ([1, 1], [2049, 300], 16, 2, 128, 64, "NHD", 7, 0, 3),
    ([1, 1, 1], [130, 5, 700], 4, 1, 256, 16, "NHD", 9, 2, 2),
    ([1, 1, 1], [130, 5, 700], 24, 2, 256, 128, "HND", 2, 1, 1),
    ([1] * 4, [33, 100, 7, 258], 6, 2, 128, 1, "NHD", 40, 3, 5),
    ([1] * 4, [33, 100, 7, 258], 10, 2, 64, 4, "HND", 11, 1, 2),
    ([1, 2, 3], [40, 41, 300], 7, 1, 128, 8, "NHD", 6, 1, 1),
    ([0, 1, 0, 2, 0], [50, 60, 0, 70, 16], 4, 2, 128, 16, "NHD", 3, 1, 1),  # idle requests
    ([2, 1, 5], [0, 0, 3], 4, 2, 128, 16, "HND", 2, 1, 1),                  # rows that see no key
    ([33, 5], [33, 700], 4, 4, 128, 16, "NHD", 8, 1, 2),
    ([40, 1], [200, 300], 34, 2, 64, 16, "HND", 5, 0, 1),                   # groups of 17
    ([17, 66], [90, 66], 8, 2, 256, 32, "NHD", 2, 0, 2),
    ([100], [333], 33, 1, 128, 16, "NHD", 7, 2, 2),                         # a group of 33
    ([1, 1], [9000, 5000], 128, 1, 64, 16, "HND", 129, 1, 1),               # a group of 128
    ([20], [4100], 16, 1, 128, 64, "NHD", 16, 1, 1),
    ([3, 1], [1500, 40], 5, 5, 128, 2, "HND", 200, 1, 1),
]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%s-%s-%d.%d.%d-p%d%s-%d" % (
    "_".join(map(str, s[0])), "_".join(map(str, s[1])), *s[2:8]))
def test_selection_and_attention_equal_restated(shape, dtype):
    *base, blocks, first, last = shape
    b = Batch(*base, dtype, seed=len(shape[0]) + shape[4], pad=3)
    a = b.attention(blocks, first, last)
    got = torch.full((b.T, b.Hkv, blocks), -5, dtype=I32, device="cuda")
    a.select(b.q, b.cache, b.tables(), out=got)
    lists = b.lists(blocks, first, last)
    np.testing.assert_array_equal(got.cpu().numpy(), lists)  # rows behind the last sequence as well
    out = torch.full((b.T, b.Hq, b.D), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((b.T, b.Hq), 9.0, device="cuda")
    a.run(b.q, b.cache, b.tables(), got, out=out, lse=lse)
    assert a.device_status() == 0
    b.check(out, lse, b.want(lists))
    assert (out[-3:] == 9.0).all() and (lse[-3:] == 9.0).all()


@gpu
def test_bounds_hold_for_every_key():
    """A page's score is no less than the sum of its group's logits for any of its keys, but for what q's codes round:
    half a code (1/254 of the largest channel sum) in each channel of each part."""
    b = Batch([1] * 3, [700, 90, 1000], 12, 3, 128, 16, "NHD", torch.bfloat16, seed=2)
    q, data = host(b.q), b.cache.data.float().cpu().numpy().astype(np.float64)
    codes, scales = b.cache.bounds.cpu().numpy(), b.cache.bound_scales.cpu().numpy()
    for i in range(3):
        for h in range(3):
            g = q[i, 4 * h: 4 * h + 4]
            parts = np.concatenate([np.maximum(g, 0).sum(0), np.minimum(g, 0).sum(0)])
            unit = np.abs(parts).max() / 127
            ids = b.pages[b.page_indptr[i]: b.page_indptr[i + 1]]
            z = paged.scores(paged.query_codes(g), codes[ids, h], scales[ids, h]) * unit
            for n, page in enumerate(ids):
                keys = data[page, 0, :, h][: b.last[i] if n == len(ids) - 1 else 16]
                slack = 0.5 * unit * np.abs(codes[page, h].astype(float) * scales[page, h]).sum() * 1.01
                assert (keys @ g.sum(0)).max() <= z[n] + slack


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_selection_with_equal_scores(dtype):
    """Equal bounds, zero queries, negative zeros: the lowest indices among equals, whatever the cut."""
    for kv, blocks, first, last in (([3000, 700], 20, 0, 1), ([40000], 70, 3, 4)):
        b = Batch([1] * len(kv), kv, 4, 2, 64, 16, "NHD", dtype, seed=1)
        rng = np.random.default_rng(3)
        b.cache.bounds.copy_(b.cache.bounds[int(b.pages[0])].clone())
        b.cache.bound_scales.copy_(torch.from_numpy(rng.choice([0.0, 0.5, 1.0], b.cache.bound_scales.shape)))
        b.cache.bound_scales[0, 0] = float("inf")
        for q in (b.q.clone(), torch.zeros_like(b.q), -b.q.abs()):
            b.q = q
            got = b.attention(blocks, first, last).select(b.q, b.cache, b.tables())
            np.testing.assert_array_equal(got.cpu().numpy(), b.lists(blocks, first, last))


@gpu
@pytest.mark.parametrize("kind", ["nan", "inf", "tiny", "huge", "one"])
def test_selection_of_unusual_queries(kind):
    b = Batch([1, 1, 6], [700, 300, 500], 8, 2, 128, 16, "HND", torch.bfloat16, seed=4)
    if kind in ("nan", "inf"):
        b.q[0, 3, 5] = float(kind)
        b.q[4, 7, 127] = -float(kind)
    elif kind == "one":
        b.q.zero_()
        b.q[:, :, 17] = 3.0
    else:
        b.q *= 2.0 ** (-120 if kind == "tiny" else 120)
    got = b.attention(9, 1, 1).select(b.q, b.cache, b.tables())
    np.testing.assert_array_equal(got.cpu().numpy(), b.lists(9, 1, 1))


@gpu
@pytest.mark.parametrize("qo, kv, Hkv, page, blocks", [
    ([1], [150_000], 1, 16, 128), ([1, 1], [30_000, 9000], 3, 1, 700), ([1], [20_000], 1, 1, 4096),
    ([40, 2], [20_000, 12_000], 2, 1, 300), ([320, 2, 4], [5000, 300, 3900], 2, 1, 60),
    ([310, 300, 1], [8000, 7000, 30], 1, 1, 100), ([210, 1], [2900, 8000], 3, 1, 5), ([1] * 300, [2000] * 300, 2, 16, 20)], ids=str)
def test_selection_of_many_pages(qo, kv, Hkv, page, blocks):
    """Items cut into slices; more keys than shared memory keeps; several launches of one call."""
    b = Batch(qo, kv, 2 * Hkv, Hkv, 64, page, "NHD", torch.float16, seed=8)
    a = b.attention(blocks, 2, 3)
    got = [a.select(b.q, b.cache, b.tables()) for _ in range(3)]
    assert a.device_status() == 0
    np.testing.assert_array_equal(got[0].cpu().numpy(), b.lists(blocks, 2, 3))
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])


@gpu
def test_selection_does_not_depend_on_the_batch():
    """One request alone, in a large batch and in a chunk: the same lists, and the same attention up to how it is cut."""
    many = Batch([1] * 200, [3000] * 200, 8, 1, 128, 16, "NHD", torch.bfloat16, seed=5)
    got = many.attention(30, 1, 2).select(many.q, many.cache, many.tables())
    for r in (0, 77, 199):
        p = many.pages[many.page_indptr[r]: many.page_indptr[r + 1]]
        t = tuple(dev(x) for x in ([0, 1], [0, len(p)], p, many.last[r: r + 1]))
        a = pa.BlockAttention(1, 1, 8, 1, 128, 16, torch.bfloat16, 30, 3000, 1, 2)
        assert torch.equal(a.select(many.q[r: r + 1], many.cache, t)[0], got[r])


@gpu
def test_no_room_for_the_pages():
    b = Batch([1, 2, 1], [200, 700, 100], 4, 2, 64, 16, "NHD", torch.float16, seed=6)
    a = b.attention(5, 1, 1, max_kv=200)
    got = a.select(b.q, b.cache, b.tables()).cpu().numpy()
    assert a.device_status() == raw.PA_DEV_NO_ROOM and a.device_status() == 0
    want = b.lists(5, 1, 1)
    want[1:3] = -1
    np.testing.assert_array_equal(got, want)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunk, kv, blocks", [(40, 130, 12), (520, 1300, 64)])
def test_attention_over_the_callers_lists(chunk, kv, blocks, dtype):
    """Lists without the query's own block, empty, of blocks that the query does not see, of none that exist, out of
    order and with repetitions: for single tokens, and for chunks."""
    b = Batch([1, chunk, 1, 3], [300, kv, 40, 100], 8, 2, 128, 16, "NHD", dtype, seed=9)
    rng = np.random.default_rng(1)
    pages = np.repeat([19, -(-kv // 16), 3, 7], b.qo)
    lists = np.full((b.T, 2, blocks), -1, np.int32)
    for i in range(b.T):
        for h in range(2):
            mine = np.sort(rng.permutation(pages[i])[: rng.integers(0, min(blocks, pages[i]) + 1)])
            lists[i, h, : len(mine)] = mine
    lists[2, 1] = -1
    a = b.attention(blocks)
    out, lse = a.run(b.q, b.cache, b.tables(), dev(lists))
    b.check(out, lse, b.want(lists))
    assert a.device_status() == 0 and torch.isneginf(lse[2, 4:]).all() and not out[2, 4:].any()
    bad = lists.copy()
    bad[0, 0, :3] = [4, 4, 5]
    bad[7, 1, :4] = [0, 3, 2, 5]
    bad[20, 0, :3] = [-1, 2, 3]
    bad[1, 0, :5] = [0, 1, 2, 1, -1]  # the first token of a chunk
    bad[chunk + 1, 0, :3] = [2, 2, -1]
    bad[chunk + 1, 1, :4] = [0, -1, 1, -1]
    for wrong in (bad, lists.copy()):
        wrong[12, 0, :5] = [0, 2, pages[12], pages[12] + 70, -1]  # beyond its request's pages
        wrong[12, 0, 5:] = -1
        wrong[-1, 1, :3] = [0, 7, -1]
        wrong[-1, 1, 3:] = -1
        out, lse = a.run(b.q, b.cache, b.tables(), dev(wrong))
        assert a.device_status() == pa.PA_DEV_BAD_INDEX
        b.check(out, lse, b.want(wrong))


@gpu
@pytest.mark.parametrize("n, blocks", [(20, 5), (600, 60)])
def test_requests_longer_than_they_may_be(n, blocks):
    b = Batch([1, n, 1], [200, 700 + n, 100], 4, 2, 64, 16, "NHD", torch.float16, seed=6)
    lists = b.attention(blocks).select(b.q, b.cache, b.tables())
    want = b.attention(blocks).run(b.q, b.cache, b.tables(), lists)
    a = b.attention(blocks, max_kv=208)
    out, lse = a.run(b.q, b.cache, b.tables(), lists)
    assert a.device_status() == raw.PA_DEV_NO_ROOM and not out[1: n + 1].any() and torch.isneginf(lse[1: n + 1]).all()
    for r in (0, n + 1):
        assert torch.equal(out[r], want[0][r]) and torch.equal(lse[r], want[1][r])


CHUNKS = [
    # qo, kv, Hq, Hkv, D, page, layout, blocks: long requests of a million keys of single tokens or more
    ([600], [1200], 8, 1, 128, 16, "NHD", 128), ([270, 64, 1, 9], [3000, 64, 900, 40], 8, 2, 128, 16, "HND", 100),
    ([400, 33], [1111, 2000], 16, 2, 64, 32, "NHD", 40), ([450], [6000], 8, 1, 256, 64, "HND", 40),
    ([140, 170], [900, 175], 20, 4, 128, 8, "NHD", 110), ([460], [2500], 3, 3, 64, 128, "NHD", 6),
    ([560], [2901], 2, 1, 128, 16, "HND", 120), ([320, 17], [1600, 300], 48, 1, 64, 16, "NHD", 200),
    ([65], [1500], 72, 1, 64, 64, "NHD", 260), ([65], [700], 7, 1, 256, 8, "HND", 2100),
    ([40] * 30 + [1] * 50, [300] * 40 + [77] * 40, 8, 1, 64, 16, "NHD", 56), ([512], [20_000], 8, 1, 128, 16, "NHD", 130),
    ([64, 0, 2, 64], [10, 5, 2, 100], 4, 1, 128, 16, "HND", 4096), ([700], [4000], 8, 1, 128, 16, "NHD", 100),
    ([300, 20], [3000, 500], 16, 2, 64, 16, "HND", 120), ([280], [5000], 4, 1, 256, 64, "NHD", 60),
    ([500, 90, 4], [2000, 90, 900], 5, 1, 128, 32, "NHD", 60), ([40, 3], [700, 90], 8, 1, 128, 16, "NHD", 30)]


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", CHUNKS, ids=lambda s: "%s-%d.%d.%d-p%d%s" % ("_".join(map(str, s[0][:4])), *s[2:7]))
def test_chunks_equal_restated(shape, dtype):
    """Long requests through row tiles, beside short ones; the same lists through single tokens agree within both bounds."""
    *base, blocks = shape
    b = Batch(*base, dtype, seed=len(shape[0]) + shape[4], pad=2)
    a = b.attention(blocks, 1, 1)
    lists = a.select(b.q, b.cache, b.tables())
    np.testing.assert_array_equal(lists.cpu().numpy()[:-2], b.lists(blocks, 1, 1)[:-2])
    want = b.want(lists.cpu().numpy())
    out = torch.full((b.T, b.Hq, b.D), 9.0, dtype=dtype, device="cuda")
    lse = torch.full((b.T, b.Hq), 9.0, device="cuda")
    for _ in range(2):
        a.run(b.q, b.cache, b.tables(), lists, out=out, lse=lse)
        assert a.device_status() == 0
        b.check(out, lse, want)
        assert (out[-2:] == 9.0).all() and (lse[-2:] == 9.0).all()
    long = sum(n for n in b.qo if n > 1 and n * (b.Hq // b.Hkv) > 32)
    assert long * b.Hkv * blocks * b.page >= 1 << 20 or b.qo == [40, 3]
    one = b.attention(blocks, 1, 1, max_qo_len=1)  # a bound that does not hold costs time, not results
    out, lse = one.run(b.q, b.cache, b.tables(), lists)
    b.check(out, lse, want)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kv, Hq, Hkv, D, page, blocks", [
    ([20_000], 8, 1, 128, 16, 1250), ([5000, 3, 900], 6, 2, 64, 64, 79), ([9000], 16, 1, 128, 1, 4096),
    ([3000, 2000], 8, 2, 256, 32, 94), ([30_000], 128, 1, 64, 128, 235)], ids=str)
def test_attention_of_cut_lists(kv, Hq, Hkv, D, page, blocks, dtype):
    """Few queries of long lists: slices joined by the last of them, run after run in one workspace, bit for bit."""
    b = Batch([1] * len(kv), kv, Hq, Hkv, D, page, "HND", dtype, seed=12)
    a = b.attention(blocks, 0, 1)
    lists = a.select(b.q, b.cache, b.tables())
    runs = [a.run(b.q, b.cache, b.tables(), lists) for _ in range(3)]
    assert a.device_status() == 0
    b.check(*runs[0], b.want(lists.cpu().numpy()))
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kv", [900, 9000])
def test_attention_keeps_a_long_tail(kv, dtype):
    """One key of 2^20 times the others' weight and values of zero: the outputs are the others' sum.

    With the reference 7 below the dominant logit the others' P is 2^7 * 2^-20, which fp16 rounds by at most 2^-25:
    2^-12 of it; logits and weights add less than 2^-10, the output rounds by half a step (v keeps it a normal number)."""
    H, D, page = 2, 128, 16
    n = -(-kv // page)
    cache = pa.KvCache(n, page, H, D, dtype)
    k = torch.zeros(kv, H, D, dtype=dtype, device="cuda")
    v = torch.full((kv, H, D), 16384.0, dtype=dtype, device="cuda")
    k[kv // 5, :, 0] = 4.0
    v[kv // 5] = 0.0
    cache.append(k, v, torch.arange(kv, device="cuda"))
    q = torch.zeros(1, 2 * H, D, dtype=dtype, device="cuda")
    q[..., 0] = 20 * np.log(2) * D ** 0.5 / 4
    a = pa.BlockAttention(1, 1, 2 * H, H, D, page, dtype, n, kv)
    tables = tuple(dev(x) for x in ([0, 1], [0, n], range(n), [kv - (n - 1) * page]))
    out, lse = a.run(q, cache, tables, torch.arange(n, dtype=I32, device="cuda").expand(1, H, n).contiguous())
    logit = float(q[0, 0, 0]) * 4 / D ** 0.5
    w = (kv - 1) * np.exp(-logit)
    rel = (out.double() / (16384 * w / (1 + w)) - 1).abs().max().item()
    assert rel <= 2.0 ** -12 + 2.0 ** -10 + torch.finfo(dtype).eps / 2, rel
    assert (lse.double() - (logit + np.log1p(w))).abs().max().item() <= 2.0 ** -17


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("qo, kv, Hq, D, page, gain", [
    ([1, 1, 1], [700, 9, 3000], 16, 64, 16, 1e4), ([1], [5000], 8, 128, 2, 1e4), ([1, 1], [900, 40], 8, 256, 32, 1e4),
    ([1, 2], [333, 600], 24, 128, 16, 500.0), ([300], [900], 16, 128, 16, 500.0)], ids=str)
def test_attention_of_large_logits(qo, kv, Hq, D, page, gain, dtype):
    """Logits of 10^8 and more (or 10^6): rows whose largest stands out take its value.

    Its weight is off by half a step of the type at most, as is the output: twice eps / 2.  The others' logits lie
    two bounds of the fp32 sums and 40 below it: less than 2^-40 together.  lse: that bound, 2^-20 for
    exp2 and log2, and six roundings of 2^-24 (two factors, their products, the reference, its sum with the log)."""
    b = Batch(qo, kv, Hq, Hq // 2 if len(qo) == 1 and qo[0] > 1 else 2, D, page, "NHD", dtype, seed=8, q_gain=gain)
    b.cache.data.mul_(gain)
    b.cache.data[:, 1].div_(gain)
    b.cache.data.clamp_(-6e4, 6e4)
    b.q.clamp_(-6e4, 6e4)
    blocks = -(-max(kv) // page)
    lists = np.broadcast_to(np.arange(blocks, dtype=np.int32), (b.T, b.Hkv, blocks)).copy()
    for i, (_, _, n, _) in enumerate(paged.queries(b.qo_indptr, b.page_indptr, b.last, page)):
        lists[i, :, n:] = -1
    ref, ref_lse, sp = b.want(lists)
    ds = 2.0 ** -22 * (D / 16 + 2) * sp["s"]
    G = b.Hq // b.Hkv
    data, q = b.cache.data.double().cpu().numpy(), host(b.q)
    clear = np.zeros((b.T, b.Hq), bool)
    for i, (_, start, n, pos) in enumerate(paged.queries(b.qo_indptr, b.page_indptr, b.last, page)):
        k = data[b.pages[start: start + n], 0].reshape(-1, b.Hkv, D)[: pos + 1]
        z = np.sort(np.einsum("nhd,hgd->hgn", k, q[i].reshape(b.Hkv, G, D)).reshape(b.Hq, -1) / np.sqrt(D))
        clear[i] = z[:, -1] - z[:, -2] > 2 * ds[i] + 40
    assert clear.mean() > 0.8 and np.abs(ref_lse).max() > (1e8 if gain > 1e3 else 1e5)
    a = b.attention(blocks)
    out, lse = a.run(b.q, b.cache, b.tables(), dev(lists))
    assert a.device_status() == 0
    out, lse = host(out), host(lse)
    assert np.isfinite(out).all()
    assert (np.abs(lse - ref_lse) <= ds + 6 * 2.0 ** -24 * np.abs(ref_lse) + 2.0 ** -20)[clear].all()
    eps = torch.finfo(dtype).eps
    assert (np.abs(out - ref) <= eps * (1 + eps) * np.abs(ref) + 2.0 ** -25)[clear].all()


@gpu
def test_attention_nan_stays_its_own():
    """A NaN of q reaches its row, one of K or V the rows of its kv head that list its page and see it."""
    b = Batch([1, 2, 1], [100, 100, 100], 8, 2, 128, 16, "NHD", torch.float16, seed=2)
    a = b.attention(7)
    lists = a.select(b.q, b.cache, b.tables())
    clean, _ = a.run(b.q, b.cache, b.tables(), lists)
    b.q[0, 3, 5] = float("nan")
    page = int(b.pages[b.page_indptr[1] + 6])
    b.cache.data[page, 0, 3, 1, 7] = float("nan")  # key 99, the second query's own
    b.cache.data[int(b.pages[b.page_indptr[2]]), 1, 4, 0, 9] = float("inf")
    out, lse = a.run(b.q, b.cache, b.tables(), lists)
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[0, 3] = True
    hit[2, 4:] = True
    assert torch.equal(torch.isnan(out), hit)
    assert (out[3, :4, 9] == float("inf")).all()
    hit[3, :4, 9] = True
    assert torch.equal(out[~hit], clean[~hit])


@gpu
def test_strided_q_no_lse_and_layouts():
    for layout in ("NHD", "HND"):
        b = Batch([1, 5], [100, 330], 8, 2, 64, 16, layout, torch.float16, seed=12)
        fused = torch.zeros(b.T, 8 * 64 + 24, dtype=torch.float16, device="cuda")
        fused[:, 8: 8 + 512] = b.q.flatten(1)
        q, a = fused[:, 8: 520].view(b.T, 8, 64), b.attention(6)
        lists = a.select(q, b.cache, b.tables())
        assert torch.equal(lists, a.select(b.q, b.cache, b.tables()))
        want, _ = a.run(b.q, b.cache, b.tables(), lists)
        out, lse = a.run(q, b.cache, b.tables(), lists, return_lse=False)
        assert lse is None and torch.equal(out, want)


@gpu
def test_bad_tables_are_contained():
    b = Batch([1, 1, 1], [100, 60, 40], 8, 2, 128, 16, "NHD", torch.float16, seed=13)
    lists = b.attention(3).select(b.q, b.cache, b.tables())
    want = b.attention(3).run(b.q, b.cache, b.tables(), lists)
    for which, at, value in (("last", 1, 17), ("last", 1, 0), ("pages", int(b.page_indptr[1]), 1 << 20),
                             ("pages", int(b.page_indptr[1]), -1), ("page_indptr", 2, 1 << 20), ("qo_indptr", 2, 5)):
        good = getattr(b, which).copy()
        getattr(b, which)[at] = value
        a = b.attention(3)
        some = torch.full_like(lists, -5)
        a.select(b.q, b.cache, b.tables(), out=some)
        assert a.device_status() == pa.PA_DEV_BAD_INDEX
        out, lse = a.run(b.q, b.cache, b.tables(), lists)
        flags = a.device_status()
        assert flags == (pa.PA_DEV_BAD_INDEX if which != "pages" or (lists[1] == 0).any() else 0)
        keep = (0,) if which.endswith("indptr") else (0, 2)
        for r in keep:
            assert torch.equal(some[r], lists[r]) and torch.equal(out[r], want[0][r]) and torch.equal(lse[r], want[1][r])
        setattr(b, which, good)


@gpu
def test_empty_calls():
    cache = pa.KvCache(4, 16, 2, 64, torch.float16, bounds=True)
    z = lambda *s: torch.zeros(s, dtype=I32, device="cuda")  # noqa: E731
    for B, T in ((0, 0), (3, 0), (0, 4), (3, 4)):
        a = pa.BlockAttention(B, T, 4, 2, 64, 16, torch.float16, 3, 100)
        out = torch.full((T, 4, 64), 5.0, dtype=torch.float16, device="cuda")
        lists = torch.full((T, 2, 3), -5, dtype=I32, device="cuda")
        tables = (z(B + 1), z(B + 1), z(0), z(B))
        a.select(torch.zeros_like(out), cache, tables, out=lists)
        got, lse = a.run(torch.zeros_like(out), cache, tables, lists, out=out)
        assert (got == 5.0).all() and (lists == -5).all() and a.device_status() == 0
    k = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    cache.append(k, k, torch.zeros(0, dtype=torch.int64, device="cuda"))
    cache.update_bounds(torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert cache.device_status() == 0


@gpu
def test_block_attention_python_refusals():
    b = Batch([1, 5], [100, 30], 8, 2, 64, 16, "NHD", torch.float16, seed=12)
    for kw in (dict(first=-1), dict(last=0), dict(first=3, last=3), dict(num_blocks=0), dict(num_blocks=5000, last=1),
               dict(dtype=torch.float32), dict(head_dim=96), dict(max_kv_len=-1), dict(workspace=torch.zeros(9, device="cuda")),
               dict(workspace=pa.Kv4Attention(1, 1, 1, 1, 64, 16, torch.float16))):
        with pytest.raises(pa.PagedAttnError):
            pa.BlockAttention(**{**dict(batch_size=2, num_tokens=6, num_qo_heads=8, num_kv_heads=2, head_dim=64, page_size=16,
                                        dtype=torch.float16, num_blocks=5, max_kv_len=100), **kw})
    a, t = b.attention(5), b.tables()
    lists = a.select(b.q, b.cache, t)
    plain = pa.KvCache(9, 16, 2, 64, torch.float16)
    for kw in (dict(q=b.q[:5]), dict(q=b.q.bfloat16()), dict(cache=plain), dict(tables=t[:3] + (t[3][:1],)),
               dict(tables=(t[0].long(), *t[1:])), dict(out=lists[:, :, :4]), dict(out=lists.long()),
               dict(cache=pa.KvCache(9, 16, 2, 64, torch.bfloat16, bounds=True))):
        with pytest.raises(pa.PagedAttnError):
            a.select(**{**dict(q=b.q, cache=b.cache, tables=t), **kw})
    for kw in (dict(blocks=lists[:, :, :4]), dict(blocks=lists.long()), dict(lse=lists), dict(out=b.q[:5]),
               dict(cache=pa.KvCache(9, 32, 2, 64, torch.float16))):
        with pytest.raises(pa.PagedAttnError):
            a.run(**{**dict(q=b.q, cache=b.cache, tables=t, blocks=lists), **kw})
    a.run(b.q, plain, t, lists)  # the attention needs no bounds


# ---------------------------------------------------------------- the step


@gpu
@pytest.mark.parametrize("layout, dtype", [("NHD", torch.bfloat16), ("HND", torch.float16)])
def test_captured_step_grows_requests(layout, dtype):
    """Tables, append with rotation and bounds, selection and attention in one graph, replayed while requests grow."""
    B, page, Hq, Hkv, D, blocks, steps, num_pages = 3, 4, 4, 2, 64, 5, 30, 60
    rng = np.random.default_rng(0)
    kv = np.array([9, 0, 22])
    table = np.full((B, 20), -1, np.int32)
    ids = rng.permutation(num_pages).astype(np.int32)
    held = -(-kv // page)
    at = 0
    for r in range(B):
        table[r, : held[r]] = ids[at: at + held[r]]
        at += held[r]
    free = ids[at:]
    tables = pa.BatchTables(B, B + 2, num_pages, page, num_pages)
    cache = pa.KvCache(num_pages, page, Hkv, D, dtype, layout, bounds=True)
    cache.data.fill_(float("nan"))
    w = frequencies(24)
    rope, att = pa.Rope(w, interleaved=True), pa.BlockAttention(B, B + 2, Hq, Hkv, D, page, dtype, blocks, 80, 1, 2)
    # the keys cached so far, as an earlier append left them
    k0, v0 = (torch.from_numpy(rng.standard_normal((int(kv.sum()), Hkv, D))).to(dtype).cuda() for _ in range(2))
    t = np.concatenate([np.arange(n) for n in kv])
    slots0 = np.concatenate([table[r, np.arange(n) // page] * page + np.arange(n) % page for r, n in enumerate(kv)])
    cache.append(k0, v0, dev(slots0, torch.int64), rope=rope, positions=dev(t))
    qo, table_t, free_t = dev(np.ones(B)), dev(table), dev(free)
    tables.kv_lens.copy_(dev(kv))
    tables.free_count.fill_(len(free))
    qkv = torch.zeros(B + 2, (Hq + 2 * Hkv) * D, dtype=dtype, device="cuda")
    q, k, v = (qkv[:, a * D: (a + n) * D].view(B + 2, n, D) for a, n in ((0, Hq), (Hq, Hkv), (Hq + Hkv, Hkv)))

    def step():
        tables.build(qo, tables.kv_lens, table_t, free_t, tables.free_count)
        turned = cache.append(k, v, tables.slot_mapping, rope=rope, positions=tables.positions, q=q)
        lists = att.select(turned, cache, tables)
        return (turned, lists, *att.run(turned, cache, tables, lists))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        turned, lists, out, lse = step()
    for i in range(steps):
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape)))
        graph.replay()
        kv = kv + 1
        assert np.array_equal(tables.kv_lens.cpu().numpy(), kv)
        want_q, size = paged.rope(host(q[:B]), (kv - 1)[None], w, None, True)
        check_rotated(turned[:B], want_q, size, dtype)
        b = Batch.__new__(Batch)
        b.qo = [1] * B
        b.qo_indptr, b.page_indptr = np.arange(B + 1), tables.kv_page_indptr.cpu().numpy()
        b.pages, b.last = tables.kv_page_indices.cpu().numpy(), tables.kv_last_page_len.cpu().numpy()
        b.q, b.cache, b.page, b.Hq, b.Hkv, b.D, b.T, b.pad, b.hnd, b.dtype = turned, cache, page, Hq, Hkv, D, B + 2, 2, \
            layout == "HND", dtype
        want = b.lists(blocks, 1, 2)
        assert np.array_equal(lists.cpu().numpy()[:B], want[:B])
        if i % 7 == 0 or i == steps - 1:
            b.check(out, lse, b.want(want))
            n = b.page_indptr[-1]
            filled = np.concatenate([[page] * (m - 1) + [int(b.last[r])] for r, m in enumerate(np.diff(b.page_indptr))])
            check_bounds(cache, b.pages[:n], filled.astype(int), [])
    assert tables.device_status() == cache.device_status() == att.device_status() == 0
    x = host(cache.data if layout == "NHD" else cache.data.transpose(2, 3))
    turned0, size0 = paged.rope(host(k0), t[None], w, None, True)
    check_rotated(torch.from_numpy(x[slots0 // page, 0, slots0 % page]), turned0, size0, dtype)  # old rows as they were


@gpu
def test_calls_on_another_stream():
    """Objects made while their stream is busy, used by hand on another one and under it; memory outlives the calls."""
    b = Batch([1] * 4, [3000] * 4, 8, 1, 128, 16, "NHD", torch.bfloat16, seed=3)
    a, tables = b.attention(40, 1, 2), b.tables()
    lists = a.select(b.q, b.cache, tables)
    want = a.run(b.q, b.cache, tables, lists)
    w, pos = frequencies(64), torch.arange(4, dtype=I32, device="cuda") * 1000
    turned, _ = pa.Rope(w).apply(b.q, None, pos)
    rows, slots = torch.randn(4, 1, 128, device="cuda").bfloat16(), torch.arange(4, device="cuda") * 16
    ref = pa.KvCache(9, 16, 1, 128, torch.bfloat16, bounds=True)
    ref.append(rows, rows, slots, rope=pa.Rope(w), positions=pos)
    side = torch.cuda.Stream()
    for by_hand in (True, False):
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)  # the objects' zeroing waits behind this
        a2, rope = b.attention(40, 1, 2), pa.Rope(w)
        cache = pa.KvCache(9, 16, 1, 128, torch.bfloat16, bounds=True)
        kw = dict(stream=side) if by_hand else {}
        with torch.cuda.stream(torch.cuda.current_stream() if by_hand else side):
            got_q, _ = rope.apply(b.q, None, pos, **kw)
            cache.append(rows, rows, slots, rope=rope, positions=pos, **kw)
            cache.update_bounds(slots, **kw)
            got_lists = a2.select(b.q, b.cache, tables, **kw)
            got = a2.run(b.q, b.cache, tables, got_lists, **kw)
        assert a2.device_status(side) == cache.device_status(side) == 0
        torch.cuda.synchronize()
        assert torch.equal(got_q, turned) and torch.equal(got_lists, lists)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for name in ("data", "bounds", "bound_scales"):
            assert torch.equal(getattr(cache, name), getattr(ref, name)), name


@gpu
@pytest.mark.parametrize("qo, kv, Hkv, blocks", [([1] * 3, [3000, 700, 9000], 1, 200), ([550], [3000], 2, 60)], ids=str)
def test_two_objects_on_two_streams_and_a_replayed_graph(qo, kv, Hkv, blocks):
    """Runs that overlap, each in its own workspace; a captured one replayed between them, over queries that change."""
    bs = [Batch(qo, kv, 8 * Hkv, Hkv, 128, 16, "NHD", torch.bfloat16, seed=s) for s in (1, 2, 3)]
    objs, tables = [b.attention(blocks, 1, 1) for b in bs], [b.tables() for b in bs]
    both = lambda i: (lists := objs[i].select(bs[i].q, bs[i].cache, tables[i]),  # noqa: E731
                      *objs[i].run(bs[i].q, bs[i].cache, tables[i], lists))
    want = [both(i) for i in range(3)]
    queries = [bs[2].q.clone(), -bs[2].q]
    bs[2].q.copy_(queries[1])
    other = both(2)
    graph, streams = torch.cuda.CUDAGraph(), [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = both(2)
    torch.cuda.synchronize()
    for n in range(20):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append(both(i))
        bs[2].q.copy_(queries[n % 2])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((*got, captured), (*want[:2], (want[2], other)[n % 2])):
            assert all(torch.equal(a, b) for a, b in zip(x, y))
    assert all(a.device_status() == 0 for a in objs)


@gpu
def test_objects_that_share_a_workspace():
    bs = [Batch([1, 1], [3000, 900], 8, 1, 128, 16, "NHD", torch.float16, seed=1),
          Batch([40, 1], [2100, 1900], 16, 2, 64, 16, "NHD", torch.bfloat16, seed=3),
          Batch([2], [1700], 6, 2, 256, 16, "NHD", torch.bfloat16, seed=4)]
    first = bs[0].attention(100, workspace=torch.full((64 << 20,), 0x5A, dtype=torch.uint8, device="cuda"))
    objs = [first] + [b.attention(100, workspace=first) for b in bs[1:]]
    want = [b.lists(100) for b in bs]
    for _ in range(3):
        for b, a, w in zip(bs, objs, want):
            lists = a.select(b.q, b.cache, b.tables())
            np.testing.assert_array_equal(lists.cpu().numpy(), w)
            out, lse = a.run(b.q, b.cache, b.tables(), lists)
            b.check(out, lse, b.want(w))
    assert all(a.device_status() == 0 for a in objs)


@gpu
def test_offsets_beyond_32_bits():
    """Pages behind 4 GB of a cache: rows, bounds, selection and attention find them."""
    page, H, D = 64, 8, 128
    num_pages = 20_000  # 5.2 GB
    cache = pa.KvCache(num_pages, page, H, D, torch.bfloat16, bounds=True)
    n = 5
    pages = np.array([num_pages - 1, 3, num_pages - 7, num_pages // 2 + 1, num_pages - 2])
    t = np.arange(n * page - 9)
    k, v = (torch.randn(len(t), H, D, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(1, 2 * H, D, device="cuda").bfloat16()
    small = pa.KvCache(n, page, H, D, torch.bfloat16, bounds=True)
    got = []
    for c, ids in ((cache, pages), (small, np.arange(n))):
        c.append(k, v, dev(ids[t // page].astype(np.int64) * page + t % page, torch.int64))
        a = pa.BlockAttention(1, 1, 2 * H, H, D, page, torch.bfloat16, 3, n * page)
        tables = tuple(dev(x) for x in ([0, 1], [0, n], ids, [page - 9]))
        lists = a.select(q, c, tables)
        got.append((lists, *a.run(q, c, tables, lists), c.bounds[dev(ids, torch.int64)]))
        assert a.device_status() == c.device_status() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)


def test_turns_are_the_nearest_fractions():
    """w / 2 pi modulo 1 in units of 2^-64, to the unit, for frequencies of either sign and any size."""
    from fractions import Fraction
    from attention_paged_kv_gb300 import _paged
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582")
    rng = np.random.default_rng(0)
    for w in [0.0, 1.0, -2.5, 6.283185307179586, 5e-324, 1e-9, 123.456, *rng.uniform(-3, 3, 50), *10.0 ** rng.uniform(-12, 6, 50)]:
        exact = Fraction(float(w)) / two_pi * (1 << 64)
        got = _paged._turns(float(w))
        assert -(1 << 63) <= got < 1 << 63
        assert abs((exact - got + (1 << 63)) % (1 << 64) - (1 << 63)) <= Fraction(1, 2) + Fraction(1, 1 << 40) * max(1, abs(exact) / (1 << 64))


# ---------------------------------------------------------------- bounds of slots with others between them


@gpu
@pytest.mark.parametrize("h, page, n, gaps", [
    (1, 16, 40, [1]), (8, 16, 30, [1, 2, 7]), (2, 64, 100, [1, 250, 256, 3]), (1, 128, 5, [300, 1400, 9000]),
    (8, 16, 3000, [1, 1, 40]), (3, 32, 5000, [2, 500, 1]), (4, 8, 20, [256, 255, 257, 1023, 1024, 1025, 2])], ids=str)
def test_bounds_pass_over_rows_without_a_slot(h, page, n, gaps):
    """Negative slots, and slots beyond the cache, between two of one page: the bounds are those of all its slots.

    From one token a warp to 32, the next row within the CTA's tokens, within what it loads ahead, and beyond."""
    rng = np.random.default_rng(n)
    num_pages = -(-n // page) + 2
    ids = rng.permutation(num_pages)
    t = np.arange(n)
    slots, named, at = [], ids[t // page] * page + t % page, 0
    while at < n:
        take = int(rng.integers(1, 5))
        slots += list(named[at: at + take])
        gap = gaps[int(rng.integers(len(gaps)))] if rng.random() < min(1.0, 200 / n) else 0
        slots += list(rng.choice([-1, -7, -(1 << 40)], gap))
        at += take
    slots = np.array(slots + [-1] * 3000, np.int64)
    used = -(-n // page)
    filled = [page] * (used - 1) + [n - (used - 1) * page]
    for beyond in (False, True):
        if beyond:
            free = np.flatnonzero(slots < 0)
            slots[free[:: 3]] = num_pages * page + rng.integers(0, 1 << 40, len(free[:: 3]))
        for use in ("update_bounds", "append"):
            cache = pa.KvCache(num_pages, page, h, 64, torch.bfloat16, bounds=True)
            cache.data.copy_(torch.randn(cache.data.shape, device="cuda"))
            cache.bounds.fill_(77)
            cache.bound_scales.fill_(77)
            for _ in range(3):
                if use == "append":
                    k = torch.randn(len(slots), h, 64, device="cuda").bfloat16()
                    cache.append(k, k, dev(slots, torch.int64))
                else:
                    cache.update_bounds(dev(slots, torch.int64))
                assert cache.device_status() == (raw.PA_DEV_BAD_INDEX if beyond else 0)
                check_bounds(cache, ids[:used], filled, ids[used:])


@gpu
def test_bounds_of_slots_out_of_order_are_reported():
    cache = pa.KvCache(4, 16, 2, 64, torch.float16, bounds=True)
    for slots, bad in (([3, 4, 5, 16, 17], False), ([4, 3], True), ([4, -1, 3], True), ([4, 4], True),
                       ([15, 14], True), ([4] + [-1] * 700 + [2], True), ([4] + [-1] * 700 + [18], False),
                       ([15, 0 + 16, 31, 32], False)):
        cache.update_bounds(torch.tensor(slots, device="cuda"))
        assert cache.device_status() == (raw.PA_DEV_BAD_INDEX if bad else 0), slots


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H, kv, page, D", [(5, 9000, 16, 128), (5, 8200, 128, 64), (3, 9000, 32, 256), (1, 9000, 16, 128)])
def test_chunks_keep_a_long_tail(H, kv, page, D, dtype):
    """As test_attention_keeps_a_long_tail, for a chunk: the tail's weights are 2^-20.45 of the largest, between two
    fp16 subnormals (11.7 of them) where the reference is the largest logit itself.

    With the reference 7 below it they are 2^-13.45, rounded by at most 2^-25, which is 2^-11.55 of them; bf16 rounds by
    2^-8.  Logits, weights and sums add less than 2^-10, the output rounds by half a step."""
    n, qo, G = -(-kv // page), 600, 16  # (few kv heads: keys cut into parts of their own references)
    cache = pa.KvCache(n, page, H, D, dtype)
    k = torch.zeros(kv, H, D, dtype=dtype, device="cuda")
    v = torch.full((kv, H, D), 16384.0, dtype=dtype, device="cuda")
    k[kv // 5, :, 0] = 4.0
    v[kv // 5] = 0.0
    cache.append(k, v, torch.arange(kv, device="cuda"))
    q = torch.zeros(qo, G * H, D, dtype=dtype, device="cuda")
    q[..., 0] = 20.45 * np.log(2) * D ** 0.5 / 4
    a = pa.BlockAttention(1, qo, G * H, H, D, page, dtype, n, kv)
    tables = tuple(dev(x) for x in ([0, qo], [0, n], range(n), [kv - (n - 1) * page]))
    assert qo * H * n * page >= 1 << 20  # a chunk, by the rule of its kernel
    lists = torch.arange(n, dtype=I32, device="cuda").expand(qo, H, n).contiguous()
    out, lse = a.run(q, cache, tables, lists)
    assert a.device_status() == 0
    logit = float(q[0, 0, 0]) * 4 / D ** 0.5
    w = torch.arange(kv - qo, kv, device="cuda", dtype=torch.float64).view(-1, 1, 1) * np.exp(-logit)
    rel = (out.double() / (16384 * w / (1 + w)) - 1).abs().max().item()
    eps = torch.finfo(dtype).eps / 2
    assert rel <= (2.0 ** -11.5 if dtype == torch.float16 else eps) + 2.0 ** -10 + eps, rel
    assert (lse.double() - (logit + torch.log1p(w[..., 0]))).abs().max().item() <= 2.0 ** -17


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("qo, kv, Hq, Hkv, D, page, layout, blocks, short", [
    ([600], [600], 8, 1, 128, 16, "NHD", 128, False), ([700, 300], [700, 303], 16, 2, 64, 8, "HND", 130, False),
    ([500], [500], 4, 1, 256, 32, "NHD", 100, False), ([600], [6000], 8, 1, 128, 16, "NHD", 128, True),
    ([300], [5000], 12, 3, 64, 128, "HND", 12, True), ([400], [3000], 8, 1, 256, 64, "NHD", 60, True)], ids=str)
def test_chunks_keep_rows_of_few_keys(qo, kv, Hq, Hkv, D, page, layout, blocks, short, dtype):
    """Rows of a chunk that see fewer than 128 keys: the weights' rounding does not average out there, and they are held in
    two terms, 2^-16 of bf16's weights (2^-22 of fp16's, and 2^-25 of the largest where the second is a subnormal).

    The other terms are those of Batch.check.  short: the callers' lists of none to three blocks at far positions, with
    others of many in the same tiles."""
    b = Batch(qo, kv, Hq, Hkv, D, page, layout, dtype, seed=5)
    a = b.attention(blocks)
    assert sum(qo) * Hkv * blocks * page >= 1 << 20 or short
    rng = np.random.default_rng(2)
    lists = np.full((b.T, Hkv, blocks), -1, np.int32)
    for i, (_, _, _, pos) in enumerate(paged.queries(b.qo_indptr, b.page_indptr, b.last, page)):
        n = pos // page + 1
        for h in range(Hkv):
            count = min(n, blocks) if not short or i % 11 == 3 else int(rng.integers(0, 4))
            mine = np.sort(rng.permutation(n)[:count])
            if count and i % 2:
                mine[-1] = n - 1  # the query's own, in part
            lists[i, h, :count] = mine
    ref, ref_lse, sp = b.want(lists)
    out, lse = a.run(b.q, b.cache, b.tables(), dev(lists))
    assert a.device_status() == 0
    b.check(out, lse, (ref, ref_lse, sp))
    eps = torch.finfo(dtype).eps / 2
    ds = 2.0 ** -22 * (D / 16 + 2) * sp["s"]
    rel = 2 * (ds + 2.0 ** -21) + (2.0 ** -22 if dtype == torch.float16 else 2.0 ** -16) + 2.0 ** -23 * (sp["n"] / 16 + 8)
    bound = (rel[..., None] * sp["av"] + 2.0 ** -25 * sp["v"]) * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25
    few = sp["n"] < 128
    err = np.abs(host(out) - ref)
    assert few.sum() >= 100 * Hkv and (err <= bound)[few].all(), (err / bound)[few].max()


@gpu
@pytest.mark.parametrize("qo, kv", [([1, 2, 1], [200, 330, 100]), ([40, 700], [330, 200 + 700])])
def test_no_room_although_the_list_has_some(qo, kv):
    """More pages than the object allows for, but no more than a list holds: no list and no output, as with longer ones."""
    b = Batch(qo, kv, 4, 2, 64, 16, "NHD", torch.float16, seed=6)
    a = b.attention(60, 1, 1, max_kv=208)
    got = a.select(b.q, b.cache, b.tables())
    assert a.device_status() == raw.PA_DEV_NO_ROOM and a.device_status() == 0
    want = b.lists(60, 1, 1)
    over = np.array([pos // 16 + 1 > 13 for _, _, _, pos in paged.queries(b.qo_indptr, b.page_indptr, b.last, 16)])
    assert over.any() and not over.all()
    want[over] = -1
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    out, lse = a.run(b.q, b.cache, b.tables(), got)
    assert a.device_status() == raw.PA_DEV_NO_ROOM
    at = torch.from_numpy(over).cuda()
    assert not out[at].any() and torch.isneginf(lse[at]).all() and torch.isfinite(lse[~at]).all()


@gpu
def test_overlapping_requests_of_many_tokens():
    """A qo_indptr that goes back and forth over 2^27 tokens 512 times: its tiles alone would pass 2^32."""
    n, B = 1 << 27, 1024
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    cache = pa.KvCache(4, 16, 1, 64, torch.float16, bounds=True)
    a = pa.BlockAttention(B, n, 1, 1, 64, 16, torch.float16, 1, 64, 0, 1, max_qo_len=n)
    qo = torch.tensor([0, n] * (B // 2) + [0], dtype=I32, device="cuda")
    # every request has 4 pages of its own: a long one's last token is at position 63
    tables = (qo, 4 * torch.arange(B + 1, dtype=I32, device="cuda"), torch.arange(4, dtype=I32, device="cuda").repeat(B),
              torch.full((B,), 16, dtype=I32, device="cuda"))
    q = torch.zeros(n, 1, 64, dtype=torch.float16, device="cuda")
    out = torch.full((n, 1, 1), 7, dtype=I32, device="cuda")
    a.select(q, cache, tables, out=out)
    assert a.device_status() == raw.PA_DEV_BAD_INDEX
    # the first request's tokens are there: only the last 64 see a key, each its own block
    want = torch.full((n,), -1, dtype=I32, device="cuda")
    want[-64:] = torch.arange(64, device="cuda", dtype=I32) // 16
    assert torch.equal(out.view(-1), want)


# ---------------------------------------------------------------- the rotation under autograd


def oracle_gradient(y, positions, w, interleaved, inverse, dtype, scale=1.0):
    """The gradient of sum(y * rope(x)) in x, and check_rotated's size of it."""
    return paged.rope(host(y), positions, w, None, interleaved, scale, inverse=not inverse)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved, inverse, scale, needs", [
    (False, False, 1.0, "qk"), (True, False, 1.5, "q"), (False, True, 0.75, "k"), (True, True, 1.0, "qk")])
def test_rope_is_recorded_by_autograd(interleaved, inverse, scale, needs, dtype):
    """backward() gives the formula's gradient, of q, k or both, as slices of a projection that is the leaf."""
    rng = np.random.default_rng(4)
    n, H, h, d = 37, 4, 2, 96
    w = frequencies(40)
    r = pa.Rope(w, interleaved=interleaved, scale=scale)
    positions = rng.integers(0, 9000, (1, n))
    pos = dev(positions[0])
    leaf = torch.from_numpy(rng.standard_normal((n, (H + h) * d))).to(dtype).cuda().requires_grad_()
    q, k = leaf[:, : H * d].view(n, H, d), leaf[:, H * d:].view(n, h, d)
    q, k = q if "q" in needs else q.detach(), k if "k" in needs else k.detach()
    a, b = r.apply(q, k, pos, inverse=inverse)
    with torch.no_grad():
        plain = r.apply(q, k, pos, inverse=inverse)
    assert plain[0].grad_fn is None and torch.equal(a, plain[0]) and torch.equal(b, plain[1])
    pos.fill_(7)  # the next step's: the backward pass has those of its own
    y, z = (torch.from_numpy(rng.standard_normal(t.shape)).to(dtype).cuda() for t in (a, b))
    torch.autograd.backward([a, b], [y, z])
    got = leaf.grad.view(n, H + h, d)
    for part, g, need in ((got[:, :H], y, "q"), (got[:, H:], z, "k")):
        if need in needs:
            check_rotated(part, *oracle_gradient(g, positions, w, interleaved, inverse, dtype, scale), dtype)
        else:
            assert not part.any()


@gpu
def test_rope_gradients_of_unusual_calls():
    """One value expanded, a part of the results used, no k, given outputs, a given stream, the gradient's gradient, and
    differences: a rotation is linear, so a step along e changes the sum by the gradient's product with e."""
    rng = np.random.default_rng(5)
    n, d = 20, 64
    w, positions = frequencies(32), rng.integers(0, 500, (1, n))
    r, pos = pa.Rope(w), dev(positions[0])
    x = torch.from_numpy(rng.standard_normal((n, 3, d))).half().cuda().requires_grad_()
    ones = torch.ones_like(x)
    out, none = r.apply(x, None, pos)
    assert none is None
    out.sum().backward()
    check_rotated(x.grad, *oracle_gradient(ones, positions, w, False, False, x.dtype), x.dtype)
    a, b = r.apply(x, x, pos)
    only_b, = torch.autograd.grad(b, x, ones, retain_graph=True)
    both, = torch.autograd.grad([a, b], x, [ones, ones])
    assert torch.equal(only_b, x.grad) and torch.equal(both, x.grad + x.grad)
    given = torch.empty_like(x)
    assert r.apply(x, None, pos, q_out=given)[0] is given and not given.requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    far, _ = r.apply(x, None, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    there, = torch.autograd.grad(far, x, ones)
    torch.cuda.synchronize()
    assert torch.equal(there, x.grad)
    # y -> gradient in x is a rotation of y: its own gradient along v is rope(v)
    y = ones.clone().requires_grad_()
    g, = torch.autograd.grad(r.apply(x, None, pos)[0], x, y, create_graph=True)
    v = torch.from_numpy(rng.standard_normal((n, 3, d))).half().cuda()
    gg, = torch.autograd.grad(g, y, v)
    assert torch.equal(gg, r.apply(v, None, pos)[0])
    # differences, of values whose sums are exact in fp16: each result is half a step off, and 2^-20 of its pairs as of check_rotated
    x0, e = (torch.from_numpy(rng.integers(-64, 65, (n, 3, d)) / 32).half().cuda() for _ in range(2))
    here, moved = (host(r.apply(t, None, pos)[0]) for t in (x0, x0 + e))
    bound = 2.0 ** -11 * (np.abs(here).sum() + np.abs(moved).sum() + (np.abs(host(x.grad)) * np.abs(host(e))).sum()) + \
        2.0 ** -20 * 2 * (np.abs(host(x0)).sum() + np.abs(host(x0 + e)).sum() + np.abs(host(e)).sum())
    assert abs((moved - here).sum() - (host(x.grad) * host(e)).sum()) <= bound


@gpu
def test_rope_with_its_gradient_in_a_graph():
    n, d = 33, 128
    r, pos = pa.Rope(frequencies(64)), torch.arange(n, dtype=I32, device="cuda")
    x, y = (torch.randn(n, 2, d, device="cuda").half() for _ in range(2))
    x.requires_grad_()

    def step():
        out, _ = r.apply(x, None, pos)
        return out, torch.autograd.grad(out, x, y)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, grad = step()
    for gain in (1.0, -2.0):
        with torch.no_grad():
            x.mul_(gain)
            y.mul_(gain)
        pos.add_(5)
        g.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            assert torch.equal(out, r.apply(x, None, pos)[0]) and torch.equal(grad, r.apply(y, None, pos, inverse=True)[0])


@gpu
def test_workspaces_are_shared_within_a_class():
    kv4 = pa.Kv4Attention(1, 1, 2, 1, 64, 16, torch.float16)
    block = pa.BlockAttention(1, 1, 2, 1, 64, 16, torch.float16, 4, 100)
    cache = pa.KvCache(2, 16, 1, 64, torch.float16)
    for make in (lambda w: pa.Kv4Attention(1, 1, 2, 1, 64, 16, torch.float16, workspace=w),
                 lambda w: pa.BlockAttention(1, 1, 2, 1, 64, 16, torch.float16, 4, 100, workspace=w)):
        refusals = 0
        for w in (kv4, block, cache):
            try:
                make(w)
            except pa.PagedAttnError as e:
                refusals += "another class" in str(e)
        assert refusals == 2


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("qo, kv, D, page, blocks", [
    ([1, 2, 1], [100, 100, 100], 128, 16, 7), ([1, 1], [5000, 300], 64, 32, 160), ([1], [900], 256, 4, 225)], ids=str)
def test_attention_of_an_infinite_value(qo, kv, D, page, blocks, dtype):
    """An infinity of V, of either sign, is the result of its channel in the rows of its kv head that see it, and of none
    else: their weights are positive, however they are held."""
    b = Batch(qo, kv, 8, 2, D, page, "NHD", dtype, seed=2)
    a = b.attention(blocks)
    lists = a.select(b.q, b.cache, b.tables())
    clean, clean_lse = a.run(b.q, b.cache, b.tables(), lists)
    assert torch.isfinite(clean).all()
    at = kv[0] // 3  # a key of the first request
    page_id, slot = int(b.pages[at // page]), at % page
    b.cache.data[page_id, 1, slot, 1, 9] = float("inf")
    b.cache.data[page_id, 1, slot, 1, 40] = -float("inf")
    out, lse = a.run(b.q, b.cache, b.tables(), lists)
    want = clean.clone()
    want[0, 4:, 9], want[0, 4:, 40] = float("inf"), -float("inf")
    assert torch.equal(out, want) and torch.equal(lse, clean_lse)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D, page, heads", [(128, 16, 8), (64, 32, 32), (256, 4, 4)], ids=str)
def test_single_tokens_hold_weights_in_two_terms(D, page, heads, dtype):
    """Batch.check's bound with the weights' rounding by two terms, the first cut: 2^-21 of fp16's (and 2^-24 where the second
    is a subnormal, 2^-31 of the largest, which is 2^7 or more), 2^-15 of bf16's.  Requests of 1 to 120 keys, where one
    term's roundings do not average out."""
    kv = list(range(1, 121))
    b = Batch([1] * len(kv), kv, heads, 2, D, page, "NHD", dtype, seed=3, q_gain=0.3)
    blocks = -(-kv[-1] // page)
    a = b.attention(blocks)
    lists = a.select(b.q, b.cache, b.tables())
    ref, ref_lse, sp = b.want(lists.cpu().numpy())
    out, lse = a.run(b.q, b.cache, b.tables(), lists)
    eps = torch.finfo(dtype).eps / 2
    ds = 2.0 ** -22 * (D / 16 + 2) * sp["s"]
    rel = 2 * (ds + 2.0 ** -21) + (2.0 ** -21 if dtype == torch.float16 else 2.0 ** -15) + 2.0 ** -23 * (sp["n"] / 16 + 8)
    bound = (rel[..., None] * sp["av"] + 2.0 ** -31 * sp["v"]) * (1 + eps) + eps * np.abs(ref) + 2.0 ** -25
    err = np.abs(host(out) - ref)
    assert (err <= bound).all(), (err / bound).max()
