"""Binding of the calls over the 16-bit cache through device tables (include/pagedattn.h).

A step of a serving loop whose queries attend to a part of their keys:

    rope = Rope(inv_freq)                                                      # or several axes: Rope(inv_freq, axes=[...])
    cache = KvCache(num_pages, page_size, num_kv_heads, head_dim, dtype, bounds=True)
    attention = BlockAttention(batch_size, max_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, dtype,
                               num_blocks, max_kv_len)

    tables.build(qo_lens, kv_lens, block_table, free_pages, free_count)        # a BatchTables
    q = cache.append(k, v, tables.slot_mapping, rope=rope, positions=tables.positions, q=q)
    blocks = attention.select(q, cache, tables)
    out, lse = attention.run(q, cache, tables, blocks)

The calls only launch kernels, so the step can be captured into a CUDA graph,
as with the objects of the 4-bit cache.  ``cache.data`` is laid out as
``Plan.run`` takes it.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import struct

from . import _binding as _b
from ._kv4 import BatchTables, _call, _device, _is, _Object, _on, _refuse, _rows

# The arguments' structures (include/pagedattn.h) packed directly.
_ROPE_ROWS = struct.Struct("@4P4qPq6i0P")
_KV_ROWS = struct.Struct("@4P4q2PqP2i0P")
_BLOCK_BATCH = struct.Struct("@4P9i0P")

# 2 pi as a ratio of whole numbers, good to 50 digits
_TWO_PI = (2 * 314159265358979323846264338327950288419716939937510582, 10 ** 53)


def _turns(w):
    """w radians in turns modulo 1, as the nearest multiple of 2^-64 (its numerator, signed: torch has no unsigned)."""
    n, d = w.as_integer_ratio()
    a, b = n * (_TWO_PI[1] << 64), d * _TWO_PI[0]
    t = (2 * a + b) // (2 * b) & ((1 << 64) - 1)
    return t - (1 << 64) if t >> 63 else t


@functools.lru_cache(None)
def _recorded():
    """Rope.apply as a function of autograd: the gradient of a rotation is the rotation by the negative angle."""
    import torch

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rope, q, k, positions, inverse):
            ctx.rope, ctx.inverse = rope, inverse
            ctx.save_for_backward(positions)
            ctx.set_materialize_grads(False)
            return rope.apply(q, k, positions, inverse=inverse)

        @staticmethod
        def backward(ctx, dq, dk):
            # a gradient may be missing, or not laid out as rows (that of a sum is one value, expanded)
            dq, dk = (None if d is None else d.contiguous() for d in (dq, dk))
            if dq is None and dk is not None:
                dk, _ = ctx.rope.apply(dk, None, *ctx.saved_tensors, inverse=not ctx.inverse)
            elif dq is not None:
                dq, dk = ctx.rope.apply(dq, dk, *ctx.saved_tensors, inverse=not ctx.inverse)
            return None, dq, dk, None, None

    return Turn


class Rope(_Object):
    """A rotation of queries and keys by their positions.

    inv_freq: radians a position of each pair (float64 values; scaled for long
    contexts by the caller where wanted); twice as many values of each head are
    rotated, a multiple of 16, those behind them are left.  Pairs are value i and
    value i + len(inv_freq), or neighbours with ``interleaved``.  axes: the axis
    of each pair, for positions of several axes ([0] * 16 + [1] * 24 + [2] * 24
    for sections of time, height and width); None for one position a token.
    scale multiplies cosines and sines.
    """

    def __init__(self, inv_freq, interleaved=False, axes=None, scale=1.0, device=None):
        import torch
        freq = [float(w) for w in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
        pairs = len(freq)
        if pairs < 8 or pairs % 8 or pairs > 128:
            _refuse("inv_freq must have a multiple of 8 entries, 8 to 128")
        if not all(abs(w) < float("inf") for w in freq):
            _refuse("inv_freq must be finite")
        axes = None if axes is None else [int(a) for a in (axes.tolist() if hasattr(axes, "tolist") else axes)]
        if axes is not None and (len(axes) != pairs or min(axes) < 0):
            _refuse(f"axes must name an axis for each of the {pairs} pairs")
        self.rotary_dim, self.num_axes = 2 * pairs, 1 if axes is None else max(axes) + 1
        self.interleaved, self.scale = bool(interleaved), float(scale)
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        self.turns = torch.tensor([_turns(w) for w in freq], dtype=torch.int64, device=self.device)
        self.axes = None if axes is None else torch.tensor(axes, dtype=torch.int32, device=self.device)
        self._args = _b.Rotation(self.turns.data_ptr(), None if axes is None else self.axes.data_ptr(), self.num_axes,
                                 self.rotary_dim, self.interleaved, self.scale)
        self._made(*(t for t in (self.turns, self.axes) if t is not None))

    def _positions(self, positions, n, index):
        """Pointer and stride between axes of int32 positions [n] or [num_axes, n]."""
        import torch
        axes = self.num_axes
        if positions.dtype != torch.int32 or positions.get_device() != index or positions.shape not in \
                (((n,), (1, n)) if axes == 1 else ((axes, n),)):
            _refuse(f"positions must be int32 of shape {[n] if axes == 1 else [axes, n]} on cuda:{index}")
        if n > 1 and positions.stride(-1) != 1:
            _refuse("positions: each axis must be contiguous")
        return positions.data_ptr(), positions.stride(0) if positions.dim() == 2 else n

    def apply(self, q, k, positions, q_out=None, k_out=None, inverse=False, stream=None):
        """(q, k) rotated by their positions, int32 [n] or [num_axes, n].

        q, k [n, heads, head_dim] (k may be None): any token stride that is a
        multiple of 8; head_dim a multiple of 16 up to 256.  q_out and k_out
        (allocated where not given) may be q and k themselves.  inverse: by the
        negative angle, as gradients pass through the rotation (with scale 1, the
        rotation back).  Autograd records the call where q or k needs a gradient
        and no outputs are given (positions are copied for it); outputs that are
        given carry none, nor do the results of the other calls here.  A backward
        pass is captured into a graph with torch.autograd.grad, or with leaves
        that no eager graph still holds.  See pagedattn_rope.
        """
        import torch
        at = self._index
        if q.dim() != 3:
            _refuse("q must be of shape [tokens, heads, head_dim]")
        size = n, _, dim = q.shape
        k_heads = 0 if k is None else (k.shape[1] if k.dim() == 3 else -1)
        shape = (n, k_heads, dim)
        q_stride = _rows(q, "q", size, at)
        k_stride = 0 if k is None else _rows(k, "k", shape, at)
        if q_out is not None:
            _rows(q_out, "q_out", size, at)
        if k_out is not None:
            if k is None:
                _refuse("k_out without k")
            _rows(k_out, "k_out", shape, at)
        for t in (k, q_out, k_out):
            if t is not None and t.dtype != q.dtype:
                _refuse("q, k and their outputs must be of one type")
        code = _b.PA_BF16 if q.dtype == torch.bfloat16 else _b.dtype_code(q.dtype)
        pos, pos_stride = self._positions(positions, n, at)
        handle, guard = _on(at, stream, (self,), (q, k, positions, q_out, k_out))
        if q_out is None and k_out is None and torch.is_grad_enabled() and \
                (q.requires_grad or (k is not None and k.requires_grad)):
            with guard or contextlib.nullcontext():
                return _recorded().apply(self, q, k, positions.clone(), inverse)
        if guard is not None:
            with guard:  # the outputs are allocated on the stream that writes them
                return self._launch(q, k, size, k_heads, q_stride, k_stride, q_out, k_out, pos, pos_stride, inverse,
                                    code, handle)
        return self._launch(q, k, size, k_heads, q_stride, k_stride, q_out, k_out, pos, pos_stride, inverse, code,
                            handle)

    def _launch(self, q, k, size, k_heads, q_stride, k_stride, q_out, k_out, pos, pos_stride, inverse, code, handle):
        import torch
        n, heads, dim = size
        if q_out is None:  # (alike but for the tokens' stride: twice as quick as with type, shape and device by name)
            q_out = torch.empty_like(q)
        if k is not None and k_out is None:
            k_out = torch.empty_like(k)
        more = n > 1
        rows = _ROPE_ROWS.pack(q.data_ptr(), 0 if k is None else k.data_ptr(), q_out.data_ptr(),
                               0 if k is None else k_out.data_ptr(), q_stride, k_stride,
                               q_out.stride(0) if more else heads * dim,
                               0 if k is None else (k_out.stride(0) if more else k_heads * dim), pos, pos_stride, n, heads,
                               k_heads, dim, bool(inverse), code)
        status = self._lib.pagedattn_rope(ctypes.byref(self._args), rows, handle)
        if status != _b.PA_OK:
            _b.check(status)
        return q_out, k_out


class KvCache(_Object):
    """A paged KV cache in 16 bits, and the bounds of its pages' keys.

    ``data`` [num_pages, 2, page_size, num_kv_heads, head_dim] ("NHD"; "HND"
    exchanges page_size and num_kv_heads), as ``Plan.run`` takes it.  With
    bounds=True ``bounds`` int8 [num_pages, num_kv_heads, 2, head_dim] and
    ``bound_scales`` float32 [num_pages, num_kv_heads] hold codes that enclose the
    keys of each page (largest, smallest) and what code 1 stands for; appends
    keep them.  Pass tensors to take over existing memory (bounds and
    bound_scales together).  A page copied to another takes its bounds along.
    """

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, dtype, kv_layout="NHD", data=None, bounds=False,
                 bound_scales=None, device=None):
        import torch
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.kv_layout, code = _b.layout_code(kv_layout), _b.dtype_code(dtype)
        self.dtype = (torch.float16, torch.bfloat16)[code]
        if min(self.num_pages, self.page_size, self.num_kv_heads) < 1 or self.head_dim not in (64, 128, 256):
            _refuse("num_pages, page_size and num_kv_heads must be positive, head_dim 64, 128 or 256")
        if device is None and data is not None:
            device = data.device
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        h, d = self.num_kv_heads, self.head_dim
        mid = (h, self.page_size) if self.kv_layout == _b.PA_LAYOUT_HND else (self.page_size, h)
        given = isinstance(bounds, torch.Tensor)
        if given != (bound_scales is not None):
            _refuse("bounds and bound_scales are given together")
        wanted = [("data", data, (self.num_pages, 2, *mid, d), self.dtype)]
        if given or bounds:
            wanted += [("bounds", bounds if given else None, (self.num_pages, h, 2, d), torch.int8),
                       ("bound_scales", bound_scales, (self.num_pages, h), torch.float32)]
        else:
            self.bounds = self.bound_scales = None
        for name, t, shape, kind in wanted:
            if t is None:
                t = torch.zeros(shape, dtype=kind, device=self.device)
            _is(t, name, kind, shape, self._index)
            setattr(self, name, t)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._status_ptr = self.status.data_ptr()
        own = (self.data, self.bounds, self.bound_scales)
        self._args = _b.KvCacheArgs(*(None if t is None else t.data_ptr() for t in own), self.num_pages, self.page_size,
                                    h, d, self.kv_layout, code)
        self._made(*(t for t in own if t is not None), self.status)

    def append(self, k, v, slot_mapping, rope=None, positions=None, q=None, q_out=None, stream=None):
        """Rows k, v [n, num_kv_heads, head_dim] into the slots of slot_mapping (int64 [n]); returns q, rotated.

        Rows with a negative slot are skipped; the others' slots must be
        distinct.  rope: a Rope that turns k, and q [n, heads, head_dim] where
        given, by the positions (int32 [n], or [num_axes, n]); q_out (allocated
        where not given) may be q.  Tokens at any stride that is a multiple of 8.
        Bounds, where the cache has them, follow, and then the slots of a page
        have to stand together in ascending order (see update_bounds).  See
        pagedattn_kv_append.
        """
        import torch
        at, n = self._index, slot_mapping.shape[0] if slot_mapping.dim() else 0
        shape = (n, self.num_kv_heads, self.head_dim)
        k_stride, v_stride = _rows(k, "k", shape, at), _rows(v, "v", shape, at)
        _is(slot_mapping, "slot_mapping", torch.int64, (n,), at)
        if rope is None:
            if q is not None or positions is not None:
                _refuse("q and positions need a rope")
        elif rope._index != at or positions is None:
            _refuse(f"the rope must be on cuda:{at}, and positions are needed with it")
        q_heads = q_stride = 0
        if q is not None:
            q_heads = q.shape[1] if q.dim() == 3 else -1
            q_stride = _rows(q, "q", (n, q_heads, self.head_dim), at)
            if q_out is not None:
                _rows(q_out, "q_out", q.shape, at)
        elif q_out is not None:
            _refuse("q_out without q")
        for t in (k, v, q, q_out):
            if t is not None and t.dtype != self.dtype:
                _refuse("k, v, q and q_out must be of the cache's type")
        pos, pos_stride = (0, 0) if rope is None else rope._positions(positions, n, at)
        handle, guard = _on(at, stream, (self,) if rope is None else (self, rope),
                            (k, v, slot_mapping, positions, q, q_out))
        if guard is not None:
            with guard:
                return self._append(k, v, slot_mapping, rope, q, q_out, k_stride, v_stride, q_stride, q_heads, pos,
                                    pos_stride, n, handle)
        return self._append(k, v, slot_mapping, rope, q, q_out, k_stride, v_stride, q_stride, q_heads, pos, pos_stride,
                            n, handle)

    def _append(self, k, v, slots, rope, q, q_out, k_stride, v_stride, q_stride, q_heads, pos, pos_stride, n, handle):
        import torch
        if q is not None and q_out is None:
            q_out = torch.empty_like(q)
        out_stride = 0 if q is None else (q_out.stride(0) if n > 1 else q_heads * self.head_dim)
        rows = _KV_ROWS.pack(k.data_ptr(), v.data_ptr(), 0 if q is None else q.data_ptr(),
                             0 if q is None else q_out.data_ptr(), k_stride, v_stride, q_stride, out_stride,
                             slots.data_ptr(), pos, pos_stride, self._status_ptr, n, q_heads)
        status = self._lib.pagedattn_kv_append(ctypes.byref(self._args), None if rope is None else
                                               ctypes.byref(rope._args), rows, handle)
        if status != _b.PA_OK:
            _b.check(status)
        return q_out

    def update_bounds(self, slot_mapping, stream=None):
        """The bounds of the pages that the slots (int64 [n]) name, each over its slots up to the one named last.

        For keys that came into ``data`` by other ways than append.  The slots of
        a page stand together in ascending order, as BatchTables lays them out, none
        of another page between them; negative ones may stand anywhere and are
        skipped.  See pagedattn_kv_bounds.
        """
        import torch
        if self.bounds is None:
            _refuse("the cache has no bounds")
        n = slot_mapping.shape[0] if slot_mapping.dim() else 0
        _is(slot_mapping, "slot_mapping", torch.int64, (n,), self._index)
        handle, guard = _on(self._index, stream, (self,), (slot_mapping,))
        _call(guard, self._lib.pagedattn_kv_bounds, ctypes.byref(self._args), slot_mapping.data_ptr(), n,
              self._status_ptr, handle)


class BlockAttention(_Object):
    """Attention of each query over the pages selected for it, through tables in device memory.

    num_tokens: rows of q.  num_blocks: pages of a query's list (of each kv
    head), at most 4096.  max_kv_len: most keys of a request.  first, last: pages
    that are always selected, from the start of the request and back from the
    query's own.  max_qo_len: a bound of the requests' query lengths, by which the
    kernels are chosen (a longer request is computed too, slower); by default 1
    where there are as many tokens as requests, else num_tokens.  Pass 1 for a
    decode step with a few rows to spare (64 requests in 256 rows: attention 75
    us, by default 87); with many, the default is the quicker (in 2048 rows 136
    and 90).  Holds the workspace, so two calls that overlap on the device
    need two objects with a workspace each; workspace: as for Kv4Attention.
    """

    def __init__(self, batch_size, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, dtype, num_blocks,
                 max_kv_len, first=1, last=1, max_qo_len=None, workspace=None, device=None):
        import torch
        self.batch_size, self.num_tokens = int(batch_size), int(num_tokens)
        self.num_qo_heads, self.num_kv_heads = int(num_qo_heads), int(num_kv_heads)
        self.head_dim, self.page_size = int(head_dim), int(page_size)
        self.num_blocks, self.first, self.last = int(num_blocks), int(first), int(last)
        if self.page_size < 1 or int(max_kv_len) < 0:
            _refuse("page_size must be positive and max_kv_len not negative")
        self.max_pages = -(-int(max_kv_len) // self.page_size)
        if self.first < 0 or self.last < 1 or self.first + self.last > self.num_blocks:
            _refuse("first must not be negative, last positive, and both fit num_blocks")
        if max_qo_len is None:
            max_qo_len = 1 if self.num_tokens == self.batch_size else self.num_tokens
        self.max_qo_len = int(max_qo_len)
        self._dtype = (torch.float16, torch.bfloat16)[_b.dtype_code(dtype)]
        self._shape = (self.num_tokens, self.num_qo_heads, self.head_dim)
        self._lists = (self.num_tokens, self.num_kv_heads, self.num_blocks)
        if device is None and workspace is not None:
            device = workspace.device
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        need = ctypes.c_size_t(0)
        with torch.cuda.device(self.device):
            sizes = self._sizes(0, 0, 0, 0, 0)
            _b.check(self._lib.pagedattn_blocks_workspace_size(self.num_kv_heads, self.head_dim, self.page_size, sizes,
                                                               ctypes.byref(need)))
            self._take_workspace(workspace, need.value, BlockAttention)
        # what allocated outputs are like
        self._a_list = self.status.expand(self._lists)
        self._an_lse = self.status.view(torch.float32).expand(self._shape[:2])

    def _sizes(self, qo_indptr, page_indptr, pages, last, nnz):
        return _BLOCK_BATCH.pack(qo_indptr, page_indptr, pages, last, self.batch_size, nnz, self.num_tokens,
                                 self.num_qo_heads, self.num_blocks, self.first, self.last, self.max_pages,
                                 self.max_qo_len)

    def _batch(self, q, cache, tables):
        """(q's stride, packed batch, the objects and the tensors of a call), checked."""
        import torch
        at, B = self._index, self.batch_size
        stride = _rows(q, "q", self._shape, at)
        if q.dtype != self._dtype or cache.dtype != self._dtype:
            _refuse("q's or the cache's dtype differs from the object's")
        if cache._index != at or cache.num_kv_heads != self.num_kv_heads or cache.head_dim != self.head_dim or \
                cache.page_size != self.page_size:
            _refuse("the cache's heads, head_dim, page_size or device differ from the object's")
        objects = (self, cache)
        if isinstance(tables, BatchTables):
            objects = (self, cache, tables)
            if tables.batch_size != B or tables.page_size != self.page_size or tables._index != at:
                _refuse("the tables' batch, page_size or device differ from the object's")
            tables = (tables.qo_indptr, tables.kv_page_indptr, tables.kv_page_indices, tables.kv_last_page_len)
            nnz = tables[2].shape[0]
        else:
            qo_indptr, page_indptr, pages, last = tables
            nnz, i32 = pages.numel(), torch.int32
            _is(qo_indptr, "qo_indptr", i32, (B + 1,), at)
            _is(page_indptr, "kv_page_indptr", i32, (B + 1,), at)
            _is(pages, "kv_page_indices", i32, (nnz,), at)
            _is(last, "kv_last_page_len", i32, (B,), at)
        batch = self._sizes(tables[0].data_ptr(), tables[1].data_ptr(), tables[2].data_ptr(), tables[3].data_ptr(), nnz)
        return stride, batch, objects, tables

    def select(self, q, cache, tables, out=None, stream=None):
        """The blocks of each query and kv head, int32 [num_tokens, num_kv_heads, num_blocks], ascending, -1 behind them.

        q [num_tokens, num_qo_heads, head_dim], rotated as the cache's keys are (any
        token stride that is a multiple of 8); a cache with bounds; tables: a
        BatchTables, or (qo_indptr, kv_page_indptr, kv_page_indices,
        kv_last_page_len) as int32 device tensors.  Rows behind the last
        request's are left as they are.  See pagedattn_select_blocks.
        """
        import torch
        if cache.bounds is None:
            _refuse("the cache has no bounds")
        stride, batch, objects, tables = self._batch(q, cache, tables)
        if out is not None:
            _is(out, "out", torch.int32, self._lists, self._index)
        handle, guard = _on(self._index, stream, objects, (q, out, *tables))
        if out is None:
            if guard is None:
                out = torch.empty_like(self._a_list)
            else:
                with guard:  # allocated on the stream that writes it
                    out = torch.empty_like(self._a_list)
                handle, guard = _on(self._index, stream, ())
        _call(guard, self._lib.pagedattn_select_blocks, ctypes.byref(cache._args), batch, q.data_ptr(), stride,
              out.data_ptr(), self._ws_ptr, self._ws_bytes, handle)
        return out

    def run(self, q, cache, tables, blocks, out=None, lse=None, return_lse=True, stream=None):
        """out, lse of q over the listed blocks (of select, or any int32 lists of that shape).

        Lists ascend, with negative entries behind them; blocks behind a query's
        own are skipped.  out must not overlap q.  See pagedattn_blocks_run.
        """
        import torch
        at = self._index
        stride, batch, objects, tables = self._batch(q, cache, tables)
        _is(blocks, "blocks", torch.int32, self._lists, at)
        if out is not None:
            _is(out, "out", q.dtype, self._shape, at)
        if lse is not None:
            _is(lse, "lse", torch.float32, self._shape[:2], at)
        handle, guard = _on(at, stream, objects, (q, out, lse, blocks, *tables))
        if guard is None:
            return self._launch(q, stride, cache, batch, blocks, out, lse, return_lse, handle)
        with guard:
            return self._launch(q, stride, cache, batch, blocks, out, lse, return_lse, handle)

    def _launch(self, q, stride, cache, batch, blocks, out, lse, return_lse, handle):
        import torch
        if out is None:
            out = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty_like(self._an_lse)
        status = self._lib.pagedattn_blocks_run(ctypes.byref(cache._args), batch, blocks.data_ptr(), q.data_ptr(), stride,
                                                out.data_ptr(), None if lse is None else lse.data_ptr(), self._ws_ptr,
                                                self._ws_bytes, handle)
        if status != _b.PA_OK:
            _b.check(status)
        return out, lse
