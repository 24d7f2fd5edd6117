"""Binding of the device-built tables and the 4-bit cache (include/pagedattn.h).

A step of a serving loop, with no length on the host:

    tables = BatchTables(batch_size, max_tokens, max_pages, page_size, num_pages)
    cache = Kv4Cache(num_pages, page_size, num_kv_heads, head_dim)
    attention = Kv4Attention(batch_size, max_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, dtype)

    tables.build(qo_lens, kv_lens, block_table, free_pages, free_count)
    cache.append(k, v, tables.slot_mapping)
    out, lse = attention.run(q, cache, tables)

All three calls only launch kernels, so the step can be captured into a CUDA
graph; `tables.build(qo_lens, tables.kv_lens, block_table, free_pages,
tables.free_count)` then advances the lengths in place at each replay.  The
objects (and the tensors of the calls) have to live as long as such a graph.
"""
from __future__ import annotations

import ctypes
import struct

from . import _binding as _b
from ._binding import PA_ERR_INVALID_ARG, PagedAttnError

# The arguments' structures (include/pagedattn.h) packed directly: a ctypes
# structure of this size costs a third of a small launch to fill.
_TABLES_IN = struct.Struct("@5Pq5i0P")
_KV4_ROWS = struct.Struct("@2P2q4P2i")
_KV4_BATCH = struct.Struct("@4P7i0P")


def _refuse(msg):
    raise PagedAttnError(PA_ERR_INVALID_ARG, msg)


def _is(t, name, dtype, shape, index):
    """A contiguous tensor of this type and shape on device `index`, or an error."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        _refuse(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{index}")


def _rows(t, name, shape, index):
    """Tokens of contiguous [heads, head_dim] blocks at any stride; returns the stride."""
    if t.shape != shape or t.get_device() != index:
        _refuse(f"{name} must be of shape {list(shape)} on cuda:{index}")
    n, h, d = shape
    st = t.stride()
    if st[2] != 1 or (h > 1 and st[1] != d):
        _refuse(f"{name}: each token's [heads, head_dim] block must be contiguous")
    return st[0] if n > 1 else h * d


def _on(index, stream, objects, tensors=()):
    """(stream handle, context or None) for a call with these objects on device `index`.

    Without a stream the device's current one is used.  With another one, the
    tensors of the call are recorded on it, so that their memory is not given
    away before it has passed the call.  The context makes device and stream
    current where they are not.
    """
    import torch
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None:
        handle = current
    else:
        handle = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    if handle != current:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(handle, device=index)
        if stream.device.index != index:
            _refuse(f"the stream is not one of cuda:{index}")
    for o in objects:
        if handle not in o._streams:
            o._enter(handle)
    if handle != current:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return handle, torch.cuda.stream(stream)  # sets the device too
    if torch.cuda.current_device() != index:
        return handle, torch.cuda.device(index)
    return handle, None


def _device(device):
    import torch
    device = torch.device("cuda") if device is None else torch.device(device)
    if device.type != "cuda":
        _refuse(f"device must be a CUDA device, not {device}")
    return torch.device("cuda", torch.cuda.current_device() if device.index is None else device.index)


def _call(guard, function, *args):
    if guard is None:
        status = function(*args)
    else:
        with guard:
            status = function(*args)
    if status != _b.PA_OK:
        _b.check(status)


class _Object:
    """Device memory of an object's own: initialised by the stream that is current when the object is made.

    The first call on another stream, current or given, records the memory on
    it, so that it is not given away before it has passed the object's calls,
    and makes it wait for the initialisation.  (A stream under capture cannot
    wait: what it captures has to be replayed after the initialisation, as it is
    where the capture began with a wait for the device.  The memory of an object
    made under capture is initialised by each replay, and the object belongs to
    that graph.)  What a program itself does with the object's tensors on
    another stream it has to order, as with any tensor.
    """

    def _made(self, *own):
        import torch
        self._own = own
        with torch.cuda.device(self._index):
            self._streams, self._ready = {torch._C._cuda_getCurrentRawStream(self._index)}, None
            if not torch.cuda.is_current_stream_capturing():
                self._ready = torch.cuda.Event()
                self._ready.record()

    def _enter(self, handle):
        import torch
        stream = torch.cuda.ExternalStream(handle, device=self._index)
        for t in self._own:
            t.record_stream(stream)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return
            if self._ready is not None:
                stream.wait_event(self._ready)
        self._streams.add(handle)

    def device_status(self, stream=None) -> int:
        """Waits for the stream; the PA_DEV_* bits since the last read, which clears them."""
        flags = ctypes.c_int32(0)
        handle, guard = _on(self._index, stream, (self,))
        try:
            _call(guard, self._lib.pagedattn_status_word, self.status.data_ptr(), handle, ctypes.byref(flags))
        except PagedAttnError as e:
            if e.status not in (_b.PA_ERR_TIMEOUT, _b.PA_ERR_DEVICE_CHECK):
                raise
        return int(flags.value)


class BatchTables(_Object):
    """Page tables, slot maps and positions of a step, built on the device.

    Holds the outputs, all on the device: ``qo_indptr``, ``kv_page_indptr``,
    ``new_page_indptr`` [batch_size + 1]; ``kv_page_indices`` [max_pages];
    ``kv_last_page_len``, ``kv_lens`` [batch_size]; ``slot_mapping`` (int64),
    ``positions`` [max_tokens]; ``free_count`` [1].
    """

    def __init__(self, batch_size, max_tokens, max_pages, page_size, num_pages, device=None):
        import torch
        self.batch_size, self.max_tokens, self.max_pages = int(batch_size), int(max_tokens), int(max_pages)
        self.page_size, self.num_pages = int(page_size), int(num_pages)
        if min(self.batch_size, self.max_tokens, self.max_pages) < 0:
            _refuse("batch_size, max_tokens and max_pages must not be negative")
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        i32 = dict(dtype=torch.int32, device=self.device)
        self.qo_indptr = torch.zeros(self.batch_size + 1, **i32)
        self.kv_page_indptr = torch.zeros(self.batch_size + 1, **i32)
        self.new_page_indptr = torch.zeros(self.batch_size + 1, **i32)
        self.kv_page_indices = torch.full((self.max_pages,), -1, **i32)
        self.kv_last_page_len = torch.zeros(self.batch_size, **i32)
        self.kv_lens = torch.zeros(self.batch_size, **i32)
        self.slot_mapping = torch.full((self.max_tokens,), -1, dtype=torch.int64, device=self.device)
        self.positions = torch.zeros(self.max_tokens, **i32)
        self.free_count = torch.zeros(1, **i32)
        self.status = torch.zeros(2, **i32)  # the second word is the library's
        self._out = _b.TablesOut(*(getattr(self, n).data_ptr() for n, t in _b.TablesOut._fields_
                                   if t is ctypes.c_void_p), self.max_tokens, self.max_pages)
        self._made(*(t for t in vars(self).values() if isinstance(t, torch.Tensor)))

    def build(self, qo_lens, kv_lens, block_table, free_pages, free_count, stream=None):
        """Builds the tables of a step; see pagedattn_build_tables.

        qo_lens, kv_lens: int32 [batch_size]; block_table: int32 [batch_size,
        width], rows contiguous; free_pages: int32, a stack of page ids whose
        top is free_pages[free_count - 1]; free_count: int32 [1].  kv_lens may
        be ``self.kv_lens`` and free_count ``self.free_count``: the step then
        advances them in place.
        """
        i32, B, at, cap = self.qo_indptr.dtype, self.batch_size, self._index, free_pages.numel()
        _is(qo_lens, "qo_lens", i32, (B,), at)
        _is(kv_lens, "kv_lens", i32, (B,), at)
        _is(free_count, "free_count", i32, (1,), at)
        _is(free_pages, "free_pages", i32, (cap,), at)
        if block_table.dtype != i32 or block_table.dim() != 2 or block_table.shape[0] != B or \
                block_table.get_device() != at:
            _refuse(f"block_table must be an int32 tensor of shape [{B}, width] on cuda:{at}")
        width, (row, col) = block_table.shape[1], block_table.stride()
        if width > 1 and col != 1:
            _refuse("block_table: each row must be contiguous")
        handle, guard = _on(at, stream, (self,), (qo_lens, kv_lens, block_table, free_pages, free_count))
        _call(guard, self._lib.pagedattn_build_tables,
              _TABLES_IN.pack(qo_lens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(),
                              free_count.data_ptr(), row if B > 1 else width, width, cap, B, self.page_size,
                              self.num_pages), ctypes.byref(self._out), handle)
        return self


class Kv4Cache(_Object):
    """A paged KV cache in 4 bits: e2m1 codes with an e4m3 scale for each 16 values along head_dim.

    ``codes`` uint8 [num_pages, 2, page_size, num_kv_heads, head_dim / 2] and
    ``scales`` uint8 [..., head_dim / 16] ("NHD"; "HND" exchanges page_size
    and num_kv_heads); pass them to take over existing memory.  A value is
    code * scale * k_scale (or v_scale).
    """

    def __init__(self, num_pages, page_size, num_kv_heads, head_dim, kv_layout="NHD", k_scale=1.0, v_scale=1.0,
                 codes=None, scales=None, device=None):
        import torch
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.num_kv_heads, self.head_dim = int(num_kv_heads), int(head_dim)
        self.kv_layout = _b.layout_code(kv_layout)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        mid = (self.num_kv_heads, self.page_size) if self.kv_layout == _b.PA_LAYOUT_HND else \
            (self.page_size, self.num_kv_heads)
        if min(self.num_pages, self.page_size, self.num_kv_heads) < 1 or self.head_dim not in (64, 128, 256):
            _refuse("num_pages, page_size and num_kv_heads must be positive, head_dim 64, 128 or 256")
        if device is None and codes is not None:
            device = codes.device
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        for name, given, last in (("codes", codes, self.head_dim // 2), ("scales", scales, self.head_dim // 16)):
            shape = (self.num_pages, 2, *mid, last)
            if given is None:
                given = torch.zeros(shape, dtype=torch.uint8, device=self.device)
            _is(given, name, torch.uint8, shape, self._index)
            setattr(self, name, given)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._status_ptr = self.status.data_ptr()
        self._args = _b.Kv4CacheArgs(self.codes.data_ptr(), self.scales.data_ptr(), self.num_pages, self.page_size,
                                     self.num_kv_heads, self.head_dim, self.kv_layout, self.k_scale, self.v_scale)
        self._made(self.codes, self.scales, self.status)

    def append(self, k, v, slot_mapping, k_values=None, v_values=None, stream=None):
        """Quantises the rows k, v [n, num_kv_heads, head_dim] into the slots of slot_mapping (int64 [n]).

        Rows with a negative slot are skipped; the others' slots must be
        distinct.  k and v may have any token stride that is a multiple of 8.
        k_values, v_values (contiguous, of k's shape and type) receive the rows
        as later reads see them.  See pagedattn_kv4_append.
        """
        import torch
        at, n = self._index, slot_mapping.shape[0] if slot_mapping.dim() else 0
        shape = (n, self.num_kv_heads, self.head_dim)
        k_stride, v_stride = _rows(k, "k", shape, at), _rows(v, "v", shape, at)
        if v.dtype != k.dtype:
            _refuse("k and v must be of one type")
        _is(slot_mapping, "slot_mapping", torch.int64, (n,), at)
        if k_values is not None:
            _is(k_values, "k_values", k.dtype, shape, at)
        if v_values is not None:
            _is(v_values, "v_values", k.dtype, shape, at)
        rows = _KV4_ROWS.pack(k.data_ptr(), v.data_ptr(), k_stride, v_stride,
                              0 if k_values is None else k_values.data_ptr(),
                              0 if v_values is None else v_values.data_ptr(), slot_mapping.data_ptr(),
                              self._status_ptr, n,
                              _b.PA_BF16 if k.dtype == torch.bfloat16 else _b.dtype_code(k.dtype))
        handle, guard = _on(at, stream, (self,), (k, v, slot_mapping, k_values, v_values))
        _call(guard, self._lib.pagedattn_kv4_append, ctypes.byref(self._args), rows, handle)


class Kv4Attention(_Object):
    """Attention over a Kv4Cache, through tables in device memory.

    num_tokens: rows of q; max_qo_len: a bound of the requests' query lengths
    (default num_tokens), by which the kernels are chosen: pass 1 for decode
    steps.  (A longer request is computed too, slower, but with max_qo_len <= 1
    its rows may share a NaN of K or V that only some of them see.)  Holds the
    workspace, so two runs that overlap on the device need two objects with a
    workspace each.

    workspace: None to allocate one; another Kv4Attention, to share its
    workspace as it stands (and its status word); or a tensor, which is cleared:
    the constructor then waits for the device before and after (under capture
    the clearing becomes part of the graph instead).
    """

    def __init__(self, batch_size, num_tokens, num_qo_heads, num_kv_heads, head_dim, page_size, dtype, causal=True,
                 max_qo_len=None, workspace=None, device=None):
        import torch
        self.batch_size, self.num_tokens = int(batch_size), int(num_tokens)
        self.num_qo_heads, self.num_kv_heads = int(num_qo_heads), int(num_kv_heads)
        self.head_dim, self.page_size = int(head_dim), int(page_size)
        self.dtype_code, self.causal = _b.dtype_code(dtype), bool(causal)
        self.max_qo_len = self.num_tokens if max_qo_len is None else int(max_qo_len)
        if device is None and workspace is not None:
            device = workspace.device
        self._lib = _b.load()
        self.device = _device(device)
        self._index = self.device.index
        self._dtype = (torch.float16, torch.bfloat16)[self.dtype_code]
        self._shape = (self.num_tokens, self.num_qo_heads, self.head_dim)
        need = ctypes.c_size_t(0)
        with torch.cuda.device(self.device):
            _b.check(_b.load().pagedattn_kv4_workspace_size(self.num_qo_heads, self.num_kv_heads, self.head_dim,
                                                            self.max_qo_len, ctypes.byref(need)))
            shared = workspace if isinstance(workspace, Kv4Attention) else None
            given = workspace is not None
            if shared is not None:
                workspace = shared.workspace
            elif not given:
                workspace = torch.empty(need.value, dtype=torch.uint8, device=self.device)
            if workspace.device != self.device or not workspace.is_contiguous():
                _refuse(f"workspace must be a contiguous tensor on {self.device}")
            self.workspace = workspace
            self._ws_bytes = workspace.numel() * workspace.element_size()
            if self._ws_bytes < need.value:
                raise PagedAttnError(_b.PA_ERR_WORKSPACE_TOO_SMALL,
                                     f"workspace needs {need.value} bytes, got {self._ws_bytes}")
            self._ws_ptr = workspace.data_ptr()
            memory = workspace.view(-1).view(torch.uint8)
            self.status = memory[:4].view(torch.int32)
            if shared is not None:
                self._own, self._streams, self._ready = shared._own, shared._streams, shared._ready
                return
            wait = given and not torch.cuda.is_current_stream_capturing()
            if wait:  # runs in it keep their counts there until they end
                torch.cuda.synchronize(self.device)
            memory[:need.value].zero_()
            if wait:  # the next run in it may be on any stream
                torch.cuda.current_stream(self.device).synchronize()
        self._made(workspace)

    def run(self, q, cache, tables, out=None, lse=None, return_lse=True, stream=None):
        """out, lse of q [num_tokens, num_qo_heads, head_dim] (any token stride that is a multiple of 8).

        tables: a BatchTables, or (qo_indptr, kv_page_indptr, kv_page_indices,
        kv_last_page_len) as int32 device tensors.  out must not overlap q.  The
        size of kv_page_indices (a BatchTables' max_pages) helps to choose the
        kernels: one far above the pages in use costs short prompts time.  See
        pagedattn_kv4_run.
        """
        import torch
        at, B, shape = self._index, self.batch_size, self._shape
        stride = _rows(q, "q", shape, at)
        if q.dtype != self._dtype:
            _refuse("q's dtype differs from the object's")
        if cache._index != at or cache.num_kv_heads != self.num_kv_heads or cache.head_dim != self.head_dim or \
                cache.page_size != self.page_size:
            _refuse("the cache's heads, head_dim, page_size or device differ from the object's")
        objects = (self, cache)
        if isinstance(tables, BatchTables):
            objects = (self, cache, tables)
            if tables.batch_size != B or tables.page_size != self.page_size or tables._index != at:
                _refuse("the tables' batch, page_size or device differ from the object's")
            qo_indptr, page_indptr, pages, last = tables = (tables.qo_indptr, tables.kv_page_indptr,
                                                            tables.kv_page_indices, tables.kv_last_page_len)
            nnz = pages.shape[0]
        else:
            qo_indptr, page_indptr, pages, last = tables
            nnz, i32 = pages.numel(), torch.int32
            _is(qo_indptr, "qo_indptr", i32, (B + 1,), at)
            _is(page_indptr, "kv_page_indptr", i32, (B + 1,), at)
            _is(pages, "kv_page_indices", i32, (nnz,), at)
            _is(last, "kv_last_page_len", i32, (B,), at)
        if out is not None:
            _is(out, "out", q.dtype, shape, at)
        if lse is not None:
            _is(lse, "lse", torch.float32, shape[:2], at)
        handle, guard = _on(at, stream, objects, (q, out, lse, *tables))
        if guard is None:
            return self._launch(q, stride, cache, qo_indptr, page_indptr, pages, last, nnz, out, lse, return_lse, handle)
        with guard:  # the outputs are allocated on the stream that writes them
            return self._launch(q, stride, cache, qo_indptr, page_indptr, pages, last, nnz, out, lse, return_lse, handle)

    def _launch(self, q, stride, cache, qo_indptr, page_indptr, pages, last, nnz, out, lse, return_lse, handle):
        import torch
        shape = self._shape
        if out is None:
            out = torch.empty(shape, dtype=self._dtype, device=self.device)
        if lse is None and return_lse:
            lse = torch.empty(shape[:2], dtype=torch.float32, device=self.device)
        batch = _KV4_BATCH.pack(qo_indptr.data_ptr(), page_indptr.data_ptr(), pages.data_ptr(), last.data_ptr(),
                                self.batch_size, nnz, shape[0], self.max_qo_len, shape[1], self.causal,
                                self.dtype_code)
        status = self._lib.pagedattn_kv4_run(ctypes.byref(cache._args), batch, q.data_ptr(), stride, out.data_ptr(),
                                             None if lse is None else lse.data_ptr(), self._ws_ptr, self._ws_bytes,
                                             handle)
        if status != _b.PA_OK:
            _b.check(status)
        return out, lse
