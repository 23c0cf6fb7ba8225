"""Split-KV flash attention over a partitioned KV cache, for GB300 (sm_103a).

A thin Python layer over libsplitkv.so (C ABI: include/splitkv.h).  The
functions below carry the C names without the ``skv_`` prefix and only
marshal arguments (torch tensors -> device pointers, streams); all compute
runs in the library's CUDA kernels.  PyTorch provides device memory and
streams.

    h = Handle(0)
    o, lse = attn_partial(h, q, k, v, Hk=8, kv_rows=rows)        # unified cache
    o, lse = attn_window_tail(h, q, k_win, v_win, k_tail, v_tail, Hk=8, ...)
    o, lse = attn_combine(h, o_parts, lse_parts)
    x = kv_dequant_q8_0(h, blocks, n_values)

    pool = Q8Pool.empty(n_pages, D=128)                          # 8-bit pages of 64 tokens of one KV head
    q8_append(h, pool, k_new, v_new, page_ids, kv_len)           # write tokens (kv_len is the caller's to advance)
    o, lse = q8_attn(h, pool, q, page_ids, kv_len, mass=mass)    # attend; mass += each page's attention weight
    sel = q8_select(h, pool, q, page_ids, kv_len, n_sel=64)      # the pages of the largest score bounds ...
    o, lse = q8_attn(h, pool, q, page_ids, kv_len, sel=sel)      # ... and attention over those alone
    page_ids, mass, kv_len, freed = q8_evict(h, page_ids, mass, kv_len, n_keep=512)

    spec = Rope(D, freq)                                         # rotation (and norm) of queries and keys
    q = rope_append(h, spec, x_q, x_k, x_v, pos, rows, K, V)     # q as attention takes it; k, v into cache rows
    q, k = rope(h, spec, x_q, x_k, pos, q_weight=wq, k_weight=wk)
    dq, dk, dv = attn_backward(h, q, k, v, o, lse, d_o, Hk=8, q_pos=pos)
    dx_q, dx_k, dwq, dwk = rope_backward(h, spec, dq, dk, pos, q=x_q, k=x_k, q_weight=wq, k_weight=wk)
"""
from __future__ import annotations

import ctypes
import math

from . import _lib
from ._lib import BF16, F16, F32, Q4_0, Q8_0, Q8_PAGE, SkvCacheDst, SkvQ8Pool, SkvRopeSpec, SkvShape

__all__ = ["Handle", "SplitKVError", "F16", "Q8_0", "Q4_0", "attn_partial", "attn_combine", "attn_window_tail",
           "attn_paged", "BlockCache", "kv_dequant_q8_0", "kv_dequant_q4_0", "gather_rows", "kv_append", "plan_splits", "plan_prefill_splits", "plan_q8_tokens",
           "segment_bytes", "Q8_PAGE", "Q8Pool", "q8_append", "q8_attn", "q8_select", "q8_evict",
           "Rope", "rope", "rope_append", "rope_backward", "attn_backward"]


class SplitKVError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_lib.STATUS.get(status, status)}: {msg}")
        self.status = status


def segment_bytes(type_: int, D: int) -> int:
    return {F16: 2 * D, Q8_0: 34 * (D // 32), Q4_0: 18 * (D // 32)}[type_]


def _torch():
    import torch
    return torch


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Handle:
    """Owns the library handle: copy stream, events, workspace, tail ring."""

    def __init__(self, device: int = 0):
        self._h = ctypes.c_void_p()
        rc = _lib.lib().skv_create(int(device), ctypes.byref(self._h))
        if rc != 0:
            raise SplitKVError(rc, "skv_create failed")
        self.device = device

    @property
    def ptr(self):
        return self._h

    def check(self, rc: int):
        if rc != 0:
            msg = _lib.lib().skv_last_error(self._h).decode(errors="replace")
            raise SplitKVError(rc, msg)

    def reserve(self, workspace_bytes: int = 0, ring_bytes_per_slot: int = 0, n_slots: int = 0):
        self.check(_lib.lib().skv_reserve(self._h, workspace_bytes, ring_bytes_per_slot, n_slots))

    def scratch_info(self):
        ws, ring, n = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int32()
        self.check(_lib.lib().skv_scratch_info(self._h, ctypes.byref(ws), ctypes.byref(ring), ctypes.byref(n)))
        return ws.value, ring.value, n.value

    def sm_count(self) -> int:
        n = ctypes.c_int32()
        self.check(_lib.lib().skv_sm_count(self._h, ctypes.byref(n)))
        return n.value

    def status(self) -> int:
        """Synchronise and read/clear the device status word (raises on a timeout)."""
        code = ctypes.c_int32()
        self.check(_lib.lib().skv_status(self._h, ctypes.byref(code)))
        return code.value

    def set_profile_events(self, before=None, after=None):
        """Bracket later attention-kernel launches with these torch.cuda.Events."""
        b = ctypes.c_void_p(before.cuda_event) if before is not None else None
        a = ctypes.c_void_p(after.cuda_event) if after is not None else None
        self.check(_lib.lib().skv_set_profile_events(self._h, b, a))

    def close(self):
        if self._h:
            _lib.lib().skv_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_prefill_splits(S, nq, H, Hk, n_keys, sm_count, *, k_type=F16, v_type=F16, D=128, rows=False):
    """The split plan a prefill call of this shape gets on the tensor-core
    path (no GPU needed): returns (split_len, n_splits, n_ctas)."""
    sh = SkvShape(int(S), int(nq), int(H), int(Hk), int(D), 1.0 / math.sqrt(D), int(k_type), int(v_type),
                  int(Hk) * segment_bytes(k_type, D), int(Hk) * segment_bytes(v_type, D))
    sl, ns, nc = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int64()
    rc = _lib.lib().skv_plan_prefill_splits(ctypes.byref(sh), int(n_keys), int(sm_count), int(bool(rows)),
                                            ctypes.byref(sl), ctypes.byref(ns), ctypes.byref(nc))
    if rc != 0:
        raise SplitKVError(rc, "skv_plan_prefill_splits rejected its arguments")
    return sl.value, ns.value, nc.value


def plan_splits(n_keys, n_units, sm_count, ctas_per_sm, tile=64, max_split=0):
    """Host-side split planner (no GPU needed): returns (split_len, n_splits)."""
    sl, ns = ctypes.c_int64(), ctypes.c_int32()
    rc = _lib.lib().skv_plan_splits(int(n_keys), int(n_units), int(sm_count), int(ctas_per_sm), int(tile),
                                    int(max_split), ctypes.byref(sl), ctypes.byref(ns))
    if rc != 0:
        raise SplitKVError(rc, "skv_plan_splits rejected its arguments")
    return sl.value, ns.value


def plan_window(per_cell_bytes, kv_size, free_bytes, target_bytes=0, reserve_bytes=1536 << 20, n_pad=256):
    """Host-side resident-window sizing (no GPU needed): cells kept on the device."""
    out = ctypes.c_int64()
    rc = _lib.lib().skv_plan_window(int(per_cell_bytes), int(kv_size), int(free_bytes), int(target_bytes),
                                    int(reserve_bytes), int(n_pad), ctypes.byref(out))
    if rc != 0:
        raise SplitKVError(rc, "skv_plan_window rejected its arguments")
    return out.value


def plan_tail_tile(n_keys, per_key_bytes, n_slots=4, slot_cap_bytes=512 << 20, target_keys=32768, align=256):
    """Host-side tail-tile sizing (no GPU needed): (tile_rows, n_tiles)."""
    rows, n = ctypes.c_int64(), ctypes.c_int32()
    rc = _lib.lib().skv_plan_tail_tile(int(n_keys), int(per_key_bytes), int(n_slots), int(slot_cap_bytes),
                                       int(target_keys), int(align), ctypes.byref(rows), ctypes.byref(n))
    if rc != 0:
        raise SplitKVError(rc, "skv_plan_tail_tile rejected its arguments")
    return rows.value, n.value


def _shape(q, Hk, k_type, v_type, k_row_bytes, v_row_bytes, scale):
    S, nq, H, D = (int(x) for x in q.shape)
    if k_row_bytes is None:
        k_row_bytes = Hk * segment_bytes(k_type, D)
    if v_row_bytes is None:
        v_row_bytes = Hk * segment_bytes(v_type, D)
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    return SkvShape(S, nq, H, int(Hk), D, sc, int(k_type), int(v_type), int(k_row_bytes), int(v_row_bytes))


def _outputs(q, o, lse):
    torch = _torch()
    S, nq, H, D = q.shape
    if o is None:
        o = torch.empty((S, nq, H, D), dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty((S, nq, H), dtype=torch.float32, device=q.device)
    return o, lse


def attn_partial(h: Handle, q, k, v, *, Hk, k_type=F16, v_type=F16, k_row_bytes=None, v_row_bytes=None,
                 scale=None, kv_begin=0, kv_end=None, kv_rows=None, kv_rows_per_head=False,
                 mask=None, q_pos=None, key_pos0=0, o=None, lse=None, stream=None):
    """skv_attn_partial: attention over logical keys [kv_begin, kv_end)."""
    sh = _shape(q, Hk, k_type, v_type, k_row_bytes, v_row_bytes, scale)
    if kv_end is None:
        kv_end = int(kv_rows.shape[-1]) if kv_rows is not None else int(k.shape[0])
    rows_ld = int(kv_rows.shape[-1]) if kv_rows is not None else 0
    mask_ld = int(mask.shape[-1]) if mask is not None else 0
    o, lse = _outputs(q, o, lse)
    h.check(_lib.lib().skv_attn_partial(h.ptr, ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), _ptr(mask), mask_ld,
                                        _ptr(q_pos), int(key_pos0), _ptr(kv_rows), rows_ld,
                                        int(bool(kv_rows_per_head)), int(kv_begin), int(kv_end), _ptr(o),
                                        _ptr(lse), _stream(stream)))
    return o, lse


def attn_combine(h: Handle, o_parts, lse_parts, *, o=None, lse=None, stream=None):
    """skv_attn_combine: o_parts [P, rows, D] fp32, lse_parts [P, rows] -> (o [rows, D], lse [rows])."""
    torch = _torch()
    P, rows, D = (int(x) for x in o_parts.shape)
    if o is None:
        o = torch.empty((rows, D), dtype=torch.float32, device=o_parts.device)
    if lse is None:
        lse = torch.empty((rows,), dtype=torch.float32, device=o_parts.device)
    h.check(_lib.lib().skv_attn_combine(h.ptr, P, _ptr(o_parts), _ptr(lse_parts), rows, D, _ptr(o), _ptr(lse),
                                        _stream(stream)))
    return o, lse


def attn_window_tail(h: Handle, q, k_win, v_win, k_tail_host, v_tail_host, *, Hk, n_win=None, n_tail=None,
                     tile_rows=0, k_type=F16, v_type=F16, k_row_bytes=None, v_row_bytes=None, scale=None,
                     mask=None, q_pos=None, o=None, lse=None, stream=None):
    """skv_attn_window_tail: window rows on the device, tail rows in pinned host memory.

    tile_rows <= 0 lets the library size the tail tiles (skv_plan_tail_tile)."""
    sh = _shape(q, Hk, k_type, v_type, k_row_bytes, v_row_bytes, scale)
    if n_win is None:
        n_win = int(k_win.shape[0]) if k_win is not None else 0
    if n_tail is None:
        n_tail = int(k_tail_host.shape[0]) if k_tail_host is not None else 0
    mask_ld = int(mask.shape[-1]) if mask is not None else 0
    o, lse = _outputs(q, o, lse)
    h.check(_lib.lib().skv_attn_window_tail(h.ptr, ctypes.byref(sh), _ptr(q), _ptr(k_win), _ptr(v_win), int(n_win),
                                            _ptr(k_tail_host), _ptr(v_tail_host), int(n_tail), int(tile_rows),
                                            _ptr(mask), mask_ld, _ptr(q_pos), _ptr(o), _ptr(lse), _stream(stream)))
    return o, lse


def attn_paged(h: Handle, q, k_pages, v_pages, page_ids, *, Hk, page_rows, scale=None, o=None, lse=None,
               stream=None):
    """skv_attn_paged: page_ids int32 [S, Hk, pages_per_list] into pools of
    page_rows x D fp16 pages (one KV head per page)."""
    sh = _shape(q, Hk, F16, F16, None, None, scale)
    o, lse = _outputs(q, o, lse)
    h.check(_lib.lib().skv_attn_paged(h.ptr, ctypes.byref(sh), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                      int(page_rows), _ptr(page_ids), int(page_ids.shape[-1]), _ptr(o), _ptr(lse),
                                      _stream(stream)))
    return o, lse


class BlockCache:
    """Device block cache over a pinned paged host copy [n_blocks][Hk][block_rows][D] fp16."""

    def __init__(self, h: Handle, host_k, host_v, *, n_blocks, block_rows, Hk, D, n_slots=0, max_lookups=0,
                 ring_blocks=0, max_seqs=1):
        """ring_blocks > 0 makes a ring (static table block -> block % ring_blocks)."""
        self.h = h
        self.Hk, self.D, self.block_rows = int(Hk), int(D), int(block_rows)
        self.ring_blocks = int(ring_blocks)
        self._c = ctypes.c_void_p()
        if self.ring_blocks > 0:
            h.check(_lib.lib().skv_bcache_create_ring(h.ptr, int(n_blocks), int(block_rows), int(Hk), int(D),
                                                      self.ring_blocks, int(max_seqs), _ptr(host_k), _ptr(host_v),
                                                      ctypes.byref(self._c)))
        else:
            h.check(_lib.lib().skv_bcache_create(h.ptr, int(n_blocks), int(block_rows), int(Hk), int(D),
                                                 int(n_slots), int(max_lookups), _ptr(host_k), _ptr(host_v),
                                                 ctypes.byref(self._c)))
        self._keep = (host_k, host_v)

    def ring_restore(self, n_keys, stream=None):
        self.h.check(_lib.lib().skv_bcache_ring_restore(self._c, int(n_keys), _stream(stream)))

    def ring_attn(self, q, n_keys, window=0, *, scale=None, o=None, lse=None, stream=None):
        sh = _shape(q, self.Hk, F16, F16, None, None, scale)
        o, lse = _outputs(q, o, lse)
        self.h.check(_lib.lib().skv_bcache_ring_attn(self._c, ctypes.byref(sh), _ptr(q), int(n_keys), int(window),
                                                     _ptr(o), _ptr(lse), _stream(stream)))
        return o, lse

    def reset(self, stream=None):
        self.h.check(_lib.lib().skv_bcache_reset(self._c, _stream(stream)))

    def resolve(self, sel, page_ids=None, stream=None):
        S, _, n_sel = (int(x) for x in sel.shape)
        self.h.check(_lib.lib().skv_bcache_resolve(self._c, _ptr(sel), S, n_sel, _ptr(page_ids), _stream(stream)))
        return page_ids

    def append(self, k_new, v_new, positions, stream=None):
        """Write-through append of fp32 rows [n][Hk][D] at cache positions."""
        self.h.check(_lib.lib().skv_bcache_append(self._c, _ptr(k_new), _ptr(v_new), _ptr(positions),
                                                  int(positions.numel()), _stream(stream)))

    def attn(self, q, sel, *, scale=None, o=None, lse=None, stream=None):
        sh = _shape(q, self.Hk, F16, F16, None, None, scale)
        o, lse = _outputs(q, o, lse)
        self.h.check(_lib.lib().skv_bcache_attn(self._c, ctypes.byref(sh), _ptr(q), _ptr(sel), int(sel.shape[-1]),
                                                _ptr(o), _ptr(lse), _stream(stream)))
        return o, lse

    def stats(self):
        c = _lib.SkvBcacheCounters()
        self.h.check(_lib.lib().skv_bcache_stats(self._c, ctypes.byref(c)))
        return {k: getattr(c, k) for k, _ in c._fields_}

    def check(self) -> int:
        v = ctypes.c_int32()
        self.h.check(_lib.lib().skv_bcache_check(self._c, ctypes.byref(v)))
        return v.value

    def pool(self):
        k, v, n, ids = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_void_p()
        self.h.check(_lib.lib().skv_bcache_pool(self._c, ctypes.byref(k), ctypes.byref(v), ctypes.byref(n),
                                                ctypes.byref(ids)))
        return k.value, v.value, n.value, ids.value

    def close(self):
        if self._c:
            _lib.lib().skv_bcache_destroy(self._c)
            self._c = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _dequant(fn, h, blocks, n_values, out, stream):
    torch = _torch()
    if out is None:
        out = torch.empty((n_values,), dtype=torch.float32, device=blocks.device)
    h.check(fn(h.ptr, _ptr(blocks), int(n_values), _ptr(out), _stream(stream)))
    return out


def kv_dequant_q8_0(h: Handle, blocks, n_values, *, out=None, stream=None):
    return _dequant(_lib.lib().skv_kv_dequant_q8_0, h, blocks, n_values, out, stream)


def kv_dequant_q4_0(h: Handle, blocks, n_values, *, out=None, stream=None):
    return _dequant(_lib.lib().skv_kv_dequant_q4_0, h, blocks, n_values, out, stream)


def gather_rows(h: Handle, src, rows, *, row_bytes=None, out=None, stream=None):
    """dst[i] = src[rows[i]]; negative rows give zero rows."""
    torch = _torch()
    n = int(rows.numel())
    if row_bytes is None:
        row_bytes = src[0].numel() * src.element_size()
    if out is None:
        out = torch.empty((n, row_bytes), dtype=torch.uint8, device=src.device)
    h.check(_lib.lib().skv_gather_rows(h.ptr, _ptr(src), int(row_bytes), _ptr(rows), n, _ptr(out),
                                       _stream(stream)))
    return out


def selftest_wait_timeout(h: Handle, budget_ns: int = 5_000_000, stream=None):
    """skv_selftest_wait_timeout: a bounded device-side wait that nothing
    completes gives up after budget_ns and marks the handle's status word."""
    h.check(_lib.lib().skv_selftest_wait_timeout(h.ptr, int(budget_ns), _stream(stream)))


def kv_append(h: Handle, x, positions, dst0, dst1=None, *, type_=F16, n_rows0=None, n_rows1=None, row_bytes=None,
              stream=None):
    """Write x (fp32 [n][Hk][D], device) into a two-region cell-major cache:
    position p < n_rows0 goes to row p of dst0, otherwise row p - n_rows0 of
    dst1 (device or page-locked host).  Rows are converted to fp16 or
    quantised to q8_0 / q4_0 according to type_."""
    n, Hk, D = (int(s) for s in x.shape)
    if row_bytes is None:
        row_bytes = Hk * segment_bytes(type_, D)
    if n_rows0 is None:
        n_rows0 = 0 if dst0 is None else dst0.numel() * dst0.element_size() // row_bytes
    if n_rows1 is None:
        n_rows1 = 0 if dst1 is None else dst1.numel() * dst1.element_size() // row_bytes
    h.check(_lib.lib().skv_kv_append(h.ptr, int(type_), Hk, D, int(row_bytes), _ptr(x), _ptr(positions), n,
                                     _ptr(dst0), int(n_rows0), _ptr(dst1), int(n_rows1), _stream(stream)))


class Q8Pool:
    """8-bit pages (see include/splitkv.h): k, v int8 [n_pages][64][D], k_scale,
    v_scale fp32 [n_pages], k_min, k_max int8 [n_pages][D].  The tensors stay
    the caller's; the pool keeps references to them."""

    def __init__(self, k, v, k_scale, v_scale, k_min, k_max):
        torch = _torch()
        if k.dim() != 3:
            raise SplitKVError(1, f"k: want int8 [n_pages, {Q8_PAGE}, D], got {list(k.shape)}")
        n, _, D = (int(x) for x in k.shape)
        want = [("k", k, torch.int8, (n, Q8_PAGE, D)), ("v", v, torch.int8, (n, Q8_PAGE, D)),
                ("k_scale", k_scale, torch.float32, (n,)), ("v_scale", v_scale, torch.float32, (n,)),
                ("k_min", k_min, torch.int8, (n, D)), ("k_max", k_max, torch.int8, (n, D))]
        for name, x, dtype, shape in want:
            _need(name, x, dtype, shape, k.get_device())
        self.n_pages, self.D, self.device, self.scale = n, D, k.get_device(), 1.0 / math.sqrt(max(1, D))
        self.k, self.v, self.k_scale, self.v_scale, self.k_min, self.k_max = k, v, k_scale, v_scale, k_min, k_max
        self._c = SkvQ8Pool(n, D, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                            k_min.data_ptr(), k_max.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages, D, device="cuda"):
        """A pool of unwritten pages (appends need nothing cleared)."""
        torch = _torch()
        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=device)
        n, D = int(n_pages), int(D)
        return cls(new((n, Q8_PAGE, D), torch.int8), new((n, Q8_PAGE, D), torch.int8), new((n,), torch.float32),
                   new((n,), torch.float32), new((n, D), torch.int8), new((n, D), torch.int8))


def _need(name, x, dtype, shape, device):
    """Raise SKV_EINVAL unless x is a contiguous tensor of this type, shape and
    device (an index, -1 for the CPU)."""
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or not x.is_contiguous():
        raise SplitKVError(1, f"{name}: want contiguous {dtype} {list(shape)} on device {device}, got "
                              f"{'' if x.is_contiguous() else 'non-contiguous '}{x.dtype} {list(x.shape)} on {x.device}")


def _q8_stream(h, stream, device):
    """The raw stream of a call over 8-bit pages (default: the current one of the tensors' device)."""
    if device != h.device:
        raise SplitKVError(1, f"tensors on device {device}, handle on cuda:{h.device}")
    if stream is None:
        return _raw_stream()(device)
    return _stream(stream)


def _on_stream(stream, device):
    """Context in which the results of a call on a given stream are allocated: they
    belong to that stream, so that memory freed on another one is not written early."""
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


_raw_stream_fn = None


def _raw_stream():
    global _raw_stream_fn
    if _raw_stream_fn is None:
        torch = _torch()
        # the same number as torch.cuda.current_stream(device).cuda_stream, without the objects
        _raw_stream_fn = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream_fn


def _q8_lists(torch, page_ids, kv_len, device):
    shape = page_ids.shape
    if len(shape) != 3:
        raise SplitKVError(1, f"page_ids: want int32 [S, Hk, pages_per_list], got {list(shape)}")
    _need("page_ids", page_ids, torch.int32, shape, device)
    _need("kv_len", kv_len, torch.int32, shape[:1], device)
    return shape


def _q8_query(torch, pool, q, page_ids, kv_len, q_pos, scale):
    dev, D = pool.device, pool.D
    lists, shape = page_ids.shape, q.shape
    # all checks in one expression; what fails is found again below, with its message
    if not (len(lists) == 3 and len(shape) == 4 and page_ids.dtype is torch.int32 and kv_len.dtype is torch.int32
            and q.dtype is torch.float16 and kv_len.shape == lists[:1] and shape[0] == lists[0] and shape[3] == D
            and page_ids.get_device() == dev and kv_len.get_device() == dev and q.get_device() == dev
            and page_ids.is_contiguous() and kv_len.is_contiguous() and q.is_contiguous()):
        _q8_lists(torch, page_ids, kv_len, dev)
        if len(shape) != 4:
            raise SplitKVError(1, f"q: want fp16 [S, nq, H, D], got {list(shape)}")
        _need("q", q, torch.float16, (lists[0], shape[1], shape[2], D), dev)
    S, Hk, cap = lists
    _, nq, H, _ = shape
    if q_pos is not None:
        _need("q_pos", q_pos, torch.int32, (S, nq), dev)
    return SkvShape(S, nq, H, Hk, D, pool.scale if scale is None else float(scale), 0, 0, 0, 0), S, nq, H, Hk, cap


def q8_append(h: Handle, pool: Q8Pool, k_new, v_new, page_ids, kv_len, *, n_new=None, stream=None):
    """skv_q8_append: write k_new, v_new (fp32 or fp16 [S, n, Hk, D]) as tokens
    kv_len[s] .. of each sequence; n_new int32 [S]: how many of the n rows."""
    torch = _torch()
    S, Hk, cap = _q8_lists(torch, page_ids, kv_len, pool.device)
    st = _q8_stream(h, stream, pool.device)
    if k_new.dim() != 4 or k_new.dtype not in (torch.float32, torch.float16):
        raise SplitKVError(1, f"k_new: want fp32 or fp16 [S, n, Hk, D], got {k_new.dtype} {list(k_new.shape)}")
    n = k_new.shape[1]
    _need("k_new", k_new, k_new.dtype, (S, n, Hk, pool.D), pool.device)
    _need("v_new", v_new, k_new.dtype, (S, n, Hk, pool.D), pool.device)
    if n_new is not None:
        _need("n_new", n_new, torch.int32, (S,), pool.device)
    h.check(_lib.lib().skv_q8_append(h.ptr, pool._ref, S, Hk, n, F32 if k_new.dtype == torch.float32 else F16,
                                     k_new.data_ptr(), v_new.data_ptr(), page_ids.data_ptr(), cap,
                                     kv_len.data_ptr(), _ptr(n_new), st))


def q8_attn(h: Handle, pool: Q8Pool, q, page_ids, kv_len, *, scale=None, q_pos=None, sel=None, mass=None,
            o_dtype=None, o=None, lse=None, stream=None):
    """skv_q8_attn: attention of q over the lists (sel: over those pages of
    them); mass fp32 [S, Hk, pages_per_list] is added to.  o is fp32 unless
    o_dtype (or a given o) is torch.float16."""
    torch = _torch()
    dev = pool.device
    sh, S, nq, H, Hk, cap = _q8_query(torch, pool, q, page_ids, kv_len, q_pos, scale)
    st = _q8_stream(h, stream, dev)
    if o is None:
        if o_dtype is None:
            o_dtype = torch.float32
        if stream is None:
            o = torch.empty_like(q, dtype=o_dtype)
        else:
            with _on_stream(stream, dev):
                o = torch.empty_like(q, dtype=o_dtype)
    else:
        _need("o", o, o.dtype, q.shape, dev)
    if o.dtype is torch.float32:
        o_type = F32
    elif o.dtype is torch.float16:
        o_type = F16
    else:
        raise SplitKVError(1, f"o: fp32 or fp16 is wanted, got {o.dtype}")
    if o_dtype is not None and o.dtype is not o_dtype:
        raise SplitKVError(1, f"o is {o.dtype}, o_dtype {o_dtype}")
    if lse is None:
        if stream is None:
            lse = torch.empty((S, nq, H), dtype=torch.float32, device=q.device)
        else:
            with _on_stream(stream, dev):
                lse = torch.empty((S, nq, H), dtype=torch.float32, device=q.device)
    else:
        _need("lse", lse, torch.float32, (S, nq, H), dev)
    n_sel, sel_ptr, mass_ptr = 0, None, None
    if sel is not None:
        n_sel = sel.shape[-1]
        _need("sel", sel, torch.int32, (S, nq, Hk, n_sel), dev)
        sel_ptr = sel.data_ptr()
    if mass is not None:
        _need("mass", mass, torch.float32, (S, Hk, cap), dev)
        mass_ptr = mass.data_ptr()
    rc = _lib.lib().skv_q8_attn(h._h, pool._ref, ctypes.byref(sh), q.data_ptr(), page_ids.data_ptr(), cap,
                                kv_len.data_ptr(), None if q_pos is None else q_pos.data_ptr(), sel_ptr, n_sel,
                                mass_ptr, o_type, o.data_ptr(), lse.data_ptr(), st)
    if rc:
        h.check(rc)
    return o, lse


def plan_q8_tokens(S, nq, H, Hk, pages_per_list, *, n_sel=0, mass=False):
    """skv_plan_q8_tokens: the tokens that one launch of q8_attn takes for calls of
    this shape (n_sel 0: over whole lists).  Needs no GPU."""
    sh, n = SkvShape(int(S), int(nq), int(H), int(Hk), 128, 1.0, 0, 0, 0, 0), ctypes.c_int32()
    rc = _lib.lib().skv_plan_q8_tokens(ctypes.byref(sh), int(pages_per_list), int(n_sel), int(bool(mass)), ctypes.byref(n))
    if rc != 0:
        raise SplitKVError(rc, "skv_plan_q8_tokens rejected its arguments")
    return n.value


def q8_select(h: Handle, pool: Q8Pool, q, page_ids, kv_len, *, n_sel, n_first=1, n_last=1, q_pos=None, sel=None,
              stream=None):
    """skv_q8_select: the n_sel list indices int32 [S, nq, Hk, n_sel] (ascending,
    -1 padded) of the pages with the largest score bounds for each query and
    KV head, the first n_first and last n_last among them."""
    torch = _torch()
    sh, S, nq, H, Hk, cap = _q8_query(torch, pool, q, page_ids, kv_len, q_pos, None)
    st = _q8_stream(h, stream, pool.device)
    n_sel = int(n_sel)
    if sel is None:
        shape = (S, nq, Hk, max(0, n_sel))
        if stream is None:
            sel = torch.empty(shape, dtype=torch.int32, device=q.device)
        else:
            with _on_stream(stream, pool.device):
                sel = torch.empty(shape, dtype=torch.int32, device=q.device)
    else:
        _need("sel", sel, torch.int32, (S, nq, Hk, n_sel), pool.device)
    rc = _lib.lib().skv_q8_select(h._h, pool._ref, ctypes.byref(sh), q.data_ptr(), page_ids.data_ptr(), cap,
                                  kv_len.data_ptr(), None if q_pos is None else q_pos.data_ptr(), n_sel, int(n_first),
                                  int(n_last), sel.data_ptr(), st)
    if rc:
        h.check(rc)
    return sel


def q8_evict(h: Handle, page_ids, mass, kv_len, *, n_keep, n_first=1, n_last=1, stream=None):
    """skv_q8_evict: lists cut to n_keep pages (the first n_first, the last
    n_last, the others of largest mass): (page_ids, mass, kv_len, freed)."""
    torch = _torch()
    dev = page_ids.get_device()
    S, Hk, cap = _q8_lists(torch, page_ids, kv_len, dev)
    st = _q8_stream(h, stream, dev)
    _need("mass", mass, torch.float32, (S, Hk, cap), dev)
    def results():
        return (torch.empty_like(page_ids), torch.empty_like(mass), torch.empty_like(kv_len),
                torch.empty_like(page_ids))
    if stream is None:
        ids_out, mass_out, len_out, freed = results()
    else:
        with _on_stream(stream, dev):
            ids_out, mass_out, len_out, freed = results()
    h.check(_lib.lib().skv_q8_evict(h.ptr, S, Hk, cap, page_ids.data_ptr(), mass.data_ptr(), kv_len.data_ptr(),
                                    int(n_keep), int(n_first), int(n_last), ids_out.data_ptr(), mass_out.data_ptr(),
                                    len_out.data_ptr(), freed.data_ptr(), st))
    return ids_out, mass_out, len_out, freed


class Rope:
    """How rows turn (see include/splitkv.h): freq fp32 [rot_dims/2] (device), the
    angle of each pair per position; axis int32 [rot_dims/2]: the axis of pos that a
    pair turns with (None: the first); interleaved: pairs (2i, 2i+1) instead of
    (i, i + rot_dims/2); factor: on cos and sin; eps: of the norm.  The tensors stay
    the caller's; the spec keeps references to them."""

    def __init__(self, D, freq, *, axis=None, interleaved=False, factor=1.0, eps=1e-6, n_axes=None):
        torch = _torch()
        if freq.dim() != 1:
            raise SplitKVError(1, f"freq: want fp32 [rot_dims/2], got {list(freq.shape)}")
        half, self.device = int(freq.shape[0]), freq.get_device()
        _need("freq", freq, torch.float32, (half,), self.device)
        if axis is not None:
            _need("axis", axis, torch.int32, (half,), self.device)
            if n_axes is None:
                n_axes = int(axis.max().item()) + 1 if half else 1
        self.D, self.rot_dims, self.n_axes, self.freq, self.axis = int(D), 2 * half, int(n_axes or 1), freq, axis
        self._c = SkvRopeSpec(self.D, 2 * half, int(bool(interleaved)), self.n_axes, freq.data_ptr(), _ptr(axis),
                              float(factor), float(eps))
        self._d = (self.D,)
        self._ref = ctypes.byref(self._c)


_row_types = None


def _row_type(name, dtype):
    global _row_types
    if _row_types is None:
        torch = _torch()
        _row_types = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    t = _row_types.get(dtype)
    if t is None:
        raise SplitKVError(1, f"{name}: fp32, fp16 or bf16 is wanted, got {dtype}")
    return t


def _token_rows(name, x, lead, D, dtype, device):
    """Heads and token stride of rows [*lead, heads, D] whose heads stand side by side and whose tokens a fixed
    stride apart (a part of a packed projection, say), which holds a token's heads: broadcast or overlapping tokens are
    refused."""
    shape, stride, k = x.shape, x.stride(), len(lead)
    ok = x.dtype is dtype and x.get_device() == device
    if (k == 1 and ok and len(shape) == 3 and shape[0] == lead[0] and shape[2] == D and stride[2] == 1 and stride[1] == D
            and (stride[0] >= shape[1] * D or shape[0] <= 1)):
        return shape[1], stride[0]                            # the usual case, without the loop
    ok = (ok and len(shape) == k + 2 and shape[:k] == lead and shape[-1] == D
          and (stride[-1] == 1 and (stride[-2] == D or shape[-2] == 1) or x.numel() == 0))
    step = want = None                                        # None: no dimension has more than one token
    if ok:
        for i in range(k - 1, -1, -1):
            if shape[i] > 1:
                if want is None:
                    step = stride[i]
                    want = step * shape[i]
                elif stride[i] != want:
                    ok = x.numel() == 0
                    break
                else:
                    want *= shape[i]
        if step is not None and step < shape[-2] * D and x.numel():
            ok = False
    if not ok:
        raise SplitKVError(1, f"{name}: want {dtype} [{', '.join(map(str, lead))}, heads, {D}] on device {device} with heads side by side "
                              f"and tokens a fixed stride apart, got {x.dtype} {list(shape)} of strides {list(stride)} on {x.device}")
    return int(shape[-2]), int(shape[-2]) * D if step is None else int(step)


def _tokens(lead):
    n = 1
    for m in lead:
        n *= m
    return n


def _positions(torch, name, pos, axes, lead, n, device):
    """Pointer of positions of n tokens: int32 [axes, *lead] or [axes, n]; for one axis also without it."""
    shape = pos.shape
    if not ((shape == (axes, n) or axes == 1 and (shape == lead or shape == (n,)) or shape == (axes, *lead))
            and pos.dtype is torch.int32 and pos.get_device() == device and pos.is_contiguous()):
        want = ", ".join(map(str, (axes, *lead) if axes > 1 else lead))
        raise SplitKVError(1, f"{name}: want contiguous int32 [{want}] (positions) on device {device}, got "
                              f"{'' if pos.is_contiguous() else 'non-contiguous '}{pos.dtype} {list(shape)} on {pos.device}")
    return pos.data_ptr()


def _weight(torch, name, w, spec):
    if w is None:
        return None
    if w.dtype is not torch.float32 or w.shape != spec._d or w.get_device() != spec.device or not w.is_contiguous():
        _need(name, w, torch.float32, spec._d, spec.device)
    return w.data_ptr()


def _new(torch, shape, dtype, like, stream, device):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _on_stream(stream, device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _rope_inputs(torch, h, spec, q, k, pos, stream):
    """stream, leading shape, tokens, H, q stride, Hk, k stride, row type, pointer of pos"""
    some = k if k is not None else q
    if some is None:
        raise SplitKVError(1, "q or k is wanted")
    lead, dev, D, dtype = some.shape[:-2], spec.device, spec.D, some.dtype
    st = _q8_stream(h, stream, dev)
    xt = _row_type("q" if some is q else "k", dtype)
    H, qs = _token_rows("q", q, lead, D, dtype, dev) if q is not None else (0, 0)
    Hk, ks = _token_rows("k", k, lead, D, dtype, dev) if k is not None else (0, 0)
    n = lead[0] if len(lead) == 1 else _tokens(lead)
    return st, lead, n, H, qs, Hk, ks, xt, _positions(torch, "pos", pos, spec.n_axes, lead, n, dev)


def rope(h: Handle, spec: Rope, q, k, pos, *, q_weight=None, k_weight=None, o_dtype=None, q_out=None, k_out=None,
         stream=None):
    """skv_rope: norm (where a weight fp32 [D] is given) and rotation of q [..., H, D] and k [..., Hk, D]
    (fp32, fp16 or bf16; either may be None); pos int32 [n_axes, ...] or, tokens in one line, [n_axes, n] (without the
    axis for one).
    Results are fp16 unless o_dtype (or a given q_out, k_out) says otherwise."""
    torch = _torch()
    st, lead, n, H, qs, Hk, ks, xt, pp = _rope_inputs(torch, h, spec, q, k, pos, stream)
    wq, wk = _weight(torch, "q_weight", q_weight, spec), _weight(torch, "k_weight", k_weight, spec)
    if o_dtype is None:
        o_dtype = q_out.dtype if q_out is not None else k_out.dtype if k_out is not None else torch.float16
    ot, D = _row_type("o_dtype", o_dtype), spec.D
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = _new(torch, (*lead, H, D), o_dtype, q, stream, spec.device)
    else:
        _need("q_out", q_out, o_dtype, (*lead, H, D), spec.device)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = _new(torch, (*lead, Hk, D), o_dtype, k, stream, spec.device)
    else:
        _need("k_out", k_out, o_dtype, (*lead, Hk, D), spec.device)
    rc = _lib.lib().skv_rope(h._h, spec._ref, n, H, Hk, xt, _ptr(q), qs, _ptr(k), ks, wq, wk, pp, ot, _ptr(q_out),
                             _ptr(k_out), st)
    if rc:
        h.check(rc)
    return q_out, k_out


def _region_rows(torch, name, x, half, need, row_bytes, n_rows, device):
    """Rows of `need` bytes, row_bytes apart, that a cache region's tensor holds (or n_rows of them): contiguous memory, or
    rows with that pitch (a part of a packed cache, say).  half: fp16 rows."""
    dtype = x.dtype
    if dtype is not torch.uint8 and dtype.is_floating_point and not (half and dtype is torch.float16):
        raise SplitKVError(1, f"{name}: want {'fp16 or ' if half else ''}bytes, got {dtype}")
    at = x.get_device()
    if at != device and at >= 0:
        raise SplitKVError(1, f"{name}: on device {at}, other tensors on {device}")
    if row_bytes < need or row_bytes < 1:
        raise SplitKVError(1, f"{name}: a row stride of {row_bytes} bytes, a row has {need}")
    if x.is_contiguous():
        held = x.nbytes
        n = held // row_bytes or int(held >= need)            # (one row needs no padding behind it)
    else:
        row, size = x[0], x.element_size()
        if x.stride(0) * size != row_bytes or not row.is_contiguous() or row.numel() * size < need:
            raise SplitKVError(1, f"{name}: {list(x.shape)} of strides {list(x.stride())} is not contiguous and holds no rows "
                                  f"{row_bytes} bytes apart (rows of another pitch want their row bytes)")
        n = x.shape[0]
    if n_rows is None:
        return n
    if n_rows > n and (n_rows - 1) * row_bytes + need > x.untyped_storage().nbytes() - x.element_size() * x.storage_offset():
        raise SplitKVError(1, f"{name}: {n_rows} rows lie beyond its memory at {row_bytes} bytes a row")
    return n_rows


def _cache_dst(torch, name, type_, Hk, D, dst0, dst1, n_rows0, n_rows1, row_bytes, device):
    if type_ not in (F16, Q8_0, Q4_0):
        raise SplitKVError(1, f"{name}_type: unknown element type {type_}")
    half, p0, p1 = type_ == F16, None, None
    need = Hk * 2 * D if half else Hk * segment_bytes(type_, D)
    if row_bytes is None:
        row_bytes = need
    if dst0 is not None:
        n_rows0, p0 = _region_rows(torch, name + "_dst0", dst0, half, need, row_bytes, n_rows0, device), dst0.data_ptr()
    if dst1 is not None:
        n_rows1, p1 = _region_rows(torch, name + "_dst1", dst1, half, need, row_bytes, n_rows1, device), dst1.data_ptr()
    return SkvCacheDst(type_, row_bytes, p0, n_rows0 or 0, p1, n_rows1 or 0)


def rope_append(h: Handle, spec: Rope, q, k, v, pos, positions, k_dst0, v_dst0, k_dst1=None, v_dst1=None, *,
                q_weight=None, k_weight=None, k_type=F16, v_type=F16, n_rows0=None, n_rows1=None, k_row_bytes=None,
                v_row_bytes=None, q_out=None, stream=None):
    """skv_rope_append: norm and rotation of q [..., H, D] and k [..., Hk, D]; q is returned as fp16 rows, k and
    v [..., Hk, D] go to the cache rows `positions` (int32 [...]) of two-region caches as for kv_append.  A region is a
    contiguous tensor (fp16 rows or bytes), or one whose rows are k_row_bytes, v_row_bytes apart (a part of a packed
    cache: its pitch), on the device or page-locked."""
    torch = _torch()
    if k is None or v is None:
        raise SplitKVError(1, "k and v are wanted")
    st, lead, n, H, qs, Hk, ks, xt, pp = _rope_inputs(torch, h, spec, q, k, pos, stream)
    D, dev = spec.D, spec.device
    Hv, vs = _token_rows("v", v, lead, D, k.dtype, dev)
    if Hv != Hk:
        raise SplitKVError(1, f"v has {Hv} heads, k {Hk}")
    wq, wk = _weight(torch, "q_weight", q_weight, spec), _weight(torch, "k_weight", k_weight, spec)
    at = _positions(torch, "positions", positions, 1, lead, n, dev)
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = _new(torch, (*lead, H, D), torch.float16, q, stream, dev)
    else:
        _need("q_out", q_out, torch.float16, (*lead, H, D), dev)
    kd = _cache_dst(torch, "k", k_type, Hk, D, k_dst0, k_dst1, n_rows0, n_rows1, k_row_bytes, dev)
    vd = _cache_dst(torch, "v", v_type, Hk, D, v_dst0, v_dst1, n_rows0, n_rows1, v_row_bytes, dev)
    rc = _lib.lib().skv_rope_append(h._h, spec._ref, n, H, Hk, xt, _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                                    wq, wk, pp, at, _ptr(q_out), ctypes.byref(kd), ctypes.byref(vd), st)
    if rc:
        h.check(rc)
    return q_out


def rope_backward(h: Handle, spec: Rope, dq_out, dk_out, pos, *, q=None, k=None, q_weight=None, k_weight=None,
                  x_dtype=None, dq=None, dk=None, stream=None):
    """skv_rope_backward: (dq, dk, dq_weight, dk_weight) from the gradients of rope's results.  q, k: rope's
    inputs, wanted where a weight is given; the gradients have their type, or x_dtype (the results' gradients'
    type by default).  dq, dk may be given (rows of a packed gradient, say)."""
    torch = _torch()
    some = dq_out if dq_out is not None else dk_out
    if some is None:
        raise SplitKVError(1, "dq_out or dk_out is wanted")
    lead, dev, D = some.shape[:-2], spec.device, spec.D
    st = _q8_stream(h, stream, dev)
    g_dtype = some.dtype
    gt = _row_type("dq_out" if some is dq_out else "dk_out", g_dtype)
    n = lead[0] if len(lead) == 1 else _tokens(lead)
    pp = _positions(torch, "pos", pos, spec.n_axes, lead, n, dev)
    wq, wk = _weight(torch, "q_weight", q_weight, spec), _weight(torch, "k_weight", k_weight, spec)
    if x_dtype is None:
        x_dtype = next((x.dtype for x in (q, k, dq, dk) if x is not None), g_dtype)
    xt = _row_type("x_dtype", x_dtype)

    def side(name, g, x, w, out):
        """heads, pointer and stride of x, of the gradient, the gradient and that of the weight"""
        if g is None:
            if w is not None:
                raise SplitKVError(1, f"{name}_weight without d{name}_out")
            return 0, None, 0, None, 0, None
        shape = g.shape
        if len(shape) != len(lead) + 2:
            raise SplitKVError(1, f"d{name}_out: want [..., heads, {D}], got {list(shape)}")
        hd = shape[-2]
        _need(f"d{name}_out", g, g_dtype, (*lead, hd, D), dev)
        ptr = dw = None
        stride = 0
        if w is not None:
            if x is None:
                raise SplitKVError(1, f"{name} is wanted with its weight")
            xh, stride = _token_rows(name, x, lead, D, x_dtype, dev)
            if xh != hd:
                raise SplitKVError(1, f"{name} has {xh} heads, d{name}_out {hd}")
            ptr, dw = x.data_ptr(), _new(torch, spec._d, torch.float32, g, stream, dev)
        if out is None:
            return hd, ptr, stride, _new(torch, shape, x_dtype, g, stream, dev), hd * D, dw
        oh, ostride = _token_rows(f"d{name}", out, lead, D, x_dtype, dev)
        if oh != hd:
            raise SplitKVError(1, f"d{name} has {oh} heads, d{name}_out {hd}")
        return hd, ptr, stride, out, ostride, dw

    H, qp, qs, dq, dqs, dwq = side("q", dq_out, q, q_weight, dq)
    Hk, kp, ks, dk, dks, dwk = side("k", dk_out, k, k_weight, dk)
    rc = _lib.lib().skv_rope_backward(h._h, spec._ref, n, H, Hk, xt, qp, qs, kp, ks, wq, wk, pp, gt, _ptr(dq_out),
                                      _ptr(dk_out), _ptr(dq), dqs, _ptr(dk), dks, _ptr(dwq), _ptr(dwk), st)
    if rc:
        h.check(rc)
    return dq, dk, dwq, dwk


def attn_backward(h: Handle, q, k, v, o, lse, d_o, *, Hk, scale=None, kv_begin=0, kv_end=None, kv_rows=None,
                  kv_rows_per_head=False, q_pos=None, key_pos0=0, k_row_bytes=None, v_row_bytes=None, d_lse=None,
                  need_dq=True, need_dkv=True, g_dtype=None, dq=None, dk=None, dv=None, stream=None):
    """skv_attn_backward: (dq, dk, dv) of attn_partial over fp16 rows, from its o, lse and their gradients d_o (fp16
    or fp32) and d_lse.  Results are fp32 unless g_dtype (or a given result) is torch.float16; need_dq=False or
    need_dkv=False leaves a part out (None).  Products take fp16 operands whatever the types: results are good to about
    11 bits in fp32 too, of small calls to about 14 (the header says which, and what small gradients beside large ones lose)."""
    torch = _torch()
    shape, dev, f16, f32 = q.shape, q.get_device(), torch.float16, torch.float32
    if len(shape) != 4:
        raise SplitKVError(1, f"q: want fp16 [S, nq, H, D], got {list(shape)}")
    S, nq, H, D = shape
    st = _q8_stream(h, stream, dev)
    d_type, rows3 = d_o.dtype, shape[:3]
    # all checks in one expression; what fails is found again below, with its message
    if not (q.dtype is f16 and o.dtype is f32 and lse.dtype is f32 and (d_type is f16 or d_type is f32) and k.dtype is f16
            and v.dtype is f16 and o.shape == shape and d_o.shape == shape and lse.shape == rows3 and o.get_device() == dev
            and lse.get_device() == dev and d_o.get_device() == dev and k.get_device() == dev and v.get_device() == dev
            and q.is_contiguous() and o.is_contiguous() and lse.is_contiguous() and d_o.is_contiguous()
            and (k_row_bytes is not None or k.is_contiguous()) and (v_row_bytes is not None or v.is_contiguous())):
        if d_type not in (f16, f32):
            raise SplitKVError(1, f"d_o: fp16 or fp32 is wanted, got {d_type}")
        for name, x, t, want in (("q", q, f16, shape), ("o", o, f32, shape), ("lse", lse, f32, rows3), ("d_o", d_o, d_type, shape)):
            _need(name, x, t, want, dev)
        for name, x in (("k", k), ("v", v)):
            if x.dtype is not f16 or x.get_device() != dev:
                raise SplitKVError(1, f"{name}: want fp16 rows on device {dev}, got {x.dtype} on {x.device}")
        raise SplitKVError(1, "k or v: rows that are not contiguous need k_row_bytes and v_row_bytes")
    if d_lse is not None:
        _need("d_lse", d_lse, f32, rows3, dev)
    if q_pos is not None:
        _need("q_pos", q_pos, torch.int32, (S, nq), dev)
    Hk, per_head, rows_ld = int(Hk), bool(kv_rows_per_head), 0
    if kv_rows is not None:
        rows_ld = kv_rows.shape[-1]
        _need("kv_rows", kv_rows, torch.int32, (S, Hk, rows_ld) if per_head else (S, rows_ld), dev)
    if kv_end is None:
        if kv_rows is None and k.shape[0] != v.shape[0]:
            raise SplitKVError(1, f"k has {k.shape[0]} rows, v {v.shape[0]}, and no kv_end says how many are wanted")
        kv_end = rows_ld if kv_rows is not None else k.shape[0]
    kv_begin, kv_end = int(kv_begin), int(kv_end)
    n = max(0, kv_end - kv_begin)
    if kv_rows is None and (kv_end > k.shape[0] or kv_end > v.shape[0]):
        raise SplitKVError(1, f"kv_end {kv_end} lies beyond k's {k.shape[0]} or v's {v.shape[0]} rows")
    row = Hk * 2 * D
    if k_row_bytes is None and k.numel() != k.shape[0] * Hk * D or v_row_bytes is None and v.numel() != v.shape[0] * Hk * D:
        raise SplitKVError(1, f"k {list(k.shape)} or v {list(v.shape)}: rows of {Hk} heads of {D} are wanted")
    if kv_rows is None and n:
        for name, x, step in (("k", k, k_row_bytes), ("v", v, v_row_bytes)):
            if step is not None and (kv_end - 1) * step + row > x.untyped_storage().nbytes() - 2 * x.storage_offset():
                raise SplitKVError(1, f"kv_end {kv_end} lies beyond {name}'s memory at {step} bytes a row")
    sh = SkvShape(S, nq, H, Hk, D, 1.0 / math.sqrt(D) if scale is None else float(scale), F16, F16,
                  row if k_row_bytes is None else int(k_row_bytes), row if v_row_bytes is None else int(v_row_bytes))
    if g_dtype is None:
        g_dtype = next((x.dtype for x in (dq, dk, dv) if x is not None), f32)
    if g_dtype is not f16 and g_dtype is not f32:
        raise SplitKVError(1, f"g_dtype: fp32 or fp16 is wanted, got {g_dtype}")
    kv_shape = (n, Hk, D) if kv_rows is None else (S, n, Hk, D)

    def result(name, x, want, need):
        if not need:
            return None
        if x is None:
            return _new(torch, want, g_dtype, q, stream, dev)
        _need(name, x, g_dtype, want, dev)
        return x

    outs = (result("dq", dq, shape, need_dq), result("dk", dk, kv_shape, need_dkv), result("dv", dv, kv_shape, need_dkv))
    rc = _lib.lib().skv_attn_backward(h._h, ctypes.byref(sh), q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(q_pos),
                                      int(key_pos0), _ptr(kv_rows), rows_ld, int(per_head), kv_begin, kv_end,
                                      o.data_ptr(), lse.data_ptr(), F16 if d_type is f16 else F32,
                                      d_o.data_ptr(), _ptr(d_lse), F16 if g_dtype is f16 else F32,
                                      _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), st)
    if rc:
        h.check(rc)
    return outs
