"""B200 (sm_100a) head-wise sparse attention layer: Python binding of librtp.

The functions below keep the C names of include/rtp.h and only marshal
arguments (torch tensors -> device pointers, the current CUDA stream); every
step of the layer runs in the library's CUDA kernels.  There is no CPU
fallback: importing this package loads librtp.so or raises.

`Layer` is a convenience holder for one layer's configuration, cache and
scratch memory, all allocated with torch (PyTorch supplies memory and streams).
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _abi
from ._abi import (EXPORTS, RTP_BF16, RTP_DEV_POSITION, RTP_DEV_SEQ_LEN, RTP_DEV_TIMEOUT, RTP_FP32,
                   RTP_DEV_BLOCKS, RTP_NOALLOC_SCRATCH_BYTES, STAGES, RtpError, rtp_cache, rtp_layer_cfg,
                   rtp_q8_cache, rtp_rope_axes)

_lib = _abi.load()

__all__ = ["Layer", "RtpError", "rtp_layer_cfg", "rtp_cache", "rtp_cache_bytes",
           "rtp_decode_workspace_bytes", "rtp_prefill_workspace_bytes", "rtp_append_kv",
           "rtp_decode_attn", "rtp_decode_attn_noalloc", "rtp_decode_recall", "rtp_prefill_attn",
           "rtp_trace_stage",
           "rtp_debug_wait_expiry",
           "rtp_last_error", "RTP_NOALLOC_SCRATCH_BYTES",
           "rtp_version", "make_cfg", "STAGES",
           "library_path", "EXPORTS", "RTP_BF16", "RTP_FP32", "RTP_DEV_SEQ_LEN",
           "RTP_DEV_POSITION", "RTP_DEV_TIMEOUT", "RTP_DEV_BLOCKS",
           "PagedLayer", "rtp_q8_cache", "rtp_rope_axes", "make_q8_cache", "make_rope", "rtp_q8_cache_bytes",
           "rtp_page_plan", "rtp_append_q8", "rtp_attn_q8_workspace_bytes", "rtp_attn_q8"]


def library_path() -> str:
    return _abi.LIB_PATH


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, torch.Tensor):
        if not x.is_cuda:
            raise ValueError("expected a CUDA tensor")
        if not x.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)} as a device pointer")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def make_cfg(batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, max_ctx: int,
             n_sink: int, window: int, top_p: float, retrieval: Sequence[int],
             dtype: str = "bf16", rope_base: float = 10000.0, idx_dim: int = 16,
             local_cap: int = 0, top_k: int = 0) -> rtp_layer_cfg:
    mask = 0
    for h in retrieval:
        mask |= 1 << int(h)
    return rtp_layer_cfg(batch, n_q_heads, n_kv_heads, head_dim, idx_dim, max_ctx, n_sink, window,
                         top_p, rope_base, mask, RTP_BF16 if dtype == "bf16" else RTP_FP32,
                         int(local_cap), int(top_k))


def rtp_version() -> str:
    return _lib.rtp_version().decode()


def rtp_last_error() -> str:
    return _lib.rtp_last_error().decode()


def rtp_trace_stage(stage, start_event=None, stop_event=None) -> None:
    """Arm CUDA events (torch.cuda.Event with timing) around the next launch of a stage."""
    sid = STAGES[stage] if isinstance(stage, str) else int(stage)
    handles = []
    for ev in (start_event, stop_event):
        if ev is None:
            handles.append(None)
            continue
        if not ev.cuda_event:  # torch creates its events lazily, at the first record
            ev.record()
        handles.append(ev.cuda_event)
    _abi.check(_lib.rtp_trace_stage(sid, handles[0], handles[1]))


def rtp_debug_wait_expiry(polls: int) -> None:
    """Arm the next rtp_decode_attn call on this thread to let its bounded waits expire."""
    _abi.check(_lib.rtp_debug_wait_expiry(int(polls)))


def rtp_cache_bytes(cfg: rtp_layer_cfg):
    k, v, ki = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _abi.check(_lib.rtp_cache_bytes(ctypes.byref(cfg), ctypes.byref(k), ctypes.byref(v), ctypes.byref(ki)))
    return k.value, v.value, ki.value


def rtp_decode_workspace_bytes(cfg: rtp_layer_cfg) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib.rtp_decode_workspace_bytes(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def rtp_prefill_workspace_bytes(cfg: rtp_layer_cfg, T: int) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib.rtp_prefill_workspace_bytes(ctypes.byref(cfg), int(T), ctypes.byref(n)))
    return n.value


def rtp_append_kv(cfg, cache, k_pre, v_in, start_pos, T, w_k, stream=None) -> None:
    _abi.check(_lib.rtp_append_kv(ctypes.byref(cfg), ctypes.byref(cache), _ptr(k_pre), _ptr(v_in),
                                  _ptr(start_pos), int(T), _ptr(w_k), _stream(stream)))


def rtp_decode_attn(cfg, cache, q_pre, seq_len, max_seq_len, w_q, out, sel_bitmask=None,
                    sel_count=None, workspace=None, workspace_bytes=0, stream=None) -> None:
    _abi.check(_lib.rtp_decode_attn(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q_pre),
                                    _ptr(seq_len), int(max_seq_len), _ptr(w_q), _ptr(out),
                                    _ptr(sel_bitmask), _ptr(sel_count), _ptr(workspace),
                                    int(workspace_bytes), _stream(stream)))


def rtp_decode_attn_noalloc(cfg, cache, q_pre, seq_len, max_seq_len, w_q, out, sel_bitmask=None,
                            sel_count=None, stream=None) -> None:
    """rtp_decode_attn with the library's fixed device scratch instead of a workspace."""
    _abi.check(_lib.rtp_decode_attn_noalloc(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q_pre),
                                            _ptr(seq_len), int(max_seq_len), _ptr(w_q), _ptr(out),
                                            _ptr(sel_bitmask), _ptr(sel_count), _stream(stream)))


def rtp_decode_recall(cfg, cache, q_pre, seq_len, max_seq_len, sel_bitmask, recall, workspace=None,
                      workspace_bytes=0, stream=None) -> None:
    _abi.check(_lib.rtp_decode_recall(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q_pre),
                                      _ptr(seq_len), int(max_seq_len), _ptr(sel_bitmask), _ptr(recall),
                                      _ptr(workspace), int(workspace_bytes), _stream(stream)))


def rtp_prefill_attn(cfg, cache, q_pre, start_pos, T, w_q, out, sel_bitmask=None, sel_tau=None,
                     sel_jcut=None, sel_count=None, workspace=None, workspace_bytes=0,
                     stream=None) -> None:
    _abi.check(_lib.rtp_prefill_attn(ctypes.byref(cfg), ctypes.byref(cache), _ptr(q_pre),
                                     _ptr(start_pos), int(T), _ptr(w_q), _ptr(out),
                                     _ptr(sel_bitmask), _ptr(sel_tau), _ptr(sel_jcut),
                                     _ptr(sel_count), _ptr(workspace), int(workspace_bytes),
                                     _stream(stream)))


def make_q8_cache(k, v, k_scale, v_scale, status) -> rtp_q8_cache:
    """Describe a pool of blocks: k, v [n_blocks, Hkv, block_size, D] (float8_e4m3fn or
    uint8), scales [n_blocks, Hkv] fp32, status one int32, all on one device.  It
    holds addresses only (keep the tensors alive), and the pool's heads, head_dim
    and device, which rtp_append_q8 and rtp_attn_q8 hold against the call's."""
    if v.shape != k.shape or k.dim() != 4 or k.element_size() != 1 or v.element_size() != 1:
        raise ValueError("k and v must be [n_blocks, Hkv, block_size, D] of one byte an element")
    if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2] or k_scale.dtype != torch.float32 \
            or v_scale.dtype != torch.float32:
        raise ValueError("k_scale and v_scale must be [n_blocks, Hkv] float32")
    if status.dtype != torch.int32 or status.numel() != 1:
        raise ValueError("status must be one int32")
    if any(x.device != k.device for x in (v, k_scale, v_scale, status)):
        raise ValueError("k, v, k_scale, v_scale and status must be on one device")
    cache = rtp_q8_cache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(status), k.shape[0], k.shape[2])
    cache.made_for = (k.shape[1], k.shape[3], k.get_device())
    return cache


def make_rope(head_dim: int, sections: Sequence[int], interleaved: bool = False) -> rtp_rope_axes:
    """Rotary axes: axis a turns sections[a] of the head_dim / 2 rotary pairs.
    The axes' pairs follow one another, or, interleaved, are dealt out in turn
    (axis 0, 1, 2, 0, ...) until an axis has its number."""
    left = [int(s) for s in sections]
    if sum(left) != head_dim // 2 or min(left) < 0 or not 1 <= len(left) <= 4:
        raise ValueError("one to four sections that sum to head_dim / 2")
    r = rtp_rope_axes(len(left))
    if interleaved:
        k = 0
        while k < head_dim // 2:
            for a in range(len(left)):
                if left[a] > 0:
                    r.axis[k] = a
                    left[a] -= 1
                    k += 1
    else:
        r.axis[:head_dim // 2] = [a for a, s in enumerate(left) for _ in range(s)]
    return r


def rtp_q8_cache_bytes(cfg: rtp_layer_cfg, n_blocks: int, block_size: int):
    kv, sc = ctypes.c_size_t(), ctypes.c_size_t()
    _abi.check(_lib.rtp_q8_cache_bytes(ctypes.byref(cfg), int(n_blocks), int(block_size), ctypes.byref(kv),
                                       ctypes.byref(sc)))
    return kv.value, sc.value


def _arg(x, dtype, name, dev, n=-1) -> int:
    """Address of a dense tensor whose element type, device and number of elements the call fixes.
    Kernels run on the current device `dev`: a tensor of another one is refused."""
    if x.dtype is not dtype or x.get_device() != dev or not x.is_contiguous() or (n >= 0 and x.numel() != n):
        _refuse(x, dtype, name, dev, n)
    return x.data_ptr()


def _refuse(x, dtype, name, dev, n) -> None:
    if x.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, not on the current CUDA device")
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError(f"{name} must have {n} elements")


def _packed(x, D: int, dt, heads: int, name, dev):
    """(address, elements between tokens) of packed [N, heads, D] rows of dt, dense or a slice of wider rows."""
    shape = x.shape
    if x.dtype is not dt or len(shape) != 3 or shape[1] != heads or shape[2] != D:
        raise ValueError(f"{name} must be a CUDA [N, {heads}, {D}] tensor of {dt}")
    if x.get_device() != dev:
        _refuse(x, dt, name, dev, -1)
    s0, s1, s2 = x.stride()
    if (s2 != 1 or s1 != D) and shape[0] > 0:
        raise ValueError(f"{name}: a token's heads must be dense")
    if shape[0] > 1 and s0 < heads * D:  # (0, a broadcast, would reach the library as "dense")
        raise ValueError(f"{name}: tokens must not overlap")
    return x.data_ptr(), s0 if shape[0] > 1 else 0


def _check_pool(cache, heads: int, D: int, dev) -> None:
    """The call's heads, head_dim and device are the pool's (a description made of bare addresses has none to hold)."""
    if cache.made_for is not None and cache.made_for != (heads, D, dev):
        raise ValueError(f"the pool has (n_kv_heads, head_dim, CUDA device) {cache.made_for}, the call {(heads, D, dev)}")


def _device(x, name) -> int:
    """The device of a call's first tensor, which has to be the current one."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {x.device}, not on the current CUDA device")
    return dev


def _table_cols(cfg, block_size) -> int:
    """Entries of a block table's row (none for a block size that the library refuses)."""
    return -(-cfg.max_ctx // block_size) if block_size > 0 else 0


def _raw_stream(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def rtp_page_plan(cfg, block_size, ctx_len, new_len, block_table, free_list, n_free, seq_len, cu_new,
                  slot_map, positions, n_free_out, status, stream=None) -> None:
    i32, dev, B = torch.int32, _device(ctx_len, "ctx_len"), cfg.batch
    cols = _table_cols(cfg, block_size)
    n = slot_map.numel()
    rc = _lib.rtp_page_plan(cfg, block_size, _arg(ctx_len, i32, "ctx_len", dev, B), _arg(new_len, i32, "new_len", dev, B),
                            _arg(block_table, i32, "block_table", dev, B * cols), _arg(free_list, i32, "free_list", dev),
                            free_list.numel(), _arg(n_free, i32, "n_free", dev, 1), _arg(seq_len, i32, "seq_len", dev, B),
                            _arg(cu_new, i32, "cu_new", dev, B + 1), _arg(slot_map, torch.int64, "slot_map", dev),
                            _arg(positions, i32, "positions", dev, n), n, _arg(n_free_out, i32, "n_free_out", dev, 1),
                            _arg(status, i32, "status", dev, 1), _raw_stream(stream, dev))
    if rc:
        _abi.check(rc)


def rtp_append_q8(cfg, cache, k_pre, v_in, slot_map, pos, rope=None, stream=None) -> None:
    dev, n = _device(k_pre, "k_pre"), k_pre.shape[0]
    heads, D, dt = cfg.n_kv_heads, cfg.head_dim, torch.bfloat16 if cfg.dtype == RTP_BF16 else torch.float32
    _check_pool(cache, heads, D, dev)
    k, ks = _packed(k_pre, D, dt, heads, "k_pre", dev)
    v, vs = _packed(v_in, D, dt, heads, "v_in", dev)
    if v_in.shape[0] != n:
        raise ValueError("k_pre and v_in must have as many tokens")
    rc = _lib.rtp_append_q8(cfg, cache, k, ks, v, vs, _arg(slot_map, torch.int64, "slot_map", dev, n),
                            _arg(pos, torch.int32, "pos", dev, n * (rope.n_axes if rope is not None else 1)), rope, n,
                            _raw_stream(stream, dev))
    if rc:
        _abi.check(rc)


def rtp_attn_q8_workspace_bytes(cfg: rtp_layer_cfg, block_size: int, n_tokens: int, max_q: int,
                                max_seq_len: int = 0) -> int:
    n = ctypes.c_size_t()
    _abi.check(_lib.rtp_attn_q8_workspace_bytes(ctypes.byref(cfg), int(block_size), int(n_tokens), int(max_q),
                                                int(max_seq_len), ctypes.byref(n)))
    return n.value


def rtp_attn_q8(cfg, cache, q_pre, cu_q, seq_len, block_table, pos, out, max_q, max_seq_len=0, rope=None,
                workspace=None, workspace_bytes=0, stream=None) -> None:
    if workspace is None:
        raise ValueError("workspace is missing: rtp_attn_q8_workspace_bytes says how much")
    i32, dev, n, B = torch.int32, _device(q_pre, "q_pre"), q_pre.shape[0], cfg.batch
    D = cfg.head_dim
    _check_pool(cache, cfg.n_kv_heads, D, dev)
    q, qs = _packed(q_pre, D, torch.bfloat16 if cfg.dtype == RTP_BF16 else torch.float32, cfg.n_q_heads, "q_pre", dev)
    if out.shape != q_pre.shape:
        raise ValueError("out must have q_pre's shape")
    if workspace.numel() < workspace_bytes:
        raise ValueError("workspace_bytes is more than the workspace has")
    rc = _lib.rtp_attn_q8(cfg, cache, q, qs, _arg(cu_q, i32, "cu_q", dev, B + 1), _arg(seq_len, i32, "seq_len", dev, B),
                          _arg(block_table, i32, "block_table", dev, B * _table_cols(cfg, cache.block_size)),
                          _arg(pos, i32, "pos", dev, n * (rope.n_axes if rope is not None else 1)), rope, n, max_q,
                          max_seq_len, _arg(out, q_pre.dtype, "out", dev), _arg(workspace, torch.uint8, "workspace", dev),
                          workspace_bytes, _raw_stream(stream, dev))
    if rc:
        _abi.check(rc)


class _Memory:
    """Torch-allocated memory that is used on whatever streams its owner's calls
    name.  Torch orders a buffer's former and next users on the stream that was
    current when it was allocated; the other streams are seen to here."""

    def _settle(self, dev: int) -> None:
        """What the current stream still does to memory just allocated (its former
        user's work, its filling) is waited for, so that any stream may use it."""
        self._dev = dev
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()

    def _on(self, stream) -> int:
        """The handle of a call's stream; torch is told of streams that it has not
        seen, so that freed memory waits for them (not of streams made elsewhere,
        which may be gone by then: synchronise those before the owner goes)."""
        handle = _raw_stream(stream, self._dev)
        if handle not in self._streams:
            self._streams[handle] = None
            if not isinstance(stream, int):
                s = torch.cuda.current_stream(self._dev) if stream is None else stream
                if handle == 0 or s.stream_id != handle:  # (an outside stream's id is its handle)
                    self._streams[handle] = s
                    for t in self._tensors():
                        t.record_stream(s)
        return handle

    def _scratch(self, n: int, dev: int) -> torch.Tensor:
        t = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev))
        self._settle(dev)
        for s in self._streams.values():
            if s is not None:
                t.record_stream(s)
        return t


class PagedLayer(_Memory):
    """One layer's configuration with a pool of 8-bit blocks and scratch, all
    torch-allocated.  Requests' block tables come from rtp_page_plan and are
    shared by a model's layers; pass the step's to append() and attend().
    attend() calls share one scratch, so they must not overlap each other;
    layers that run side by side, and graphs replayed side by side, take an
    object each.  Scratch that has to grow waits for the current stream: where
    that matters, and before a capture, reserve() the largest call's."""

    def __init__(self, shape, max_ctx: int, n_blocks: int, block_size: int = 64, device="cuda", rope=None):
        self.shape = shape
        self.cfg = make_cfg(shape.batch, shape.n_q_heads, shape.n_kv_heads, shape.head_dim, max_ctx, shape.n_sink,
                            shape.window, 1.0, shape.retrieval, shape.dtype, shape.rope_base, shape.idx_dim)
        rtp_q8_cache_bytes(self.cfg, n_blocks, block_size)  # refuses what the library does not take
        self.rope = rope
        size = (n_blocks, shape.n_kv_heads, block_size, shape.head_dim)
        self.k = torch.zeros(size, dtype=torch.float8_e4m3fn, device=device)
        self.v = torch.zeros(size, dtype=torch.float8_e4m3fn, device=device)
        self.k_scale = torch.ones(size[:2], dtype=torch.float32, device=device)
        self.v_scale = torch.ones(size[:2], dtype=torch.float32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.cache = make_q8_cache(self.k, self.v, self.k_scale, self.v_scale, self.status)
        self.ws = torch.empty(0, dtype=torch.uint8, device=device)
        self._outgrown = []  # scratch that a captured graph or another stream may still use
        self._streams = {}
        self._settle(self.k.get_device())

    def reserve(self, n_tokens: int, max_q: int, max_seq_len: int = 0) -> None:
        """Scratch for attend() calls of that size; call it before capturing one in a graph."""
        n = rtp_attn_q8_workspace_bytes(self.cfg, self.cache.block_size, n_tokens, max_q, max_seq_len)
        if n > self.ws.numel():
            if self.ws.numel():
                self._outgrown.append(self.ws)
            # at least twice the last, so that all outgrown ones together are no larger
            self.ws = self._scratch(max(n, 2 * self.ws.numel()), self._dev)

    def _tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale, self.status, self.ws

    def append(self, k_pre, v_in, slot_map, pos, stream=None) -> None:
        rtp_append_q8(self.cfg, self.cache, k_pre, v_in, slot_map, pos, self.rope, self._on(stream))

    def attend(self, q_pre, cu_q, seq_len, block_table, pos, out, max_q: int, max_seq_len: int = 0, stream=None) -> None:
        self.reserve(q_pre.shape[0], max_q, max_seq_len)
        rtp_attn_q8(self.cfg, self.cache, q_pre, cu_q, seq_len, block_table, pos, out, max_q, max_seq_len, self.rope,
                    self.ws, self.ws.numel(), self._on(stream))

    def device_status(self) -> int:
        return int(self.status.item())


class Layer(_Memory):
    """One layer's configuration plus its device cache and scratch (torch-allocated).
    Calls that share scratch must not overlap; prefill scratch that has to grow
    waits for the current stream (reserve_prefill() the longest chunk's).

    local_cap > 0 selects ring mode: local heads keep only their sinks and a
    ring of local_cap window rows.  k and v are then flat [B, rows, D] buffers
    (head_rows() gives each head's slice); otherwise [B, Hkv, max_ctx, D]."""

    def __init__(self, shape, max_ctx: int, device="cuda", prefill_T: int = 0, local_cap: int = 0):
        self.shape = shape
        self.cfg = make_cfg(shape.batch, shape.n_q_heads, shape.n_kv_heads, shape.head_dim, max_ctx,
                            shape.n_sink, shape.window, shape.top_p, shape.retrieval, shape.dtype,
                            shape.rope_base, shape.idx_dim, local_cap, getattr(shape, "top_k", 0))
        self.max_ctx = max_ctx
        dt = torch.bfloat16 if shape.dtype == "bf16" else torch.float32
        B, Hkv, D, R = shape.batch, shape.n_kv_heads, shape.head_dim, shape.n_retrieval
        es = 2 if shape.dtype == "bf16" else 4
        k_bytes, _, _ = rtp_cache_bytes(self.cfg)
        rows = k_bytes // (B * D * es)
        self.ring = rows != Hkv * max_ctx
        if self.ring:
            self.k = torch.empty((B, rows, D), dtype=dt, device=device)
        else:
            self.k = torch.empty((B, Hkv, max_ctx, D), dtype=dt, device=device)
        self.v = torch.empty_like(self.k)
        # indexer keys [B, R, Lk, d] (Lk = max_ctx, or max_ctx rounded up to even
        # for 8-byte bf16 d = 4 rows); kidx views the first max_ctx rows of each block
        d = shape.idx_dim
        _, _, ki_bytes = rtp_cache_bytes(self.cfg)
        Lk = ki_bytes // (B * max(R, 1) * d * es) if R > 0 else max_ctx
        self.kidx_full = torch.empty((B, max(R, 1), Lk, d), dtype=dt, device=device)
        self.kidx = self.kidx_full[:, :, :max_ctx]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.cache = rtp_cache(self.k.data_ptr(), self.v.data_ptr(), self.kidx_full.data_ptr(),
                               self.status.data_ptr())
        self.ws_decode_bytes = rtp_decode_workspace_bytes(self.cfg)
        self.ws_decode = torch.empty(self.ws_decode_bytes, dtype=torch.uint8, device=device)
        self.ws_prefill = None
        self.ws_prefill_bytes = 0
        self._outgrown = []  # prefill scratch that a captured graph or another stream may still use
        self._streams = {}
        self._settle(self.k.get_device())
        if prefill_T:
            self.reserve_prefill(prefill_T)

    def reserve_prefill(self, T: int) -> None:
        n = rtp_prefill_workspace_bytes(self.cfg, T)
        if n > self.ws_prefill_bytes:
            if self.ws_prefill is not None:
                self._outgrown.append(self.ws_prefill)
                # twice the last, up to the GiB that chunks need at most: so outgrown ones stay few
                n = max(n, min(2 * self.ws_prefill_bytes, 1 << 30))
            self.ws_prefill_bytes = n
            self.ws_prefill = self._scratch(n, self._dev)

    def _tensors(self):
        t = (self.k, self.v, self.kidx_full, self.status, self.ws_decode)
        return t if self.ws_prefill is None else t + (self.ws_prefill,)

    def append(self, k_pre, v_in, start_pos, w_k, stream=None) -> None:
        rtp_append_kv(self.cfg, self.cache, k_pre, v_in, start_pos, k_pre.shape[1], w_k, self._on(stream))

    def decode(self, q_pre, seq_len, w_q, out, max_seq_len: int = 0, sel_bitmask=None,
               sel_count=None, stream=None) -> None:
        rtp_decode_attn(self.cfg, self.cache, q_pre, seq_len, max_seq_len, w_q, out, sel_bitmask,
                        sel_count, self.ws_decode, self.ws_decode_bytes, self._on(stream))

    def recall(self, q_pre, seq_len, sel_bitmask, recall, max_seq_len: int = 0, stream=None) -> None:
        rtp_decode_recall(self.cfg, self.cache, q_pre, seq_len, max_seq_len, sel_bitmask, recall,
                          self.ws_decode, self.ws_decode_bytes, self._on(stream))

    def prefill(self, q_pre, start_pos, w_q, out, sel_bitmask=None, sel_tau=None, sel_jcut=None,
                sel_count=None, stream=None) -> None:
        T = q_pre.shape[1]
        self.reserve_prefill(T)
        rtp_prefill_attn(self.cfg, self.cache, q_pre, start_pos, T, w_q, out, sel_bitmask, sel_tau,
                         sel_jcut, sel_count, self.ws_prefill, self.ws_prefill_bytes, self._on(stream))

    def device_status(self) -> int:
        return int(self.status.item())
