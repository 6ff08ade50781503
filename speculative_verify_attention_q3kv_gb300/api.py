"""Thin Python layer over the C ABI: torch tensors in, raw pointers out.

Argument marshalling only -- every step of the hot path runs in the CUDA
library.  Names follow ``include/q3kv.h``.  Device buffers are torch tensors the
caller owns; the library never allocates device memory.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import numpy as np
import torch

from . import _lib
from ._lib import CacheDesc, Q3KVError, RopePlan, check  # noqa: F401  (re-exported)

HEAD_DIM = 256
PAGE_SIZE = 256
GROUP = 8


def make_desc(num_layers: int, num_kv_heads: int, num_pages: int) -> CacheDesc:
    return CacheDesc(num_layers, num_kv_heads, GROUP * num_kv_heads, HEAD_DIM, PAGE_SIZE, num_pages)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to q3kv must be contiguous")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return _lib.Q3KV_BF16
    if dtype is torch.float32:
        return _lib.Q3KV_F32
    raise TypeError(f"q3kv inputs must be float32 or bfloat16, got {t.dtype}")


def _on_gpu(name: str, t: Optional[torch.Tensor], dev: int, dtype=None, min_numel: int = 0,
            optional: bool = False) -> None:
    """Refuse, before any launch, a tensor the kernels could not address safely.

    The C ABI takes raw device pointers; a host tensor, a tensor on another
    device, a wrong element type or a buffer shorter than the call's counts
    would be read or written out of bounds on the GPU.  Values inside device
    arrays (lengths, offsets, page ids) are checked by the kernels.
    """
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    idx = _device_index(t)
    if idx < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if idx != dev:
        raise ValueError(f"{name} is on cuda:{idx}, the current device is cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs at least {min_numel}")


# CUDA device index of a tensor; -1 for a tensor in host memory
_device_index = torch.Tensor.get_device

_cuda_seen = False                # asking torch whether CUDA is there costs microseconds; a yes stays a yes


def _current_device() -> int:
    """The current CUDA device; -2, which no tensor is on, where there is none."""
    global _cuda_seen
    if not _cuda_seen:
        if not torch.cuda.is_available():
            return -2
        torch.cuda.init()
        _cuda_seen = True
    return torch._C._cuda_getDevice()


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _check_cache_args(desc: CacheDesc, pool: torch.Tensor, need_pool_bytes: int, page_table: torch.Tensor,
                      lens: torch.Tensor, counts: torch.Tensor, offsets: torch.Tensor,
                      status: Optional[torch.Tensor], dev: int) -> int:
    """Common checks of the append / verify / prefill calls; returns num_slots."""
    _on_gpu("pool", pool, dev)
    if _nbytes(pool) < need_pool_bytes:
        raise ValueError(f"pool holds {_nbytes(pool)} bytes, the cache needs {need_pool_bytes}")
    _on_gpu("lengths", lens, dev, torch.int32)
    if lens.dim() != 1:
        raise ValueError("per-slot lengths must be one-dimensional")
    n = lens.shape[0]
    _on_gpu("page_table", page_table, dev, torch.int32)
    if page_table.dim() != 2 or page_table.shape[1] < 1 or (n > 0 and page_table.shape[0] < n):
        raise ValueError(f"page_table must be int32 [num_slots >= {n}, max_pages_per_slot >= 1], "
                         f"got {tuple(page_table.shape)}")
    _on_gpu("per-slot token counts", counts, dev, torch.int32, n)
    _on_gpu("row offsets", offsets, dev, torch.int32, n)
    _on_gpu("status", status, dev, torch.int32, 1, optional=True)
    return n


def _check_rows(name: str, t: torch.Tensor, heads: int, dev: int) -> None:
    _on_gpu(name, t, dev)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must be [rows, {heads}, {HEAD_DIM}], got {tuple(t.shape)}")


def _check_append(desc, pool, pool_bytes_fn, page_table, slot_len, n_new, row_offsets, k, v, status) -> None:
    dev = _current_device()
    _check_cache_args(desc, pool, pool_bytes_fn(desc), page_table, slot_len, n_new, row_offsets, status, dev)
    if k.dtype != v.dtype:
        raise TypeError("k and v must share a dtype")
    _check_rows("k", k, desc.num_kv_heads, dev)
    _check_rows("v", v, desc.num_kv_heads, dev)
    if k.shape != v.shape:
        raise ValueError(f"k and v differ in shape: {tuple(k.shape)} vs {tuple(v.shape)}")


def _check_verify(desc, pool, pool_bytes_fn, page_table, ctx_len, n_q, q_offsets, q, out, workspace,
                  status) -> None:
    dev = _current_device()
    _check_cache_args(desc, pool, pool_bytes_fn(desc), page_table, ctx_len, n_q, q_offsets, status, dev)
    _check_rows("q", q, desc.num_q_heads, dev)
    if out.dtype != torch.float32:
        raise TypeError("out must be float32")
    _check_rows("out", out, desc.num_q_heads, dev)
    if out.shape[0] < q.shape[0]:
        raise ValueError(f"out has {out.shape[0]} rows, q has {q.shape[0]}")
    _on_gpu("workspace", workspace, dev, optional=True)


def _pointers(dev: int, *args):
    """Checks of several tensors in one pass (a call of a step costs microseconds): for every (name, tensor, dtype or
    None, elements needed) what _on_gpu and _ptr check, and the data pointers.  A tensor of None gives None."""
    out = []
    index, tensor = _device_index, torch.Tensor
    for name, t, dtype, need in args:
        if t is None:
            out.append(None)
            continue
        if not isinstance(t, tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if index(t) != dev or (t.dtype is not dtype and dtype is not None) or (need and t.numel() < need):
            _on_gpu(name, t, dev, dtype, need)
        if not t.is_contiguous():
            raise ValueError("tensors passed to q3kv must be contiguous")
        out.append(t.data_ptr())
    return out


def _cache_pointers(desc: CacheDesc, pool, need_pool_bytes: int, page_table, lens, counts, offsets, status, dev: int,
                    names=("per-slot token counts", "row offsets")):
    """_check_cache_args with the pointers: (num_slots, max_pages_per_slot, [pool, page_table, lens, counts, offsets, status])."""
    if pool is None or page_table is None or lens is None or counts is None or offsets is None:
        _required(**{"pool": pool, "page_table": page_table, "lengths": lens, names[0]: counts, names[1]: offsets})
    if lens.dim() != 1:
        raise ValueError("per-slot lengths must be one-dimensional")
    n = lens.numel()
    ptrs = _pointers(dev, ("pool", pool, None, 0), ("page_table", page_table, torch.int32, 0), ("lengths", lens, torch.int32, 0),
                     (names[0], counts, torch.int32, n), (names[1], offsets, torch.int32, n), ("status", status, torch.int32, 1))
    shape = page_table.shape
    if len(shape) != 2 or shape[1] < 1 or (n > 0 and shape[0] < n):
        raise ValueError(f"page_table must be int32 [num_slots >= {n}, max_pages_per_slot >= 1], "
                         f"got {tuple(shape)}")
    if _nbytes(pool) < need_pool_bytes:
        raise ValueError(f"pool holds {_nbytes(pool)} bytes, the cache needs {need_pool_bytes}")
    return n, shape[1], ptrs


@functools.lru_cache(maxsize=64)
def _pool_need(pool_bytes_fn, lib, desc_bytes: bytes) -> int:
    """The pool size that a format's function and the library `lib` give for a CacheDesc with these bytes."""
    return pool_bytes_fn(CacheDesc.from_buffer_copy(desc_bytes))


def _required(**tensors) -> None:
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def pool_bytes(desc: CacheDesc) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_pool_bytes(ctypes.byref(desc), ctypes.byref(n)), "q3kv_pool_bytes")
    return n.value


def workspace_bytes(desc: CacheDesc, num_slots: int, max_ctx_len: int, max_n_q: int,
                    impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_workspace_bytes(ctypes.byref(desc), num_slots, max_ctx_len, max_n_q, impl,
                                           split_positions, ctypes.byref(n)), "q3kv_workspace_bytes")
    return n.value


class Allocator:
    """Host free-list page allocator (q3kv_allocator_*)."""

    def __init__(self, num_pages: int, num_slots: int, max_pages_per_slot: int):
        self._lib = _lib.load()
        h = ctypes.c_void_p()
        check(self._lib.q3kv_allocator_create(num_pages, num_slots, max_pages_per_slot, ctypes.byref(h)),
              "q3kv_allocator_create")
        self._h = h
        self.max_pages_per_slot = max_pages_per_slot

    def alloc_pages(self, slot: int, n_positions: int) -> np.ndarray:
        row = np.full(self.max_pages_per_slot, -1, dtype=np.int32)
        n = ctypes.c_int32()
        check(self._lib.q3kv_alloc_pages(self._h, slot, n_positions,
                                         row.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ctypes.byref(n)),
              "q3kv_alloc_pages")
        return row

    def free_slot(self, slot: int) -> None:
        check(self._lib.q3kv_free_slot(self._h, slot), "q3kv_free_slot")

    def free_pages(self) -> int:
        n = ctypes.c_int32()
        check(self._lib.q3kv_free_pages(self._h, ctypes.byref(n)), "q3kv_free_pages")
        return n.value

    def close(self) -> None:
        if self._h:
            self._lib.q3kv_allocator_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def append(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, slot_len: torch.Tensor,
           n_new: torch.Tensor, row_offsets: torch.Tensor, max_n_new: int, layer: int,
           k: torch.Tensor, v: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_append: quantise and store k, v [rows, kv_heads, 256] for each slot."""
    _check_append(desc, pool, pool_bytes, page_table, slot_len, n_new, row_offsets, k, v, status)
    rc = _lib.load().q3kv_append(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                 page_table.shape[1], _ptr(slot_len), _ptr(n_new), _ptr(row_offsets),
                                 slot_len.shape[0], max_n_new, layer, _ptr(k), _ptr(v), _dtype_code(k),
                                 _ptr(status))
    check(rc, "q3kv_append")


def verify_attn(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_verify_attn: out[rows, q_heads, 256] (float32) for every slot's query tokens."""
    _check_verify(desc, pool, pool_bytes, page_table, ctx_len, n_q, q_offsets, q, out, workspace, status)
    rc = _lib.load().q3kv_verify_attn(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                      page_table.shape[1], _ptr(ctx_len), _ptr(n_q), _ptr(q_offsets),
                                      ctx_len.shape[0], max_ctx_len, max_n_q, layer, _ptr(q), _dtype_code(q),
                                      _ptr(out), impl, split_positions, _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _ptr(status))
    check(rc, "q3kv_verify_attn")


def verify_attn_noalloc(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                        n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                        q: torch.Tensor, out: torch.Tensor, impl: int = _lib.Q3KV_IMPL_AUTO,
                        split_positions: int = 0, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_verify_attn_noalloc: verify_attn with the library's fixed scratch instead of a workspace.

    For callers that cannot provide device scratch memory; calls that overlap
    on the GPU share that scratch and must not run concurrently.
    """
    _check_verify(desc, pool, pool_bytes, page_table, ctx_len, n_q, q_offsets, q, out, None, status)
    rc = _lib.load().q3kv_verify_attn_noalloc(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                              page_table.shape[1], _ptr(ctx_len), _ptr(n_q), _ptr(q_offsets),
                                              ctx_len.shape[0], max_ctx_len, max_n_q, layer, _ptr(q),
                                              _dtype_code(q), _ptr(out), impl, split_positions, _ptr(status))
    check(rc, "q3kv_verify_attn_noalloc")


def prefill_workspace_bytes(desc: CacheDesc, num_slots: int, max_ctx_len: int, max_n_new: int,
                            impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_prefill_workspace_bytes(ctypes.byref(desc), num_slots, max_ctx_len, max_n_new, impl,
                                                   split_positions, ctypes.byref(n)), "q3kv_prefill_workspace_bytes")
    return n.value


def prefill_attn(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                 n_new: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_new: int, layer: int,
                 q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                 impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                 status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_prefill_attn: causal attention of up to 8192 appended tokens per slot over the 3-bit cache."""
    _check_verify(desc, pool, pool_bytes, page_table, ctx_len, n_new, q_offsets, q, out, workspace, status)
    rc = _lib.load().q3kv_prefill_attn(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                       page_table.shape[1], _ptr(ctx_len), _ptr(n_new), _ptr(q_offsets),
                                       ctx_len.shape[0], max_ctx_len, max_n_new, layer, _ptr(q), _dtype_code(q),
                                       _ptr(out), impl, split_positions, _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(status))
    check(rc, "q3kv_prefill_attn")


def t5k_pool_bytes(desc: CacheDesc) -> int:
    """q3kv_t5k_pool_bytes: bytes of a turbo5k-style pool (164-byte K, 112-byte V records)."""
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_t5k_pool_bytes(ctypes.byref(desc), ctypes.byref(n)), "q3kv_t5k_pool_bytes")
    return n.value


def t5k_append(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, slot_len: torch.Tensor,
               n_new: torch.Tensor, row_offsets: torch.Tensor, max_n_new: int, layer: int,
               k: torch.Tensor, v: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_t5k_append: 5-bit Lloyd-Max K and 3-bit V records for k, v [rows, kv_heads, 256]."""
    _check_append(desc, pool, t5k_pool_bytes, page_table, slot_len, n_new, row_offsets, k, v, status)
    rc = _lib.load().q3kv_t5k_append(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                     page_table.shape[1], _ptr(slot_len), _ptr(n_new), _ptr(row_offsets),
                                     slot_len.shape[0], max_n_new, layer, _ptr(k), _ptr(v), _dtype_code(k),
                                     _ptr(status))
    check(rc, "q3kv_t5k_append")


def t5k_verify_attn(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                    n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                    q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                    impl: int = _lib.Q3KV_IMPL_FMA, split_positions: int = 0,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_t5k_verify_attn: verify attention over the turbo5k-style cache (CUDA-core leg)."""
    _check_verify(desc, pool, t5k_pool_bytes, page_table, ctx_len, n_q, q_offsets, q, out, workspace, status)
    rc = _lib.load().q3kv_t5k_verify_attn(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                          page_table.shape[1], _ptr(ctx_len), _ptr(n_q), _ptr(q_offsets),
                                          ctx_len.shape[0], max_ctx_len, max_n_q, layer, _ptr(q), _dtype_code(q),
                                          _ptr(out), impl, split_positions, _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(status))
    check(rc, "q3kv_t5k_verify_attn")


def fp8_pool_bytes(desc: CacheDesc) -> int:
    """q3kv_fp8_pool_bytes: bytes of an fp8 E4M3 comparison pool (256-byte records)."""
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_fp8_pool_bytes(ctypes.byref(desc), ctypes.byref(n)), "q3kv_fp8_pool_bytes")
    return n.value


def fp8_append(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, slot_len: torch.Tensor,
               n_new: torch.Tensor, row_offsets: torch.Tensor, max_n_new: int, layer: int,
               k: torch.Tensor, v: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_fp8_append: store k, v [rows, kv_heads, 256] as E4M3 records (the comparison cache)."""
    _check_append(desc, pool, fp8_pool_bytes, page_table, slot_len, n_new, row_offsets, k, v, status)
    rc = _lib.load().q3kv_fp8_append(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                     page_table.shape[1], _ptr(slot_len), _ptr(n_new), _ptr(row_offsets),
                                     slot_len.shape[0], max_n_new, layer, _ptr(k), _ptr(v), _dtype_code(k),
                                     _ptr(status))
    check(rc, "q3kv_fp8_append")


def fp8_verify_attn(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                    n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                    q: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                    impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_fp8_verify_attn: verify attention over the fp8 comparison cache (tensor-core leg)."""
    _check_verify(desc, pool, fp8_pool_bytes, page_table, ctx_len, n_q, q_offsets, q, out, workspace, status)
    rc = _lib.load().q3kv_fp8_verify_attn(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                          page_table.shape[1], _ptr(ctx_len), _ptr(n_q), _ptr(q_offsets),
                                          ctx_len.shape[0], max_ctx_len, max_n_q, layer, _ptr(q), _dtype_code(q),
                                          _ptr(out), impl, split_positions, _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(status))
    check(rc, "q3kv_fp8_verify_attn")


def _check_accept(logits, q_offsets, n_q, tokens, ctx_len, n_accepted, next_token, committed_len, workspace,
                  status):
    """Checks common to the acceptance calls; returns (rows, vocab) of the logits."""
    dev = _current_device()
    _on_gpu("logits", logits, dev)
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, vocab], got {tuple(logits.shape)}")
    _dtype_code(logits)
    rows, vocab = logits.shape
    _on_gpu("n_q", n_q, dev, torch.int32)
    if n_q.dim() != 1:
        raise ValueError("n_q must be one-dimensional")
    n = n_q.shape[0]
    for name, t in (("q_offsets", q_offsets), ("ctx_len", ctx_len), ("n_accepted", n_accepted),
                    ("next_token", next_token), ("committed_len", committed_len)):
        _on_gpu(name, t, dev, torch.int32, n)
    _on_gpu("tokens", tokens, dev, torch.int32, rows)
    _on_gpu("workspace", workspace, dev, optional=True)
    _on_gpu("status", status, dev, torch.int32, 1, optional=True)
    return rows, vocab


def accept_workspace_bytes(num_rows: int, vocab: int) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_accept_workspace_bytes(num_rows, vocab, ctypes.byref(n)), "q3kv_accept_workspace_bytes")
    return n.value


def accept_greedy(logits: torch.Tensor, q_offsets: torch.Tensor, n_q: torch.Tensor, tokens: torch.Tensor,
                  max_n_q: int, ctx_len: torch.Tensor, n_accepted: torch.Tensor, next_token: torch.Tensor,
                  committed_len: torch.Tensor, workspace: Optional[torch.Tensor],
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_accept_greedy: logits [rows, vocab] (f32 or bf16); int32 per-slot outputs."""
    rows, vocab = _check_accept(logits, q_offsets, n_q, tokens, ctx_len, n_accepted, next_token, committed_len,
                                workspace, status)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.load().q3kv_accept_greedy(_stream(stream), _ptr(logits), _dtype_code(logits), vocab, _ptr(q_offsets),
                                        _ptr(n_q), _ptr(tokens), n_q.shape[0], rows, max_n_q, _ptr(ctx_len),
                                        _ptr(n_accepted), _ptr(next_token), _ptr(committed_len), _ptr(workspace),
                                        nbytes, _ptr(status))
    check(rc, "q3kv_accept_greedy")


def accept_sample(logits: torch.Tensor, q_offsets: torch.Tensor, n_q: torch.Tensor, tokens: torch.Tensor,
                  max_n_q: int, ctx_len: torch.Tensor, temperature: float, uniforms: torch.Tensor, seed: int,
                  n_accepted: torch.Tensor, next_token: torch.Tensor, committed_len: torch.Tensor,
                  workspace: Optional[torch.Tensor], status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_accept_sample: rejection-sampled acceptance; uniforms float32 [rows]."""
    rows, vocab = _check_accept(logits, q_offsets, n_q, tokens, ctx_len, n_accepted, next_token, committed_len,
                                workspace, status)
    _on_gpu("uniforms", uniforms, _current_device(), torch.float32, rows)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.load().q3kv_accept_sample(_stream(stream), _ptr(logits), _dtype_code(logits), vocab, _ptr(q_offsets),
                                        _ptr(n_q), _ptr(tokens), n_q.shape[0], rows, max_n_q, _ptr(ctx_len),
                                        float(temperature), _ptr(uniforms), int(seed) & ((1 << 64) - 1),
                                        _ptr(n_accepted), _ptr(next_token), _ptr(committed_len), _ptr(workspace),
                                        nbytes, _ptr(status))
    check(rc, "q3kv_accept_sample")


def accept_sample_nucleus(logits: torch.Tensor, q_offsets: torch.Tensor, n_q: torch.Tensor, tokens: torch.Tensor,
                          max_n_q: int, ctx_len: torch.Tensor, temperature: float, top_p: float,
                          uniforms: torch.Tensor, seed: int, n_accepted: torch.Tensor, next_token: torch.Tensor,
                          committed_len: torch.Tensor, workspace: Optional[torch.Tensor],
                          status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_accept_sample_nucleus: rejection-sampled acceptance with the top-p nucleus."""
    rows, vocab = _check_accept(logits, q_offsets, n_q, tokens, ctx_len, n_accepted, next_token, committed_len,
                                workspace, status)
    _on_gpu("uniforms", uniforms, _current_device(), torch.float32, rows)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.load().q3kv_accept_sample_nucleus(_stream(stream), _ptr(logits), _dtype_code(logits), vocab,
                                                _ptr(q_offsets), _ptr(n_q), _ptr(tokens), n_q.shape[0], rows,
                                                max_n_q, _ptr(ctx_len), float(temperature), float(top_p),
                                                _ptr(uniforms), int(seed) & ((1 << 64) - 1), _ptr(n_accepted),
                                                _ptr(next_token), _ptr(committed_len), _ptr(workspace), nbytes,
                                                _ptr(status))
    check(rc, "q3kv_accept_sample_nucleus")


def verify_attn_lse(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                    n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                    q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                    impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                    status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_verify_attn_lse: verify_attn that also stores lse[rows, q_heads] (float32) for attn_mass."""
    _verify_lse("q3kv_verify_attn_lse", pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len, max_n_q,
                layer, q, out, lse, workspace, impl, split_positions, status, stream)


def prefill_attn_lse(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                     n_new: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_new: int, layer: int,
                     q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                     impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_prefill_attn_lse: prefill_attn that also stores lse[rows, q_heads] (float32)."""
    _verify_lse("q3kv_prefill_attn_lse", pool_bytes, desc, pool, page_table, ctx_len, n_new, q_offsets, max_ctx_len,
                max_n_new, layer, q, out, lse, workspace, impl, split_positions, status, stream)


def fp8_verify_attn_lse(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                        n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                        q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                        impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_fp8_verify_attn_lse: fp8_verify_attn that also stores lse[rows, q_heads] (float32)."""
    _verify_lse("q3kv_fp8_verify_attn_lse", fp8_pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len,
                max_n_q, layer, q, out, lse, workspace, impl, split_positions, status, stream)


def t5k_verify_attn_lse(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                        n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                        q: torch.Tensor, out: torch.Tensor, lse: torch.Tensor, workspace: torch.Tensor,
                        impl: int = _lib.Q3KV_IMPL_AUTO, split_positions: int = 0,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_t5k_verify_attn_lse: t5k_verify_attn (AUTO: the tensor-core leg) that also stores lse[rows, q_heads]."""
    _verify_lse("q3kv_t5k_verify_attn_lse", t5k_pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len,
                max_n_q, layer, q, out, lse, workspace, impl, split_positions, status, stream)


def _check_lse(lse: torch.Tensor, q: torch.Tensor, heads: int, dev: int) -> None:
    _on_gpu("lse", lse, dev, torch.float32)
    if lse.dim() != 2 or lse.shape[1] != heads or lse.shape[0] < q.shape[0]:
        raise ValueError(f"lse must be [rows >= {q.shape[0]}, {heads}], got {tuple(lse.shape)}")


def _verify_lse(name, pool_bytes_fn, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len, max_n_q, layer, q, out,
                lse, workspace, impl, split_positions, status, stream) -> None:
    _check_verify(desc, pool, pool_bytes_fn, page_table, ctx_len, n_q, q_offsets, q, out, workspace, status)
    _check_lse(lse, q, desc.num_q_heads, _current_device())
    rc = getattr(_lib.load(), name)(_stream(stream), ctypes.byref(desc), _ptr(pool), _ptr(page_table),
                                    page_table.shape[1], _ptr(ctx_len), _ptr(n_q), _ptr(q_offsets), ctx_len.shape[0],
                                    max_ctx_len, max_n_q, layer, _ptr(q), _dtype_code(q), _ptr(out), _ptr(lse), impl,
                                    split_positions, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _ptr(status))
    check(rc, name)


def attn_mass(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor, n_q: torch.Tensor,
              q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int, q: torch.Tensor, lse: torch.Tensor,
              decay: float, mass: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_attn_mass: mass[slots, kv_heads, >= max_ctx_len] (float32) = decay * mass + the step's attention weights."""
    _attn_mass("q3kv_attn_mass", pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len, max_n_q, layer,
               q, lse, decay, mass, status, stream)


def fp8_attn_mass(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                  n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                  q: torch.Tensor, lse: torch.Tensor, decay: float, mass: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_fp8_attn_mass: attn_mass over the fp8 comparison cache."""
    _attn_mass("q3kv_fp8_attn_mass", fp8_pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len,
               max_n_q, layer, q, lse, decay, mass, status, stream)


def t5k_attn_mass(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                  n_q: torch.Tensor, q_offsets: torch.Tensor, max_ctx_len: int, max_n_q: int, layer: int,
                  q: torch.Tensor, lse: torch.Tensor, decay: float, mass: torch.Tensor,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_t5k_attn_mass: attn_mass over the turbo5k-style cache."""
    _attn_mass("q3kv_t5k_attn_mass", t5k_pool_bytes, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len,
               max_n_q, layer, q, lse, decay, mass, status, stream)


def _attn_mass(name, pool_bytes_fn, desc, pool, page_table, ctx_len, n_q, q_offsets, max_ctx_len, max_n_q, layer, q, lse,
               decay, mass, status, stream) -> None:
    dev, lib = _current_device(), _lib.load()
    n, pages, (p_pool, p_table, p_ctx, p_nq, p_off, p_status) = _cache_pointers(
        desc, pool, _pool_need(pool_bytes_fn, lib, bytes(desc)), page_table, ctx_len, n_q, q_offsets, status, dev)
    if q is None or lse is None or mass is None:
        _required(q=q, lse=lse, mass=mass)
    p_q, p_lse, p_mass = _pointers(dev, ("q", q, None, 0), ("lse", lse, torch.float32, 0), ("mass", mass, torch.float32, 0))
    hq, hk = desc.num_q_heads, desc.num_kv_heads
    shape = q.shape
    if len(shape) != 3 or shape[1] != hq or shape[2] != HEAD_DIM:
        raise ValueError(f"q must be [rows, {hq}, {HEAD_DIM}], got {tuple(shape)}")
    rows, shape = shape[0], lse.shape
    if len(shape) != 2 or shape[1] != hq or shape[0] < rows:
        raise ValueError(f"lse must be [rows >= {rows}, {hq}], got {tuple(shape)}")
    shape = mass.shape
    if len(shape) != 3 or shape[0] < n or shape[1] != hk or shape[2] < max_ctx_len:
        raise ValueError(f"mass must be [slots >= {n}, {hk}, positions >= {max_ctx_len}], got {tuple(shape)}")
    end = p_mass + 4 * shape[0] * hk * shape[2]
    if (p_mass < p_q + q.nbytes and p_q < end) or (p_mass < p_lse + lse.nbytes and p_lse < end) or (p_mass < p_pool + pool.nbytes and p_pool < end):
        raise ValueError("mass overlaps q, lse or the pool")
    rc = getattr(lib, name)(_stream(stream), ctypes.byref(desc), p_pool, p_table, pages, p_ctx, p_nq, p_off,
                                    n, max_ctx_len, max_n_q, layer, p_q, _dtype_code(q), p_lse, float(decay), p_mass, shape[2],
                                    p_status)
    check(rc, name)


def evict(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor, max_ctx_len: int,
          budget: torch.Tensor, max_budget: int, n_sink: int, n_recent: int, layer: int, mass: torch.Tensor,
          dst_page_table: torch.Tensor, kept: torch.Tensor, mass_out: Optional[torch.Tensor], new_len: torch.Tensor,
          status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_evict: keep budget[b] positions of every slot by mass[layers, slots, kv_heads, >= max_ctx_len] and compact
    their records into the pages of dst_page_table; kept and mass_out are [layers, slots, kv_heads, max_budget]."""
    _evict("q3kv_evict", pool_bytes, desc, pool, page_table, ctx_len, max_ctx_len, budget, max_budget, n_sink, n_recent,
           layer, mass, dst_page_table, kept, mass_out, new_len, status, stream)


def fp8_evict(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor, max_ctx_len: int,
              budget: torch.Tensor, max_budget: int, n_sink: int, n_recent: int, layer: int, mass: torch.Tensor,
              dst_page_table: torch.Tensor, kept: torch.Tensor, mass_out: Optional[torch.Tensor], new_len: torch.Tensor,
              status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_fp8_evict: evict over the fp8 comparison cache."""
    _evict("q3kv_fp8_evict", fp8_pool_bytes, desc, pool, page_table, ctx_len, max_ctx_len, budget, max_budget, n_sink,
           n_recent, layer, mass, dst_page_table, kept, mass_out, new_len, status, stream)


def t5k_evict(desc: CacheDesc, pool: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor, max_ctx_len: int,
              budget: torch.Tensor, max_budget: int, n_sink: int, n_recent: int, layer: int, mass: torch.Tensor,
              dst_page_table: torch.Tensor, kept: torch.Tensor, mass_out: Optional[torch.Tensor], new_len: torch.Tensor,
              status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_t5k_evict: evict over the turbo5k-style cache."""
    _evict("q3kv_t5k_evict", t5k_pool_bytes, desc, pool, page_table, ctx_len, max_ctx_len, budget, max_budget, n_sink,
           n_recent, layer, mass, dst_page_table, kept, mass_out, new_len, status, stream)


def _evict(name, pool_bytes_fn, desc, pool, page_table, ctx_len, max_ctx_len, budget, max_budget, n_sink, n_recent, layer,
           mass, dst_page_table, kept, mass_out, new_len, status, stream) -> None:
    dev, lib = _current_device(), _lib.load()
    n, pages, (p_pool, p_table, p_ctx, p_budget, p_new, p_status) = _cache_pointers(
        desc, pool, _pool_need(pool_bytes_fn, lib, bytes(desc)), page_table, ctx_len, budget, new_len, status, dev,
        ("budget", "new_len"))
    if dst_page_table is None or mass is None or kept is None:
        _required(dst_page_table=dst_page_table, mass=mass, kept=kept)
    i32, f32 = torch.int32, torch.float32
    p_dst, p_mass, p_kept, p_out = _pointers(dev, ("dst_page_table", dst_page_table, i32, 0), ("mass", mass, f32, 0),
                                             ("kept", kept, i32, 0), ("mass_out", mass_out, f32, 0))
    dst_shape = dst_page_table.shape
    if len(dst_shape) != 2 or dst_shape[1] < 1 or dst_shape[0] < n:
        raise ValueError(f"dst_page_table must be int32 [num_slots >= {n}, max_pages_per_slot >= 1], "
                         f"got {tuple(dst_shape)}")
    heads, shape = desc.num_kv_heads, mass.shape
    if len(shape) != 4 or shape[1] != n or shape[2] != heads or shape[3] < max_ctx_len:
        raise ValueError(f"mass must be [layers, {n}, {heads}, positions >= {max_ctx_len}], got {tuple(shape)}")
    want = (shape[0], n, heads, max_budget)
    if kept.shape != want or (mass_out is not None and mass_out.shape != want):
        what, t = ("kept", kept) if kept.shape != want else ("mass_out", mass_out)
        raise ValueError(f"{what} must be {want}, got {tuple(t.shape)}")
    rc = getattr(lib, name)(_stream(stream), ctypes.byref(desc), p_pool, p_table, pages, p_ctx, n, max_ctx_len,
                                    p_budget, max_budget, n_sink, n_recent, layer, shape[0], p_mass, shape[3], p_dst,
                                    dst_shape[1], p_kept, p_out, p_new, p_status)
    check(rc, name)


def make_rope_plan(rotary_dim: int, theta: float, sections, deal_axes: bool = False, axis_freqs: bool = False,
                   adjacent: bool = False) -> RopePlan:
    """q3kv_rope_plan_init: sections[a] pairs turn with axis a's position (their sum is rotary_dim / 2)."""
    if len(sections) > _lib.Q3KV_ROPE_MAX_AXES:
        raise ValueError(f"at most {_lib.Q3KV_ROPE_MAX_AXES} axes, got {len(sections)}")
    flags = ((_lib.Q3KV_ROPE_ADJACENT if adjacent else 0) | (_lib.Q3KV_ROPE_DEAL_AXES if deal_axes else 0)
             | (_lib.Q3KV_ROPE_AXIS_FREQS if axis_freqs else 0))
    config = _lib.RopeConfig(theta, rotary_dim, len(sections), (ctypes.c_int32 * 4)(*sections), flags, 0)
    plan = RopePlan()
    check(_lib.load().q3kv_rope_plan_init(ctypes.byref(config), ctypes.byref(plan)), "q3kv_rope_plan_init")
    return plan


def _strided_rows(name: str, t: torch.Tensor, rows: int, dev: int):
    """Pointer, row stride and heads of [rows, heads, 256] rows whose heads are contiguous; rows may be strided."""
    if not isinstance(t, torch.Tensor) or _device_index(t) != dev:
        _on_gpu(name, t, dev)
    shape = t.shape
    if len(shape) != 3 or shape[0] != rows or shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must be [{rows}, heads, {HEAD_DIM}], got {tuple(shape)}")
    heads = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), heads * HEAD_DIM, heads
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != HEAD_DIM):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.data_ptr(), row if rows > 1 else heads * HEAD_DIM, heads


def _rows_meet(a: int, a_step: int, b: int, b_step: int, width: int, rows: int) -> bool:
    """Whether rows [a + i a_step, + width) and [b + j b_step, + width) share a byte, i, j < rows, steps >= width if rows > 1."""
    if a_step == b_step:
        d = min((width - 1 + a - b) // b_step, rows - 1)     # the last j - i whose row of b begins before a's ends
        return d > -rows and b - a + d * b_step > -width
    for at in range(a, a + rows * a_step, a_step):
        j = min((width - 1 + at - b) // b_step, rows - 1)
        if j >= 0 and b + j * b_step + width > at:
            return True
    return False


def rope(plan: RopePlan, positions: torch.Tensor, q: torch.Tensor, q_out: torch.Tensor, k: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_rope: rotate q and k [rows, heads, 256] by positions int32 [rows, axes] into q_out and k_out.

    Rows may be strided (slices of one projection); an output may be its input.
    """
    dev = _current_device()
    p_pos, = _pointers(dev, ("positions", positions, torch.int32, 0))
    if p_pos is None or positions.dim() != 2:
        raise ValueError(f"positions must be [rows, {plan.num_axes}]"
                         + (f", got {tuple(positions.shape)}" if positions is not None else ""))
    rows, axes = positions.shape
    if axes != plan.num_axes:
        raise ValueError(f"positions must be [rows, {plan.num_axes}], got {(rows, axes)}")
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out come together")
    if not isinstance(q, torch.Tensor):
        _on_gpu("q", q, dev)
    args = []
    code = _dtype_code(q)
    dtype, size = q.dtype, 4 if code == _lib.Q3KV_F32 else 2
    for name, x, y in (("q", q, q_out),) if k is None else (("q", q, q_out), ("k", k, k_out)):
        src, src_stride, heads = _strided_rows(name, x, rows, dev)
        dst, dst_stride, out_heads = _strided_rows(name + "_out", y, rows, dev)
        if heads != out_heads or x.dtype is not dtype or y.dtype is not dtype:
            raise ValueError(f"{name} and {name}_out must have the heads of one another and the dtype of q")
        if rows and heads and not (src == dst and src_stride == dst_stride):
            # an exact in-place call is fine, any other overlap is not (the library looks at the other operands)
            if (src < dst + ((rows - 1) * dst_stride + heads * HEAD_DIM) * size
                    and dst < src + ((rows - 1) * src_stride + heads * HEAD_DIM) * size
                    and _rows_meet(src, src_stride * size, dst, dst_stride * size, heads * HEAD_DIM * size, rows)):
                raise ValueError(f"{name}_out overlaps {name} without being the same rows")
        args += (src, src_stride, dst, dst_stride, heads)
    if k is None:
        args += (None, 0, None, 0, 0)
    rc = _lib.load().q3kv_rope(_stream(stream), ctypes.byref(plan), p_pos, rows, *args, code)
    check(rc, "q3kv_rope")


def accept_draft_workspace_bytes(num_slots: int, num_rows: int, vocab: int) -> int:
    n = ctypes.c_size_t()
    check(_lib.load().q3kv_accept_draft_workspace_bytes(num_slots, num_rows, vocab, ctypes.byref(n)),
          "q3kv_accept_draft_workspace_bytes")
    return n.value


def accept_draft(logits: torch.Tensor, draft_probs: torch.Tensor, q_offsets: torch.Tensor, n_q: torch.Tensor,
                 tokens: torch.Tensor, max_n_q: int, ctx_len: torch.Tensor, temperature: float, uniforms: torch.Tensor,
                 seed: int, n_accepted: torch.Tensor, next_token: torch.Tensor, committed_len: torch.Tensor,
                 workspace: Optional[torch.Tensor], accept_prob: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> None:
    """q3kv_accept_draft: rejection-sampled acceptance of drafts drawn from draft_probs [rows, vocab] (f32 or bf16)."""
    if (logits is None or draft_probs is None or q_offsets is None or n_q is None or tokens is None or ctx_len is None
            or uniforms is None or n_accepted is None or next_token is None or committed_len is None):
        _required(logits=logits, draft_probs=draft_probs, q_offsets=q_offsets, n_q=n_q, tokens=tokens, ctx_len=ctx_len,
                  uniforms=uniforms, n_accepted=n_accepted, next_token=next_token, committed_len=committed_len)
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError(f"logits must be [rows, vocab], got {tuple(shape)}")
    if n_q.dim() != 1:
        raise ValueError("n_q must be one-dimensional")
    rows, vocab = shape
    n, i32, f32 = n_q.numel(), torch.int32, torch.float32
    p = _pointers(_current_device(), ("logits", logits, None, 0), ("draft_probs", draft_probs, None, 0),
                  ("q_offsets", q_offsets, i32, n), ("n_q", n_q, i32, 0), ("tokens", tokens, i32, rows), ("ctx_len", ctx_len, i32, n),
                  ("uniforms", uniforms, f32, rows), ("n_accepted", n_accepted, i32, n), ("next_token", next_token, i32, n),
                  ("committed_len", committed_len, i32, n), ("accept_prob", accept_prob, f32, rows),
                  ("workspace", workspace, None, 0), ("status", status, i32, 1))
    if draft_probs.shape != shape:
        raise ValueError(f"draft_probs must be {tuple(shape)}, got {tuple(draft_probs.shape)}")
    rc = _lib.load().q3kv_accept_draft(_stream(stream), p[0], _dtype_code(logits), vocab, p[1], _dtype_code(draft_probs), p[2], p[3],
                                       p[4], n, rows, max_n_q, p[5], float(temperature), p[6], int(seed) & ((1 << 64) - 1), p[7],
                                       p[8], p[9], p[10], p[11], 0 if workspace is None else workspace.nbytes, p[12])
    check(rc, "q3kv_accept_draft")
