"""Python binding of libpa.so: paged-KV GQA attention for one GB300 (sm_103a).

This module only marshals arguments: it takes torch CUDA tensors, checks their dtype,
device and layout, and passes raw pointers, sizes and the current CUDA stream to the
C ABI declared in include/pa.h (the calls of the 8-bit cache and of rotation by axes through a
compiled module, csrc/pa_bind.cpp, where their arguments are as usual: a small call's time is its
checks).  Every step of the computation runs in the library's
CUDA kernels.  There is no CPU or PyTorch fallback: if libpa.so is missing or cannot be
loaded, every call raises.  The module is an option: without it those calls are checked in Python,
with one warning.

Functions (names follow the C ABI):
    slot_mapping(positions, block_table, block_size, seq_idx=None)    -> int64 slots
    decode_input_prep(positions, block_tables, block_sizes, sampled_ids=None)
                                                                      -> step inputs
    reshape_and_cache(key, value, k_cache, v_cache, slot_mapping)     (in place)
    decode_workspace_size(...), decode(q, k_cache, v_cache, block_table, seq_lens, ...)
    prefill_workspace_size(...), prefill_chunk(q, k_cache, v_cache, block_table, q_start,
                                               causal, scale, workspace=None)
    prefill_varlen_workspace_size(...), prefill_varlen(q, k_cache, v_cache, block_table,
                                               cu_seqlens_q, seq_lens_k, causal, scale)
    prefill_plan(q_len, q_start, causal, num_q_heads, block_size, num_ctas)  (host only)
    batch_input_prep(num_computed, num_new, block_tables, block_sizes, free_pages, num_tokens)
                                                                      -> mixed-step inputs
    qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps)   -> q, k
    qk_norm_rope_cache(q, k, v, ..., eps, k_cache, v_cache, slot_mapping)
                                                                      -> q (K/V in place)
    4-bit cache (uint8 tensors of q4_cache_shape(num_pages, block_size, num_kv_heads)):
    reshape_and_cache_q4(...) (in place), gather_cache_q4(...) -> key, value
    decode_q4(...), prefill_chunk_q4(...), prefill_varlen_q4(...) and their
    *_workspace_size functions: as the calls without _q4
    8-bit cache (float8_e4m3fn codes and uint8 scales, shapes of q8_cache_shapes(...)):
    reshape_and_cache_q8(...) (in place), gather_cache_q8(...) -> key, value
    decode_q8(...), prefill_chunk_q8(...), prefill_varlen_q8(...) and their
    *_workspace_size functions: as the calls without _q8
    qk_norm_mrope(...), qk_norm_mrope_cache(...): qk_norm_rope(_cache) with positions on several
    axes; mrope_axes(sections, ...) -> the axis of each frequency
    device_errors(clear=True)
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
import warnings

import torch

from . import _build

__all__ = ["load", "build", "slot_mapping", "decode_input_prep", "reshape_and_cache",
           "decode_workspace_size",
           "decode", "decode_append", "prefill_chunk", "prefill_varlen", "prefill_plan",
           "prefill_workspace_size", "prefill_varlen_workspace_size", "prefill_plan_pieces", "device_errors", "set_kernel_events", "build_info", "PAError",
           "DEVERR_PAGE", "DEVERR_SEQLEN", "DEVERR_SLOT", "DEVERR_TIMEOUT", "DEVERR_POSITION", "DEVERR_LAYOUT",
           "DEVERR_NO_PAGES", "Q4_ROW_BYTES", "batch_input_prep", "qk_norm_rope",
           "qk_norm_rope_cache", "q4_cache_shape", "reshape_and_cache_q4", "gather_cache_q4",
           "decode_q4", "decode_q4_workspace_size", "prefill_chunk_q4",
           "prefill_q4_workspace_size", "prefill_varlen_q4", "prefill_varlen_q4_workspace_size",
           "Q8_TOKENS", "q8_cache_shapes", "reshape_and_cache_q8", "gather_cache_q8", "decode_q8",
           "decode_q8_workspace_size", "prefill_chunk_q8", "prefill_q8_workspace_size",
           "prefill_varlen_q8", "prefill_varlen_q8_workspace_size", "mrope_axes", "qk_norm_mrope",
           "qk_norm_mrope_cache",
           "LIB_PATH"]

LIB_PATH = _build.LIB
DEVERR_PAGE, DEVERR_SEQLEN, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_POSITION = 1, 2, 4, 8, 16
DEVERR_LAYOUT, DEVERR_NO_PAGES = 32, 64
Q4_ROW_BYTES = 144  # PA_Q4_ROW_BYTES: a token of one KV head in the 4-bit cache
Q8_TOKENS = 16  # PA_Q8_TOKENS: tokens of a page under one scale of the 8-bit cache
ERR_TIMEOUT = 4  # PA_ERR_TIMEOUT

_lib = None
_bind = None  # the module of the short calls
_lock = threading.Lock()


class PAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = _lib.pa_status_string(status).decode() if _lib is not None else str(status)
        super().__init__(f"{where}: {name}")


def build(force: bool = False) -> str:
    """Compile libpa.so (nvcc, sm_103a) in-tree."""
    return _build.build(force=force)


def load():
    """Load libpa.so and declare the C signatures.  Raises if it is not built."""
    global _lib, _bind
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpa.so not built ({LIB_PATH}); run __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
        sig = {
            "pa_slot_mapping": ([P, P, P, i32, i64, i32, i32, i32, P, P], i32),
            "pa_reshape_and_cache": ([P, P, P, P, i64, i64, P, i32, i32, i32, i32, P], i32),
            "pa_decode_input_prep": ([P, P, P, P, P, i32, i32, P, P, P, P, P, P], i32),
            "pa_decode_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
            "pa_decode": ([P, P, P, i64, i64, P, i64, P, i32, i32, i32, i32, i32, i32, f32, P, P,
                           sz, P, P, P, P], i32),
            "pa_decode_append": ([P, P, P, i64, i64, P, i64, P, i32, i32, i32, i32, i32, i32, f32,
                                  P, P, sz, P, P, P, P], i32),
            "pa_prefill_workspace_size": ([i32, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_chunk": ([P, P, P, i64, i64, P, i32, i32, i32, i32, i32, i32, i32, f32,
                                  P, P, sz, P], i32),
            "pa_prefill_varlen_workspace_size": ([P, P, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_plan": ([i32, i32, i32, i32, i32, i32, i32, P, P, P], i32),
            "pa_prefill_plan_pieces": ([i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, P, P, P,
                                        P,
                                        P], i32),
            "pa_prefill_varlen": ([P, P, P, i64, i64, P, i64, P, P, i32, i32, i32, i32, i32,
                                   i32, f32, P, P, sz, P], i32),
            "pa_batch_input_prep": ([P, P, i32, i32, P, P, P, P, P, P, i32, P, P, P, P, P, P, P],
                                    i32),
            "pa_qk_norm_rope": ([P, i64, P, i64, P, P, f32, f32, P, i32, i32, i32, P, i32, i32,
                                 i32, i32, P, i64, P, i64, P], i32),
            "pa_qk_norm_rope_cache": ([P, i64, P, i64, P, i64, P, P, f32, f32, P, i32, i32, i32,
                                       P, i32, i32, i32, i32, P, i64, i32, P, P, i64, i64, P, i32,
                                       P], i32),
            "pa_reshape_and_cache_q4": ([P, i64, P, i64, P, P, i64, i64, P, i32, i32, i32, i32,
                                         P], i32),
            "pa_gather_cache_q4": ([P, P, i64, i64, P, i32, i32, i32, i32, P, P, P], i32),
            "pa_decode_q4_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
            "pa_decode_q4": ([P, P, P, i64, i64, P, i64, P, i32, i32, i32, i32, i32, i32, f32, P,
                              P, sz, P], i32),
            "pa_prefill_q4_workspace_size": ([i32, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_chunk_q4": ([P, P, P, i64, i64, P, i32, i32, i32, i32, i32, i32, i32,
                                     f32, P, P, sz, P], i32),
            "pa_prefill_varlen_q4_workspace_size": ([P, P, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_varlen_q4": ([P, P, P, i64, i64, P, i64, P, P, i32, i32, i32, i32, i32,
                                      i32, f32, P, P, sz, P], i32),
            "pa_reshape_and_cache_q8": ([P, i64, P, i64, P, P, P, P, i64, i64, i64, P, i32, i32,
                                         i32, i32, P], i32),
            "pa_gather_cache_q8": ([P, P, P, P, i64, i64, i64, P, i32, i32, i32, i32, P, P, P],
                                   i32),
            "pa_decode_q8_workspace_size": ([i32, i32, i32, i32, i32, i32], sz),
            "pa_decode_q8": ([P, P, P, P, P, i64, i64, i64, P, i64, P, i32, i32, i32, i32, i32,
                              i32, f32, P, P, sz, P], i32),
            "pa_prefill_q8_workspace_size": ([i32, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_chunk_q8": ([P, P, P, P, P, i64, i64, i64, P, i32, i32, i32, i32, i32,
                                     i32, i32, f32, P, P, sz, P], i32),
            "pa_prefill_varlen_q8_workspace_size": ([P, P, i32, i32, i32, i32, i32, i32], sz),
            "pa_prefill_varlen_q8": ([P, P, P, P, P, i64, i64, i64, P, i64, P, P, i32, i32, i32,
                                      i32, i32, i32, f32, P, P, sz, P], i32),
            "pa_qk_norm_mrope": ([P, i64, P, i64, P, P, f32, f32, P, i32, i32, i32, P, i64, i32,
                                  ctypes.c_char_p, i32, i32, i32, i32, P, i64, P, i64, P], i32),
            "pa_qk_norm_mrope_cache": ([P, i64, P, i64, P, i64, P, P, f32, f32, P, i32, i32, i32,
                                        P, i64, i32, ctypes.c_char_p, i32, i32, i32, i32, P, i64,
                                        i32, P, P, i64, i64, P, i32, P], i32),
            "pa_copy": ([P, P, sz, P], i32),
            "pa_get_device_errors": ([ctypes.POINTER(ctypes.c_uint), i32, P], i32),
            "pa_set_kernel_events": ([P, P], i32),
            "pa_status_string": ([i32], ctypes.c_char_p),
            "pa_build_info": ([], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _bind, _lib = _load_bind(), lib
        return lib


class _NoShortCalls:
    """In the place of the module of the short calls where it is missing: takes no call, so that each
    is checked and made in Python (some 10 us slower), and says so once."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        why, self._why = self._why, None
        if why is not None:
            warnings.warn(f"no pa_bind module ({why}): the short calls take the way through ctypes; "
                          "__graft_entry__.build() makes it", RuntimeWarning, stacklevel=3)
        return lambda *args: None


def _load_bind():
    try:
        loader = importlib.machinery.ExtensionFileLoader("pa_bind", _build.BIND)
        bind = importlib.util.module_from_spec(importlib.util.spec_from_loader("pa_bind", loader))
        loader.exec_module(bind)
        bind.load(LIB_PATH)
        return bind
    except (ImportError, RuntimeError) as e:  # not there, of another Python or torch, of another libpa.so
        return _NoShortCalls(str(e))


def _stream():
    # torch.cuda.current_stream() builds a Stream object: 2.8 us of a call's host time
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _check_out(out, like):
    """A caller's decode output: BF16, contiguous, shaped like q, on the GPU or in
    page-locked host memory (which the combine kernel writes directly)."""
    if not isinstance(out, torch.Tensor) or not (out.is_cuda or out.is_pinned()):
        raise TypeError("out must be a CUDA tensor or a pinned host tensor")
    if out.dtype != torch.bfloat16 or out.shape != like.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous BF16 tensor shaped like q")


def _check_cache(k_cache, v_cache):
    for n, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        _check(c, n, torch.bfloat16, 4)
        if c.stride(3) != 1 or c.stride(2) != c.shape[3] or c.stride(1) != c.shape[2] * c.shape[3]:
            raise ValueError(f"{n}: each page must be a contiguous [BS, Hkv, D] block")
    if k_cache.shape != v_cache.shape or k_cache.stride(0) != v_cache.stride(0):
        raise ValueError("k_cache and v_cache must have the same shape and page stride")
    return k_cache.stride(0)


def _raise(rc, where):
    if rc != 0:
        raise PAError(rc, where)


def build_info() -> str:
    return load().pa_build_info().decode()


def slot_mapping(positions, block_table, block_size, seq_idx=None, max_blocks=None, out=None):
    """int64 slot of each position (see pa_slot_mapping)."""
    lib = load()
    _check(positions, "positions", torch.int32, 1)
    _check(block_table, "block_table", torch.int32)
    bt = block_table if block_table.dim() == 2 else block_table.view(1, -1)
    if bt.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    if seq_idx is not None:
        _check(seq_idx, "seq_idx", torch.int32, 1)
    n = positions.numel()
    if out is None:
        out = torch.empty(n, dtype=torch.int64, device=positions.device)
    mb = bt.shape[1] if max_blocks is None else int(max_blocks)
    _raise(lib.pa_slot_mapping(_ptr(positions.contiguous()), _ptr(seq_idx), _ptr(bt),
                               bt.shape[0], bt.stride(0), mb, n, int(block_size), _ptr(out),
                               _stream()), "pa_slot_mapping")
    return out


def decode_input_prep(positions, block_tables, block_sizes, sampled_ids=None, max_blocks=None,
                      out=None):
    """One decode step's inputs for several KV-cache groups in one launch (see
    pa_decode_input_prep).  block_tables / block_sizes: one int32 [S, n] table and one
    block size per group.  Returns a dict with seq_lens, query_start_loc, input_ids (when
    sampled_ids is given) and slot_mappings (a list, one int64 [S] tensor per group);
    `out` may pass that dict back in to reuse its tensors."""
    lib = load()
    _check(positions, "positions", torch.int32, 1)
    S, G = positions.shape[0], len(block_tables)
    if len(block_sizes) != G or not 1 <= G <= 8:
        raise ValueError("one block size per group, 1..8 groups")
    dev = positions.device
    if out is None:
        out = {"seq_lens": torch.empty(S, dtype=torch.int32, device=dev),
               "query_start_loc": torch.empty(S + 1, dtype=torch.int32, device=dev),
               "slot_mappings": [torch.empty(S, dtype=torch.int64, device=dev) for _ in range(G)]}
        if sampled_ids is not None:
            out["input_ids"] = torch.empty(S, dtype=torch.int32, device=dev)
    tables = []
    for t in block_tables:
        _check(t, "block_table", torch.int32, 2)
        if t.shape[0] < S or t.stride(1) != 1:
            raise ValueError("block tables: one row per sequence, contiguous rows")
        tables.append(t)
    mb = max_blocks if max_blocks is not None else [t.shape[1] for t in tables]
    arr = lambda ctype, vals: (ctype * G)(*vals)
    bt_ptrs = arr(ctypes.c_void_p, [t.data_ptr() for t in tables])
    sm_ptrs = arr(ctypes.c_void_p, [m.data_ptr() for m in out["slot_mappings"]])
    strides = arr(ctypes.c_int64, [t.stride(0) for t in tables])
    mbs = arr(ctypes.c_int, [int(x) for x in mb])
    bss = arr(ctypes.c_int, [int(x) for x in block_sizes])
    sid = None
    if sampled_ids is not None:
        _check(sampled_ids, "sampled_ids", torch.int32, 1)
        sid = sampled_ids.contiguous()
    _raise(lib.pa_decode_input_prep(_ptr(positions.contiguous()), _ptr(sid),
                                    _ptr(out.get("input_ids")), _ptr(out["seq_lens"]),
                                    _ptr(out["query_start_loc"]), S, G, bt_ptrs, strides, mbs,
                                    bss, sm_ptrs, _stream()), "pa_decode_input_prep")
    return out


def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping_):
    """Write key/value [T, Hkv, D] into the caches at slot_mapping_ (in place)."""
    lib = load()
    _check(key, "key", torch.bfloat16, 3)
    _check(value, "value", torch.bfloat16, 3)
    _check(slot_mapping_, "slot_mapping", torch.int64, 1)
    ps = _check_cache(k_cache, v_cache)
    key, value = key.contiguous(), value.contiguous()
    T, hkv, d = key.shape
    _raise(lib.pa_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), ps,
                                    k_cache.shape[0], _ptr(slot_mapping_), T, hkv, d,
                                    k_cache.shape[1], _stream()), "pa_reshape_and_cache")


def copy(dst, src):
    """Copy src into dst (same byte size, both contiguous) with a kernel on the current
    stream (see pa_copy).  Each tensor may live on the GPU or in pinned host memory."""
    lib = load()
    for t, nm in ((dst, "dst"), (src, "src")):
        if not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{nm} must be a CUDA tensor or pinned host memory")
    nb = dst.numel() * dst.element_size()
    if nb != src.numel() * src.element_size():
        raise ValueError("dst and src differ in size")
    _raise(lib.pa_copy(ctypes.c_void_p(dst.data_ptr()), ctypes.c_void_p(src.data_ptr()), nb,
                       _stream()), "pa_copy")
    return dst


def decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                          max_seq_len) -> int:
    return int(load().pa_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                               block_size, max_seq_len))


def decode(q, k_cache, v_cache, block_table, seq_lens, scale, max_seq_len, out=None,
           workspace=None, new_k=None, new_v=None, new_slots=None):
    """q=1 paged decode (see pa_decode).  Returns out [S, Hq, D] BF16."""
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    ps = _check_cache(k_cache, v_cache)
    q = q.contiguous()
    S, hq, d = q.shape
    _, bs, hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q)
    need = decode_workspace_size(S, hq, hkv, d, bs, max_seq_len)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    if new_k is not None:
        new_k, new_v = new_k.contiguous(), new_v.contiguous()
    _raise(lib.pa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), ps, k_cache.shape[0],
                         _ptr(block_table), block_table.stride(0), _ptr(seq_lens), S,
                         int(max_seq_len), hq, hkv, d, bs, float(scale), _ptr(out),
                         _ptr(workspace), workspace.numel() * workspace.element_size(),
                         _ptr(new_k), _ptr(new_v), _ptr(new_slots), _stream()), "pa_decode")
    return out


def decode_append(q, k_cache, v_cache, block_table, seq_lens, scale, max_seq_len, new_k, new_v,
                  out=None, workspace=None, slot_mapping=None):
    """Decode step that appends each sequence's newest token (position seq_lens[s] - 1)
    from new_k / new_v at the slot the kernel derives from the block table, then attends
    (see pa_decode_append).  slot_mapping, if given (int64 [S]), receives those slots.
    Returns out [S, Hq, D] BF16."""
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _check(new_k, "new_k", torch.bfloat16, 3)
    _check(new_v, "new_v", torch.bfloat16, 3)
    if slot_mapping is not None:
        _check(slot_mapping, "slot_mapping", torch.int64, 1)
        if not slot_mapping.is_contiguous() or slot_mapping.numel() < q.shape[0]:
            raise ValueError("slot_mapping must be a contiguous int64 tensor of num_seqs entries")
    ps = _check_cache(k_cache, v_cache)
    q = q.contiguous()
    new_k, new_v = new_k.contiguous(), new_v.contiguous()
    S, hq, d = q.shape
    _, bs, hkv, _ = k_cache.shape
    if new_k.shape != (S, hkv, d) or new_v.shape != (S, hkv, d):
        raise ValueError("new_k / new_v must be [num_seqs, num_kv_heads, head_dim]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_out(out, q)
    need = decode_workspace_size(S, hq, hkv, d, bs, max_seq_len)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _raise(lib.pa_decode_append(_ptr(q), _ptr(k_cache), _ptr(v_cache), ps, k_cache.shape[0],
                                _ptr(block_table), block_table.stride(0), _ptr(seq_lens), S,
                                int(max_seq_len), hq, hkv, d, bs, float(scale), _ptr(out),
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(new_k), _ptr(new_v), _ptr(slot_mapping), _stream()),
           "pa_decode_append")
    return out


def prefill_workspace_size(q_len, q_start, causal, num_q_heads, num_kv_heads, head_dim,
                           block_size):
    """Bytes of workspace with which pa_prefill_chunk may split items (0: none would pay)."""
    return int(load().pa_prefill_workspace_size(int(q_len), int(q_start), int(bool(causal)),
                                                num_q_heads, num_kv_heads, head_dim,
                                                block_size))


def _workspace_arg(workspace, need, device):
    """(pointer, bytes) of a caller's workspace, or of a fresh one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    return workspace, workspace.numel() * workspace.element_size()


def prefill_chunk(q, k_cache, v_cache, block_table, q_start, causal, scale, out=None,
                  workspace=None):
    """Causal (or full) chunk attention of one sequence (see pa_prefill_chunk).  Without a
    workspace, one of pa_prefill_workspace_size bytes is allocated for the call."""
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(block_table, "block_table", torch.int32)
    ps = _check_cache(k_cache, v_cache)
    q = q.contiguous()
    bt = block_table.reshape(-1).contiguous()
    q_len, hq, d = q.shape
    _, bs, hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = prefill_workspace_size(q_len, q_start, causal, hq, hkv, d, bs)
    ws, ws_bytes = _workspace_arg(workspace, need if workspace is None else 0, q.device)
    _raise(lib.pa_prefill_chunk(_ptr(q), _ptr(k_cache), _ptr(v_cache), ps, k_cache.shape[0],
                                _ptr(bt), q_len, int(q_start), int(bool(causal)), hq, hkv, d,
                                bs, float(scale), _ptr(out), _ptr(ws), ws_bytes, _stream()),
           "pa_prefill_chunk")
    return out


def prefill_varlen_workspace_size(cu_seqlens_q, seq_lens_k, causal, num_q_heads, num_kv_heads,
                                  head_dim, block_size):
    """Bytes of workspace with which pa_prefill_varlen may split items."""
    B = len(seq_lens_k)
    cu = (ctypes.c_int32 * (B + 1))(*[int(x) for x in cu_seqlens_q])
    sk = (ctypes.c_int32 * max(B, 1))(*[int(x) for x in seq_lens_k])
    return int(load().pa_prefill_varlen_workspace_size(cu, sk, B, int(bool(causal)),
                                                       num_q_heads, num_kv_heads, head_dim,
                                                       block_size))


def prefill_varlen(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, causal, scale,
                   out=None, workspace=None):
    """Chunks of several sequences stacked row-wise in q (see pa_prefill_varlen).
    cu_seqlens_q and seq_lens_k are host sequences of ints (lists or arrays).  Without a
    workspace, one of pa_prefill_varlen_workspace_size bytes is allocated for the call."""
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(block_table, "block_table", torch.int32, 2)
    ps = _check_cache(k_cache, v_cache)
    q = q.contiguous()
    if block_table.stride(1) != 1:
        raise ValueError("block_table rows must be contiguous")
    B = len(seq_lens_k)
    if len(cu_seqlens_q) != B + 1 or int(cu_seqlens_q[-1]) != q.shape[0]:
        raise ValueError("cu_seqlens_q: num_seqs + 1 offsets ending at q's row count")
    cu = (ctypes.c_int32 * (B + 1))(*[int(x) for x in cu_seqlens_q])
    sk = (ctypes.c_int32 * max(B, 1))(*[int(x) for x in seq_lens_k])
    _, hq, d = q.shape
    _, bs, hkv, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    need = 0
    if workspace is None:
        need = int(lib.pa_prefill_varlen_workspace_size(cu, sk, B, int(bool(causal)), hq, hkv,
                                                        d, bs))
    ws, ws_bytes = _workspace_arg(workspace, need, q.device)
    _raise(lib.pa_prefill_varlen(_ptr(q), _ptr(k_cache), _ptr(v_cache), ps, k_cache.shape[0],
                                 _ptr(block_table), block_table.stride(0), cu, sk, B,
                                 int(bool(causal)), hq, hkv, d, bs, float(scale), _ptr(out),
                                 _ptr(ws), ws_bytes, _stream()), "pa_prefill_varlen")
    return out


def prefill_plan(q_len, q_start, causal, num_q_heads, num_kv_heads, block_size, num_ctas):
    """The static work assignment of prefill_chunk (see pa_prefill_plan): returns
    (cta_of_item, max_cost) with cta_of_item a list indexed by work item."""
    lib = load()
    n = ctypes.c_int(0)
    mc = ctypes.c_int(0)
    args = (int(q_len), int(q_start), int(bool(causal)), int(num_q_heads), int(num_kv_heads),
            int(block_size), int(num_ctas))
    _raise(lib.pa_prefill_plan(*args, None, ctypes.byref(n), None), "pa_prefill_plan")
    cta = (ctypes.c_int32 * n.value)()
    _raise(lib.pa_prefill_plan(*args, cta, ctypes.byref(n), ctypes.byref(mc)), "pa_prefill_plan")
    return list(cta), mc.value


def prefill_plan_pieces(q_len, q_start, causal, num_q_heads, num_kv_heads, block_size,
                        num_ctas, max_pieces=480):
    """The plan used with a workspace (host only, see pa_prefill_plan_pieces): returns
    (cta_of_item with -1 for split items, [(item, tile_begin, tile_end, cta), ...], max_cost)."""
    lib = load()
    ni, npc, mc = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    items = (ctypes.c_int32 * (-(-int(q_len) // 128) * num_q_heads))()  # an upper bound
    arrs = [(ctypes.c_int32 * max(1, max_pieces))() for _ in range(4)]
    _raise(lib.pa_prefill_plan_pieces(int(q_len), int(q_start), int(bool(causal)), num_q_heads,
                                      num_kv_heads, block_size, num_ctas, max_pieces, items,
                                      *arrs, ctypes.byref(ni), ctypes.byref(npc),
                                      ctypes.byref(mc)),
           "pa_prefill_plan_pieces")
    pieces = [(arrs[0][p], arrs[1][p], arrs[2][p], arrs[3][p]) for p in range(npc.value)]
    return list(items)[:ni.value], pieces, mc.value


def _short():
    """The module of the short calls, whose functions give None where the arguments are not as usual,
    and a status where the library refuses them."""
    if _bind is None:
        load()
    return _bind


_BF16, _I32, _I64, _U8, _F32 = (torch.bfloat16, torch.int32, torch.int64, torch.uint8,
                                torch.float32)
_E4M3 = torch.float8_e4m3fn


def _device():
    """The current device, on whose stream a call is queued (none: no tensor is on it)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


def _i32(x, name):
    """x as an int that a C int holds (ctypes would wrap it)."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must be within 32 bits, got {x}")
    return x


def _need(t, name, dtype, ndim, dev):
    """t's shape, if it is a `dtype` tensor of ndim dims on device dev, the current one."""
    try:
        if t.dtype is dtype and t.get_device() == dev:
            shape = t.shape
            if len(shape) == ndim:
                return shape
    except AttributeError:  # not a tensor
        pass
    _check(t, name, dtype, ndim)
    raise ValueError(f"{name} must be on the current CUDA device")


def _vector(t, name, dtype, n, dev):
    """Checks a contiguous vector of n entries (any number for None); returns its address."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.dim() == 1 and t.is_contiguous() and \
                (n is None or t.numel() == n):
            return t.data_ptr()
    except AttributeError:  # not a tensor
        pass
    _need(t, name, dtype, 1, dev)
    raise ValueError(f"{name} must be contiguous" + (f" and have {n} entries" if n is not None else ""))


def _table(t, name, rows, dev):
    """Checks an int32 block table of at least `rows` rows, each contiguous; returns (width,
    distance between rows)."""
    have, width = _need(t, name, _I32, 2, dev)
    row, col = t.stride()
    if have < rows or (have and width > 1 and col != 1):
        raise ValueError(f"{name}: one row per sequence, contiguous rows")
    return width, row if have > 1 else width


def _token_rows(t, name, tokens, heads, dim, dev):
    """Checks BF16 [tokens, heads, dim] rows, each token's heads contiguous; returns the
    distance between tokens."""
    shape = _need(t, name, _BF16, 3, dev)
    if shape != (tokens, heads, dim):
        raise ValueError(f"{name} must be [{tokens}, {heads}, {dim}], got {tuple(shape)}")
    return _row_stride(t, name, tokens, heads, dim)


def _row_stride(t, name, tokens, heads, dim):
    a, b, c = t.stride()
    if (c != 1 and dim > 1) or (b != dim and heads > 1):
        raise ValueError(f"{name}: each token's rows must be contiguous")
    return a if tokens > 1 else heads * dim


# (void *, int, int64_t) arrays of each length up to the number of groups
_ARRAYS = [(ctypes.c_void_p * n, ctypes.c_int * n, ctypes.c_int64 * n) for n in range(9)]


def batch_input_prep(num_computed, num_new, block_tables, block_sizes, free_pages, num_tokens,
                     out=None):
    """One mixed step's inputs from the requests' lengths (see pa_batch_input_prep).
    num_computed, num_new: int32 [S]; per KV-cache group an int32 [S, n] block table, which
    receives the new pages, a block size and an int32 list of free pages.  num_tokens: rows
    of the per-token outputs, at least the step's tokens.  Returns a dict with seq_lens,
    query_start_loc, positions, seq_idx, slot_mappings (one per group) and pages_taken (int32
    [groups]); `out` may pass that dict back in to reuse its tensors, but none of them may be an
    input (the seq_lens of one step are copied to be the num_computed of the next)."""
    lib, dev = _lib or load(), _device()
    G, T = len(block_tables), _i32(num_tokens, "num_tokens")
    if len(block_sizes) != G or len(free_pages) != G or not 1 <= G <= 8:
        raise ValueError("one block size and one free list per group, 1..8 groups")
    computed = _vector(num_computed, "num_computed", _I32, None, dev)
    S = num_computed.shape[0]
    new = _vector(num_new, "num_new", _I32, S, dev)
    widths, strides = zip(*[_table(t, "block_table", S, dev) for t in block_tables])
    free = [_vector(f, "free_pages", _I32, None, dev) for f in free_pages]
    if out is None:
        at = num_computed.device
        out = {"seq_lens": torch.empty(S, dtype=_I32, device=at),
               "query_start_loc": torch.empty(S + 1, dtype=_I32, device=at),
               "positions": torch.empty(T, dtype=_I32, device=at),
               "seq_idx": torch.empty(T, dtype=_I32, device=at),
               "slot_mappings": [torch.empty(T, dtype=_I64, device=at) for _ in range(G)],
               "pages_taken": torch.empty(G, dtype=_I32, device=at)}
    slots = out["slot_mappings"]
    if len(slots) != G:
        raise ValueError("out: one slot mapping per group")
    pointers, ints, longs = _ARRAYS[G]
    _raise(lib.pa_batch_input_prep(
        computed, new, S, G, pointers(*[t.data_ptr() for t in block_tables]),
        longs(*strides), ints(*widths), ints(*[_i32(b, "block size") for b in block_sizes]),
        pointers(*free), ints(*[f.shape[0] for f in free_pages]), T,
        _vector(out["seq_lens"], "seq_lens", _I32, S, dev),
        _vector(out["query_start_loc"], "query_start_loc", _I32, S + 1, dev),
        _vector(out["positions"], "positions", _I32, T, dev),
        _vector(out["seq_idx"], "seq_idx", _I32, T, dev),
        pointers(*[_vector(m, "slot_mapping", _I64, T, dev) for m in slots]),
        _vector(out["pages_taken"], "pages_taken", _I32, G, dev), _stream()),
        "pa_batch_input_prep")
    return out


def _rope_args(q, k, q_weight, k_weight, cos_sin, dev):
    """(tokens, query heads, KV heads, head_dim, token strides of q and k, the addresses of the
    weights, the table's sizes)"""
    T, hq, d = _need(q, "q", _BF16, 3, dev)
    kt, hkv, kd = _need(k, "k", _BF16, 3, dev)
    if kt != T or kd != d:
        raise ValueError(f"k must be [{T}, {hkv}, {d}], got [{kt}, {hkv}, {kd}]")
    qs, ks = _row_stride(q, "q", T, hq, d), _row_stride(k, "k", T, hkv, d)
    rows, rot = _need(cos_sin, "cos_sin", _F32, 2, dev)
    if not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous")
    return (T, hq, hkv, d, qs, ks, _vector(q_weight, "q_weight", _BF16, d, dev),
            _vector(k_weight, "k_weight", _BF16, d, dev), rows, rot)


def _rope_cache(v, k_cache, v_cache, slot_mapping, T, hkv, d, dev):
    """(token stride of v, address of the slots, cache format, pages, page stride, block size)"""
    vs = _token_rows(v, "v", T, hkv, d, dev)
    slots = _vector(slot_mapping, "slot_mapping", _I64, T, dev)
    fmt = 1 if isinstance(k_cache, torch.Tensor) and k_cache.dtype is _U8 else 0
    if fmt:
        pages, ps, bs, heads = _q4_cache(k_cache, v_cache, dev)
        dim = 256
    else:
        shape = _need(k_cache, "k_cache", _BF16, 4, dev)
        pages, bs, heads, dim = shape
        strides = k_cache.stride()
        ps = strides[0]
        if _need(v_cache, "v_cache", _BF16, 4, dev) != shape or v_cache.stride() != strides or \
                strides[1:] != (heads * dim, dim, 1):
            _check_cache(k_cache, v_cache)  # says what is wrong
            raise ValueError("k_cache and v_cache must have the same shape and strides")
    if heads != hkv or dim != d:
        raise ValueError("the caches' heads must be k's")
    return vs, slots, fmt, pages, ps, bs


def _rope_q_out(q_out, q, T, hq, d, dev):
    if q_out is None:
        return torch.empty((T, hq, d), dtype=_BF16, device=q.device), hq * d
    return q_out, _token_rows(q_out, "q_out", T, hq, d, dev)


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved=False,
                 weight_bias=0.0, q_out=None, k_out=None):
    """RMS norm of each query and key head and rotation by position (see pa_qk_norm_rope).
    q [T, Hq, D], k [T, Hkv, D] (views of a packed projection are taken as they are); cos_sin
    fp32 [max_position, rotary_dim], cosines then sines.  q_out / k_out may be q / k.  Rows of
    negative positions are left as they were.  Returns (q_out, k_out)."""
    lib, dev = _lib or load(), _device()
    T, hq, hkv, d, qs, ks, qw, kw, rows, rot = _rope_args(q, k, q_weight, k_weight, cos_sin, dev)
    pos = _vector(positions, "positions", _I32, T, dev)
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=_BF16, device=q.device)
    if k_out is None:
        k_out = torch.empty((T, hkv, d), dtype=_BF16, device=k.device)
    qos = _token_rows(q_out, "q_out", T, hq, d, dev)
    kos = _token_rows(k_out, "k_out", T, hkv, d, dev)
    _raise(lib.pa_qk_norm_rope(
        q.data_ptr(), qs, k.data_ptr(), ks, qw, kw, float(weight_bias), float(eps),
        cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, pos, T, hq, hkv, d,
        q_out.data_ptr(), qos, k_out.data_ptr(), kos, _stream()), "pa_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_cache(q, k, v, q_weight, k_weight, cos_sin, positions, eps, k_cache, v_cache,
                       slot_mapping, interleaved=False, weight_bias=0.0, q_out=None):
    """qk_norm_rope with the KV write in the same launch: the keys, and the values v as they
    are, go to their slots of the caches (see pa_qk_norm_rope_cache), BF16 [num_pages,
    block_size, Hkv, D] or 4-bit (uint8, q4_cache_shape).  Returns q_out."""
    lib, dev = _lib or load(), _device()
    T, hq, hkv, d, qs, ks, qw, kw, rows, rot = _rope_args(q, k, q_weight, k_weight, cos_sin, dev)
    pos = _vector(positions, "positions", _I32, T, dev)
    vs, slots, fmt, pages, ps, bs = _rope_cache(v, k_cache, v_cache, slot_mapping, T, hkv, d, dev)
    q_out, qos = _rope_q_out(q_out, q, T, hq, d, dev)
    _raise(lib.pa_qk_norm_rope_cache(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, float(weight_bias),
        float(eps), cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, pos, T, hq, hkv, d,
        q_out.data_ptr(), qos, fmt, k_cache.data_ptr(), v_cache.data_ptr(), ps, pages, slots, bs,
        _stream()), "pa_qk_norm_rope_cache")
    return q_out


def mrope_axes(sections, in_turn=False):
    """The axis of each frequency, for qk_norm_mrope: sections[a] frequencies turn by axis a.
    In runs, axis after axis; or in turn, frequency i by axis i % len(sections) while that axis
    has frequencies left, and by axis 0 afterwards."""
    n, count = sum(sections), len(sections)
    if in_turn:
        return bytes(i % count if i // count < sections[i % count] else 0 for i in range(n))
    return bytes(a for a, m in enumerate(sections) for _ in range(m))


def _axis_rows(positions, axes, T, rot, dev):
    """(address of the positions, distance between axes, axes, the frequencies' axes as bytes)"""
    n, tokens = _need(positions, "positions", _I32, 2, dev)
    row, col = positions.stride()
    if tokens != T or not 1 <= n <= 4 or (col != 1 and T > 1):
        raise ValueError(f"positions must be [axes, {T}], 1 to 4 axes, each row contiguous")
    axes = bytes(axes)
    if len(axes) != rot // 2:
        raise ValueError(f"axes must have an entry for each of {rot // 2} frequencies")
    return positions.data_ptr(), row if n > 1 else T, n, axes


def qk_norm_mrope(q, k, q_weight, k_weight, cos_sin, positions, axes, eps, interleaved=False,
                  weight_bias=0.0, q_out=None, k_out=None):
    """qk_norm_rope with positions on several axes (see pa_qk_norm_mrope): positions int32 [axes,
    T], axes the axis of each of the rotary_dim / 2 frequencies (bytes or ints, see mrope_axes).
    Returns (q_out, k_out)."""
    if q_out is None and k_out is None:
        r = (_bind or _short()).mrope(q, k, q_weight, k_weight, cos_sin, positions, axes, eps,
                                      interleaved, weight_bias)
        if r is not None:
            return r if type(r) is tuple else _raise(r, "pa_qk_norm_mrope")
    lib, dev = _lib or load(), _device()
    T, hq, hkv, d, qs, ks, qw, kw, rows, rot = _rope_args(q, k, q_weight, k_weight, cos_sin, dev)
    pos, stride, n, axes = _axis_rows(positions, axes, T, rot, dev)
    q_out, qos = _rope_q_out(q_out, q, T, hq, d, dev)
    if k_out is None:
        k_out = torch.empty((T, hkv, d), dtype=_BF16, device=k.device)
    kos = _token_rows(k_out, "k_out", T, hkv, d, dev)
    _raise(lib.pa_qk_norm_mrope(
        q.data_ptr(), qs, k.data_ptr(), ks, qw, kw, float(weight_bias), float(eps),
        cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, pos, stride, n, axes, T, hq, hkv, d,
        q_out.data_ptr(), qos, k_out.data_ptr(), kos, _stream()), "pa_qk_norm_mrope")
    return q_out, k_out


def qk_norm_mrope_cache(q, k, v, q_weight, k_weight, cos_sin, positions, axes, eps, k_cache,
                        v_cache, slot_mapping, interleaved=False, weight_bias=0.0, q_out=None):
    """qk_norm_rope_cache with positions on several axes (see qk_norm_mrope).  Returns q_out."""
    if q_out is None:
        r = (_bind or _short()).mrope_cache(q, k, q_weight, k_weight, cos_sin, positions, axes, eps,
                                            interleaved, weight_bias, v, k_cache, v_cache, slot_mapping)
        if r is not None:
            return r if type(r) is not int else _raise(r, "pa_qk_norm_mrope_cache")
    lib, dev = _lib or load(), _device()
    T, hq, hkv, d, qs, ks, qw, kw, rows, rot = _rope_args(q, k, q_weight, k_weight, cos_sin, dev)
    pos, stride, n, axes = _axis_rows(positions, axes, T, rot, dev)
    vs, slots, fmt, pages, ps, bs = _rope_cache(v, k_cache, v_cache, slot_mapping, T, hkv, d, dev)
    q_out, qos = _rope_q_out(q_out, q, T, hq, d, dev)
    _raise(lib.pa_qk_norm_mrope_cache(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, qw, kw, float(weight_bias),
        float(eps), cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, pos, stride, n, axes, T,
        hq, hkv, d, q_out.data_ptr(), qos, fmt, k_cache.data_ptr(), v_cache.data_ptr(), ps, pages,
        slots, bs, _stream()), "pa_qk_norm_mrope_cache")
    return q_out


def q4_cache_shape(num_pages, block_size, num_kv_heads):
    """Shape of a 4-bit K or V cache (uint8; see pa.h for its bytes)."""
    return (num_pages, num_kv_heads, block_size * Q4_ROW_BYTES)


def _q4_cache(k_cache, v_cache, dev):
    """(pages, page stride in bytes, block size, KV heads) of a pair of 4-bit caches."""
    shape = _need(k_cache, "k_cache", _U8, 3, dev)
    pages, heads, run = shape
    stride = k_cache.stride()
    if _need(v_cache, "v_cache", _U8, 3, dev) != shape or \
            (v_cache.stride() != stride and not (k_cache.is_contiguous() and
                                                 v_cache.is_contiguous())):
        raise ValueError("k_cache and v_cache must have the same shape and page stride")
    if run % Q4_ROW_BYTES or run == 0 or stride[2] != 1 or (heads > 1 and stride[1] != run):
        raise ValueError("each page of a 4-bit cache must be a contiguous [Hkv, block_size * "
                         f"{Q4_ROW_BYTES}] block of bytes")
    return pages, stride[0] if pages > 1 else heads * run, run // Q4_ROW_BYTES, heads


def reshape_and_cache_q4(key, value, k_cache, v_cache, slot_mapping):
    """Quantise key/value [T, Hkv, 256] into the 4-bit caches at slot_mapping (in place)."""
    lib, dev = _lib or load(), _device()
    pages, ps, bs, hkv = _q4_cache(k_cache, v_cache, dev)
    T, heads, dim = _need(key, "key", _BF16, 3, dev)
    if heads != hkv or dim != 256:
        raise ValueError(f"key must be [{T}, {hkv}, 256], got [{T}, {heads}, {dim}]")
    ks = _row_stride(key, "key", T, hkv, 256)
    vs = _token_rows(value, "value", T, hkv, 256, dev)
    _raise(lib.pa_reshape_and_cache_q4(
        key.data_ptr(), ks, value.data_ptr(), vs, k_cache.data_ptr(), v_cache.data_ptr(), ps,
        pages, _vector(slot_mapping, "slot_mapping", _I64, T, dev), T, hkv, 256, bs, _stream()),
        "pa_reshape_and_cache_q4")


def _gather_out(t, name, tokens, heads, like, dev):
    if t is None:
        return torch.empty((tokens, heads, 256), dtype=_BF16, device=like.device)
    if _need(t, name, _BF16, 3, dev) != (tokens, heads, 256) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [T, Hkv, 256] tensor")
    return t


def gather_cache_q4(k_cache, v_cache, slot_mapping, k_out=None, v_out=None):
    """The tokens at slot_mapping [T] as BF16 (k, v), each [T, Hkv, 256]; zeros for negative
    slots."""
    lib, dev = _lib or load(), _device()
    pages, ps, bs, hkv = _q4_cache(k_cache, v_cache, dev)
    slots = _vector(slot_mapping, "slot_mapping", _I64, None, dev)
    T = slot_mapping.shape[0]
    k_out = _gather_out(k_out, "k_out", T, hkv, k_cache, dev)
    v_out = _gather_out(v_out, "v_out", T, hkv, v_cache, dev)
    _raise(lib.pa_gather_cache_q4(k_cache.data_ptr(), v_cache.data_ptr(), ps, pages, slots, T, hkv,
                                  256, bs, k_out.data_ptr(), v_out.data_ptr(), _stream()),
           "pa_gather_cache_q4")
    return k_out, v_out


def decode_q4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             max_seq_len) -> int:
    return int(load().pa_decode_q4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                  block_size, _i32(max_seq_len, "max_seq_len")))


def _q4_out(out, q, dev):
    if out is None:
        return torch.empty_like(q)
    if _need(out, "out", _BF16, 3, dev) != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous BF16 tensor shaped like q")
    return out


def _q4_workspace(workspace, need, dev, device):
    """(tensor, address, bytes) of a caller's workspace, or of a fresh one of need() bytes."""
    if workspace is None:
        workspace = torch.empty(max(need(), 256), dtype=_U8, device=device)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or \
            not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on the current CUDA device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def decode_q4(q, k_cache, v_cache, block_table, seq_lens, scale, max_seq_len, out=None,
              workspace=None):
    """q=1 decode over the 4-bit cache (see pa_decode_q4): row s of q [S, Hq, 256] attends to
    sequence s of seq_lens [S] and of block_table (S rows or more).  Returns out [S, Hq, 256]
    BF16; rows of sequences of length 0 are zeros.  (A step's tokens are packed: with idle entries
    before others, row t belongs to sequence seq_idx[t] instead, and is moved there first.)"""
    lib, dev = _lib or load(), _device()
    S, hq, d = _need(q, "q", _BF16, 3, dev)
    q = q.contiguous()
    pages, ps, bs, hkv = _q4_cache(k_cache, v_cache, dev)
    width, row = _table(block_table, "block_table", S, dev)
    lens = _vector(seq_lens, "seq_lens", _I32, S, dev)  # one entry per row of q
    max_seq_len = _i32(max_seq_len, "max_seq_len")
    if width * bs < max_seq_len:
        raise ValueError("block_table rows are too short for max_seq_len")
    out = _q4_out(out, q, dev)
    _keep, ws, ws_bytes = _q4_workspace(
        workspace, lambda: decode_q4_workspace_size(S, hq, hkv, d, bs, max_seq_len), dev, q.device)
    _raise(lib.pa_decode_q4(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ps, pages,
                            block_table.data_ptr(), row, lens, S, max_seq_len,
                            hq, hkv, d, bs, float(scale), out.data_ptr(), ws, ws_bytes, _stream()),
           "pa_decode_q4")
    return out


def prefill_q4_workspace_size(q_len, q_start, causal, num_q_heads, num_kv_heads, head_dim,
                              block_size) -> int:
    """Bytes of workspace for prefill_chunk_q4 (the expanded operands, and room for split items)."""
    return int(load().pa_prefill_q4_workspace_size(_i32(q_len, "q_len"), _i32(q_start, "q_start"),
                                                   int(bool(causal)),
                                                   num_q_heads, num_kv_heads, head_dim,
                                                   block_size))


def prefill_chunk_q4(q, k_cache, v_cache, block_table, q_start, causal, scale, out=None,
                     workspace=None):
    """Causal (or full) chunk attention of one sequence over the 4-bit cache (see
    pa_prefill_chunk_q4).  Without a workspace, one of prefill_q4_workspace_size bytes is
    allocated for the call."""
    _check(q, "q", _BF16, 3)
    _check(block_table, "block_table", _I32)
    bt = block_table.reshape(1, -1)
    return prefill_varlen_q4(q, k_cache, v_cache, bt, [0, q.shape[0]],
                             [int(q_start) + q.shape[0]], causal, scale, out, workspace)


def _varlen_lens(cu_seqlens_q, seq_lens_k):
    B = len(seq_lens_k)
    if len(cu_seqlens_q) != B + 1:
        raise ValueError("cu_seqlens_q: num_seqs + 1 offsets")
    return ((ctypes.c_int32 * (B + 1))(*[_i32(x, "cu_seqlens_q") for x in cu_seqlens_q]),
            (ctypes.c_int32 * max(B, 1))(*[_i32(x, "seq_lens_k") for x in seq_lens_k]), B)


def prefill_varlen_q4_workspace_size(cu_seqlens_q, seq_lens_k, causal, num_q_heads, num_kv_heads,
                                     head_dim, block_size) -> int:
    """Bytes of workspace for prefill_varlen_q4 (the expanded operands, and room for split items)."""
    cu, sk, B = _varlen_lens(cu_seqlens_q, seq_lens_k)
    return int(load().pa_prefill_varlen_q4_workspace_size(cu, sk, B, int(bool(causal)),
                                                          num_q_heads, num_kv_heads, head_dim,
                                                          block_size))


def prefill_varlen_q4(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, causal, scale,
                      out=None, workspace=None):
    """Chunks of several sequences stacked row-wise in q, over the 4-bit cache (see
    pa_prefill_varlen_q4).  cu_seqlens_q and seq_lens_k are host sequences of ints.  Without a
    workspace, one of prefill_varlen_q4_workspace_size bytes is allocated for the call."""
    lib, dev = _lib or load(), _device()
    rows, hq, d = _need(q, "q", _BF16, 3, dev)
    q = q.contiguous()
    pages, ps, bs, hkv = _q4_cache(k_cache, v_cache, dev)
    cu, sk, B = _varlen_lens(cu_seqlens_q, seq_lens_k)
    if cu[B] != rows:
        raise ValueError("cu_seqlens_q must end at q's row count")
    width, stride = _table(block_table, "block_table", B, dev)
    if B and width * bs < max(sk):
        raise ValueError("block_table rows are too short for the sequences' keys")
    out = _q4_out(out, q, dev)
    causal = 1 if causal else 0
    _keep, ws, ws_bytes = _q4_workspace(
        workspace, lambda: int(lib.pa_prefill_varlen_q4_workspace_size(cu, sk, B, causal, hq, hkv,
                                                                       d, bs)), dev, q.device)
    _raise(lib.pa_prefill_varlen_q4(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), ps, pages, block_table.data_ptr(),
        stride, cu, sk, B, causal, hq, hkv, d, bs, float(scale), out.data_ptr(), ws, ws_bytes,
        _stream()), "pa_prefill_varlen_q4")
    return out


def q8_cache_shapes(num_pages, block_size, num_kv_heads):
    """Shapes of an 8-bit K or V cache: its codes (float8_e4m3fn) and its scales (uint8)."""
    return ((num_pages, block_size, num_kv_heads, 256),
            (num_pages, -(-block_size // Q8_TOKENS), num_kv_heads))


def _q8_cache(k_cache, v_cache, k_scales, v_scales, dev):
    """(the four addresses, page stride and scale stride in bytes, pages), block size, KV heads of
    an 8-bit cache."""
    shape = _need(k_cache, "k_cache", _E4M3, 4, dev)
    pages, bs, heads, dim = shape
    stride = k_cache.stride()
    if _need(v_cache, "v_cache", _E4M3, 4, dev) != shape or \
            (v_cache.stride() != stride and not (k_cache.is_contiguous() and
                                                 v_cache.is_contiguous())):
        raise ValueError("k_cache and v_cache must have the same shape and page stride")
    if dim != 256 or stride[3] != 1 or (heads > 1 and stride[2] != 256) or \
            (bs > 1 and stride[1] != heads * 256):
        raise ValueError("each page of an 8-bit cache must be a contiguous [block_size, Hkv, 256] "
                         "block of codes")
    want = (pages, (bs - 1) // Q8_TOKENS + 1, heads)
    got = _need(k_scales, "k_scales", _U8, 3, dev)
    sstride = k_scales.stride()
    if got != want or _need(v_scales, "v_scales", _U8, 3, dev) != want or \
            (v_scales.stride() != sstride and not (k_scales.is_contiguous() and
                                                   v_scales.is_contiguous())) or \
            (heads > 1 and sstride[2] != 1) or (want[1] > 1 and sstride[1] != heads):
        raise ValueError(f"k_scales and v_scales must be {want}, each page contiguous, with the "
                         "same page stride")
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
            stride[0] if pages > 1 else bs * heads * 256, sstride[0] if pages > 1 else want[1] * heads,
            pages), bs, heads


def reshape_and_cache_q8(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping):
    """Quantise key/value [T, Hkv, 256] into the 8-bit caches at slot_mapping (in place; see
    pa_reshape_and_cache_q8 for how a block's scale follows its tokens)."""
    r = (_bind or _short()).write_q8(key, value, k_cache, v_cache, k_scales, v_scales, slot_mapping)
    if r is not None:
        return None if r is True else _raise(r, "pa_reshape_and_cache_q8")
    lib, dev = _lib or load(), _device()
    cache, bs, hkv = _q8_cache(k_cache, v_cache, k_scales, v_scales, dev)
    T, heads, dim = _need(key, "key", _BF16, 3, dev)
    if heads != hkv or dim != 256:
        raise ValueError(f"key must be [{T}, {hkv}, 256], got [{T}, {heads}, {dim}]")
    ks = _row_stride(key, "key", T, hkv, 256)
    vs = _token_rows(value, "value", T, hkv, 256, dev)
    _raise(lib.pa_reshape_and_cache_q8(
        key.data_ptr(), ks, value.data_ptr(), vs, *cache,
        _vector(slot_mapping, "slot_mapping", _I64, T, dev), T, hkv, 256, bs, _stream()),
        "pa_reshape_and_cache_q8")


def gather_cache_q8(k_cache, v_cache, k_scales, v_scales, slot_mapping, k_out=None, v_out=None):
    """The tokens at slot_mapping [T] as BF16 (k, v), each [T, Hkv, 256]; zeros for negative
    slots."""
    if k_out is None and v_out is None:
        r = (_bind or _short()).gather_q8(k_cache, v_cache, k_scales, v_scales, slot_mapping)
        if r is not None:
            return r if type(r) is tuple else _raise(r, "pa_gather_cache_q8")
    lib, dev = _lib or load(), _device()
    cache, bs, hkv = _q8_cache(k_cache, v_cache, k_scales, v_scales, dev)
    slots = _vector(slot_mapping, "slot_mapping", _I64, None, dev)
    T = slot_mapping.shape[0]
    k_out = _gather_out(k_out, "k_out", T, hkv, k_cache, dev)
    v_out = _gather_out(v_out, "v_out", T, hkv, v_cache, dev)
    _raise(lib.pa_gather_cache_q8(*cache, slots, T, hkv, 256, bs, k_out.data_ptr(),
                                  v_out.data_ptr(), _stream()), "pa_gather_cache_q8")
    return k_out, v_out


def decode_q8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                             max_seq_len) -> int:
    return int(load().pa_decode_q8_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                  block_size, _i32(max_seq_len, "max_seq_len")))


def decode_q8(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, scale, max_seq_len,
              out=None, workspace=None):
    """q=1 decode over the 8-bit cache (see pa_decode_q8): row s of q [S, Hq, 256] attends to
    sequence s of seq_lens [S] and of block_table (S rows or more).  Returns out [S, Hq, 256]
    BF16; rows of sequences of length 0 are zeros."""
    r = (_bind or _short()).decode_q8(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens,
                                      scale, max_seq_len, out, workspace)
    if r is not None:
        return r if type(r) is not int else _raise(r, "pa_decode_q8")
    lib, dev = _lib or load(), _device()
    S, hq, d = _need(q, "q", _BF16, 3, dev)
    q = q.contiguous()
    cache, bs, hkv = _q8_cache(k_cache, v_cache, k_scales, v_scales, dev)
    width, row = _table(block_table, "block_table", S, dev)
    lens = _vector(seq_lens, "seq_lens", _I32, S, dev)  # one entry per row of q
    max_seq_len = _i32(max_seq_len, "max_seq_len")
    if width * bs < max_seq_len:
        raise ValueError("block_table rows are too short for max_seq_len")
    out = _q4_out(out, q, dev)
    _keep, ws, ws_bytes = _q4_workspace(
        workspace, lambda: decode_q8_workspace_size(S, hq, hkv, d, bs, max_seq_len), dev, q.device)
    _raise(lib.pa_decode_q8(q.data_ptr(), *cache, block_table.data_ptr(), row, lens, S, max_seq_len,
                            hq, hkv, d, bs, float(scale), out.data_ptr(), ws, ws_bytes, _stream()),
           "pa_decode_q8")
    return out


def prefill_q8_workspace_size(q_len, q_start, causal, num_q_heads, num_kv_heads, head_dim,
                              block_size) -> int:
    """Bytes of workspace for prefill_chunk_q8 (the expanded operands, and room for split items)."""
    return int(load().pa_prefill_q8_workspace_size(_i32(q_len, "q_len"), _i32(q_start, "q_start"),
                                                   int(bool(causal)), num_q_heads, num_kv_heads,
                                                   head_dim, block_size))


def prefill_chunk_q8(q, k_cache, v_cache, k_scales, v_scales, block_table, q_start, causal, scale,
                     out=None, workspace=None):
    """Causal (or full) chunk attention of one sequence over the 8-bit cache (see
    pa_prefill_chunk_q8).  Without a workspace, one of prefill_q8_workspace_size bytes is
    allocated for the call."""
    _check(q, "q", _BF16, 3)
    _check(block_table, "block_table", _I32)
    bt = block_table.reshape(1, -1)
    return prefill_varlen_q8(q, k_cache, v_cache, k_scales, v_scales, bt, [0, q.shape[0]],
                             [int(q_start) + q.shape[0]], causal, scale, out, workspace)


def prefill_varlen_q8_workspace_size(cu_seqlens_q, seq_lens_k, causal, num_q_heads, num_kv_heads,
                                     head_dim, block_size) -> int:
    """Bytes of workspace for prefill_varlen_q8 (the expanded operands, and room for split items)."""
    cu, sk, B = _varlen_lens(cu_seqlens_q, seq_lens_k)
    return int(load().pa_prefill_varlen_q8_workspace_size(cu, sk, B, int(bool(causal)),
                                                          num_q_heads, num_kv_heads, head_dim,
                                                          block_size))


def prefill_varlen_q8(q, k_cache, v_cache, k_scales, v_scales, block_table, cu_seqlens_q,
                      seq_lens_k, causal, scale, out=None, workspace=None):
    """Chunks of several sequences stacked row-wise in q, over the 8-bit cache (see
    pa_prefill_varlen_q8).  cu_seqlens_q and seq_lens_k are host sequences of ints.  Without a
    workspace, one of prefill_varlen_q8_workspace_size bytes is allocated for the call."""
    r = (_bind or _short()).prefill_q8(q, k_cache, v_cache, k_scales, v_scales, block_table,
                                       cu_seqlens_q, seq_lens_k, causal, scale, out, workspace)
    if r is not None:
        return r if type(r) is not int else _raise(r, "pa_prefill_varlen_q8")
    lib, dev = _lib or load(), _device()
    rows, hq, d = _need(q, "q", _BF16, 3, dev)
    q = q.contiguous()
    cache, bs, hkv = _q8_cache(k_cache, v_cache, k_scales, v_scales, dev)
    cu, sk, B = _varlen_lens(cu_seqlens_q, seq_lens_k)
    if cu[B] != rows:
        raise ValueError("cu_seqlens_q must end at q's row count")
    width, stride = _table(block_table, "block_table", B, dev)
    if B and width * bs < max(sk):
        raise ValueError("block_table rows are too short for the sequences' keys")
    out = _q4_out(out, q, dev)
    causal = 1 if causal else 0
    _keep, ws, ws_bytes = _q4_workspace(
        workspace, lambda: int(lib.pa_prefill_varlen_q8_workspace_size(cu, sk, B, causal, hq, hkv,
                                                                       d, bs)), dev, q.device)
    _raise(lib.pa_prefill_varlen_q8(
        q.data_ptr(), *cache, block_table.data_ptr(), stride, cu, sk, B, causal, hq, hkv, d, bs,
        float(scale), out.data_ptr(), ws, ws_bytes, _stream()), "pa_prefill_varlen_q8")
    return out


def set_kernel_events(start, stop):
    """Measurement hook: the next decode / prefill_chunk call records these
    torch.cuda.Event objects around its main kernel (see pa_set_kernel_events)."""
    lib = load()
    for e in (start, stop):
        if not e.cuda_event:          # torch creates the CUDA event on first record
            e.record()
    _raise(lib.pa_set_kernel_events(ctypes.c_void_p(start.cuda_event),
                                    ctypes.c_void_p(stop.cuda_event)), "pa_set_kernel_events")


def device_errors(clear: bool = True) -> int:
    """Waits for the current stream and returns (and by default clears) the error bits.
    A bounded wait that ran out shows as DEVERR_TIMEOUT among them (the C call then
    returns PA_ERR_TIMEOUT, which is not raised here)."""
    lib = load()
    v = ctypes.c_uint(0)
    rc = lib.pa_get_device_errors(ctypes.byref(v), int(clear), _stream())
    if rc != ERR_TIMEOUT:
        _raise(rc, "pa_get_device_errors")
    return int(v.value)
