"""ctypes binding of libpagedkv.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
turns torch tensors into device pointers, passes the current CUDA stream and
raises on a non-OK status.  If the library is missing it raises: there is no
fallback path.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "pagedkv.h")

KV_BF16, KV_FP8_E4M3 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "workspace missing or too small",
          4: "CUDA error", 5: "device-side index or length error", 6: "device-side wait timed out",
          7: "no free cache block and none evictable", 8: "unknown (or already registered) sequence id"}
DEVERR_BLOCK_ID, DEVERR_LENGTH, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_RANGE = 1, 2, 4, 8, 16
DEVERR_NO_BLOCKS = 32

_lock = threading.Lock()
_lib = None


class PagedKVError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, 'unknown')} (status {status})")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


ROPE_MAX_PAIRS = 128


class RopeDesc(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("magnitude", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("inv_freq", ctypes.c_double * ROPE_MAX_PAIRS)]


def lib():
    """Load libpagedkv.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libpagedkv.so not found at {LIB_PATH}: build it first "
                                   "(`python -m paged_kv_decode_14_gb300.build`)")
            L = ctypes.CDLL(LIB_PATH)
            c = ctypes
            vp, i32, i64 = c.c_void_p, c.c_int32, c.c_int64
            L.pkv_paged_kv_append.restype = c.c_int
            L.pkv_paged_kv_append.argtypes = [c.POINTER(CacheDesc), vp, vp, vp, i64, vp, vp]
            L.pkv_attention_workspace_size.restype = c.c_size_t
            L.pkv_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
            L.pkv_workspace_init.restype = c.c_int
            L.pkv_workspace_init.argtypes = [vp, c.c_size_t, vp]
            L.pkv_paged_attention.restype = c.c_int
            L.pkv_paged_attention.argtypes = [c.POINTER(CacheDesc), vp, i32, vp, i32, vp, vp, i32, i32,
                                              c.c_float, vp, vp, c.c_size_t, i32, vp]
            L.pkv_paged_attention_noalloc.restype = c.c_int
            L.pkv_paged_attention_noalloc.argtypes = [c.POINTER(CacheDesc), vp, i32, vp, i32, vp, vp, i32, i32,
                                                      c.c_float, vp, i32, vp, vp]
            L.pkv_paged_prefill.restype = c.c_int
            L.pkv_paged_prefill.argtypes = [c.POINTER(CacheDesc), vp, i32, vp, i32, vp, vp, i32, i32, c.c_float, vp,
                                            vp, vp]
            L.pkv_kvmgr_create.restype = vp
            L.pkv_kvmgr_create.argtypes = [i64]
            L.pkv_kvmgr_destroy.restype = None
            L.pkv_kvmgr_destroy.argtypes = [vp]
            L.pkv_kvmgr_add_sequence.restype = c.c_int
            L.pkv_kvmgr_add_sequence.argtypes = [vp, i64, vp, i64, c.POINTER(i64), vp]
            L.pkv_kvmgr_append.restype = c.c_int
            L.pkv_kvmgr_append.argtypes = [vp, i64, vp, i64, vp, vp, c.POINTER(i32)]
            for nm in ("pkv_kvmgr_commit", "pkv_kvmgr_release"):
                getattr(L, nm).restype = c.c_int
                getattr(L, nm).argtypes = [vp, i64]
            L.pkv_kvmgr_fork.restype = c.c_int
            L.pkv_kvmgr_fork.argtypes = [vp, i64, i64]
            L.pkv_kvmgr_tables.restype = c.c_int
            L.pkv_kvmgr_tables.argtypes = [vp, vp, i32, i32, vp, vp]
            L.pkv_kvmgr_num_free.restype = i64
            L.pkv_kvmgr_num_free.argtypes = [vp]
            L.pkv_kvmgr_num_cached.restype = i64
            L.pkv_kvmgr_num_cached.argtypes = [vp]
            L.pkv_kvmgr_refcount.restype = i32
            L.pkv_kvmgr_refcount.argtypes = [vp, i32]
            L.pkv_cascade_workspace_size.restype = c.c_size_t
            L.pkv_cascade_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
            L.pkv_paged_attention_cascade.restype = c.c_int
            L.pkv_paged_attention_cascade.argtypes = [c.POINTER(CacheDesc), vp, i32, vp, i32, vp, vp, i32, i32, vp, vp,
                                                      i32, i32, c.c_float, vp, vp, c.c_size_t, vp]
            L.pkv_paged_kv_append_rope.restype = c.c_int
            L.pkv_paged_kv_append_rope.argtypes = [c.POINTER(CacheDesc), vp, vp, vp, i64, vp, c.c_float, vp, i32,
                                                   i32, vp, vp]
            pc = c.POINTER(CacheDesc)
            L.pkv_rope_init.restype = c.c_int
            L.pkv_rope_init.argtypes = [c.POINTER(RopeDesc), i32, i32, c.c_double, i32, c.c_double, i64, c.c_double,
                                        c.c_double]
            L.pkv_qk_norm_rope.restype = c.c_int
            L.pkv_qk_norm_rope.argtypes = [vp, vp, vp, vp, i32, i32, i64, vp, vp, i32, vp, vp, c.c_float, vp]
            L.pkv_paged_kv_append_norm_rope.restype = c.c_int
            L.pkv_paged_kv_append_norm_rope.argtypes = [pc, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, c.c_float,
                                                        i32, vp, vp]
            L.pkv_paged_kv_read.restype = c.c_int
            L.pkv_paged_kv_read.argtypes = [pc, vp, i32, vp, vp, i32, i64, vp, vp, i32, vp, vp]
            L.pkv_prompt_workspace_size.restype = c.c_size_t
            L.pkv_prompt_workspace_size.argtypes = []
            L.pkv_prompt_attention.restype = c.c_int
            L.pkv_prompt_attention.argtypes = [vp, vp, vp, vp, vp, i32, i32, i64, i64, vp, vp, vp, vp, i32, i32,
                                               c.c_float, vp, c.c_size_t, vp, vp]
            L.pkv_masked_workspace_size.restype = c.c_size_t
            L.pkv_masked_workspace_size.argtypes = []
            masked = [vp, vp, vp, vp, i64, vp, i32, vp, vp, vp, i32, i32]
            L.pkv_paged_attention_window.restype = c.c_int
            L.pkv_paged_attention_window.argtypes = masked + [i32, i32, c.c_float, vp, c.c_size_t, vp]
            L.pkv_paged_attention_tree.restype = c.c_int
            L.pkv_paged_attention_tree.argtypes = masked + [vp, i32, c.c_float, vp, c.c_size_t, vp]
            L.pkv_block_tables_update.restype = L.pkv_block_tables_update_padded.restype = c.c_int
            L.pkv_block_tables_update.argtypes = L.pkv_block_tables_update_padded.argtypes = [vp, i32, vp, vp, i32, vp, vp, i64, vp, vp, vp, vp, i64, vp, vp]
            L.pkv_paged_kv_keep_path.restype = c.c_int
            L.pkv_paged_kv_keep_path.argtypes = [vp, vp, i32, vp, vp, vp, i32, vp, i32, vp, vp]
            L.pkv_copy_blocks.restype = c.c_int
            L.pkv_copy_blocks.argtypes = [c.POINTER(CacheDesc), vp, i32, vp, vp, vp]
            L.pkv_debug_set_wait_limit.restype = None
            L.pkv_debug_set_wait_limit.argtypes = [c.c_uint64, vp]
            L.pkv_read_device_error.restype = c.c_int
            L.pkv_read_device_error.argtypes = [vp, c.POINTER(i32), vp]
            L.pkv_status_string.restype = c.c_char_p
            L.pkv_status_string.argtypes = [c.c_int]
            L.pkv_version.restype = c.c_char_p
            L.pkv_version.argtypes = []
            _lib = L
    return _lib


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


class PagedKVCache:
    """A paged K/V cache in the library's layout: two device buffers of
    [num_blocks][num_kv_heads][16 * head_dim] elements (bf16 or e4m3 bytes),
    plus the per-(block, kv-head) fp32 scales of an FP8 cache."""

    def __init__(self, num_blocks: int, num_kv_heads: int, head_dim: int, kv_dtype: str = "bf16",
                 device="cuda", k=None, v=None, k_scales=None, v_scales=None):
        self.num_blocks, self.num_kv_heads, self.head_dim = num_blocks, num_kv_heads, head_dim
        self.kv_dtype = kv_dtype
        tdt = torch.uint8 if kv_dtype == "fp8" else torch.bfloat16
        shape = (num_blocks, num_kv_heads, 16 * head_dim)
        self.k = k if k is not None else torch.empty(shape, dtype=tdt, device=device)
        self.v = v if v is not None else torch.empty(shape, dtype=tdt, device=device)
        self.k_scales, self.v_scales = k_scales, v_scales
        if kv_dtype == "fp8" and (k_scales is None or v_scales is None):
            raise ValueError("an FP8 cache needs k_scales and v_scales")

    def desc(self) -> CacheDesc:
        for t in (self.k, self.v):
            if not t.is_contiguous():
                raise ValueError("cache buffers must be contiguous")
        for t in (self.k_scales, self.v_scales):
            if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()):
                raise ValueError("scales must be contiguous float32")
        return CacheDesc(self.num_blocks, 16, self.num_kv_heads, self.head_dim,
                         KV_FP8_E4M3 if self.kv_dtype == "fp8" else KV_BF16,
                         self.k.data_ptr(), self.v.data_ptr(),
                         None if self.k_scales is None else self.k_scales.data_ptr(),
                         None if self.v_scales is None else self.v_scales.data_ptr())


def _check(st: int, what: str):
    if st != 0:
        raise PagedKVError(st, what)


def append(cache: PagedKVCache, k_new, v_new, slot_mapping, device_error=None, stream=None):
    """pkv_paged_kv_append: k_new/v_new bf16 [T, Hkv, D], slot_mapping int64 [T]."""
    for t in (k_new, v_new):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("k_new / v_new must be contiguous bfloat16")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    d = cache.desc()
    st = lib().pkv_paged_kv_append(ctypes.byref(d), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                   int(slot_mapping.numel()), _ptr(device_error), _stream(stream))
    _check(st, "pkv_paged_kv_append")


def append_rope(cache: PagedKVCache, k_new, v_new, slot_mapping, positions=None, theta: float = 10000.0, q=None,
                fp8_scales_from_values: bool = False, device_error=None, stream=None):
    """pkv_paged_kv_append_rope: append with K rotated at `positions` (int32
    [T], None = no rotation), q rows [T, Hq, D] rotated in place, and
    optionally the FP8 scales of the blocks this call starts chosen from the
    values (written into cache.k_scales / v_scales)."""
    for t in (k_new, v_new):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("k_new / v_new must be contiguous bfloat16")
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if positions is not None and (positions.dtype != torch.int32 or not positions.is_contiguous()):
        raise ValueError("positions must be contiguous int32")
    if q is not None and (q.dtype != torch.bfloat16 or not q.is_contiguous()):
        raise ValueError("q must be contiguous bfloat16")
    d = cache.desc()
    st = lib().pkv_paged_kv_append_rope(ctypes.byref(d), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                        int(slot_mapping.numel()), _ptr(positions), float(theta), _ptr(q),
                                        int(q.shape[1]) if q is not None else 0, int(bool(fp8_scales_from_values)),
                                        _ptr(device_error), _stream(stream))
    _check(st, "pkv_paged_kv_append_rope")


def workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_q_len, num_ctas=0) -> int:
    n = lib().pkv_attention_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_q_len, num_ctas)
    if n == 0:
        raise PagedKVError(1, "pkv_attention_workspace_size")
    return int(n)


def make_workspace(num_seqs, num_q_heads, num_kv_heads, head_dim, max_q_len, num_ctas=0, device="cuda",
                   stream=None):
    n = workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_q_len, num_ctas)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _check(lib().pkv_workspace_init(_ptr(ws), n, _stream(stream)), "pkv_workspace_init")
    return ws


def workspace_init(workspace, stream=None):
    """pkv_workspace_init: zero a workspace (needed once, and after a timeout)."""
    _check(lib().pkv_workspace_init(_ptr(workspace), int(workspace.numel()), _stream(stream)), "pkv_workspace_init")


def attention(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, scale: float,
              workspace, out=None, num_ctas: int = 0, stream=None):
    """pkv_paged_attention: q bf16 [sum q_lens, Hq, D] -> out bf16 of the same shape."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be contiguous bfloat16 [rows, Hq, D]")
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"), (q_lens, "q_lens")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    if out is None:
        out = torch.empty_like(q)
    d = cache.desc()
    st = lib().pkv_paged_attention(ctypes.byref(d), _ptr(q), int(q.shape[1]), _ptr(block_tables),
                                   int(block_tables.shape[1]), _ptr(context_lens), _ptr(q_lens),
                                   int(context_lens.numel()), int(max_q_len), float(scale), _ptr(out),
                                   _ptr(workspace), int(workspace.numel()), int(num_ctas), _stream(stream))
    _check(st, "pkv_paged_attention")
    return out


def make_cascade_workspace(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_q_len, max_group_q_len,
                           device="cuda", stream=None):
    n = lib().pkv_cascade_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, max_q_len,
                                         max_group_q_len)
    if n == 0:
        raise PagedKVError(1, "pkv_cascade_workspace_size")
    ws = torch.empty(int(n), dtype=torch.uint8, device=device)
    _check(lib().pkv_workspace_init(_ptr(ws), int(n), _stream(stream)), "pkv_workspace_init")
    return ws


def attention_cascade(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, group_starts,
                      group_prefix_lens, max_group_q_len: int, scale: float, workspace, out=None, stream=None):
    """pkv_paged_attention_cascade: attention with each group's shared prefix
    attended once for the whole group (group_starts int32 [G + 1],
    group_prefix_lens int32 [G], device)."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be contiguous bfloat16 [rows, Hq, D]")
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"), (q_lens, "q_lens"),
                    (group_starts, "group_starts"), (group_prefix_lens, "group_prefix_lens")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    if out is None:
        out = torch.empty_like(q)
    d = cache.desc()
    st = lib().pkv_paged_attention_cascade(ctypes.byref(d), _ptr(q), int(q.shape[1]), _ptr(block_tables),
                                           int(block_tables.shape[1]), _ptr(context_lens), _ptr(q_lens),
                                           int(context_lens.numel()), int(max_q_len), _ptr(group_starts),
                                           _ptr(group_prefix_lens), int(group_prefix_lens.numel()),
                                           int(max_group_q_len), float(scale), _ptr(out), _ptr(workspace),
                                           int(workspace.numel()), _stream(stream))
    _check(st, "pkv_paged_attention_cascade")
    return out


def attention_noalloc(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, scale: float,
                      out=None, num_ctas: int = 0, device_error=None, stream=None):
    """pkv_paged_attention_noalloc: like attention(), with the library's static
    scratch array instead of a caller workspace (for callers that cannot
    allocate device memory).  Calls that overlap on the GPU race."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be contiguous bfloat16 [rows, Hq, D]")
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"), (q_lens, "q_lens")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    if out is None:
        out = torch.empty_like(q)
    d = cache.desc()
    st = lib().pkv_paged_attention_noalloc(ctypes.byref(d), _ptr(q), int(q.shape[1]), _ptr(block_tables),
                                           int(block_tables.shape[1]), _ptr(context_lens), _ptr(q_lens),
                                           int(context_lens.numel()), int(max_q_len), float(scale), _ptr(out),
                                           int(num_ctas), _ptr(device_error), _stream(stream))
    _check(st, "pkv_paged_attention_noalloc")
    return out


def prefill(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, scale: float, out=None,
            device_error=None, stream=None):
    """pkv_paged_prefill: causal attention of long query windows (prompts or
    prompt chunks) on the tensor cores; q bf16 [sum q_lens, Hq, D] -> out of
    the same shape.  bf16 caches, Hq / Hkv dividing 128."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be contiguous bfloat16 [rows, Hq, D]")
    for t, name in ((block_tables, "block_tables"), (context_lens, "context_lens"), (q_lens, "q_lens")):
        if t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32")
    if out is None:
        out = torch.empty_like(q)
    d = cache.desc()
    st = lib().pkv_paged_prefill(ctypes.byref(d), _ptr(q), int(q.shape[1]), _ptr(block_tables),
                                 int(block_tables.shape[1]), _ptr(context_lens), _ptr(q_lens),
                                 int(context_lens.numel()), int(max_q_len), float(scale), _ptr(out),
                                 _ptr(device_error), _stream(stream))
    _check(st, "pkv_paged_prefill")
    return out


# ------------------------------------------------------------------ rows

_ROWS = struct.Struct("@Pqqi4x")            # pkv_rows
_CACHE = struct.Struct("@qiiiiPPPP")        # pkv_cache
_ROW_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "bands": 3, "ramp": 4}


class Rope:
    """A rotation (pkv_rope_init): the first `rotary_dim` dimensions of a head,
    in pairs (i, i + rotary_dim / 2) or, interleaved, (2i, 2i + 1), with
    frequencies theta^(-2i / rotary_dim) scaled by one of ROPE_SCALINGS.
    `inv_freq` and `magnitude` are the values in use."""

    def __init__(self, rotary_dim: int, theta: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_len: int = 0, low: float = 1.0, high: float = 4.0):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        self.desc = RopeDesc()
        _check(lib().pkv_rope_init(ctypes.byref(self.desc), int(rotary_dim), int(bool(interleaved)), float(theta),
                                   ROPE_SCALINGS[scaling], float(factor), int(original_len), float(low), float(high)),
               "pkv_rope_init")
        self._ref = ctypes.addressof(self.desc)

    @property
    def rotary_dim(self) -> int:
        return int(self.desc.rotary_dim)

    @property
    def magnitude(self) -> float:
        return float(self.desc.magnitude)

    @property
    def inv_freq(self):
        return list(self.desc.inv_freq[:self.rotary_dim // 2])


def _row_view(t, name, dtype, device, shape):
    """pkv_rows of t, of the given [tokens, heads, dim] (any strides but the last)."""
    strides = t.stride()
    if t.shape != shape or t.dtype is not dtype or strides[2] != 1 or t.get_device() != device:
        raise ValueError(f"{name} must be {list(shape)} in {dtype} on the same GPU, with consecutive elements in a "
                         f"row: got {list(t.shape)} in {t.dtype}, strides {list(strides)}")
    return _ROWS.pack(t.data_ptr(), strides[0], strides[1], shape[1])


def _new(stream, make, *args, **kw):
    """make(...), the memory belonging to the stream that will write it: memory of another stream
    could be handed out while that stream's earlier work still reads it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _row_output(t, name, like, dtype, device, shape, stream):
    """(output, its pkv_rows): t, or a new contiguous tensor of the shape."""
    if t is not None:
        return t, _row_view(t, name, dtype, device, shape)
    t = _new(stream, torch.empty_like, like, memory_format=torch.contiguous_format)
    return t, _ROWS.pack(t.data_ptr(), shape[1] * shape[2], shape[2], shape[1])


def _vector(t, name, dtype, device, numel):
    if t.dtype is not dtype or t.numel() != numel or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be {numel} contiguous {dtype} values on the same GPU")
    return t.data_ptr()


def _weight(t, name, dtype, device, dim):
    return None if t is None else _vector(t, name, dtype, device, dim)


def _error_word(t, device):
    return None if t is None else _vector(t, "device_error", torch.int32, device, 1)


def _device_of(t, name):
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on a GPU")
    return device


def _call(name, device, stream, *args):
    """Entry point `name` with the tensors' device current and, unless a stream
    is given, on that device's current stream."""
    fn = getattr(_lib or lib(), name)
    if device != torch.cuda.current_device():
        with torch.cuda.device(device):
            st = fn(*args, _stream(stream))
    else:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else int(stream.cuda_stream))
    if st != 0:
        raise PagedKVError(st, name)


def _check_norm_rope(q_weight, k_weight, eps, rope, positions):
    if eps is None:
        if q_weight is not None or k_weight is not None:
            raise ValueError("weights without eps")
    elif not eps >= 0:
        raise ValueError("eps must not be negative")
    if rope is not None and positions is None:
        raise ValueError("rope without positions")


def _check_cache_device(cache, device):
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        if t is not None and t.get_device() != device:
            raise ValueError("the cache must be on the same GPU as the other tensors")


def qk_norm_rope(q, k=None, positions=None, rope: Rope | None = None, q_weight=None, k_weight=None, eps=None,
                 q_out=None, k_out=None, inverse: bool = False, stream=None):
    """pkv_qk_norm_rope: query rows q [T, Hq, D] and key rows k [T, Hkv, D]
    (views of a fused projection are fine; bf16, fp16 or fp32), normed per head
    where eps is given, rotated at int32 positions [T] where rope is.  Returns
    (q_out, k_out): new tensors unless given (q_out=q: in place)."""
    device, dtype, shape = _device_of(q, "q"), q.dtype, q.shape
    if len(shape) != 3 or dtype not in _ROW_DTYPES:
        raise ValueError("q must be [tokens, heads, head_dim] in bfloat16, float16 or float32")
    T, _, D = shape
    _check_norm_rope(q_weight, k_weight, eps, rope, positions)
    qr = _row_view(q, "q", dtype, device, shape)
    q_out, qo = _row_output(q_out, "q_out", q, dtype, device, shape, stream)
    kr = ko = None
    if k is not None:
        kshape = (T, k.shape[1] if k.dim() == 3 else 0, D)
        kr = _row_view(k, "k", dtype, device, kshape)
        k_out, ko = _row_output(k_out, "k_out", k, dtype, device, kshape, stream)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call("pkv_qk_norm_rope", device, stream, qr, qo, kr, ko, _ROW_DTYPES[dtype], D, T,
          None if positions is None else _vector(positions, "positions", torch.int32, device, T),
          None if rope is None else rope._ref, inverse, _weight(q_weight, "q_weight", dtype, device, D),
          _weight(k_weight, "k_weight", dtype, device, D), -1.0 if eps is None else eps)
    return q_out, k_out


def append_norm_rope(cache: PagedKVCache, q, k, v, slot_mapping, positions=None, rope: Rope | None = None,
                     q_weight=None, k_weight=None, eps=None, q_out=None, k_out=None,
                     fp8_scales_from_values: bool = False, device_error=None, stream=None):
    """pkv_paged_kv_append_norm_rope: the rows of a step normed and rotated as
    by qk_norm_rope (bf16), K and V written into their slots (int64 [T]).
    Returns q_out (a new tensor unless given; None for q=None).  k_out, if
    given, receives the normed and rotated key rows too."""
    device, bf16 = _device_of(k, "k"), torch.bfloat16
    T, D = k.shape[0], cache.head_dim
    kshape = (T, cache.num_kv_heads, D)
    _check_cache_device(cache, device)
    _check_norm_rope(q_weight, k_weight, eps, rope, positions)
    qr = qo = None
    if q is not None:
        qshape = (T, q.shape[1] if q.dim() == 3 else 0, D)
        qr = _row_view(q, "q", bf16, device, qshape)
        q_out, qo = _row_output(q_out, "q_out", q, bf16, device, qshape, stream)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _call("pkv_paged_kv_append_norm_rope", device, stream, ctypes.byref(cache.desc()), qr, qo,
          _row_view(k, "k", bf16, device, kshape), _row_view(v, "v", bf16, device, kshape),
          None if k_out is None else _row_view(k_out, "k_out", bf16, device, kshape),
          _vector(slot_mapping, "slot_mapping", torch.int64, device, T), T,
          None if positions is None else _vector(positions, "positions", torch.int32, device, T),
          None if rope is None else rope._ref, _weight(q_weight, "q_weight", bf16, device, D),
          _weight(k_weight, "k_weight", bf16, device, D), -1.0 if eps is None else eps,
          bool(fp8_scales_from_values), _error_word(device_error, device))
    return q_out


def read_cache(cache: PagedKVCache, block_tables, lens, num_rows: int, starts=None, dtype=torch.bfloat16, k_out=None,
               v_out=None, device_error=None, stream=None):
    """pkv_paged_kv_read: positions starts[b] .. starts[b] + lens[b] - 1 of each
    sequence (starts None: 0) as packed rows; num_rows >= sum(lens).  Returns
    (k, v) [num_rows, Hkv, D]: new tensors of `dtype` unless given."""
    device, n = _device_of(block_tables, "block_tables"), lens.numel()
    shape = (int(num_rows), cache.num_kv_heads, cache.head_dim)
    if k_out is None:
        k_out = _new(stream, torch.empty, shape, dtype=dtype if v_out is None else v_out.dtype, device=block_tables.device)
    dtype = k_out.dtype
    if dtype not in _ROW_DTYPES:
        raise ValueError("rows must be bfloat16, float16 or float32")
    v_out, vr = _row_output(v_out, "v_out", k_out, dtype, device, shape, stream)
    _check_cache_device(cache, device)
    if block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    _call("pkv_paged_kv_read", device, stream, ctypes.byref(cache.desc()),
          _vector(block_tables, "block_tables", torch.int32, device, block_tables.numel()), block_tables.shape[1],
          None if starts is None else _vector(starts, "starts", torch.int32, device, n),
          _vector(lens, "lens", torch.int32, device, n), n, shape[0], _row_view(k_out, "k_out", dtype, device, shape),
          vr, _ROW_DTYPES[dtype], _error_word(device_error, device))
    return k_out, v_out


def prompt_workspace_size() -> int:
    n = lib().pkv_prompt_workspace_size()
    if n == 0:
        raise PagedKVError(4, "pkv_prompt_workspace_size")
    return int(n)


def make_prompt_workspace(device="cuda"):
    """A workspace for prompt_attention on the given device (uninitialised:
    it needs none)."""
    with torch.cuda.device(device):
        return torch.empty(prompt_workspace_size(), dtype=torch.uint8, device=device)


def prompt_attention(q, k, v, q_lens, kv_lens, max_q_len: int, scale: float, out=None, lse=None, q_starts=None,
                     kv_starts=None, workspace=None, device_error=None, stream=None):
    """pkv_prompt_attention: causal attention of packed prompts over key and
    value rows (bf16 or fp16; q [Tq, Hq, D], k and v [Tk, Hkv, D], views are
    fine).  Returns (out, lse): new tensors unless given; lse fp32 [Tq, Hq],
    natural logarithm.  With starts, rows outside every sequence are not
    written.  Without a workspace (make_prompt_workspace) a few rows over long
    contexts run on a few SMs only."""
    device, dtype, shape = _device_of(q, "q"), q.dtype, q.shape
    if len(shape) != 3 or (dtype is not torch.bfloat16 and dtype is not torch.float16):
        raise ValueError("q must be [rows, heads, head_dim] in bfloat16 or float16")
    (Tq, Hq, D), n = shape, q_lens.numel()
    kshape = (k.shape[0], k.shape[1] if k.dim() == 3 else 0, D)
    qr, kr = _row_view(q, "q", dtype, device, shape), _row_view(k, "k", dtype, device, kshape)
    vr = _row_view(v, "v", dtype, device, kshape)
    out, orow = _row_output(out, "out", q, dtype, device, shape, stream)
    if lse is None:
        lse = _new(stream, torch.empty, (Tq, Hq), dtype=torch.float32, device=q.device)
    if workspace is not None and (workspace.get_device() != device or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous on the same GPU")
    _call("pkv_prompt_attention", device, stream, qr, kr, vr, orow, _vector(lse, "lse", torch.float32, device, Tq * Hq),
          _ROW_DTYPES[dtype], D, Tq, kshape[0], _vector(q_lens, "q_lens", torch.int32, device, n),
          _vector(kv_lens, "kv_lens", torch.int32, device, n),
          None if q_starts is None else _vector(q_starts, "q_starts", torch.int64, device, n),
          None if kv_starts is None else _vector(kv_starts, "kv_starts", torch.int64, device, n), n, max_q_len, scale,
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel() * workspace.element_size(), _error_word(device_error, device))
    return out, lse


# ------------------------------------------------------------------ a step on the GPU


def make_masked_workspace(device="cuda", stream=None):
    """A workspace for attention_window and attention_tree on the given device, zeroed on its current stream (or
    `stream`): calls on other streams wait for that."""
    with torch.cuda.device(device):
        ws = _new(stream, torch.empty, int(lib().pkv_masked_workspace_size()), dtype=torch.uint8, device=device)
        workspace_init(ws, stream)
    return ws


def _cache_pack(cache, device):
    """pkv_cache of a cache on the given GPU."""
    k, v, ks, vs = cache.k, cache.v, cache.k_scales, cache.v_scales
    if k.get_device() != device or v.get_device() != device:
        raise ValueError("the cache must be on the same GPU as the other tensors")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("cache buffers must be contiguous")
    for t in (ks, vs):
        if t is not None and (t.dtype is not torch.float32 or not t.is_contiguous() or t.get_device() != device):
            raise ValueError("scales must be contiguous float32 on the same GPU")
    return _CACHE.pack(cache.num_blocks, 16, cache.num_kv_heads, cache.head_dim,
                       KV_FP8_E4M3 if cache.kv_dtype == "fp8" else KV_BF16, k.data_ptr(), v.data_ptr(),
                       0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr())


def _tables_of(block_tables, device, n):
    """Pointer and width of block_tables [n, width]."""
    if block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("block_tables must be [num_seqs, max_blocks_per_seq]")
    return _vector(block_tables, "block_tables", torch.int32, device, block_tables.numel()), block_tables.shape[1]


def _masked(cache, q, block_tables, context_lens, q_lens, workspace, out, lse, q_starts, stream):
    """(device, out, lse, the arguments that both masked attentions begin with, the workspace's)."""
    device, bf16, shape = _device_of(q, "q"), torch.bfloat16, q.shape
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise ValueError("q must be [rows, heads, head_dim of the cache]")
    n, rows, i32 = context_lens.numel(), shape[0], torch.int32
    qr = _row_view(q, "q", bf16, device, shape)
    out, orow = _row_output(out, "out", q, bf16, device, shape, stream)
    if lse is None:
        lse = _new(stream, torch.empty, (rows, shape[1]), dtype=torch.float32, device=q.device)
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the same GPU")
    args = (_cache_pack(cache, device), qr, orow, _vector(lse, "lse", torch.float32, device, rows * shape[1]), rows,
            *_tables_of(block_tables, device, n), _vector(context_lens, "context_lens", i32, device, n),
            _vector(q_lens, "q_lens", i32, device, n),
            None if q_starts is None else _vector(q_starts, "q_starts", torch.int64, device, n), n)
    return device, out, lse, args, (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def attention_window(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, window: int,
                     sinks: int, scale: float, workspace, out=None, lse=None, q_starts=None, stream=None):
    """pkv_paged_attention_window: attention over the cache in which a query sees the last `window` positions up to
    its own and the first `sinks`; q bf16 [rows, Hq, D] (views are fine), single tokens to prompts.  Returns
    (out, lse): new tensors unless given; lse fp32 [rows, Hq], natural logarithm.  With q_starts (int64
    [num_seqs]), rows outside every sequence are not written.  workspace: make_masked_workspace."""
    device, out, lse, args, ws = _masked(cache, q, block_tables, context_lens, q_lens, workspace, out, lse, q_starts,
                                         stream)
    _call("pkv_paged_attention_window", device, stream, *args, max_q_len, window, sinks, scale, *ws)
    return out, lse


def attention_tree(cache: PagedKVCache, q, block_tables, context_lens, q_lens, max_q_len: int, tree_mask,
                   scale: float, workspace, out=None, lse=None, q_starts=None, stream=None):
    """pkv_paged_attention_tree: attention of a tree of drafted tokens, whose keys and values are the last q_lens
    positions of each context: a row sees the context before them and the nodes whose bits are set in its row of
    tree_mask (int32 [rows, words], bit j % 32 of word j / 32).  Otherwise as attention_window."""
    device, out, lse, args, ws = _masked(cache, q, block_tables, context_lens, q_lens, workspace, out, lse, q_starts,
                                         stream)
    if tree_mask.dim() != 2 or tree_mask.shape[0] != q.shape[0]:
        raise ValueError("tree_mask must be [rows, words]")
    _call("pkv_paged_attention_tree", device, stream, *args, max_q_len,
          _vector(tree_mask, "tree_mask", torch.int32, device, tree_mask.numel()), tree_mask.shape[1], scale, *ws)
    return out, lse


class BlockPool:
    """The free blocks of a cache as a stack on the GPU (update_tables): `free` int32 [num_blocks], of which the first
    `count` (int32 [1]) are free.  Without them: all are, and 0 is taken first."""

    def __init__(self, num_blocks: int, device="cuda", free=None, count=None):
        if (free is None) != (count is None):
            raise ValueError("free and count go together")
        self.num_blocks = int(num_blocks)
        if free is None:
            free = torch.arange(self.num_blocks - 1, -1, -1, dtype=torch.int32, device=device)
            count = torch.full((1,), self.num_blocks, dtype=torch.int32, device=device)
        self.free, self.count = free, count
        at = _device_of(free, "free")
        _vector(free, "free", torch.int32, at, self.num_blocks)
        _vector(count, "count", torch.int32, at, 1)


def update_tables(pool: BlockPool, block_tables, context_lens, grow, num_rows: int, slots=None, positions=None,
                  granted=None, row_starts=None, device_error=None, stream=None, pad=None):
    """pkv_block_tables_update: requests grow by (or, negative, drop) grow tokens: block_tables, context_lens and the
    pool are updated in place.  num_rows >= sum(max(grow, 0)).  Returns (slots int64, positions int32 [num_rows],
    granted int32, row_starts int64 [num_seqs]), new tensors unless given: what an append and the attention of
    the new tokens take as slot_mapping, positions, q_lens and q_starts.
    pad (pkv_block_tables_update_padded): rows behind the last request's get slot -1, which appends skip, and
    position 0; else they are left as they were.  By default so where slots are new.  With slots given, say pad=True
    where num_rows is more than the rows there are and an append of all of them follows."""
    device, n, num_rows = _device_of(block_tables, "block_tables"), context_lens.numel(), int(num_rows)
    i32, i64 = torch.int32, torch.int64
    if num_rows < 0:
        raise ValueError("num_rows must not be negative")

    pad = slots is None if pad is None else pad

    def output(t, name, dtype, numel):
        if t is None:
            t = _new(stream, torch.empty, numel, dtype=dtype, device=block_tables.device)
            return t, t.data_ptr()
        return t, _vector(t, name, dtype, device, numel)

    slots, sp = output(slots, "slots", i64, num_rows)
    positions, pp = output(positions, "positions", i32, num_rows)
    granted, gp = output(granted, "granted", i32, n)
    row_starts, rp = output(row_starts, "row_starts", i64, n)
    _call("pkv_block_tables_update_padded" if pad else "pkv_block_tables_update", device, stream, *_tables_of(block_tables, device, n),
          _vector(context_lens, "context_lens", i32, device, n), _vector(grow, "grow", i32, device, n), n,
          _vector(pool.free, "pool.free", i32, device, pool.num_blocks), _vector(pool.count, "pool.count", i32, device, 1),
          pool.num_blocks, sp, pp, gp, rp, num_rows, _error_word(device_error, device))
    return slots, positions, granted, row_starts


def keep_path(cache: PagedKVCache, block_tables, context_lens, q_lens, path, path_lens, device_error=None, stream=None):
    """pkv_paged_kv_keep_path: the accepted nodes of each sequence's tree (path int32 [num_seqs, max_path], strictly
    ascending, path_lens int32 [num_seqs] of them) moved to the places behind the context, in the cache."""
    device, n, i32 = _device_of(block_tables, "block_tables"), context_lens.numel(), torch.int32
    if path.dim() != 2 or path.shape[0] != n:
        raise ValueError("path must be [num_seqs, max_path]")
    _call("pkv_paged_kv_keep_path", device, stream, _cache_pack(cache, device), *_tables_of(block_tables, device, n),
          _vector(context_lens, "context_lens", i32, device, n), _vector(q_lens, "q_lens", i32, device, n),
          _vector(path, "path", i32, device, path.numel()), path.shape[1],
          _vector(path_lens, "path_lens", i32, device, n), n, _error_word(device_error, device))


def read_device_error(error_word, stream=None) -> int:
    """Read and clear a device error word (workspace or append flag); syncs."""
    code = ctypes.c_int32(0)
    st = lib().pkv_read_device_error(_ptr(error_word), ctypes.byref(code), _stream(stream))
    if st not in (0, 5, 6):
        _check(st, "pkv_read_device_error")
    return int(code.value)


class KVManager:
    """The library's host-side block manager (pkv_kvmgr_*): block allocation,
    reference counts, copy-on-write and radix prefix reuse; it hands out the
    slots and block tables the append and attention calls take.  Host memory
    only (numpy arrays in and out)."""

    def __init__(self, num_blocks: int):
        self._lib = lib()
        self._h = self._lib.pkv_kvmgr_create(int(num_blocks))
        if not self._h:
            raise PagedKVError(1, "pkv_kvmgr_create")
        self.num_blocks = int(num_blocks)

    def close(self):
        if self._h:
            self._lib.pkv_kvmgr_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _i32(a):
        import numpy as np
        return np.ascontiguousarray(a, dtype=np.int32)

    def add_sequence(self, seq: int, tokens):
        """-> (cached_tokens, slots of the other prompt tokens: int64 array)."""
        import numpy as np
        t = self._i32(tokens)
        slots = np.zeros(len(t), dtype=np.int64)
        cached = ctypes.c_int64(0)
        _check(self._lib.pkv_kvmgr_add_sequence(self._h, int(seq), t.ctypes.data, len(t), ctypes.byref(cached),
                                                slots.ctypes.data), "pkv_kvmgr_add_sequence")
        return int(cached.value), slots[:len(t) - int(cached.value)].copy()

    def append(self, seq: int, tokens):
        """-> (slots: int64 array, copy-on-write pair (src, dst) or None)."""
        import numpy as np
        t = self._i32(tokens)
        slots = np.zeros(len(t), dtype=np.int64)
        copy = np.zeros(2, dtype=np.int32)
        ncopy = ctypes.c_int32(0)
        _check(self._lib.pkv_kvmgr_append(self._h, int(seq), t.ctypes.data, len(t), slots.ctypes.data,
                                          copy.ctypes.data, ctypes.byref(ncopy)), "pkv_kvmgr_append")
        return slots, (int(copy[0]), int(copy[1])) if ncopy.value else None

    def commit(self, seq: int):
        _check(self._lib.pkv_kvmgr_commit(self._h, int(seq)), "pkv_kvmgr_commit")

    def fork(self, parent: int, child: int):
        _check(self._lib.pkv_kvmgr_fork(self._h, int(parent), int(child)), "pkv_kvmgr_fork")

    def release(self, seq: int):
        _check(self._lib.pkv_kvmgr_release(self._h, int(seq)), "pkv_kvmgr_release")

    def tables(self, seqs, max_blocks: int):
        """-> (block_tables int32 [n, max_blocks] (-1 padded), context_lens int32 [n])."""
        import numpy as np
        s = np.ascontiguousarray(seqs, dtype=np.int64)
        bt = np.zeros((len(s), max_blocks), dtype=np.int32)
        lens = np.zeros(len(s), dtype=np.int32)
        _check(self._lib.pkv_kvmgr_tables(self._h, s.ctypes.data, len(s), int(max_blocks), bt.ctypes.data,
                                          lens.ctypes.data), "pkv_kvmgr_tables")
        return bt, lens

    def num_free(self) -> int:
        return int(self._lib.pkv_kvmgr_num_free(self._h))

    def num_cached(self) -> int:
        return int(self._lib.pkv_kvmgr_num_cached(self._h))

    def refcount(self, block: int) -> int:
        return int(self._lib.pkv_kvmgr_refcount(self._h, int(block)))


def copy_blocks(cache: PagedKVCache, pairs, stream=None):
    """pkv_copy_blocks: device int32 [n, 2] (src, dst) block pairs; an FP8
    cache's scales are copied too."""
    if pairs.dtype != torch.int32 or not pairs.is_contiguous():
        raise ValueError("pairs must be contiguous int32 [n, 2]")
    d = cache.desc()
    fp8 = cache.kv_dtype == "fp8"
    _check(lib().pkv_copy_blocks(ctypes.byref(d), _ptr(pairs), int(pairs.shape[0]),
                                 _ptr(cache.k_scales) if fp8 else None, _ptr(cache.v_scales) if fp8 else None,
                                 _stream(stream)), "pkv_copy_blocks")


def debug_set_wait_limit(limit_ns: int = 0, hold_flag=None):
    """Test hook of the timeout path (pkv_debug_set_wait_limit): the wait
    limit of later attention launches (0 = the default 2 s) and an optional
    device int32 flag the kernel waits on before its first K/V copy."""
    lib().pkv_debug_set_wait_limit(int(limit_ns), _ptr(hold_flag))


def version() -> str:
    return lib().pkv_version().decode()
