"""Python binding of libnvfp4kv.so, the NVFP4 paged KV cache library for GB300.

Argument marshalling only: every step of the cache paths runs in the CUDA
kernels behind the C ABI (include/nvfp4kv.h).  PyTorch provides device
memory and streams.  There is no CPU fallback: importing this package on a
machine without the built library, or calling it without a CUDA device,
raises.

The three paths of "Accelerating Long-Context and Agentic Inference with
NVFP4 KV Cache" (section A2):

  quantize_append(cache, k, v, slot_mapping)             paths 1 and 2 (write)
  paged_decode_attention(cache, q, block_table, seq_lens) path 3 (decode)
  prefix_dequant(cache, block_table, prefix_lens, cu)     path 2 (extend)

beside them a cache of latents (one shared vector a token) with its two
attention forms, and the eviction of cached tokens by accumulated attention
weight:

  latent_quantize_append, latent_decode_attention (absorbed form),
  latent_prefix_dequant, latent_extend_attention (expanded form)
  accumulate_attention_weights, evict
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libnvfp4kv.so")

DTYPE_NVFP4 = 0
DTYPE_FP8_E4M3 = 1
HEAD_DIM = 128
LATENT_DIM = 512
ROPE_DIM = 64

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported configuration", -3: "CUDA error",
          -4: "a kernel skipped an out-of-range index"}


class NVFP4KVError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" % (what, STATUS.get(status, "unknown"), status))
        self.status = status


class _CacheDesc(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_global_scale", ctypes.c_float), ("v_global_scale", ctypes.c_float)]


class _LatentDesc(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("global_scale", ctypes.c_float)]


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libnvfp4kv.so is not built; run __graft_entry__.build() (nvcc, sm_103a) first: %s"
                          % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    D = ctypes.POINTER(_CacheDesc)
    sig = {
        "nvfp4kv_version": (i32, []),
        "nvfp4kv_status_string": (ctypes.c_char_p, [i32]),
        "nvfp4kv_slab_bytes": (sz, [D]),
        "nvfp4kv_pool_bytes": (sz, [D]),
        "nvfp4_kv_quantize_append": (i32, [D, P, P, i64, i64, P, P]),
        "nvfp4kv_decode_workspace_bytes": (sz, [D, i32, i32, i32]),
        "nvfp4kv_decode_auto_splits": (i32, [D, i32]),
        "nvfp4kv_decode_launch_count": (i32, [D, i32, i32, i32, i32]),
        "nvfp4_paged_decode_attention": (i32, [D, P, i32, i32, P, i32, P, f32, P, P, sz, i32, P]),
        "nvfp4_prefix_dequant": (i32, [D, P, i32, P, P, i32, i64, P, P, P]),
        "nvfp4kv_check_device_errors": (i32, [P]),
        "nvfp4kv_selftest_bounded_wait": (i32, [i32, ctypes.c_uint, P, P]),
        "nvfp4kv_calibrate_global_scales": (i32, [P, P, i64, i32, i64, P, P]),
        "nvfp4_extend_attention": (i32, [P, P, P, P, i64, P, P, P, i64, i32, i32, i32, i32, f32, P, P]),
        "nvfp4_extend_attention_paged": (i32, [D, P, P, i32, P, P, P, P, i64, i32, i32, i32, f32, P, P]),
        "nvfp4_paged_decode_attention_append": (i32, [D, P, P, i64, P, i32, i32, P, i32, P, f32, P, P, sz, i32, P]),
        "nvfp4kv_cascade_workspace_bytes": (sz, [D, i32, i32, i32, i32]),
        "nvfp4_cascade_decode_attention": (i32, [D, P, i32, i32, P, i32, P, i32, P, f32, P, P, sz, i32, P]),
        "nvfp4kv_profile_decode": (i32, [P, P, i32, i32]),
        "nvfp4_paged_decode_attention_noalloc": (i32, [D, P, i32, i32, P, i32, P, f32, P, i32, P]),
        "nvfp4kv_latent_slab_bytes": (sz, [P]),
        "nvfp4_latent_quantize_append": (i32, [P, P, i64, P, i64, i64, P, P]),
        "nvfp4_latent_prefix_dequant": (i32, [P, P, i32, P, P, i32, i64, P, P, P]),
        "nvfp4kv_latent_decode_workspace_bytes": (sz, [P, i32, i32, i32]),
        "nvfp4_latent_decode_attention": (i32, [P, P, P, i32, i32, P, i32, P, f32, P, P, sz, i32, P]),
        "nvfp4_latent_extend_attention": (i32, [P, P, P, i64, i64, P, P, i64, P, P, i64, i64, P, P, i64, i32, i32, i32,
                                                f32, P, P]),
        "nvfp4kv_weights_workspace_bytes": (sz, [D, i32, i32]),
        "nvfp4_accumulate_attention_weights": (i32, [D, P, i32, i32, P, i32, P, f32, P, i64, P, sz, P]),
        "nvfp4_evict": (i32, [D, P, i64, i32, P, i32, P, P, i32, i32, i32, i32, P, P, P, i64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load_library()

EXPORTED_SYMBOLS = ("nvfp4kv_version", "nvfp4kv_status_string", "nvfp4kv_slab_bytes", "nvfp4kv_pool_bytes",
                    "nvfp4_kv_quantize_append", "nvfp4kv_decode_workspace_bytes", "nvfp4kv_decode_auto_splits",
                    "nvfp4kv_decode_launch_count",
                    "nvfp4_paged_decode_attention", "nvfp4_prefix_dequant", "nvfp4kv_check_device_errors",
                    "nvfp4kv_profile_decode", "nvfp4_paged_decode_attention_noalloc",
                    "nvfp4kv_selftest_bounded_wait", "nvfp4kv_calibrate_global_scales", "nvfp4_extend_attention",
                    "nvfp4_extend_attention_paged",
                    "nvfp4_paged_decode_attention_append", "nvfp4kv_cascade_workspace_bytes",
                    "nvfp4_cascade_decode_attention", "nvfp4kv_latent_slab_bytes", "nvfp4_latent_quantize_append",
                    "nvfp4_latent_prefix_dequant", "nvfp4kv_latent_decode_workspace_bytes",
                    "nvfp4_latent_decode_attention", "nvfp4_latent_extend_attention",
                    "nvfp4kv_weights_workspace_bytes", "nvfp4_accumulate_attention_weights", "nvfp4_evict")

NOALLOC_SCRATCH_BYTES = 64 << 20  # NVFP4KV_NOALLOC_SCRATCH_BYTES of the header


def library():
    """The loaded ctypes library (for tests of the raw ABI)."""
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        raise NVFP4KVError(rc, what)


def _stream(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr() if t is not None else 0)


def _require(t: torch.Tensor, name: str, dtype: torch.dtype):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


class PagedCache:
    """A caller-owned page pool (uint8 [num_pages][num_kv_heads][slab]) and its format."""

    def __init__(self, num_pages: int, page_size: int, num_kv_heads: int, dtype: int = DTYPE_NVFP4,
                 k_global_scale: float = 1.0, v_global_scale: float = 1.0, device="cuda",
                 pool: Optional[torch.Tensor] = None):
        self.num_pages, self.page_size, self.num_kv_heads = int(num_pages), int(page_size), int(num_kv_heads)
        self.dtype = int(dtype)
        self.k_global_scale, self.v_global_scale = float(k_global_scale), float(v_global_scale)
        slab = slab_bytes(self.dtype, self.page_size, self.num_kv_heads)
        self.slab = slab
        if pool is None:
            pool = torch.zeros((self.num_pages, self.num_kv_heads, slab), dtype=torch.uint8, device=device)
        _require(pool, "pool", torch.uint8)
        if pool.numel() != self.num_pages * self.num_kv_heads * slab:
            raise ValueError("pool has %d bytes, expected %d" % (pool.numel(), self.num_pages * self.num_kv_heads * slab))
        self.pool = pool
        self._desc = _CacheDesc(pool.data_ptr(), self.num_pages, self.page_size, self.num_kv_heads, HEAD_DIM,
                                self.dtype, self.k_global_scale, self.v_global_scale)

    @property
    def desc(self):
        return ctypes.byref(self._desc)

    @property
    def num_slots(self) -> int:
        return self.num_pages * self.page_size


def slab_bytes(dtype: int, page_size: int, num_kv_heads: int = 1) -> int:
    d = _CacheDesc(256, 1, page_size, num_kv_heads, HEAD_DIM, dtype, 1.0, 1.0)
    n = _lib.nvfp4kv_slab_bytes(ctypes.byref(d))
    if n == 0:
        raise NVFP4KVError(-2, "slab_bytes(dtype=%d, page_size=%d)" % (dtype, page_size))
    return int(n)


def quantize_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                    stream: Optional[torch.cuda.Stream] = None):
    """k, v: BF16 [T][Hkv][128] or [T][stride >= Hkv*128]; slot_mapping: int64 [T]."""
    T = int(slot_mapping.shape[0])
    _require(slot_mapping, "slot_mapping", torch.int64)
    row = cache.num_kv_heads * HEAD_DIM
    for name, x in (("k", k), ("v", v)):
        if not x.is_cuda or x.dtype != torch.bfloat16:
            raise ValueError("%s must be a CUDA bfloat16 tensor" % name)
        if x.shape[0] != T:
            raise ValueError("%s has %d tokens, slot_mapping %d" % (name, x.shape[0], T))
        # each token's Hkv*128 values contiguous; tokens may be strided (a view of a wider QKV buffer)
        if T > 0 and (not x[0].is_contiguous() or x[0].numel() != row):
            raise ValueError("%s: each token must hold %d contiguous values" % (name, row))
    stride = int(k.stride(0)) if T > 0 else row
    if T > 0 and int(v.stride(0)) != stride:
        raise ValueError("k and v must share a token stride")
    rc = _lib.nvfp4_kv_quantize_append(cache.desc, _ptr(k), _ptr(v), T, stride, _ptr(slot_mapping), _stream(stream))
    _check(rc, "nvfp4_kv_quantize_append")


def calibrate_global_scales(k: torch.Tensor, v: torch.Tensor, num_kv_heads: int,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Per-tensor FP32 global scales {g_K, g_V} = amax / (6 * 448) of BF16 K and V
    ([T][Hkv][128] or token-strided, as for quantize_append), as a device float32
    tensor [2] (1.0 for an all-zero tensor)."""
    T = int(k.shape[0])
    row = int(num_kv_heads) * HEAD_DIM
    for name, x in (("k", k), ("v", v)):
        if not x.is_cuda or x.dtype != torch.bfloat16:
            raise ValueError("%s must be a CUDA bfloat16 tensor" % name)
        if x.shape[0] != T:
            raise ValueError("k and v must have the same number of tokens")
        if T > 0 and (not x[0].is_contiguous() or x[0].numel() != row):
            raise ValueError("%s: each token must hold %d contiguous values" % (name, row))
    stride = int(k.stride(0)) if T > 0 else row
    if T > 0 and int(v.stride(0)) != stride:
        raise ValueError("k and v must share a token stride")
    scales = torch.empty(2, dtype=torch.float32, device=k.device)
    rc = _lib.nvfp4kv_calibrate_global_scales(_ptr(k), _ptr(v), T, int(num_kv_heads), stride, _ptr(scales),
                                              _stream(stream))
    _check(rc, "nvfp4kv_calibrate_global_scales")
    return scales


def decode_workspace_bytes(cache: PagedCache, batch: int, num_q_heads: int, num_splits: int = 0) -> int:
    n = _lib.nvfp4kv_decode_workspace_bytes(cache.desc, int(batch), int(num_q_heads), int(num_splits))
    if n == 0 and batch > 0:
        raise NVFP4KVError(-1, "decode_workspace_bytes")
    return int(n)


def decode_auto_splits(cache: PagedCache, num_q_heads: int) -> int:
    return int(_lib.nvfp4kv_decode_auto_splits(cache.desc, int(num_q_heads)))


def decode_launch_count(cache: PagedCache, batch: int, num_q_heads: int, num_splits: int = 0,
                        shared_len: int = 0) -> int:
    """Kernel launches of one decode (shared_len = 0) or cascade call of this shape."""
    return int(_lib.nvfp4kv_decode_launch_count(cache.desc, int(batch), int(num_q_heads), int(num_splits),
                                                int(shared_len)))


def alloc_decode_workspace(cache: PagedCache, batch: int, num_q_heads: int, num_splits: int = 0) -> torch.Tensor:
    n = decode_workspace_bytes(cache, batch, num_q_heads, num_splits)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.pool.device)


def paged_decode_attention(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                           sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, num_splits: int = 0,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """q: BF16 [B][Hq][128]; block_table int32 [B][max_pages]; seq_lens int32 [B] -> BF16 [B][Hq][128]."""
    _require(q, "q", torch.bfloat16)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    B, Hq = int(q.shape[0]), int(q.shape[1])
    if q.shape[2] != HEAD_DIM:
        raise ValueError("head_dim must be 128")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if out is None:
        out = torch.empty_like(q)
    _require(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = alloc_decode_workspace(cache, B, Hq, num_splits)
    _require(workspace, "workspace", torch.uint8)
    rc = _lib.nvfp4_paged_decode_attention(cache.desc, _ptr(q), B, Hq, _ptr(block_table), int(block_table.shape[1]),
                                           _ptr(seq_lens), float(sm_scale), _ptr(out), _ptr(workspace),
                                           workspace.numel(), int(num_splits), _stream(stream))
    _check(rc, "nvfp4_paged_decode_attention")
    return out


def paged_decode_attention_append(cache: PagedCache, k_new: torch.Tensor, v_new: torch.Tensor, q: torch.Tensor,
                                  block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: Optional[float] = None,
                                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                                  num_splits: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode step with the new token appended in the same launch: row b of
    k_new / v_new (BF16 [B][Hkv][128], or token-strided) is quantised into
    position seq_lens[b] - 1 of sequence b, then attention as paged_decode_attention."""
    _require(q, "q", torch.bfloat16)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    B, Hq = int(q.shape[0]), int(q.shape[1])
    if q.shape[2] != HEAD_DIM:
        raise ValueError("head_dim must be 128")
    row = cache.num_kv_heads * HEAD_DIM
    for name, x in (("k_new", k_new), ("v_new", v_new)):
        if not x.is_cuda or x.dtype != torch.bfloat16 or x.shape[0] != B:
            raise ValueError("%s must be a CUDA bfloat16 tensor with one row per sequence" % name)
        if B > 0 and (not x[0].is_contiguous() or x[0].numel() != row):
            raise ValueError("%s: each row must hold %d contiguous values" % (name, row))
    stride = int(k_new.stride(0)) if B > 0 else row
    if B > 0 and int(v_new.stride(0)) != stride:
        raise ValueError("k_new and v_new must share a row stride")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if out is None:
        out = torch.empty_like(q)
    _require(out, "out", torch.bfloat16)
    if workspace is None:
        workspace = alloc_decode_workspace(cache, B, Hq, num_splits)
    _require(workspace, "workspace", torch.uint8)
    rc = _lib.nvfp4_paged_decode_attention_append(cache.desc, _ptr(k_new), _ptr(v_new), stride, _ptr(q), B, Hq,
                                                  _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                                  float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                                  int(num_splits), _stream(stream))
    _check(rc, "nvfp4_paged_decode_attention_append")
    return out


def cascade_workspace_bytes(cache: PagedCache, batch: int, num_q_heads: int, shared_len: int,
                            num_splits: int = 0) -> int:
    n = _lib.nvfp4kv_cascade_workspace_bytes(cache.desc, int(batch), int(num_q_heads), int(num_splits),
                                             int(shared_len))
    if n == 0 and batch > 0:
        raise NVFP4KVError(-1, "cascade_workspace_bytes")
    return int(n)


def cascade_decode_attention(cache: PagedCache, q: torch.Tensor, shared_pages: torch.Tensor, shared_len: int,
                             block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: Optional[float] = None,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             num_splits: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Decode attention for sequences sharing their first shared_len tokens (pages
    shared_pages, int32 [shared_len / P]); the shared part is attended once per kv
    head for all sequences, then merged with each sequence's own part."""
    _require(q, "q", torch.bfloat16)
    _require(shared_pages, "shared_pages", torch.int32)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    B, Hq = int(q.shape[0]), int(q.shape[1])
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if out is None:
        out = torch.empty_like(q)
    _require(out, "out", torch.bfloat16)
    if workspace is None:
        n = cascade_workspace_bytes(cache, B, Hq, shared_len, num_splits)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=cache.pool.device)
    _require(workspace, "workspace", torch.uint8)
    rc = _lib.nvfp4_cascade_decode_attention(cache.desc, _ptr(q), B, Hq, _ptr(shared_pages), int(shared_len),
                                             _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                             float(sm_scale), _ptr(out), _ptr(workspace), workspace.numel(),
                                             int(num_splits), _stream(stream))
    _check(rc, "nvfp4_cascade_decode_attention")
    return out


def paged_decode_attention_noalloc(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor,
                                   seq_lens: torch.Tensor, sm_scale: Optional[float] = None,
                                   out: Optional[torch.Tensor] = None, num_splits: int = 0,
                                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Same as paged_decode_attention, with the split scratch taken from the
    library's static device array instead of a workspace, for callers that
    cannot allocate device memory.  `out` must then be provided by the caller
    too (passing None allocates it here, through torch)."""
    _require(q, "q", torch.bfloat16)
    _require(block_table, "block_table", torch.int32)
    _require(seq_lens, "seq_lens", torch.int32)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    if out is None:
        out = torch.empty_like(q)
    _require(out, "out", torch.bfloat16)
    rc = _lib.nvfp4_paged_decode_attention_noalloc(cache.desc, _ptr(q), int(q.shape[0]), int(q.shape[1]),
                                                   _ptr(block_table), int(block_table.shape[1]), _ptr(seq_lens),
                                                   float(sm_scale), _ptr(out), int(num_splits), _stream(stream))
    _check(rc, "nvfp4_paged_decode_attention_noalloc")
    return out


def prefix_dequant(cache: PagedCache, block_table: torch.Tensor, prefix_lens: torch.Tensor,
                   cu_prefix_lens: torch.Tensor, total_prefix_tokens: int, k_ws: Optional[torch.Tensor] = None,
                   v_ws: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Returns (k_ws, v_ws), BF16 [total][Hkv][128]."""
    _require(block_table, "block_table", torch.int32)
    _require(prefix_lens, "prefix_lens", torch.int32)
    _require(cu_prefix_lens, "cu_prefix_lens", torch.int32)
    shape = (int(total_prefix_tokens), cache.num_kv_heads, HEAD_DIM)
    dev = cache.pool.device
    if k_ws is None:
        k_ws = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if v_ws is None:
        v_ws = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    _require(k_ws, "k_ws", torch.bfloat16)
    _require(v_ws, "v_ws", torch.bfloat16)
    rc = _lib.nvfp4_prefix_dequant(cache.desc, _ptr(block_table), int(block_table.shape[1]), _ptr(prefix_lens),
                                   _ptr(cu_prefix_lens), int(prefix_lens.shape[0]), int(total_prefix_tokens),
                                   _ptr(k_ws), _ptr(v_ws), _stream(stream))
    _check(rc, "nvfp4_prefix_dequant")
    return k_ws, v_ws


def profile_decode(before, after, every: int = 1):
    """Benchmark hook: record torch.cuda.Event pairs around the decode-kernel
    launch of every `every`-th following call (the j-th such call uses pair
    j % len).  Pass empty lists to stop."""
    if not before:
        _check(_lib.nvfp4kv_profile_decode(None, None, 0, 1), "nvfp4kv_profile_decode")
        return
    n = len(before)
    assert len(after) == n
    for e in list(before) + list(after):
        if not e.cuda_event:      # torch creates the CUDA event on first record
            e.record()
    arr_b = (ctypes.c_void_p * n)(*[e.cuda_event for e in before])
    arr_a = (ctypes.c_void_p * n)(*[e.cuda_event for e in after])
    _check(_lib.nvfp4kv_profile_decode(arr_b, arr_a, n, int(every)), "nvfp4kv_profile_decode")


def selftest_bounded_wait(arrive: bool, poll_limit: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Failure-path self-test: one warp waits (at most poll_limit polls) on an
    mbarrier phase that completes only if `arrive`.  Returns a device int32
    tensor [1]: 1 if the wait gave up (the device error word then holds the
    timeout bit), else 0."""
    result = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _check(_lib.nvfp4kv_selftest_bounded_wait(1 if arrive else 0, int(poll_limit), _ptr(result), _stream(stream)),
           "nvfp4kv_selftest_bounded_wait")
    return result


def extend_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, cu_prefix_lens: torch.Tensor,
                     k_chunk: torch.Tensor, v_chunk: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int,
                     sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Each request's chunk attends to [its prefix rows || the chunk], causally in
    the chunk.  q: BF16 [total_q][Hq][128]; k_prefix, v_prefix: BF16
    [total_prefix][Hkv][128] (e.g. from prefix_dequant); k_chunk, v_chunk: BF16
    [total_q][Hkv][128]; cu_*: int32 [R+1]; max_q_len: bound on chunk lengths."""
    for name, x in (("q", q), ("k_prefix", k_prefix), ("v_prefix", v_prefix), ("k_chunk", k_chunk),
                    ("v_chunk", v_chunk)):
        if not x.is_cuda or x.dtype != torch.bfloat16 or not x.is_contiguous() or x.dim() != 3 or x.shape[2] != HEAD_DIM:
            raise ValueError("%s must be a contiguous CUDA bfloat16 tensor [rows][heads][128]" % name)
    _require(cu_prefix_lens, "cu_prefix_lens", torch.int32)
    _require(cu_q_lens, "cu_q_lens", torch.int32)
    R = int(cu_q_lens.shape[0]) - 1
    if int(cu_prefix_lens.shape[0]) != R + 1:
        raise ValueError("cu_prefix_lens and cu_q_lens must have the same length")
    hq, hkv = int(q.shape[1]), int(k_chunk.shape[1])
    if k_prefix.shape[1] != hkv or v_prefix.shape[1] != hkv or v_chunk.shape[1] != hkv:
        raise ValueError("K/V head counts differ")
    if k_chunk.shape[0] != q.shape[0] or v_chunk.shape[0] != q.shape[0]:
        raise ValueError("chunk K/V must have one row per query token")
    if out is None:
        out = torch.empty_like(q)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    # an empty prefix still needs a valid aligned pointer
    kp = k_prefix if k_prefix.numel() else torch.zeros((1, hkv, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
    vp = v_prefix if v_prefix.numel() else kp
    rc = _lib.nvfp4_extend_attention(_ptr(q), _ptr(kp), _ptr(vp), _ptr(cu_prefix_lens), int(kp.shape[0]),
                                     _ptr(k_chunk), _ptr(v_chunk), _ptr(cu_q_lens), int(q.shape[0]), R,
                                     int(max_q_len), hq, hkv, float(sm_scale), _ptr(out), _stream(stream))
    _check(rc, "nvfp4_extend_attention")
    return out


def extend_attention_paged(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, prefix_lens: torch.Tensor,
                           k_chunk: torch.Tensor, v_chunk: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int,
                           sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """extend_attention with request r's prefix read from the NVFP4 cache: tokens
    0 .. prefix_lens[r] - 1 of its pages (block_table row r, int32 [R][max_pages]),
    expanded to BF16 inside the kernel; equals prefix_dequant + extend_attention."""
    for name, x in (("q", q), ("k_chunk", k_chunk), ("v_chunk", v_chunk)):
        if not x.is_cuda or x.dtype != torch.bfloat16 or not x.is_contiguous() or x.dim() != 3 or x.shape[2] != HEAD_DIM:
            raise ValueError("%s must be a contiguous CUDA bfloat16 tensor [rows][heads][128]" % name)
    _require(block_table, "block_table", torch.int32)
    _require(prefix_lens, "prefix_lens", torch.int32)
    _require(cu_q_lens, "cu_q_lens", torch.int32)
    R = int(cu_q_lens.shape[0]) - 1
    if int(prefix_lens.shape[0]) != R or int(block_table.shape[0]) != R:
        raise ValueError("prefix_lens and block_table need one entry / row per request")
    hq = int(q.shape[1])
    if k_chunk.shape[1] != cache.num_kv_heads or v_chunk.shape[1] != cache.num_kv_heads:
        raise ValueError("chunk K/V must have the cache's kv heads")
    if k_chunk.shape[0] != q.shape[0] or v_chunk.shape[0] != q.shape[0]:
        raise ValueError("chunk K/V must have one row per query token")
    if out is None:
        out = torch.empty_like(q)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(HEAD_DIM)
    rc = _lib.nvfp4_extend_attention_paged(cache.desc, _ptr(q), _ptr(block_table), int(block_table.shape[1]),
                                           _ptr(prefix_lens), _ptr(k_chunk), _ptr(v_chunk), _ptr(cu_q_lens),
                                           int(q.shape[0]), R, int(max_q_len), hq, float(sm_scale), _ptr(out),
                                           _stream(stream))
    _check(rc, "nvfp4_extend_attention_paged")
    return out


# ---------------------------------------------------------------- latent cache and eviction

# (the calls below are short: their checks are written to cost little on the host)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _complain(t, name: str, dtype: torch.dtype, shape, dev: int):
    """The error that the failed check of _want describes."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the call's other tensors on cuda:%d" % (name, t.get_device(), dev))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _want(t, name: str, dtype: torch.dtype, shape, dev: int) -> int:
    """Checks a contiguous CUDA tensor (shape None: any) and returns its address."""
    if (not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous() or (shape is not None and t.shape != shape)):
        _complain(t, name, dtype, shape, dev)
    return t.data_ptr()


def _want_table(t, name: str, rows: int, dev: int) -> int:
    p = _want(t, name, torch.int32, None, dev)
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError("%s must be [%d][pages], a row per sequence" % (name, rows))
    return p


def _launch_stream(dev: int, stream: Optional[torch.cuda.Stream]) -> int:
    """The stream handle of a call whose tensors lie on device dev: the current
    device (the library launches there), and the stream on it."""
    if _current_device() != dev:
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % dev)
    if stream is None:
        return _raw_stream(dev)
    if stream.device.index != dev:
        raise ValueError("the stream is on %s, the tensors on cuda:%d" % (stream.device, dev))
    return stream.cuda_stream


def _keep_until_done(stream: Optional[torch.cuda.Stream], *tensors):
    """Tensors allocated here on the current stream, used on another one: their
    memory is not given out again before that stream has passed this point."""
    if stream is not None and tensors and stream.cuda_stream != _raw_stream(stream.device.index):
        stream.wait_stream(torch.cuda.current_stream())   # memory that earlier work here may still use
        for t in tensors:
            t.record_stream(stream)


class LatentCache:
    """A caller-owned pool of latent pages (uint8 [num_pages][416 * page_size]): 512
    NVFP4 latent values and 64 BF16 rotary values a token."""

    def __init__(self, num_pages: int, page_size: int, global_scale: float = 1.0, device="cuda",
                 pool: Optional[torch.Tensor] = None):
        self.num_pages, self.page_size, self.global_scale = int(num_pages), int(page_size), float(global_scale)
        self.slab = latent_slab_bytes(self.page_size)
        if pool is None:
            pool = torch.zeros((self.num_pages, self.slab), dtype=torch.uint8, device=device)
        _require(pool, "pool", torch.uint8)
        if pool.numel() != self.num_pages * self.slab:
            raise ValueError("pool has %d bytes, expected %d" % (pool.numel(), self.num_pages * self.slab))
        self.pool = pool
        self._desc = _LatentDesc(pool.data_ptr(), self.num_pages, self.page_size, LATENT_DIM, ROPE_DIM,
                                 self.global_scale)
        self.desc = ctypes.byref(self._desc)

    @property
    def num_slots(self) -> int:
        return self.num_pages * self.page_size


def latent_slab_bytes(page_size: int) -> int:
    d = _LatentDesc(256, 1, int(page_size), LATENT_DIM, ROPE_DIM, 1.0)
    n = _lib.nvfp4kv_latent_slab_bytes(ctypes.byref(d))
    if n == 0:
        raise NVFP4KVError(-2, "latent_slab_bytes(page_size=%d)" % page_size)
    return int(n)


def _rows(t, name: str, T: int, width: int, dev: int):
    """Address and row stride of BF16 [T][width] whose rows may be strided."""
    st = t.stride() if isinstance(t, torch.Tensor) else None
    if (st is None or t.dtype is not torch.bfloat16 or t.get_device() != dev
            or t.shape != (T, width) or (T > 0 and st[1] != 1)):
        if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == (T, width):
            raise ValueError("%s: each token must hold %d contiguous values" % (name, width))
        _complain(t, name, torch.bfloat16, (T, width), dev)
    # (a single row's stride says nothing: torch may give it any value)
    return t.data_ptr(), st[0] if T > 1 else width


def latent_quantize_append(cache: LatentCache, latent: torch.Tensor, k_rope: torch.Tensor, slot_mapping: torch.Tensor,
                           stream: Optional[torch.cuda.Stream] = None):
    """latent: BF16 [T][512], k_rope: BF16 [T][64] (rows may be strided: views of one
    wider row); slot_mapping: int64 [T].  Quantises the latents, stores the rotary
    parts as they are."""
    dev = cache.pool.get_device()
    sp = _want(slot_mapping, "slot_mapping", torch.int64, None, dev)
    T = slot_mapping.numel()
    if slot_mapping.dim() != 1:
        raise ValueError("slot_mapping must be [tokens]")
    lp, ls = _rows(latent, "latent", T, LATENT_DIM, dev)
    rp, rs = _rows(k_rope, "k_rope", T, ROPE_DIM, dev)
    rc = _lib.nvfp4_latent_quantize_append(cache.desc, lp, ls, rp, rs, T, sp, _launch_stream(dev, stream))
    if rc:
        _check(rc, "nvfp4_latent_quantize_append")


def latent_prefix_dequant(cache: LatentCache, block_table: torch.Tensor, prefix_lens: torch.Tensor,
                          cu_prefix_lens: torch.Tensor, total_prefix_tokens: int,
                          latent_ws: Optional[torch.Tensor] = None, rope_ws: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None):
    """Returns (latent_ws BF16 [total][512], rope_ws BF16 [total][64]): the cached
    prefixes' rows, the input of the up-projections to per-head K and V."""
    dev, total = cache.pool.get_device(), int(total_prefix_tokens)
    pp = _want(prefix_lens, "prefix_lens", torch.int32, None, dev)
    R = prefix_lens.numel()
    cp = _want(cu_prefix_lens, "cu_prefix_lens", torch.int32, (R + 1,), dev)
    bp = _want_table(block_table, "block_table", R, dev)
    s = _launch_stream(dev, stream)
    made = []
    if latent_ws is None:
        latent_ws = torch.empty((total, LATENT_DIM), dtype=torch.bfloat16, device=cache.pool.device)
        made.append(latent_ws)
        lp = latent_ws.data_ptr()
    else:
        lp = _want(latent_ws, "latent_ws", torch.bfloat16, (total, LATENT_DIM), dev)
    if rope_ws is None:
        rope_ws = torch.empty((total, ROPE_DIM), dtype=torch.bfloat16, device=cache.pool.device)
        made.append(rope_ws)
        rp = rope_ws.data_ptr()
    else:
        rp = _want(rope_ws, "rope_ws", torch.bfloat16, (total, ROPE_DIM), dev)
    if stream is not None:
        _keep_until_done(stream, *made)
    rc = _lib.nvfp4_latent_prefix_dequant(cache.desc, bp, block_table.shape[1], pp, cp, R, total, lp, rp, s)
    if rc:
        _check(rc, "nvfp4_latent_prefix_dequant")
    return latent_ws, rope_ws


def latent_decode_workspace_bytes(cache: LatentCache, batch: int, num_heads: int, num_splits: int = 0) -> int:
    n = _lib.nvfp4kv_latent_decode_workspace_bytes(cache.desc, int(batch), int(num_heads), int(num_splits))
    if n == 0:
        raise NVFP4KVError(-1, "latent_decode_workspace_bytes")
    return int(n)


def alloc_latent_decode_workspace(cache: LatentCache, batch: int, num_heads: int, num_splits: int = 0) -> torch.Tensor:
    n = latent_decode_workspace_bytes(cache, batch, num_heads, num_splits)
    return torch.empty(n, dtype=torch.uint8, device=cache.pool.device)


def latent_decode_attention(cache: LatentCache, q_latent: torch.Tensor, q_rope: torch.Tensor,
                            block_table: torch.Tensor, seq_lens: torch.Tensor, sm_scale: Optional[float] = None,
                            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            num_splits: int = 0, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Absorbed form, one query a sequence.  q_latent: BF16 [B][H][512] (the queries
    times the up-projection of K); q_rope: BF16 [B][H][64]; block_table int32
    [B][max_pages]; seq_lens int32 [B] -> BF16 [B][H][512], each head's weighted
    mean of the latents (its up-projection to V is left to the caller).  H <= 128;
    sm_scale defaults to 1 / sqrt(128 + 64)."""
    dev = cache.pool.get_device()
    qp = _want(q_latent, "q_latent", torch.bfloat16, None, dev)
    if q_latent.dim() != 3 or q_latent.shape[2] != LATENT_DIM:
        raise ValueError("q_latent must be [batch][heads][512]")
    B, H, _ = q_latent.shape
    rp = _want(q_rope, "q_rope", torch.bfloat16, (B, H, ROPE_DIM), dev)
    lp = _want(seq_lens, "seq_lens", torch.int32, (B,), dev)
    bp = _want_table(block_table, "block_table", B, dev)
    s = _launch_stream(dev, stream)
    made = []
    if out is None:
        out = torch.empty_like(q_latent)
        made.append(out)
        op = out.data_ptr()
    else:
        op = _want(out, "out", torch.bfloat16, (B, H, LATENT_DIM), dev)
    if workspace is None:
        workspace = alloc_latent_decode_workspace(cache, B, H, num_splits)
        made.append(workspace)
    wp = _want(workspace, "workspace", torch.uint8, None, dev)
    if stream is not None:
        _keep_until_done(stream, *made)
    rc = _lib.nvfp4_latent_decode_attention(cache.desc, qp, rp, B, H, bp, block_table.shape[1], lp,
                                            _LATENT_SCALE if sm_scale is None else float(sm_scale), op, wp,
                                            workspace.numel(), int(num_splits), s)
    if rc:
        _check(rc, "nvfp4_latent_decode_attention")
    return out


_LATENT_SCALE = 1.0 / math.sqrt(HEAD_DIM + ROPE_DIM)


def _heads(k, v, where: str, rows: int, H: int, dev: int):
    """Addresses and (token, head) strides of BF16 K and V [rows][H][128], which share them."""
    shape, strides = (rows, H, HEAD_DIM), []
    for name, x in (("k_", k), ("v_", v)):
        st = x.stride() if isinstance(x, torch.Tensor) else None
        if (st is None or x.dtype is not torch.bfloat16 or x.get_device() != dev or x.shape != shape
                or (rows > 0 and st[2] != 1)):
            if st is not None and x.dtype is torch.bfloat16 and x.get_device() == dev and x.shape == shape:
                raise ValueError("%s%s: the 128 values of a head must be contiguous" % (name, where))
            _complain(x, name + where, torch.bfloat16, shape, dev)
        strides.append(st)
    sk, sv = strides
    # strides of axes of length 1 say nothing: torch may give them any value
    st = sk[0] if rows > 1 else H * HEAD_DIM
    sh = sk[1] if H > 1 else HEAD_DIM
    if sk != sv and ((rows > 1 and sv[0] != st) or (H > 1 and rows > 0 and sv[1] != sh)):
        raise ValueError("k_%s and v_%s must share their strides" % (where, where))
    return k.data_ptr(), v.data_ptr(), st, sh


def latent_extend_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, rope_prefix: torch.Tensor,
                            cu_prefix_lens: torch.Tensor, k_chunk: torch.Tensor, v_chunk: torch.Tensor,
                            rope_chunk: torch.Tensor, cu_q_lens: torch.Tensor, max_q_len: int,
                            sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Expanded form: each request's chunk attends to [its prefix || the chunk],
    causally in the chunk.  q: BF16 [total_q][H][192], the last 64 the rotary part;
    k_*, v_*: BF16 [rows][H][128], the up-projected latents (any token and head
    strides that are multiples of 8: halves of one [rows][H][256] projection
    output); rope_*: BF16 [rows][64], shared by the heads; cu_*: int32 [R+1];
    max_q_len: bound on chunk lengths -> BF16 [total_q][H][128].  sm_scale > 0
    defaults to 1 / sqrt(192)."""
    dev = q.get_device()
    qp = _want(q, "q", torch.bfloat16, None, dev)
    if dev < 0 or q.dim() != 3 or q.shape[2] != HEAD_DIM + ROPE_DIM:
        raise ValueError("q must be a CUDA tensor [total_q][heads][192]")
    TQ, H, _ = q.shape
    np_ = _want(cu_q_lens, "cu_q_lens", torch.int32, None, dev)
    R = cu_q_lens.numel() - 1
    pp = _want(cu_prefix_lens, "cu_prefix_lens", torch.int32, (R + 1,), dev)
    TP = k_prefix.shape[0]
    k0, v0, ps, ph = _heads(k_prefix, v_prefix, "prefix", TP, H, dev)
    k1, v1, cs, ch = _heads(k_chunk, v_chunk, "chunk", TQ, H, dev)
    r0 = _want(rope_prefix, "rope_prefix", torch.bfloat16, (TP, ROPE_DIM), dev)
    r1 = _want(rope_chunk, "rope_chunk", torch.bfloat16, (TQ, ROPE_DIM), dev)
    s = _launch_stream(dev, stream)
    if out is None:
        out = torch.empty((TQ, H, HEAD_DIM), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
        if stream is not None:
            _keep_until_done(stream, out)
    else:
        op = _want(out, "out", torch.bfloat16, (TQ, H, HEAD_DIM), dev)
    rc = _lib.nvfp4_latent_extend_attention(qp, k0, v0, ps, ph, r0, pp, TP, k1, v1, cs, ch, r1, np_, TQ, R,
                                            int(max_q_len), H, _LATENT_SCALE if sm_scale is None else float(sm_scale),
                                            op, s)
    if rc:
        _check(rc, "nvfp4_latent_extend_attention")
    return out


def weights_workspace_bytes(cache: PagedCache, batch: int, num_q_heads: int) -> int:
    n = _lib.nvfp4kv_weights_workspace_bytes(cache.desc, int(batch), int(num_q_heads))
    if n == 0:
        raise NVFP4KVError(-1, "weights_workspace_bytes")
    return int(n)


def alloc_weights_workspace(cache: PagedCache, batch: int, num_q_heads: int) -> torch.Tensor:
    return torch.empty(weights_workspace_bytes(cache, batch, num_q_heads), dtype=torch.uint8, device=cache.pool.device)


def accumulate_attention_weights(cache: PagedCache, q: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                                 scores: torch.Tensor, sm_scale: Optional[float] = None,
                                 workspace: Optional[torch.Tensor] = None,
                                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Adds to scores (float32 [B][Hkv][S], in place) the attention weights that the
    queries q (BF16 [B][Hq][128]) put on every cached token: entry [b][h][t] grows
    by the sum over kv head h's query heads of their softmax weight of token t <
    seq_lens[b].  Returns scores."""
    dev = cache.pool.get_device()
    qp = _want(q, "q", torch.bfloat16, None, dev)
    if q.dim() != 3 or q.shape[2] != HEAD_DIM:
        raise ValueError("q must be [batch][heads][128]")
    B, Hq, _ = q.shape
    lp = _want(seq_lens, "seq_lens", torch.int32, (B,), dev)
    bp = _want_table(block_table, "block_table", B, dev)
    cp = _want(scores, "scores", torch.float32, None, dev)
    if scores.dim() != 3 or scores.shape[0] != B or scores.shape[1] != cache.num_kv_heads:
        raise ValueError("scores must be [batch][kv heads][tokens]")
    s = _launch_stream(dev, stream)
    if workspace is None:
        workspace = alloc_weights_workspace(cache, B, Hq)
        _keep_until_done(stream, workspace)
    wp = _want(workspace, "workspace", torch.uint8, None, dev)
    rc = _lib.nvfp4_accumulate_attention_weights(cache.desc, qp, B, Hq, bp, block_table.shape[1], lp,
                                                 _HEAD_SCALE if sm_scale is None else float(sm_scale), cp,
                                                 scores.shape[2], wp, workspace.numel(), s)
    if rc:
        _check(rc, "nvfp4_accumulate_attention_weights")
    return scores


_HEAD_SCALE = 1.0 / math.sqrt(HEAD_DIM)


def evict(cache: PagedCache, scores: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
          new_block_table: torch.Tensor, keep: int, recent: int = 0, sink: int = 0,
          new_lens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
          new_scores: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Keeps, for every sequence and kv head, the `keep` tokens of largest score (and
    always the first `sink` and the last `recent`; ties to the lowest index), in
    their order, and copies their rows into the pages of new_block_table (int32
    [B][new pages]), none of which may be in use.  scores: float32 [B][Hkv][S].
    Returns (new_lens int32 [B], kept int32 [B][Hkv][keep]: the old row of every new
    one, -1 behind the last, new_scores float32 [B][Hkv][>= keep]: theirs, then zeros;
    S or keep wide, the larger, by default)."""
    dev, Hkv, keep = cache.pool.get_device(), cache.num_kv_heads, int(keep)
    lp = _want(seq_lens, "seq_lens", torch.int32, None, dev)
    B = seq_lens.numel()
    cp = _want(scores, "scores", torch.float32, None, dev)
    if scores.dim() != 3 or scores.shape[0] != B or scores.shape[1] != Hkv:
        raise ValueError("scores must be [batch][kv heads][tokens]")
    if keep < 1:
        raise ValueError("keep must be at least 1")
    S = scores.shape[2]
    bp = _want_table(block_table, "block_table", B, dev)
    np_ = _want_table(new_block_table, "new_block_table", B, dev)
    s = _launch_stream(dev, stream)
    where, made = cache.pool.device, []
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=where)
        made.append(new_lens)
        nlp = new_lens.data_ptr()
    else:
        nlp = _want(new_lens, "new_lens", torch.int32, (B,), dev)
    if kept is None:
        kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=where)
        made.append(kept)
        kp = kept.data_ptr()
    else:
        kp = _want(kept, "kept", torch.int32, (B, Hkv, keep), dev)
    if new_scores is None:
        new_scores = torch.empty((B, Hkv, max(S, keep)), dtype=torch.float32, device=where)
        made.append(new_scores)
        nsp = new_scores.data_ptr()
    else:
        nsp = _want(new_scores, "new_scores", torch.float32, None, dev)
        if (new_scores.dim() != 3 or new_scores.shape[0] != B or new_scores.shape[1] != Hkv
                or new_scores.shape[2] < keep):
            raise ValueError("new_scores must be [batch][kv heads][at least keep]")
    if stream is not None:
        _keep_until_done(stream, *made)
    rc = _lib.nvfp4_evict(cache.desc, cp, S, B, bp, block_table.shape[1], lp, np_, new_block_table.shape[1], keep,
                          int(recent), int(sink), nlp, kp, nsp, new_scores.shape[2], s)
    if rc:
        _check(rc, "nvfp4_evict")
    return new_lens, kept, new_scores


def check_device_errors(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream and return (and clear) the device error status (0 = none)."""
    return int(_lib.nvfp4kv_check_device_errors(_stream(stream)))
