"""Thin Python binding of the C ABI in include/kvq.h (argument marshalling only).

Every step of the path runs in the CUDA library ``_build/libkvq.so``; torch
supplies device memory and streams.  If the library is missing the calls raise
``KVQError`` -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkvq.so")

KVQ_FMT_INT4_G32, KVQ_FMT_FP4_E2M1_S16, KVQ_FMT_CB2_OUTLIER, KVQ_FMT_TIERED, KVQ_FMT_CB2_STATIC = 0, 1, 2, 3, 4
KVQ_FMT_ASYM3_OUTLIER, KVQ_FMT_CB2_GROUP4 = 5, 6
KVQ_BF16, KVQ_F16, KVQ_F32 = 0, 1, 2
KVQ_DECODE_AUTO, KVQ_DECODE_TENSOR_CORES, KVQ_DECODE_CUDA_CORES = 0, 1, 2
KVQ_TIER_BIT = 1 << 31
KVQ_STATUS_BAD_PAGE, KVQ_STATUS_CAPACITY, KVQ_STATUS_SEQ_TOO_LONG, KVQ_STATUS_TIMEOUT = 1, 2, 4, 8
KVQ_STATUS_BAD_ROWS = 16
KVQ_OK, KVQ_ERR_INVALID_ARG, KVQ_ERR_UNSUPPORTED, KVQ_ERR_WORKSPACE, KVQ_ERR_CAPACITY, KVQ_ERR_CUDA = range(6)

_DTYPE = {torch.bfloat16: KVQ_BF16, torch.float16: KVQ_F16, torch.float32: KVQ_F32}


class KVQError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = kvq_status_string(status) if _lib is not None else str(status)
        if status == KVQ_ERR_CUDA and _lib is not None:   # the runtime's own error name
            msg += f" {_lib.kvq_cuda_error_name(_lib.kvq_last_cuda_error()).decode()}"
        super().__init__(f"{what}: {msg} (status {status})" if what else msg)


class kvq_config(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("pages_per_seq_max", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("num_tier_pages", ctypes.c_int32), ("format", ctypes.c_int32), ("lloyd_iters", ctypes.c_int32),
                ("sigma", ctypes.c_double), ("static_channels", ctypes.c_int32),
                ("decode_math", ctypes.c_int32)]


class kvq_cache(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("tier_pool", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seq_lens", ctypes.c_void_p), ("staging", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("static_mask", ctypes.c_void_p)]


_lib = None
_lock = threading.Lock()
EXPORTS = ("kvq_block_bytes", "kvq_cache_bytes", "kvq_quantize_append", "kvq_project_append",
           "kvq_decode_workspace_bytes",
           "kvq_decode_num_splits", "kvq_decode_split", "kvq_decode_combine", "kvq_decode_attention",
           "kvq_decode_attention_noalloc", "kvq_tree_workspace_bytes", "kvq_tree_attention", "kvq_page_mass",
           "kvq_evict_pages", "kvq_norm_rope", "kvq_prompt_attention", "kvq_select_static_channels", "kvq_dequantize",
           "kvq_status_string",
           "kvq_last_cuda_error", "kvq_cuda_error_name", "kvq_version")


def lib() -> ctypes.CDLL:
    """Load libkvq.so (built by __graft_entry__.build() / sub_byte_quantized_kvq_gb300.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise KVQError(-1, f"CUDA library not built: {LIB_PATH} is missing")
            L = ctypes.CDLL(LIB_PATH)
            P, I, S, L64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int64
            pcfg, pcache = ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache)
            sig = {
                "kvq_block_bytes": (I, [pcfg, I, ctypes.POINTER(S)]),
                "kvq_cache_bytes": (I, [pcfg, ctypes.POINTER(S), ctypes.POINTER(S), ctypes.POINTER(S)]),
                "kvq_quantize_append": (I, [pcfg, pcache, P, P, I, I, P, P]),
                "kvq_project_append": (I, [pcfg, pcache, P, I, P, P, I, P, P, P]),
                "kvq_decode_workspace_bytes": (I, [pcfg, I, I, I, ctypes.POINTER(S)]),
                "kvq_decode_num_splits": (I, [pcfg, I, I, ctypes.POINTER(I)]),
                "kvq_decode_split": (I, [pcfg, pcache, P, I, ctypes.c_float, I, I, P, S, P]),
                "kvq_decode_combine": (I, [pcfg, I, I, I, P, S, P, I, P]),
                "kvq_decode_attention": (I, [pcfg, pcache, P, I, ctypes.c_float, I, I, P, I, P, S, P]),
                "kvq_decode_attention_noalloc": (I, [pcfg, pcache, P, I, ctypes.c_float, I, I, P, I, P]),
                "kvq_tree_workspace_bytes": (I, [pcfg, I, I, I, I, ctypes.POINTER(S)]),
                "kvq_tree_attention": (I, [pcfg, pcache, P, I, I, P, P, P, I, P, ctypes.c_float, I, I, P, I, P, P, P, S,
                                           P]),
                "kvq_page_mass": (I, [pcfg, I, I, I, P, P, P, ctypes.c_float, P, P, P]),
                "kvq_evict_pages": (I, [pcfg, pcache, P, I, I, I, P, P, P, P, P]),
                "kvq_norm_rope": (I, [pcfg, P, L64, I, P, L64, I, I, P, P, ctypes.c_float, P, I, P, I, P, I, P, L64, P, L64, I,
                                      P]),
                "kvq_prompt_attention": (I, [pcfg, P, L64, P, L64, P, L64, I, I, I, P, P, I, ctypes.c_float, I, P, L64, I, P, P,
                                             P]),
                "kvq_select_static_channels": (I, [pcfg, P, P, I, I, P, P]),
                "kvq_dequantize": (I, [pcfg, pcache, I, I, I, I, I, P, P]),
                "kvq_status_string": (ctypes.c_char_p, [I]),
                "kvq_last_cuda_error": (I, []),
                "kvq_cuda_error_name": (ctypes.c_char_p, [I]),
                "kvq_version": (ctypes.c_char_p, []),
            }
            for name, (res, args) in sig.items():
                f = getattr(L, name)
                f.restype, f.argtypes = res, args
            _lib = L
    return _lib


def _check(status: int, what: str):
    if status != KVQ_OK:
        raise KVQError(status, what)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _made_on(stream, make, returned: bool = False) -> torch.Tensor:
    """make(), a tensor allocated here for a call on `stream` (None: the current stream), from that stream's
    memory: what another stream's pending work still uses is never handed to it.  returned: the caller
    goes on with it on the current stream."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make()
    if returned:
        t.record_stream(here)
    return t


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def kvq_status_string(status: int) -> str:
    return lib().kvq_status_string(status).decode()


def kvq_version() -> str:
    return lib().kvq_version().decode()


class QuantizedKVCache:
    """Device buffers of one paged, quantized cache (allocated with torch)."""

    def __init__(self, fmt: int, num_seqs: int, num_kv_heads: int, head_dim: int, pages_per_seq_max: int,
                 num_pages: int, num_tier_pages: int = 0, sigma: float = 3.0, lloyd_iters: int = 16,
                 page_table: torch.Tensor | None = None, device="cuda", static_channels: int = 0,
                 decode_math: int = KVQ_DECODE_AUTO):
        """static_channels (KVQ_FMT_CB2_STATIC): fp16 channels per (kv head, K|V);
        fill `static_mask` ([Hkv, 2, n]) before the first append, e.g. with
        kvq_select_static_channels.  decode_math: KVQ_DECODE_* (cfg.decode_math
        may be changed between calls)."""
        self.cfg = kvq_config(num_seqs, num_kv_heads, head_dim, pages_per_seq_max, num_pages, num_tier_pages, fmt,
                              lloyd_iters, sigma, static_channels, decode_math)
        pb, tb, sb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().kvq_cache_bytes(ctypes.byref(self.cfg), ctypes.byref(pb), ctypes.byref(tb), ctypes.byref(sb)),
               "kvq_cache_bytes")
        self.device = torch.device(device)
        self.pool = torch.zeros(pb.value, dtype=torch.uint8, device=self.device)
        self.tier_pool = torch.zeros(tb.value, dtype=torch.uint8, device=self.device) if tb.value else None
        self.staging = torch.zeros(sb.value // 4, dtype=torch.float32, device=self.device) if sb.value else None
        if page_table is None:
            page_table = torch.arange(num_seqs * pages_per_seq_max, dtype=torch.int64).view(num_seqs, -1) % num_pages
        self.page_table = torch.as_tensor(page_table).to(torch.int32).to(self.device).contiguous()
        self.seq_lens = torch.zeros(num_seqs, dtype=torch.int32, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self.static_mask = (torch.zeros((num_kv_heads, 2, static_channels), dtype=torch.uint8, device=self.device)
                            if fmt == KVQ_FMT_CB2_STATIC else None)
        self.c = kvq_cache(self.pool.data_ptr(), self.tier_pool.data_ptr() if self.tier_pool is not None else None,
                           self.page_table.data_ptr(), self.seq_lens.data_ptr(),
                           self.staging.data_ptr() if self.staging is not None else None, self.status.data_ptr(),
                           self.static_mask.data_ptr() if self.static_mask is not None else None)

    @classmethod
    def from_buffers(cls, fmt: int, num_kv_heads: int, head_dim: int, pool: torch.Tensor, page_table: torch.Tensor,
                     seq_lens: torch.Tensor, status: torch.Tensor, staging: torch.Tensor | None = None,
                     tier_pool: torch.Tensor | None = None, static_mask: torch.Tensor | None = None,
                     sigma: float = 3.0, lloyd_iters: int = 16, decode_math: int = KVQ_DECODE_AUTO) -> "QuantizedKVCache":
        """A handle on device buffers the caller owns (page_table int32
        [num_seqs, pages_per_seq_max], seq_lens int32 [num_seqs], status int32
        [1], pool / tier_pool uint8 of whole blocks, 16-byte aligned, staging
        fp32); nothing is allocated or copied, and the pools' sizes give the
        page counts."""
        num_seqs, ppsm = page_table.shape
        buffers = [pool, page_table, seq_lens, status, staging, tier_pool, static_mask]
        assert all(t is None or (t.is_contiguous() and t.device == pool.device) for t in buffers)
        assert page_table.dtype == seq_lens.dtype == status.dtype == torch.int32 and seq_lens.numel() == num_seqs
        for t in (pool, tier_pool):
            assert t is None or (t.dtype == torch.uint8 and t.data_ptr() % 16 == 0)
        assert static_mask is None or static_mask.dtype == torch.uint8
        self = cls.__new__(cls)
        self.cfg = kvq_config(num_seqs, num_kv_heads, head_dim, ppsm, 1, 1 if tier_pool is not None else 0, fmt,
                              lloyd_iters, sigma, static_mask.shape[-1] if static_mask is not None else 0, decode_math)
        main = 2 * num_kv_heads * kvq_block_bytes(self.cfg, 0)
        self.cfg.num_pages = pool.numel() * pool.element_size() // main
        if tier_pool is not None:
            self.cfg.num_tier_pages = (tier_pool.numel() * tier_pool.element_size() //
                                       (2 * num_kv_heads * kvq_block_bytes(self.cfg, 1)))
        pb, tb, sb = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().kvq_cache_bytes(ctypes.byref(self.cfg), ctypes.byref(pb), ctypes.byref(tb), ctypes.byref(sb)),
               "kvq_cache_bytes")
        if sb.value:   # a page format
            assert staging is not None and staging.dtype == torch.float32 and staging.numel() * 4 >= sb.value
        self.device, self.pool, self.tier_pool, self.staging = pool.device, pool, tier_pool, staging
        self.page_table, self.seq_lens, self.status, self.static_mask = page_table, seq_lens, status, static_mask
        self.c = kvq_cache(*[None if t is None else t.data_ptr()
                             for t in (pool, tier_pool, page_table, seq_lens, staging, status, static_mask)])
        return self

    @property
    def head_dim(self) -> int:
        return self.cfg.head_dim

    def block_bytes(self, tier: int = 0) -> int:
        return kvq_block_bytes(self.cfg, tier)

    def status_word(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF


def kvq_block_bytes(cfg: kvq_config, tier: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(lib().kvq_block_bytes(ctypes.byref(cfg), tier, ctypes.byref(n)), "kvq_block_bytes")
    return n.value


def kvq_quantize_append(cache: QuantizedKVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                        t_per_seq: torch.Tensor | None = None, stream=None):
    """k_new, v_new: [num_seqs, t_new, Hkv, D] bf16/f16/f32 on the cache's device."""
    assert k_new.shape == v_new.shape and k_new.dtype == v_new.dtype and k_new.is_contiguous() and v_new.is_contiguous()
    assert k_new.dim() == 4 and k_new.shape[0] == cache.cfg.num_seqs
    if t_per_seq is not None:
        given = t_per_seq
        t_per_seq = _made_on(stream, lambda: given.to(torch.int32).contiguous())
    _check(lib().kvq_quantize_append(ctypes.byref(cache.cfg), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new),
                                     _DTYPE[k_new.dtype], k_new.shape[1], _ptr(t_per_seq), _stream(stream)),
           "kvq_quantize_append")


def kvq_project_append(cache: QuantizedKVCache, x: torch.Tensor, w_k: torch.Tensor, w_v: torch.Tensor,
                       t_per_seq: torch.Tensor | None = None, kv_out: torch.Tensor | None = None, stream=None):
    """x: bf16 [num_seqs, t_new, hidden]; w_k, w_v: bf16 [Hkv * D, hidden].  K = x w_k^T and
    V = x w_v^T are projected on the tensor cores and quantized into the cache in one kernel.
    kv_out: optional fp32 [2, num_seqs, t_new, Hkv, D] that receives the projected K and V."""
    cfg = cache.cfg
    assert x.dtype == torch.bfloat16 and w_k.dtype == torch.bfloat16 and w_v.dtype == torch.bfloat16
    assert x.is_contiguous() and w_k.is_contiguous() and w_v.is_contiguous()
    assert x.dim() == 3 and x.shape[0] == cfg.num_seqs
    hidden = x.shape[2]
    assert w_k.shape == (cfg.num_kv_heads * cfg.head_dim, hidden) and w_v.shape == w_k.shape
    if kv_out is not None:
        assert kv_out.dtype == torch.float32 and kv_out.is_contiguous()
        assert kv_out.shape == (2, cfg.num_seqs, x.shape[1], cfg.num_kv_heads, cfg.head_dim)
    if t_per_seq is not None:
        given = t_per_seq
        t_per_seq = _made_on(stream, lambda: given.to(torch.int32).contiguous())
    _check(lib().kvq_project_append(ctypes.byref(cfg), ctypes.byref(cache.c), _ptr(x), hidden, _ptr(w_k), _ptr(w_v),
                                    x.shape[1], _ptr(t_per_seq), _ptr(kv_out), _stream(stream)),
           "kvq_project_append")


def kvq_decode_num_splits(cache: QuantizedKVCache, num_q_heads: int, max_seq_len: int) -> int:
    n = ctypes.c_int32()
    _check(lib().kvq_decode_num_splits(ctypes.byref(cache.cfg), num_q_heads, max_seq_len, ctypes.byref(n)),
           "kvq_decode_num_splits")
    return n.value


def kvq_decode_workspace_bytes(cache: QuantizedKVCache, num_q_heads: int, max_seq_len: int,
                               num_splits: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(lib().kvq_decode_workspace_bytes(ctypes.byref(cache.cfg), num_q_heads, max_seq_len, num_splits,
                                            ctypes.byref(n)), "kvq_decode_workspace_bytes")
    return n.value


def kvq_decode_attention(cache: QuantizedKVCache, q: torch.Tensor, softmax_scale: float, max_seq_len: int,
                         num_splits: int = 0, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q: [num_seqs, Hq, D] bf16 -> out [num_seqs, Hq, D] (bf16 or f32)."""
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    Hq = q.shape[1]
    if out is None:
        out = _made_on(stream, lambda: torch.empty(q.shape, dtype=out_dtype, device=q.device), returned=True)
    if workspace is None:
        workspace = _made_on(stream, lambda: alloc_workspace(cache, Hq, max_seq_len, num_splits))   # (zeroed on `stream`)
    _check(lib().kvq_decode_attention(ctypes.byref(cache.cfg), ctypes.byref(cache.c), _ptr(q), Hq,
                                      float(softmax_scale), max_seq_len, num_splits, _ptr(out), _DTYPE[out.dtype],
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "kvq_decode_attention")
    return out


def kvq_select_static_channels(cache: QuantizedKVCache, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Fill cache.static_mask from calibration values k, v [t, Hkv, D] (device)."""
    assert k.shape == v.shape and k.dim() == 3 and k.dtype == v.dtype and k.is_contiguous() and v.is_contiguous()
    _check(lib().kvq_select_static_channels(ctypes.byref(cache.cfg), _ptr(k), _ptr(v), _DTYPE[k.dtype], k.shape[0],
                                            _ptr(cache.static_mask), _stream(stream)), "kvq_select_static_channels")
    return cache.static_mask


def alloc_workspace(cache: QuantizedKVCache, num_q_heads: int, max_seq_len: int, num_splits: int = 0) -> torch.Tensor:
    nbytes = kvq_decode_workspace_bytes(cache, num_q_heads, max_seq_len, num_splits)
    # zeroed once: its head holds the fused split merge's arrival counters
    return torch.zeros((nbytes + 15) // 16 * 4, dtype=torch.float32, device=cache.device)


def kvq_decode_split(cache: QuantizedKVCache, q: torch.Tensor, softmax_scale: float, max_seq_len: int,
                     workspace: torch.Tensor, num_splits: int = 0, stream=None):
    """Stage 1 of kvq_decode_attention: split partials into `workspace`."""
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    _check(lib().kvq_decode_split(ctypes.byref(cache.cfg), ctypes.byref(cache.c), _ptr(q), q.shape[1],
                                  float(softmax_scale), max_seq_len, num_splits, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)), "kvq_decode_split")


def kvq_decode_combine(cache: QuantizedKVCache, num_q_heads: int, max_seq_len: int, workspace: torch.Tensor,
                       out: torch.Tensor, num_splits: int = 0, stream=None) -> torch.Tensor:
    """Stage 2 of kvq_decode_attention: merge the split partials into `out`."""
    _check(lib().kvq_decode_combine(ctypes.byref(cache.cfg), num_q_heads, max_seq_len, num_splits, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _ptr(out), _DTYPE[out.dtype],
                                    _stream(stream)), "kvq_decode_combine")
    return out


NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


def kvq_decode_attention_noalloc(cache: QuantizedKVCache, q: torch.Tensor, softmax_scale: float, max_seq_len: int,
                                 num_splits: int = 0, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                                 stream=None) -> torch.Tensor:
    """kvq_decode_attention without a workspace, for callers that may not
    allocate device memory while they decode (the library's own fixed scratch
    holds the split partials).  `out` should be passed by such callers; it is
    allocated here only as a convenience when omitted.  Concurrent calls on
    different streams share that scratch and must be serialised."""
    assert q.dtype == torch.bfloat16 and q.is_contiguous() and q.dim() == 3
    if out is None:
        out = _made_on(stream, lambda: torch.empty(q.shape, dtype=out_dtype, device=q.device), returned=True)
    st = lib().kvq_decode_attention_noalloc(ctypes.byref(cache.cfg), ctypes.byref(cache.c), _ptr(q), q.shape[1],
                                            float(softmax_scale), max_seq_len, num_splits, _ptr(out),
                                            _DTYPE[out.dtype], _stream(stream))
    if st == KVQ_ERR_WORKSPACE:
        need = kvq_decode_workspace_bytes(cache, q.shape[1], max_seq_len, num_splits)
        raise KVQError(st, f"kvq_decode_attention_noalloc: split partials need {need} bytes, more than the "
                           f"{NOALLOC_SCRATCH_BYTES}-byte built-in scratch")
    _check(st, "kvq_decode_attention_noalloc")
    return out


KVQ_TREE_MAX_NODES = 64


# These calls are short, so their binding is lean: the checks read each tensor's
# properties once, and pointers go to ctypes as plain integers.
def _check_on(index: int, *tensors):
    """Every tensor (None apart) lies on CUDA device `index`."""
    for t in tensors:
        if t is not None and (index < 0 or t.get_device() != index):
            raise ValueError(f"a tensor on {t.device} beside a cache on CUDA device {index}")


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _call(what: str, index: int, stream, *args):
    """The library's function `what` with `args` and the stream, device `index` current; stream None
    is that device's current stream."""
    f = getattr(_lib or lib(), what)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = f(*args, raw)
    else:
        with torch.cuda.device(index):
            status = f(*args, raw)
    if status != KVQ_OK:
        raise KVQError(status, what)


def _refs(cache: "QuantizedKVCache"):
    """References to the cache's C structures, and its device."""
    return ctypes.byref(cache.cfg), ctypes.byref(cache.c), cache.pool.get_device()


def kvq_tree_workspace_bytes(cache: QuantizedKVCache, num_q_heads: int, num_nodes: int, max_seq_len: int,
                             num_splits: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(lib().kvq_tree_workspace_bytes(ctypes.byref(cache.cfg), num_q_heads, num_nodes, max_seq_len, num_splits,
                                          ctypes.byref(n)), "kvq_tree_workspace_bytes")
    return n.value


def alloc_tree_workspace(cache: QuantizedKVCache, num_q_heads: int, num_nodes: int, max_seq_len: int,
                         num_splits: int = 0) -> torch.Tensor:
    """A workspace for kvq_tree_attention calls of this shape (needs no initialisation)."""
    nbytes = kvq_tree_workspace_bytes(cache, num_q_heads, num_nodes, max_seq_len, num_splits)
    return torch.empty((nbytes + 15) // 16 * 4, dtype=torch.float32, device=cache.device)


def tree_mask_from_parents(parents) -> torch.Tensor:
    """Ancestor words (int64, CPU) of trees given by parent indices [.., T] (a
    parent comes before its children, -1 for a root): each node attends to
    itself and its ancestors."""
    p = torch.as_tensor(parents).to("cpu", torch.int64)
    T = p.shape[-1]
    if T > KVQ_TREE_MAX_NODES or bool((p >= torch.arange(T)).any()) or bool((p < -1).any()):
        raise ValueError("parents: at most 64 nodes, each parent before its children, -1 for a root")
    words = torch.zeros_like(p)
    for t in range(T):
        up = words.gather(-1, p[..., t:t + 1].clamp_min(0)) * (p[..., t:t + 1] >= 0)
        words[..., t:t + 1] = up | (-(1 << 63) if t == 63 else 1 << t)
    return words


def kvq_tree_attention(cache: QuantizedKVCache, q: torch.Tensor, softmax_scale: float, max_seq_len: int,
                       k_tree: torch.Tensor | None = None, v_tree: torch.Tensor | None = None,
                       tree_mask: torch.Tensor | None = None, nodes_per_seq: torch.Tensor | None = None,
                       num_splits: int = 0, out: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                       lse: torch.Tensor | None = None, page_lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q: [num_seqs, T, Hq, D] bf16 -> out [num_seqs, T, Hq, D] (bf16 or f32); T <= 64 drafted
    tokens with k_tree, v_tree [num_seqs, T, Hkv, D] bf16 (None: the cache alone).
    tree_mask: int64 ancestor words [T] or [num_seqs, T] (None: a chain).  lse fp32
    [num_seqs, T, Hq] and page_lse fp32 [num_seqs, T, Hq, ceil(max_seq_len / 16)] are
    filled when given."""
    cfg, (pcfg, pcache, index) = cache.cfg, _refs(cache)
    assert q.dtype is torch.bfloat16 and q.is_contiguous() and q.dim() == 4
    shape = q.shape
    B, T, Hq, D = shape
    assert B == cfg.num_seqs and D == cfg.head_dim
    assert (k_tree is None) == (v_tree is None)
    if k_tree is not None:
        kv = (B, T, cfg.num_kv_heads, D)
        assert k_tree.dtype is torch.bfloat16 and k_tree.is_contiguous() and k_tree.shape == kv
        assert v_tree.dtype is torch.bfloat16 and v_tree.is_contiguous() and v_tree.shape == kv
    per_seq = 0
    if tree_mask is not None:
        per_seq = tree_mask.dim() - 1
        assert tree_mask.dtype is torch.int64 and tree_mask.is_contiguous()
        assert tree_mask.shape == ((B, T) if per_seq else (T,))
    if nodes_per_seq is not None:
        assert nodes_per_seq.dtype is torch.int32 and nodes_per_seq.is_contiguous() and nodes_per_seq.shape == (B,)
    if out is None:
        out = _made_on(stream, lambda: torch.empty(shape, dtype=out_dtype, device=q.device), returned=True)
    dt = _DTYPE[out.dtype]
    assert dt != KVQ_F16 and out.is_contiguous() and out.shape == shape
    if lse is not None:
        assert lse.dtype is torch.float32 and lse.is_contiguous() and lse.shape == (B, T, Hq)
    if page_lse is not None:
        P = (min(max_seq_len, 16 * cfg.pages_per_seq_max) + 15) // 16
        assert page_lse.dtype is torch.float32 and page_lse.is_contiguous() and page_lse.shape == (B, T, Hq, P)
    if workspace is None:
        workspace = _made_on(stream, lambda: alloc_tree_workspace(cache, Hq, T, max_seq_len, num_splits))
    _check_on(index, q, k_tree, v_tree, tree_mask, nodes_per_seq, out, lse, page_lse, workspace)
    _call("kvq_tree_attention", index, stream, pcfg, pcache, q.data_ptr(), Hq, T, _addr(k_tree), _addr(v_tree),
          _addr(tree_mask), per_seq, _addr(nodes_per_seq), float(softmax_scale), max_seq_len, num_splits, out.data_ptr(), dt,
          _addr(lse), _addr(page_lse), workspace.data_ptr(), workspace.nbytes)
    return out


def kvq_page_mass(cache: QuantizedKVCache, lse: torch.Tensor, page_lse: torch.Tensor, mass: torch.Tensor,
                  node_mask: torch.Tensor | None = None, decay: float = 1.0, mass_out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """mass_out = decay * mass + the page weights of the marked nodes (node_mask int64
    [num_seqs], bit t = node t; None: all).  lse [num_seqs, T, Hq] and page_lse
    [num_seqs, T, Hq, P] as kvq_tree_attention wrote them; mass fp32 [num_seqs,
    pages_per_seq_max], updated in place unless mass_out is given."""
    cfg, (pcfg, _, index) = cache.cfg, _refs(cache)
    B, T, Hq, P = page_lse.shape
    if mass_out is None:
        mass_out = mass
    f32, shape = torch.float32, (B, cfg.pages_per_seq_max)
    assert B == cfg.num_seqs and lse.shape == (B, T, Hq) and mass.shape == shape and mass_out.shape == shape
    assert lse.dtype is f32 and page_lse.dtype is f32 and mass.dtype is f32 and mass_out.dtype is f32
    assert lse.is_contiguous() and page_lse.is_contiguous() and mass.is_contiguous() and mass_out.is_contiguous()
    if node_mask is not None:
        assert node_mask.dtype is torch.int64 and node_mask.is_contiguous() and node_mask.shape == (B,)
    _check_on(index, lse, page_lse, mass, node_mask, mass_out)
    _call("kvq_page_mass", index, stream, pcfg, Hq, T, P, lse.data_ptr(), page_lse.data_ptr(), _addr(node_mask), float(decay),
          mass.data_ptr(), mass_out.data_ptr())
    return mass_out


def kvq_evict_pages(cache: QuantizedKVCache, mass: torch.Tensor, keep_pages: int, sink_pages: int = 0,
                    recent_pages: int = 0, page_table_out: torch.Tensor | None = None,
                    seq_lens_out: torch.Tensor | None = None, mass_out: torch.Tensor | None = None,
                    evicted: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Evict the lightest full pages of every sequence down to keep_pages; returns the int32
    [num_seqs] counts.  Updates cache.page_table, cache.seq_lens and mass in place, each
    unless its output tensor is given."""
    cfg, (pcfg, pcache, index) = cache.cfg, _refs(cache)
    B = cfg.num_seqs
    shape = (B, cfg.pages_per_seq_max)
    page_table_out = cache.page_table if page_table_out is None else page_table_out
    seq_lens_out = cache.seq_lens if seq_lens_out is None else seq_lens_out
    mass_out = mass if mass_out is None else mass_out
    if evicted is None:
        evicted = _made_on(stream, lambda: torch.empty(B, dtype=torch.int32, device=cache.device), returned=True)
    f32, i32 = torch.float32, torch.int32
    assert mass.dtype is f32 and mass_out.dtype is f32 and mass.is_contiguous() and mass_out.is_contiguous()
    assert mass.shape == shape and mass_out.shape == shape and page_table_out.shape == shape
    assert page_table_out.dtype is i32 and seq_lens_out.dtype is i32 and evicted.dtype is i32
    assert page_table_out.is_contiguous() and seq_lens_out.is_contiguous() and evicted.is_contiguous()
    assert seq_lens_out.shape == (B,) and evicted.shape == (B,)
    _check_on(index, mass, page_table_out, seq_lens_out, mass_out, evicted)
    _call("kvq_evict_pages", index, stream, pcfg, pcache, mass.data_ptr(), keep_pages, sink_pages, recent_pages,
          page_table_out.data_ptr(), seq_lens_out.data_ptr(), mass_out.data_ptr(), evicted.data_ptr())
    return evicted


def _token_rows(t: torch.Tensor, heads: int, D: int):
    """(rows, elements from a row to the next) of a tensor [..., heads, D] whose last two dimensions are
    dense and whose others step evenly: a contiguous tensor, or a part of one projection's rows."""
    shape = t.shape
    if len(shape) < 3 or shape[-1] != D or shape[-2] != heads:
        raise ValueError(f"a tensor of shape {tuple(shape)} where [..., {heads}, {D}] is wanted")
    if t.is_contiguous():
        return t.numel() // (heads * D), heads * D
    strides = t.stride()
    if len(shape) == 3 and strides[2] == 1 and (heads == 1 or strides[1] == D):   # (what the loop below says, for one dimension)
        return shape[0], strides[0] if shape[0] != 1 else heads * D
    rows, step = 1, None
    for i in range(len(shape) - 3, -1, -1):
        n = shape[i]
        if n != 1:
            if step is None:
                step = strides[i]
            elif strides[i] != step * rows:
                raise ValueError(f"rows of a tensor with strides {strides} are not evenly spaced")
            rows *= n
    if strides[-1] != 1 or (heads > 1 and strides[-2] != D):
        raise ValueError(f"a tensor with strides {strides}: the heads of a row have to be contiguous")
    return rows, heads * D if step is None else step


def kvq_norm_rope(cache: QuantizedKVCache, q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None,
                  inv_freq: torch.Tensor | None, q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                  eps: float | None = 1e-6, interleaved: bool = False, pair_axis=None, q_out: torch.Tensor | None = None,
                  k_out: torch.Tensor | None = None, out_dtype=None, stream=None):
    """Per-head RMS norm (eps None: none) of q [..., Hq, D] and k [..., Hkv, D] (bf16, f16 or f32; either may be
    None) and their rotary positions in one pass; returns (q_out, k_out).  positions: int32, one a row ([rows] or
    q's leading shape), or [axes, rows] with pair_axis, the axis of each of the rot_dim / 2 pairs (a sequence).
    inv_freq: fp32 [rot_dim / 2] (None: norms alone).  q_weight, k_weight: fp32 [D] gains (None: ones).  The outputs
    may be the inputs."""
    cfg, (pcfg, _, index) = cache.cfg, _refs(cache)
    D, Hkv = cfg.head_dim, cfg.num_kv_heads
    x = k if q is None else q
    if x is None:
        raise ValueError("q or k is wanted")
    dtype = x.dtype
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else k_out.dtype if k_out is not None else dtype
    Hq = rows = qp = qs = qop = qos = kp = ks = kop = kos = 0
    if q is None:
        q_out = None
    else:
        Hq = q.shape[-2]
        rows, qs = _token_rows(q, Hq, D)
        if q_out is None:
            q_out = _made_on(stream, lambda: torch.empty(q.shape, dtype=out_dtype, device=q.device), returned=True)
        n, qos = _token_rows(q_out, Hq, D)
        if n != rows or q_out.dtype is not out_dtype:
            raise ValueError(f"q_out: {n} rows of {q_out.dtype} for {rows} of {out_dtype}")
        qp, qop = q.data_ptr(), q_out.data_ptr()
    if k is None:
        k_out = None
    else:
        n, ks = _token_rows(k, Hkv, D)
        if k.dtype is not dtype or (q is not None and n != rows):
            raise ValueError(f"k: {n} rows of {k.dtype} beside {rows} of {dtype}")
        rows = n
        if k_out is None:
            k_out = _made_on(stream, lambda: torch.empty(k.shape, dtype=out_dtype, device=k.device), returned=True)
        n, kos = _token_rows(k_out, Hkv, D)
        if n != rows or k_out.dtype is not out_dtype:
            raise ValueError(f"k_out: {n} rows of {k_out.dtype} for {rows} of {out_dtype}")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    rot, axes, pp, fp, pairs = 0, 1, None, None, None
    if inv_freq is not None:
        assert inv_freq.dtype is torch.float32 and inv_freq.dim() == 1 and inv_freq.is_contiguous()
        assert positions is not None and positions.dtype is torch.int32 and positions.is_contiguous()
        rot, pp, fp = 2 * inv_freq.numel(), positions.data_ptr(), inv_freq.data_ptr()
        if pair_axis is not None:
            axes = positions.shape[0]
        if positions.numel() != axes * rows:
            raise ValueError(f"{positions.numel()} positions for {rows} rows of {axes} axes")
    if pair_axis is not None:
        if len(pair_axis) != rot // 2 or (rot and not 0 <= min(pair_axis) <= max(pair_axis) < axes):
            raise ValueError(f"pair_axis: an axis below {axes} for each of the {rot // 2} pairs")
        pairs = bytes(list(pair_axis))   # (not an array's own bytes)
    if q_weight is not None:
        assert q_weight.dtype is torch.float32 and q_weight.is_contiguous() and q_weight.shape == (D,)
    if k_weight is not None:
        assert k_weight.dtype is torch.float32 and k_weight.is_contiguous() and k_weight.shape == (D,)
    if eps is None:
        eps = -1.0
    else:
        eps = float(eps)
        if not eps >= 0:
            raise ValueError("eps has to be at least 0 (None: no norm)")
    _check_on(index, q, k, q_out, k_out, None if rot == 0 else positions, inv_freq, q_weight, k_weight)
    if rows:
        _call("kvq_norm_rope", index, stream, pcfg, qp or None, qs, Hq, kp or None, ks, _DTYPE[dtype], rows, _addr(q_weight),
              _addr(k_weight), eps, pp, axes, fp, rot, pairs, 1 if interleaved else 0, qop or None, qos, kop or None, kos,
              _DTYPE[out_dtype])
    return q_out, k_out


def kvq_prompt_attention(cache: QuantizedKVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, softmax_scale: float,
                         t_per_seq: torch.Tensor | None = None, first_row: torch.Tensor | None = None, t_new: int | None = None,
                         causal: bool = True, out: torch.Tensor | None = None, out_dtype=None, lse: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Attention of whole prompts, each over its own tokens (causal or full).  A padded batch: q [num_seqs, t_new,
    Hq, D], k and v [num_seqs, t_new, Hkv, D] (bf16 or f16), sequence b's first t_per_seq[b] tokens (int32
    [num_seqs]; None: all).  Packed sequences: q [rows, Hq, D], ..., first_row and t_per_seq int32 [num_seqs] on the
    device, t_new a bound on the lengths.  lse: fp32 of q's leading shape x Hq, filled when given.  Rows of no
    sequence are left as they were (an `out` made here: uninitialised)."""
    cfg, (pcfg, _, index) = cache.cfg, _refs(cache)
    B, D = cfg.num_seqs, cfg.head_dim
    shape, dtype = q.shape, q.dtype
    Hq = shape[-2]
    code = _DTYPE[dtype]
    if code == KVQ_F32 or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("q, k and v have to be of one type, bf16 or f16")
    if first_row is not None:
        if t_per_seq is None or t_new is None:
            raise ValueError("packed sequences: t_per_seq and t_new are wanted")
        assert len(shape) == 3 and first_row.dtype is torch.int32 and first_row.is_contiguous() and first_row.shape == (B,)
    else:
        assert len(shape) == 4 and shape[0] == B and t_new in (None, shape[1])
        t_new = shape[1]
    if t_per_seq is not None:
        assert t_per_seq.dtype is torch.int32 and t_per_seq.is_contiguous() and t_per_seq.shape == (B,)
    rows, qs = _token_rows(q, Hq, D)
    kshape, Hkv = k.shape, cfg.num_kv_heads
    _, ks = _token_rows(k, Hkv, D)
    _, vs = _token_rows(v, Hkv, D)
    if out is None:
        made = out_dtype or dtype
        out = _made_on(stream, lambda: torch.empty(shape, dtype=made, device=q.device), returned=True)
    od = out.dtype
    assert kshape[:-2] == shape[:-2] and v.shape == kshape and out.shape == shape
    assert (od is dtype or od is torch.float32) and out_dtype in (None, od)
    _, outs = _token_rows(out, Hq, D)
    if lse is not None:
        assert lse.dtype is torch.float32 and lse.is_contiguous() and lse.shape == shape[:-1]
    _check_on(index, q, k, v, t_per_seq, first_row, out, lse)
    if rows:
        _call("kvq_prompt_attention", index, stream, pcfg, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, code, Hq, rows,
              _addr(first_row), _addr(t_per_seq), t_new, float(softmax_scale), 1 if causal else 0, out.data_ptr(), outs, _DTYPE[od],
              _addr(lse), cache.status.data_ptr())
    return out


def kvq_dequantize(cache: QuantizedKVCache, seq: int, kv_head: int, which: int, tok_begin: int, tok_end: int,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Values tokens [tok_begin, tok_end) of (seq, kv_head, K=0 / V=1) stand for, fp32 [n, D]."""
    if out is None:
        shape = (max(tok_end - tok_begin, 0), cache.head_dim)
        out = _made_on(stream, lambda: torch.empty(shape, dtype=torch.float32, device=cache.device), returned=True)
    _check(lib().kvq_dequantize(ctypes.byref(cache.cfg), ctypes.byref(cache.c), seq, kv_head, which, tok_begin,
                                tok_end, _ptr(out), _stream(stream)), "kvq_dequantize")
    return out
