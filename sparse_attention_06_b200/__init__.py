"""Python binding of the DSA hot-path library (``libdsa.so``, C ABI in ``include/dsa.h``).

Argument marshalling only: every function below takes torch CUDA tensors, checks that they are
laid out as the C ABI expects, and calls the C entry point of the same name.  Every step of the
path runs in the library's CUDA kernels; there is no Python or CPU fallback, and calling any
function without the built library raises ``DsaLibraryMissing``.

Build the library with ``python -m sparse_attention_06_b200.build`` (nvcc, sm_100a).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA, DSA_ERR_DEVICE_FAULT = range(5)
DSA_F32, DSA_BF16, DSA_E4M3, DSA_LATENT_E4M3 = 0, 1, 2, 3

LATENT_E4M3_DIM, LATENT_E4M3_BYTES = 576, 640  # elements and data bytes of a quantised latent row

DEVERR_BLOCK_ID = 1
DEVERR_INDEX = 2
DEVERR_REQUEST = 4
DEVERR_NAN_SCORE = 8
DEVERR_TIMEOUT = 16
DEVERR_QUERY_GROUP = 32
DEVERR_SCALE = 64
DEVERR_NONFINITE = 128

# Symbols the C ABI exports (checked by the CPU test suite).
EXPORTED = (
    "dsa_indexer_scores", "dsa_topk_select", "dsa_indexer_topk", "dsa_sparse_mla_decode",
    "dsa_sparse_mla_prefill", "dsa_mla_workspace_size", "dsa_get_device_error",
    "dsa_clear_device_error", "dsa_status_string", "dsa_last_error_message", "dsa_abi_version",
    "dsa_kernel_launch_count", "dsa_sparse_mla_decode_noalloc", "dsa_selftest_bounded_wait",
    "dsa_indexer_topk_workspace_size", "dsa_selftest_gather_rate", "dsa_cache_append", "dsa_cache_read",
    "dsa_chunk_mla", "dsa_chunk_mla_workspace_size",
)


class DsaLibraryMissing(RuntimeError):
    pass


class DsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s (status %d)" % (message, status))
        self.status = status


class _PagedCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64),
                ("block_size", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("num_queries", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
                ("q_req", ctypes.c_void_p), ("q_pos", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32),
                ("max_context", ctypes.c_int32), ("query_group", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _Chunks(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_reqs", ctypes.c_int32),
                ("cu_tokens", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32),
                ("max_context", ctypes.c_int32)]


_lib = None


def load_library():
    """Load libdsa.so (raises DsaLibraryMissing if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise DsaLibraryMissing(
            "libdsa.so not found at %s; build it with `python -m sparse_attention_06_b200.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    PC, PB, PK = ctypes.POINTER(_PagedCache), ctypes.POINTER(_Batch), ctypes.POINTER(_Chunks)
    sig = {
        "dsa_indexer_scores": [P, I32, P, I32, I32, P, PC, PB, P, I64, P, P],
        "dsa_topk_select": [P, I64, P, I32, I32, P, P, P],
        "dsa_indexer_topk": [P, I32, P, I32, I32, P, PC, PB, I32, P, I64, P, P, ctypes.c_size_t, P],
        "dsa_sparse_mla_decode": [P, I32, I32, I32, I32, PC, PB, P, I32, F, P, P, P, ctypes.c_size_t, P],
        "dsa_sparse_mla_prefill": [P, I32, I32, I32, I32, PC, PB, P, I32, F, P, P, P, ctypes.c_size_t, P],
        "dsa_sparse_mla_decode_noalloc": [P, I32, I32, I32, I32, PC, PB, P, I32, F, P, P, P],
        "dsa_cache_append": [P, I64, P, I64, I32, PC, PC, PK, P],
        "dsa_cache_read": [PC, PK, P, I32, P],
        "dsa_chunk_mla": [P, I32, I32, I32, I32, PC, PK, F, P, P, P, ctypes.c_size_t, P],
        "dsa_get_device_error": [ctypes.POINTER(I32), P],
        "dsa_clear_device_error": [P],
        "dsa_selftest_bounded_wait": [I64, P],
        "dsa_selftest_gather_rate": [PC, P, I32, I32, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.dsa_mla_workspace_size.argtypes = [I32, I32, I32, I32]
    lib.dsa_mla_workspace_size.restype = ctypes.c_size_t
    lib.dsa_indexer_topk_workspace_size.argtypes = [I32]
    lib.dsa_indexer_topk_workspace_size.restype = ctypes.c_size_t
    lib.dsa_chunk_mla_workspace_size.argtypes = [I32, I32, I32, I32, I32]
    lib.dsa_chunk_mla_workspace_size.restype = ctypes.c_size_t
    lib.dsa_status_string.argtypes = [ctypes.c_int]
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_last_error_message.restype = ctypes.c_char_p
    lib.dsa_abi_version.restype = I32
    lib.dsa_kernel_launch_count.restype = I64
    _lib = lib
    return lib


def _check(status: int):
    if status != DSA_OK:
        lib = load_library()
        msg = (lib.dsa_last_error_message() or b"").decode() or lib.dsa_status_string(status).decode()
        raise DsaError(status, msg)


# A device's current stream without the wrapper object torch.cuda builds (0.1 us for 1.3).  It neither initialises CUDA nor
# notices a forked process; torch.cuda.current_device, which every call asks first, does both.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev_ptr(t: Optional[torch.Tensor], what: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


_DTYPE_CODES = {torch.float32: DSA_F32, torch.bfloat16: DSA_BF16, torch.uint8: DSA_E4M3,
                torch.float8_e4m3fn: DSA_E4M3}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return code


@dataclasses.dataclass
class PagedCache:
    """A paged per-token cache: data [num_blocks, block_size, dim] (f32 / bf16 / e4m3 codes as
    uint8), scale [num_blocks, block_size] (or [num_blocks, block_size, 1]) f32 for e4m3.  A quantised latent cache has data
    [num_blocks, 64, 640] uint8 (512 e4m3 codes, 64 RoPE elements in bf16) and scale
    [num_blocks, 64, 4] f32, powers of two (include/dsa.h)."""
    data: torch.Tensor
    scale: Optional[torch.Tensor] = None

    @property
    def dim(self) -> int:
        """Elements of a row."""
        return LATENT_E4M3_DIM if self._quantised_latent() else self.data.shape[2]

    def _quantised_latent(self) -> bool:
        # (scales [num_blocks, 64, 1] are a key cache's, one per row)
        scale = self.scale
        return scale is not None and scale.dim() == 3 and scale.shape[2] != 1 and _DTYPE_CODES.get(self.data.dtype) == DSA_E4M3

    def _c(self) -> _PagedCache:
        data, scale = self.data, self.scale
        nb, bs, dim = data.shape
        dtype = _dtype_code(data)
        if dtype == DSA_E4M3 and scale is not None:
            shape = scale.shape
            if len(shape) == 3 and shape[2] != 1:
                if dim != LATENT_E4M3_BYTES:
                    raise ValueError("a quantised latent cache has data [num_blocks, 64, 640] uint8")
                if scale.dtype is not torch.float32 or shape != (nb, bs, 4):
                    raise ValueError("a quantised latent cache has scale [num_blocks, 64, 4] float32")
                dim, dtype = LATENT_E4M3_DIM, DSA_LATENT_E4M3
            elif scale.dtype is not torch.float32 or scale.numel() < nb * bs:
                # the calls read, and an append writes, one f32 per row through it
                raise ValueError("an e4m3 cache has scale [num_blocks, block_size] float32")
        return _PagedCache(_dev_ptr(data, "cache data"), _dev_ptr(scale, "cache scale"), nb, bs, dim, dtype, 0)


@dataclasses.dataclass
class Batch:
    """Queries of one call: q_req [T], q_pos [T] and block_table [B, max_blocks] int32 CUDA
    tensors; max_context bounds q_pos + 1 (host int); query_group as in dsa.h."""
    q_req: torch.Tensor
    q_pos: torch.Tensor
    block_table: torch.Tensor
    max_context: int
    query_group: int = 1

    def _c(self) -> _Batch:
        for n in ("q_req", "q_pos", "block_table"):
            if getattr(self, n).dtype != torch.int32:
                raise ValueError("%s must be int32" % n)
        B, mb = self.block_table.shape
        return _Batch(self.q_req.numel(), B, _dev_ptr(self.q_req, "q_req"), _dev_ptr(self.q_pos, "q_pos"),
                      _dev_ptr(self.block_table, "block_table"), mb, int(self.max_context),
                      int(self.query_group), 0)


@dataclasses.dataclass
class Chunks:
    """Chunks of new tokens of several requests, side by side: cu_tokens [B + 1], seq_len [B] and
    block_table [B, max_blocks] int32 CUDA tensors; max_context bounds seq_len (host int)."""
    cu_tokens: torch.Tensor
    seq_len: torch.Tensor
    block_table: torch.Tensor
    max_context: int

    def _c(self, num_tokens) -> _Chunks:
        cu, seq, table = self.cu_tokens, self.seq_len, self.block_table
        i32 = torch.int32
        if cu.dtype is not i32 or seq.dtype is not i32 or table.dtype is not i32:
            raise ValueError("cu_tokens, seq_len and block_table must be int32")
        B, mb = table.shape
        if cu.shape != (B + 1,) or seq.shape != (B,):
            raise ValueError("cu_tokens must have B + 1 entries and seq_len B, for the B rows of block_table")
        return _Chunks(num_tokens, B, _dev_ptr(cu, "cu_tokens"), _dev_ptr(seq, "seq_len"),
                       _dev_ptr(table, "block_table"), mb, int(self.max_context))


def _same_device(*tensors) -> int:
    """The library runs on the current device: every tensor has to be there.  Returns the device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensor on %s, but the current device is cuda:%d" % (t.device, dev))
    return dev


def dsa_indexer_scores(q, w, keys: PagedCache, batch: Batch, scores, stream=None, q_scale=None, key_hist=None):
    """scores[t, s] = sum_h w[t,h] ReLU(qhat[t,h] . khat[s]) for s <= q_pos[t] (include/dsa.h);
    e4m3 queries (uint8 codes) come with q_scale [T, Hi] f32; key_hist [T, 4096] int32/uint32
    (optional) receives the scores' order-key digit counts."""
    lib = load_library()
    T, Hi, Di = q.shape
    kc, bc = keys._c(), batch._c()
    _check(lib.dsa_indexer_scores(_dev_ptr(q, "q"), _dtype_code(q), _dev_ptr(q_scale, "q_scale"), Hi, Di,
                                  _dev_ptr(w, "w"), ctypes.byref(kc), ctypes.byref(bc), _dev_ptr(scores, "scores"),
                                  scores.shape[1], _dev_ptr(key_hist, "key_hist"), _stream(stream)))
    return scores


def dsa_topk_select(scores, q_pos, k, idx, stream=None, key_hist=None):
    """idx[t] = the k best positions of scores[t, :q_pos[t]+1], ascending, -1 padded; key_hist
    (optional) places the threshold and is left zeroed (include/dsa.h)."""
    lib = load_library()
    _check(lib.dsa_topk_select(_dev_ptr(scores, "scores"), scores.shape[1], _dev_ptr(q_pos, "q_pos"),
                               q_pos.numel(), k, _dev_ptr(idx, "idx"), _dev_ptr(key_hist, "key_hist"),
                               _stream(stream)))
    return idx


def dsa_indexer_topk(q, w, keys: PagedCache, batch: Batch, k, scores, idx, stream=None, q_scale=None,
                     workspace=None):
    """Indexer scores fused with the top-K selection; workspace (optional, zero-filled before its
    first use, left zero-filled) holds the order-key digit histograms (include/dsa.h)."""
    lib = load_library()
    T, Hi, Di = q.shape
    kc, bc = keys._c(), batch._c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.dsa_indexer_topk(_dev_ptr(q, "q"), _dtype_code(q), _dev_ptr(q_scale, "q_scale"), Hi, Di,
                                _dev_ptr(w, "w"), ctypes.byref(kc), ctypes.byref(bc), k, _dev_ptr(scores, "scores"),
                                scores.shape[1], _dev_ptr(idx, "idx"), _dev_ptr(workspace, "workspace"), ws_bytes,
                                _stream(stream)))
    return idx


def dsa_indexer_topk_workspace_size(num_queries) -> int:
    return int(load_library().dsa_indexer_topk_workspace_size(num_queries))


def _mla(fn_name, q, latent: PagedCache, batch: Batch, idx, softmax_scale, out, lse, workspace, stream, k=None):
    lib = load_library()
    T, H, dqk = q.shape
    d_v = out.shape[-1]
    lc, bc = latent._c(), batch._c()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if k is None:
        k = idx.shape[1] if idx is not None else int(batch.max_context)
    _check(getattr(lib, fn_name)(_dev_ptr(q, "q"), _dtype_code(q), H, d_v, dqk - d_v, ctypes.byref(lc),
                                 ctypes.byref(bc), _dev_ptr(idx, "idx"), int(k), float(softmax_scale),
                                 _dev_ptr(out, "out"), _dev_ptr(lse, "lse"), _dev_ptr(workspace, "workspace"),
                                 ws_bytes, _stream(stream)))
    return out


def dsa_sparse_mla_decode(q, latent: PagedCache, batch: Batch, idx, softmax_scale, out, lse=None,
                          workspace=None, stream=None, k=None):
    """Sparse MQA-mode MLA over the selected latent rows, split-K across CTAs (include/dsa.h).
    ``idx=None`` is the dense case: every visible position, with k (default max_context) rows."""
    return _mla("dsa_sparse_mla_decode", q, latent, batch, idx, softmax_scale, out, lse, workspace, stream, k)


def dsa_sparse_mla_prefill(q, latent: PagedCache, batch: Batch, idx, softmax_scale, out, lse=None,
                           workspace=None, stream=None, k=None):
    return _mla("dsa_sparse_mla_prefill", q, latent, batch, idx, softmax_scale, out, lse, workspace, stream, k)


def dsa_sparse_mla_decode_noalloc(q, latent: PagedCache, batch: Batch, idx, softmax_scale, out, lse=None,
                                  stream=None):
    """dsa_sparse_mla_decode for callers that cannot allocate device memory: the split partials
    live in the library's fixed 32 MiB device scratch (see include/dsa.h)."""
    lib = load_library()
    T, H, dqk = q.shape
    d_v = out.shape[-1]
    lc, bc = latent._c(), batch._c()
    _check(lib.dsa_sparse_mla_decode_noalloc(_dev_ptr(q, "q"), _dtype_code(q), H, d_v, dqk - d_v,
                                             ctypes.byref(lc), ctypes.byref(bc), _dev_ptr(idx, "idx"),
                                             idx.shape[1], float(softmax_scale), _dev_ptr(out, "out"),
                                             _dev_ptr(lse, "lse"), _stream(stream)))
    return out


def _rows(x, dim, what):
    """Pointer and row stride (elements) of [num_tokens, dim] inputs whose rows may be apart."""
    if x.dim() != 2 or x.shape[1] != dim:
        raise ValueError("%s must be [num_tokens, %d]" % (what, dim))
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    row, one = x.stride()
    if x.shape[0] == 1:
        row = dim
    if one != 1 or row < dim:
        raise ValueError("%s: the elements of a row must be contiguous, and rows must not overlap" % what)
    return x.data_ptr(), row


def dsa_cache_append(k, kv, keys: Optional[PagedCache], latent: Optional[PagedCache], chunks: Chunks, stream=None):
    """Writes the new tokens' indexer keys k [num_tokens, key dim] and latent rows kv
    [num_tokens, 576] into their paged caches, quantising where a cache is quantised
    (include/dsa.h).  k and keys, or kv and latent, may be None; rows of k and kv may be apart
    (a slice of a wider projection)."""
    lib = load_library()
    if (k is None) != (keys is None) or (kv is None) != (latent is None):
        raise ValueError("k comes with keys, and kv with latent")
    x = k if k is not None else kv
    if x is None:
        raise ValueError("nothing to append")
    T = x.shape[0]
    kp = vp = kc = lc = None
    ks = vs = 0
    if keys is not None:
        kc = keys._c()
        kp, ks = _rows(k, kc.dim, "k")
    if latent is not None:
        lc = latent._c()
        vp, vs = _rows(kv, lc.dim, "kv")
        if kv.shape[0] != T or kv.dtype is not x.dtype:
            raise ValueError("k and kv must have the same tokens and dtype")
    cc = chunks._c(T)
    dev = _same_device(k, kv, chunks.cu_tokens, chunks.seq_len, chunks.block_table, keys and keys.data,
                       keys and keys.scale, latent and latent.data, latent and latent.scale)
    if T == 0:
        return
    status = lib.dsa_cache_append(kp, ks, vp, vs, _dtype_code(x), kc, lc, cc, _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check(status)


def dsa_cache_read(cache: PagedCache, chunks: Chunks, out, stream=None):
    """out[t] = the values of the cached row at token t's position; out [num_tokens, row elements]
    bf16 or f32 (include/dsa.h)."""
    lib = load_library()
    c = cache._c()
    if out.dim() != 2 or out.shape[1] != c.dim:
        raise ValueError("out must be [num_tokens, %d]" % c.dim)
    T = out.shape[0]
    cc = chunks._c(T)
    dev = _same_device(cache.data, cache.scale, out, chunks.cu_tokens, chunks.seq_len, chunks.block_table)
    if T:
        status = lib.dsa_cache_read(c, cc, _dev_ptr(out, "out"), _dtype_code(out),
                                    _raw_stream(dev) if stream is None else _stream(stream))
        if status:
            _check(status)
    return out


def dsa_chunk_mla(q, latent: PagedCache, chunks: Chunks, softmax_scale, out, lse=None, workspace=None, stream=None):
    """Dense MQA-mode MLA of chunks of new tokens: the token at position p attends to the positions
    0..p of its request (include/dsa.h).  q [num_tokens, H, 576], out [num_tokens, H, 512],
    workspace of dsa_chunk_mla_workspace_size(...) bytes (uint8, its own for calls that may overlap)."""
    lib = load_library()
    T, H, dqk = q.shape
    d_v = out.shape[-1]
    if out.shape != (T, H, d_v) or out.dtype is not q.dtype:
        raise ValueError("out must be [num_tokens, H, d_v] of q's dtype")
    if lse is not None and (lse.shape != (T, H) or lse.dtype is not torch.float32):
        raise ValueError("lse must be [num_tokens, H] float32")
    lc, cc = latent._c(), chunks._c(T)
    dev = _same_device(q, latent.data, latent.scale, out, lse, workspace, chunks.cu_tokens, chunks.seq_len, chunks.block_table)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if T:
        status = lib.dsa_chunk_mla(_dev_ptr(q, "q"), _dtype_code(q), H, d_v, dqk - d_v, lc, cc, float(softmax_scale),
                                   _dev_ptr(out, "out"), _dev_ptr(lse, "lse"), _dev_ptr(workspace, "workspace"), ws_bytes,
                                   _raw_stream(dev) if stream is None else _stream(stream))
        if status:
            _check(status)
    return out


def dsa_chunk_mla_workspace_size(num_tokens, num_reqs, H, d_v, max_context) -> int:
    return int(load_library().dsa_chunk_mla_workspace_size(num_tokens, num_reqs, H, d_v, max_context))


def dsa_mla_workspace_size(num_queries, H, d_v, k) -> int:
    return int(load_library().dsa_mla_workspace_size(num_queries, H, d_v, k))


def dsa_get_device_error(stream=None) -> int:
    """Synchronises the stream and returns the device error word (0 = no fault)."""
    code = ctypes.c_int32(0)
    st = load_library().dsa_get_device_error(ctypes.byref(code), _stream(stream))
    if st not in (DSA_OK, DSA_ERR_DEVICE_FAULT):
        _check(st)
    return int(code.value)


def dsa_kernel_launch_count() -> int:
    """Kernels the library has enqueued in this process so far."""
    return int(load_library().dsa_kernel_launch_count())


def dsa_selftest_bounded_wait(limit_cycles, stream=None):
    """Diagnostic: a kernel whose bounded wait on a phase that never completes gives up after
    ``limit_cycles`` SM cycles and sets DEVERR_TIMEOUT (include/dsa.h)."""
    _check(load_library().dsa_selftest_bounded_wait(int(limit_cycles), _stream(stream)))


def dsa_selftest_gather_rate(latent: PagedCache, rows, tiles_per_cta, num_ctas, cycles, stream=None):
    """Diagnostic: gathers latent pool rows with the sparse MLA's TMA pattern and nothing else;
    rows: int32 [num_ctas * tiles_per_cta * 64] pool row indices; cycles: int64 [num_ctas]
    receives each CTA's SM cycles (include/dsa.h)."""
    if rows.dtype != torch.int32 or rows.numel() < num_ctas * tiles_per_cta * 64:
        raise ValueError("rows must be int32 with num_ctas * tiles_per_cta * 64 entries")
    if cycles.dtype != torch.int64 or cycles.numel() < num_ctas:
        raise ValueError("cycles must be int64 with num_ctas entries")
    lc = latent._c()
    _check(load_library().dsa_selftest_gather_rate(ctypes.byref(lc), _dev_ptr(rows, "rows"), int(tiles_per_cta),
                                                   int(num_ctas), _dev_ptr(cycles, "cycles"), _stream(stream)))
    return cycles


def dsa_clear_device_error(stream=None):
    _check(load_library().dsa_clear_device_error(_stream(stream)))
