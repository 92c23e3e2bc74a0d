"""Python binding of libcsa2.so, the GB300 CSA2 decode hot-path library.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams; tensors are passed by
``data_ptr()`` and the current CUDA stream.  The names follow the C ABI in
``include/csa2.h``.  Importing this module loads the library and raises if it
is missing -- there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, fields

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))  # package directory
LIB_PATH = os.path.join(_PKG, "_build", "libcsa2.so")

LATENT, ROPE, DQK, PAGE, BLOCK = 512, 64, 576, 64, 8
IDXK_E4M3, IDXK_F32, IDXK_FP4 = 0, 1, 2
MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2
MAX_QLEN = 4
IDX_EARLY_INPUTS = 1
KV_EARLY_INPUTS = 1
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_PARTS, ROPE_BASE = 0, 1, 2, 3
DENSE_ALL_POSITIONS = 1
IDX_NORM_NONE, IDX_NORM_RMS, IDX_NORM_LAYER = 0, 1, 2

STATUS = {0: "CSA2_OK", 1: "CSA2_ERR_INVALID_ARG", 2: "CSA2_ERR_UNSUPPORTED_SHAPE",
          3: "CSA2_ERR_WORKSPACE_TOO_SMALL", 4: "CSA2_ERR_CUDA",
          5: "CSA2_ERR_DEVICE_ASSERT", 6: "CSA2_ERR_TIMEOUT"}

# exported symbols and their ctypes signatures
_P, _I32, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


class CKernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_double)]


class CDims(ctypes.Structure):
    _fields_ = [("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("idx_k_dtype", ctypes.c_int32), ("pool_blocks", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("heads", ctypes.c_int32), ("swa", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("max_ctx", ctypes.c_int64)]


class CRope(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("mscale", ctypes.c_float), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_ctx", ctypes.c_double), ("turns_lo", ctypes.c_double), ("turns_hi", ctypes.c_double)]


SIGNATURES = {
    "csa2_version": (_I32, []),
    "csa2_status_string": (ctypes.c_char_p, [_I32]),
    "csa2_workspace_size": (_I32, [ctypes.POINTER(CDims), _I32, ctypes.POINTER(_SZ)]),
    "fp4_kv_quantize": (_I32, [_P, _I64, _P, _P, _P]),
    "fp4_kv_quantize_scatter": (_I32, [_P, _I64, _P, _P, _P, _P]),
    "fp4_kv_quantize_scatter_ex": (_I32, [_P, _I64, _P, _P, _P, _I32, _P]),
    "fp4_idx_k_quantize_scatter": (_I32, [_P, _I64, _P, _P, _I64, _P]),
    "fp4_kv_dequantize": (_I32, [_P, _P, _I64, _P, _P]),
    "indexer_full_topk": (_I32, [ctypes.POINTER(CDims), _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _P, _SZ, _P]),
    "indexer_reindex_topk": (_I32, [ctypes.POINTER(CDims), _I32, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _SZ, _P]),
    "indexer_full_topk_ex": (_I32, [ctypes.POINTER(CDims), _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _SZ, _P]),
    "indexer_reindex_topk_ex": (_I32, [ctypes.POINTER(CDims), _I32, _I32, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _SZ, _P]),
    "csa2_sparse_attn_decode": (_I32, [ctypes.POINTER(CDims), _I32, _I32, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _P, _F, _P, _P, _P, _SZ, _P]),
    "csa2_sparse_attn_decode_mq": (_I32, [ctypes.POINTER(CDims), _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                          _P, _P, _P, _P, _F, _P, _P, _P, _SZ, _P]),
    "csa2_sparse_attn_decode_noalloc": (_I32, [ctypes.POINTER(CDims), _I32, _I32, _P, _P, _P, _P,
                                               _P, _P, _P, _P, _P, _F, _P, _P, _P, _P]),
    "csa2_rope_apply": (_I32, [ctypes.POINTER(CRope), _I32, _P, _P, _P, _I64, _I32, _I32, _I32, _I64, _I64, _I64,
                               _I64, _I32, _P]),
    "csa2_kv_append": (_I32, [ctypes.POINTER(CRope), _P, _I64, _I64, _P, _F, _P, _P, _P, _P, _P, _I64, _P, _P]),
    "csa2_dense_attn_workspace_size": (_I32, [ctypes.POINTER(CDims), _I32, _I64, ctypes.POINTER(_SZ)]),
    "csa2_dense_attn_chunk": (_I32, [ctypes.POINTER(CDims), _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _F, _I32, _I32,
                                     _P, _P, _P, _SZ, _P]),
    "csa2_window_append": (_I32, [ctypes.POINTER(CRope), _P, _I64, _I64, _P, _F, _P, _P, _P, _I64, _P]),
    "csa2_idx_k_append": (_I32, [ctypes.POINTER(CRope), _I32, _P, _I64, _I64, _I32, _I32, _P, _P, _F, _P, _P, _P, _I64, _P]),
    "csa2_window_attn_workspace_size": (_I32, [ctypes.POINTER(CDims), _I32, _I64, ctypes.POINTER(_SZ)]),
    "csa2_window_attn_chunk": (_I32, [ctypes.POINTER(CDims), _I32, _I64, _P, _P, _P, _P, _P, _F, _I32, _I32, _P, _P, _P, _P,
                                      _P, _SZ, _P]),
    "csa2_get_device_status": (_I32, [_P, _P, ctypes.POINTER(_I32)]),
    "csa2_profile_enable": (_I32, [_I32]),
    "csa2_profile_read": (_I32, [ctypes.POINTER(CKernelTime), _I32, ctypes.POINTER(_I32)]),
    "csa2_clear_device_status": (_I32, [_P, _P]),
    "csa2_selftest_wait_timeout": (_I32, [_P, _SZ, ctypes.c_uint32, _P]),
}


class Csa2Error(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"libcsa2.so not built ({path}); run __graft_entry__.build() or "
                          "python -m compressed_sparse_attention_fp4_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def _check(name: str, code: int):
    if code != 0:
        raise Csa2Error(name, code)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:                                # (torch.cuda.current_stream() takes 2.9 us of host time, this 0.2)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """A new output of a call on `stream`, from the memory of that stream: a block of the current
    stream's may still be in use by work queued there, and would go back there while `stream` writes it.
    To use the output on a third stream, wait and ``record_stream`` as for any tensor."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


@dataclass
class Dims:
    """Python view of ``csa2_dims`` (see include/csa2.h)."""
    idx_heads: int = 16
    idx_dim: int = 128
    idx_k_dtype: int = IDXK_E4M3
    pool_blocks: int = 2048
    topk: int = 512
    heads: int = 64
    swa: int = 128
    max_pages: int = 0
    num_pages: int = 0
    max_ctx: int = 131072

    def c(self) -> CDims:
        return CDims(self.idx_heads, self.idx_dim, self.idx_k_dtype, self.pool_blocks,
                     self.topk, self.heads, self.swa, self.max_pages, self.num_pages,
                     self.max_ctx)


def version() -> int:
    return _lib.csa2_version()


def workspace_size(dims: Dims, batch: int) -> int:
    out = ctypes.c_size_t(0)
    _check("csa2_workspace_size", _lib.csa2_workspace_size(ctypes.byref(dims.c()), batch, ctypes.byref(out)))
    return out.value


def alloc_workspace(dims: Dims, batch: int, device="cuda") -> torch.Tensor:
    """Zeroed workspace tensor (uint8, 256-byte aligned by the allocator)."""
    return torch.zeros(workspace_size(dims, batch), dtype=torch.uint8, device=device)


def fp4_kv_quantize(x: torch.Tensor, codes: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None, stream=None):
    """bf16 [n, 512] -> (codes uint8 [n, 256], scales uint8 [n, 32])."""
    n = x.shape[0]
    if codes is None:
        codes = _new((n, LATENT // 2), torch.uint8, x.device, stream)
    if scales is None:
        scales = _new((n, LATENT // 16), torch.uint8, x.device, stream)
    _check("fp4_kv_quantize", _lib.fp4_kv_quantize(_ptr(x), n, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def fp4_kv_quantize_scatter(x: torch.Tensor, dst_rows: torch.Tensor, codes: torch.Tensor,
                            scales: torch.Tensor, stream=None, flags: int = 0):
    """Quantize row i of x into cache row dst_rows[i] (int64).  flags:
    KV_EARLY_INPUTS (see fp4_kv_quantize_scatter_ex in include/csa2.h) or 0."""
    if flags:
        _check("fp4_kv_quantize_scatter_ex",
               _lib.fp4_kv_quantize_scatter_ex(_ptr(x), x.shape[0], _ptr(dst_rows), _ptr(codes),
                                               _ptr(scales), int(flags), _stream(stream)))
        return
    _check("fp4_kv_quantize_scatter",
           _lib.fp4_kv_quantize_scatter(_ptr(x), x.shape[0], _ptr(dst_rows), _ptr(codes),
                                        _ptr(scales), _stream(stream)))


def fp4_idx_k_quantize_scatter(x: torch.Tensor, idx_k: torch.Tensor, cache_rows: int,
                               dst_rows: torch.Tensor | None = None, stream=None):
    """bf16 [n, 128] indexer keys into the two-plane FP4 indexer-K buffer
    ``idx_k`` (uint8, cache_rows * 72 bytes: codes [rows][64], then scales
    [rows][8]); row i goes to dst_rows[i] (int64) or to row i."""
    _check("fp4_idx_k_quantize_scatter",
           _lib.fp4_idx_k_quantize_scatter(_ptr(x), x.shape[0], _ptr(dst_rows), _ptr(idx_k), int(cache_rows),
                                           _stream(stream)))


def fp4_idx_k_planes(idx_k: torch.Tensor, cache_rows: int):
    """Views (codes [rows, 64], scales [rows, 8]) of a two-plane FP4 indexer-K buffer."""
    flat = idx_k if idx_k.dim() == 1 and idx_k.is_contiguous() else idx_k.reshape(-1)
    _need("fp4_idx_k_planes", 0 <= cache_rows * 72 <= flat.numel())
    at, step = flat.storage_offset(), flat.stride(0)
    return (flat.as_strided((cache_rows, 64), (64 * step, step), at),
            flat.as_strided((cache_rows, 8), (8 * step, step), at + cache_rows * 64 * step))


def fp4_kv_dequantize(codes: torch.Tensor, scales: torch.Tensor, y: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """(codes, scales) -> bf16 [n, 512]."""
    n = codes.shape[0]
    if y is None:
        y = _new((n, LATENT), torch.bfloat16, codes.device, stream)
    _check("fp4_kv_dequantize", _lib.fp4_kv_dequantize(_ptr(codes), _ptr(scales), n, _ptr(y), _stream(stream)))
    return y


def indexer_full_topk(dims: Dims, batch: int, idx_k, page_table, ctx_len, idx_q, w,
                      pool_out, pool_len_out, topk_out, ws, stream=None, flags: int = 0):
    """flags: IDX_EARLY_INPUTS (see indexer_full_topk_ex in include/csa2.h) or 0."""
    if flags:
        _check("indexer_full_topk_ex", _lib.indexer_full_topk_ex(
            ctypes.byref(dims.c()), batch, int(flags), _ptr(idx_k), _ptr(page_table), _ptr(ctx_len),
            _ptr(idx_q), _ptr(w), _ptr(pool_out), _ptr(pool_len_out), _ptr(topk_out), _ptr(ws), ws.numel(),
            _stream(stream)))
        return
    _check("indexer_full_topk", _lib.indexer_full_topk(
        ctypes.byref(dims.c()), batch, _ptr(idx_k), _ptr(page_table), _ptr(ctx_len), _ptr(idx_q),
        _ptr(w), _ptr(pool_out), _ptr(pool_len_out), _ptr(topk_out), _ptr(ws), ws.numel(),
        _stream(stream)))


def indexer_reindex_topk(dims: Dims, batch: int, idx_k, page_table, ctx_len, idx_q, w,
                         pool_blocks, pool_len, topk_out, ws, stream=None, flags: int = 0):
    """flags: IDX_EARLY_INPUTS (see indexer_reindex_topk_ex in include/csa2.h) or 0."""
    if flags:
        _check("indexer_reindex_topk_ex", _lib.indexer_reindex_topk_ex(
            ctypes.byref(dims.c()), batch, int(flags), _ptr(idx_k), _ptr(page_table), _ptr(ctx_len),
            _ptr(idx_q), _ptr(w), _ptr(pool_blocks), _ptr(pool_len), _ptr(topk_out), _ptr(ws), ws.numel(),
            _stream(stream)))
        return
    _check("indexer_reindex_topk", _lib.indexer_reindex_topk(
        ctypes.byref(dims.c()), batch, _ptr(idx_k), _ptr(page_table), _ptr(ctx_len), _ptr(idx_q),
        _ptr(w), _ptr(pool_blocks), _ptr(pool_len), _ptr(topk_out), _ptr(ws), ws.numel(),
        _stream(stream)))


def csa2_sparse_attn_decode(dims: Dims, batch: int, mode: int, q, kv_codes, kv_scales, kv_rope,
                            page_table, ctx_len, topk, swa_kv, swa_len, scale: float, out, lse,
                            ws, stream=None):
    _check("csa2_sparse_attn_decode", _lib.csa2_sparse_attn_decode(
        ctypes.byref(dims.c()), batch, mode, _ptr(q), _ptr(kv_codes), _ptr(kv_scales),
        _ptr(kv_rope), _ptr(page_table), _ptr(ctx_len), _ptr(topk), _ptr(swa_kv), _ptr(swa_len),
        float(scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def csa2_sparse_attn_decode_mq(dims: Dims, batch: int, q_len: int, mode: int, q, kv_codes, kv_scales,
                               kv_rope, page_table, ctx_len, topk, swa_kv, swa_len, scale: float, out, lse,
                               ws, stream=None):
    """Multi-query decode attention: q bf16 [B, q_len, H, 576] (the newest
    q_len tokens, oldest first), out fp32 [B, q_len, H, 512], lse [B, q_len, H]."""
    _check("csa2_sparse_attn_decode_mq", _lib.csa2_sparse_attn_decode_mq(
        ctypes.byref(dims.c()), batch, int(q_len), mode, _ptr(q), _ptr(kv_codes), _ptr(kv_scales),
        _ptr(kv_rope), _ptr(page_table), _ptr(ctx_len), _ptr(topk), _ptr(swa_kv), _ptr(swa_len),
        float(scale), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))


def csa2_sparse_attn_decode_noalloc(dims: Dims, batch: int, mode: int, q, kv_codes, kv_scales,
                                    kv_rope, page_table, ctx_len, topk, swa_kv, swa_len,
                                    scale: float, out, lse, err_word=None, stream=None):
    """Decode attention without a workspace: for callers that cannot allocate.

    The split-KV scratch is a fixed array inside the library (12 MiB per GPU,
    kept until exit); calls that overlap on the GPU race on it.  err_word is
    an optional device int32 tensor that receives the call's device error bits.
    """
    _check("csa2_sparse_attn_decode_noalloc", _lib.csa2_sparse_attn_decode_noalloc(
        ctypes.byref(dims.c()), batch, mode, _ptr(q), _ptr(kv_codes), _ptr(kv_scales),
        _ptr(kv_rope), _ptr(page_table), _ptr(ctx_len), _ptr(topk), _ptr(swa_kv), _ptr(swa_len),
        float(scale), _ptr(out), _ptr(lse), _ptr(err_word), _stream(stream)))


@dataclass(frozen=True)
class Rope:
    """Python view of ``csa2_rope``: a rotary configuration (see include/csa2.h)."""
    rot: int = ROPE
    theta: float = 10000.0
    layout: int = ROPE_INTERLEAVED
    scaling: int = ROPE_PLAIN
    factor: float = 1.0
    orig_ctx: float = 0.0
    turns_lo: float = 1.0
    turns_hi: float = 32.0
    mscale: float = 1.0

    def __post_init__(self):
        # whole numbers that ctypes would cut to 32 bits; what they mean is checked by the calls
        _need("csa2_rope", all(-1 << 31 <= v < 1 << 31 for v in (self.rot, self.layout, self.scaling)))
        object.__setattr__(self, "_c", CRope(self.rot, self.layout, self.scaling, self.mscale, self.theta, self.factor,
                                             self.orig_ctx, self.turns_lo, self.turns_hi))
        object.__setattr__(self, "_ref", ctypes.byref(self._c))

    def __reduce__(self):
        # copies and pickles carry the fields; a reference to a C structure cannot be copied
        return Rope, tuple(getattr(self, f.name) for f in fields(self))

    def ref(self):
        """The C structure, by reference."""
        return self._ref


def _need(fn: str, ok: bool):
    """A tensor that the C call cannot check (type, shape, stride, device): the same error as its own checks."""
    if not ok:
        raise Csa2Error(fn, 1)


def _plane(t, dtype, n, dev) -> bool:
    """A contiguous tensor of n elements of dtype on CUDA device number dev (-1: the host)."""
    return t.dtype is dtype and t.numel() == n and t.is_contiguous() and t.get_device() == dev


def _call(fn: str, dev: int, stream, args):
    """Calls the library on CUDA device number dev (made current for the call: a library call
    launches on the current device) and on its current stream, or on `stream`."""
    f = getattr(_lib, fn)
    if dev < 0:
        _need(fn, False)
    if stream is None and dev == torch._C._cuda_getDevice():
        _check(fn, f(*args, torch._C._cuda_getCurrentRawStream(dev)))
        return
    with torch.cuda.device(dev):
        _check(fn, f(*args, _stream(stream)))


def csa2_rope_apply(cfg: Rope, x: torch.Tensor, pos: torch.Tensor, y: torch.Tensor | None = None, offset: int = 0,
                    inverse: bool = False, stream=None) -> torch.Tensor:
    """Rotary positions on channels [offset, offset + cfg.rot) of x [tokens, heads, dim]
    (bf16 or fp32, any strides but the last axis's 1) into y (None: a new tensor, of the
    memory of `stream`; y=x: in place).  pos: int32 [tokens].  inverse=True is the gradient's turn."""
    fn = "csa2_rope_apply"
    dt, dev = x.dtype, x.get_device()
    if y is None:
        y = _new(x.shape, dt, x.device, stream)
    _need(fn, x.dim() == 3 and (dt is torch.bfloat16 or dt is torch.float32))
    tokens, heads, dim = x.shape
    xt, xh, xc = x.stride()
    if y is x:
        yt, yh = xt, xh
    else:
        _need(fn, y.shape == x.shape and y.dtype is dt and y.get_device() == dev)
        yt, yh, yc = y.stride()
        _need(fn, yc == 1 or dim <= 1)
    _need(fn, (xc == 1 or dim <= 1) and 0 <= offset <= dim and _plane(pos, torch.int32, tokens, dev))
    _call(fn, dev, stream, (cfg.ref(), 1 if dt is torch.float32 else 0, x.data_ptr(), y.data_ptr(), pos.data_ptr(),
                            tokens, heads, dim, offset, xt, xh, yt, yh, 1 if inverse else 0))
    return y


def csa2_kv_append(cfg: Rope, x: torch.Tensor, pos: torch.Tensor, dst_rows: torch.Tensor, codes: torch.Tensor,
                   scales: torch.Tensor, rope: torch.Tensor, norm_w: torch.Tensor | None = None, eps: float = 1e-6,
                   entry: torch.Tensor | None = None, stream=None):
    """Norm, rotate, quantize and write row i of x (bf16 [n, 576], rows strided) to cache
    row dst_rows[i] (int64; outside the cache: no cache row) of the planes codes
    [rows, 256], scales [rows, 32], rope [rows, 64]; entry (bf16 [n, 576]) also
    receives the row in bf16."""
    fn = "csa2_kv_append"
    _need(fn, x.dim() == 2 and x.shape[1] == DQK and x.dtype is torch.bfloat16 and x.stride(1) == 1)
    n, dev, rows = x.shape[0], x.get_device(), codes.numel() // (LATENT // 2)
    _need(fn, _plane(pos, torch.int32, n, dev) and _plane(dst_rows, torch.int64, n, dev)
          and _plane(codes, torch.uint8, rows * (LATENT // 2), dev) and _plane(scales, torch.uint8, rows * (LATENT // 16), dev)
          and _plane(rope, torch.bfloat16, rows * ROPE, dev)
          and (norm_w is None or _plane(norm_w, torch.bfloat16, LATENT, dev))
          and (entry is None or _plane(entry, torch.bfloat16, n * DQK, dev)))
    _call(fn, dev, stream, (cfg.ref(), x.data_ptr(), n, x.stride(0), _ptr(norm_w), eps, pos.data_ptr(), dst_rows.data_ptr(),
                            codes.data_ptr(), scales.data_ptr(), rope.data_ptr(), rows, _ptr(entry)))


def dense_attn_workspace_size(dims: Dims, batch: int, total_q: int) -> int:
    out = ctypes.c_size_t(0)
    _need("csa2_dense_attn_workspace_size", -1 << 31 <= batch < 1 << 31)
    _check("csa2_dense_attn_workspace_size",
           _lib.csa2_dense_attn_workspace_size(ctypes.byref(dims.c()), batch, total_q, ctypes.byref(out)))
    return out.value


def alloc_dense_attn_workspace(dims: Dims, batch: int, total_q: int, device="cuda") -> torch.Tensor:
    """Workspace of csa2_dense_attn_chunk (uint8; its error word zeroed)."""
    ws = torch.empty(dense_attn_workspace_size(dims, batch, total_q), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def csa2_dense_attn_chunk(dims: Dims, batch: int, q, q_start, kv_codes, kv_scales, kv_rope, page_table, ctx_len,
                          scale: float, out, lse, ws, window: int = 0, flags: int = 0, stream=None):
    """Dense attention of packed query tokens q bf16 [total_q, H, 576] over every visible
    cache position: out bf16 [total_q, H, 512], lse fp32 [total_q, H].  flags:
    DENSE_ALL_POSITIONS (no causal mask) or 0; window > 0: the last `window` positions."""
    fn = "csa2_dense_attn_chunk"
    total, h, dev = q.shape[0], dims.heads, q.get_device()
    rows = batch * dims.max_ctx if page_table is None else dims.num_pages * PAGE
    _need(fn, _plane(q, torch.bfloat16, total * h * DQK, dev) and _plane(out, torch.bfloat16, total * h * LATENT, dev)
          and _plane(lse, torch.float32, total * h, dev) and _plane(q_start, torch.int32, batch + 1, dev)
          and _plane(ctx_len, torch.int32, batch, dev)
          and (page_table is None or _plane(page_table, torch.int32, batch * dims.max_pages, dev)))
    for t, dt, width in ((kv_codes, torch.uint8, LATENT // 2), (kv_scales, torch.uint8, LATENT // 16),
                         (kv_rope, torch.bfloat16, ROPE)):
        _need(fn, t.dtype is dt and t.numel() >= rows * width and t.is_contiguous() and t.get_device() == dev)
    # whole numbers that ctypes would cut to 32 bits
    _need(fn, ws.dtype is torch.uint8 and ws.is_contiguous() and ws.get_device() == dev and 0 <= window < 1 << 31
          and 0 <= flags < 1 << 31)
    _call(fn, dev, stream, (ctypes.byref(dims.c()), batch, total, q.data_ptr(), q_start.data_ptr(), kv_codes.data_ptr(),
                            kv_scales.data_ptr(), kv_rope.data_ptr(), _ptr(page_table), ctx_len.data_ptr(), scale, window,
                            flags, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel()))


def csa2_window_append(cfg: Rope, x: torch.Tensor, pos: torch.Tensor, dst_rows: torch.Tensor, kv: torch.Tensor,
                       norm_w: torch.Tensor | None = None, eps: float = 1e-6, stream=None):
    """Norm, rotate and write row i of x (bf16 [n, 576], rows strided) in bf16 to row
    dst_rows[i] (int64; outside the cache: skipped) of the window cache kv [rows, 576]."""
    fn = "csa2_window_append"
    _need(fn, x.dim() == 2 and x.shape[1] == DQK and x.dtype is torch.bfloat16 and x.stride(1) == 1)
    n, dev, rows = x.shape[0], x.get_device(), kv.numel() // DQK
    _need(fn, _plane(pos, torch.int32, n, dev) and _plane(dst_rows, torch.int64, n, dev)
          and _plane(kv, torch.bfloat16, rows * DQK, dev)
          and (norm_w is None or _plane(norm_w, torch.bfloat16, LATENT, dev)))
    _call(fn, dev, stream, (cfg.ref(), x.data_ptr(), n, x.stride(0), _ptr(norm_w), eps, pos.data_ptr(), dst_rows.data_ptr(),
                            kv.data_ptr(), rows))


# an indexer key: type and channels of its row before the append, bytes of it in the cache
_KEY_ROW = {IDXK_E4M3: (torch.bfloat16, 128, 128), IDXK_F32: (torch.float32, 64, 256), IDXK_FP4: (torch.bfloat16, 128, 72)}


def csa2_idx_k_append(cfg: Rope | None, kind: int, x: torch.Tensor, pos: torch.Tensor | None, dst_rows: torch.Tensor,
                      idx_k: torch.Tensor, cache_rows: int, offset: int = 0, norm: int = IDX_NORM_NONE,
                      norm_w: torch.Tensor | None = None, norm_b: torch.Tensor | None = None, eps: float = 1e-6, stream=None):
    """Norm, rotate (cfg on channels [offset, offset + cfg.rot); None: not) and write row i
    of x (bf16 [n, 128], fp32 [n, 64] for IDXK_F32; rows strided) to row dst_rows[i] (int64;
    outside the cache: skipped) of the indexer keys idx_k of `kind` (IDXK_E4M3, IDXK_FP4,
    IDXK_F32; cache_rows rows).  norm: IDX_NORM_*, norm_w and norm_b of x's type."""
    fn = "csa2_idx_k_append"
    _need(fn, kind in _KEY_ROW)
    dt, dim, size = _KEY_ROW[kind]
    n, dev = x.numel() // dim, x.get_device()
    strides = x.stride()
    # (whole numbers that ctypes would cut to 32 bits, too)
    _need(fn, x.dtype is dt and len(strides) == 2 and x.shape[1] == dim and strides[1] == 1 and 0 <= offset < 1 << 31
          and 0 <= norm < 1 << 31 and _plane(dst_rows, torch.int64, n, dev) and (pos is None or _plane(pos, torch.int32, n, dev))
          and (norm_w is None or _plane(norm_w, dt, dim, dev)) and (norm_b is None or _plane(norm_b, dt, dim, dev))
          and idx_k.numel() * idx_k.element_size() == cache_rows * size and idx_k.is_contiguous() and idx_k.get_device() == dev)
    _call(fn, dev, stream, (None if cfg is None else cfg.ref(), kind, x.data_ptr(), n, strides[0], offset, norm, _ptr(norm_w),
                            _ptr(norm_b), eps, _ptr(pos), dst_rows.data_ptr(), idx_k.data_ptr(), cache_rows))


def window_attn_workspace_size(dims: Dims, batch: int, total_q: int) -> int:
    out = ctypes.c_size_t(0)
    _need("csa2_window_attn_workspace_size", -1 << 31 <= batch < 1 << 31)
    _check("csa2_window_attn_workspace_size",
           _lib.csa2_window_attn_workspace_size(ctypes.byref(dims.c()), batch, total_q, ctypes.byref(out)))
    return out.value


def alloc_window_attn_workspace(dims: Dims, batch: int, total_q: int, device="cuda") -> torch.Tensor:
    """Workspace of csa2_window_attn_chunk (uint8; its error word zeroed)."""
    ws = torch.empty(window_attn_workspace_size(dims, batch, total_q), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def csa2_window_attn_chunk(dims: Dims, batch: int, q, q_start, kv, page_table, ctx_len, scale: float, window: int, out, lse,
                           ws, sinks: int = 0, prev_out=None, prev_lse=None, stream=None):
    """Attention of packed query tokens q bf16 [total_q, H, 576] over exact rows kv bf16
    [rows, 576]: the last `window` positions of each and the first `sinks`; joined in one softmax
    with prev_out / prev_lse (another attention's results for these queries; may be out / lse).
    out bf16 [total_q, H, 512], lse fp32 [total_q, H]."""
    fn = "csa2_window_attn_chunk"
    total, h, dev = q.shape[0], dims.heads, q.get_device()
    rows = batch * dims.max_ctx if page_table is None else dims.num_pages * PAGE
    _need(fn, _plane(q, torch.bfloat16, total * h * DQK, dev) and _plane(out, torch.bfloat16, total * h * LATENT, dev)
          and _plane(lse, torch.float32, total * h, dev) and _plane(q_start, torch.int32, batch + 1, dev)
          and _plane(ctx_len, torch.int32, batch, dev)
          and (page_table is None or _plane(page_table, torch.int32, batch * dims.max_pages, dev))
          and (prev_out is None or _plane(prev_out, torch.bfloat16, total * h * LATENT, dev))
          and (prev_lse is None or _plane(prev_lse, torch.float32, total * h, dev))
          and kv.dtype is torch.bfloat16 and kv.numel() >= rows * DQK and kv.is_contiguous() and kv.get_device() == dev)
    # whole numbers that ctypes would cut to 32 bits
    _need(fn, ws.dtype is torch.uint8 and ws.is_contiguous() and ws.get_device() == dev and 0 <= window < 1 << 31
          and 0 <= sinks < 1 << 31 and -1 << 31 <= batch < 1 << 31)
    _call(fn, dev, stream, (ctypes.byref(dims.c()), batch, total, q.data_ptr(), q_start.data_ptr(), kv.data_ptr(),
                            _ptr(page_table), ctx_len.data_ptr(), scale, window, sinks, _ptr(prev_out), _ptr(prev_lse),
                            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel()))


def get_device_status(ws: torch.Tensor, stream=None) -> int:
    """The workspace's device error word (synchronises the stream)."""
    word = ctypes.c_int32(0)
    code = _lib.csa2_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(word))
    if code not in (0, 5, 6):
        raise Csa2Error("csa2_get_device_status", code)
    return word.value


def profile_enable(on: bool = True):
    """Bracket every library kernel launch with CUDA events (not during capture)."""
    _check("csa2_profile_enable", _lib.csa2_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{kernel name: (launches, total ms)} of the launches recorded so far."""
    arr = (CKernelTime * 64)()
    n = ctypes.c_int32(0)
    _check("csa2_profile_read", _lib.csa2_profile_read(arr, 64, ctypes.byref(n)))
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(min(n.value, 64))}


def clear_device_status(ws: torch.Tensor, stream=None):
    _check("csa2_clear_device_status", _lib.csa2_clear_device_status(_ptr(ws), _stream(stream)))


def selftest_wait_timeout(ws: torch.Tensor, limit_us: int = 2000, stream=None):
    """Runs the device timeout path on purpose: a bounded wait on an mbarrier
    nothing arrives at gives up after limit_us and sets CSA2_DEV_TIMEOUT in
    the error word of ws (read it with get_device_status)."""
    _check("csa2_selftest_wait_timeout",
           _lib.csa2_selftest_wait_timeout(_ptr(ws), ws.numel(), int(limit_us), _stream(stream)))
