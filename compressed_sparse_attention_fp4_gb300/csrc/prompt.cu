// prompt.cu -- C entry points of the prompt-side calls: rotary positions, the
// cache append and dense chunk attention.  As in api.cu, every call validates on
// the host and launches nothing when an argument is wrong.
#include <cmath>
#include <cstdint>

#include "checks.cuh"
#include "dense.cuh"
#include "kernels.cuh"
#include "rope.cuh"

using namespace csa2;

namespace {

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

csa2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

// Rows of a [tokens][heads][dim] output that do not overlap: token-major or head-major.
bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  if (ts < 0 || hs < 0) return false;
  if (tokens <= 1) return heads <= 1 || hs >= dim;
  if (heads <= 1) return ts >= dim;
  return (hs >= dim && ts >= (heads - 1) * hs + dim) || (ts >= dim && hs >= (tokens - 1) * ts + dim);
}

// Last element index of a strided [tokens][heads][dim] block, or -1 where it passes 2^62.
int64_t extent(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  const __int128 e = __int128(tokens - 1) * ts + __int128(heads - 1) * hs + dim;
  return e > (__int128(1) << 59) ? -1 : int64_t(e);
}

csa2_status check_dense_dims(const csa2_dims* d, int32_t batch, int64_t total_q) {
  if (!d || batch < 0 || total_q < 0) return CSA2_ERR_INVALID_ARG;
  if (d->heads < 1 || d->heads > kMaxHeads) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (d->max_ctx < 1 || d->max_ctx > kMaxCtx) return CSA2_ERR_UNSUPPORTED_SHAPE;
  // rows (and positions less a window) are counted in 32 bits with room to spare
  if (batch > (1 << 20) || total_q > (1 << 30) / d->heads) return CSA2_ERR_UNSUPPORTED_SHAPE;
  return CSA2_OK;
}

}  // namespace

extern "C" {

csa2_status csa2_rope_apply(const csa2_rope* r, int32_t dtype, const void* x, void* y, const int32_t* pos,
                            int64_t tokens, int32_t heads, int32_t dim, int32_t offset, int64_t x_token,
                            int64_t x_head, int64_t y_token, int64_t y_head, int32_t inverse, void* stream) {
  csa2_status st = check_rope(r);
  if (st != CSA2_OK) return st;
  if ((dtype != CSA2_ROPE_BF16 && dtype != CSA2_ROPE_F32) || (inverse != 0 && inverse != 1)) return CSA2_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > (int64_t(1) << 31) || heads < 0 || heads > 65535 || dim < 1 || offset < 0 ||
      int64_t(offset) + r->rot > dim)
    return CSA2_ERR_UNSUPPORTED_SHAPE;
  // pieces of one CTA (kRopeTok tokens, all heads) are counted in 32 bits
  if (int64_t(heads) * dim > (int64_t(1) << 27)) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0 || heads == 0) return CSA2_OK;
  const uintptr_t size = dtype == CSA2_ROPE_F32 ? 4 : 2;
  if (!x || !y || !pos || !is_aligned(x, size) || !is_aligned(y, size) || !is_aligned(pos, 4)) return CSA2_ERR_INVALID_ARG;
  if (x_token < 0 || x_head < 0 || !rows_apart(tokens, heads, dim, y_token, y_head)) return CSA2_ERR_INVALID_ARG;
  const int64_t ex = extent(tokens, heads, dim, x_token, x_head), ey = extent(tokens, heads, dim, y_token, y_head);
  if (ex < 0 || ey < 0) return CSA2_ERR_UNSUPPORTED_SHAPE;
  // in place means the same elements in the same places; strides of axes of length 1 say nothing
  if (x == y && ((tokens > 1 && x_token != y_token) || (heads > 1 && x_head != y_head))) return CSA2_ERR_INVALID_ARG;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
  if (x != y && xa < ya + uintptr_t(ey) * size && ya < xa + uintptr_t(ex) * size)
    return CSA2_ERR_INVALID_ARG;
  RopeArgs a = {};
  a.cfg = *r;
  a.fp32 = dtype == CSA2_ROPE_F32;
  a.inverse = inverse != 0;
  a.x = x;
  a.y = y;
  a.pos = pos;
  a.tokens = tokens;
  a.heads = heads;
  a.dim = dim;
  a.offset = offset;
  a.x_token = tokens > 1 ? x_token : 0;
  a.x_head = heads > 1 ? x_head : 0;
  a.y_token = tokens > 1 ? y_token : 0;
  a.y_head = heads > 1 ? y_head : 0;
  return from_cuda(launch_rope(a, as_stream(stream)));
}

csa2_status csa2_kv_append(const csa2_rope* r, const uint16_t* x, int64_t n, int64_t x_stride,
                           const uint16_t* norm_w, float eps, const int32_t* pos, const int64_t* dst_rows,
                           uint8_t* codes, uint8_t* scales, uint16_t* rope, int64_t cache_rows, uint16_t* entry,
                           void* stream) {
  csa2_status st = check_rope(r);
  if (st != CSA2_OK) return st;
  if (r->rot != kRope) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (n < 0 || cache_rows < 0 || (norm_w && !(eps > 0.0f && eps <= 1.0f))) return CSA2_ERR_INVALID_ARG;
  if (n == 0) return CSA2_OK;
  if (!x || !pos || !dst_rows || !codes || !scales || !rope) return CSA2_ERR_INVALID_ARG;
  if (!is_aligned(x, 16) || !is_aligned(codes, 16) || !is_aligned(scales, 2) || !is_aligned(rope, 16) ||
      !is_aligned(pos, 4) || !is_aligned(dst_rows, 8) || (norm_w && !is_aligned(norm_w, 16)) ||
      (entry && !is_aligned(entry, 16)))
    return CSA2_ERR_INVALID_ARG;
  if (n > 1 && (x_stride < kDqk || x_stride % 8 != 0)) return CSA2_ERR_INVALID_ARG;
  if (entry) {
    const __int128 last = __int128(n - 1) * (n > 1 ? x_stride : 0) + kDqk;
    if (last > (__int128(1) << 59) || n > (int64_t(1) << 49)) return CSA2_ERR_UNSUPPORTED_SHAPE;
    const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ea = reinterpret_cast<uintptr_t>(entry);
    if (xa < ea + uintptr_t(n) * kDqk * 2 && ea < xa + uintptr_t(last) * 2) return CSA2_ERR_INVALID_ARG;
  }
  AppendArgs a = {};
  a.cfg = *r;
  a.x = x;
  a.n = n;
  a.x_stride = n > 1 ? x_stride : 0;
  a.norm_w = norm_w;
  a.eps = eps;
  a.pos = pos;
  a.dst_rows = dst_rows;
  a.codes = codes;
  a.scales = scales;
  a.rope = rope;
  a.cache_rows = cache_rows;
  a.entry = entry;
  return from_cuda(launch_append(a, as_stream(stream)));
}

csa2_status csa2_dense_attn_workspace_size(const csa2_dims* d, int32_t batch, int64_t total_q, size_t* bytes) {
  if (!bytes) return CSA2_ERR_INVALID_ARG;
  const csa2_status st = check_dense_dims(d, batch, total_q);
  if (st != CSA2_OK) return st;
  *bytes = size_t(make_dense_layout(*d, batch, total_q).total);
  return CSA2_OK;
}

csa2_status csa2_dense_attn_chunk(const csa2_dims* d, int32_t batch, int64_t total_q, const uint16_t* q,
                                  const int32_t* q_start, const uint8_t* kv_codes, const uint8_t* kv_scales,
                                  const uint16_t* kv_rope, const int32_t* page_table, const int32_t* ctx_len,
                                  float scale, int32_t window, int32_t flags, uint16_t* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream) {
  csa2_status st = check_dense_dims(d, batch, total_q);
  if (st != CSA2_OK) return st;
  if ((flags & ~int32_t(CSA2_DENSE_ALL_POSITIONS)) != 0 || window < 0 || !std::isfinite(scale)) return CSA2_ERR_INVALID_ARG;
  const bool causal = (flags & CSA2_DENSE_ALL_POSITIONS) == 0;
  if (!causal && window > 0) return CSA2_ERR_INVALID_ARG;
  if ((st = check_paging(d, page_table)) != CSA2_OK) return st;
  if (!ws || !is_aligned(ws, 256)) return CSA2_ERR_INVALID_ARG;
  const DenseLayout L = make_dense_layout(*d, batch, total_q);
  if (ws_bytes < size_t(L.total)) return CSA2_ERR_WORKSPACE_TOO_SMALL;
  // the cache is addressed by 32-bit row coordinates
  const __int128 rows = page_table ? __int128(d->num_pages) * kPage : __int128(batch) * d->max_ctx;
  if (rows > INT32_MAX) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (batch == 0 || total_q == 0) return CSA2_OK;
  if (!q || !q_start || !kv_codes || !kv_scales || !kv_rope || !ctx_len || !out || !lse) return CSA2_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(q_start, 4) || !is_aligned(kv_codes, 16) || !is_aligned(kv_scales, 16) ||
      !is_aligned(kv_rope, 16) || !is_aligned(ctx_len, 4) || !is_aligned(out, 16) || !is_aligned(lse, 4))
    return CSA2_ERR_INVALID_ARG;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DenseArgs a = {};
  a.d = *d;
  a.batch = batch;
  a.total_q = int(total_q);
  a.causal = causal ? 1 : 0;
  a.window = int(min64(window, kMaxCtx));          // a longer one is no window at all
  a.q = q;
  a.q_start = q_start;
  a.codes = kv_codes;
  a.scales = kv_scales;
  a.rope = kv_rope;
  a.page_table = page_table;
  a.ctx_len = ctx_len;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.ws = w;
  a.plan.head = reinterpret_cast<int4*>(w + L.head);
  a.plan.runs = reinterpret_cast<int4*>(w + L.runs);
  a.plan.seqs = reinterpret_cast<int4*>(w + L.seqs);
  a.plan.tiles = reinterpret_cast<int4*>(w + L.tiles);
  a.plan.before = reinterpret_cast<int64_t*>(w + L.before);
  a.part_lse = reinterpret_cast<float*>(w + L.part_lse);
  a.part_o = reinterpret_cast<float*>(w + L.part_o);
  return from_cuda(launch_dense(a, as_stream(stream)));
}

}  // extern "C"
