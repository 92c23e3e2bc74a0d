// newrows.cu -- what a layer's new tokens leave for the tokens after them, beside the FP4 rows:
// exact bf16 rows (the SWA window's form) and indexer keys, normed, rotated and written to their
// cache rows in one pass.
//
// Both kernels are bound by memory: a row is read once and written once.
#include <cmath>

#include "fp4.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rope.cuh"
#include "rows.cuh"

namespace csa2 {

namespace {

// ---------------------------------------------------------------------------
// Exact rows: one warp a row, in the layout of the FP4 append (rows.cuh): latent =
// bf16(x w / sqrt(mean x^2 + eps)) rounded once, rope = bf16(rotary(x)).
// ---------------------------------------------------------------------------
constexpr int kWinAppThreads = 256;
constexpr int kWinAppBlocks = 3;                     // resident on an SM

template <bool kHalf, bool kNorm>
__global__ void __launch_bounds__(kWinAppThreads, kWinAppBlocks)
    window_append_kernel(const __grid_constant__ RopeTable tab, const uint16_t* __restrict__ x, int64_t n, int64_t stride,
                         const uint16_t* __restrict__ norm_w, float eps, int least_ex, const int32_t* __restrict__ pos,
                         const int64_t* __restrict__ dst_rows, uint16_t* __restrict__ kv, int64_t cache_rows) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (int64_t(gridDim.x) * blockDim.x) >> 5;
  pdl_wait();
  pdl_launch_dependents();
  float w[2][8];
  if (kNorm) {
#pragma unroll
    for (int r = 0; r < 2; ++r) Io<uint16_t>::unpack(__ldg(reinterpret_cast<const uint4*>(norm_w) + r * 32 + lane), w[r]);
  }
  if (warp >= n) return;
  AppendRow next = append_load<kHalf>(x, stride, pos, dst_rows, warp, lane);
  for (int64_t row = warp; row < n; row += nwarps) {
    uint4 v[2] = {next.v[0], next.v[1]};
    const float u0 = __uint_as_float(next.p << 16), u1 = __uint_as_float(kHalf ? next.p2 << 16 : next.p & 0xFFFF0000u);
    const int32_t ps = next.pos;
    const int64_t dst = next.dst;
    next = append_load<kHalf>(x, stride, pos, dst_rows, min64(row + nwarps, n - 1), lane);
    if (dst < 0 || dst >= cache_rows) continue;       // the same for the whole warp
    if (kNorm) norm_row(v, w, eps, least_ex);
    const float2 cs = rope_cs(tab, lane, ps);
    const float2 uv = turn_pair(u0, u1, cs);
    const uint32_t turned = bf16x2_rn(uv.x, uv.y);
    uint16_t* to = kv + dst * kDqk;
#pragma unroll
    for (int r = 0; r < 2; ++r) reinterpret_cast<uint4*>(to)[r * 32 + lane] = v[r];
    if (kHalf) {
      to[kLatent + lane] = uint16_t(turned);
      to[kLatent + 32 + lane] = uint16_t(turned >> 16);
    } else {
      reinterpret_cast<uint32_t*>(to + kLatent)[lane] = turned;
    }
  }
}

// ---------------------------------------------------------------------------
// Indexer keys: eight lanes a row, four rows a warp.  Lane l of a row holds its 16-byte pieces l
// and l + 8: of 128 bf16 channels (E4M3, FP4 keys) or 64 fp32 channels.
//   y = x, x w / sqrt(mean x^2 + eps), or (x - mu) w / sqrt(mean (x - mu)^2 + eps) + b,
//   then rotary on [offset, offset + rot), then the key's format: E4M3 from fp32, FP4 from bf16
//   (its grid's rounding is exact for bf16 values: fp4.cuh), fp32 as it is.
// All in fp32: the keys' formats are coarse beside its roundings (2^-22 of a row's size), so no
// compensated sums as for the latent rows.
// The angles' (cos, sin) of a row are formed once, spread over the warp, and go through shared
// memory, as do the values that half-split pairs exchange.
// ---------------------------------------------------------------------------
constexpr int kKeyThreads = 256;
constexpr int kKeyBlocks = 3;                        // resident on an SM
constexpr int kKeyPairs = 64;                        // most pairs of a key

struct KeyRow {
  uint4 v[2];
  int32_t pos;
  int64_t dst;
};
template <typename T>
__device__ inline KeyRow key_load(const T* x, int64_t stride, const int32_t* pos, const int64_t* dst, int64_t row, int64_t n,
                                  int l) {
  KeyRow k;
  const int64_t at = min64(row, n - 1);
  const uint4* xr = reinterpret_cast<const uint4*>(x + at * stride);
  k.v[0] = __ldcs(xr + l);
  k.v[1] = __ldcs(xr + l + 8);
  k.pos = pos ? __ldg(pos + at) : 0;
  k.dst = row < n ? __ldg(dst + at) : -1;
  return k;
}

__device__ inline float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <typename T> struct Piece;
template <> struct Piece<uint16_t> {
  static constexpr int kC = 8;
  __device__ static void get(uint4 v, float* f) {
    float t[8];
    Io<uint16_t>::unpack(v, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = t[i];
  }
};
template <> struct Piece<float> {
  static constexpr int kC = 4;
  __device__ static void get(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};

__device__ inline uint32_t e4m3x4_rn(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// vec: every piece is rotated as a whole or not at all, and so is its partner.
template <int kKind, bool kHalf>
__global__ void __launch_bounds__(kKeyThreads, kKeyBlocks)
    idx_append_kernel(const __grid_constant__ RopeTable tab, const void* __restrict__ xv, int64_t n, int64_t stride, int norm,
                      const void* __restrict__ wv, const void* __restrict__ bv, float eps, int offset, int vec,
                      const int32_t* __restrict__ pos, const int64_t* __restrict__ dst_rows, uint8_t* __restrict__ keys,
                      uint8_t* __restrict__ scales, int64_t cache_rows) {
  using T = std::conditional_t<kKind == CSA2_IDXK_F32, float, uint16_t>;
  constexpr int C = Piece<T>::kC, D = 16 * C;
  __shared__ __align__(16) float2 s_cs[kKeyThreads / 32][4][kKeyPairs];
  __shared__ __align__(16) float s_y[kKeyThreads / 32][4][D];
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3, wid = threadIdx.x >> 5;
  const int64_t warp = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (int64_t(gridDim.x) * blockDim.x) >> 5;
  const T* x = static_cast<const T*>(xv);
  const int pairs = tab.pairs, rot = 2 * pairs;
  pdl_wait();
  pdl_launch_dependents();
  if (4 * warp >= n) return;
  KeyRow next = key_load(x, stride, pos, dst_rows, 4 * warp + sub, n, l);
  float w[2 * C], b[2 * C];
#pragma unroll
  for (int i = 0; i < 2 * C; ++i) {
    w[i] = 1.0f;
    b[i] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (norm != CSA2_IDX_NORM_NONE) Piece<T>::get(__ldg(static_cast<const uint4*>(wv) + l + 8 * j), w + j * C);
    if (bv) Piece<T>::get(__ldg(static_cast<const uint4*>(bv) + l + 8 * j), b + j * C);
  }
  uint64_t turn[2];                                  // the lane's pairs
#pragma unroll
  for (int k = 0; k < 2; ++k) turn[k] = lane + 32 * k < pairs ? tab.turn[lane + 32 * k] : 0;
  for (int64_t g = warp; 4 * g < n; g += nwarps) {
    const KeyRow now = next;
    next = key_load(x, stride, pos, dst_rows, 4 * (g + nwarps) + sub, n, l);
    float y[2 * C];
#pragma unroll
    for (int j = 0; j < 2; ++j) Piece<T>::get(now.v[j], y + j * C);
    if (norm != CSA2_IDX_NORM_NONE) {
      float up = 1.0f;
      for (int again = 0;; ++again) {
        float d[2 * C], mean = 0.0f, q = 0.0f;
        if (norm == CSA2_IDX_NORM_LAYER) {
#pragma unroll
          for (int i = 0; i < 2 * C; ++i) mean += y[i] * up;
          mean = row_sum(mean) * (1.0f / D);
        }
#pragma unroll
        for (int i = 0; i < 2 * C; ++i) {
          d[i] = __fmaf_rn(y[i], up, -mean);
          q = __fmaf_rn(d[i], d[i], q);
        }
        q = row_sum(q) * (1.0f / D);
        // squares past fp32 (a row of values above 2^60): once more, scaled down; eps is nothing there
        if (again == 0 && __any_sync(0xFFFFFFFFu, !(q < 1.0e37f))) {
          up = q < 1.0e37f ? 1.0f : 1.2621774483536189e-29f;     // 2^-96
          continue;
        }
        const float r = rsqrtf(q + eps * up * up);
#pragma unroll
        for (int i = 0; i < 2 * C; ++i) y[i] = __fmaf_rn(d[i] * r, w[i], b[i]);
        break;
      }
    }
    if (pairs > 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int32_t ps = __shfl_sync(0xFFFFFFFFu, now.pos, 8 * r);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (lane + 32 * k < pairs) s_cs[wid][r][lane + 32 * k] = rope_cs(turn[k], tab.mscale, ps);
      }
      float* ys = s_y[wid][sub];
      const float2* cs = s_cs[wid][sub];
      if (vec) {
        if (kHalf) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < C; i += 4)
              *reinterpret_cast<float4*>(ys + C * (l + 8 * j) + i) = make_float4(y[j * C + i], y[j * C + i + 1], y[j * C + i + 2], y[j * C + i + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = C * (l + 8 * j) - offset;    // channel in the rotated part
          if (c >= 0 && c < rot) {
            if (kHalf) {
              const bool v = c >= pairs;
              const int p = v ? c - pairs : c;
              const float* other = ys + offset + (v ? p : p + pairs);
#pragma unroll
              for (int i = 0; i < C; ++i) {
                const float a = y[j * C + i], o = other[i];
                const float2 t = turn_pair(v ? o : a, v ? a : o, cs[p + i]);
                y[j * C + i] = v ? t.y : t.x;
              }
            } else {
#pragma unroll
              for (int i = 0; i < C; i += 2) {
                const float2 t = turn_pair(y[j * C + i], y[j * C + i + 1], cs[(c + i) / 2]);
                y[j * C + i] = t.x;
                y[j * C + i + 1] = t.y;
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < C; ++i) ys[C * (l + 8 * j) + i] = y[j * C + i];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < C; ++i) {
            const int c = C * (l + 8 * j) + i - offset;
            if (c < 0 || c >= rot) continue;
            const bool v = kHalf ? c >= pairs : c & 1;
            const int p = kHalf ? (v ? c - pairs : c) : c >> 1;
            const float2 t = turn_pair(ys[offset + (kHalf ? p : 2 * p)], ys[offset + (kHalf ? p + pairs : 2 * p + 1)], cs[p]);
            y[j * C + i] = v ? t.y : t.x;
          }
      }
      __syncwarp();
    }
    const bool keep = now.dst >= 0 && now.dst < cache_rows;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = l + 8 * j;
      const float* f = y + j * C;
      if constexpr (kKind == CSA2_IDXK_E4M3) {
        if (keep)
          *reinterpret_cast<uint2*>(keys + now.dst * D + 8 * k) =
              make_uint2(e4m3x4_rn(f[0], f[1], f[2], f[3]), e4m3x4_rn(f[4], f[5], f[6], f[7]));
      } else if constexpr (kKind == CSA2_IDXK_F32) {
        if (keep) *reinterpret_cast<float4*>(keys + now.dst * (4 * D) + 16 * k) = make_float4(f[0], f[1], f[2], f[3]);
      } else {
        uint32_t sc;                                 // all lanes take part
        const uint32_t packed = fp4_quantize_half_group(
            make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]), bf16x2_rn(f[6], f[7])), &sc);
        if (keep) {
          *reinterpret_cast<uint32_t*>(keys + now.dst * (D / 2) + 4 * k) = packed;
          if ((k & 1) == 0) scales[now.dst * (D / 16) + (k >> 1)] = uint8_t(sc);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_window_append(const WindowAppendArgs& a, cudaStream_t st) {
  const RopeTable tab = rope_table(a.cfg);
  // one row a warp up to what is resident at once, then rows in turn
  const int64_t want = (a.n + 7) / 8, cap = int64_t(device_sms()) * kWinAppBlocks;
  const bool half = a.cfg.layout == CSA2_ROPE_HALF;
  auto kernel = a.norm_w ? (half ? window_append_kernel<true, true> : window_append_kernel<false, true>)
                         : (half ? window_append_kernel<true, false> : window_append_kernel<false, false>);
  cudaError_t e;
  CSA2_PROFILED(st, "window_append",
                (e = launch_pdl(kernel, dim3(unsigned(min64(want, cap))), dim3(kWinAppThreads), 0, st, 1, tab, a.x, a.n,
                                a.x_stride, a.norm_w, a.eps, a.norm_w ? norm_least_exponent(a.eps) : 0, a.pos, a.dst_rows,
                                a.kv, a.cache_rows)));
  return e;
}

cudaError_t launch_idx_append(const IdxAppendArgs& a, cudaStream_t st) {
  RopeTable tab = {};
  if (a.rotate) tab = rope_table(a.cfg);
  const bool half = a.rotate && a.cfg.layout == CSA2_ROPE_HALF;
  const int c = a.kind == CSA2_IDXK_F32 ? 4 : 8, rot = a.rotate ? a.cfg.rot : 0;
  const int vec = a.offset % c == 0 && (half ? rot / 2 : rot) % c == 0;
  const int64_t want = (a.n + 31) / 32, cap = int64_t(device_sms()) * kKeyBlocks;
  uint8_t* keys = static_cast<uint8_t*>(a.idx_k);
  uint8_t* scales = a.kind == CSA2_IDXK_FP4 ? keys + a.cache_rows * 64 : nullptr;
  auto kernel = a.kind == CSA2_IDXK_E4M3  ? (half ? idx_append_kernel<CSA2_IDXK_E4M3, true> : idx_append_kernel<CSA2_IDXK_E4M3, false>)
                : a.kind == CSA2_IDXK_F32 ? (half ? idx_append_kernel<CSA2_IDXK_F32, true> : idx_append_kernel<CSA2_IDXK_F32, false>)
                                          : (half ? idx_append_kernel<CSA2_IDXK_FP4, true> : idx_append_kernel<CSA2_IDXK_FP4, false>);
  cudaError_t e;
  CSA2_PROFILED(st, "idx_append",
                (e = launch_pdl(kernel, dim3(unsigned(min64(want, cap))), dim3(kKeyThreads), 0, st, 1, tab, a.x, a.n,
                                a.x_stride, a.norm, a.norm_w, a.norm_b, a.eps, a.offset, vec, a.pos, a.dst_rows, keys, scales,
                                a.cache_rows)));
  return e;
}

}  // namespace csa2
