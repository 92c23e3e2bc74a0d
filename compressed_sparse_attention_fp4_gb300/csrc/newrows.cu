// newrows.cu -- what a layer's new tokens leave for the tokens after them, beside the FP4 rows:
// exact bf16 rows (the SWA window's form) and indexer keys, normed, rotated and written to their
// cache rows in one pass.
//
// A row is read once and written once; beside that the exact rows cost little, the keys their angles.
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
// Resident on an SM.  131,072 rows: 57.5 us with 3 blocks, 58.3 with 4, 70.8 with 5 (which spills): 5.3 TB/s
// of reads and writes, and one row a warp at a time below a grid's worth of rows (a decode batch: 2.1 us).
constexpr int kWinAppBlocks = 3;

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
//
// What bounds it is instructions and shared memory's cycles, both: 16 values a lane and row, and a third of
// the work for the angles, whose (cos, sin) are formed once a row, spread over the warp, two rows at a time.
// So values are held in pairs, for two fp32 operations an instruction, and the angles' results and the values
// that half-split pairs exchange go through shared memory, laid out so that the eight lanes of a row read 128
// bytes in a row.
//
// A million rows (layer norm, 64 of 128 channels turned, E4M3): 122 us.  It took 206 us with arithmetic on
// single values and angles formed by the lanes that use them, 135 with the weights in shared memory (four
// wavefronts a load, 87 % of its cycles) at 4 blocks of 256 threads.  (With the hardware's sine and cosine, which
// are off by 2^-21 and more whatever they are themselves, 112: E4M3 keys then come out a step off next to a
// rounding border, by many steps where a large channel meets a small sine.)
// ---------------------------------------------------------------------------
constexpr int kKeyThreads = 128;
constexpr int kKeyBlocks = 4;                        // resident on an SM: 128 registers a thread hold the weights, too (5: 135 us)
constexpr int kKeyPairs = 64;                        // most pairs of a key

using f32x2 = uint64_t;                              // low half first
__device__ inline f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ inline float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ inline f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ inline f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

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

// A 16-byte piece as pairs of channels.
template <typename T> struct Piece;
template <> struct Piece<uint16_t> {
  static constexpr int kC = 8;
  __device__ static void get(uint4 v, f32x2* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};
template <> struct Piece<float> {
  static constexpr int kC = 4;
  __device__ static void get(uint4 v, f32x2* f) {
    f[0] = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};

__device__ inline uint32_t e4m3x4_rn(f32x2 a, f32x2 b) {
  const float2 x = unpack2(a), y = unpack2(b);
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ inline uint32_t bf16x2_rn(f32x2 v) {
  const float2 x = unpack2(v);
  return bf16x2_rn(x.x, x.y);
}

// rope_cs (rope.cuh) of two positions: (cos, cos), (sin, sin) times mscale.
__device__ inline void rope_cs2(uint64_t turn, f32x2 mscale, int32_t p0, int32_t p1, float2& c, float2& s) {
  const uint32_t a0 = uint32_t((uint64_t(int64_t(p0)) * turn) >> 32), a1 = uint32_t((uint64_t(int64_t(p1)) * turn) >> 32);
  const uint32_t q0 = (a0 + 0x20000000u) >> 30, q1 = (a1 + 0x20000000u) >> 30;
  const f32x2 unit = pack2(1.4629180792671596e-9f, 1.4629180792671596e-9f);                 // 2 pi / 2^32
  const f32x2 x = mul2(pack2(float(int32_t(a0 - (q0 << 30))), float(int32_t(a1 - (q1 << 30)))), unit), z = mul2(x, x);
  const auto k = [](float v) { return pack2(v, v); };
  const f32x2 si = fma2(mul2(x, z), fma2(z, fma2(z, fma2(z, k(1.0f / 362880), k(-1.0f / 5040)), k(1.0f / 120)), k(-1.0f / 6)), x);
  const f32x2 co = fma2(z, fma2(z, fma2(z, fma2(z, k(1.0f / 40320), k(-1.0f / 720)), k(1.0f / 24)), k(-0.5f)), k(1.0f));
  const float2 u = unpack2(mul2(co, mscale)), v = unpack2(mul2(si, mscale));
  // quarters: (c, s), (-s, c), (-c, -s), (s, -c)
  c.x = __uint_as_float(__float_as_uint(q0 & 1 ? v.x : u.x) ^ ((q0 + 1) << 30 & 0x80000000u));
  c.y = __uint_as_float(__float_as_uint(q1 & 1 ? v.y : u.y) ^ ((q1 + 1) << 30 & 0x80000000u));
  s.x = __uint_as_float(__float_as_uint(q0 & 1 ? u.x : v.x) ^ (q0 << 30 & 0x80000000u));
  s.y = __uint_as_float(__float_as_uint(q1 & 1 ? u.y : v.y) ^ (q1 << 30 & 0x80000000u));
}

// Places (floats) of a row's channel c and pair p in shared memory: where pieces have two quads of
// channels, the first quads of eight pieces stand before their second ones (pairs, 48 apart: the 32
// lanes that store them meet all banks).
template <int C> __device__ inline int y_place(int c) { return C == 8 ? (c >> 6) * 64 + (c >> 2 & 1) * 32 + (c >> 3 & 7) * 4 + (c & 3) : c; }
template <int C, bool kHalf> __device__ inline int cs_place(int p) { return C == 8 && kHalf ? (p >> 2 & 1) * 48 + (p >> 3) * 4 + (p & 3) : p; }
constexpr int kCsRow = 80;

// vec: every piece is rotated as a whole or not at all, and so is its partner.
template <int kKind, bool kHalf, int kNorm>
__global__ void __launch_bounds__(kKeyThreads, kKeyBlocks)
    idx_append_kernel(const __grid_constant__ RopeTable tab, const void* __restrict__ xv, int64_t n, int64_t stride,
                      const void* __restrict__ wv, const void* __restrict__ bv, float eps, int offset, int vec,
                      const int32_t* __restrict__ pos, const int64_t* __restrict__ dst_rows, uint8_t* __restrict__ keys,
                      uint8_t* __restrict__ scales, int64_t cache_rows) {
  using T = std::conditional_t<kKind == CSA2_IDXK_F32, float, uint16_t>;
  constexpr int C = Piece<T>::kC, D = 16 * C, P = C / 2;               // channels and pairs of a piece
  __shared__ __align__(16) float s_c[kKeyThreads / 32][4][kCsRow], s_s[kKeyThreads / 32][2][4][kCsRow];   // (sin: and -sin)
  __shared__ __align__(16) float s_y[kKeyThreads / 32][4][D];
  __shared__ uint64_t s_turn[kKeyPairs];
  const int lane = threadIdx.x & 31, l = lane & 7, sub = lane >> 3, wid = threadIdx.x >> 5;
  const int64_t warp = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t nwarps = (int64_t(gridDim.x) * blockDim.x) >> 5;
  const T* x = static_cast<const T*>(xv);
  const int pairs = tab.pairs, rot = 2 * pairs;
  pdl_wait();
  pdl_launch_dependents();
  uint4 wr[2], br[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (kNorm != CSA2_IDX_NORM_NONE) wr[j] = __ldg(static_cast<const uint4*>(wv) + l + 8 * j);
    if (kNorm == CSA2_IDX_NORM_LAYER) br[j] = bv ? __ldg(static_cast<const uint4*>(bv) + l + 8 * j) : make_uint4(0, 0, 0, 0);
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kKeyPairs) s_turn[threadIdx.x - 64] = tab.turn[threadIdx.x - 64];
  __syncthreads();
  if (4 * warp >= n) return;
  KeyRow next = key_load(x, stride, pos, dst_rows, 4 * warp + sub, n, l);
  const f32x2 mscale = pack2(tab.mscale, tab.mscale);
  for (int64_t g = warp; 4 * g < n; g += nwarps) {
    const KeyRow now = next;
    next = key_load(x, stride, pos, dst_rows, 4 * (g + nwarps) + sub, n, l);
    f32x2 y[2 * P];
#pragma unroll
    for (int j = 0; j < 2; ++j) Piece<T>::get(now.v[j], y + j * P);
    if (kNorm != CSA2_IDX_NORM_NONE) {
      const auto deviations = [&]() {                // y less its mean; the mean of their squares
        if (kNorm == CSA2_IDX_NORM_LAYER) {
          f32x2 m = add2(y[0], y[1]);
#pragma unroll
          for (int i = 2; i < 2 * P; ++i) m = add2(y[i], m);
          const float2 t = unpack2(m);
          const float mean = row_sum(t.x + t.y) * (-1.0f / D);
#pragma unroll
          for (int i = 0; i < 2 * P; ++i) y[i] = add2(y[i], pack2(mean, mean));
        }
        f32x2 q = mul2(y[0], y[0]);
#pragma unroll
        for (int i = 1; i < 2 * P; ++i) q = fma2(y[i], y[i], q);
        const float2 t = unpack2(q);
        return row_sum(t.x + t.y) * (1.0f / D);
      };
      float v = deviations(), e = eps;
      // squares past fp32 (a row of values above 2^60): once more, scaled down; eps is nothing there
      const bool large = !(v < 1.0e37f);
      if (__any_sync(0xFFFFFFFFu, large)) {
        const float up = large ? 1.2621774483536189e-29f : 1.0f;       // 2^-96
#pragma unroll
        for (int j = 0; j < 2; ++j) Piece<T>::get(now.v[j], y + j * P);
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) y[i] = mul2(y[i], pack2(up, up));
        v = deviations();
        e = large ? 0.0f : eps;
      }
      const float r = __frsqrt_rn(v + e);
      const f32x2 rs = pack2(r, r);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f32x2 w[P], b[P];
        Piece<T>::get(wr[j], w);
        if (kNorm == CSA2_IDX_NORM_LAYER) Piece<T>::get(br[j], b);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const f32x2 t = mul2(y[j * P + i], rs);
          y[j * P + i] = kNorm == CSA2_IDX_NORM_LAYER ? fma2(t, w[i], b[i]) : mul2(t, w[i]);
        }
      }
    }
    if (pairs > 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k > 0 && pairs <= 32) break;
        const int i = lane + 32 * k;
        const uint64_t turn = s_turn[i];
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          float2 c, s;
          const int32_t p0 = __shfl_sync(0xFFFFFFFFu, now.pos, 8 * r), p1 = __shfl_sync(0xFFFFFFFFu, now.pos, 8 * r + 8);
          rope_cs2(turn, mscale, p0, p1, c, s);
          if (i < pairs) {
            const int to = cs_place<C, kHalf>(i);
            s_c[wid][r][to] = c.x;
            s_c[wid][r + 1][to] = c.y;
            s_s[wid][0][r][to] = s.x;
            s_s[wid][0][r + 1][to] = s.y;
            if (kHalf) {
              s_s[wid][1][r][to] = -s.x;
              s_s[wid][1][r + 1][to] = -s.y;
            }
          }
        }
      }
      float* ys = s_y[wid][sub];
      const float *cs = s_c[wid][sub], *ss = s_s[wid][0][sub];
      if (vec) {
        if (kHalf) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = C * (l + 8 * j);
            if (c - offset < 0 || c - offset >= rot) continue;
#pragma unroll
            for (int i = 0; i < P; i += 2)
              *reinterpret_cast<ulonglong2*>(ys + y_place<C>(c + 2 * i)) = make_ulonglong2(y[j * P + i], y[j * P + i + 1]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = C * (l + 8 * j) - offset;    // channel in the rotated part
          if (c >= 0 && c < rot) {
            if (kHalf) {
              const bool v = c >= pairs;             // v: (u s + v c); u: (u c + v (-s))
              const int p = v ? c - pairs : c;
              const float* si = v ? ss : s_s[wid][1][sub];
#pragma unroll
              for (int i = 0; i < P; i += 2) {
                const ulonglong2 o2 = *reinterpret_cast<const ulonglong2*>(ys + y_place<C>(offset + (v ? p : p + pairs) + 2 * i));
                const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(cs + cs_place<C, true>(p + 2 * i));
                const ulonglong2 s2 = *reinterpret_cast<const ulonglong2*>(si + cs_place<C, true>(p + 2 * i));
                y[j * P + i] = fma2(y[j * P + i], c2.x, mul2(o2.x, s2.x));
                y[j * P + i + 1] = fma2(y[j * P + i + 1], c2.y, mul2(o2.y, s2.y));
              }
            } else {
#pragma unroll
              for (int i = 0; i < P; ++i) {
                const float2 t = unpack2(y[j * P + i]);
                const float co = cs[c / 2 + i], si = ss[c / 2 + i];
                y[j * P + i] = fma2(y[j * P + i], pack2(co, co), mul2(pack2(t.y, t.x), pack2(-si, si)));
              }
            }
          }
        }
      } else {
        // odd offsets and sizes: all values through shared memory, a pair a lane at a time
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < P; ++i) *reinterpret_cast<f32x2*>(ys + y_place<C>(C * (l + 8 * j) + 2 * i)) = y[j * P + i];
        __syncwarp();
#pragma unroll 1
        for (int p = l; p < pairs; p += 8) {
          float *u = ys + y_place<C>(offset + (kHalf ? p : 2 * p)), *v = ys + y_place<C>(offset + (kHalf ? p + pairs : 2 * p + 1));
          const int at = cs_place<C, kHalf>(p);
          const float2 r = turn_pair(*u, *v, make_float2(cs[at], ss[at]));
          *u = r.x;
          *v = r.y;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < P; ++i) y[j * P + i] = *reinterpret_cast<const f32x2*>(ys + y_place<C>(C * (l + 8 * j) + 2 * i));
      }
      __syncwarp();
    }
    const bool keep = now.dst >= 0 && now.dst < cache_rows;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = l + 8 * j;
      const f32x2* f = y + j * P;
      if constexpr (kKind == CSA2_IDXK_E4M3) {
        if (keep) *reinterpret_cast<uint2*>(keys + now.dst * D + 8 * k) = make_uint2(e4m3x4_rn(f[0], f[1]), e4m3x4_rn(f[2], f[3]));
      } else if constexpr (kKind == CSA2_IDXK_F32) {
        if (keep) *reinterpret_cast<ulonglong2*>(keys + now.dst * (4 * D) + 16 * k) = make_ulonglong2(f[0], f[1]);
      } else {
        uint32_t sc;                                 // all lanes take part
        const uint32_t packed = fp4_quantize_half_group(make_uint4(bf16x2_rn(f[0]), bf16x2_rn(f[1]), bf16x2_rn(f[2]), bf16x2_rn(f[3])), &sc);
        if (keep) {
          *reinterpret_cast<uint32_t*>(keys + now.dst * (D / 2) + 4 * k) = packed;
          if ((k & 1) == 0) scales[now.dst * (D / 16) + (k >> 1)] = uint8_t(sc);
        }
      }
    }
  }
}

using IdxKernel = void (*)(const RopeTable, const void*, int64_t, int64_t, const void*, const void*, float, int, int, const int32_t*,
                           const int64_t*, uint8_t*, uint8_t*, int64_t);
template <int kKind, bool kHalf>
IdxKernel idx_kernel(int norm) {
  return norm == CSA2_IDX_NORM_NONE  ? idx_append_kernel<kKind, kHalf, CSA2_IDX_NORM_NONE>
         : norm == CSA2_IDX_NORM_RMS ? idx_append_kernel<kKind, kHalf, CSA2_IDX_NORM_RMS>
                                     : idx_append_kernel<kKind, kHalf, CSA2_IDX_NORM_LAYER>;
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
  const int64_t want = (a.n + kKeyThreads / 8 - 1) / (kKeyThreads / 8), cap = int64_t(device_sms()) * kKeyBlocks;
  uint8_t* keys = static_cast<uint8_t*>(a.idx_k);
  uint8_t* scales = a.kind == CSA2_IDXK_FP4 ? keys + a.cache_rows * 64 : nullptr;
  const IdxKernel kernel = a.kind == CSA2_IDXK_E4M3  ? (half ? idx_kernel<CSA2_IDXK_E4M3, true>(a.norm) : idx_kernel<CSA2_IDXK_E4M3, false>(a.norm))
                           : a.kind == CSA2_IDXK_F32 ? (half ? idx_kernel<CSA2_IDXK_F32, true>(a.norm) : idx_kernel<CSA2_IDXK_F32, false>(a.norm))
                                                     : (half ? idx_kernel<CSA2_IDXK_FP4, true>(a.norm) : idx_kernel<CSA2_IDXK_FP4, false>(a.norm));
  cudaError_t e;
  CSA2_PROFILED(st, "idx_append",
                (e = launch_pdl(kernel, dim3(unsigned(min64(want, cap))), dim3(kKeyThreads), 0, st, 1, tab, a.x, a.n,
                                a.x_stride, a.norm_w, a.norm_b, a.eps, a.offset, vec, a.pos, a.dst_rows, keys, scales,
                                a.cache_rows)));
  return e;
}

}  // namespace csa2
