// rope.cu -- rotary positions of query / key heads, and the cache append that
// norms, rotates and quantizes a token's row in one pass.
//
// Both kernels are bound by memory: every value is read once and written once,
// and the arithmetic between is kept under the time of the bytes.
#include <cmath>

#include "fp4.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "rope.cuh"

namespace csa2 {

namespace {

// ---------------------------------------------------------------------------
// Rotary positions: y = m R(angle) x on channels [offset, offset + rot) of every
// head, the other channels copied (or left, in place).
//
// A CTA takes kRopeTok tokens and a range of heads: it asks for its first 16-byte pieces,
// four a thread, forms the (cos, sin) of its tokens in shared memory meanwhile (rot / 2 of
// them a token, against heads * rot values to turn) and then walks the pieces, four in
// flight.  Measured (kernel in a graph): 8,192 tokens x 64 heads x 64 fp32 channels in place,
// 268 MB, 44.0 us (90 % of the copy rate); 4,099 x 16 heads x 128 bf16 channels into another
// buffer, half layout, 34 MB, 7.4 us.  Loads behind the angles: 45.5 and 12; tiles of 8 tokens:
// 43.9 and 8.1; 2: 43.1 and 10.0; three CTAs an SM instead of four: 44.0 and 7.9, five: 44.2
// and 12.3; one piece in flight and two divisions a piece: 68 for the first.  (At four CTAs an
// SM, 64 registers, the half layouts spill 44 (fp32) and 68 bytes a thread.)
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeTok = 4;

template <typename T> struct Io;
template <> struct Io<float> {
  static constexpr int kVec = 4;
  // the values of a word (fp32: one, twice) and back
  __device__ static float2 word(uint32_t w) { return make_float2(__uint_as_float(w), __uint_as_float(w)); }
  __device__ static uint32_t unword(float a, float) { return __float_as_uint(a); }
  __device__ static float get(float v) { return v; }
  __device__ static float put(float v) { return v; }
};
__device__ inline uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <> struct Io<uint16_t> {
  static constexpr int kVec = 8;
  __device__ static void unpack(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static float2 word(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
  __device__ static uint32_t unword(float a, float b) { return bf16x2_rn(a, b); }
  __device__ static uint4 pack(const float (&f)[8]) {
    return make_uint4(bf16x2_rn(f[0], f[1]), bf16x2_rn(f[2], f[3]), bf16x2_rn(f[4], f[5]), bf16x2_rn(f[6], f[7]));
  }
  __device__ static float get(uint16_t v) { return bf16_to_f32(v); }
  __device__ static uint16_t put(float v) { return uint16_t(bf16x2_rn(v, 0.0f)); }
};

// A turned pair, (u c - v s, u s + v c), in the same operations wherever it is formed: a result
// depends neither on strides and alignment nor on the kernel (left to the compiler, the product
// that is rounded first differed between the paths).
__device__ inline float2 turn_pair(float u, float v, float2 cs) {
  return make_float2(__fmaf_rn(u, cs.x, -__fmul_rn(v, cs.y)), __fmaf_rn(v, cs.x, __fmul_rn(u, cs.y)));
}

// x, y and the strides count elements of T; sign is -1 for the inverse.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads, 4)
    rope_kernel(const __grid_constant__ RopeTable tab, const T* x, T* y, const int32_t* __restrict__ pos, int64_t tokens,
                int heads, int dim, int offset, int64_t xt, int64_t xh, int64_t yt, int64_t yh, int heads_per, int copy,
                int vec, float sign) {
  __shared__ float2 cs[kRopeTok * kMaxPairs];
  pdl_wait();
  pdl_launch_dependents();
  const int pairs = tab.pairs, tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kRopeTok;
  const int nt = int(min64(kRopeTok, tokens - t0));
  const int h0 = blockIdx.y * heads_per, nh = min(heads_per, heads - h0);
  // pieces of a head: turned (kHalf: two pieces rot / 2 apart at once), then copied.  A
  // thread keeps to one piece and walks the (token, head) rows, four in flight.
  constexpr int V = Io<T>::kVec;
  const int nturn = kHalf ? pairs / V : 2 * pairs / V, per = nturn + (copy ? (dim - 2 * pairs) / V : 0);
  const int rows = nt * nh;
  const float inv = 1.0f / float(nh);                // rows < 2^20: (r + 1/2) / nh truncates to r / nh
  uint4 u4[4], v4[4];
  int tk[4];
  int64_t yo[4];
  int c, at, r, apart;
  const auto place = [&](int c0) {                   // the thread's piece and first row among those from c0 on
    const int here = min(per - c0, kRopeThreads);
    apart = kRopeThreads / here;
    c = c0 + tid % here;
    r = tid / here < apart ? tid / here : rows;      // threads left over: none
    at = c < nturn ? offset + c * V : (c - nturn) * V;
    if (c >= nturn && at >= offset) at += 2 * pairs;
  };
  const auto load = [&]() {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int rr = min(r + b * apart, rows - 1);
      tk[b] = __float2int_rz((float(rr) + 0.5f) * inv);
      const int h = h0 + rr - tk[b] * nh;
      const T* xs = x + (t0 + tk[b]) * xt + int64_t(h) * xh + at;
      yo[b] = (t0 + tk[b]) * yt + int64_t(h) * yh + at;
      u4[b] = *reinterpret_cast<const uint4*>(xs);
      if (kHalf && c < nturn) v4[b] = *reinterpret_cast<const uint4*>(xs + pairs);
    }
  };
  // the first rows are on their way while the angles are formed
  if (vec) {
    place(0);
    if (r < rows) load();
  }
  for (int i = tid; i < nt * pairs; i += kRopeThreads) {
    const int t = i / pairs, p = i - t * pairs;
    float2 v = rope_cs(tab, p, __ldg(pos + t0 + t));
    v.y *= sign;
    cs[t * kMaxPairs + p] = v;
  }
  __syncthreads();
  if (vec) {
    for (int c0 = 0; c0 < per; c0 += kRopeThreads) {
      if (c0 > 0) {
        place(c0);
        if (r < rows) load();
      }
      const bool turn = c < nturn;
      while (r < rows) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          if (r + b * apart >= rows) break;
          T* ys = y + yo[b];
          if (!turn) {
            *reinterpret_cast<uint4*>(ys) = u4[b];
            continue;
          }
          // word by word: few values are held widened at a time
          const float2* e2 = cs + tk[b] * kMaxPairs + (kHalf ? c * V : c * (V / 2));
          uint32_t uw[4] = {u4[b].x, u4[b].y, u4[b].z, u4[b].w};
          if (kHalf) {
            uint32_t vw[4] = {v4[b].x, v4[b].y, v4[b].z, v4[b].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 u = Io<T>::word(uw[k]), v = Io<T>::word(vw[k]);
              const float2 e = e2[k * (V / 4)], f = V == 8 ? e2[2 * k + 1] : e;
              const float2 a = turn_pair(u.x, v.x, e), b = turn_pair(u.y, v.y, f);
              uw[k] = Io<T>::unword(a.x, b.x);
              vw[k] = Io<T>::unword(a.y, b.y);
            }
            *reinterpret_cast<uint4*>(ys + pairs) = make_uint4(vw[0], vw[1], vw[2], vw[3]);
          } else if (V == 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 u = Io<T>::word(uw[k]), e = e2[k];
              const float2 a = turn_pair(u.x, u.y, e);
              uw[k] = Io<T>::unword(a.x, a.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const float u = __uint_as_float(uw[k]), v = __uint_as_float(uw[k + 1]);
              const float2 a = turn_pair(u, v, e2[k / 2]);
              uw[k] = __float_as_uint(a.x);
              uw[k + 1] = __float_as_uint(a.y);
            }
          }
          *reinterpret_cast<uint4*>(ys) = make_uint4(uw[0], uw[1], uw[2], uw[3]);
        }
        r += 4 * apart;
        if (r < rows) load();
      }
    }
  } else {
    // odd sizes, strides or addresses: one pair, or one copied channel, at a time
    const int ncopy = copy ? dim - 2 * pairs : 0;
    const int per = pairs + ncopy, per_t = nh * per, all = nt * per_t;
    for (int i = tid; i < all; i += kRopeThreads) {
      const int t = i / per_t, r = i - t * per_t, h = r / per, c = r - h * per;
      const T* xs = x + (t0 + t) * xt + int64_t(h0 + h) * xh;
      T* ys = y + (t0 + t) * yt + int64_t(h0 + h) * yh;
      if (c >= pairs) {
        int at = c - pairs;
        if (at >= offset) at += 2 * pairs;
        ys[at] = xs[at];
      } else {
        const float2 e = cs[t * kMaxPairs + c];
        const int iu = offset + (kHalf ? c : 2 * c), iv = offset + (kHalf ? c + pairs : 2 * c + 1);
        const float u = Io<T>::get(xs[iu]), v = Io<T>::get(xs[iv]);
        const float2 a = turn_pair(u, v, e);
        ys[iu] = Io<T>::put(a.x);
        ys[iv] = Io<T>::put(a.y);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Cache append: one warp a row.  Lane l holds latent channels 8 l .. 8 l + 7 of
// both halves (the layout of the FP4 write) and rotary pair l.
//
// RMS norm y = x w / sqrt(mean x^2 + eps), rounded once, from the exact value,
// to bf16: the FP4 codes then follow the 64-bit definition bit for bit, as the
// codec's do.  fp32 arithmetic alone would round some thousandths of a percent
// of the values the other way, so
//   * x is scaled by the power of two that brings the row's largest value into
//     [1, 2), or, where the row is so small that eps outweighs its squares, eps to
//     1 or more (the squares' sums are right to 2^-40 of that); a lane adds its
//     16 squares to 64 (each step's rounding error is then exact in fp32 and summed
//     beside it), and both sums are added over the warp as integers;
//   * 1/sqrt is rsqrtf and one Newton step kept as a second fp32 part;
//   * x w is exact in fp32 (8 + 8 bits); only a product within 8 units of a
//     bf16 midpoint (one in 4,000) needs the low parts.
// Bound by its instructions, 584 a warp and row, and by the latencies between them: issue
// slots are 69 % busy with the 24 warps an SM that 79 registers leave.  131,072 rows with
// the bf16 rows written, 357 MB, in 89 us (4.0 TB/s; 53 us at the copy rate).
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendBlocks = 3;                    // resident on an SM

// xw * (r + rl) rounded once to bf16, for a product p = xw * r near a midpoint.
__device__ __noinline__ float near_midpoint(float xw, float r, float rl, float p) {
  const float e = __fmaf_rn(xw, r, -p) + xw * rl;
  float q = p + e;
  const float rest = (p - q) + e;
  if ((__float_as_uint(q) & 0xFFFFu) == 0x8000u && rest != 0.0f)
    q = __uint_as_float(__float_as_uint(q) + (((rest < 0.0f) == (q < 0.0f)) ? 1u : 0xFFFFFFFFu));
  return q;
}

// Largest magnitude bits of 8 bf16 values, two candidates in one word.
__device__ inline uint32_t bf16x8_top(uint4 v) {
  constexpr uint32_t m = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

// 8 scaled inputs g and weights w: bf16(g w (r + rl)), rounded once.
__device__ inline uint4 norm8(const float (&g)[8], const float (&w)[8], float r, float rl) {
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = g[i] * w[i];
    y[i] = x[i] * r;
  }
  // low halves within 8 of a midpoint, two values at a time (the carry between the two
  // halves of the sum widens the test of the upper one by 1)
  uint32_t near = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    near = __vminu2(near, __byte_perm(__float_as_uint(y[i]), __float_as_uint(y[i + 1]), 0x5410) + 0x80088008u);
  if ((near & 0xFFFFu) <= 17u || (near >> 16) <= 17u) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (((__float_as_uint(y[i]) + 0x8008u) & 0xFFFFu) <= 16u) y[i] = near_midpoint(x[i], r, rl, y[i]);
  }
  return Io<uint16_t>::pack(y);
}

// What a lane reads of a row.
struct AppendRow {
  uint4 v[2];
  uint32_t p, p2;                                    // rotary pair: one word, or (kHalf) one value each
  int32_t pos;
  int64_t dst;
};
template <bool kHalf>
__device__ inline AppendRow append_load(const uint16_t* x, int64_t stride, const int32_t* pos, const int64_t* dst, int64_t row,
                                        int lane) {
  AppendRow a;
  const uint16_t* xr = x + row * stride;
#pragma unroll
  for (int r = 0; r < 2; ++r) a.v[r] = __ldcs(reinterpret_cast<const uint4*>(xr) + r * 32 + lane);
  if (kHalf) {                                       // not put together here: that would wait for them
    a.p = __ldcs(xr + kLatent + lane);
    a.p2 = __ldcs(xr + kLatent + 32 + lane);
  } else {
    a.p = __ldcs(reinterpret_cast<const uint32_t*>(xr + kLatent) + lane);
    a.p2 = 0;
  }
  a.pos = __ldg(pos + row);
  a.dst = __ldg(dst + row);
  return a;
}

// The next row's loads are on their way while a row is worked on.
template <bool kHalf, bool kNorm>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks)
    append_kernel(const __grid_constant__ RopeTable tab, const uint16_t* __restrict__ x, int64_t n, int64_t stride,
                  const uint16_t* __restrict__ norm_w, float eps, int least_ex, const int32_t* __restrict__ pos,
                  const int64_t* __restrict__ dst_rows, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                  uint16_t* __restrict__ rope, int64_t cache_rows, uint16_t* __restrict__ entry) {
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
    if (kNorm) {
      const uint32_t b2 = __vmaxu2(bf16x8_top(v[0]), bf16x8_top(v[1]));
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(b2 & 0xFFFFu, b2 >> 16));
      // an infinity or a NaN in the row: its values as they are times 0 or NaN (below)
      const bool whole = top < 0x7F80u;
      // exponent of the row's largest value, at least least_ex (launch_append)
      const int ex = max(int(top >> 7) - 127, least_ex);
      const float up = whole ? __uint_as_float(uint32_t(127 - ex) << 23 | (ex == 127 ? 0x00400000u : 0u)) : 1.0f;
      float g[2][8], s = 64.0f, e = 0.0f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        Io<uint16_t>::unpack(v[r], g[r]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          g[r][i] *= up;
          const float t = __fmaf_rn(g[r][i], g[r][i], s);
          e += __fmaf_rn(g[r][i], g[r][i], s - t);
          s = t;
        }
      }
      // s - 64 < 64 in steps of 2^-17, |e| < 2^-13: integer sums over the warp
      const int hi = __reduce_add_sync(0xFFFFFFFFu, int((s - 64.0f) * 131072.0f));
      const int lo = __reduce_add_sync(0xFFFFFFFFu, __float2int_rn(e * 274877906944.0f));       // 2^38
      // mean + eps, scaled like x^2, as two fp32 parts
      const float m0 = float(hi & ~31) * 1.4901161193847656e-8f;                               // 2^-26
      const float m1 = float(hi & 31) * 1.4901161193847656e-8f + float(lo) * 7.105427357601002e-15f;   // 2^-47
      const float es = eps * up * up;
      const float ms = m0 + es, back = ms - m0;
      const float ml0 = (m0 - (ms - back)) + (es - back) + m1;
      const float mh = ms + ml0, ml = (ms - mh) + ml0;
      const float r0 = whole ? rsqrtf(mh) : top > 0x7F80u ? __uint_as_float(0x7FC00000u) : 0.0f;
      const float p = r0 * r0, pe = __fmaf_rn(r0, r0, -p);
      const float d = __fmaf_rn(-mh, p, 1.0f) - __fmaf_rn(mh, pe, ml * p);
      const float rl = 0.5f * r0 * d;
#pragma unroll
      for (int r = 0; r < 2; ++r) v[r] = norm8(g[r], w[r], r0, rl);
    }
    const float2 cs = rope_cs(tab, lane, ps);
    const float2 uv = turn_pair(u0, u1, cs);
    const uint32_t turned = bf16x2_rn(uv.x, uv.y);
    if (entry) {
      uint16_t* er = entry + row * kDqk;
#pragma unroll
      for (int r = 0; r < 2; ++r) __stcs(reinterpret_cast<uint4*>(er) + r * 32 + lane, v[r]);
      if (kHalf) {
        er[kLatent + lane] = uint16_t(turned);
        er[kLatent + 32 + lane] = uint16_t(turned >> 16);
      } else {
        __stcs(reinterpret_cast<uint32_t*>(er + kLatent) + lane, turned);
      }
    }
    if (dst < 0 || dst >= cache_rows) continue;       // the same for the whole warp
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t sc;
      codes[dst * 64 + r * 32 + lane] = fp4_quantize_half_group(v[r], &sc);
      if ((lane & 1) == 0) scales[dst * 32 + r * 16 + (lane >> 1)] = uint8_t(sc);
    }
    uint16_t* rr = rope + dst * kRope;
    if (kHalf) {
      rr[lane] = uint16_t(turned);
      rr[32 + lane] = uint16_t(turned >> 16);
    } else {
      reinterpret_cast<uint32_t*>(rr)[lane] = turned;
    }
  }
}

template <typename T>
cudaError_t rope_typed(const RopeArgs& a, cudaStream_t st) {
  constexpr int V = Io<T>::kVec;
  const RopeTable tab = rope_table(a.cfg);
  const bool half = a.cfg.layout == CSA2_ROPE_HALF;
  const int rot = a.cfg.rot;
  const bool copy = a.x != a.y;
  // 16-byte pieces wherever every piece of every head is whole and aligned
  const int64_t strides = a.x_token | a.x_head | a.y_token | a.y_head | a.offset | (half ? rot / 2 : rot) |
                          (copy ? a.dim : 0);
  const bool vec = strides % V == 0 && (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y)) % 16 == 0;
  const int64_t gx = (a.tokens + kRopeTok - 1) / kRopeTok;
  // few tokens: the heads are spread over CTAs (down to one a CTA), up to about four CTAs an SM
  int hper = a.heads;
  const int64_t want = int64_t(device_sms()) * 4;
  if (gx < want) {
    const int64_t split = min64(a.heads, (want + gx - 1) / gx);
    hper = int((a.heads + split - 1) / split);
  }
  const unsigned gy = unsigned((a.heads + hper - 1) / hper);
  cudaError_t e;
  auto kernel = half ? rope_kernel<T, true> : rope_kernel<T, false>;
  CSA2_PROFILED(st, "rope",
                (e = launch_pdl(kernel, dim3(unsigned(gx), gy), dim3(kRopeThreads), 0, st, 1, tab,
                                static_cast<const T*>(a.x), static_cast<T*>(a.y), a.pos, a.tokens, a.heads, a.dim,
                                a.offset, a.x_token, a.x_head, a.y_token, a.y_head, hper, copy ? 1 : 0, vec ? 1 : 0,
                                a.inverse ? -1.0f : 1.0f)));
  return e;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  return a.fp32 ? rope_typed<float>(a, st) : rope_typed<uint16_t>(a, st);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  const RopeTable tab = rope_table(a.cfg);
  // one row a warp up to what is resident at once (kAppendBlocks an SM), then rows in turn
  const int64_t want = (a.n + 7) / 8, cap = int64_t(device_sms()) * kAppendBlocks;
  const unsigned grid = unsigned(want < cap ? want : cap);
  const bool half = a.cfg.layout == CSA2_ROPE_HALF;
  auto kernel = a.norm_w ? (half ? append_kernel<true, true> : append_kernel<false, true>)
                         : (half ? append_kernel<true, false> : append_kernel<false, false>);
  // least power of two that rows are scaled by, as the exponent that it takes to 0: where it acts,
  // eps / 2^(2 ex) is 1 or more (eps 2^-149, the least, and ex -75: 2)
  const int least_ex = a.norm_w ? int(min64(-40, std::ilogb(a.eps) >> 1)) : 0;
  cudaError_t e;
  CSA2_PROFILED(st, "kv_append",
                (e = launch_pdl(kernel, dim3(grid), dim3(kAppendThreads), 0, st, 1, tab, a.x, a.n, a.x_stride, a.norm_w,
                                a.eps, least_ex, a.pos, a.dst_rows, reinterpret_cast<uint32_t*>(a.codes), a.scales, a.rope,
                                a.cache_rows, a.entry)));
  return e;
}

}  // namespace csa2
