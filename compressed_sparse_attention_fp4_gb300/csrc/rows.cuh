// rows.cuh -- a projection's row of 576 channels (512 latent, 64 rotary) in one warp: loads, the
// latent's RMS norm, the turn of a pair.  Shared by the FP4 cache append (rope.cu) and the append
// of exact rows (newrows.cu).
#pragma once

#include <cmath>

#include "common.cuh"

namespace csa2 {

// least power of two that rows are scaled by, as the exponent that it takes to 0: where it acts,
// eps / 2^(2 ex) is 1 or more (eps 2^-149, the least, and ex -75: 2)
inline int norm_least_exponent(float eps) { return int(min64(-40, std::ilogb(eps) >> 1)); }

namespace {

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

// RMS norm y = x w / sqrt(mean x^2 + eps), rounded once, from the exact value,
// to bf16.  fp32 arithmetic alone would round some thousandths of a percent
// of the values the other way, so
//   * x is scaled by the power of two that brings the row's largest value into
//     [1, 2), or, where the row is so small that eps outweighs its squares, eps to
//     1 or more (the squares' sums are right to 2^-40 of that); a lane adds its
//     16 squares to 64 (each step's rounding error is then exact in fp32 and summed
//     beside it), and both sums are added over the warp as integers;
//   * 1/sqrt is rsqrtf and one Newton step kept as a second fp32 part;
//   * x w is exact in fp32 (8 + 8 bits); only a product within 8 units of a
//     bf16 midpoint (one in 4,000) needs the low parts.
// Lane l holds channels 8 l .. 8 l + 7 of both halves of the row (v) and of the weights (w).
__device__ __forceinline__ void norm_row(uint4 (&v)[2], const float (&w)[2][8], float eps, int least_ex) {
  const uint32_t b2 = __vmaxu2(bf16x8_top(v[0]), bf16x8_top(v[1]));
  const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(b2 & 0xFFFFu, b2 >> 16));
  // an infinity or a NaN in the row: its values as they are times 0 or NaN (below)
  const bool whole = top < 0x7F80u;
  // exponent of the row's largest value, at least least_ex (norm_least_exponent)
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

}  // namespace

}  // namespace csa2
