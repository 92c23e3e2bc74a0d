// rope.cuh -- rotary positions: configurations (host) and angles (device).
//
// Pair i of a rotated part of `rot` channels turns by the angle pos * f_i.  The
// pages apply rotary positions to the 64 bf16 key channels and the matching
// query channels before the cache and the attention are reached; the layouts
// and the context scalings here are the published ones (rotary embedding;
// position interpolation; the base change and the by-parts rule of YaRN).
//
// Angles: pos reaches 2^20 and more, where an fp32 product pos * f_i is off by
// hundredths of a radian.  f_i / 2 pi is therefore held as a 64-bit fraction of
// a turn, and pos * F_i modulo 2^64 is the angle modulo one turn, exactly: one
// integer multiply in place of 64-bit floating point, which this GPU runs at a
// small part of its fp32 rate.  The top 32 bits give the angle: to 2^-32 turns, and
// 2^-34 for the fraction's own rounding at the farthest positions (rope_table.cuh).
// The sine and cosine are fp32.
#pragma once

#include <cmath>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "rope_table.cuh"

namespace csa2 {

// make_rope_table, remembered: a table is a pure function of its configuration, and the
// powers of 32 to 128 frequencies take longer than a decode step's kernel.
inline RopeTable rope_table(const csa2_rope& r) {
  struct Entry {
    bool used;
    csa2_rope r;
    RopeTable t;
  };
  constexpr int kEntries = 8;
  static std::mutex mu;
  static Entry cache[kEntries];
  static int next = 0;
  const auto same = [](const csa2_rope& a, const csa2_rope& b) {
    return a.rot == b.rot && a.scaling == b.scaling && a.mscale == b.mscale && a.theta == b.theta && a.factor == b.factor &&
           a.orig_ctx == b.orig_ctx && a.turns_lo == b.turns_lo && a.turns_hi == b.turns_hi;
  };
  std::lock_guard<std::mutex> lk(mu);
  for (const Entry& e : cache)
    if (e.used && same(e.r, r)) return e.t;
  Entry& e = cache[next];
  next = (next + 1) % kEntries;
  e.t = make_rope_table(r);
  e.r = r;
  e.used = true;
  return e.t;
}

// Checks of a rotary configuration (host).
inline csa2_status check_rope(const csa2_rope* r) {
  if (!r) return CSA2_ERR_INVALID_ARG;
  if (r->layout != CSA2_ROPE_INTERLEAVED && r->layout != CSA2_ROPE_HALF) return CSA2_ERR_INVALID_ARG;
  if (r->scaling < CSA2_ROPE_PLAIN || r->scaling > CSA2_ROPE_BASE) return CSA2_ERR_INVALID_ARG;
  if (r->rot < 2 || r->rot > kMaxRot || (r->rot & 1)) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (!(r->theta > 1.0) || !std::isfinite(r->theta) || !std::isfinite(r->mscale)) return CSA2_ERR_INVALID_ARG;
  if (r->scaling != CSA2_ROPE_PLAIN && (!(r->factor >= 1.0) || !std::isfinite(r->factor))) return CSA2_ERR_INVALID_ARG;
  if (r->scaling == CSA2_ROPE_PARTS &&
      (!(r->orig_ctx > 0.0) || !std::isfinite(r->orig_ctx) || !(r->turns_lo >= 0.0) || !(r->turns_hi > r->turns_lo) ||
       !std::isfinite(r->turns_hi)))
    return CSA2_ERR_INVALID_ARG;
  return CSA2_OK;
}

// (cos, sin) * mscale of pair i at position pos.  The angle, a 32-bit fraction of a turn,
// is taken to within an eighth of a turn of a multiple of a quarter, where the Taylor
// series about 0 to the 9th and 8th power are right to 2.5e-8 (the first terms left out,
// (pi/4)^11 / 11! and (pi/4)^10 / 10!).
__device__ inline float2 rope_cs(uint64_t turn, float mscale, int32_t pos) {
  const uint32_t a = uint32_t((uint64_t(int64_t(pos)) * turn) >> 32);           // modulo one turn
  const uint32_t q = (a + 0x20000000u) >> 30;                                    // nearest quarter
  const float x = float(int32_t(a - (q << 30))) * 1.4629180792671596e-9f;        // 2 pi / 2^32
  const float z = x * x;
  const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  // quarters: (c, s), (-s, c), (-c, -s), (s, -c)
  const float u = (q & 1) ? s : c, v = (q & 1) ? c : s;
  return make_float2(((q + 1) & 2) ? -u * mscale : u * mscale, (q & 2) ? -v * mscale : v * mscale);
}
__device__ inline float2 rope_cs(const RopeTable& t, int i, int32_t pos) { return rope_cs(t.turn[i], t.mscale, pos); }

}  // namespace csa2
