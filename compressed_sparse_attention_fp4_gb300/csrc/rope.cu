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
#include "rows.cuh"

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
// The norm is norm_row's (rows.cuh): the FP4 codes follow the 64-bit definition bit for bit, as
// the codec's do.
// Bound by its instructions, 584 a warp and row, and by the latencies between them: issue
// slots are 69 % busy with the 24 warps an SM that 79 registers leave.  131,072 rows with
// the bf16 rows written, 357 MB, in 89 us (4.0 TB/s; 53 us at the copy rate).
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendBlocks = 3;                    // resident on an SM

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
    if (kNorm) norm_row(v, w, eps, least_ex);
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
  const int least_ex = a.norm_w ? norm_least_exponent(a.eps) : 0;
  cudaError_t e;
  CSA2_PROFILED(st, "kv_append",
                (e = launch_pdl(kernel, dim3(grid), dim3(kAppendThreads), 0, st, 1, tab, a.x, a.n, a.x_stride, a.norm_w,
                                a.eps, least_ex, a.pos, a.dst_rows, reinterpret_cast<uint32_t*>(a.codes), a.scales, a.rope,
                                a.cache_rows, a.entry)));
  return e;
}

}  // namespace csa2
