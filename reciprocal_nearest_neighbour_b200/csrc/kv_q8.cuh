// A paged key-value cache of 8-bit codes: new tokens go in (keys rotated by their
// positions on the way), cached tokens come back as 16-bit values.
//
// A row is one token's d channels x of one head, the rotated key or the value, in fp32
// (the rotated key is not rounded to 16 bits in between).  Its scale is
//   s = max(max |x| / top, 2^-126),  top = 448 (e4m3) or 127 (int8),
// and its codes are x * (1 / s), rounded to nearest even; code * s is off by at most half
// a step: 2^-4 of the value (e4m3, 2^-10 s below 2^-6 s) or s / 2 (int8).  Both quotients
// are rounded to nearest, so scales and codes are functions of the fp32 row.  With a
// scale for each row, a token's codes never change when another token is added, and the
// smallest scale keeps 1 / s finite for rows of zeros too.  A row with a NaN or an
// infinity gets a NaN for its scale and reads back as NaN.
//
// Bound by memory: a 16-bit channel is read, a code and d-th of a scale written (append),
// or the other way round (read).
#pragma once
#include <cstdint>
#include "kv_append.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kQ8Warps = 4;
// Rows in flight a lane.
constexpr int kQ8Batch = 3;
constexpr float kQ8MinScale = 1.1754943508222875e-38f;  // 2^-126

enum CodeFormat : int { kE4m3 = 0, kInt8 = 1 };

struct AppendQ8Params {
  const uint16_t *q, *k, *v;        // q may be null
  uint16_t *q_out, *k_out;          // k_out may be null
  uint8_t *kc, *vc;
  float* scales;                    // [page][head][row][key, value]
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;  // elements
  int64_t kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs, s_ps, s_hs;
  const int32_t *table, *start, *cu, *positions;  // positions may be null
  int64_t table_bs, pos_ts, num_pages;
  const double* inv_freq;
  int T, B, Hq, Hkv, d;             // Hq = 0 without queries
  int max_pages, page_size;
  int pairs, axes;                  // channel pairs per axis, axes (0: no rotation)
  int paired;                       // pairs side by side instead of half a block apart
  int share;                        // log2 of the warps that share a token
  int row_lanes;                    // log2 of the lanes of a row, 8 channels each
};

// Codes of 8 channels, 4 a word.
template <int kFmt>
__device__ __forceinline__ uint2 q8_codes(const float (&x)[8], float inv) {
  uint2 r;
  uint32_t* w = &r.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // (products of their own: fused with the sum below they would be rounded once only)
    const float a = __fmul_rn(x[4 * h], inv), b = __fmul_rn(x[4 * h + 1], inv);
    const float c = __fmul_rn(x[4 * h + 2], inv), e = __fmul_rn(x[4 * h + 3], inv);
    if constexpr (kFmt == kE4m3) {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(e), "f"(c));
      w[h] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    } else {
      // added to 1.5 * 2^23, a number of up to 2^22 rounds to the integer that its
      // lowest bits then hold
      constexpr float kTo = 12582912.f;
      const uint32_t i0 = __float_as_uint(a + kTo), i1 = __float_as_uint(b + kTo);
      const uint32_t i2 = __float_as_uint(c + kTo), i3 = __float_as_uint(e + kTo);
      w[h] = __byte_perm(__byte_perm(i0, i1, 0x0040), __byte_perm(i2, i3, 0x0040), 0x5410);
    }
  }
  return r;
}

// The fp32 values of 4 codes.
template <int kFmt>
__device__ __forceinline__ void q8_floats(uint32_t w, float (&x)[4]) {
  if constexpr (kFmt == kE4m3) {
    uint32_t lo, hi;  // e4m3 is exact in fp16
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(w)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(w >> 16)));
    const float2 a = unpack2<false>(lo), b = unpack2<false>(hi);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = static_cast<float>(static_cast<int8_t>(w >> (8 * e)));
  }
}

// Row of a token in the caches, or nothing.
struct CachePlace {
  int64_t page;  // -1: not there
  int row;
};
__device__ __forceinline__ CachePlace cache_place(int64_t place, const int32_t* table, int max_pages,
                                                  int page_size, int64_t num_pages) {
  CachePlace at{-1, 0};
  if (place >= 0 && place < static_cast<int64_t>(max_pages) * page_size) {
    const int pg = static_cast<int>(place / page_size);
    at.row = static_cast<int>(place - static_cast<int64_t>(pg) * page_size);
    const int64_t id = __ldg(table + pg);
    if (id >= 0 && id < num_pages) at.page = id;
  }
  return at;
}

// A lane holds 8 neighbouring channels of a row and fetches their partners of the
// rotation again beside them (from the first-level cache, in pieces of kVec channels,
// the widest that divides the pairs), so that rows of every layout are read, reduced to
// their maximum and written in their natural order, by 1 to 32 lanes each.
template <bool kBf16, int kFmt, int kVec>
__global__ void __launch_bounds__(kQ8Warps * 32, 8) kv_append_q8_kernel(const AppendQ8Params p) {
  using V = typename VecOf<kVec>::T;
  constexpr float kTop = kFmt == kE4m3 ? 448.f : 127.f;
  extern __shared__ __align__(16) float2 app_turns[];  // [warp][axes * pairs] cos, sin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kQ8Warps + warp;
  if ((gw >> p.share) >= p.T) return;
  const int t = static_cast<int>(gw >> p.share);
  const int part = static_cast<int>(gw) & ((1 << p.share) - 1);
  const int angles = p.axes * p.pairs, rotated = 2 * angles;
  float2* turn = app_turns + warp * ((angles + 1) & ~1);
  const int c0 = (lane & ((1 << p.row_lanes) - 1)) * 8;  // this lane's channels
  const bool live = c0 < p.d;
  const int per_pass = 32 >> p.row_lanes;                // rows of a pass over the warp
  const int n_rows = p.Hq + 2 * p.Hkv;                   // queries, keys, values
  const int first = part * per_pass + (lane >> p.row_lanes), step = per_pass << p.share;

  uint4 x[kQ8Batch];
  union Partner { uint4 v; V part[8 / kVec]; } y[kQ8Batch];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kQ8Batch; ++i) {
      const int r = r0 + i * step;
      if (r >= n_rows || !live) break;
      const uint16_t* src = r < p.Hq             ? p.q + t * p.q_ts + r * p.q_hs
                            : r < p.Hq + p.Hkv   ? p.k + t * p.k_ts + (r - p.Hq) * p.k_hs
                                                 : p.v + t * p.v_ts + (r - p.Hq - p.Hkv) * p.v_hs;
      x[i] = *reinterpret_cast<const uint4*>(src + c0);
      if (p.paired || r >= p.Hq + p.Hkv) continue;
#pragma unroll
      for (int s = 0; s < 8 / kVec; ++s) {
        const int c = c0 + s * kVec;
        if (c >= rotated) break;
        const int in = c >= 2 * p.pairs ? c - 2 * p.pairs : c;  // within its axis
        y[i].part[s] =
            *reinterpret_cast<const V*>(src + (in < p.pairs ? c + p.pairs : c - p.pairs));
      }
    }
  };
  fetch(first);
  // ---- the token's sequence, cache row and angles
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0 || b >= p.B) return;
  const int64_t place = static_cast<int64_t>(__ldg(p.start + b)) + t - __ldg(p.cu + b);
  const CachePlace at =
      cache_place(place, p.table + b * p.table_bs, p.max_pages, p.page_size, p.num_pages);
  for (int a = lane; a < angles; a += 32) {
    const int axis = a >= p.pairs ? 1 : 0;
    const double pos = p.positions ? static_cast<double>(__ldg(p.positions + t * p.pos_ts + axis))
                                   : static_cast<double>(place);
    double turns = pos * __ldg(p.inv_freq + (a - axis * p.pairs)) * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns), &s, &c);
    turn[a] = make_float2(c, s);
  }
  __syncwarp();
  // (the bound is the warp's, so that all its lanes reach the reductions)
  for (int r0 = first; r0 - (lane >> p.row_lanes) < n_rows; r0 += kQ8Batch * step) {
    if (r0 != first) fetch(r0);
    __syncwarp();  // rows rotated in place are written behind every lane's reads
#pragma unroll
    for (int i = 0; i < kQ8Batch; ++i) {
      const int r = r0 + i * step;
      if (r - (lane >> p.row_lanes) >= n_rows) break;
      const bool here = live && r < n_rows;
      const bool is_q = r < p.Hq, is_k = !is_q && r < p.Hq + p.Hkv;
      float f[8];
      const uint32_t xw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 u = here ? unpack2<kBf16>(xw[e]) : make_float2(0.f, 0.f);
        f[2 * e] = u.x, f[2 * e + 1] = u.y;
      }
      if (here && (is_q || is_k) && c0 < rotated) {
        if (p.paired) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c0 + 2 * e >= rotated) break;
            const float2 cs = turn[c0 / 2 + e];
            const float one = f[2 * e], two = f[2 * e + 1];
            f[2 * e] = one * cs.x - two * cs.y;
            f[2 * e + 1] = two * cs.x + one * cs.y;
          }
        } else {
          const uint32_t yw[4] = {y[i].v.x, y[i].v.y, y[i].v.z, y[i].v.w};
          float g[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = unpack2<kBf16>(yw[e]);
            g[2 * e] = u.x, g[2 * e + 1] = u.y;
          }
#pragma unroll
          for (int s = 0; s < 8 / kVec; ++s) {
            const int c = c0 + s * kVec;
            if (c >= rotated) break;
            const int axis = c >= 2 * p.pairs ? 1 : 0, in = c - 2 * axis * p.pairs;
            const bool second = in >= p.pairs;
            const float2* cs = turn + axis * p.pairs + (second ? in - p.pairs : in);
#pragma unroll
            for (int e = s * kVec; e < (s + 1) * kVec; ++e) {
              const float2 z = cs[e - s * kVec];
              f[e] = f[e] * z.x + g[e] * (second ? z.y : -z.y);
            }
          }
        }
      }
      if (here && (is_q || (is_k && p.k_out))) {
        uint16_t* dst = is_q ? p.q_out + t * p.qo_ts + r * p.qo_hs
                             : p.k_out + t * p.ko_ts + (r - p.Hq) * p.ko_hs;
        *reinterpret_cast<uint4*>(dst + c0) =
            make_uint4(pack2<kBf16>(f[0], f[1]), pack2<kBf16>(f[2], f[3]),
                       pack2<kBf16>(f[4], f[5]), pack2<kBf16>(f[6], f[7]));
      }
      if (r - (lane >> p.row_lanes) + per_pass <= p.Hq) continue;  // queries only
      // the largest magnitude by its bits: a NaN's are above infinity's
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
      for (int o = 1; o < (1 << p.row_lanes); o <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!here || is_q || at.page < 0) continue;
      float scale = fmaxf(__fdiv_rn(__uint_as_float(top), kTop), kQ8MinScale);
      if (top >= 0x7F800000u) scale = __uint_as_float(0x7FC00000u);
      const uint2 codes = q8_codes<kFmt>(f, __fdiv_rn(1.f, scale));
      const int h = is_k ? r - p.Hq : r - p.Hq - p.Hkv;
      uint8_t* dst = is_k ? p.kc + at.page * p.kc_ps + at.row * p.kc_ts + h * p.kc_hs
                          : p.vc + at.page * p.vc_ps + at.row * p.vc_ts + h * p.vc_hs;
      *reinterpret_cast<uint2*>(dst + c0) = codes;
      if (c0 == 0)
        p.scales[at.page * p.s_ps + h * p.s_hs + 2 * at.row + (is_k ? 0 : 1)] = scale;
    }
  }
}

struct ReadQ8Params {
  const uint8_t *kc, *vc;
  const float* scales;
  uint16_t *k, *v;
  int64_t kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs, s_ps, s_hs;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int32_t *table, *start, *cu;  // start may be null
  int64_t table_bs, num_pages;
  int T, B, Hkv, d, max_pages, page_size;
  int share;
  FastDiv by_row;                   // 8-channel units of a row
};

constexpr int kReadBatch = 4;

// One warp a token (for few tokens up to 8); a unit is 8 channels of a head, the keys'
// units first.
template <bool kBf16, int kFmt>
__global__ void __launch_bounds__(kQ8Warps * 32) kv_read_q8_kernel(const ReadQ8Params p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kQ8Warps + warp;
  if ((gw >> p.share) >= p.T) return;
  const int t = static_cast<int>(gw >> p.share);
  const int part = static_cast<int>(gw) & ((1 << p.share) - 1);
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0 || b >= p.B) return;
  const int64_t place =
      static_cast<int64_t>(p.start ? __ldg(p.start + b) : 0) + t - __ldg(p.cu + b);
  const CachePlace at =
      cache_place(place, p.table + b * p.table_bs, p.max_pages, p.page_size, p.num_pages);
  const int row_units = p.by_row.div, half = p.Hkv * row_units;
  const int step = 32 << p.share;
  for (int u0 = part * 32 + lane; u0 < 2 * half; u0 += kReadBatch * step) {
    uint2 w[kReadBatch];
    float s[kReadBatch];
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int u = u0 + i * step;
      if (u >= 2 * half) break;
      const bool is_v = u >= half;
      const int in = is_v ? u - half : u, h = fdiv(in, p.by_row), c = (in - h * row_units) * 8;
      w[i] = make_uint2(0u, 0u);
      s[i] = 0.f;
      if (at.page >= 0) {
        const uint8_t* src = is_v ? p.vc + at.page * p.vc_ps + at.row * p.vc_ts + h * p.vc_hs
                                  : p.kc + at.page * p.kc_ps + at.row * p.kc_ts + h * p.kc_hs;
        w[i] = __ldg(reinterpret_cast<const uint2*>(src + c));
        s[i] = __ldg(p.scales + at.page * p.s_ps + h * p.s_hs + 2 * at.row + (is_v ? 1 : 0));
      }
    }
#pragma unroll
    for (int i = 0; i < kReadBatch; ++i) {
      const int u = u0 + i * step;
      if (u >= 2 * half) break;
      const bool is_v = u >= half;
      const int in = is_v ? u - half : u, h = fdiv(in, p.by_row), c = (in - h * row_units) * 8;
      float a[4], e[4];
      q8_floats<kFmt>(w[i].x, a);
      q8_floats<kFmt>(w[i].y, e);
      uint16_t* dst = is_v ? p.v + t * p.v_ts + h * p.v_hs : p.k + t * p.k_ts + h * p.k_hs;
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(
          pack2<kBf16>(a[0] * s[i], a[1] * s[i]), pack2<kBf16>(a[2] * s[i], a[3] * s[i]),
          pack2<kBf16>(e[0] * s[i], e[1] * s[i]), pack2<kBf16>(e[2] * s[i], e[3] * s[i]));
    }
  }
}

}  // namespace rnn
