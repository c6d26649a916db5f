// Append of packed new tokens to a paged key-value cache, keys and queries
// rotated by their positions on the way.
//
// Token t of sequence b (cu[b] <= t < cu[b+1]) is number start[b] + t - cu[b]
// of its sequence and goes to row (number % page_size) of page
// table[b][number / page_size].  A rotated pair of channels (x1, x2) becomes
// (x1 cos a - x2 sin a, x2 cos a + x1 sin a) with a = position * inv_freq[i].
//
// Bound by memory: every channel is read once and written once or twice.  A
// block takes a few tokens: first a warp per token looks its sequence and its
// cache row up and makes the token's cosines and sines once (in 64 bits up to
// the fraction of a turn: at position 10^6 a 32-bit angle is off by 0.06),
// then all threads move the heads' channels in units of up to 2 x 16 bytes
// (both halves of kVec pairs), which read the angles from shared memory.
#pragma once
#include <cstdint>
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kAppThreads = 256;
constexpr int kAppMaxTokens = 8;

struct AppendParams {
  const uint16_t *q, *k, *v;        // q may be null
  uint16_t *q_out, *k_out;          // k_out may be null
  uint16_t *kc, *vc;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;  // elements
  int64_t kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs;
  const int32_t *table, *start, *cu, *positions;  // positions may be null
  int64_t table_bs, pos_ts, num_pages;
  const double* inv_freq;
  int T, B, Hq, Hkv, d;             // Hq = 0 without queries
  int max_pages, page_size;
  int pairs, axes;                  // channel pairs per axis, axes (0: no rotation)
  int paired;                       // pairs side by side instead of half a block apart
  int tokens;                       // tokens per block
  FastDiv by_row, by_unit, by_vunit;  // units of a token's rotated rows, of one such row, of a
                                      // value row
};

// Sequence of token t: the last b with cu[b] <= t, -1 before the first and B
// behind the last.  The 32 lanes look at 32 places at a time.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
  int lo = -1, left = B + 1;  // cu[lo] <= t, candidates lo+1 .. lo+left
  while (left > 0) {
    const int step = (left + 31) >> 5;
    const int at = (lane + 1) * step;
    const bool in = at <= left;
    const unsigned le = __ballot_sync(0xffffffffu, in && __ldg(cu + lo + at) <= t);
    const int c = __popc(le & ~(le + 1u));  // leading run of lanes below t
    lo += c * step;
    left = min(step - 1, left - c * step);
  }
  return lo;
}

template <int kVec>
struct VecOf;
template <> struct VecOf<8> { using T = uint4; };
template <> struct VecOf<4> { using T = uint2; };
template <> struct VecOf<2> { using T = uint32_t; };
template <> struct VecOf<1> { using T = uint16_t; };

template <bool kBf16>
__device__ __forceinline__ float app_float(uint16_t h) {
  return kBf16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
}
template <bool kBf16>
__device__ __forceinline__ uint16_t app_bits(float x) {
  return kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
               : __half_as_ushort(__float2half_rn(x));
}

// One unit of a rotated row: kVec pairs, or kVec channels behind the rotated
// ones.  Outputs are rounded once from fp32.
template <bool kBf16, int kVec>
__device__ __forceinline__ void app_unit(const uint16_t* src, uint16_t* dst0, uint16_t* dst1,
                                         int unit, const AppendParams& p, const float2* turn) {
  using V = typename VecOf<kVec>::T;
  const int per_axis = p.pairs / kVec, rot = p.axes * per_axis;
  if (unit >= rot) {
    const int c = 2 * p.axes * p.pairs + (unit - rot) * kVec;
    const V x = *reinterpret_cast<const V*>(src + c);
    if (dst0) *reinterpret_cast<V*>(dst0 + c) = x;
    if (dst1) *reinterpret_cast<V*>(dst1 + c) = x;
    return;
  }
  const int axis = (p.axes > 1 && unit >= per_axis) ? 1 : 0;
  const int i0 = (unit - axis * per_axis) * kVec;          // first pair
  const int base = 2 * axis * p.pairs;
  const int ca = base + (p.paired ? 2 * i0 : i0);
  const int cb = p.paired ? ca + kVec : ca + p.pairs;
  union { V v[2]; uint16_t h[2 * kVec]; } x, y;
  x.v[0] = *reinterpret_cast<const V*>(src + ca);
  x.v[1] = *reinterpret_cast<const V*>(src + cb);
  const float2* cs = turn + axis * p.pairs + i0;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float2 t = cs[e];
    // pair e: elements (e, kVec + e) of halves, (2e, 2e + 1) side by side
    const float a0 = app_float<kBf16>(x.h[e]), a1 = app_float<kBf16>(x.h[kVec + e]);
    const float b0 = app_float<kBf16>(x.h[2 * e]), b1 = app_float<kBf16>(x.h[2 * e + 1]);
    const float x1 = p.paired ? b0 : a0, x2 = p.paired ? b1 : a1;
    const uint16_t r1 = app_bits<kBf16>(x1 * t.x - x2 * t.y);
    const uint16_t r2 = app_bits<kBf16>(x2 * t.x + x1 * t.y);
    if (p.paired) {
      y.h[2 * e] = r1;
      y.h[2 * e + 1] = r2;
    } else {
      y.h[e] = r1;
      y.h[kVec + e] = r2;
    }
  }
  if (dst0) {
    *reinterpret_cast<V*>(dst0 + ca) = y.v[0];
    *reinterpret_cast<V*>(dst0 + cb) = y.v[1];
  }
  if (dst1) {
    *reinterpret_cast<V*>(dst1 + ca) = y.v[0];
    *reinterpret_cast<V*>(dst1 + cb) = y.v[1];
  }
}

template <bool kBf16, int kVec>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const AppendParams p) {
  extern __shared__ float2 app_turn[];  // [tokens][axes * pairs] cos, sin
  __shared__ int64_t k_at[kAppMaxTokens], v_at[kAppMaxTokens];  // cache rows, -1: nowhere
  __shared__ int alive[kAppMaxTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, p.T - t0);
  const int angles = p.axes * p.pairs;
  for (int i = warp; i < nt; i += kAppThreads / 32) {
    const int t = t0 + i;
    const int b = find_sequence(p.cu, p.B, t, lane);
    const bool live = b >= 0 && b < p.B;
    int64_t place = 0, ka = -1, va = -1;
    if (live) {
      place = static_cast<int64_t>(__ldg(p.start + b)) + t - __ldg(p.cu + b);
      if (place >= 0 && place < static_cast<int64_t>(p.max_pages) * p.page_size) {
        const int pg = static_cast<int>(place / p.page_size);
        const int row = static_cast<int>(place - static_cast<int64_t>(pg) * p.page_size);
        const int64_t id = __ldg(p.table + b * p.table_bs + pg);
        if (id >= 0 && id < p.num_pages) {
          ka = id * p.kc_ps + row * p.kc_ts;
          va = id * p.vc_ps + row * p.vc_ts;
        }
      }
      for (int a = lane; a < angles; a += 32) {
        const int axis = a >= p.pairs ? 1 : 0;
        const double pos = p.positions
                               ? static_cast<double>(p.positions[t * p.pos_ts + axis])
                               : static_cast<double>(place);
        double turns = pos * __ldg(p.inv_freq + (a - axis * p.pairs)) * 0.15915494309189533577;
        turns -= rint(turns);
        float s, c;
        sincospif(2.0f * static_cast<float>(turns), &s, &c);
        app_turn[i * angles + a] = make_float2(c, s);
      }
    }
    if (lane == 0) {
      alive[i] = live;
      k_at[i] = ka;
      v_at[i] = va;
    }
  }
  __syncthreads();
  const int row_units = p.by_unit.div, tok_units = p.by_row.div;  // rotated rows
  const int n_rot = nt * tok_units;
  for (int u = threadIdx.x; u < n_rot; u += kAppThreads) {
    const int i = fdiv(u, p.by_row);
    if (!alive[i]) continue;
    const int r = u - i * tok_units;
    const int h = fdiv(r, p.by_unit), unit = r - h * row_units;
    const int64_t t = t0 + i;
    const uint16_t* src;
    uint16_t *dst0, *dst1 = nullptr;
    if (h < p.Hq) {
      src = p.q + t * p.q_ts + h * p.q_hs;
      dst0 = p.q_out + t * p.qo_ts + h * p.qo_hs;
    } else {
      const int hk = h - p.Hq;
      src = p.k + t * p.k_ts + hk * p.k_hs;
      dst0 = p.k_out ? p.k_out + t * p.ko_ts + hk * p.ko_hs : nullptr;
      dst1 = k_at[i] >= 0 ? p.kc + k_at[i] + hk * p.kc_hs : nullptr;
    }
    app_unit<kBf16, kVec>(src, dst0, dst1, unit, p, app_turn + i * angles);
  }
  const int vrow = p.by_vunit.div, tok_v = p.Hkv * vrow;
  for (int i = 0; i < nt; ++i) {
    if (v_at[i] < 0) continue;
    const int64_t t = t0 + i;
    for (int r = threadIdx.x; r < tok_v; r += kAppThreads) {
      const int h = fdiv(r, p.by_vunit), c = (r - h * vrow) * 8;
      *reinterpret_cast<uint4*>(p.vc + v_at[i] + h * p.vc_hs + c) =
          *reinterpret_cast<const uint4*>(p.v + t * p.v_ts + h * p.v_hs + c);
    }
  }
}

}  // namespace rnn
