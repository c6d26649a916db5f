// Append of packed new tokens to a paged key-value cache, keys and queries
// rotated by their positions on the way.
//
// Token t of sequence b (cu[b] <= t < cu[b+1]) is number start[b] + t - cu[b]
// of its sequence and goes to row (number % page_size) of page
// table[b][number / page_size].  A rotated pair of channels (x1, x2) becomes
// (x1 cos a - x2 sin a, x2 cos a + x1 sin a) with a = position * inv_freq[i].
//
// Bound by memory: every channel is read once and written once or twice.  One
// warp takes a token (for few tokens up to 8 warps share one), so nothing
// waits at block level: it fetches its first units, looks the token's sequence
// and cache row up under that latency, makes the token's cosines and sines once
// (in 64 bits up to the fraction of a turn: at position 10^6 a 32-bit angle is
// off by 0.06), and then moves the heads' channels in batches of kAppBatch units
// of up to 2 x 16 bytes a lane.
#pragma once
#include <cstdint>
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace rnn {

// Blocks of 4 warps of at most 64 registers, 3 units in flight a lane.  14 prompt
// chunks (21326 tokens, 32/8 heads of 128, 568 MB) and 24 frames (18432 tokens, 12
// heads of 64, 198 MB): 99 and 35 us; with 4 units 97 and 36.  (Before the words were
// converted in pairs: 107 and 35, blocks of 8 warps with 4 units 110 and 39, blocks
// of 2 warps 110 and 35.)
constexpr int kAppWarps = 4;
constexpr int kAppBatch = 3;

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
  int share;                        // log2 of the warps that share a token
  FastDiv by_unit, by_vunit;        // units of a query or key row, of a value row
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

// A unit of a query or key row: kVec pairs (two vectors), or kVec channels
// behind the rotated ones (one vector).
template <int kVec>
struct AppUnit {
  using V = typename VecOf<kVec>::T;
  V a, b;
};
struct AppPlace {
  int ca, cb, turn;  // channels of the two vectors (cb < 0: one), first pair's angle
};
template <int kVec>
__device__ __forceinline__ AppPlace app_place(int unit, const AppendParams& p) {
  const int per_axis = p.pairs / kVec, rot = p.axes * per_axis;
  AppPlace at;
  if (unit >= rot) {
    at.ca = 2 * p.axes * p.pairs + (unit - rot) * kVec;
    at.cb = -1;
    at.turn = 0;
    return at;
  }
  const int axis = unit >= per_axis ? 1 : 0;
  const int i0 = (unit - axis * per_axis) * kVec;  // first pair
  const int base = 2 * axis * p.pairs;
  at.ca = base + (p.paired ? 2 * i0 : i0);
  at.cb = p.paired ? at.ca + kVec : at.ca + p.pairs;
  at.turn = axis * p.pairs + i0;
  return at;
}

// Rotated in fp32, rounded once.  Two channels a word: (x1, x2) of one pair when
// they lie side by side, else two pairs' x1 in `a` and their x2 in `b`.
template <bool kBf16, int kVec>
__device__ __forceinline__ void app_rotate(AppUnit<kVec>& u, const float2* cs, bool paired) {
  if constexpr (kVec == 1) {
    const float x1 = app_float<kBf16>(u.a), x2 = app_float<kBf16>(u.b);
    u.a = app_bits<kBf16>(x1 * cs->x - x2 * cs->y);
    u.b = app_bits<kBf16>(x2 * cs->x + x1 * cs->y);
  } else {
    constexpr int kWords = kVec / 2;
    union Words { typename VecOf<kVec>::T v; uint32_t w[kWords]; } a, b;
    a.v = u.a;
    b.v = u.b;
    const float4* turns = reinterpret_cast<const float4*>(cs);  // cos, sin of two pairs
    if (paired) {
      uint32_t x[2 * kWords];
#pragma unroll
      for (int e = 0; e < kWords; ++e) x[e] = a.w[e], x[kWords + e] = b.w[e];
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        const float4 t = turns[e];
        const float2 p = unpack2<kBf16>(x[2 * e]), q = unpack2<kBf16>(x[2 * e + 1]);
        x[2 * e] = pack2<kBf16>(p.x * t.x - p.y * t.y, p.y * t.x + p.x * t.y);
        x[2 * e + 1] = pack2<kBf16>(q.x * t.z - q.y * t.w, q.y * t.z + q.x * t.w);
      }
#pragma unroll
      for (int e = 0; e < kWords; ++e) a.w[e] = x[e], b.w[e] = x[kWords + e];
    } else {
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        const float4 t = turns[e];
        const float2 x1 = unpack2<kBf16>(a.w[e]), x2 = unpack2<kBf16>(b.w[e]);
        a.w[e] = pack2<kBf16>(x1.x * t.x - x2.x * t.y, x1.y * t.z - x2.y * t.w);
        b.w[e] = pack2<kBf16>(x2.x * t.x + x1.x * t.y, x2.y * t.z + x1.y * t.w);
      }
    }
    u.a = a.v;
    u.b = b.v;
  }
}

template <bool kBf16, int kVec>
__global__ void __launch_bounds__(kAppWarps * 32, 8) kv_append_kernel(const AppendParams p) {
  using V = typename VecOf<kVec>::T;
  extern __shared__ __align__(16) float2 app_turns[];  // [warp][axes * pairs] cos, sin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kAppWarps + warp;
  if ((gw >> p.share) >= p.T) return;
  const int t = static_cast<int>(gw >> p.share);
  const int part = static_cast<int>(gw) & ((1 << p.share) - 1);
  const int first = part * 32 + lane, step = 32 << p.share;
  const int angles = p.axes * p.pairs;
  float2* turn = app_turns + warp * angles;
  const int row_units = p.by_unit.div;
  const int n_units = (p.Hq + p.Hkv) * row_units;
  const uint16_t* q_row = p.q + t * p.q_ts;  // never read without queries
  const uint16_t* k_row = p.k + t * p.k_ts;
  AppUnit<kVec> u[kAppBatch];
  auto fetch = [&](int u0) {
#pragma unroll
    for (int i = 0; i < kAppBatch; ++i) {
      const int r = u0 + i * step;
      if (r >= n_units) break;
      const int h = fdiv(r, p.by_unit);
      const AppPlace at = app_place<kVec>(r - h * row_units, p);
      const uint16_t* src = h < p.Hq ? q_row + h * p.q_hs : k_row + (h - p.Hq) * p.k_hs;
      u[i].a = *reinterpret_cast<const V*>(src + at.ca);
      if (at.cb >= 0) u[i].b = *reinterpret_cast<const V*>(src + at.cb);
    }
  };
  fetch(first);
  // ---- the token's sequence, cache row and angles
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0 || b >= p.B) return;
  const int64_t place = static_cast<int64_t>(__ldg(p.start + b)) + t - __ldg(p.cu + b);
  int64_t ka = -1, va = -1;  // its row in the caches, -1: nowhere
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
    const double pos = p.positions ? static_cast<double>(__ldg(p.positions + t * p.pos_ts + axis))
                                   : static_cast<double>(place);
    double turns = pos * __ldg(p.inv_freq + (a - axis * p.pairs)) * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns), &s, &c);
    turn[a] = make_float2(c, s);
  }
  __syncwarp();
  // ---- queries and keys
  for (int u0 = first; u0 < n_units; u0 += kAppBatch * step) {
    if (u0 != first) fetch(u0);
#pragma unroll
    for (int i = 0; i < kAppBatch; ++i) {
      const int r = u0 + i * step;
      if (r >= n_units) break;
      const int h = fdiv(r, p.by_unit);
      const AppPlace at = app_place<kVec>(r - h * row_units, p);
      const bool two = at.cb >= 0;
      if (two) app_rotate<kBf16, kVec>(u[i], turn + at.turn, p.paired != 0);
      auto store = [&](uint16_t* dst) {
        *reinterpret_cast<V*>(dst + at.ca) = u[i].a;
        if (two) *reinterpret_cast<V*>(dst + at.cb) = u[i].b;
      };
      if (h < p.Hq) {
        store(p.q_out + t * p.qo_ts + h * p.qo_hs);
      } else {
        if (p.k_out) store(p.k_out + t * p.ko_ts + (h - p.Hq) * p.ko_hs);
        if (ka >= 0) store(p.kc + ka + (h - p.Hq) * p.kc_hs);
      }
    }
  }
  // ---- values
  if (va < 0) return;
  const int vrow = p.by_vunit.div, n_v = p.Hkv * vrow;
  const uint16_t* v_row = p.v + t * p.v_ts;
  uint16_t* v_dst = p.vc + va;
  for (int r0 = first; r0 < n_v; r0 += kAppBatch * step) {
    uint4 x[kAppBatch];
#pragma unroll
    for (int i = 0; i < kAppBatch; ++i) {
      const int r = r0 + i * step, h = fdiv(r, p.by_vunit);
      if (r < n_v)
        x[i] = *reinterpret_cast<const uint4*>(v_row + h * p.v_hs + (r - h * vrow) * 8);
    }
#pragma unroll
    for (int i = 0; i < kAppBatch; ++i) {
      const int r = r0 + i * step, h = fdiv(r, p.by_vunit);
      if (r < n_v) *reinterpret_cast<uint4*>(v_dst + h * p.vc_hs + (r - h * vrow) * 8) = x[i];
    }
  }
}

}  // namespace rnn
