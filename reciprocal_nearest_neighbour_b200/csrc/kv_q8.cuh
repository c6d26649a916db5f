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
// or the other way round (read).  What an append takes is enough reads under way (a warp has
// three passes over its rows on their way to shared memory), few instructions a pass, and
// whole sectors.  Measured, in a CUDA graph: 11 prompt chunks, 25825 tokens of 32/8 heads of
// 128, bf16 to e4m3, 583 MB, 94 us (6.2 TB/s, 0.95 of a copy's rate); with rows of 72
// channels, whose 36 pairs come in pieces of 4, 122 us for 328 MB (2.7 TB/s).  One token 3.4 us.
#pragma once
#include <cstdint>
#include <type_traits>
#include "kv_append.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kQ8Warps = 4;
// Passes of a warp (32 lanes of up to 16 channels) in its ring, all but one of them on
// their way while one is worked on.
constexpr int kQ8Ring = 4, kQ8PassBytes = 1024;
constexpr float kQ8MinScale = 1.1754943508222875e-38f;  // 2^-126

enum CodeFormat : int { kE4m3 = 0, kInt8 = 1 };

struct AppendQ8Params {
  const uint16_t *q, *k, *v;        // q may be null
  uint16_t *q_out, *k_out;          // k_out may be null
  uint8_t *kc, *vc;
  float2* scales;                   // [page][head][row] of key, value
  // strides in units of 8 elements, of scales in pairs
  int q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  int kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs, s_ps, s_hs;
  const int32_t *table, *start, *cu, *positions;  // positions may be null
  int64_t table_bs, pos_ts, num_pages;
  const double* inv_freq;
  int T, B, Hq, Hkv, d;             // Hq = 0 without queries
  int max_pages;
  FastDiv page;
  int pairs, axes;                  // channel pairs per axis, axes (0: no rotation)
  int share;                        // log2 of the warps that share a token
  int row_lanes;                    // log2 of the lanes of a row, up to 16 channels each
};

// 16 bytes to shared memory.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Codes of 8 channels, 4 a word.
template <int kFmt>
__device__ __forceinline__ uint2 q8_codes(const float* x, float inv) {
  uint2 r;
  uint32_t* w = &r.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // (products of their own: fused with the sum below they would be rounded once only)
    const float a = __fmul_rn(x[4 * h], inv), b = __fmul_rn(x[4 * h + 1], inv);
    const float c = __fmul_rn(x[4 * h + 2], inv), e = __fmul_rn(x[4 * h + 3], inv);
    if constexpr (kFmt == kE4m3) {
      asm("{\n\t.reg .b16 lo, hi;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
          "mov.b32 %0, {lo, hi};\n\t}"
          : "=r"(w[h])
          : "f"(a), "f"(b), "f"(c), "f"(e));
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

// The largest magnitude, NaN if one of them is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
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
    // a byte with its sign bit flipped, planted into 2^23: 128 + 2^23 above its value
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + e)) - 8388736.f;
  }
}

// Row of a token in the caches, or nothing.
struct CachePlace {
  int page;  // -1: not there
  int row;
};
__device__ __forceinline__ CachePlace cache_place(int64_t place, const int32_t* table, int max_pages,
                                                  const FastDiv& page, int64_t num_pages) {
  CachePlace at{-1, 0};
  if (place >= 0 && place < static_cast<int64_t>(max_pages) * page.div) {
    // (a division of 64 bits costs a hundred instructions)
    const int pg = static_cast<int>(place < 0x7FFFFFFF ? fdiv(static_cast<uint32_t>(place), page)
                                                       : place / page.div);
    at.row = static_cast<int>(place - static_cast<int64_t>(pg) * page.div);
    const int id = __ldg(table + pg);
    if (id >= 0 && id < num_pages) at.page = id;
  }
  return at;
}

// x * stride in 64 bits, with strides in units of 8 elements (of 2 for scales).
__device__ __forceinline__ int64_t times(int x, int stride) {
  return static_cast<int64_t>(x) * stride;
}

// A lane's channels of a row: two vectors of 8 (cb < 0: one; ca = d: none), so that
// neighbouring lanes have neighbouring vectors.  Where channels i and pairs + i of an axis
// form a pair and 8 divides the pairs (kVec = 8), a lane of the rotated channels has 8
// pairs.  (With 16 neighbouring channels a lane, a warp's access would take half of each
// sector: 25825 prompt tokens with pairs side by side 146 us.)
struct Q8Place {
  int ca, cb, turn;  // turn: the first pair, < 0 behind the rotated channels
};
template <int kVec>
__device__ __forceinline__ Q8Place q8_place(int unit, const AppendQ8Params& p) {
  int first = 0;  // channel where the vectors start that have no partner
  if (kVec == 8) {
    const int per_axis = p.pairs >> 3, rot = p.axes * per_axis;
    if (unit < rot) {
      const int axis = unit >= per_axis ? 1 : 0, i0 = (unit - axis * per_axis) * 8;
      const int ca = 2 * axis * p.pairs + i0;
      return Q8Place{ca, ca + p.pairs, axis * p.pairs + i0};
    }
    first = 2 * p.axes * p.pairs;
    unit -= rot;
  }
  const int units = (p.d - first + 15) >> 4;
  Q8Place at{unit < units ? first + unit * 8 : p.d, first + (unit + units) * 8, -1};
  if (at.ca >= p.d || at.cb >= p.d) at.cb = -1;
  return at;
}

constexpr int kNeighbours = 16;

// A row takes 1 to 16 lanes with up to 16 channels each, and is reduced to its maximum
// between them; a pass takes the rows that fit the warp, of queries, keys or values.  A
// lane fetches its own channels ahead, into a place of its own, so that a row rotated in
// place is written behind its reads.  Partners of pairs that do not come in eights
// (kVec < 8) are read from the other lanes' places, in pieces of kVec channels.
template <bool kBf16, int kFmt, int kVec>
__global__ void __launch_bounds__(kQ8Warps * 32, kVec >= 8 ? 8 : 6)
kv_append_q8_kernel(const AppendQ8Params p) {
  constexpr int kPiece = kVec >= 8 ? 8 : kVec;
  using V = typename VecOf<kPiece>::T;
  constexpr float kTop = kFmt == kE4m3 ? 448.f : 127.f;
  extern __shared__ __align__(16) uint8_t app_smem[];  // rings, then [warp][axes * pairs] cos, sin
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kQ8Warps + warp;
  if ((gw >> p.share) >= p.T) return;
  const int t = static_cast<int>(gw >> p.share);
  const int part = static_cast<int>(gw) & ((1 << p.share) - 1);
  const int angles = p.axes * p.pairs, rotated = 2 * angles;
  uint8_t* const ring = app_smem + warp * (kQ8Ring * kQ8PassBytes);
  float2* const turn = reinterpret_cast<float2*>(app_smem + kQ8Warps * kQ8Ring * kQ8PassBytes) +
                       warp * ((angles + 7) & ~7);
  // Lanes with 8 pairs (or 4, in pieces and side by side) read them two at a time: those of
  // all lanes lie side by side, the first two, the next two and so on, so that eight lanes
  // meet no bank twice (25825 prompt tokens 95 us, 109 with the pairs in order).
  constexpr int kOf = kVec == 8 ? 8 : kVec >= 4 ? 4 : 2;
  const int groups = (angles + kOf - 1) / kOf;
  auto turn_at = [&](int a) {
    return kVec >= 4 ? (((a % kOf >> 1) * groups + a / kOf) << 1) + (a & 1) : a;
  };
  const int sub = lane >> p.row_lanes;                   // row of the pass
  const int unit = lane & ((1 << p.row_lanes) - 1);
  const Q8Place at = q8_place<kVec>(unit, p);
  const bool live = at.ca < p.d, both = at.cb >= 0;
  // passes: the queries', the keys', the values'
  const int rows_log = 5 - p.row_lanes, fill = (1 << rows_log) - 1;
  const int q_passes = (p.Hq + fill) >> rows_log, k_passes = (p.Hkv + fill) >> rows_log;
  const int passes = q_passes + 2 * k_passes, step = 1 << p.share;
  // The next pass to fetch, its kind's end, this lane's row of it, and where that is.
  // (Pointers move on along a kind: with every pass's kind looked at and its addresses made
  // anew, 80 instructions a pass more, 25825 prompt tokens took 122 us where they then took 114.)
  int f_pass = part, f_end = 0, f_row = 0, f_rows = 0;
  const uint16_t* f_src = nullptr;
  int64_t f_step = 0;
  const uint32_t mine = smem_u32(ring) + lane * 16;
  uint32_t f_to = mine;
  auto fetch = [&]() {
    if (f_pass < passes) {
      if (f_pass >= f_end) {  // on to the kind that this pass is of
        const bool is_q = f_pass < q_passes, is_k = !is_q && f_pass < q_passes + k_passes;
        const int begin = is_q ? 0 : is_k ? q_passes : q_passes + k_passes;
        const int hs = is_q ? p.q_hs : is_k ? p.k_hs : p.v_hs;
        f_end = begin + (is_q ? q_passes : k_passes);
        f_rows = is_q ? p.Hq : p.Hkv;
        f_row = ((f_pass - begin) << rows_log) + sub;
        f_src = (is_q ? p.q : is_k ? p.k : p.v) +
                8 * (times(t, is_q ? p.q_ts : is_k ? p.k_ts : p.v_ts) + times(f_row, hs)) + at.ca;
        f_step = 8 * times(step << rows_log, hs);
      }
      if (live && f_row < f_rows) {
        cp_async16(f_to, f_src);
        if (both) cp_async16(f_to + 512, f_src + (at.cb - at.ca));
      }
      f_pass += step;
      f_row += step << rows_log;
      f_src += f_step;
    }
    f_to = f_to == mine + (kQ8Ring - 1) * kQ8PassBytes ? mine : f_to + kQ8PassBytes;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kQ8Ring - 1; ++i) fetch();
  // ---- the token's sequence, cache row and angles
  const int b = find_sequence(p.cu, p.B, t, lane);
  if (b < 0 || b >= p.B) {
    cp_async_wait<0>();
    return;
  }
  const int64_t place = static_cast<int64_t>(__ldg(p.start + b)) + t - __ldg(p.cu + b);
  const CachePlace to =
      cache_place(place, p.table + b * p.table_bs, p.max_pages, p.page, p.num_pages);
  for (int a = lane; a < angles; a += 32) {
    const int axis = a >= p.pairs ? 1 : 0;
    const double pos = p.positions ? static_cast<double>(__ldg(p.positions + t * p.pos_ts + axis))
                                   : static_cast<double>(place);
    double turns = pos * __ldg(p.inv_freq + (a - axis * p.pairs)) * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * static_cast<float>(turns), &s, &c);
    turn[turn_at(a)] = make_float2(c, s);
  }
  int slot = 0, pass = part;
  auto walk = [&](auto kind) {
    constexpr bool is_q = decltype(kind)::value == 0, is_v = decltype(kind)::value == 2;
    const int begin = is_q ? 0 : is_v ? q_passes + k_passes : q_passes;
    const int end = begin + (is_q ? q_passes : k_passes), rows = is_q ? p.Hq : p.Hkv;
    if (pass >= end) return;
    int r = ((pass - begin) << rows_log) + sub;
    const int r_step = step << rows_log;
    // this lane's places in the 16-bit output, the codes and the scales
    uint16_t* out = is_q ? p.q_out + 8 * (times(t, p.qo_ts) + times(r, p.qo_hs))
                         : p.k_out + 8 * (times(t, p.ko_ts) + times(r, p.ko_hs));
    const bool with_out = is_q || (!is_v && p.k_out);
    const int ps = is_v ? p.vc_ps : p.kc_ps, ts = is_v ? p.vc_ts : p.kc_ts;
    uint8_t* codes = (is_v ? p.vc : p.kc) +
                     8 * (times(to.page, ps) + times(to.row, ts) + times(r, is_v ? p.vc_hs : p.kc_hs));
    float2* scales = p.scales + (times(to.page, p.s_ps) + to.row + times(r, p.s_hs));
    out += at.ca;
    codes += at.ca;
    const int apart = at.cb - at.ca;
#pragma unroll 1
    for (; pass < end; pass += step, r += r_step, out += 8 * times(r_step, is_q ? p.qo_hs : p.ko_hs),
                       codes += 8 * times(r_step, is_v ? p.vc_hs : p.kc_hs),
                       scales += times(r_step, p.s_hs)) {
      cp_async_wait<kQ8Ring - 2>();
      __syncwarp();  // others' channels and the angles are there, and the last pass's are read
      fetch();
      const bool here = live && r < rows, two = here && both;
      const uint8_t* const from = ring + slot * kQ8PassBytes;
      slot = slot + 1 == kQ8Ring ? 0 : slot + 1;
      uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
      if (here) x0 = *reinterpret_cast<const uint4*>(from + lane * 16);
      if (two) x1 = *reinterpret_cast<const uint4*>(from + 512 + lane * 16);
      float f[16];
      {
        const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 u = unpack2<kBf16>(w[e]);
          f[2 * e] = u.x, f[2 * e + 1] = u.y;
        }
      }
      if (!is_v && here) {
        if constexpr (kVec == kNeighbours) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = (e < 2 ? at.ca : at.cb) + 4 * (e & 1);
            if (c >= rotated || (e >= 2 && !both)) continue;
            const float4 z = reinterpret_cast<const float4*>(turn)[(e & 1) * groups + (c >> 3)];
            const float a0 = f[4 * e], b0 = f[4 * e + 1], a1 = f[4 * e + 2], b1 = f[4 * e + 3];
            f[4 * e] = a0 * z.x - b0 * z.y;
            f[4 * e + 1] = b0 * z.x + a0 * z.y;
            if (c + 2 < rotated) {
              f[4 * e + 2] = a1 * z.z - b1 * z.w;
              f[4 * e + 3] = b1 * z.z + a1 * z.w;
            }
          }
        } else if constexpr (kVec == 8) {
          if (at.turn >= 0) {
            const float4* cs = reinterpret_cast<const float4*>(turn) + (at.turn >> 3);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 z = cs[e * groups];
              const float a0 = f[2 * e], a1 = f[2 * e + 1], b0 = f[8 + 2 * e], b1 = f[9 + 2 * e];
              f[2 * e] = a0 * z.x - b0 * z.y;
              f[2 * e + 1] = a1 * z.z - b1 * z.w;
              f[8 + 2 * e] = b0 * z.x + a0 * z.y;
              f[9 + 2 * e] = b1 * z.z + a1 * z.w;
            }
          }
        } else {
          const uint8_t* row = from + (sub << p.row_lanes) * 16;
          const int units = (p.d + 15) >> 4;  // first vectors, and so lanes, of a row
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < 8 / kPiece; ++s) {
              const int c = (h ? at.cb : at.ca) + s * kPiece;
              if (c >= rotated || (h && !both)) break;
              const int axis = c >= 2 * p.pairs ? 1 : 0, in_axis = c - 2 * axis * p.pairs;
              const bool second = in_axis >= p.pairs;
              const int o = second ? c - p.pairs : c + p.pairs;  // the partners
              union { V v; uint16_t e[kPiece]; uint32_t w[(kPiece + 1) / 2]; } g;
              const int vec = o >> 3, second_vec = vec >= units;
              g.v = *reinterpret_cast<const V*>(row + second_vec * 512 +
                                                (vec - second_vec * units) * 16 + (o & 7) * 2);
              const int a = axis * p.pairs + (second ? in_axis - p.pairs : in_axis);
              float* y = f + 8 * h + s * kPiece;
              if constexpr (kPiece == 1) {
                const float2 z = turn[a];
                y[0] = y[0] * z.x + app_float<kBf16>(g.e[0]) * (second ? z.y : -z.y);
              } else {
                const float4* cs = reinterpret_cast<const float4*>(turn) + a / kOf;
#pragma unroll
                for (int e = 0; e < kPiece / 2; ++e) {
                  const float4 z = cs[e * groups];
                  const float2 u = unpack2<kBf16>(g.w[e]);
                  y[2 * e] = y[2 * e] * z.x + u.x * (second ? z.y : -z.y);
                  y[2 * e + 1] = y[2 * e + 1] * z.z + u.y * (second ? z.w : -z.w);
                }
              }
            }
        }
      }
      if (here && with_out) {
        *reinterpret_cast<uint4*>(out) =
            make_uint4(pack2<kBf16>(f[0], f[1]), pack2<kBf16>(f[2], f[3]),
                       pack2<kBf16>(f[4], f[5]), pack2<kBf16>(f[6], f[7]));
        if (two)
          *reinterpret_cast<uint4*>(out + apart) =
              make_uint4(pack2<kBf16>(f[8], f[9]), pack2<kBf16>(f[10], f[11]),
                         pack2<kBf16>(f[12], f[13]), pack2<kBf16>(f[14], f[15]));
      }
      if (is_q || to.page < 0) continue;
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max_abs(top, f[2 * e], f[2 * e + 1]);
      for (int o = 1; o < (1 << p.row_lanes); o <<= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float scale = top < -kNegInf ? fmaxf(__fdiv_rn(top, kTop), kQ8MinScale)
                                         : __uint_as_float(0x7FC00000u);
      const float inv = __frcp_rn(scale);
      if (here) *reinterpret_cast<uint2*>(codes) = q8_codes<kFmt>(f, inv);
      if (two) *reinterpret_cast<uint2*>(codes + apart) = q8_codes<kFmt>(f + 8, inv);
      if (here && unit == 0) reinterpret_cast<float*>(scales)[is_v ? 1 : 0] = scale;
    }
  };
  walk(std::integral_constant<int, 0>{});
  walk(std::integral_constant<int, 1>{});
  walk(std::integral_constant<int, 2>{});
  cp_async_wait<0>();
}

struct ReadQ8Params {
  const uint8_t *kc, *vc;
  const float2* scales;
  uint16_t *k, *v;
  // strides in units of 8 elements, of scales in pairs
  int kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs, s_ps, s_hs;
  int k_ts, k_hs, v_ts, v_hs;
  const int32_t *table, *start, *cu;  // start may be null
  int64_t table_bs, num_pages;
  int T, B, Hkv, d, max_pages;
  FastDiv page;
  int share;                        // log2 of the warps that share a token
  FastDiv by_row;                   // 8-channel units of a row
};

constexpr int kReadBatch = 4;

// One warp a token (for few tokens up to 8 share one); a unit is 8 channels of a head.
// Measured: 54012 tokens of 24 sequences, 8 heads of 128, e4m3 to bf16, 335 MB, 59 us (5.7
// TB/s, 0.87 of a copy's rate); four tokens a warp, looked up together, take as long, and
// so do 8 units in flight a lane in place of 4.  One short conversation (333 tokens): 3.4 us.
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
      cache_place(place, p.table + b * p.table_bs, p.max_pages, p.page, p.num_pages);
  const int page = at.page, row = at.row;
  const int row_units = p.by_row.div, units = p.Hkv * row_units;
  const int step = 32 << p.share;
  const float2* const sc = p.scales + times(page, p.s_ps) + row;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const uint8_t* const from =
        kind ? p.vc + 8 * (times(page, p.vc_ps) + times(row, p.vc_ts))
             : p.kc + 8 * (times(page, p.kc_ps) + times(row, p.kc_ts));
    uint16_t* const to = kind ? p.v + 8 * times(t, p.v_ts) : p.k + 8 * times(t, p.k_ts);
    const int from_hs = kind ? p.vc_hs : p.kc_hs, to_hs = kind ? p.v_hs : p.k_hs;
    for (int u0 = part * 32 + lane; u0 < units; u0 += kReadBatch * step) {
      uint2 w[kReadBatch];
      float s[kReadBatch];
      int h[kReadBatch], c[kReadBatch];  // head, and unit of its row
#pragma unroll
      for (int j = 0; j < kReadBatch; ++j) {
        const int u = u0 + j * step;
        if (u >= units) break;
        h[j] = fdiv(u, p.by_row), c[j] = u - h[j] * row_units;
        w[j] = make_uint2(0u, 0u);
        s[j] = 0.f;
        if (page >= 0) {
          w[j] = __ldg(reinterpret_cast<const uint2*>(from) + (times(h[j], from_hs) + c[j]));
          s[j] = __ldg(reinterpret_cast<const float*>(sc + times(h[j], p.s_hs)) + kind);
        }
      }
#pragma unroll
      for (int j = 0; j < kReadBatch; ++j) {
        if (u0 + j * step >= units) break;
        float a[4], e[4];
        q8_floats<kFmt>(w[j].x, a);
        q8_floats<kFmt>(w[j].y, e);
        reinterpret_cast<uint4*>(to)[times(h[j], to_hs) + c[j]] = make_uint4(
            pack2<kBf16>(a[0] * s[j], a[1] * s[j]), pack2<kBf16>(a[2] * s[j], a[3] * s[j]),
            pack2<kBf16>(e[0] * s[j], e[1] * s[j]), pack2<kBf16>(e[2] * s[j], e[3] * s[j]));
      }
    }
  }
}

}  // namespace rnn
