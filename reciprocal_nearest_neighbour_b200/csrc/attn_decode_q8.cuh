// attn_decode over a cache of 8-bit codes (kv_q8.cuh):
//   out = sum_t softmax_t(scale ks_t q.kc_t) vs_t vc_t
// with the codes kc_t, vc_t and scales ks_t, vs_t of cached row t.
//
// Bound by memory as attn_decode is, by half its bytes.  The split of the cache into
// tiles and of their list into the CTAs' shares, the four warps with a softmax state
// each, the ring of asynchronous copies, the parts and their join are attn_decode's; a
// tile has 4 x 32 keys here.  Codes stay codes on their way through shared memory and
// become fp16 in registers, exactly: e4m3 by the conversion instruction (two codes, 64
// lanes a cycle and SM), int8 by planting the byte into the mantissa of 1024 and taking
// 1152 off.  The matrix instruction adds its 16 depth steps in any order, so a lane reads
// 16 neighbouring codes of a key row and takes them as its share of four steps; the
// queries' fragments follow the same order.  The values' fragments pair neighbouring
// keys of one channel: the byte permutation that gathers the codes for the conversion
// also transposes them.
//
// Measured, in a CUDA graph with the join: 90 streams of 50 to 9000 keys, 32/8 heads of 128,
// e4m3, pages of 16, 0.32 GB, 65 us (4.9 TB/s; attn_decode takes 1.6 times as long over twice
// the bytes; 62 us with a head's rows of a page side by side); 4 streams of 80 001 to 131 000
// keys, 32/4 heads, int8, 0.44 GB, 80 us (5.4 TB/s, 0.83 of a copy's rate); the 90 streams
// with 32/2 heads (kNT = 2) 40 us (2.0 TB/s).  It is latency and issue that are left: about 720 instructions (e4m3, 830
// int8) a warp and tile, of which the conversions are 200 at half rate, with three warps a
// scheduler in 168 registers.  (Two CTAs per SM with three tiles a warp: 83 and 100 us, when
// the others took 71 and 97.)
//
// Range.  Queries are scaled by a power of two to below 2^15 for fp16, and their scores
// back together with ks_t, in fp32.  The second product's operand is the weight
// p_t vs_t with any size of vs_t, as fp16, which holds 2^-24 to 2^16.  So the running
// reference z of a head is that of score + log2 vs, not of the score: with p_t =
// 2^(score - z) the largest weight is put at 2^6 when z is chosen, and z is chosen again,
// the sums following, when a weight passes 2^15.  The totals sum p_t in fp32, which z
// keeps below 2^100, and whose least 2^-126 a value beyond about 2^100 would come near:
// z is no less than the largest score - 60.  Where that leaves the weights below 2^6
// (scales below 2^-54) they take a further factor 2^lift on their way into the product,
// which brings the largest to 2^5 at least; a pair's end, or what is held, takes it out
// again.  A power of two up to 2^72 (an append's scales are 2^-126 and more), it is exact
// in fp32 both ways.
#pragma once
#include <cstdint>
#include "attn_decode.cuh"
#include "attn_prompt.cuh"
#include "kv_q8.cuh"

namespace rnn {

constexpr int kQ8Keys = 32;  // keys per warp and tile, the lanes of a warp
// What a pair costs beside its tiles, in tiles.  90 streams of 50 to 9000 keys, 8 key
// heads: of 128 channels 86 us without it, 65 at 1, 66 at 2, 68 at 4; of 96 channels 91, 74,
// 78 and 82.
constexpr int kQ8PairCost = 1;
// Three CTAs per SM for up to 8 query heads a key head, with two tiles each a warp.
template <int kDP>
struct DecQ8Shape {
  static constexpr int kTile = kDecWarps * kQ8Keys;
  static constexpr int kStageBytes = 2 * kQ8Keys * kDP + kQ8Keys * 8;  // K, V, scales
  static constexpr int kStages = 256 / kDP;                            // 17 KB a warp
  static constexpr int kMergeRow = kDP + 4;                            // floats
  // a warp's sums of two times 8 heads take the place of the tile it has just used
  static_assert(2 * 8 * kMergeRow * 4 <= kStageBytes, "");
  static constexpr size_t kSmem = size_t(kDecWarps) * kStages * kStageBytes +
                                  kDecWarps * kDecRows * 8;
};

// 1 / x of a power of two between 2^-126 and 2^126.
__device__ __forceinline__ float inverse_pow2(float x) {
  return __uint_as_float(0x7F000000u - __float_as_uint(x));
}

// 8 bytes to shared memory; with `live` false they are zeroed and nothing is read.
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool live) {
  const int n = live ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// The two codes of a half word as fp16; kHigh: of the upper half.  int8 codes come with
// their sign bits flipped (q8_raw).
template <int kFmt>
__device__ __forceinline__ uint32_t q8_raw(uint32_t w) {
  return kFmt == kInt8 ? w ^ 0x80808080u : w;
}
template <int kFmt, bool kHigh>
__device__ __forceinline__ uint32_t q8_halves(uint32_t w) {
  uint32_t r;
  if constexpr (kFmt == kE4m3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(kHigh ? w >> 16 : w)));
  } else {
    const uint32_t m = __byte_perm(w, 0x64646464u, kHigh ? 0x4342 : 0x4140);  // 1024 + byte
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));      // 1024 + 128
  }
  return r;
}

template <bool kBf16, int kFmt, int kDP, int kNT, bool kLong>
__global__ void __launch_bounds__(kDecWarps * 32, kNT == 1 ? 3 : 2)
attn_decode_q8_kernel(const DecodeParams p) {
  using S = DecQ8Shape<kDP>;
  constexpr int kStages = S::kStages;
  constexpr int kMT = kQ8Keys / 16;      // 16-key groups
  constexpr int kSteps = kDP / 16;       // depth steps of K Q^T, channel pairs of V^T P^T
  constexpr int kChunks = kDP / 16;      // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks; // rows moved by one warp-wide copy
  constexpr int kLaneCh = kDP / 8;       // a lane's channels of a value row
  constexpr float kWeightTop = 32768.f, kTotalTop = 1.2676506e30f;  // 2^15, 2^100
  constexpr float kAim = 6.f, kTotalAim = 60.f, kMostLift = 80.f;    // log2
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* const tiles = dec_smem + warp * kStages * S::kStageBytes;
  const uint32_t ring = smem_u32(tiles);
  float2* ml = reinterpret_cast<float2*>(dec_smem + kDecWarps * kStages * S::kStageBytes);  // [warp][16]

  const int Hv = p.Hkv * p.hblocks;
  DecCursor ld, cur;
  int64_t hi, total, grid;
  if (!dec_begin<S::kTile, kQ8PairCost>(p, warp, lane, ld, hi, total, grid)) return;
  cur = ld;
  auto advance = [&](DecCursor& k) { dec_advance<S::kTile, kQ8PairCost>(p, Hv, k); };
  // Page of key `lane` of a tile, -1 where there is none.
  auto page_of = [&](const DecCursor& k) -> int {
    const int t = k.j * S::kTile + warp * kQ8Keys + lane;
    if (t >= k.len) return -1;
    const int id = __ldg(p.table + k.b * p.table_bs + fdiv(t, p.page));
    return (id >= 0 && id < p.num_pages) ? id : -1;
  };
  // Offsets of a row, from strides in units of 8 bytes.
  auto row_at = [](int page, int row, int hk, const int (&stride)[3]) {
    const int64_t units = static_cast<int64_t>(page) * stride[0] +
                          static_cast<int64_t>(row) * stride[1] + static_cast<int64_t>(hk) * stride[2];
    return units * 8;
  };
  // Where chunk ch of row r lies, so that eight lanes that read together (two key rows,
  // or two chunks of every second value row) meet no bank twice.
  auto k_at = [](int r, int ch) {
    return r * kDP + ((kDP == 128 ? ch ^ ((r & 1) << 2) : ch) << 4);
  };
  auto v_at = [](int r, int ch) {
    return r * kDP + ((kDP == 128 ? ch ^ (((r >> 1) & 3) << 1) : ch ^ (((r >> 2) & 1) << 1)) << 4);
  };
  const int ch = lane % kChunks, sub = lane / kChunks;
  const int ch_bytes = p.d - ch * 16;  // live bytes of this lane's chunk
  auto copy = [&](uint32_t dst, const uint8_t* src, const uint8_t* none, bool live) {
    if (p.wide) {
      live = live && ch_bytes > 0;
      cp_async16(dst, live ? src : none, live);
    } else {
      const bool a = live && ch_bytes > 0, b = live && ch_bytes > 8;
      cp_async8(dst, a ? src : none, a);
      cp_async8(dst + 8, b ? src + 8 : none, b);
    }
  };
  auto issue = [&](int stage, const DecCursor& k, int id) -> unsigned {
    const int t0 = k.j * S::kTile + warp * kQ8Keys;
    const int hk = p.hblocks == 1 ? k.h : k.h / p.hblocks;
    const unsigned valid = __ballot_sync(0xffffffffu, id >= 0);
    const uint32_t dst = ring + stage * S::kStageBytes, vdst = dst + kQ8Keys * kDP;
    const int t = t0 + lane;
    const int my_row = t - static_cast<int>(fdiv(t, p.page)) * static_cast<int>(p.page.div);
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(p.scales);
    if (id >= 0) sc += row_at(id, my_row, hk, p.s_s8);
    cp_async8(vdst + kQ8Keys * kDP + lane * 8, sc, id >= 0);
    if (p.page16) {
      // pages are whole 16-key groups: one base per group, no shuffles per row
      const bool all = p.wide && valid == 0xffffffffu && kChunks * 16 == p.d;
      const int64_t k_step = int64_t{kRowsPer * 8} * p.k_s8[1];
      const int64_t v_step = int64_t{kRowsPer * 8} * p.v_s8[1];
#pragma unroll
      for (int g = 0; g < kMT; ++g) {
        const int page = max(0, __shfl_sync(0xffffffffu, id, g * 16));
        const int row = __shfl_sync(0xffffffffu, my_row, g * 16) + sub;
        const uint8_t* ks = p.kc8 + row_at(page, row, hk, p.k_s8) + ch * 16;
        const uint8_t* vs = p.vc8 + row_at(page, row, hk, p.v_s8) + ch * 16;
        if (all) {
#pragma unroll
          for (int i = 0; i < 16 / kRowsPer; ++i) {
            const int r = g * 16 + i * kRowsPer + sub;
            cp_async16(dst + k_at(r, ch), ks);
            cp_async16(vdst + v_at(r, ch), vs);
            ks += k_step;
            vs += v_step;
          }
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16 / kRowsPer; ++i) {
          const int r = g * 16 + i * kRowsPer + sub;
          const bool live = (valid >> r) & 1u;
          copy(dst + k_at(r, ch), ks, p.kc8, live);
          copy(vdst + v_at(r, ch), vs, p.vc8, live);
          ks += k_step;
          vs += v_step;
        }
      }
      return valid;
    }
    const int64_t ko = row_at(id, my_row, hk, p.k_s8), vo = row_at(id, my_row, hk, p.v_s8);
#pragma unroll
    for (int i = 0; i < kQ8Keys / kRowsPer; ++i) {
      const int r = i * kRowsPer + sub;
      const int64_t k_off = __shfl_sync(0xffffffffu, ko, r);
      const int64_t v_off = __shfl_sync(0xffffffffu, vo, r);
      const bool live = (valid >> r) & 1u;
      copy(dst + k_at(r, ch), p.kc8 + k_off + ch * 16, p.kc8, live);
      copy(vdst + v_at(r, ch), p.vc8 + v_off + ch * 16, p.vc8, live);
    }
    return valid;
  };

  int fill = 0, stage = 0;  // ring places of the next load and of the current tile
  int next_id = page_of(ld);
  unsigned there[kStages];  // keys of the tiles in the ring, the current one's first
  auto issue_next = [&]() {
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) there[i] = there[i + 1];
    if (ld.at < hi) {
      const DecCursor now = ld;
      const int id = next_id;
      advance(ld);
      if (ld.at < hi) next_id = page_of(ld);  // the next tile's pages are looked up a tile ahead
      there[kStages - 1] = issue(fill, now, id);
    }
    fill = fill + 1 == kStages ? 0 : fill + 1;
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) issue_next();

  const int g = lane >> 2, q = lane & 3, q2 = q * 2;
  uint32_t qf[kNT][kSteps][2];
  float o[kNT][kSteps][4];   // channel kLaneCh g + 2 c (+ 1 in 2, 3), head 8 n + 2 q (+ 1 in 1, 3)
  float ch_scale[kNT][2];    // of those heads: scale * log2(e) / the queries' factor
  float z[kNT][2], l[kNT][2];
  float lift[kNT][2];        // the factor 2^lift of those heads' weights and sums
  constexpr int kSums = kNT * kSteps * 4, kHoldTiles = kDecHoldKeys / kQ8Keys;
  volatile float held[kSums + 4 * kNT];  // sums taken out, their totals and references
  bool any_held = false;
  int until = kHoldTiles;
  auto add_held = [&]() {
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = held[kSums + 2 * kNT + 2 * n + e];
        const float a = ref == kNegInf ? 0.f : exp2_approx(ref - z[n][e]);
        l[n][e] = fmaf(held[kSums + 2 * n + e], a, l[n][e]);
        const float up = a * lift[n][e];
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
#pragma unroll
          for (int h = e; h < 4; h += 2)
            o[n][c][h] = fmaf(held[(n * kSteps + c) * 4 + h], up, o[n][c][h]);
      }
  };
  bool fresh = true, lifted = false;  // lifted: one of the warp's factors is not 1
  bool whole = cur.j == 0;   // the pair started in this share
#pragma unroll 1
  while (cur.at < hi) {
    const int hk = p.hblocks == 1 ? cur.h : cur.h / p.hblocks, hb = cur.h - hk * p.hblocks;
    const int rows = min(kDecRows, p.group - hb * kDecRows);
    const int head0 = hk * p.group + hb * kDecRows;
    if (fresh) {  // under the wait for the first tile
      const uint16_t* qb = p.q + cur.b * p.q_bs;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const bool row_live = n * 8 + g < rows;
        const uint16_t* qr = qb + (head0 + (row_live ? n * 8 + g : 0)) * p.q_hs;
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const int c = (s >> 2) * 64 + 16 * q + (s & 3) * 4;
          const uint2 w = row_live && c < p.d ? *reinterpret_cast<const uint2*>(qr + c)
                                              : make_uint2(0u, 0u);
          qf[n][s][0] = w.x, qf[n][s][1] = w.y;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack2<kBf16>(qf[n][s][e]);
            top = max(top, max(__float_as_uint(x.x) & 0x7FFFFFFFu,
                               __float_as_uint(x.y) & 0x7FFFFFFFu));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest magnitude to [2^14, 2^15); below 2^-112 to what 2^126 makes of it
        const int k = min(126, 14 + 127 - static_cast<int>(top >> 23));
        const float to = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = unpack2<kBf16>(qf[n][s][e]);
            qf[n][s][e] = pack2<false>(x.x * to, x.y * to);
          }
        const float back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ch_scale[n][e] = __shfl_sync(0xffffffffu, back, (q2 + e) * 4) * p.c;
          z[n][e] = kNegInf;
          l[n][e] = 0.f;
          lift[n][e] = 1.f;
        }
        lifted = false;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][s][e] = 0.f;
      }
      fresh = false;
    }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue_next();
    const uint8_t* const kb = tiles + stage * S::kStageBytes;
    const uint8_t* const vb = kb + kQ8Keys * kDP;
    const float2* const sb = reinterpret_cast<const float2*>(vb + kQ8Keys * kDP);
    const unsigned valid = there[0];  // (after the next tile's issue the current one is first)
    if (valid) {
      float s[kMT][kNT][4];
      float vscale[kMT][2];
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][n][e] = 0.f;
        const int ra = t * 16 + g, rb = ra + 8;
#pragma unroll
        for (int hh = 0; hh < kDP / 64; ++hh) {
          const uint4 wa = *reinterpret_cast<const uint4*>(kb + k_at(ra, hh * 4 + q));
          const uint4 wb = *reinterpret_cast<const uint4*>(kb + k_at(rb, hh * 4 + q));
          const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, b[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const uint32_t x = q8_raw<kFmt>(a[st]), y = q8_raw<kFmt>(b[st]);
            const uint32_t frag[4] = {q8_halves<kFmt, false>(x), q8_halves<kFmt, false>(y),
                                      q8_halves<kFmt, true>(x), q8_halves<kFmt, true>(y)};
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              mma_16816<false>(s[t][n], frag, qf[n][hh * 4 + st][0],
                               qf[n][hh * 4 + st][1]);
          }
        }
        const float2 sa = sb[ra], sc = sb[rb];
        vscale[t][0] = sa.y, vscale[t][1] = sc.y;
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[t][n][e] *= sa.x * ch_scale[n][e];
            s[t][n][e + 2] *= sc.x * ch_scale[n][e];
          }
      }
      if (valid != 0xffffffffu) {
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((valid >> (t * 16 + g + (e >> 1) * 8)) & 1u))
#pragma unroll
              for (int n = 0; n < kNT; ++n) s[t][n][e] = kNegInf;
      }
      // ---- p = 2^(score - z), and the weights p vs 2^lift (in this order: vs 2^lift may
      // be infinite where p is 0)
      float pr[kMT][kNT][4], w[kMT][kNT][4];
      auto weigh = [&](int n, int e) {
        const float zz = z[n][e] == kNegInf ? 0.f : z[n][e];
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pr[t][n][e + 2 * h] = exp2_approx(s[t][n][e + 2 * h] - zz);
            w[t][n][e + 2 * h] = pr[t][n][e + 2 * h] * vscale[t][h];
          }
        if (lifted) {
#pragma unroll
          for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[t][n][e + 2 * h] *= lift[n][e];
        }
      };
      bool over = false;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          weigh(n, e);
          float tw = fmaxf(w[0][n][e], w[0][n][e + 2]), tp = fmaxf(pr[0][n][e], pr[0][n][e + 2]);
#pragma unroll
          for (int t = 1; t < kMT; ++t) {
            tw = fmax3(tw, w[t][n][e], w[t][n][e + 2]);
            tp = fmax3(tp, pr[t][n][e], pr[t][n][e + 2]);
          }
          over = over || tw > kWeightTop || tp > kTotalTop || z[n][e] == kNegInf;
        }
      // ---- the reference
      if (__any_sync(0xffffffffu, over)) {
        bool any = false;
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the reference, and where the largest weight so far and here would be at 2^6
            const int had = static_cast<int>(__float_as_uint(lift[n][e]) >> 23) - 127;
            float put = z[n][e] - had, y = z[n][e];
#pragma unroll
            for (int t = 0; t < kMT; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = s[t][n][e + 2 * h];
                put = fmaxf(put, x + (log2f(vscale[t][h]) - kAim));
                y = fmaxf(y, x - kTotalAim);
              }
#pragma unroll
            for (int h = 4; h < 32; h *= 2) {
              put = fmaxf(put, __shfl_xor_sync(0xffffffffu, put, h));
              y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, h));
            }
            y = fmaxf(y, put);
            const float a = z[n][e] == kNegInf ? 0.f : exp2_approx(z[n][e] - y);
            // (all scales so far 0: the most; no score so far: 2^0)
            const int up = y == kNegInf ? 0 : static_cast<int>(fminf(floorf(y - put), kMostLift));
            const float b = a * __uint_as_float(static_cast<uint32_t>(127 + up - had) << 23);
            lift[n][e] = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            any = any || up > 0;
            z[n][e] = y;
            l[n][e] *= a;
#pragma unroll
            for (int c = 0; c < kSteps; ++c) {
              o[n][c][e] *= b;
              o[n][c][e + 2] *= b;
            }
          }
        lifted = __any_sync(0xffffffffu, any);
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) weigh(n, e);
      }
      uint32_t pf[kMT][kNT][2];
#pragma unroll
      for (int t = 0; t < kMT; ++t)
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          l[n][0] += pr[t][n][0] + pr[t][n][2];
          l[n][1] += pr[t][n][1] + pr[t][n][3];
          // weights round to fp16 for the second product (half a step: 2^-12)
          pf[t][n][0] = movmatrix_t(pack2<false>(w[t][n][0], w[t][n][1]));
          pf[t][n][1] = movmatrix_t(pack2<false>(w[t][n][2], w[t][n][3]));
        }
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        const int r = t * 16 + q2;
        constexpr int kWords = kLaneCh / 4;
        uint32_t v4[4][kWords];  // rows r, r + 1, r + 8, r + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = r + (i & 1) + (i >> 1) * 8;
          if constexpr (kDP == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vb + v_at(row, g));
            v4[i][0] = v.x, v4[i][1] = v.y, v4[i][2] = v.z, v4[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vb + v_at(row, g >> 1) + (g & 1) * 8);
            v4[i][0] = v.x, v4[i][1] = v.y;
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // codes of channels 2 h, 2 h + 1 of a word, key by key
            const uint32_t x = q8_raw<kFmt>(__byte_perm(v4[0][j], v4[1][j], h ? 0x7362 : 0x5140));
            const uint32_t y = q8_raw<kFmt>(__byte_perm(v4[2][j], v4[3][j], h ? 0x7362 : 0x5140));
            const uint32_t frag[4] = {q8_halves<kFmt, false>(x), q8_halves<kFmt, true>(x),
                                      q8_halves<kFmt, false>(y), q8_halves<kFmt, true>(y)};
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              mma_16816<false>(o[n][2 * j + h], frag, pf[t][n][0], pf[t][n][1]);
          }
      }
    }
    const int used = stage;
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool last = cur.j == cur.n - 1;
    if (kLong && --until == 0) {
      if (any_held) add_held();
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          held[kSums + 2 * n + e] = l[n][e];
          held[kSums + 2 * kNT + 2 * n + e] = z[n][e];
          l[n][e] = 0.f;
          const float down = inverse_pow2(lift[n][e]);
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
#pragma unroll
            for (int h = e; h < 4; h += 2) {
              held[(n * kSteps + c) * 4 + h] = o[n][c][h] * down;
              o[n][c][h] = 0.f;
            }
        }
      any_held = true;
      until = kHoldTiles;
    }
    if (last || cur.at + 1 >= hi) {
      if (kLong) {
        if (any_held) add_held();
        any_held = false;
        until = kHoldTiles;
      }
      // ---- the pair ends here, or goes on in the next share
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = l[n][e];
          y += __shfl_xor_sync(0xffffffffu, y, 4);
          y += __shfl_xor_sync(0xffffffffu, y, 8);
          y += __shfl_xor_sync(0xffffffffu, y, 16);
          if (g == 0) ml[warp * kDecRows + n * 8 + q2 + e] = make_float2(z[n][e], y);
        }
      __syncthreads();
      const bool done = whole && last;
      // a pair that began in an earlier share fills slot 0, one that goes on slot 1
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (whole ? 1 : 0);
      // the warps' sums, at the pair's reference, in the places of the tiles they used
      float* const mine = reinterpret_cast<float*>(tiles + used * S::kStageBytes);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if (n * 8 >= rows) break;
        float r[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = kNegInf;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * kDecRows + n * 8 + q2 + e].x);
          r[e] = z[n][e] == kNegInf ? 0.f : exp2_approx(z[n][e] - M) * inverse_pow2(lift[n][e]);
        }
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(mine + (n * 8 + q2 + e) * S::kMergeRow + kLaneCh * g + 2 * c) =
                make_float2(o[n][c][e] * r[e], o[n][c][e + 2] * r[e]);
      }
      __syncthreads();
      {
        const int used_all = used * S::kStageBytes;  // (the same in every warp)
        for (int row = warp; row < rows; row += kDecWarps) {
          float M = kNegInf, L = 0.f;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * kDecRows + row].x);
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float2 a = ml[w * kDecRows + row];
            // without a reference the total is 0, or NaN if its scores were
            L += a.x == kNegInf ? a.y : a.y * exp2_approx(a.x - M);
          }
          const float inv = L != 0.f ? 1.f / L : 0.f;
          for (int c = lane * 2; c < kDP; c += 64) {
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
              const float2 a = *reinterpret_cast<const float2*>(
                  dec_smem + w * kStages * S::kStageBytes + used_all + (row * S::kMergeRow + c) * 4);
              sum.x += a.x, sum.y += a.y;
            }
            if (!done)
              *reinterpret_cast<float2*>(p.part + (slot * kDecRows + row) * kDP + c) = sum;
            else if (c < p.d)
              *reinterpret_cast<uint32_t*>(p.out + cur.b * p.o_bs + (head0 + row) * p.o_hs + c) =
                  pack2<kBf16>(sum.x * inv, sum.y * inv);
          }
          if (lane == 0) {
            if (!done)
              p.part_ml[slot * kDecRows + row] = make_float2(M, L);
            else if (p.lse)
              p.lse[static_cast<int64_t>(cur.b) * p.Hq + head0 + row] =
                  L != 0.f ? (M + log2f(L)) * 0.69314718f : kNegInf;
          }
        }
      }
      if (whole && threadIdx.x == 0) {
        int c1 = blockIdx.x;
        if (!last) c1 = dec_owner(cur.at + (cur.n - 1 - cur.j), total, grid);
        p.span[static_cast<int64_t>(cur.b) * Hv + cur.h] = make_int2(blockIdx.x, c1);
      }
      __syncthreads();  // the next pair's totals and sums come behind these reads
      fresh = true;
      whole = true;
    }
    advance(cur);
  }
  cp_async_wait<0>();
}

}  // namespace rnn
