// Attention of one new token per sequence over a paged key-value cache:
//   out = sum_t softmax_t(scale q.k_t) v_t,  lse = log sum_t exp(scale q.k_t)
// for each query head, over the lens[b] cached rows of its sequence.
//
// Bound by memory: each cached row is read once for all the query heads that
// share it (up to 16; more heads read the rows again), and 2 x 16 x d
// multiply-adds a row are far below what the warp-level matrix path delivers,
// so tcgen05 would gain nothing at 8 or 16 rows and cost a tensor-memory round
// trip per tile.  Keys are the 16 rows of the matrix instruction and the query
// heads its 8 columns (S^T = K Q^T, then O^T += V^T P^T): with the heads as
// rows, half of each instruction would be padding for up to 8 heads.
//
// Split.  The cache is cut into tiles of 4 x kKeys keys; the tiles of all
// (sequence, key head) pairs form one list, which the CTAs (two per SM) cut
// into equal contiguous shares, whatever the lengths.  A pair that lies in
// one share is finished there; the others leave unnormalised fp32 parts with
// their running maximum and total in the workspace, and a second kernel joins
// them in a fixed order.  Each of the four warps loads and reduces its own
// kKeys keys of a tile with its own softmax state, so the loop has no block
// barrier; the warps meet once per pair.  The loads run kStages - 1 tiles
// ahead, over the ends of pairs.
//
// The reference maximum of a head moves only when a score exceeds it by more
// than 2^8 (its weights then reach 2^8, and 2^15 of fp16's 2^16 with that type's
// factor of 2^7): one vote per tile instead of a reduction across the warp.
//
// Measured (bf16, 128 channels): 4 streams of 90 001 to 131 000 keys, 32/4 heads,
// 0.96 GB, 148 us (6.5 TB/s, 0.99 of a copy's rate); 96 streams of 50 to 8000 keys,
// 32/8 heads, pages of 16, 0.66 GB, 107 us (6.1 TB/s).  64 streams of 2000 to 4000
// keys with 16 heads of 64 that share nothing, 0.75 GB: 139 us (5.4 TB/s).
#pragma once
#include <cstdint>
#include <type_traits>
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kDecWarps = 4;
constexpr int kDecRows = 16;    // query heads per unit
constexpr int kDecMaxKeys = 0x7fffffff - 1023;  // whole tiles stay below 2^31
// Keys that meet in one accumulator.  A warp takes a quarter of a pair's keys at most.
constexpr int kDecHoldKeys = 65536, kDecShortKeys = 4 * kDecHoldKeys;

// kDP: channels padded to 64 or 128.  kKeys: keys per warp and tile, 8 KB of
// keys and values in either case.
template <int kDP>
struct DecShape {
  static constexpr int kKeys = 2048 / kDP;
  static constexpr int kTile = kDecWarps * kKeys;
  static constexpr int kRowBytes = kDP * 2;
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // per warp, K then V
  static constexpr int kStages = 3;
  static constexpr int kMergeRow = kDP + 4;                  // floats; 4 against bank conflicts
  static constexpr int kMergeBytes = 2 * 8 * kMergeRow * 4;  // of two warps, 8 heads
  static constexpr size_t kSmem = size_t(kDecWarps) * kStages * kStageBytes + kMergeBytes +
                                  kDecWarps * kDecRows * 8 + kDecWarps * kStages * 4;
};
// What a pair costs beside its tiles (its queries' latency, the warps' merge),
// in tiles, counted when the list is cut into shares.  96 streams of 50 to 8000
// keys, 8 key heads of 128: 145 us without it, 108 at 2, 109 at 4, 114 at 8;
// even lengths change by 1 %.
constexpr int kDecPairCost = 2;
constexpr float kDecSlack = 8.f;  // log2 growth of the maximum before a rescale
// Scaled log2 scores beyond this lose their exponents' last bits (a sixteenth and more)
// where the reference is taken off behind the scaling, and at 2^128 all of it; it is
// taken off before for such heads.
constexpr float kDecFar = 1048576.f;

struct DecodeParams {
  const uint16_t *q, *kc, *vc;
  uint16_t* out;
  float* lse;                      // [B][Hq] or null
  int64_t q_bs, q_hs, o_bs, o_hs;  // strides in elements
  int64_t k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;
  const int32_t *table, *lens;
  int64_t table_bs, num_pages;
  int B, Hq, Hkv, group, hblocks;  // group: query heads per key head; hblocks = ceil(group/16)
  int d, max_pages;
  int page16;                      // page_size is a multiple of 16
  FastDiv page;
  float scale, c;                  // c = scale * log2(e)
  float* part;                     // [grid][2][16][kDP] unnormalised parts
  float2* part_ml;                 // [grid][2][16] maximum, total
  int* err;                        // status word, cleared: no wait here can run out
  int2* span;                      // [B][Hkv * hblocks] first and last CTA of a pair
};

__device__ __forceinline__ int dec_len(const DecodeParams& p, int b) {
  int64_t room = static_cast<int64_t>(p.max_pages) * p.page.div;
  if (room > kDecMaxKeys) room = kDecMaxKeys;
  const int64_t n = __ldg(p.lens + b);
  return static_cast<int>(n < 0 ? 0 : (n < room ? n : room));
}
// places of a sequence's pairs in the list: per pair its cost, then its tiles
template <int kTile>
__device__ __forceinline__ int64_t dec_places(const DecodeParams& p, int b) {
  const int n = dec_len(p, b);
  return n > 0 ? (n + kTile - 1) / kTile + kDecPairCost : 0;
}
__device__ __forceinline__ int64_t dec_share(int64_t c, int64_t total, int64_t grid) {
  return c * total / grid;
}
// the CTA whose share holds place w
__device__ __forceinline__ int dec_owner(int64_t w, int64_t total, int64_t grid) {
  int64_t c = w * grid / total;
  while (c + 1 < grid && dec_share(c + 1, total, grid) <= w) ++c;
  while (c > 0 && dec_share(c, total, grid) > w) --c;
  return static_cast<int>(c);
}

// kLong: page tables with room for more than kDecShortKeys keys.  The matrix instruction
// cuts what it adds off at the accumulator's last bits instead of rounding it, so a sum
// of n weights of one size loses about n 2^-27 (65536 keys: less than 2^-11, half a step
// of fp16; 2^22 in one warp: 2.7 %).  There a warp takes its sums out of the accumulator
// every kDecHoldKeys keys and adds them up itself, rounded to nearest, in local memory.
template <bool kBf16, int kDP, int kNT, bool kLong>
__global__ void __launch_bounds__(kDecWarps * 32, 2) attn_decode_kernel(const DecodeParams p) {
  using S = DecShape<kDP>;
  constexpr int kKeys = S::kKeys, kStages = S::kStages;
  constexpr int kMT = kKeys / 16;        // 16-key groups
  constexpr int kSteps = kDP / 16;       // depth steps of K Q^T, channel groups of V^T P^T
  constexpr int kChunks = kDP / 8;       // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks; // rows moved by one warp-wide copy
  // fp16 keeps a probability down to 2^-24 only: scaled by 2^7 at the reference
  // (2^15 with the slack), many small ones do not vanish from the weighted sum
  // while the fp32 total keeps them
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  // with 0.6 for the exponent's rounding up to kDecFar
  static_assert(kBias + kDecSlack + 0.6f < 15.99f, "weights have to stay inside fp16");
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(dec_smem) + warp * kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(dec_smem + kDecWarps * kStages * S::kStageBytes);
  float2* ml = reinterpret_cast<float2*>(merge + 2 * 8 * S::kMergeRow);  // [warp][16]
  uint32_t* masks = reinterpret_cast<uint32_t*>(ml + kDecWarps * kDecRows) + warp * kStages;

  const int Hv = p.Hkv * p.hblocks;
  // ---- this CTA's share of the tile list, and the pair it starts in
  __shared__ int64_t scan[kDecWarps];
  __shared__ int64_t sh_before;
  __shared__ int sh_b;
  const int per = (p.B + kDecWarps * 32 - 1) / (kDecWarps * 32);
  const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += dec_places<S::kTile>(p, b);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  if (threadIdx.x == 0) sh_b = p.B;
  __syncthreads();
  int64_t before = incl - mine, places = 0;
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += scan[w];
    places += scan[w];
  }
  const int64_t total = places * Hv;
  // CTAs with a share: no more than places, so that none inside a pair's span is empty
  const int64_t grid = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= grid) return;
  const int64_t lo = dec_share(blockIdx.x, total, grid);
  const int64_t hi = dec_share(blockIdx.x + 1, total, grid);
  if (lo >= before * Hv && lo < (before + mine) * Hv) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const int64_t n = dec_places<S::kTile>(p, b);
      if (lo < (at + n) * Hv) {
        sh_b = b;
        sh_before = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  struct Cursor {
    int b, h, j, n, len;  // sequence, head unit, tile, tiles, keys
    int64_t at;           // place of the tile in the list
  } ld, cur;
  ld.b = sh_b;
  ld.len = dec_len(p, ld.b);
  ld.n = (ld.len + S::kTile - 1) / S::kTile;
  {
    // the share's first place is a tile, or stands for its pair's cost
    const int64_t r = lo - sh_before * Hv, per_pair = ld.n + kDecPairCost;
    ld.h = static_cast<int>(r / per_pair);
    ld.j = max(0, static_cast<int>(r - ld.h * per_pair) - kDecPairCost);
    ld.at = sh_before * Hv + ld.h * per_pair + kDecPairCost + ld.j;
  }
  cur = ld;
  auto advance = [&](Cursor& k) {
    ++k.at;
    if (++k.j < k.n) return;
    k.j = 0;
    k.at += kDecPairCost;
    if (++k.h < Hv) return;
    k.h = 0;
    do {
      if (++k.b >= p.B) return;
      k.len = dec_len(p, k.b);
      k.n = (k.len + S::kTile - 1) / S::kTile;
    } while (k.n == 0);
  };
  // Page of key (lane % kKeys) of a tile, -1 where there is none.
  const int my_row = lane & (kKeys - 1);
  auto page_of = [&](const Cursor& k) -> int {
    const int t = k.j * S::kTile + warp * kKeys + my_row;
    if (t >= k.len) return -1;
    const int id = __ldg(p.table + k.b * p.table_bs + fdiv(t, p.page));
    return (id >= 0 && id < p.num_pages) ? id : -1;
  };
  const int ch = lane % kChunks, sub = lane / kChunks;
  const bool ch_live = ch * 8 < p.d;
  auto issue = [&](int stage, const Cursor& k, int id) {
    const int t0 = k.j * S::kTile + warp * kKeys;
    const int hk = p.hblocks == 1 ? k.h : k.h / p.hblocks;
    const unsigned valid = __ballot_sync(0xffffffffu, id >= 0) &
                           static_cast<unsigned>((1ull << kKeys) - 1u);
    if (lane == 0) masks[stage] = valid;
    const uint32_t dst = ring + stage * S::kStageBytes;
    if (p.page16) {
      // pages are whole 16-key groups: one base per group, no shuffles per row
#pragma unroll
      for (int g = 0; g < kMT; ++g) {
        const int64_t page = max(0, __shfl_sync(0xffffffffu, id, g * 16));
        const int t = t0 + g * 16;
        const int row = t - static_cast<int>(fdiv(t, p.page)) * static_cast<int>(p.page.div) + sub;
        const uint16_t* ks = p.kc + (page * p.k_ps + hk * p.k_hs + row * p.k_ts + ch * 8);
        const uint16_t* vs = p.vc + (page * p.v_ps + hk * p.v_hs + row * p.v_ts + ch * 8);
#pragma unroll
        for (int i = 0; i < 16 / kRowsPer; ++i) {
          const int r = g * 16 + i * kRowsPer + sub;
          const bool live = ((valid >> r) & 1u) && ch_live;
          const uint32_t at = dst + r * S::kRowBytes + ((ch ^ (r & 7)) << 4);
          cp_async16(at, live ? ks : p.kc, live);
          cp_async16(at + kKeys * S::kRowBytes, live ? vs : p.vc, live);
          ks += kRowsPer * p.k_ts;
          vs += kRowsPer * p.v_ts;
        }
      }
      return;
    }
    const int t = t0 + my_row;
    const int row = t - static_cast<int>(fdiv(t, p.page)) * static_cast<int>(p.page.div);
    const int64_t ko = id * p.k_ps + row * p.k_ts + hk * p.k_hs;
    const int64_t vo = id * p.v_ps + row * p.v_ts + hk * p.v_hs;
#pragma unroll
    for (int i = 0; i < kKeys / kRowsPer; ++i) {
      const int r = i * kRowsPer + sub;
      const int64_t k_at = __shfl_sync(0xffffffffu, ko, r);
      const int64_t v_at = __shfl_sync(0xffffffffu, vo, r);
      const bool live = ((valid >> r) & 1u) && ch_live;
      const uint32_t at = dst + r * S::kRowBytes + ((ch ^ (r & 7)) << 4);
      cp_async16(at, live ? p.kc + k_at + ch * 8 : p.kc, live);
      cp_async16(at + kKeys * S::kRowBytes, live ? p.vc + v_at + ch * 8 : p.vc, live);
    }
  };

  int fill = 0, stage = 0;  // ring places of the next load and of the current tile
  int next_id = page_of(ld);
  auto issue_next = [&]() {
    if (ld.at < hi) {
      const Cursor now = ld;
      const int id = next_id;
      advance(ld);
      if (ld.at < hi) next_id = page_of(ld);  // the next tile's pages are looked up a tile ahead
      issue(fill, now, id);
    }
    fill = fill + 1 == kStages ? 0 : fill + 1;
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) issue_next();

  uint32_t qf[kNT][kSteps][2];
  float o[kNT][kSteps][4];   // channel 16 c + lane/4 (+ 8), head 8 n + 2 (lane%4) (+ 1)
  float m[kNT][2], l[kNT][2];
  const int g = lane >> 2, q2 = (lane & 3) * 2;
  // sums taken out so far, then their totals and reference maxima; tiles until the next
  constexpr int kSums = kNT * kSteps * 4, kHoldTiles = kDecHoldKeys / kKeys;
  volatile float held[kSums + 4 * kNT];
  bool any_held = false;
  int until = kHoldTiles;
  // m, l and o with what is held added to them
  auto add_held = [&]() {
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = held[kSums + 2 * kNT + 2 * n + e];
        const float f = ref == kNegInf ? 0.f : exp2_approx((ref - m[n][e]) * p.c);
        l[n][e] = fmaf(held[kSums + 2 * n + e], f, l[n][e]);
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
#pragma unroll
          for (int h = e; h < 4; h += 2)
            o[n][c][h] = fmaf(held[(n * kSteps + c) * 4 + h], f, o[n][c][h]);
      }
  };
  auto far = [&](float ref) { return fabsf(ref * p.c) > kDecFar && fabsf(ref) < -kNegInf; };
  bool fresh = true;
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
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = s * 16 + q2 + e * 8;
            qf[n][s][e] = row_live && c < p.d ? *reinterpret_cast<const uint32_t*>(qr + c) : 0u;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][s][e] = 0.f;
        }
        m[n][0] = m[n][1] = kNegInf;
        l[n][0] = l[n][1] = 0.f;
      }
      fresh = false;
    }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue_next();
    const uint32_t kb = ring + stage * S::kStageBytes, vb = kb + kKeys * S::kRowBytes;
    const uint32_t valid = masks[stage];
    if (valid) {
      float s[kMT][kNT][4];
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        // two chains of products per score tile, added at the end
        float s1[kNT][4];
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][n][e] = s1[n][e] = 0.f;
        const int r = t * 16 + (lane & 15), half = lane >> 4;
        const uint32_t rb = kb + r * S::kRowBytes;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          uint32_t f[4];
          ldsm_x4(rb + (((2 * st + half) ^ (r & 7)) << 4), f);
#pragma unroll
          for (int n = 0; n < kNT; ++n)
            mma_16816<kBf16>(st & 1 ? s1[n] : s[t][n], f, qf[n][st][0], qf[n][st][1]);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[t][n][e] += s1[n][e];
      }
      if (valid != static_cast<unsigned>((1ull << kKeys) - 1u)) {
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((valid >> (t * 16 + g + (e >> 1) * 8)) & 1u))
#pragma unroll
              for (int n = 0; n < kNT; ++n) s[t][n][e] = kNegInf;
      }
      float x[kNT][2];
      bool up = false;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
          for (int t = 1; t < kMT; ++t) x[n][e] = fmax3(x[n][e], s[t][n][e], s[t][n][e + 2]);
          up = up || (x[n][e] - m[n][e]) * p.c > kDecSlack  // also from -inf to a number
               || fabsf(m[n][e] * p.c) > kDecFar;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y = x[n][e];
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
            y = fmaxf(y, m[n][e]);
            const float a = m[n][e] == kNegInf ? 0.f : exp2_approx((m[n][e] - y) * p.c);
            m[n][e] = y;
            l[n][e] *= a;
#pragma unroll
            for (int c = 0; c < kSteps; ++c) {
              o[n][c][e] *= a;
              o[n][c][e + 2] *= a;
            }
            const float ref = far(y) ? y : 0.f;
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
              s[t][n][e] -= ref;
              s[t][n][e + 2] -= ref;
            }
          }
      }
      uint32_t pf[kMT][kNT][2];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float z0 = (m[n][0] == kNegInf || far(m[n][0]) ? 0.f : m[n][0] * p.c) - kBias;
        const float z1 = (m[n][1] == kNegInf || far(m[n][1]) ? 0.f : m[n][1] * p.c) - kBias;
#pragma unroll
        for (int t = 0; t < kMT; ++t) {
          const float e0 = exp2_approx(fmaf(s[t][n][0], p.c, -z0));
          const float e1 = exp2_approx(fmaf(s[t][n][1], p.c, -z1));
          const float e2 = exp2_approx(fmaf(s[t][n][2], p.c, -z0));
          const float e3 = exp2_approx(fmaf(s[t][n][3], p.c, -z1));
          l[n][0] += e0 + e2;
          l[n][1] += e1 + e3;
          // probabilities round to the value type for the second product; the
          // totals above keep them in fp32
          pf[t][n][0] = movmatrix_t(pack2<kBf16>(e0, e1));
          pf[t][n][1] = movmatrix_t(pack2<kBf16>(e2, e3));
        }
      }
#pragma unroll
      for (int t = 0; t < kMT; ++t) {
        const int r = t * 16 + (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
        const uint32_t rb = vb + r * S::kRowBytes;
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          uint32_t f[4];
          ldsm_x4_t(rb + (((2 * c + half) ^ (r & 7)) << 4), f);
#pragma unroll
          for (int n = 0; n < kNT; ++n) mma_16816<kBf16>(o[n][c], f, pf[t][n][0], pf[t][n][1]);
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool last = cur.j == cur.n - 1;
    if (kLong && --until == 0) {
      if (any_held) add_held();
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          held[kSums + 2 * n + e] = l[n][e];
          held[kSums + 2 * kNT + 2 * n + e] = m[n][e];
          l[n][e] = 0.f;
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
#pragma unroll
            for (int h = e; h < 4; h += 2) {
              held[(n * kSteps + c) * 4 + h] = o[n][c][h];
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
          if (g == 0) ml[warp * kDecRows + n * 8 + q2 + e] = make_float2(m[n][e], y);
        }
      __syncthreads();
      const bool done = whole && last;
      // a pair that began in an earlier share fills slot 0, one that goes on slot 1
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (whole ? 1 : 0);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if (n * 8 >= rows) break;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = kNegInf;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * kDecRows + n * 8 + q2 + e].x);
          f[e] = m[n][e] == kNegInf ? 0.f : exp2_approx((m[n][e] - M) * p.c);
        }
        float* buf = merge + (warp & 1) * 8 * S::kMergeRow;
        auto put = [&]() {
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              buf[(q2 + (e & 1)) * S::kMergeRow + c * 16 + g + (e >> 1) * 8] =
                  o[n][c][e] * f[e & 1];
        };
        auto add = [&]() {
#pragma unroll
          for (int c = 0; c < kSteps; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& at = buf[(q2 + (e & 1)) * S::kMergeRow + c * 16 + g + (e >> 1) * 8];
              at = fmaf(o[n][c][e], f[e & 1], at);
            }
        };
        if (warp >= 2) put();      // warps 2 and 3, then 0 and 1 on top
        __syncthreads();
        if (warp < 2) add();
        __syncthreads();
        for (int r = warp; r < 8 && n * 8 + r < rows; r += kDecWarps) {
          const int row = n * 8 + r;
          float M = kNegInf, L = 0.f;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * kDecRows + row].x);
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float2 a = ml[w * kDecRows + row];
            // without a reference the total is 0, or NaN if its scores were
            L += a.x == kNegInf ? a.y : a.y * exp2_approx((a.x - M) * p.c);
          }
          const float inv = L != 0.f ? 1.f / L : 0.f;
          const float* b0 = merge + r * S::kMergeRow;
          const float* b1 = b0 + 8 * S::kMergeRow;
          if (done) {
            uint16_t* ob = p.out + cur.b * p.o_bs + (head0 + row) * p.o_hs;
            for (int c = lane * 2; c < p.d; c += 64)
              *reinterpret_cast<uint32_t*>(ob + c) =
                  pack2<kBf16>((b0[c] + b1[c]) * inv, (b0[c + 1] + b1[c + 1]) * inv);
            if (p.lse && lane == 0)
              p.lse[static_cast<int64_t>(cur.b) * p.Hq + head0 + row] =
                  L != 0.f ? M * p.scale + (log2f(L) - kBias) * 0.69314718f : kNegInf;
          } else {
            float* pb = p.part + (slot * kDecRows + row) * kDP;
            for (int c = lane * 2; c < kDP; c += 64)
              *reinterpret_cast<float2*>(pb + c) =
                  make_float2(b0[c] + b1[c], b0[c + 1] + b1[c + 1]);
            if (lane == 0) p.part_ml[slot * kDecRows + row] = make_float2(M, L);
          }
        }
        if (n + 1 < kNT) __syncthreads();  // the next heads reuse the buffer
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

// Joins the parts of the pairs that several CTAs shared, and writes the rows
// of sequences without a key.  One block per (sequence, query head); its four
// warps take the parts in turn and their sums meet in a fixed order.
template <bool kBf16, int kDP>
__global__ void __launch_bounds__(128) attn_decode_join_kernel(const DecodeParams p) {
  constexpr int kVals = kDP / 32;  // channels per lane
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  using VecT = std::conditional_t<kVals == 4, float4, float2>;
  __shared__ float acc[4][kDP];
  __shared__ float2 tot[4];
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;
  const int b = blockIdx.x / p.Hq, head = blockIdx.x - b * p.Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t* ob = p.out + b * p.o_bs + head * p.o_hs;
  if (dec_len(p, b) == 0) {
    for (int c = threadIdx.x; c < p.d; c += blockDim.x) ob[c] = 0;
    if (p.lse && threadIdx.x == 0) p.lse[static_cast<int64_t>(b) * p.Hq + head] = kNegInf;
    return;
  }
  const int hk = head / p.group, in = head - hk * p.group;
  const int hb = in / kDecRows, row = in - hb * kDecRows;
  const int2 sp = p.span[static_cast<int64_t>(b) * (p.Hkv * p.hblocks) + hk * p.hblocks + hb];
  if (sp.x == sp.y) return;
  // each warp reduces its parts with a running maximum (no pass for the maximum
  // first: a part's totals and sums are fetched together), then the four meet
  float v[kVals] = {}, M = kNegInf, L = 0.f;
#pragma unroll 4
  for (int c = sp.x + warp; c <= sp.y; c += 4) {
    const int64_t at = (static_cast<int64_t>(c) * 2 + (c == sp.x ? 1 : 0)) * kDecRows + row;
    const float2 a = p.part_ml[at];
    const VecT x = *reinterpret_cast<const VecT*>(p.part + at * kDP + lane * kVals);
    const float* xs = reinterpret_cast<const float*>(&x);
    const float top = fmaxf(M, a.x);
    const float f = a.x == kNegInf ? 0.f : exp2_approx((a.x - top) * p.c);
    const float h = M == kNegInf ? 0.f : exp2_approx((M - top) * p.c);
    M = top;
    L = L * h + a.y * f;
#pragma unroll
    for (int e = 0; e < kVals; ++e) v[e] = v[e] * h + xs[e] * f;
  }
#pragma unroll
  for (int e = 0; e < kVals; ++e) acc[warp][lane * kVals + e] = v[e];
  if (lane == 0) tot[warp] = make_float2(M, L);
  __syncthreads();
  M = fmaxf(fmaxf(tot[0].x, tot[1].x), fmaxf(tot[2].x, tot[3].x));
  float f[4];
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = tot[w].x == kNegInf ? 0.f : exp2_approx((tot[w].x - M) * p.c);
    L += tot[w].y * f[w];
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
    const float x =
        ((acc[0][c] * f[0] + acc[1][c] * f[1]) + (acc[2][c] * f[2] + acc[3][c] * f[3])) * inv;
    ob[c] = kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                  : __half_as_ushort(__float2half_rn(x));
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[static_cast<int64_t>(b) * p.Hq + head] =
        L != 0.f ? M * p.scale + (log2f(L) - kBias) * 0.69314718f : kNegInf;
}

}  // namespace rnn
