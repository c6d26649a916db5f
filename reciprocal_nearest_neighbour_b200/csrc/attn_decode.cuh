// Attention of one new token per sequence over a paged key-value cache:
//   out = sum_t softmax_t(scale q.k_t) v_t,  lse = log sum_t exp(scale q.k_t)
// for each query head, over the lens[b] cached rows of its sequence.
//
// Bound by memory: each cached row is read once for all the query heads that
// share it (up to 16, the rows of one warp-level matrix instruction; more
// heads read the rows again), and 2 x 16 x d multiply-adds a row are far
// below what the legacy matrix path delivers, so tcgen05 would gain nothing
// at 16 rows and cost a tensor-memory round trip per tile.
//
// Split.  The cache is cut into tiles of 4 x kKeys keys; the tiles of all
// (sequence, key head) pairs form one list, which the CTAs (two per SM) cut
// into equal contiguous shares, whatever the lengths.  A pair that lies in
// one share is finished there; the others leave unnormalised fp32 parts with
// their running maximum and total in the workspace, and a second kernel joins
// them in a fixed order.  Each of the four warps loads and reduces its own
// kKeys keys of a tile with its own softmax state, so the loop has no block
// barrier; the warps meet once per pair.  The loads run kStages tiles ahead,
// over the ends of pairs.
#pragma once
#include <cstdint>
#include "ptx.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kDecWarps = 4;
constexpr int kDecRows = 16;    // query heads per unit

// kDP: channels padded to 64 or 128.  kKeys: keys per warp and tile.
template <int kDP>
struct DecShape {
  static constexpr int kKeys = 16;
  static constexpr int kTile = kDecWarps * kKeys;
  static constexpr int kRowBytes = kDP * 2;
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;  // per warp, K then V
  static constexpr int kStages = 384 / kDP;
  static constexpr int kMergeBytes = 2 * kDecRows * kDP * 4;
  static constexpr size_t kSmem = size_t(kDecWarps) * kStages * kStageBytes + kMergeBytes +
                                  kDecWarps * kDecRows * 8 + kDecWarps * kStages * 4;
};
constexpr int kDecTile = DecShape<128>::kTile;

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
  FastDiv page;
  float scale, c;                  // c = scale * log2(e)
  float* part;                     // [grid][2][16][kDP] unnormalised parts
  float2* part_ml;                 // [grid][2][16] maximum, total
  int* err;                        // status word, cleared: no wait here can run out
  int2* span;                      // [B][Hkv * hblocks] first and last CTA of a pair
};

__device__ __forceinline__ int dec_len(const DecodeParams& p, int b) {
  const int64_t room = static_cast<int64_t>(p.max_pages) * p.page.div;
  const int64_t n = __ldg(p.lens + b);
  return static_cast<int>(n < 0 ? 0 : (n < room ? n : room));
}
__device__ __forceinline__ int64_t dec_share(int64_t c, int64_t total, int64_t grid) {
  return c * total / grid;
}
// the CTA whose share holds tile w
__device__ __forceinline__ int dec_owner(int64_t w, int64_t total, int64_t grid) {
  int64_t c = w * grid / total;
  while (c + 1 < grid && dec_share(c + 1, total, grid) <= w) ++c;
  while (c > 0 && dec_share(c, total, grid) > w) --c;
  return static_cast<int>(c);
}

template <bool kBf16, int kDP>
__global__ void __launch_bounds__(kDecWarps * 32, 2) attn_decode_kernel(const DecodeParams p) {
  using S = DecShape<kDP>;
  constexpr int kKeys = S::kKeys, kStages = S::kStages;
  constexpr int kSteps = kDP / 16;       // depth steps of Q K^T
  constexpr int kTilesN = kDP / 8;       // 8-channel columns of the output
  constexpr int kChunks = kDP / 8;       // 16-byte chunks of a row
  constexpr int kRowsPer = 32 / kChunks; // rows moved by one warp-wide copy
  constexpr float kBias = kBf16 ? 0.f : 15.f;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(dec_smem) + warp * kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(dec_smem + kDecWarps * kStages * S::kStageBytes);
  float2* ml = reinterpret_cast<float2*>(merge + 2 * kDecRows * kDP);     // [warp][16]
  uint32_t* masks = reinterpret_cast<uint32_t*>(ml + kDecWarps * kDecRows) + warp * kStages;

  const int Hv = p.Hkv * p.hblocks;
  // ---- this CTA's share of the tile list, and the pair it starts in
  __shared__ int64_t scan[kDecWarps];
  __shared__ int64_t sh_before;
  __shared__ int sh_b;
  const int per = (p.B + kDecWarps * 32 - 1) / (kDecWarps * 32);
  const int b_lo = min(p.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.B, b_lo + per);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += (dec_len(p, b) + S::kTile - 1) / S::kTile;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[warp] = incl;
  if (threadIdx.x == 0) sh_b = p.B;
  __syncthreads();
  int64_t before = incl - mine, tiles = 0;
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += scan[w];
    tiles += scan[w];
  }
  const int64_t total = tiles * Hv;
  // CTAs with a share: no more than tiles, so that none inside a pair's span is empty
  const int64_t grid = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= grid) return;
  const int64_t lo = dec_share(blockIdx.x, total, grid);
  const int64_t hi = dec_share(blockIdx.x + 1, total, grid);
  if (lo >= before * Hv && lo < (before + mine) * Hv) {
    int64_t at = before;
    for (int b = b_lo; b < b_hi; ++b) {
      const int64_t n = (dec_len(p, b) + S::kTile - 1) / S::kTile;
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
  } ld, cur;
  ld.b = sh_b;
  ld.len = dec_len(p, ld.b);
  ld.n = (ld.len + S::kTile - 1) / S::kTile;
  {
    const int64_t r = lo - sh_before * Hv;
    ld.h = static_cast<int>(r / ld.n);
    ld.j = static_cast<int>(r - static_cast<int64_t>(ld.h) * ld.n);
  }
  cur = ld;
  auto advance = [&](Cursor& k) {
    if (++k.j < k.n) return;
    k.j = 0;
    if (++k.h < Hv) return;
    k.h = 0;
    do {
      if (++k.b >= p.B) return;
      k.len = dec_len(p, k.b);
      k.n = (k.len + S::kTile - 1) / S::kTile;
    } while (k.n == 0);
  };
  // page of this lane's key (lane % kKeys) of a tile, -1 where there is none
  const int my_row = lane & (kKeys - 1);
  auto page_of = [&](const Cursor& k) -> int {
    const int t = k.j * S::kTile + warp * kKeys + my_row;
    if (t >= k.len) return -1;
    const int id = __ldg(p.table + k.b * p.table_bs + fdiv(t, p.page));
    return (id >= 0 && id < p.num_pages) ? id : -1;
  };
  const int64_t work = hi - lo;
  const int ch = lane % kChunks, sub = lane / kChunks;
  const bool ch_live = ch * 8 < p.d;
  auto issue = [&](int stage, const Cursor& k, int id) {
    const int t = k.j * S::kTile + warp * kKeys + my_row;
    const int row = t - static_cast<int>(fdiv(t, p.page)) * static_cast<int>(p.page.div);
    const int hk = k.h / p.hblocks;
    const int64_t ko = id * p.k_ps + row * p.k_ts + hk * p.k_hs;
    const int64_t vo = id * p.v_ps + row * p.v_ts + hk * p.v_hs;
    const unsigned valid = __ballot_sync(0xffffffffu, id >= 0) & ((1u << kKeys) - 1u);
    if (lane == 0) masks[stage] = valid;
    const uint32_t dst = ring + stage * S::kStageBytes;
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

  int64_t issued = 0;
  int fill = 0, stage = 0;  // ring places of the next load and of the current tile
  int next_id = page_of(ld);
  auto issue_next = [&]() {
    if (issued < work) {
      const Cursor now = ld;
      const int id = next_id;
      if (issued + 1 < work) {  // the next tile's pages are looked up a tile ahead
        advance(ld);
        next_id = page_of(ld);
      }
      issue(fill, now, id);
    }
    ++issued;
    fill = fill + 1 == kStages ? 0 : fill + 1;
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) issue_next();

  uint32_t qf[kSteps][4];
  float o[kTilesN][4];
  float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
  const int g = lane >> 2, q2 = (lane & 3) * 2;  // fragment row and column
  bool fresh = true;
  bool whole = cur.j == 0;  // the pair started in this share
#pragma unroll 1
  for (int64_t i = 0; i < work; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue_next();
    const int hk = cur.h / p.hblocks, hb = cur.h - hk * p.hblocks;
    const int rows = min(kDecRows, p.group - hb * kDecRows);
    const int head0 = hk * p.group + hb * kDecRows;
    if (fresh) {
      const uint16_t* qb = p.q + cur.b * p.q_bs;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = g + (e & 1) * 8, c = s * 16 + q2 + (e >> 1) * 8;
          qf[s][e] = (r < rows && c < p.d)
                         ? *reinterpret_cast<const uint32_t*>(qb + (head0 + r) * p.q_hs + c)
                         : 0u;
        }
#pragma unroll
      for (int n = 0; n < kTilesN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
      m0 = m1 = kNegInf;
      l0 = l1 = 0.f;
      fresh = false;
    }
    const uint32_t kb = ring + stage * S::kStageBytes, vb = kb + kKeys * S::kRowBytes;
    const uint32_t valid = masks[stage];
    if (valid) {
      float s[2][4] = {};
      {
        // ldmatrix rows: keys (lane % 8) and 8 + (lane % 8), depth halves
        const int r = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
        const uint32_t rb = kb + r * S::kRowBytes;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          uint32_t f[4];
          ldsm_x4(rb + (((2 * st + half) ^ (r & 7)) << 4), f);
          mma_16816<kBf16>(s[0], qf[st], f[0], f[1]);
          mma_16816<kBf16>(s[1], qf[st], f[2], f[3]);
        }
      }
      if (valid != (1u << kKeys) - 1u) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((valid >> (n * 8 + q2 + (e & 1))) & 1u)) s[n][e] = kNegInf;
      }
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
      const bool up = x0 > m0 || x1 > m1;
      if (__any_sync(0xffffffffu, up)) {
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        const float a0 = m0 == kNegInf ? 0.f : exp2_approx((m0 - n0) * p.c);
        const float a1 = m1 == kNegInf ? 0.f : exp2_approx((m1 - n1) * p.c);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < kTilesN; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a0;
          o[n][2] *= a1;
          o[n][3] *= a1;
        }
      }
      const float z0 = (m0 == kNegInf ? 0.f : m0 * p.c) - kBias;
      const float z1 = (m1 == kNegInf ? 0.f : m1 * p.c) - kBias;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        s[n][0] = exp2_approx(fmaf(s[n][0], p.c, -z0));
        s[n][1] = exp2_approx(fmaf(s[n][1], p.c, -z0));
        s[n][2] = exp2_approx(fmaf(s[n][2], p.c, -z1));
        s[n][3] = exp2_approx(fmaf(s[n][3], p.c, -z1));
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
      }
      // probabilities round to the value type for the second product; the
      // totals above keep them in fp32
      const uint32_t a[4] = {pack2<kBf16>(s[0][0], s[0][1]), pack2<kBf16>(s[0][2], s[0][3]),
                             pack2<kBf16>(s[1][0], s[1][1]), pack2<kBf16>(s[1][2], s[1][3])};
      {
        const int r = lane & 15, hi8 = lane >> 4;
        const uint32_t rb = vb + r * S::kRowBytes;
#pragma unroll
        for (int n = 0; n < kTilesN; n += 2) {
          uint32_t f[4];
          ldsm_x4_t(rb + (((n + hi8) ^ (r & 7)) << 4), f);
          mma_16816<kBf16>(o[n], a, f[0], f[1]);
          mma_16816<kBf16>(o[n + 1], a, f[2], f[3]);
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const bool last = cur.j == cur.n - 1;
    if (last || i == work - 1) {
      // ---- the pair ends here, or goes on in the next share
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if ((lane & 3) == 0) {
        ml[warp * kDecRows + g] = make_float2(m0, l0);
        ml[warp * kDecRows + g + 8] = make_float2(m1, l1);
      }
      __syncthreads();
      float M0 = kNegInf, M1 = kNegInf, L0 = 0.f, L1 = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        M0 = fmaxf(M0, ml[w * kDecRows + g].x);
        M1 = fmaxf(M1, ml[w * kDecRows + g + 8].x);
      }
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float2 a = ml[w * kDecRows + g], b = ml[w * kDecRows + g + 8];
        if (a.x != kNegInf) L0 += a.y * exp2_approx((a.x - M0) * p.c);
        if (b.x != kNegInf) L1 += b.y * exp2_approx((b.x - M1) * p.c);
      }
      const float f0 = m0 == kNegInf ? 0.f : exp2_approx((m0 - M0) * p.c);
      const float f1 = m1 == kNegInf ? 0.f : exp2_approx((m1 - M1) * p.c);
#pragma unroll
      for (int n = 0; n < kTilesN; ++n) {
        o[n][0] *= f0;
        o[n][1] *= f0;
        o[n][2] *= f1;
        o[n][3] *= f1;
      }
      // warps 2 and 3 hand theirs to 0 and 1, then warp 1 to warp 0
      auto put = [&](float* at) {
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) at[(n * 4 + e) * 32 + lane] = o[n][e];
      };
      auto add = [&](const float* at) {
#pragma unroll
        for (int n = 0; n < kTilesN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] += at[(n * 4 + e) * 32 + lane];
      };
      if (warp >= 2) put(merge + (warp - 2) * kDecRows * kDP);
      __syncthreads();
      if (warp < 2) add(merge + warp * kDecRows * kDP);
      if (warp == 1) put(merge + kDecRows * kDP);
      __syncthreads();
      if (warp == 0) {
        add(merge + kDecRows * kDP);
        if (whole && last) {
          const float i0 = L0 > 0.f ? 1.f / L0 : 0.f, i1 = L1 > 0.f ? 1.f / L1 : 0.f;
          uint16_t* ob = p.out + cur.b * p.o_bs;
#pragma unroll
          for (int n = 0; n < kTilesN; ++n) {
            const int c = n * 8 + q2;
            if (c < p.d && g < rows)
              *reinterpret_cast<uint32_t*>(ob + (head0 + g) * p.o_hs + c) =
                  pack2<kBf16>(o[n][0] * i0, o[n][1] * i0);
            if (c < p.d && g + 8 < rows)
              *reinterpret_cast<uint32_t*>(ob + (head0 + g + 8) * p.o_hs + c) =
                  pack2<kBf16>(o[n][2] * i1, o[n][3] * i1);
          }
          if (p.lse && (lane & 3) == 0) {
            float* lb = p.lse + static_cast<int64_t>(cur.b) * p.Hq + head0;
            if (g < rows)
              lb[g] = L0 > 0.f ? M0 * p.scale + (log2f(L0) - kBias) * 0.69314718f : kNegInf;
            if (g + 8 < rows)
              lb[g + 8] = L1 > 0.f ? M1 * p.scale + (log2f(L1) - kBias) * 0.69314718f : kNegInf;
          }
        } else {
          // a pair that began in an earlier share fills slot 0, one that goes on slot 1
          const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (whole ? 1 : 0);
          float* pb = p.part + slot * kDecRows * kDP;
#pragma unroll
          for (int n = 0; n < kTilesN; ++n) {
            const int c = n * 8 + q2;
            if (g < rows)
              *reinterpret_cast<float2*>(pb + g * kDP + c) = make_float2(o[n][0], o[n][1]);
            if (g + 8 < rows)
              *reinterpret_cast<float2*>(pb + (g + 8) * kDP + c) = make_float2(o[n][2], o[n][3]);
          }
          if ((lane & 3) == 0) {
            p.part_ml[slot * kDecRows + g] = make_float2(M0, L0);
            p.part_ml[slot * kDecRows + g + 8] = make_float2(M1, L1);
          }
        }
        if (whole && lane == 0) {
          int c1 = blockIdx.x;
          if (!last) c1 = dec_owner(lo + i + (cur.n - 1 - cur.j), total, grid);
          p.span[static_cast<int64_t>(cur.b) * Hv + cur.h] = make_int2(blockIdx.x, c1);
        }
      }
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
  constexpr float kBias = kBf16 ? 0.f : 15.f;
  __shared__ float acc[4][kDP];
  __shared__ float tot[4];
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
  auto slot_of = [&](int c) { return static_cast<int64_t>(c) * 2 + (c == sp.x ? 1 : 0); };
  float M = kNegInf;
  for (int c = sp.x + lane; c <= sp.y; c += 32) M = fmaxf(M, p.part_ml[slot_of(c) * kDecRows + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float v[kVals] = {}, L = 0.f;
  for (int c = sp.x + warp; c <= sp.y; c += 4) {
    const float2 a = p.part_ml[slot_of(c) * kDecRows + row];
    const float f = a.x == kNegInf ? 0.f : exp2_approx((a.x - M) * p.c);
    L += a.y * f;
    const float* pb = p.part + (slot_of(c) * kDecRows + row) * kDP + lane * kVals;
#pragma unroll
    for (int e = 0; e < kVals; ++e) v[e] += pb[e] * f;
  }
#pragma unroll
  for (int e = 0; e < kVals; ++e) acc[warp][lane * kVals + e] = v[e];
  if (lane == 0) tot[warp] = L;
  __syncthreads();
  L = (tot[0] + tot[1]) + (tot[2] + tot[3]);
  const float inv = L > 0.f ? 1.f / L : 0.f;
  for (int c = threadIdx.x; c < p.d; c += blockDim.x) {
    const float x = ((acc[0][c] + acc[1][c]) + (acc[2][c] + acc[3][c])) * inv;
    ob[c] = kBf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                  : __half_as_ushort(__float2half_rn(x));
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[static_cast<int64_t>(b) * p.Hq + head] =
        L > 0.f ? M * p.scale + (log2f(L) - kBias) * 0.69314718f : kNegInf;
}

}  // namespace rnn
