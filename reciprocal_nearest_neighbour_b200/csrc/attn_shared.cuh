// Attention of one new token per sequence where all sequences of the batch start with
// the same cached tokens:
//   out = sum_t softmax_t(scale q.k_t) v_t over the prefix's rows t and the sequence's own.
// Softmax parts over disjoint keys join exactly: with maximum m, total l and sum o of
// each part, out = sum o 2^(m - M) / sum l 2^(m - M), M the largest m.  So the prefix is
// attended to once for the whole batch (attn_prefix_kernel), each sequence's own rows as
// in attn_decode (its kernel, with parts in place of outputs), and a last kernel joins.
//
// The prefix's rows are read once per 256 query rows in place of once per sequence: the
// B * group queries of a key head are the rows of one matrix, 128 to a tile of the
// tensor cores.  Up to about 100 rows its 512 bytes a key and head (128 channels) bound
// the kernel, beyond that 4 * 128 * 128 d flops a row tile and 128 keys.
//
// attn_prefix_kernel: a CTA takes up to 256 rows of one key head and a range of the
// prefix's 128-key tiles.  With more than 128 rows (wide) its two row tiles go over the
// same keys, with up to 128 (narrow) the one row tile is there twice, for every other key
// tile, so that in either case one tile's softmax runs under the other's products:
//   warps 0-3, 4-7  fetch the queries of tile 0 and 1; then the softmax, one thread a row
//                   (as in attn_prompt): scores from tensor memory, probabilities back over
//                   them as the 16-bit A operand of the second product; in the end the
//                   rows' parts
//   warps 8, 9      issue S = Q K^T and O += P V of tile 0 and 1
//   warps 12-15     fetch K tiles (two warps) and V tiles (two) into a ring each, by 16-byte
//                   asynchronous copies: pages of any size and stride lie in shared memory
//                   as the tensor cores' 128-byte swizzle wants them
// Tensor memory: two score tiles of 128 columns, two output tiles of kDP.
//
// Measured, in a CUDA graph, all three kernels: 144 streams of 5 to 700 tokens behind 30 011,
// 32/8 heads of 128 (576 rows a key head), 126 us, of which this kernel has about 95: a wide
// step (two row tiles, 128 keys) takes 4250 cycles at 1.7 GHz, where the exponentials need
// 2048 and the products as many; a tile's chain of scores, softmax, product bounds it, as in
// attn_prompt.  32 streams behind 9001 tokens (128 rows) 34.5 us: three kernels of 10 to 13 us,
// each mostly set-up, first loads and way out.  Scores in halves of a key tile, with a
// buffer each so that the next one's product runs under the softmax: 153 us where whole ones
// took 135 (a product of 64 columns takes as long as one of 128).
#pragma once
#include <cstdint>
#include "attn_decode.cuh"
#include "attn_prompt.cuh"

namespace rnn {

constexpr int kPreThreads = 512;   // warps 10 and 11 only complete their warpgroup
constexpr int kPreMmaWarp = 8, kPreLoadWarp = 12;
constexpr int kPreUnit = 2 * kAttnM;        // query rows of a unit
// Key tiles of a row tile in one accumulator: 65536 keys (see attn_prompt).
constexpr int kPreMostTiles = 512;

template <int kDP>
struct PreShape {
  static constexpr int kTileBytes = kAttnM * kDP * 2;
  static constexpr int kBlockBytes = kAttnM * 128;
  static constexpr int kStages = kDP == 128 ? 2 : 4;  // of each ring; a power of two
  // (narrow units have one row tile less and one V slot more: 144 streams behind 30011
  // tokens waited a thousand cycles a step for their V tiles)
  static constexpr size_t kSmem = 1024 + size_t(2 + 2 * kStages) * kTileBytes + 512;
};

struct PrefixParams {
  const uint16_t *q, *kc, *vc;
  int64_t q_bs, q_hs;                  // strides in elements
  int64_t k_ps, k_ts, k_hs, v_ps, v_ts, v_hs;
  const int32_t *pages, *len;          // the prefix: its pages, and its length on the device
  int64_t num_pages;
  int max_pages, page16;
  FastDiv page, by_group;
  int rows, group, d;                  // rows: B * group
  int wide, narrow;                    // units of a key head: wide ones, and 0 or 1 narrow one
  int wide_splits, narrow_splits;      // CTAs that share a unit's keys
  int Hkv;
  float c;                             // scale * log2(e)
  uint32_t idesc_s, idesc_o;
  float* part;                         // [slot][128][kDP] unnormalised parts
  float2* part_ml;                     // [slot][128] maximum, total
  int* err;
  unsigned long long wait_limit_ns;
  int stall_loads;
};

// Slots of the parts of a unit: its splits times its two tiles.
__device__ __forceinline__ int pre_slot0(const PrefixParams& p, int hk, int unit) {
  const int per_head = 2 * (p.wide * p.wide_splits + p.narrow * p.narrow_splits);
  return hk * per_head + 2 * min(unit, p.wide) * p.wide_splits;
}

template <bool kBf16, int kDP>
__global__ void __launch_bounds__(kPreThreads, 1)
attn_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using S = PreShape<kDP>;
  constexpr int kStages = S::kStages, kCols = 512;
  constexpr int kOutCol = 2 * kAttnN;
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = smem + (2 + 2 * kStages) * S::kTileBytes;
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * (2 * kStages + 1);
  const uint32_t qfull_bar = empty_bar + 8 * (2 * kStages + 1);
  const uint32_t s_bar = qfull_bar + 8;     // scores of tile i are in tensor memory
  const uint32_t p_bar = s_bar + 16;        // its probabilities are there, by halves
  const uint32_t o_bar = p_bar + 32;        // its output is complete so far
  const uint32_t drain_bar = o_bar + 16;
  const uint32_t last_bar = drain_bar + 16; // tile i's last product is complete
  const uint32_t tmem_slot = last_bar + 16;
  const uint32_t abort_at = tmem_slot + 4;
  // Keys that exist, 4 words for each of 8 tiles: when a tile's words are written, the
  // scores of the tile four before it are done, so the softmax has read the words of the
  // one eight before it.
  const uint32_t mask_at = (tmem_slot + 8 + 15) & ~15u;
  const uint32_t turn_at = mask_at + 128;   // per softmax warp: steps whose exponentials are out

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ---- this CTA's unit and key tiles
  const int wide_ctas = p.Hkv * p.wide * p.wide_splits;
  const bool wide = static_cast<int>(blockIdx.x) < wide_ctas;
  const int splits = wide ? p.wide_splits : p.narrow_splits, units = wide ? p.wide : 1;
  int x = static_cast<int>(blockIdx.x) - (wide ? 0 : wide_ctas);
  const int unit = wide ? x % units : p.wide;
  x /= units;
  const int split = x % splits, hk = x / splits;
  const int64_t room = static_cast<int64_t>(p.max_pages) * p.page.div;
  const int64_t given = __ldg(p.len);
  const int keys = static_cast<int>(
      given < 0 ? 0 : min(given, min(room, static_cast<int64_t>(kDecMaxKeys))));
  const int all = (keys + kAttnN - 1) / kAttnN;
  const int tile0 = static_cast<int>(static_cast<int64_t>(all) * split / splits);
  const int n = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / splits) - tile0;

  // the row tiles, then the rings: K of key tile j in slot j % kStages, V behind the K slots
  const uint32_t q_tiles = smem, ring = smem + (wide ? 2 : 1) * S::kTileBytes;
  auto slot_of = [&](int j) { return j % kStages; };
  auto turn_of = [&](int j) { return j / kStages & 1; };
  auto v_slot_of = [&](int j) { return kStages + (wide ? j % kStages : j % (kStages + 1)); };
  auto v_turn_of = [&](int j) { return (wide ? j / kStages : j / (kStages + 1)) & 1; };

  auto aborted = [&]() { return lds_volatile(abort_at) != 0; };
  auto wait = [&](uint32_t bar, uint32_t parity, int code) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (true) {
      if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
      if (aborted()) return false;
      if (globaltimer_ns() - t0 > p.wait_limit_ns) {
        sts_volatile(abort_at, 1);
        atomicOr(p.err, code);
        return false;
      }
    }
  };
  if (threadIdx.x < 2 * kStages + 1) {
    mbar_init(full_bar + 8 * threadIdx.x, 2);
    mbar_init(empty_bar + 8 * threadIdx.x, wide ? 2 : 1);
    fence_barrier_init();
  } else if (threadIdx.x >= 32 && threadIdx.x < 34) {
    const int i = threadIdx.x - 32;
    mbar_init(s_bar + 8 * i, 1);
    mbar_init(p_bar + 8 * i, 4);
    mbar_init(p_bar + 8 * (2 + i), 4);
    mbar_init(o_bar + 8 * i, 1);
    mbar_init(drain_bar + 8 * i, 1);
    mbar_init(last_bar + 8 * i, 1);
    if (i == 0) mbar_init(qfull_bar, wide ? 8 : 4);
    fence_barrier_init();
  } else if (threadIdx.x >= 64 && threadIdx.x < 72) {
    sts_volatile(turn_at + 4 * (threadIdx.x - 64), 0);
    if (threadIdx.x == 64) sts_volatile(abort_at, 0);
  }
  if (warp == kPreMmaWarp) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_volatile(tmem_slot);
  // steps of tile i, and the CTA's key tile of its step k
  const int n_of[2] = {wide ? n : (n + 1) / 2, wide ? n : n / 2};
  auto tile_of = [&](int i, int k) { return wide ? k : 2 * k + i; };

  // 16-byte chunk `ch` of row r of a tile, in the 128-byte swizzle of its 64-channel block
  auto chunk_at = [](int r, int ch) {
    return (ch >> 3) * S::kBlockBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  };

  if (warp >= kPreMmaWarp) {
    regs_give<kAttnRegsOther>();
    if (warp >= kPreLoadWarp) {
      // ------------------------------------------------------------- loads
      constexpr int kChunks = kDP / 8, kRowsPer = 32 / kChunks;
      const int w = warp - kPreLoadWarp;
      const bool is_v = w >= 2;               // of the rings
      const int rows0 = (w & 1) * 64;
      auto place_of = [&](int j) { return is_v ? v_slot_of(j) : slot_of(j); };
      auto phase_of = [&](int j) { return is_v ? v_turn_of(j) : turn_of(j); };
      const int ch = lane % kChunks, sub = lane / kChunks;
      const bool ch_live = ch * 8 < p.d;
      auto at = [&](int r) { return chunk_at(r, ch); };
      // Copies are told to the tensor cores' proxy by the thread that made them, when
      // they are complete, in their order.
      int issued = 0, told = 0;
      auto tell = [&]() {
        switch (issued - told) {
          case 0: break;
          case 1: cp_async_wait<0>(); break;
          case 2: cp_async_wait<1>(); break;
          case 3: cp_async_wait<2>(); break;
          default: cp_async_wait<3>(); break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar + 8 * place_of(told));
        ++told;
      };
      const int loads = p.stall_loads ? 0 : n;
      const uint16_t* const base = is_v ? p.vc : p.kc;
      const int64_t ps = is_v ? p.v_ps : p.k_ps, ts = is_v ? p.v_ts : p.k_ts;
      const uint16_t* const head = base + hk * (is_v ? p.v_hs : p.k_hs) + ch * 8;
      bool ok = true;
      for (int j = 0; j < loads; ++j) {
        const int slot = place_of(j);
        const uint32_t eb = empty_bar + 8 * slot, parity = phase_of(j) ^ 1u;
        while (!__all_sync(0xffffffffu, mbar_test_wait(eb, parity))) {
          if (told < issued) {
            tell();
          } else {
            ok = __all_sync(0xffffffffu, wait(eb, parity, kErrWaitProducer));
            break;
          }
        }
        if (!ok) break;
        const uint32_t dst = ring + slot * S::kTileBytes;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 32 rows, a lane's page for each
          const int r0 = rows0 + half * 32, t = (tile0 + j) * kAttnN + r0 + lane;
          int id = -1;
          if (t < keys) {
            id = __ldg(p.pages + fdiv(t, p.page));
            if (id < 0 || id >= p.num_pages) id = -1;
          }
          const unsigned valid = __ballot_sync(0xffffffffu, id >= 0);
          if (!is_v && lane == 0)
            sts_volatile(mask_at + 16 * (j & 7) + (r0 >> 3), static_cast<int>(valid));
          const int row = t - static_cast<int>(fdiv(t, p.page)) * static_cast<int>(p.page.div);
          if (p.page16) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int64_t page = max(0, __shfl_sync(0xffffffffu, id, g * 16));
              const int row0 = __shfl_sync(0xffffffffu, row, g * 16) + sub;
              const uint16_t* src = head + page * ps + row0 * ts;
#pragma unroll
              for (int i = 0; i < 16 / kRowsPer; ++i) {
                const int r = g * 16 + i * kRowsPer + sub;
                const bool live = ((valid >> r) & 1u) && ch_live;
                cp_async16(dst + at(r0 + r), live ? src : base, live);
                src += kRowsPer * ts;
              }
            }
          } else {
            const int64_t off = id * ps + row * ts;
#pragma unroll 4
            for (int i = 0; i < 32 / kRowsPer; ++i) {
              const int r = i * kRowsPer + sub;
              const int64_t o = __shfl_sync(0xffffffffu, off, r);
              const bool live = ((valid >> r) & 1u) && ch_live;
              cp_async16(dst + at(r0 + r), live ? head + o : base, live);
            }
          }
        }
        cp_async_commit();
        ++issued;
        if (issued - told > 4) tell();
      }
      while (told < issued) tell();
      if (!(w & 1) && !aborted()) {
        // no arrival of a product's completion is under way when the CTA exits
        const int slots = kStages + (is_v && !wide), j = max(0, loads - slots) + lane;
        if (lane < slots && j < loads)
          settle_phase(empty_bar + 8 * place_of(j), phase_of(j), p.wait_limit_ns, p.err);
        __syncwarp();
      }
    } else if (warp < kPreMmaWarp + 2) {
      // ---------------------------------------------------------- products
      const int i = warp - kPreMmaWarp;
      const int dsteps = (p.d + 15) / 16;
      const uint64_t q_desc = make_sdesc(q_tiles + (wide ? i : 0) * S::kTileBytes, 64);
      const uint64_t k_desc = make_sdesc(ring, 64);
      const uint64_t v_desc = make_vdesc(ring);
      bool ok = true, any = false;
      auto wait_mma = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, wait(bar, parity, kErrWaitMma));
        return ok;
      };
      if (n_of[i] > 0) wait_mma(qfull_bar, 0);
      for (int k = 0; ok && k < n_of[i]; ++k) {
        const int j = tile_of(i, k), ks = slot_of(j), vs = v_slot_of(j);
        if (!wait_mma(full_bar + 8 * ks, turn_of(j))) break;
        // the probabilities lie over the scores: the product that reads them first
        if (k > 0 && !wait_mma(o_bar + 8 * i, (k - 1) & 1)) break;
        tc_fence_after();
        const uint64_t k_at = k_desc + static_cast<uint64_t>(ks * (S::kTileBytes >> 4));
        const int whole = dsteps >> 2;
#pragma unroll
        for (int c = 0; c < kDP / 64; ++c) {
          const uint32_t blk = c * (S::kBlockBytes >> 4);
          if (c < whole) {
            umma_ss_x4(tmem + i * kAttnN, q_desc + blk, k_at + blk, p.idesc_s, c > 0);
          } else {
            for (int s = 0; s < dsteps - 4 * c; ++s)
              umma_f16_warp(tmem + i * kAttnN, q_desc + blk + 2 * s, k_at + blk + 2 * s, p.idesc_s,
                            c > 0 || s > 0);
          }
        }
        umma_commit_warp(s_bar + 8 * i);
        umma_commit_warp(empty_bar + 8 * ks);
        any = true;
        if (!wait_mma(full_bar + 8 * vs, v_turn_of(j))) break;
        const uint64_t v_at = v_desc + static_cast<uint64_t>(vs * (S::kTileBytes >> 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait_mma(p_bar + 8 * (2 * h + i), k & 1)) break;
          tc_fence_after();
          umma_ts_x4(tmem + kOutCol + i * kDP, tmem + i * kAttnN + h * 32,
                     v_at + static_cast<uint64_t>(h * (8192 >> 4)), p.idesc_o,
                     (k > 0 || h > 0) ? 1u : 0u);
        }
        if (!ok) break;
        umma_commit_warp(o_bar + 8 * i);
        umma_commit_warp(empty_bar + 8 * vs);
        if (k + 1 == n_of[i]) umma_commit_warp(last_bar + 8 * i);
        __syncwarp();
      }
      // (the last arrival at this barrier too is made before the CTA exits)
      if (n_of[i] > 0) wait_mma(o_bar + 8 * i, (n_of[i] - 1) & 1);
      if (aborted() && any) {
        // let every product issued finish before tensor memory is released
        umma_commit_warp(drain_bar + 8 * i);
        __syncwarp();
        settle_phase(drain_bar + 8 * i, 0, p.wait_limit_ns, p.err);
      }
    }
  } else {
    // ----------------------------------------------------------- softmax
    regs_take<kAttnRegsSoftmax>();
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;     // row of the tile
    const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_at + i * kAttnN;
    const uint32_t o_at = tmem + lane_at + kOutCol + i * kDP;
    const int steps = i ? n_of[1] : n_of[0], steps_o = i ? n_of[0] : n_of[1];
    const int base = unit * kPreUnit + (wide ? i * kAttnM : 0);  // the tile's first row
    if (n > 0 && (wide || i == 0)) {  // (a narrow unit has its row tile once)
      constexpr int kChunks = kDP / 8, kRowsPer = 32 / kChunks;
      const int ch = lane % kChunks, sub = lane / kChunks;
      const bool row_live = base + r < p.rows;
      const int b = row_live ? fdiv(base + r, p.by_group) : 0;
      const int64_t off = b * p.q_bs + (hk * p.group + (row_live ? base + r - b * p.group : 0)) * p.q_hs;
      const unsigned rows_there = __ballot_sync(0xffffffffu, row_live);
#pragma unroll 4
      for (int x = sub; x < 32; x += kRowsPer) {
        const int64_t o = __shfl_sync(0xffffffffu, off, x);
        const bool live = ((rows_there >> x) & 1u) && ch * 8 < p.d;
        cp_async16(q_tiles + i * S::kTileBytes + chunk_at((warp & 3) * 32 + x, ch),
                   live ? p.q + o + ch * 8 : p.q, live);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull_bar);
    }
    float m = kNegInf, l = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      ok = wait(s_bar + 8 * i, k & 1, kErrWaitEpilogue);
      __syncwarp();
      tc_fence_after();
      float s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, s[c]);
      const uint4 there = lds_v4(mask_at + 16 * (tile_of(i, k) & 7));
      tmem_wait_ld_regs(s[0]);
#pragma unroll
      for (int c = 1; c < 4; ++c) reg_fence(s[c]);
      if ((there.x & there.y & there.z & there.w) != 0xffffffffu) {
        const uint32_t has[4] = {there.x, there.y, there.z, there.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((has[c] >> e) & 1u)) s[c][e] = kNegInf;
      }
      const float top = fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
      if (k == 0) m = top;
      const bool grow = (top - m) * p.c > kAttnSlack;  // also from -inf to a number
      float mc = m * p.c;
      // one vote for all: a lane whose wait gave up takes the warp with it
      if (__any_sync(0xffffffffu, grow || !ok || fabsf(mc) > kAttnFar)) {
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float f = grow ? exp2_approx((m - top) * p.c) : 1.f;
        if (grow) m = top;
        mc = m == kNegInf ? 0.f : m * p.c;
        const bool before = fabsf(mc) > kAttnFar && fabsf(m) < -kNegInf;
        if (__any_sync(0xffffffffu, before)) {
          const float ref = before ? m : 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) s[c][e] -= ref;
          if (before) mc = 0.f;
        }
        l *= f;
        if (__any_sync(0xffffffffu, grow)) {  // (only behind a first step: its product is done)
#pragma unroll
          for (int c = 0; c < kDP / 32; ++c) {
            float o[32];
            tmem_ld32(o_at + c * 32, o);
            tmem_wait_ld_regs(o);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[h * 16 + e] * f);
              tmem_st16(o_at + c * 32 + h * 16, w);
            }
          }
        }
      }
      const float z = mc - kBias;
      const uint64_t c2 = f2_make(p.c, p.c), z2 = f2_make(-z, -z);
      // the two warps of a scheduler take turns at the exponential unit, as in attn_prompt
      const int k_o = i ? k : k - 1;  // the other's step to wait for
      if (k_o >= 0 && k_o < steps_o) {
#pragma unroll 1
        for (int look = 0; look < kTurnPolls; ++look) {
          if (lds_volatile(turn_at + 4 * (warp ^ 4)) > k_o) break;
          __nanosleep(40);
        }
      }
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float a, b;
          f2_get(f2_fma(f2_make(s[c][2 * e], s[c][2 * e + 1]), c2, z2), a, b);
          a = exp2_approx(a);
          b = exp2_approx(b);
          sum[e & 1] = f2_add(sum[e & 1], f2_make(a, b));
          // the second product takes the probabilities in the value type (half a step:
          // 2^-9 of bf16, 2^-12 of fp16, of each weight); the total keeps them in fp32
          w[e] = pack2<kBf16>(a, b);
        }
        if (c == kTurnChunk && lane == 0) sts_volatile(turn_at + 4 * warp, k + 1);
        tmem_st16(s_at + c * 16, w);
        if (c & 1) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_bar + 8 * (2 * (c >> 1) + i));
        }
      }
      float a, b;
      f2_get(f2_add(sum[0], sum[1]), a, b);
      l += a + b;
    }
    // every product is complete: the rings are free for the way out
    // (told by a barrier that has one phase: the other tile may be any number of steps behind)
    ok = ok && (n_of[0] == 0 || wait(last_bar, 0, kErrWaitEpilogue)) &&
         (n_of[1] == 0 || wait(last_bar + 8, 0, kErrWaitEpilogue));
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    // ---- the rows' parts
    const int64_t at = static_cast<int64_t>(pre_slot0(p, hk, unit) + 2 * split + i) * kAttnM;
    const int mine = min(kAttnM, p.rows - base);   // rows of the tile
    if (!ok) m = l = __uint_as_float(0x7FC00000u);  // given up: its row becomes NaN
    if (r < mine) p.part_ml[at + r] = make_float2(m, l);
    if (steps > 0 && ok) {
      // 32 channels at a time through shared memory, so that a store covers whole lines
      // (straight from its row each thread would write 16 bytes of 32 lines: 5000 cycles)
      const uint32_t stage = ring + warp * 4096;
      const int ch = lane & 7;
      float* const to = p.part + at * kDP + ch * 4;
#pragma unroll 1
      for (int c = 0; c < kDP; c += 32) {
        float o[32];
        tmem_ld32(o_at + c, o);
        tmem_wait_ld_regs(o);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sts_v4(stage + lane * 128 + ((e ^ (lane & 7)) << 4),
                 make_uint4(__float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
                            __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3])));
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int x = e * 4 + (lane >> 3), row = (warp & 3) * 32 + x;
          if (row < mine)
            *reinterpret_cast<uint4*>(to + row * kDP + c) =
                lds_v4(stage + x * 128 + ((ch ^ (x & 7)) << 4));
        }
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPreMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  // This kernel starts while the one that attends to the sequences' own rows still runs,
  // and reads nothing of it; the join behind both may only wait for this one's end.  (One
  // after another: 32 streams behind 9001 tokens 37.7 us, 34.5 so.)
  pdl_wait();
}

// Joins a row's parts: the prefix's, one from each of its unit's splits (and tiles), and
// its sequence's own.  A team of kTeam warps (4, or 1 with many rows) takes a (sequence,
// query head): its lanes fetch the parts' maxima and totals at once, then its warps the
// sums in turn, several in flight, in a fixed order.
constexpr int kJoinPass = 32;  // parts whose totals a warp has at a time
template <bool kBf16, int kDP, int kTeam>
__global__ void __launch_bounds__(128)
attn_shared_join_kernel(const DecodeParams p, const __grid_constant__ PrefixParams pre) {
  constexpr int kVals = kDP / 32;  // channels per lane
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  using VecT = std::conditional_t<kVals == 4, float4, float2>;
  __shared__ float acc[4][kDP];
  __shared__ float2 tot[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int member = warp % kTeam;
  const int64_t at_row = static_cast<int64_t>(blockIdx.x) * (4 / kTeam) + warp / kTeam;
  if (at_row >= static_cast<int64_t>(p.B) * p.Hq) return;  // (never with a team of 4)
  const int b = static_cast<int>(at_row / p.Hq);
  const int head = static_cast<int>(at_row - static_cast<int64_t>(b) * p.Hq);
  const int hk = head / p.group, in = head - hk * p.group;
  const int hb = in / kDecRows, dec_row = in - hb * kDecRows;
  const int row = b * p.group + in, unit = row / kPreUnit, at = row - unit * kPreUnit;
  const bool wide = unit < pre.wide;
  const int64_t pre_slot = pre_slot0(pre, hk, unit) + (wide ? at / kAttnM : 0);
  const int64_t pre0 = pre_slot * kAttnM + (wide ? at % kAttnM : at);
  const int n_pre = wide ? pre.wide_splits : 2 * pre.narrow_splits;
  const int pre_step = (wide ? 2 : 1) * kAttnM;
  const bool own = dec_len(p, b) > 0;
  pdl_wait();
  int2 sp = make_int2(0, -1);
  if (own) sp = p.span[static_cast<int64_t>(b) * (p.Hkv * p.hblocks) + hk * p.hblocks + hb];
  const int parts = n_pre + sp.y - sp.x + 1;
  float v[kVals] = {}, M = kNegInf, L = 0.f;
  // this warp's parts: member, member + kTeam, ...
  for (int base = member; base < parts; base += kJoinPass * kTeam) {
    const int i = base + lane * kTeam;
    float2 a = make_float2(kNegInf, 0.f);
    const float* from = nullptr;
    if (i < n_pre) {
      const int64_t mine = pre0 + static_cast<int64_t>(i) * pre_step;
      a = pre.part_ml[mine];
      from = pre.part + mine * kDP;
    } else if (i < parts && sp.x == sp.y) {
      const int64_t mine = static_cast<int64_t>(b) * p.Hq + head;
      a = p.row_ml[mine];
      from = p.row_part + mine * kDP;
    } else if (i < parts) {
      const int c = sp.x + i - n_pre;
      const int64_t mine = (static_cast<int64_t>(c) * 2 + (c == sp.x ? 1 : 0)) * kDecRows + dec_row;
      a = p.part_ml[mine];
      from = p.part + mine * kDP;
    }
    // no key: its sums were not written
    const unsigned there = __ballot_sync(0xffffffffu, !(a.x == kNegInf && a.y == 0.f));
    float m = fmaxf(M, a.x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // (a NaN maximum is a part that was given up: its factor is NaN too; without a
    // reference a part's total is 0, or NaN if its scores were)
    const float f = a.x == kNegInf ? 1.f : exp2_approx((a.x - m) * p.c);
    float l = a.y * f;
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float h = M == kNegInf ? 1.f : exp2_approx((M - m) * p.c);
    L = L * h + l;
    M = m;
#pragma unroll
    for (int e = 0; e < kVals; ++e) v[e] *= h;
    const int here = min(kJoinPass, (parts - base + kTeam - 1) / kTeam);
    const uint64_t at64 = reinterpret_cast<uint64_t>(from);
#pragma unroll 8
    for (int j = 0; j < here; ++j) {
      const float g = __shfl_sync(0xffffffffu, f, j);
      const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, at64, j));
      if (!((there >> j) & 1u)) continue;
      const VecT x = *reinterpret_cast<const VecT*>(src + lane * kVals);
      const float* xs = reinterpret_cast<const float*>(&x);
#pragma unroll
      for (int e = 0; e < kVals; ++e) v[e] = fmaf(xs[e], g, v[e]);
    }
  }
  if constexpr (kTeam > 1) {
#pragma unroll
    for (int e = 0; e < kVals; ++e) acc[warp][lane * kVals + e] = v[e];
    if (lane == 0) tot[warp] = make_float2(M, L);
    __syncthreads();
    if (warp != 0) return;
    M = fmaxf(fmaxf(tot[0].x, tot[1].x), fmaxf(tot[2].x, tot[3].x));
    float f[4];
    L = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[w] = tot[w].x == kNegInf ? 1.f : exp2_approx((tot[w].x - M) * p.c);
      L += tot[w].y * f[w];
    }
#pragma unroll
    for (int e = 0; e < kVals; ++e) {
      const int c = lane * kVals + e;
      v[e] = (acc[0][c] * f[0] + acc[1][c] * f[1]) + (acc[2][c] * f[2] + acc[3][c] * f[3]);
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  uint16_t* ob = p.out + b * p.o_bs + head * p.o_hs + lane * kVals;
  if (lane * kVals < p.d) {  // (kVals divides d)
    if constexpr (kVals == 4)
      *reinterpret_cast<uint2*>(ob) =
          make_uint2(pack2<kBf16>(v[0] * inv, v[1] * inv), pack2<kBf16>(v[2] * inv, v[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(ob) = pack2<kBf16>(v[0] * inv, v[1] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[at_row] = L != 0.f ? M * p.scale + (log2f(L) - kBias) * 0.69314718f : kNegInf;
}

}  // namespace rnn
