// Attention of packed sequences: for every query row i and head of a sequence
//   out_i = sum_t softmax_t(scale q_i.k_t) v_t,  lse_i = log sum_t exp(scale q_i.k_t)
// over the keys t of the same sequence, all of them or (causal) those with
// t <= i + nk - nq, so that the last query sees the last key.
//
// One pass over the keys with a running maximum and total per row; scores and
// probabilities stay in tensor memory.  A CTA holds two tiles of 128 query
// rows (two heads of one group over the same tokens, or with an odd group two
// neighbouring token tiles of one head), both against each 128-key tile, so
// that one tile's softmax runs under the other's matrix products:
//   warps 0-3, 4-7  softmax of query tile 0 and 1: one thread per row reads
//                   its 128 scores (tcgen05.ld), exponentiates them and writes
//                   the probabilities back (tcgen05.st) over the scores as the
//                   16-bit A operand of the second product
//   warp 8          issues S = Q K^T and O += P V (tcgen05.mma), owns tensor memory
//   warp 9          TMA: query tiles, then a ring of alternating K and V tiles
// Tensor memory: two score tiles of 128 columns, two output tiles of kDP.
//
// A CTA is persistent.  The grid has one block per unit (a pair of query
// tiles); a running CTA asks for the next unit by cancelling a block that has
// not started (clusterlaunchcontrol), so units of any length are dealt as CTAs
// come free, without a counter to clear.  The TMA warp fetches units a step
// ahead and loads the next unit's tiles while the last products and the
// epilogue of this one run: the output is read, normalised and stored by the
// softmax warps while the tensor cores start on the next unit's scores.
//
// Rescaling.  A row's reference maximum only moves when its true maximum has
// grown by more than 2^8 over it (the weights then exceed 1 by at most that,
// far inside fp32 and the 16-bit types), so the output accumulator is read
// back and rescaled rarely; the softmax warps do it themselves: the barrier
// that hands them the next scores also tells that the product before it is
// complete, since the tensor pipe works in order.
//
// Bound: 4*128*128*d flops and 128*128 exponentials per tile pair; at d = 128
// the two take the same time on an SM (16 exponentials, 8192 flops a cycle),
// at d = 64 the exponentials take twice as long as the products.
#pragma once
#include <cstdint>
#include <cuda.h>
#include "ptx.cuh"
#include "nn_kernel.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kAttnM = 128;            // query rows per tile
constexpr int kAttnN = 128;            // keys per tile
constexpr int kAttnThreads = 384;      // three warpgroups; warps 10 and 11 only complete the third
// Registers: launched with 168 a thread (65536 / 384 rounded down to 8), the
// softmax warps hold 128 scores each and take what the third group gives up:
// 256 * 208 + 128 * 88 = 384 * 168.
constexpr int kAttnRegsSoftmax = 208, kAttnRegsOther = 88;
constexpr int kAttnMmaWarp = 8, kAttnTmaWarp = 9;
constexpr float kAttnSlack = 8.f;      // log2 growth of the maximum before a rescale

template <int kDP>
struct AttnShape {
  static constexpr int kBlocks = kDP / 64;               // 64-channel column blocks
  static constexpr int kTileBytes = kAttnM * kDP * 2;
  static constexpr int kBlockBytes = kAttnM * 128;
  static constexpr int kStages = kDP == 128 ? 5 : 8;
  static constexpr size_t kSmem = 1024 + size_t(2 + kStages) * kTileBytes + 512;
};

struct PromptParams {
  const int32_t *cu_q, *cu_k;
  uint16_t* out;
  float* lse;                  // [Tq][Hq] or null
  int64_t o_ts, o_hs, Tq, Tk;  // strides in elements
  int B, Hq, group, d;
  int pair_heads;              // the two tiles are heads 2u, 2u + 1 of the same tokens
  int head_units;              // Hq / 2 or Hq
  int causal;
  float scale, c;              // c = scale * log2(e)
  uint32_t idesc_s, idesc_o;   // instruction descriptors of the two products
  int* err;
  unsigned long long wait_limit_ns;
  int stall_loads;
};

__device__ __forceinline__ void umma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory descriptor of a V tile read as the B operand with its channels
// contiguous (rows of 64 channels, 128-byte swizzle): 8-key groups are 1024
// bytes apart, the 64-channel blocks a whole block.
__device__ __forceinline__ uint64_t make_vdesc(uint32_t saddr) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  desc |= static_cast<uint64_t>((kAttnN * 128) >> 4) << 16;
  desc |= static_cast<uint64_t>(1024 >> 4) << 32;
  desc |= static_cast<uint64_t>(1u) << 46;
  desc |= static_cast<uint64_t>(2u) << 61;
  return desc;
}

struct PromptUnit {
  int hu, m;            // head unit, first query row in the sequence
  int q0, nq, k0, nk;   // the sequence; nq < 0: no unit is left
};

__device__ __forceinline__ int clamp_at(const int32_t* cu, int b, int64_t top) {
  const int64_t v = __ldg(cu + b);
  return static_cast<int>(v < 0 ? 0 : (v > top ? top : v));
}

// Ask for a block of this grid that has not started; the 16-byte answer
// completes `bar`.
__device__ __forceinline__ void next_block_request(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(answer),
      "r"(bar)
      : "memory");
}
// The block's index, or -1 when every block has started.
__device__ __forceinline__ int next_block_read(uint32_t answer) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(answer)
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// What each role derives from a unit: per query tile its head, first row and
// the key tiles to visit.
struct PromptTiles {
  int head[2], row0[2], n[2], n_max, shift;
  __device__ __forceinline__ PromptTiles(const PromptParams& p, const PromptUnit& u) {
    shift = u.nk - u.nq;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      head[i] = p.pair_heads ? 2 * u.hu + i : u.hu;
      row0[i] = u.m + (p.pair_heads ? 0 : i * kAttnM);
      int keys = u.nk;
      if (p.causal) keys = min(keys, min(row0[i] + kAttnM, u.nq) + shift);
      n[i] = row0[i] < u.nq && keys > 0 ? (keys + kAttnN - 1) / kAttnN : 0;
    }
    n_max = max(n[0], n[1]);
  }
};

template <int kRegs>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <bool kBf16, int kDP>
__global__ void __launch_bounds__(kAttnThreads, 1)
attn_prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using S = AttnShape<kDP>;
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  constexpr int kUnitReaders = 9;  // softmax warps and the MMA warp
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* q_tiles = smem;
  uint8_t* ring = smem + 2 * S::kTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + S::kStages * S::kTileBytes);
  uint64_t* full_bar = bars;
  uint64_t* empty_bar = full_bar + S::kStages;
  uint64_t* qfull_bar = empty_bar + S::kStages;
  uint64_t* qempty_bar = qfull_bar + 1;
  uint64_t* s_bar = qempty_bar + 1;  // scores of tile i are in tensor memory
  uint64_t* p_bar = s_bar + 2;       // its probabilities are
  uint64_t* o_bar = p_bar + 2;       // its output is complete
  uint64_t* ofree_bar = o_bar + 2;   // its output has been read
  uint64_t* ufull_bar = ofree_bar + 2;
  uint64_t* uempty_bar = ufull_bar + 2;
  uint64_t* ask_bar = uempty_bar + 2;
  uint64_t* drain_bar = ask_bar + 1;
  uint32_t* misc = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  __shared__ __align__(16) uint8_t answer[16];
  __shared__ PromptUnit units[2];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    mbar_init(smem_u32(qfull_bar), 1);
    mbar_init(smem_u32(qempty_bar), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_bar[i]), 1);
      mbar_init(smem_u32(&p_bar[i]), 4);
      mbar_init(smem_u32(&o_bar[i]), 1);
      mbar_init(smem_u32(&ofree_bar[i]), 4);
      mbar_init(smem_u32(&ufull_bar[i]), 1);
      mbar_init(smem_u32(&uempty_bar[i]), kUnitReaders);
    }
    mbar_init(smem_u32(ask_bar), 1);
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  constexpr uint32_t kCols = 512;
  if (warp == kAttnMmaWarp) {
    tmem_alloc(smem_u32(misc), kCols);
    tmem_relinquish();
  }
  if (warp == kAttnTmaWarp && lane == 0) {
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const uint64_t lim = p.wait_limit_ns;

  // Unit number `it` of this CTA, as the TMA warp published it.
  auto take_unit = [&](int it, int code, PromptUnit& u) {
    const int slot = it & 1;
    if (!__all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(&ufull_bar[slot]), (it >> 1) & 1,
                                                 abort_flag, p.err, code, lim)))
      return false;
    u = units[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&uempty_bar[slot]));
    return u.nq >= 0;
  };

  if (warp >= kAttnMmaWarp) {
  regs_give<kAttnRegsOther>();
  if (warp == kAttnTmaWarp) {
    // ------------------------------------------------- units and loads
    const int span = p.pair_heads ? kAttnM : 2 * kAttnM;  // tokens per unit
    int base_b = 0, base_tile = 0;  // a group of 32 sequences and the tiles before it
    int block = blockIdx.x, issued = 0, q_loads = 0;
    int asked = 0;
    bool ok = true;
    auto answered = [&]() {
      if (!__all_sync(0xffffffffu, mbar_wait_sleep(smem_u32(ask_bar), (asked - 1) & 1, abort_flag,
                                                   p.err, kErrWaitProducer, lim)))
        return false;
      block = next_block_read(smem_u32(answer));
      fence_proxy_async_smem();  // read before the next answer is written
      __syncwarp();
      return true;
    };
    auto ask = [&]() {
      if (lane == 0) {
        mbar_arrive_expect_tx(smem_u32(ask_bar), 16);
        next_block_request(smem_u32(answer), smem_u32(ask_bar));
      }
      ++asked;
      __syncwarp();
    };
    for (int it = 0;; ++it) {
      PromptUnit u;
      u.nq = -1;
      while (block >= 0 && ok) {
        // the sequences' query tiles make one list, head units inside
        const int tile = block / p.head_units;
        u.hu = block - tile * p.head_units;
        if (tile < base_tile) base_b = base_tile = 0;  // blocks come in order, as a rule
        while (base_b < p.B) {
          const int b = base_b + lane;
          int q0 = 0, nq = 0;
          if (b < p.B) {
            q0 = clamp_at(p.cu_q, b, p.Tq);
            nq = max(0, clamp_at(p.cu_q, b + 1, p.Tq) - q0);
          }
          const int tiles = (nq + span - 1) / span;
          int incl = tiles;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          const unsigned behind = __ballot_sync(0xffffffffu, tile < base_tile + incl);
          if (behind) {
            const int src = __ffs(behind) - 1;
            const int before = __shfl_sync(0xffffffffu, incl - tiles, src) + base_tile;
            const int n = __shfl_sync(0xffffffffu, tiles, src);
            u.q0 = __shfl_sync(0xffffffffu, q0, src);
            u.nq = __shfl_sync(0xffffffffu, nq, src);
            u.m = (n - 1 - (tile - before)) * span;  // the rows with the most keys first
            u.k0 = clamp_at(p.cu_k, base_b + src, p.Tk);
            u.nk = max(0, clamp_at(p.cu_k, base_b + src + 1, p.Tk) - u.k0);
            break;
          }
          base_tile += __shfl_sync(0xffffffffu, incl, 31);
          base_b += 32;
        }
        if (u.nq >= 0) break;
        // behind the last tile (the grid is an upper bound): take the rest of the
        // blocks off the queue, so that none starts only to find nothing
        ask();
        ok = answered();
      }
      if (!ok) break;
      const int slot = it & 1;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_sleep(smem_u32(&uempty_bar[slot]), ((it >> 1) & 1) ^ 1u, abort_flag,
                                      p.err, kErrWaitProducer, lim));
      if (!ok) break;
      if (lane == 0) {
        units[slot] = u;
        mbar_arrive(smem_u32(&ufull_bar[slot]));
      }
      __syncwarp();
      if (u.nq < 0 || p.stall_loads) break;
      ask();
      const PromptTiles t(p, u);
      if (t.n_max > 0 && lane == 0) {
        ok = mbar_wait_sleep(smem_u32(qempty_bar), (q_loads & 1) ^ 1u, abort_flag, p.err,
                             kErrWaitProducer, lim);
        if (ok) {
          const uint32_t qb = smem_u32(qfull_bar);
          mbar_arrive_expect_tx(qb, 2 * S::kTileBytes);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            for (int c = 0; c < S::kBlocks; ++c)
              tma_load_3d(smem_u32(q_tiles) + i * S::kTileBytes + c * S::kBlockBytes, &qmap, qb,
                          c * 64, t.head[i], u.q0 + t.row0[i]);
          ++q_loads;
        }
        const int kv_head = t.head[0] / p.group;
        for (int j = 0; j < 2 * t.n_max && ok; ++j) {
          const int s = issued % S::kStages;
          ok = mbar_wait_sleep(smem_u32(&empty_bar[s]), ((issued / S::kStages) & 1) ^ 1u,
                               abort_flag, p.err, kErrWaitProducer, lim);
          if (!ok) break;
          const uint32_t fb = smem_u32(&full_bar[s]);
          mbar_arrive_expect_tx(fb, S::kTileBytes);
          for (int c = 0; c < S::kBlocks; ++c)
            tma_load_3d(smem_u32(ring) + s * S::kTileBytes + c * S::kBlockBytes,
                        j & 1 ? &vmap : &kmap, fb, c * 64, kv_head, u.k0 + (j >> 1) * kAttnN);
          ++issued;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || !answered()) break;
    }
    if (lane == 0) {
      // no copy, and no arrival of a product's completion, is under way when the
      // CTA exits, whatever the other roles did
      auto settle = [&](uint64_t* bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(bar), parity)) {
          if (globaltimer_ns() - t0 > lim) {
            atomicOr(p.err, kErrDrain);
            return;
          }
        }
      };
      if (asked > 0) settle(ask_bar, (asked - 1) & 1);
      if (q_loads > 0) settle(qfull_bar, (q_loads - 1) & 1);
      for (int q = max(0, issued - static_cast<int>(S::kStages)); q < issued; ++q)
        settle(&full_bar[q % S::kStages], (q / S::kStages) & 1);
      if (!*abort_flag) {
        if (q_loads > 0) settle(qempty_bar, (q_loads - 1) & 1);
        for (int q = max(0, issued - static_cast<int>(S::kStages)); q < issued; ++q)
          settle(&empty_bar[q % S::kStages], (q / S::kStages) & 1);
      }
    }
  } else if (warp == kAttnMmaWarp) {
    // ---------------------------------------------------------- products
    const int dsteps = (p.d + 15) / 16;
    const uint64_t q_desc = make_sdesc(smem_u32(q_tiles), 64);
    const uint64_t k_desc = make_sdesc(smem_u32(ring), 64);
    const uint64_t v_desc = make_vdesc(smem_u32(ring));
    bool ok = true, any = false;
    int used = 0, q_used = 0;       // loads taken so far
    int turns[2] = {0, 0};          // score tiles made so far per query tile
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, p.err,
                                                   kErrWaitMma, lim));
      return ok;
    };
    auto slot_of = [&](int x) { return x % S::kStages; };
    auto phase_of = [&](int x) { return static_cast<uint32_t>((x / S::kStages) & 1); };
    PromptUnit u;
    for (int it = 0; ok && take_unit(it, kErrWaitMma, u); ++it) {
      const PromptTiles t(p, u);
      if (t.n_max == 0) continue;
      auto scores = [&](int i, int slot) {  // S_i = Q_i K^T
        const uint64_t a = q_desc + static_cast<uint64_t>(i * (S::kTileBytes >> 4));
        const uint64_t b = k_desc + static_cast<uint64_t>(slot * (S::kTileBytes >> 4));
        for (int k = 0; k < dsteps; ++k) {
          const uint32_t at = (k >> 2) * (S::kBlockBytes >> 4) + (k & 3) * 2;
          umma_f16_warp(tmem + i * kAttnN, a + at, b + at, p.idesc_s, k > 0);
        }
        umma_commit_warp(smem_u32(&s_bar[i]));
        any = true;
      };
      if (!wait(qfull_bar, q_used & 1) || !wait(&full_bar[slot_of(used)], phase_of(used))) break;
      ++q_used;
      tc_fence_after();
      // the scores may overwrite the last unit's probabilities: the tensor pipe
      // works in order
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (t.n[i] > 0) scores(i, slot_of(used));
      umma_commit_warp(smem_u32(&empty_bar[slot_of(used)]));
      if (t.n_max == 1) umma_commit_warp(smem_u32(qempty_bar));
      __syncwarp();
      for (int j = 0; j < t.n_max && ok; ++j) {
        const int kx = used + 2 * j + 2, vx = used + 2 * j + 1, vs = slot_of(vx);
        if (!wait(&full_bar[vs], phase_of(vx))) break;
        const int left = u.nk - j * kAttnN;
        if (left < kAttnN) {
          // rows behind the last key belong to other sequences: whatever they
          // hold, their probabilities are 0 and 0 * NaN must not reach the sum
          uint8_t* vt = ring + vs * S::kTileBytes;
          const int chunks = (kAttnN - left) * 8;
          for (int c = 0; c < S::kBlocks; ++c)
            for (int e = lane; e < chunks; e += 32)
              *reinterpret_cast<uint4*>(vt + c * S::kBlockBytes + left * 128 + e * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        bool k_ready = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (j >= t.n[i]) continue;
          if (!wait(&p_bar[i], (turns[i] + j) & 1)) break;
          // the last unit's output must have been read before this one's begins
          if (j == 0 && it > 0 && !wait(&ofree_bar[i], (it - 1) & 1)) break;
          tc_fence_after();
          const uint64_t b = v_desc + static_cast<uint64_t>(vs * (S::kTileBytes >> 4));
#pragma unroll
          for (int k = 0; k < kAttnN / 16; ++k)  // 16 keys: 8 columns of P, 2048 bytes of V
            umma_f16_ts_warp(tmem + 2 * kAttnN + i * kDP, tmem + i * kAttnN + k * 8,
                             b + static_cast<uint64_t>(k * (2048 >> 4)), p.idesc_o,
                             (j > 0 || k > 0) ? 1u : 0u);
          if (j + 1 < t.n[i]) {
            if (!k_ready) {
              if (!wait(&full_bar[slot_of(kx)], phase_of(kx))) break;
              k_ready = true;
              tc_fence_after();
            }
            scores(i, slot_of(kx));
          } else {
            umma_commit_warp(smem_u32(&o_bar[i]));
          }
          __syncwarp();
        }
        if (!ok) break;
        umma_commit_warp(smem_u32(&empty_bar[vs]));
        if (j + 1 < t.n_max) umma_commit_warp(smem_u32(&empty_bar[slot_of(kx)]));
        if (j + 2 == t.n_max) umma_commit_warp(smem_u32(qempty_bar));
        __syncwarp();
      }
      used += 2 * t.n_max;
      turns[0] += t.n[0];
      turns[1] += t.n[1];
    }
    if (*abort_flag && any) {
      // let every product issued finish before tensor memory is released
      umma_commit_warp(smem_u32(drain_bar));
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(drain_bar), 0)) {
        if (globaltimer_ns() - t0 > lim) {
          if (lane == 0) atomicOr(p.err, kErrDrain);
          break;
        }
      }
    }
  }
  } else {
    // ----------------------------------------------------------- softmax
    regs_take<kAttnRegsSoftmax>();
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;     // row of the tile
    const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_at + i * kAttnN;
    const uint32_t o_at = tmem + lane_at + 2 * kAttnN + i * kDP;
    int turns = 0, outs = 0;                  // score tiles and outputs taken so far
    bool ok = true;
    PromptUnit u;
    for (int it = 0; take_unit(it, kErrWaitEpilogue, u); ++it) {
      const PromptTiles t(p, u);
      const int n = i ? t.n[1] : t.n[0], head = i ? t.head[1] : t.head[0];
      const int row0 = i ? t.row0[1] : t.row0[0];
      const int row = row0 + r;               // row of the sequence
      const int seen = p.causal ? min(u.nk, row + t.shift + 1) : u.nk;  // keys of this row
      const int seen_all = p.causal ? min(u.nk, row0 + t.shift + 1) : u.nk;  // of every row
      float m = kNegInf, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if (!mbar_wait(smem_u32(&s_bar[i]), (turns + j) & 1, abort_flag, p.err, kErrWaitEpilogue,
                       lim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, s[c]);
        tmem_wait_ld_regs(s[0]);
#pragma unroll
        for (int c = 1; c < 4; ++c) reg_fence(s[c]);
        if ((j + 1) * kAttnN > seen_all) {
          const int lim_col = seen - j * kAttnN;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= lim_col) s[c][e] = kNegInf;
        }
        const float x = fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
        if (j == 0) {
          m = x;
        } else {
          const bool grow = (x - m) * p.c > kAttnSlack;  // also from -inf to a number
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? exp2_approx((m - x) * p.c) : 1.f;
            if (grow) m = x;
            l *= f;
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
        const float z = (m == kNegInf ? 0.f : m * p.c) - kBias;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = exp2_approx(fmaf(s[c][2 * e], p.c, -z));
            const float b = exp2_approx(fmaf(s[c][2 * e + 1], p.c, -z));
            sum[e & 3] += a + b;
            // the second product takes the probabilities in the value type
            // (half a step: 2^-9 of bf16, 2^-12 of fp16, of each weight); the
            // total keeps them in fp32
            w[e] = pack2<kBf16>(a, b);
          }
          tmem_st16(s_at + c * 16, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_bar[i]));
      }
      if (n > 0 && ok) {
        ok = mbar_wait(smem_u32(&o_bar[i]), outs & 1, abort_flag, p.err, kErrWaitEpilogue, lim);
        ++outs;
        turns += n;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const bool live = row < u.nq;
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint16_t* ob = p.out + static_cast<int64_t>(u.q0 + row) * p.o_ts + head * p.o_hs;
#pragma unroll
      for (int c = 0; c < kDP / 32; ++c) {
        float o[32];
        if (n > 0) {
          tmem_ld32(o_at + c * 32, o);
          tmem_wait_ld_regs(o);
        }
        if (c == kDP / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ofree_bar[i]));
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int col = c * 32 + h * 8;
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = l > 0.f ? pack2<kBf16>(o[h * 8 + 2 * e] * inv, o[h * 8 + 2 * e + 1] * inv) : 0u;
          if (live && col < p.d)
            *reinterpret_cast<uint4*>(ob + col) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (live && p.lse)
        p.lse[static_cast<int64_t>(u.q0 + row) * p.Hq + head] =
            l > 0.f ? m * p.scale + (log2f(l) - kBias) * 0.69314718f : kNegInf;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace rnn
