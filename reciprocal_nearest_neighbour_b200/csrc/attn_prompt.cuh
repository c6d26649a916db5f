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
//                   the probabilities (tcgen05.st) as the 16-bit A operand of
//                   the second product
//   warps 8, 10     issue S = Q K^T and O += P V (tcgen05.mma) of query tile 0 and
//                   1; each wait and commit costs the issuing warp over a hundred
//                   cycles, and one warp for both tiles bounds the kernel
//   warp 9          TMA: query tiles, then a ring of alternating K and V tiles
//   warps 12-15     outputs: normalise and store a finished unit's rows
// Tensor memory: two score tiles of 128 columns, two output tiles of kDP, and with
// 64 channels two probability tiles (AttnShape).
//
// A CTA is persistent.  The grid has one block per unit (a pair of query
// tiles); a running CTA asks for the next unit by cancelling a block that has
// not started (clusterlaunchcontrol), so units of any length are dealt as CTAs
// come free, without a counter to clear.  The TMA warp fetches the next unit and
// its tiles, and the output warps read, normalise and store a finished unit's
// rows, while the products and the softmax of the one in between run.
//
// Rescaling.  A row's reference maximum only moves when its true maximum has
// grown by more than 2^8 over it (a weight is then at most 2^8; in fp16, where all
// weights carry a factor of 2^7 against its short range below 1, 2^15 of the 2^16
// that the type holds), so the output accumulator is read back and rescaled
// rarely; the softmax warps do it themselves.  At 128 channels the next scores are
// only made when the product before them is complete, so their barrier tells both;
// at 64 they come earlier, and the softmax warps look at the output's barrier.
//
// Bound: 4*128*128*d flops and 128*128 exponentials per query tile and key tile;
// at d = 128 the two take the same time on an SM (16 exponentials, 8192 flops a
// cycle), at d = 64 the exponentials take twice as long as the products.
// Measured (32/8 heads, bf16, in a CUDA graph): 2 x 8192 tokens, full, 128 channels
// 1.85 ms, 1.19 PFLOP/s, 0.74 of the library product's burst rate; 64 channels 1.44 ms,
// 0.76 PFLOP/s, 0.64 of the exponentials' rate at 1965 MHz; one causal prompt of 16384
// tokens of 128 channels 1.85 to 1.95 ms with the power limit, 2.15 ms call after call.
#pragma once
#include <cstdint>
#include <cuda.h>
#include "ptx.cuh"
#include "nn_kernel.cuh"
#include "warp_mma.cuh"

namespace rnn {

constexpr int kAttnM = 128;            // query rows per tile
constexpr int kAttnN = 128;            // keys per tile
constexpr int kAttnThreads = 512;      // four warpgroups; warp 11 only completes the third
// Registers: launched with 128 a thread, the softmax warps hold 128 scores each
// and take what the other groups give up: 256 * 176 + 256 * 80 = 512 * 128.
constexpr int kAttnRegsSoftmax = 176, kAttnRegsOther = 80;
constexpr int kAttnMmaWarp = 8, kAttnTmaWarp = 9, kAttnMmaWarp2 = 10,
              kAttnOutWarp = 12;
constexpr float kAttnSlack = 8.f;      // log2 growth of the maximum before a rescale
// Scaled log2 scores beyond this lose their exponents' last bits (a sixteenth and more)
// where the reference is taken off behind the scaling, and at 2^128 all of it; it is
// taken off before for such rows.
constexpr float kAttnFar = 1048576.f;
// Calls with more keys take the kernel's kLong form.  Up to this many, a unit has 512
// steps at most, about a millisecond, and what the accumulator cuts off (n 2^-27 of a
// sum of n weights of one size) stays below 2^-11, half a step of fp16.  Below the border
// the kLong form takes 108 us for 24 frames of 768 tokens (16 heads of 64; 106), 280 for
// 20 causal prompts of 17 to 4001 tokens (32/8 heads of 128; 265).  Calls with very many
// sequences or blocks take it too: the search for the next unit goes past 10 sequences
// without rows, or 3 blocks without a tile, in a microsecond.
constexpr int64_t kAttnShortKeys = 65536, kAttnFewSeqs = 1 << 20, kAttnFewUnits = 1 << 24;
// In the kLong form a row's sums leave the accumulator this often, every 65536 keys.
constexpr int kAttnHoldSteps = 512;

template <int kDP>
struct AttnShape {
  static constexpr int kBlocks = kDP / 64;               // 64-channel column blocks
  static constexpr int kTileBytes = kAttnM * kDP * 2;
  static constexpr int kBlockBytes = kAttnM * 128;
  static constexpr int kStages = kDP == 128 ? 4 : 8;
  static constexpr int kStoreBytes = 32 * 128;           // a warp's rows, 64 channels at a time
  static constexpr size_t kSmem = 1024 + size_t(2 + kStages) * kTileBytes + 4 * kStoreBytes +
                                  2048 + 512;
  // Tensor-memory columns: scores at 0 and 128, outputs at 256.  With 64
  // channels the probabilities have columns of their own behind the outputs, so
  // the next scores are made while these are exponentiated; with 128 they lie
  // over the scores, and go to the second product in two halves, so that it
  // starts while the second half is exponentiated.
  static constexpr bool kOwnP = kDP == 64;
  static constexpr int kOutCol = 2 * kAttnN;
  static constexpr int kProbCol = kOwnP ? kOutCol + 2 * kDP : 0;
  static constexpr int kProbStep = kOwnP ? kAttnN / 2 : kAttnN;  // between the two tiles
  static constexpr int kParts = kOwnP ? 1 : 2;
};
// Looks at the other warp's count, 40 ns apart, before going on anyway, and the
// 32-column chunk behind which a warp hands over.  2 x 8192 tokens, full: 64 channels
// 1.44 ms behind the third chunk, 1.50 behind the second, 1.60 behind the last and
// 1.53 without turns; 128 channels 1.84, 1.98, 1.85 and 2.00 ms.
constexpr int kTurnPolls = 100, kTurnChunk = 2;

struct PromptParams {
  const int32_t *cu_q, *cu_k;
  uint16_t* out;
  float* lse;                  // [Tq][Hq] or null
  int64_t o_ts, o_hs, Tq, Tk;  // strides in elements
  int B, Hq, group, d;
  int pair_heads;              // the two tiles are heads 2u, 2u + 1 of the same tokens
  int head_units;              // Hq / 2 or Hq
  int causal;
  int sort;                    // more units than SMs: the order of the units matters
  float scale, c;              // c = scale * log2(e)
  uint32_t idesc_s, idesc_o;   // instruction descriptors of the two products
  int* err;                    // status word or null
  unsigned long long wait_limit_ns;
  int stall_loads;
};

// Four depth steps of D (+)= A B^T with one election: 64 channels of S = Q K^T
// (both operands in shared memory, 32 bytes apart), or 64 keys of O += P V (A in
// tensor memory, 8 columns apart; B 2048 bytes apart).  Issued one by one, each
// with its own election, a product instruction costs its warp over a hundred
// cycles, and the issuing warp bounds the kernel.
__device__ __forceinline__ void umma_ss_x4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_ts_x4(uint32_t d_tmem, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
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
// 16 columns, complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
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

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t f2_make(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A load that nothing waits for.
__device__ __forceinline__ void touch(const int32_t* at) {
  asm volatile("{\n\t.reg .s32 v;\n\tld.global.nc.s32 v, [%0];\n\t}" ::"l"(at));
}

// Shared memory by 32-bit address.
__device__ __forceinline__ int lds_volatile(uint32_t at) {
  int v;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts_volatile(uint32_t at, int v) {
  asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_f2(uint32_t at, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float2 lds_f2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
// A count, with the writes before it.
__device__ __forceinline__ void st_release(uint32_t at, int v) {
  asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_acquire(uint32_t at) {
  int v;
  asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

template <int kRegs>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Wait for what must not be under way when the CTA exits.  It gives up when the limit
// has passed and 64 more looks, 20 us each, were in vain: a CTA that was itself stopped
// for that long (its GPU taken by another process) has time of its own first.
__device__ __forceinline__ bool settle_phase(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                             int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  int late = 0;
#pragma unroll 1
  while (!mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (globaltimer_ns() - t0 > limit_ns && ++late > 64) {
      if (err) atomicOr(err, kErrDrain);
      return false;
    }
  }
  return true;
}

// kLong: more than kAttnShortKeys keys in the call, so that a unit may last any time, and
// its sums may lose their small terms: the tensor pipe cuts what it adds off at the
// accumulator's last bits instead of rounding it (2^20 equal weights lost 0.7 % of a sum
// of values of one sign, 2.5 10^8 of them three quarters).  There a softmax warp takes
// its rows out of the accumulator every kAttnHoldSteps steps and adds them up itself,
// rounded to nearest, in local memory.  Also with more than kAttnFewSeqs sequences or
// kAttnFewUnits units, where the search for the next unit may last as long.
template <bool kBf16, int kDP, bool kLong>
__global__ void __launch_bounds__(kAttnThreads, 1)
attn_prompt_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap) {
  using S = AttnShape<kDP>;
  constexpr float kBias = kBf16 ? 0.f : 7.f;
  // with 0.6 for the exponent's rounding up to kAttnFar
  static_assert(kBias + kAttnSlack + 0.6f < 15.99f, "weights have to stay inside fp16");
  constexpr int kUnitReaders = 14;  // softmax, MMA and output warps
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // Shared memory by 32-bit addresses: one base, everything else a constant away.
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t q_tiles = smem;
  const uint32_t ring = smem + 2 * S::kTileBytes;
  const uint32_t staging = ring + S::kStages * S::kTileBytes;
  const uint32_t row_ml = staging + 4 * S::kStoreBytes;  // float2 [2][128]
  const uint32_t bars = row_ml + 2 * kAttnM * 8;
  const uint32_t full_bar = bars;
  const uint32_t empty_bar = full_bar + 8 * S::kStages;
  const uint32_t qfull_bar = empty_bar + 8 * S::kStages;
  const uint32_t qempty_bar = qfull_bar + 8;
  const uint32_t s_bar = qempty_bar + 8;    // scores of tile i are in tensor memory
  const uint32_t sfree_bar = s_bar + 16;    // its scores are in registers (kOwnP)
  const uint32_t p_bar = sfree_bar + 16;    // its probabilities are there, by parts
  const uint32_t o_bar = p_bar + 32;        // its output is complete so far
  const uint32_t ofree_bar = o_bar + 16;    // its output has been read
  const uint32_t ufull_bar = ofree_bar + 16;
  const uint32_t uempty_bar = ufull_bar + 16;
  const uint32_t ml_bar = uempty_bar + 16;  // its rows' maxima and totals are there
  const uint32_t mlfree_bar = ml_bar + 16;  // and have been read
  const uint32_t ask_bar = mlfree_bar + 16;
  const uint32_t drain_bar = ask_bar + 8;
  const uint32_t tmem_slot = drain_bar + 16;
  const uint32_t abort_at = tmem_slot + 4;
  // counts that only grow, where a reader may be any number of steps behind
  const uint32_t zero_at = tmem_slot + 8;   // ragged V tiles whose end is zeroed
  const uint32_t turn_at = tmem_slot + 16;  // per softmax warp: steps whose exponentials are out
  const uint32_t search_at = turn_at + 32;  // groups and blocks looked at for units (kLong)
  __shared__ __align__(16) uint8_t answer[16];
  // Units published in turn (two at a time, and those before them as long as an output
  // warp may have them in hand), how many so far, and one that was taken and not published.
  __shared__ PromptUnit units[4], unpublished;
  __shared__ int dealt;
  // What an output warp has not written when it stops: unit number x and, if y is below
  // 2, the tiles of the unit before it from tile y on.
  __shared__ int2 unwritten[4];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Waits.  A lane's outcome is its own; the warp votes before it acts on one.  They
  // suspend the warp: spinning ones take issue slots from the softmax warps of the same
  // scheduler (128 channels: a tenth slower).  The limits are read from the parameters
  // where they are needed, so that no register holds them, nor an address of a barrier,
  // through the loops.
  auto aborted = [&]() { return lds_volatile(abort_at) != 0; };
  auto give_up = [&](int code) {
    sts_volatile(abort_at, 1);
    if (p.err) atomicOr(p.err, code);
  };
  // Most last a step or two.  `whole_unit` marks those that last as long as a unit has
  // keys, or as the search for the next one: where that may be long, their limit counts
  // from the last step that a tile's first softmax warp, or the search, has done.
  auto wait = [&](uint32_t bar, uint32_t parity, int code, bool whole_unit = false) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    uint64_t t0 = globaltimer_ns();
    int steps = 0;
#pragma unroll 1
    while (true) {
      if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
      if (aborted()) return false;
      if (kLong && whole_unit) {
        const int now =
            lds_volatile(turn_at) + lds_volatile(turn_at + 16) + lds_volatile(search_at);
        if (now != steps) t0 = globaltimer_ns();
        steps = now;
      }
      if (globaltimer_ns() - t0 > p.wait_limit_ns) {
        give_up(code);
        return false;
      }
    }
  };
  if (threadIdx.x < S::kStages) {
    mbar_init(full_bar + 8 * threadIdx.x, 1);
    mbar_init(empty_bar + 8 * threadIdx.x, 2);
    fence_barrier_init();
  } else if (threadIdx.x >= 32 && threadIdx.x < 34) {
    const int i = threadIdx.x - 32;
    mbar_init(s_bar + 8 * i, 1);
    mbar_init(sfree_bar + 8 * i, 4);
    mbar_init(p_bar + 8 * i, 4);
    mbar_init(p_bar + 8 * (2 + i), 4);
    mbar_init(o_bar + 8 * i, 1);
    fence_barrier_init();
  } else if (threadIdx.x >= 64 && threadIdx.x < 66) {
    const int i = threadIdx.x - 64;
    mbar_init(ofree_bar + 8 * i, 4);
    mbar_init(ml_bar + 8 * i, 4);
    mbar_init(mlfree_bar + 8 * i, 4);
    mbar_init(ufull_bar + 8 * i, 1);
    mbar_init(uempty_bar + 8 * i, kUnitReaders);
    mbar_init(drain_bar + 8 * i, 1);
    fence_barrier_init();
  } else if (threadIdx.x == 96) {
    mbar_init(qfull_bar, 1);
    mbar_init(qempty_bar, 2);
    mbar_init(ask_bar, 1);
    fence_barrier_init();
  } else if (threadIdx.x >= 128 && threadIdx.x < 136) {
    sts_volatile(turn_at + 4 * (threadIdx.x - 128), 0);
    if (threadIdx.x == 128) {
      sts_volatile(zero_at, 0);
      sts_volatile(abort_at, 0);
      if (kLong) sts_volatile(search_at, 0);
      dealt = 0;
      unpublished.nq = -1;
    }
  }
  constexpr uint32_t kCols = 512;
  if (warp == kAttnMmaWarp) {
    tmem_alloc(tmem_slot, kCols);
    tmem_relinquish();
  }
  if (warp == kAttnTmaWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&qmap);
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    if (lane <= p.B) {  // the first offsets, into the cache under the set-up
      touch(p.cu_q + lane);
      touch(p.cu_k + lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_volatile(tmem_slot);

  // Unit number `it` of this CTA, as the TMA warp published it.
  auto take_unit = [&](int it, int code, PromptUnit& u) {
    const int slot = it & 1;
    if (!__all_sync(0xffffffffu, wait(ufull_bar + 8 * slot, (it >> 1) & 1, code, true)))
      return false;
    u = units[it & 3];
    __syncwarp();
    if (lane == 0) mbar_arrive(uempty_bar + 8 * slot);
    return u.nq >= 0;
  };

  if (warp >= kAttnMmaWarp) {
    regs_give<kAttnRegsOther>();
    if (warp == kAttnTmaWarp) {
      // ------------------------------------------------- units and loads
      const int span = p.pair_heads ? kAttnM : 2 * kAttnM;  // tokens per unit
      // The sequences in groups of 32, the lanes of this warp: a group's are dealt
      // longest keys first, so that the last units are short ones.
      int base_b = 0, base_tile = 0, loaded = -1;
      int g_q0 = 0, g_nq = 0, g_k0 = 0, g_nk = 0, g_tiles = 0, g_incl = 0;
      auto load_group = [&]() {
        const int b = base_b + lane;
        int q0 = 0, nq = 0, k0 = 0, nk = -1;
        if (b < p.B) {
          q0 = clamp_at(p.cu_q, b, p.Tq);
          nq = max(0, clamp_at(p.cu_q, b + 1, p.Tq) - q0);
          k0 = clamp_at(p.cu_k, b, p.Tk);
          nk = max(0, clamp_at(p.cu_k, b + 1, p.Tk) - k0);
        }
        const int members = min(32, p.B - base_b);
        int src = lane;
        if (p.sort) {
          int rank = 0;
          for (int o = 0; o < members; ++o) {
            const int x = __shfl_sync(0xffffffffu, nk, o);
            rank += x > nk || (x == nk && o < lane);
          }
          for (int o = 0; o < members; ++o)
            if (__shfl_sync(0xffffffffu, rank, o) == lane) src = o;
        }
        g_q0 = __shfl_sync(0xffffffffu, q0, src);
        g_nq = __shfl_sync(0xffffffffu, nq, src);
        g_k0 = __shfl_sync(0xffffffffu, k0, src);
        g_nk = __shfl_sync(0xffffffffu, nk, src);
        g_tiles = lane < members ? (g_nq + span - 1) / span : 0;
        g_incl = g_tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, g_incl, o);
          if (lane >= o) g_incl += y;
        }
        loaded = base_b;
      };
      int block = blockIdx.x, issued = 0, q_loads = 0;
      int asked = 0, searched = 0;
      bool ok = true;
      // (not cut short by an abort: a block that was handed over will not start)
      auto answered = [&]() {
        if (!__all_sync(0xffffffffu,
                        settle_phase(ask_bar, (asked - 1) & 1, p.wait_limit_ns, p.err))) {
          give_up(kErrWaitProducer);
          return false;
        }
        block = next_block_read(smem_u32(answer));
        fence_proxy_async_smem();  // read before the next answer is written
        __syncwarp();
        return true;
      };
      auto ask = [&]() {
        if (lane == 0) {
          mbar_arrive_expect_tx(ask_bar, 16);
          next_block_request(smem_u32(answer), ask_bar);
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
            if (kLong && lane == 0) sts_volatile(search_at, ++searched);
            if (loaded != base_b) load_group();
            const unsigned behind = __ballot_sync(0xffffffffu, tile < base_tile + g_incl);
            if (behind) {
              const int src = __ffs(behind) - 1;
              const int before = __shfl_sync(0xffffffffu, g_incl - g_tiles, src) + base_tile;
              const int n = __shfl_sync(0xffffffffu, g_tiles, src);
              u.q0 = __shfl_sync(0xffffffffu, g_q0, src);
              u.nq = __shfl_sync(0xffffffffu, g_nq, src);
              u.k0 = __shfl_sync(0xffffffffu, g_k0, src);
              u.nk = __shfl_sync(0xffffffffu, g_nk, src);
              u.m = (n - 1 - (tile - before)) * span;  // the rows with the most keys first
              break;
            }
            base_tile += __shfl_sync(0xffffffffu, g_incl, 31);
            base_b += 32;
          }
          if (u.nq >= 0) break;
          // behind the last tile (the grid is an upper bound): take the rest of the
          // blocks off the queue, so that none starts only to find nothing
          if (kLong && lane == 0) sts_volatile(search_at, ++searched);
          ask();
          ok = answered();
        }
        if (!ok) break;
        const int slot = it & 1;
        ok = __all_sync(0xffffffffu,
                        wait(uempty_bar + 8 * slot, ((it >> 1) & 1) ^ 1u, kErrWaitProducer));
        if (!ok) {
          if (lane == 0) unpublished = u;
          break;
        }
        if (lane == 0) {
          units[it & 3] = u;
          dealt = it + 1;
          mbar_arrive(ufull_bar + 8 * slot);
        }
        __syncwarp();
        if (u.nq < 0 || (p.stall_loads && it + 1 >= p.stall_loads)) break;
        const PromptTiles t(p, u);
        if (t.n_max > 0 && lane == 0) {
          ok = wait(qempty_bar, (q_loads & 1) ^ 1u, kErrWaitProducer);
          if (ok) {
            const uint32_t qb = qfull_bar;
            mbar_arrive_expect_tx(qb, 2 * S::kTileBytes);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              for (int c = 0; c < S::kBlocks; ++c)
                tma_load_3d(q_tiles + i * S::kTileBytes + c * S::kBlockBytes, &qmap, qb,
                            c * 64, t.head[i], u.q0 + t.row0[i]);
            ++q_loads;
          }
          const int kv_head = t.head[0] / p.group;
          for (int j = 0; j < 2 * t.n_max && ok; ++j) {
            const int s = issued % S::kStages;
            ok = wait(empty_bar + 8 * s, ((issued / S::kStages) & 1) ^ 1u, kErrWaitProducer);
            if (!ok) break;
            const uint32_t fb = full_bar + 8 * s;
            mbar_arrive_expect_tx(fb, S::kTileBytes);
            for (int c = 0; c < S::kBlocks; ++c)
              tma_load_3d(ring + s * S::kTileBytes + c * S::kBlockBytes,
                          j & 1 ? &vmap : &kmap, fb, c * 64, kv_head, u.k0 + (j >> 1) * kAttnN);
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // only now, a ring's length before the unit ends: a unit asked for early
        // would wait here while other CTAs run out of work
        ask();
        if (!answered()) break;
      }
      // no copy, and no arrival of a product's completion, is under way when the CTA
      // exits, whatever the other roles did; a lane for each barrier
      {
        issued = __shfl_sync(0xffffffffu, issued, 0);
        q_loads = __shfl_sync(0xffffffffu, q_loads, 0);
        constexpr int kEmpty = 3 + S::kStages;  // the first lane of the freed places
        static_assert(kEmpty + S::kStages <= 32, "");
        uint32_t bar = lane == 0 ? ask_bar : lane == 1 ? qfull_bar : qempty_bar;
        int phase = (lane == 0 ? asked : q_loads) - 1;
        if (lane >= 3) {
          const bool empty = lane >= kEmpty;
          const int x = max(0, issued - static_cast<int>(S::kStages)) + lane - (empty ? kEmpty : 3);
          bar = (empty ? empty_bar : full_bar) + 8 * (x % S::kStages);
          phase = x < issued ? x / S::kStages : -1;
        }
        // after an abort nobody may free the rest
        if (phase >= 0 && !((lane == 2 || lane >= kEmpty) && aborted()))
          settle_phase(bar, phase & 1, p.wait_limit_ns, p.err);
        __syncwarp();
      }
    } else if (warp == kAttnMmaWarp || warp == kAttnMmaWarp2) {
      // ---------------------------------------------------------- products
      const int i = warp == kAttnMmaWarp ? 0 : 1;  // this warp's query tile
      const int dsteps = (p.d + 15) / 16;
      const uint64_t q_desc = make_sdesc(q_tiles + i * S::kTileBytes, 64);
      const uint64_t k_desc = make_sdesc(ring, 64);
      const uint64_t v_desc = make_vdesc(ring);
      bool ok = true, any = false;
      int used = 0, q_used = 0;       // loads taken so far
      int turns = 0;                  // score tiles made so far
      int zeroed = 0;                 // ragged V tiles so far
      auto wait_mma = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, wait(bar, parity, kErrWaitMma));
        return ok;
      };
      auto slot_of = [&](int x) { return x % S::kStages; };
      auto wait_load = [&](int x) {
        return wait_mma(full_bar + 8 * slot_of(x), (x / S::kStages) & 1);
      };
      // this warp is done with a buffer: when its products so far are, or at once
      auto release = [&](uint32_t bar, bool behind_products) {
        if (behind_products)
          umma_commit_warp(bar);
        else if (lane == 0)
          mbar_arrive(bar);
      };
      auto scores = [&](int slot) {  // S_i = Q_i K^T
        const uint64_t k_at = k_desc + static_cast<uint64_t>(slot * (S::kTileBytes >> 4));
        // a last block with 16, 32 or 48 channels takes single steps
        const int whole = dsteps >> 2;
#pragma unroll
        for (int c = 0; c < S::kBlocks; ++c) {
          const uint32_t at = c * (S::kBlockBytes >> 4);
          if (c < whole) {
            umma_ss_x4(tmem + i * kAttnN, q_desc + at, k_at + at, p.idesc_s, c > 0);
          } else {
            for (int k = 0; k < dsteps - 4 * c; ++k)
              umma_f16_warp(tmem + i * kAttnN, q_desc + at + 2 * k, k_at + at + 2 * k, p.idesc_s,
                            c > 0 || k > 0);
          }
        }
        umma_commit_warp(s_bar + 8 * i);
        any = true;
      };
      // Where the probabilities lie over the scores, the product that reads them has to be
      // complete before other scores are made there: two products with different outputs
      // are not promised to run in the order of their issue.  Issued without this wait,
      // the 20 causal prompts of 17 to 4001 tokens took 250 us where this form took 266;
      // scores in two products of 64 keys, of which only the second waits, 284 us.
      auto product_done = [&](int step) {
        ok = ok && __all_sync(0xffffffffu, mbar_try_wait(o_bar + 8 * i, step & 1) ||
                                               wait(o_bar + 8 * i, step & 1, kErrWaitMma));
        return ok;
      };
      PromptUnit u;
      for (int it = 0; ok && take_unit(it, kErrWaitMma, u); ++it) {
        const PromptTiles t(p, u);
        const int n = i ? t.n[1] : t.n[0];
        // the last unit's output must have been read before this one's begins (its
        // scores may go first); waited for at every unit, so that the parity is
        // that of the last one
        auto outputs_free = [&]() { return it == 0 || wait_mma(ofree_bar + 8 * i, (it - 1) & 1); };
        if (n == 0 && !outputs_free()) break;
        if (t.n_max == 0) continue;
        if (!wait_mma(qfull_bar, q_used & 1) || !wait_load(used)) break;
        ++q_used;
        tc_fence_after();
        if (!S::kOwnP && n > 0 && turns > 0 && !product_done(turns - 1)) break;
        if (n > 0) scores(slot_of(used));
        release(empty_bar + 8 * slot_of(used), n > 0);
        if (n <= 1) release(qempty_bar, n == 1);
        __syncwarp();
        for (int j = 0; j < t.n_max; ++j) {
          const int kx = used + 2 * j + 2, vx = used + 2 * j + 1, vs = slot_of(vx);
          if (!wait_load(vx)) break;
          const int left = u.nk - j * kAttnN;
          if (left < kAttnN) {
            // rows behind the last key belong to other sequences: whatever they
            // hold, their probabilities are 0 and 0 * NaN must not reach the sum
            if (i == 0) {
              const uint32_t vt = ring + vs * S::kTileBytes + left * 128;
              const int chunks = (kAttnN - left) * 8;
              for (int c = 0; c < S::kBlocks; ++c)
                for (int e = lane; e < chunks; e += 32)
                  sts_v4(vt + c * S::kBlockBytes + e * 16, make_uint4(0, 0, 0, 0));
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) st_release(zero_at, zeroed + 1);
            } else {
              const uint64_t t0 = globaltimer_ns();
              while (ld_acquire(zero_at) <= zeroed) {
                if (!aborted() && globaltimer_ns() - t0 > p.wait_limit_ns) give_up(kErrWaitMma);
                if (aborted()) {
                  ok = false;
                  break;
                }
              }
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
            }
            ++zeroed;
          }
          if (j >= n) {
            release(empty_bar + 8 * vs, false);
            if (j + 1 < t.n_max) {
              if (!wait_load(kx)) break;
              release(empty_bar + 8 * slot_of(kx), false);
            }
            __syncwarp();
            continue;
          }
          auto next_scores = [&]() {
            if constexpr (S::kOwnP)
              if (!wait_mma(sfree_bar + 8 * i, (turns + j) & 1)) return;
            tc_fence_after();
            scores(slot_of(kx));
          };
          // (before the wait for the probabilities: a look at a barrier takes a couple
          // of hundred cycles even when it is complete)
          if (j + 1 < t.n_max && !wait_load(kx)) break;
          if constexpr (S::kOwnP)
            if (j + 1 < n) next_scores();
          if (j == 0) outputs_free();
          if (!ok) break;
          const uint64_t v_at = v_desc + static_cast<uint64_t>(vs * (S::kTileBytes >> 4));
#pragma unroll
          for (int h = 0; h < S::kParts; ++h) {
            constexpr int kGroups = kAttnN / 64 / S::kParts;  // of 64 keys
            if (!wait_mma(p_bar + 8 * (2 * h + i), (turns + j) & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int k = h * kGroups; k < (h + 1) * kGroups; ++k)
              umma_ts_x4(tmem + S::kOutCol + i * kDP,
                         tmem + S::kProbCol + i * S::kProbStep + k * 32,
                         v_at + static_cast<uint64_t>(k * (8192 >> 4)), p.idesc_o,
                         (j > 0 || k > 0) ? 1u : 0u);
          }
          if (!ok) break;
          umma_commit_warp(o_bar + 8 * i);
          if constexpr (!S::kOwnP)
            if (j + 1 < n && product_done(turns + j)) next_scores();
          if (!ok) break;
          release(empty_bar + 8 * vs, true);
          if (j + 1 < t.n_max) release(empty_bar + 8 * slot_of(kx), j + 1 < n);
          if (j + 2 == n) release(qempty_bar, true);
          __syncwarp();
        }
        used += 2 * t.n_max;
        turns += n;
      }
      if (aborted() && any) {
        // let every product issued finish before tensor memory is released
        umma_commit_warp(drain_bar + 8 * i);
        __syncwarp();
        settle_phase(drain_bar + 8 * i, 0, p.wait_limit_ns, p.err);
      }
    } else if (warp >= kAttnOutWarp) {
      // ----------------------------------------------------------- outputs
      const int quad = warp & 3;
      const uint32_t lane_at = static_cast<uint32_t>(quad * 32) << 16;
      const uint32_t mine = staging + quad * S::kStoreBytes;
      int outs[2] = {0, 0};
      bool ok = true;
      PromptUnit u;
      int it = 0, tile = 2;
      for (; ok && take_unit(it, kErrWaitEpilogue, u); ++it) {
        const PromptTiles t(p, u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (the last totals being there, the output's phase before the last is over)
          outs[i] += t.n[i];
          ok = ok && wait(ml_bar + 8 * i, it & 1, kErrWaitEpilogue, true);
          const float2 ml = lds_f2(row_ml + 8 * (i * kAttnM + quad * 32 + lane));
          ok = ok && (t.n[i] == 0 ||
                      wait(o_bar + 8 * i, (outs[i] - 1) & 1, kErrWaitEpilogue));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            tile = i;
            break;
          }
          if (lane == 0) mbar_arrive(mlfree_bar + 8 * i);
          tc_fence_after();
          const uint32_t o_at = tmem + lane_at + S::kOutCol + i * kDP;
          const int row = t.row0[i] + quad * 32;  // the warp's first row in the sequence
          const int rows = min(32, u.nq - row);
          // no key seen: the total is 0; NaN scores make it NaN, and the row with it
          const bool seen = ml.y != 0.f;
          const float inv = seen ? 1.f / ml.y : 0.f;
          uint16_t* ob = p.out + static_cast<int64_t>(u.q0 + row) * p.o_ts + t.head[i] * p.o_hs;
          // 64 channels at a time through shared memory (16-byte chunks, swizzled), so
          // that a store covers 4 whole 128-byte rows; straight from its row, each
          // thread would write 16 bytes of 32 different lines
#pragma unroll 1
          for (int c = 0; c < S::kBlocks; ++c) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float o[16];
              if (t.n[i] > 0) tmem_ld16(o_at + c * 64 + g * 16, o);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  w[e] = seen
                             ? pack2<kBf16>(o[h * 8 + 2 * e] * inv, o[h * 8 + 2 * e + 1] * inv)
                             : 0u;
                sts_v4(mine + lane * 128 + (((2 * g + h) ^ (lane & 7)) << 4),
                       make_uint4(w[0], w[1], w[2], w[3]));
              }
            }
            if (c == S::kBlocks - 1) tc_fence_before();
            __syncwarp();
            if (c == S::kBlocks - 1 && lane == 0) mbar_arrive(ofree_bar + 8 * i);
            const int ch = lane & 7, col = c * 64 + ch * 8;
#pragma unroll
            for (int h = 0; h < 8; ++h) {
              const int x = h * 4 + (lane >> 3);
              if (x < rows && col < p.d)
                *reinterpret_cast<uint4*>(ob + x * p.o_ts + col) =
                    lds_v4(mine + x * 128 + ((ch ^ (x & 7)) << 4));
            }
            __syncwarp();
          }
          if (p.lse && lane < rows)
            p.lse[static_cast<int64_t>(u.q0 + row + lane) * p.Hq + t.head[i]] =
                seen ? ml.x * p.scale + (log2f(ml.y) - kBias) * 0.69314718f : kNegInf;
        }
      }
      if (lane == 0) unwritten[quad] = make_int2(it, tile);
    }
  } else {
    // ----------------------------------------------------------- softmax
    regs_take<kAttnRegsSoftmax>();
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;     // row of the tile
    const uint32_t lane_at = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_at + i * kAttnN;
    const uint32_t o_at = tmem + lane_at + S::kOutCol + i * kDP;
    const uint32_t p_at = tmem + lane_at + S::kProbCol + i * S::kProbStep;
    int turns = 0;                            // score tiles taken so far
    int turns_o = 0;                          // the other tile's score tiles
    bool ok = true;
    PromptUnit u;
    for (int it = 0; take_unit(it, kErrWaitEpilogue, u); ++it) {
      const PromptTiles t(p, u);
      const int n = i ? t.n[1] : t.n[0], n_o = i ? t.n[0] : t.n[1];
      const int row0 = i ? t.row0[1] : t.row0[0];
      const int row = row0 + r;               // row of the sequence
      const int seen = p.causal ? min(u.nk, row + t.shift + 1) : u.nk;  // keys of this row
      const int seen_all = p.causal ? min(u.nk, row0 + t.shift + 1) : u.nk;  // of every row
      const float far = row < u.nq ? kAttnFar : -kNegInf;  // other rows do not matter
      float m = kNegInf, l = 0.f;
      // the sums taken out so far, then their total and their reference maximum
      float held[kDP + 2];
      held[kDP + 1] = kNegInf;
      // out of the accumulator, once the product of step j is complete; after the last
      // step back into it
      auto take_out = [&](int j) {
        ok = ok && wait(o_bar + 8 * i, (turns + j) & 1, kErrWaitEpilogue);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        tc_fence_after();
        const bool last = j + 1 == n, first = j + 1 == kAttnHoldSteps;
        const float f =
            held[kDP + 1] == kNegInf ? 0.f : exp2_approx((held[kDP + 1] - m) * p.c);
#pragma unroll 1
        for (int c = 0; c < kDP; c += 16) {
          float o[16];
          tmem_ld16(o_at + c, o);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (!first) o[e] = fmaf(held[c + e], f, o[e]);
            held[c + e] = o[e];
            w[e] = last ? __float_as_uint(o[e]) : 0u;
          }
          tmem_st16(o_at + c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        if (!first) l = fmaf(held[kDP], f, l);
        held[kDP] = l;
        held[kDP + 1] = m;
        if (!last) l = 0.f;
        return true;
      };
      bool s_there = false;  // the step's scores have been seen to be there
      int j = 0;
      // (a look after every step costs the 64-channel form 8 %, the loop of segments the
      // 128-channel form 4 %, where no row has that many keys)
      do {
        const int j_end = kLong && S::kOwnP ? min(n, j + kAttnHoldSteps) : n;
#pragma unroll 1
        for (; j < j_end; ++j) {
          ok = s_there || wait(s_bar + 8 * i, (turns + j) & 1, kErrWaitEpilogue);
          __syncwarp();
          tc_fence_after();
          float s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_at + c * 32, s[c]);
          tmem_wait_ld_regs(s[0]);
#pragma unroll
          for (int c = 1; c < 4; ++c) reg_fence(s[c]);
          // a look at a barrier takes a couple of hundred cycles: this one's answer is
          // used behind the comparisons, the one for the next scores in the next step
          bool o_there = !S::kOwnP || turns + j == 0;
          if (!o_there) o_there = mbar_test_wait(o_bar + 8 * i, (turns + j - 1) & 1);
          if constexpr (S::kOwnP) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sfree_bar + 8 * i);
          }
          if ((j + 1) * kAttnN > seen_all) {
            const int lim_col = seen - j * kAttnN;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e >= lim_col) s[c][e] = kNegInf;
          }
          const float x = fmaxf(fmaxf(max32(s[0]), max32(s[1])), fmaxf(max32(s[2]), max32(s[3])));
          if constexpr (S::kOwnP) {
            // the product before has read these columns, and its sum is complete
            ok = ok && (o_there || wait(o_bar + 8 * i, (turns + j - 1) & 1, kErrWaitEpilogue));
            tc_fence_after();
          }
          if (j == 0) m = x;
          const bool grow = (x - m) * p.c > kAttnSlack;  // also from -inf to a number
          float mc = m * p.c;
          // one vote for all: a lane whose wait gave up takes the warp with it (votes at
          // the waits themselves cost 2 %)
          if (__any_sync(0xffffffffu, grow || !ok || fabsf(mc) > far)) {
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const float f = grow ? exp2_approx((m - x) * p.c) : 1.f;
            if (grow) m = x;
            mc = m == kNegInf ? 0.f : m * p.c;
            const bool before = fabsf(mc) > far && fabsf(m) < -kNegInf;
            if (__any_sync(0xffffffffu, before)) {
              const float ref = before ? m : 0.f;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e) s[c][e] -= ref;
              if (before) mc = 0.f;
            }
            l *= f;
            if (__any_sync(0xffffffffu, grow)) {
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
          // The two warps of a scheduler take turns at the exponential unit, tile 0's
          // step j, tile 1's step j, tile 0's step j + 1: left alone they fall into
          // step, and both leave it idle while both load and compare.  Order only: no
          // result depends on it, and after kTurnPolls looks a warp goes on anyway.
          const int j_o = i ? j : j - 1;  // the other's step to wait for
          if (j_o >= 0 && j_o < n_o) {
#pragma unroll 1
            for (int k = 0; k < kTurnPolls; ++k) {
              if (lds_volatile(turn_at + 4 * (warp ^ 4)) > turns_o + j_o) break;
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
              // the second product takes the probabilities in the value type
              // (half a step: 2^-9 of bf16, 2^-12 of fp16, of each weight); the
              // total keeps them in fp32
              w[e] = pack2<kBf16>(a, b);
            }
            if (c == kTurnChunk && lane == 0) sts_volatile(turn_at + 4 * warp, turns + j + 1);
            if (S::kOwnP && c == 3)
              s_there = mbar_test_wait(s_bar + 8 * i, (turns + j + 1) & 1);
            tmem_st16(p_at + c * 16, w);
            if ((c + 1) % (4 / S::kParts) == 0) {
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_bar + 8 * (2 * (c / (4 / S::kParts)) + i));
            }
          }
          float a, b;
          f2_get(f2_add(sum[0], sum[1]), a, b);
          l += a + b;
          if (kLong && !S::kOwnP && n > kAttnHoldSteps &&
              ((j + 1) % kAttnHoldSteps == 0 || j + 1 == n))
            if (!take_out(j)) break;
        }
        if (kLong && S::kOwnP && ok && n > kAttnHoldSteps) take_out(j - 1);
      } while (kLong && S::kOwnP && ok && j < n);  // (ok is the same in all lanes here)
      turns += n;
      turns_o += n_o;
      if (it > 0)
        ok = ok && wait(mlfree_bar + 8 * i, (it - 1) & 1, kErrWaitEpilogue);
      if (!__all_sync(0xffffffffu, ok)) break;
      sts_f2(row_ml + 8 * (i * kAttnM + r), m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(ml_bar + 8 * i);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kAttnMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
  if (warp >= kAttnOutWarp && aborted()) {
    // what was given up becomes NaN, so that nobody takes the buffer's old bytes for rows
    const uint32_t nan2 = kBf16 ? 0x7FC07FC0u : 0x7E007E00u;
    const int2 from = unwritten[warp & 3];
#pragma unroll 1
    for (int k = from.x - 1; k <= dealt; ++k) {
      if (k < from.x && from.y == 2) continue;
      const PromptUnit u = k < dealt ? units[k & 3] : unpublished;
      if (u.nq < 0) continue;
      const int tile = k < from.x ? from.y : 0;
      const PromptTiles t(p, u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i < tile) continue;
        const int row = t.row0[i] + (warp & 3) * 32, rows = min(32, u.nq - row);
        for (int x = 0; x < rows; ++x) {
          const int64_t at = u.q0 + row + x;
          if (lane * 8 < p.d)
            *reinterpret_cast<uint4*>(p.out + at * p.o_ts + t.head[i] * p.o_hs + lane * 8) =
                make_uint4(nan2, nan2, nan2, nan2);
          if (p.lse && lane == 0)
            p.lse[at * p.Hq + t.head[i]] = __uint_as_float(0x7FC00000u);
        }
      }
    }
  }
}

}  // namespace rnn
