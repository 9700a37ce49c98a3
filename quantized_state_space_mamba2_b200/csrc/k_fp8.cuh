// k_fp8.cuh -- e4m3 matrix product with a scale for each block of 128 on the
// 5th-generation tensor cores (tcgen05, kind::f8f6f4):
//   Y[m, n] = sum_b s_a[m, b] s_w[n / 128, b] sum_{k in block b} A[m, k] W[n, k].
//
// The scales of a block are arbitrary fp32 numbers, so its sum cannot stay in
// the tensor core's accumulator: each 128-deep block is accumulated on its own
// in TMEM (four K = 32 instructions), read back, and added to fp32 registers
// with one fused multiply-add per output, acc += (s_a s_w) * block sum.  The
// TMEM accumulators form a ring, so the read-back of block b overlaps the
// MMAs of the blocks after it.
//
// Large M (8192 x 10576 x 2560, bf16 out): 258 us, 1.72 PFLOP/s.  By cycles
// (4096 rows, one clock): the MMAs alone 109 k, with their loads 128 k, with the
// hand-over of the two TMEM buffers 149 k, with the read-back and the scaling
// 173 k: the hand-over and the read-back, a chain per block, bound it, and in a
// loop the 1 kW power cap (1.5-1.8 GHz; codes and positive scales drawn evenly take
// less power: 216 us).  Pairs of CTAs (cta_group::2, 256 x 256 tiles, half the bytes
// per MMA) measured 196 k, in a version whose second CTA passed its loads on to the
// leader through a warp of its own.  Output rows that are no multiple of 16 bytes are
// stored element by element by the accumulator warps: N = 10575 302 us where N =
// 10576 takes 216, at K = 256 151 and 48.
// Small M (64 x 50000 x 2560, fp32 out): 31.4 us, 4.5 TB/s; 16 rows 26.0 us, 5.0
// TB/s.  The weight stream bounds it from below; above that are the last wave (391
// weight tiles on 148 SMs run as 3 waves, 12 % of the machine idle) and, where many
// rows wait for it, the per-block chain of the read-back.
#pragma once
#include <cuda_bf16.h>
#include "k_gemm.cuh"
#include "k_token.cuh"

namespace fm {

// Instruction descriptor, kind::f8f6f4: D = f32 (bits 4-5 = 1), A and B e4m3
// (bits 7-9 and 10-12 = 0), both K-major, N >> 3 at bits 17-22, M >> 4 at 24-28.
__host__ __device__ constexpr uint32_t e4m3_idesc(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// tcgen05.ld without its wait: the values are there after tmem_ld_wait, which
// takes them as operands so that no use can move before it
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}
// the same for values of a load that the wait just above has completed
__device__ __forceinline__ void tmem_ld_tie(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  asm volatile(""
               : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                 "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
// acc (two fp32) += (lo, hi) * c (two fp32), each a single rounding
__device__ __forceinline__ void ffma2(unsigned long long &acc, uint32_t lo, uint32_t hi,
                                      unsigned long long c) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(c));
}
// (lo, hi) * c
__device__ __forceinline__ unsigned long long fmul2(float lo, float hi, unsigned long long c) {
  unsigned long long d;
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 %0, v, %3;\n\t}"
      : "=l"(d)
      : "f"(lo), "f"(hi), "l"(c));
  return d;
}
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  return ((unsigned long long)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}

// Bounded wait for the hand-overs of a pipeline, whose limit lies in shared
// memory (a load of it from global memory costs more than such a wait).  The
// thread may stay suspended in a poll: polls that return at once take issue
// slots and shared-memory cycles from the warps at work.
__device__ __forceinline__ bool mbar_poll(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u /* ns */)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_in(uint64_t *bar, uint32_t parity,
                                             const unsigned long long &limit) {
  if (mbar_try_wait(bar, parity)) return true;  // 14 cycles; a poll that may suspend takes 50
  const unsigned long long t0 = globaltimer();
  while (true) {
    if (mbar_poll(bar, parity)) return true;
    if (globaltimer() - t0 > limit) {
      raise_error(kErrTimeout);
      return false;
    }
  }
}

// True in one lane of a converged warp.  The compiler knows that one lane runs
// the code behind it, and issues tcgen05 and TMA instructions there at once;
// behind `lane == 0` each of them costs 44 cycles, a commit among them too
// (measured: 4 MMAs of N = 16 and 2 commits 265 cycles, 157 behind this).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A position in a ring of N slots and the parity of its current round.  (A
// counter taken modulo N costs a dependent chain of multiplications per block.)
template <int N>
struct RingPos {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      round ^= 1u;
    }
  }
};

// Waits for every copy issued into the ring up to (not including) position
// `end`: they must have landed before the CTA may exit.  On the normal path all
// have been consumed and this returns at once.
template <int N>
__device__ __forceinline__ void ring_drain(uint64_t *full_bar, const RingPos<N> &end) {
  for (uint32_t i = 0; i < N; ++i) {
    // slot i was last filled in this round (i < end.at) or the one before,
    // whose parity is also what an unused slot's preceding phase counts as
    const uint32_t round = i < end.at ? end.round : end.round ^ 1u;
    if (!mbar_drain(&full_bar[i], round)) break;
  }
}

struct Fp8Args {
  const float *s_a, *s_w;  // [M, nkb], [ceil(N / 128), nkb]
  long long M, N, ldy;
  void *Y;
  int nkb, m_tiles, n_tiles;
  int tma_store;  // Y's row stride and address allow TMA stores
};

// ------------------------------------------------------------ large M
// One CTA per SM walks 128 x BN output tiles.  Warp 0 loads (TMA, a ring of
// STAGES 128-deep blocks), one lane of warp 1 issues the MMAs, warps 4..11 hold
// the fp32 accumulators: warp w the 32 rows of TMEM lane quarter w % 4 (lane =
// row) and one half of the tile's columns, so s_a s_w is one number per thread
// and block.  128 accumulators and 64 values on their way from TMEM need more
// registers than an even share: the first warpgroup hands its own over.
// A TMEM load takes about 115 cycles and another one behind it 16 more
// (measured), so 64 columns are loaded per wait and the two warps of a
// scheduler cover each other's wait.
template <int BN, int STAGES>
struct Fp8Smem {
  static constexpr int kA = kGemmBM * kGemmBK, kB = BN * kGemmBK;
  static constexpr int kStage = 4096;  // per epilogue warp: 32 rows x 128 bytes
  static constexpr int kAcc = 512 / BN;
  static constexpr int kBytes = 1024 + STAGES * (kA + kB) + 8 * kStage +
                                (2 * STAGES + 2 * kAcc + 1) * 8 + 16;
};
constexpr int kFp8Threads = 384;
// registers per thread of the first warpgroup and of the two others
constexpr int kFp8RegsLoad = 40, kFp8RegsAcc = 224;

// The 32 x 32 (fp32) or 32 x 64 (bf16) chunk of the tile at (row0, col0), from
// the lanes' rows (lane = row), 128 bytes each, through the warp's staging
// buffer: one TMA store, or row by row where Y's stride allows none.
template <typename TY>
__device__ __forceinline__ void fp8_store_chunk(const Fp8Args &a, const CUtensorMap *tm,
                                                const uint4 (&v)[8], long long row0, long long col0,
                                                uint8_t *stage, int lane) {
  constexpr int kCols = 128 / (int)sizeof(TY);
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
  uint4 *row = reinterpret_cast<uint4 *>(stage + lane * 128);
#pragma unroll
  for (int q = 0; q < 8; ++q) row[q ^ (lane & 7)] = v[q];
  if (a.tma_store) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tm, (int)col0, (int)row0, stage);
      bulk_commit();
    }
    return;
  }
  __syncwarp();
  TY *Y = (TY *)a.Y;
  for (int r = 0; r < 32 && row0 + r < a.M; ++r)
#pragma unroll
    for (int c = lane; c < kCols; c += 32) {
      const int at = c * (int)sizeof(TY);
      if (col0 + c < a.N)
        Y[(row0 + r) * a.ldy + col0 + c] = *reinterpret_cast<const TY *>(
            stage + r * 128 + ((((at >> 4) ^ (r & 7)) << 4) | (at & 15)));
    }
}

template <int BN, int STAGES, typename TY>
__global__ void __launch_bounds__(kFp8Threads, 1)
    k_fp8_gemm_tc(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, Fp8Args a) {
  using Sm = Fp8Smem<BN, STAGES>;
  constexpr int kAcc = Sm::kAcc;
  constexpr int kCols = BN / 2;  // per epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + STAGES * Sm::kA;
  uint8_t *sOut = sB + STAGES * Sm::kB;
  uint64_t *full_bar = reinterpret_cast<uint64_t *>(sOut + 8 * Sm::kStage);
  uint64_t *empty_bar = full_bar + STAGES;
  uint64_t *tfull = empty_bar + STAGES;
  uint64_t *tempty = tfull + kAcc;
  uint64_t *drain_bar = tempty + kAcc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_bar + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_tiles = a.m_tiles * a.n_tiles;

  __shared__ unsigned long long limit;  // of the waits, ns
  if (threadIdx.x == 0) {
    limit = *(volatile unsigned long long *)&g_wait_limit_ns;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    mbar_init(drain_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((unsigned long long)&tmA) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((unsigned long long)&tmB) : "memory");
    if (a.tma_store)
      asm volatile("prefetch.tensormap [%0];" ::"l"((unsigned long long)&tmY) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // every operand (the weights too: they may have been prepared just before)
  // is read after the predecessor has completed
  pdl_wait();
  pdl_trigger();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFp8RegsLoad));
    // every lane of the two warps runs the loops and the waits, one issues
    const bool lead = elect_one();
    if (warp == 0) {
      bool ok = !(g_test_stall & kStallGemm);
      RingPos<STAGES> ring;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
        const int m0 = (t / a.n_tiles) * kGemmBM, n0 = (t % a.n_tiles) * BN;
        for (int kb = 0; kb < a.nkb; ++kb, ring.next()) {
          const uint32_t s = ring.at;
          if (!mbar_wait_in(&empty_bar[s], ring.round ^ 1u, limit)) {
            ok = false;
            break;
          }
          if (lead) {
            mbar_arrive_expect_tx(&full_bar[s], (uint32_t)(Sm::kA + Sm::kB));
            tma_load_2d(sA + s * Sm::kA, &tmA, kb * kGemmBK, m0, &full_bar[s]);
            tma_load_2d(sB + s * Sm::kB, &tmB, kb * kGemmBK, n0, &full_bar[s]);
          }
        }
      }
      // every copy issued must have landed before the CTA may exit
      if (lead) ring_drain<STAGES>(full_bar, ring);
    } else if (warp == 1) {
      constexpr uint32_t idesc = e4m3_idesc(kGemmBM, BN);
      const uint64_t ad0 = sw128_desc(smem_u32(sA)), bd0 = sw128_desc(smem_u32(sB));
      RingPos<STAGES> ring;
      RingPos<kAcc> out;
      bool ok = true;
      for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x)
        for (int kb = 0; kb < a.nkb; ++kb, ring.next(), out.next()) {
          const uint32_t s = ring.at, acc = out.at;
          if (!mbar_wait_in(&tempty[acc], out.round ^ 1u, limit) ||
              !mbar_wait_in(&full_bar[s], ring.round, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lead) {
            const uint64_t ad = ad0 + s * (Sm::kA / 16), bd = bd0 + s * (Sm::kB / 16);
#pragma unroll
            for (int k = 0; k < kGemmBK / 32; ++k)
              mma_e4m3(tmem_base + acc * BN, ad + (uint64_t)(2 * k), bd + (uint64_t)(2 * k), idesc,
                       k > 0 ? 1u : 0u);
            mma_commit(&empty_bar[s]);
            mma_commit(&tfull[acc]);
          }
        }
      if (lead) {  // wait for every MMA issued so far before TMEM can be released
        mma_commit(drain_bar);
        mbar_drain(drain_bar, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8RegsAcc));
    const int e = warp - 4, quarter = warp & 3, half = e / 4;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * kCols);
    RingPos<kAcc> in;
    bool ok = true;
    for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
      const long long m0 = (long long)(t / a.n_tiles) * kGemmBM + quarter * 32;
      const long long n0 = (long long)(t % a.n_tiles) * BN + half * kCols;
      // rows and column blocks past the edge (whose operands are zeros) read
      // the last valid scale
      const float *pa = a.s_a + min(m0 + lane, a.M - 1) * a.nkb;
      const float *pw = a.s_w + (min(n0, a.N - 1) >> 7) * a.nkb;
      unsigned long long acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
      // the scales are fetched well ahead (they come from L2: shared memory
      // leaves L1 next to nothing): a row's own two blocks ahead, the column
      // block's, which the warp shares, 32 blocks in the lanes at a time
      float ca = pa[0], ca1 = pa[min(1, a.nkb - 1)];
      float cw = pw[min(lane, a.nkb - 1)];
#pragma unroll 1
      for (int kb = 0; kb < a.nkb; ++kb, in.next()) {
        const uint32_t buf = in.at;
        if (kb && (kb & 31) == 0) cw = pw[min(kb + lane, a.nkb - 1)];
        const float c = __fmul_rn(ca, __shfl_sync(0xffffffffu, cw, kb & 31));
        ca = ca1;
        if (kb + 2 < a.nkb) ca1 = pa[kb + 2];
        ok = mbar_wait_in(&tfull[buf], in.round, limit);
        ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld is warp-collective
        if (!ok) break;
        tc_fence_after();
        const unsigned long long c2 = pack2(c, c);
#pragma unroll
        for (int q = 0; q < kCols; q += 64) {
          uint32_t r0[32], r1[32];
          tmem_ld32_issue(lane_base + (uint32_t)(buf * BN + q), r0);
          tmem_ld32_issue(lane_base + (uint32_t)(buf * BN + q + 32), r1);
          tmem_ld_wait(r0);
          tmem_ld_tie(r1);
          if (q + 64 == kCols) {  // the last load has completed: hand the buffer back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) ffma2(acc[q / 2 + j], r0[2 * j], r0[2 * j + 1], c2);
#pragma unroll
          for (int j = 0; j < 16; ++j) ffma2(acc[q / 2 + 16 + j], r1[2 * j], r1[2 * j + 1], c2);
        }
      }
      if (!ok) break;
      constexpr int kChunk = 128 / (int)sizeof(TY);
#pragma unroll
      for (int c = 0; c < kCols; c += kChunk) {
        if (n0 + c >= a.N) continue;
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(TY) == 4) {
              const unsigned long long p = acc[(c + 4 * q + i) / 2];
              u[i] = i & 1 ? (uint32_t)(p >> 32) : (uint32_t)p;
            } else {
              const unsigned long long p = acc[(c + 8 * q + 2 * i) / 2];
              asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                  : "=r"(u[i])
                  : "f"(__uint_as_float((uint32_t)(p >> 32))), "f"(__uint_as_float((uint32_t)p)));
            }
          }
          v[q] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        fp8_store_chunk<TY>(a, &tmY, v, m0, n0 + c, sOut + e * Sm::kStage, lane);
      }
    }
    if (a.tma_store && lane == 0) bulk_wait_all();  // stores done before the CTA exits
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(512u)
                 : "memory");
  }
}

// ------------------------------------------------------------ small M
// A decode batch: the weights' rows take the MMA's M side (128 per tile) and
// the MP >= M activation rows its N side, so a tile costs what its real rows
// cost and the weights stream past once.  Lane = weight row n, column =
// activation row m: s_w is one number per tile and block, and s_a, which is
// the same for every tile, waits in shared memory (block by block, the MP rows
// of a block side by side; kChunk blocks at a time).  The columns are split
// over as many warps as leaves each 16 (MP = 128: 32): a block's read-back is a
// chain of waits, which the four warps of a scheduler take in turns.
template <int MP, int STAGES>
struct Fp8SmallSmem {
  static constexpr int kW = kGemmBM * kGemmBK, kA = MP * kGemmBK;
  static constexpr int kEpi = MP > 64 ? 16 : MP / 4;  // 16 columns each, 32 of MP = 128
  static constexpr int kAcc = 512 / MP < 4 ? 512 / MP : 4;
  static constexpr int kChunk = 64;
  static constexpr int kBytes = 1024 + STAGES * (kW + kA) + kChunk * MP * 4 +
                                (2 * STAGES + 2 * kAcc + 1) * 8 + 16;
};

template <int MP, int STAGES, typename TY>
__global__ void __launch_bounds__(64 + 32 * Fp8SmallSmem<MP, STAGES>::kEpi, 1)
    k_fp8_gemm_small(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmA, Fp8Args a) {
  using Sm = Fp8SmallSmem<MP, STAGES>;
  constexpr int kAcc = Sm::kAcc, kEpi = Sm::kEpi;
  constexpr int kCols = MP / (kEpi / 4);  // columns per epilogue warp
  constexpr uint32_t kTmem = kAcc * MP;  // a power of two >= 64
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sW = smem;
  uint8_t *sA = smem + STAGES * Sm::kW;
  float *coef = reinterpret_cast<float *>(sA + STAGES * Sm::kA);  // [kChunk][MP]
  uint64_t *full_bar = reinterpret_cast<uint64_t *>(coef + Sm::kChunk * MP);
  uint64_t *empty_bar = full_bar + STAGES;
  uint64_t *tfull = empty_bar + STAGES;
  uint64_t *tempty = tfull + kAcc;
  uint64_t *drain_bar = tempty + kAcc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_bar + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  __shared__ unsigned long long limit;  // of the waits, ns
  if (threadIdx.x == 0) {
    limit = *(volatile unsigned long long *)&g_wait_limit_ns;
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpi);
    }
    mbar_init(drain_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((unsigned long long)&tmW) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((unsigned long long)&tmA) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp < 2) {
    const bool lead = elect_one();
    RingPos<STAGES> ring;
    if (warp == 0) {
      bool ok = !(g_test_stall & kStallGemm);
      for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x)
        for (int kb = 0; kb < a.nkb; ++kb, ring.next()) {
          const uint32_t s = ring.at;
          if (!mbar_wait_in(&empty_bar[s], ring.round ^ 1u, limit)) {
            ok = false;
            break;
          }
          if (lead) {
            mbar_arrive_expect_tx(&full_bar[s], (uint32_t)(Sm::kW + Sm::kA));
            tma_load_2d(sW + s * Sm::kW, &tmW, kb * kGemmBK, t * kGemmBM, &full_bar[s]);
            tma_load_2d(sA + s * Sm::kA, &tmA, kb * kGemmBK, 0, &full_bar[s]);
          }
        }
      if (lead) ring_drain<STAGES>(full_bar, ring);
    } else {
      constexpr uint32_t idesc = e4m3_idesc(kGemmBM, MP);
      const uint64_t wd0 = sw128_desc(smem_u32(sW)), ad0 = sw128_desc(smem_u32(sA));
      RingPos<kAcc> out;
      bool ok = true;
      for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x)
        for (int kb = 0; kb < a.nkb; ++kb, ring.next(), out.next()) {
          const uint32_t s = ring.at, acc = out.at;
          if (!mbar_wait_in(&tempty[acc], out.round ^ 1u, limit) ||
              !mbar_wait_in(&full_bar[s], ring.round, limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lead) {
            const uint64_t wd = wd0 + s * (Sm::kW / 16), ad = ad0 + s * (Sm::kA / 16);
#pragma unroll
            for (int k = 0; k < kGemmBK / 32; ++k)
              mma_e4m3(tmem_base + acc * MP, wd + (uint64_t)(2 * k), ad + (uint64_t)(2 * k), idesc,
                       k > 0 ? 1u : 0u);
            mma_commit(&empty_bar[s]);
            mma_commit(&tfull[acc]);
          }
        }
      if (lead) {
        mma_commit(drain_bar);
        mbar_drain(drain_bar, 0);
      }
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) / 4, et = threadIdx.x - 64;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kCols);
    // the next kChunk blocks' s_a (zeros for columns past M)
    auto stage = [&](int kb0) {
      asm volatile("bar.sync 1, %0;" ::"r"(32 * kEpi) : "memory");
      const int nb = min(Sm::kChunk, a.nkb - kb0);
      for (int i = et; i < nb * MP; i += 32 * kEpi) {
        const int m = i / nb, kb = i - m * nb;
        coef[kb * MP + m] = m < a.M ? a.s_a[(long long)m * a.nkb + kb0 + kb] : 0.0f;
      }
      asm volatile("bar.sync 1, %0;" ::"r"(32 * kEpi) : "memory");
    };
    const bool resident = a.nkb <= Sm::kChunk;
    if (resident) stage(0);
    RingPos<kAcc> in;
    bool ok = true;
    // after a failed wait a warp skips its work but still meets the others
    // wherever scales are staged
    for (int t = blockIdx.x; t < a.n_tiles; t += gridDim.x) {
      const float *pw = a.s_w + (long long)t * a.nkb;
      unsigned long long acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
      float cw = pw[0];
#pragma unroll 1
      for (int kb = 0; kb < a.nkb; ++kb, in.next()) {
        if (!resident && kb % Sm::kChunk == 0) stage(kb);
        const uint32_t buf = in.at;
        const float4 *cf = reinterpret_cast<const float4 *>(coef + kb % Sm::kChunk * MP + part * kCols);
        const unsigned long long w2 = pack2(cw, cw);
        if (kb + 1 < a.nkb) cw = pw[kb + 1];
        unsigned long long c[8];  // 16 columns' factors
        auto factors = [&](int q) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = cf[4 * q + j];
            c[2 * j] = fmul2(v.x, v.y, w2);
            c[2 * j + 1] = fmul2(v.z, v.w, w2);
          }
        };
        factors(0);  // while the block is multiplied
        if (ok) ok = mbar_wait_in(&tfull[buf], in.round, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          uint32_t r[16];
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
              "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
              "tcgen05.wait::ld.sync.aligned;"
              : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
                "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
              : "r"(lane_base + buf * MP + 16 * q)
              : "memory");
          if (q + 1 == kCols / 16) {  // the last load has completed: hand the buffer back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) ffma2(acc[8 * q + j], r[2 * j], r[2 * j + 1], c[j]);
          if (q + 1 < kCols / 16) factors(q + 1);
        }
      }
      const long long n = (long long)t * kGemmBM + quarter * 32 + lane;
      if (ok && n < a.N) {
        TY *y = (TY *)a.Y + n;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const long long m = part * kCols + j;
          const uint32_t b = j & 1 ? (uint32_t)(acc[j / 2] >> 32) : (uint32_t)acc[j / 2];
          if (m < a.M) y[m * a.ldy] = (TY)__uint_as_float(b);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmem)
                 : "memory");
  }
}

}  // namespace fm
