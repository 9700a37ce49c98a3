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
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  return ((unsigned long long)__float_as_uint(hi) << 32) | __float_as_uint(lo);
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

  if (threadIdx.x == 0) {
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
    if (warp == 0) {
      if (lane == 0) {
        bool ok = !(g_test_stall & kStallGemm);
        long long it = 0;
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x) {
          const int m0 = (t / a.n_tiles) * kGemmBM, n0 = (t % a.n_tiles) * BN;
          for (int kb = 0; kb < a.nkb; ++kb, ++it) {
            const int s = (int)(it % STAGES);
            if (!mbar_wait(&empty_bar[s], ((uint32_t)(it / STAGES) & 1u) ^ 1u)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full_bar[s], (uint32_t)(Sm::kA + Sm::kB));
            tma_load_2d(sA + s * Sm::kA, &tmA, kb * kGemmBK, m0, &full_bar[s]);
            tma_load_2d(sB + s * Sm::kB, &tmB, kb * kGemmBK, n0, &full_bar[s]);
          }
        }
        // every copy issued must have landed before the CTA may exit
        for (long long j = it > STAGES ? it - STAGES : 0; j < it; ++j)
          if (!mbar_drain(&full_bar[j % STAGES], (uint32_t)(j / STAGES) & 1u)) break;
      }
    } else if (warp == 1) {
      if (lane == 0) {
        constexpr uint32_t idesc = e4m3_idesc(kGemmBM, BN);
        long long it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < num_tiles && ok; t += gridDim.x)
          for (int kb = 0; kb < a.nkb; ++kb, ++it) {
            const int s = (int)(it % STAGES), acc = (int)(it % kAcc);
            if (!mbar_wait(&tempty[acc], ((uint32_t)(it / kAcc) & 1u) ^ 1u) ||
                !mbar_wait(&full_bar[s], (uint32_t)(it / STAGES) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = sw128_desc(smem_u32(sA + s * Sm::kA));
            const uint64_t bd = sw128_desc(smem_u32(sB + s * Sm::kB));
#pragma unroll
            for (int k = 0; k < kGemmBK / 32; ++k)
              mma_e4m3(tmem_base + (uint32_t)(acc * BN), ad + (uint64_t)(2 * k),
                       bd + (uint64_t)(2 * k), idesc, k > 0 ? 1u : 0u);
            mma_commit(&empty_bar[s]);
            mma_commit(&tfull[acc]);
          }
        // wait for every MMA issued so far before TMEM can be released
        mma_commit(drain_bar);
        mbar_drain(drain_bar, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFp8RegsAcc));
    const int e = warp - 4, quarter = warp & 3, half = e / 4;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * kCols);
    long long it = 0;
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
      float ca = pa[0], cw = pw[0];
      for (int kb = 0; kb < a.nkb; ++kb, ++it) {
        const int buf = (int)(it % kAcc);
        const float c = __fmul_rn(ca, cw);
        if (kb + 1 < a.nkb) {  // the next block's scales, a block ahead
          ca = pa[kb + 1];
          cw = pw[kb + 1];
        }
        ok = mbar_wait(&tfull[buf], (uint32_t)(it / kAcc) & 1u);
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
// activation row m; s_a s_w of the block is staged in shared memory, one
// number per column.  The accumulators and the warps are as above (four
// warps; eight for MP = 128, each with 64 columns).
template <int MP, int STAGES>
struct Fp8SmallSmem {
  static constexpr int kW = kGemmBM * kGemmBK, kA = MP * kGemmBK;
  static constexpr int kEpi = MP > 64 ? 8 : 4;
  static constexpr int kAcc = 512 / MP < 4 ? 512 / MP : 4;
  static constexpr int kBytes = 1024 + STAGES * (kW + kA) + 2 * MP * 4 +
                                (2 * STAGES + 2 * kAcc + 1) * 8 + 16;
};

template <int MP, int STAGES, typename TY>
__global__ void __launch_bounds__(64 + 32 * Fp8SmallSmem<MP, STAGES>::kEpi, 1)
    k_fp8_gemm_small(const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmA, Fp8Args a) {
  using Sm = Fp8SmallSmem<MP, STAGES>;
  constexpr int kAcc = Sm::kAcc, kEpi = Sm::kEpi;
  constexpr int kCols = MP / (kEpi / 4);  // columns per epilogue warp
  constexpr int kLd = kCols < 32 ? kCols : 32;
  constexpr uint32_t kTmem = kAcc * MP;  // a power of two >= 64
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *sW = smem;
  uint8_t *sA = smem + STAGES * Sm::kW;
  float *coef = reinterpret_cast<float *>(sA + STAGES * Sm::kA);  // [2][MP]
  uint64_t *full_bar = reinterpret_cast<uint64_t *>(coef + 2 * MP);
  uint64_t *empty_bar = full_bar + STAGES;
  uint64_t *tfull = empty_bar + STAGES;
  uint64_t *tempty = tfull + kAcc;
  uint64_t *drain_bar = tempty + kAcc;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain_bar + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
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

  if (warp == 0) {
    if (lane == 0) {
      bool ok = !(g_test_stall & kStallGemm);
      long long it = 0;
      for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x)
        for (int kb = 0; kb < a.nkb; ++kb, ++it) {
          const int s = (int)(it % STAGES);
          if (!mbar_wait(&empty_bar[s], ((uint32_t)(it / STAGES) & 1u) ^ 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full_bar[s], (uint32_t)(Sm::kW + Sm::kA));
          tma_load_2d(sW + s * Sm::kW, &tmW, kb * kGemmBK, t * kGemmBM, &full_bar[s]);
          tma_load_2d(sA + s * Sm::kA, &tmA, kb * kGemmBK, 0, &full_bar[s]);
        }
      for (long long j = it > STAGES ? it - STAGES : 0; j < it; ++j)
        if (!mbar_drain(&full_bar[j % STAGES], (uint32_t)(j / STAGES) & 1u)) break;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = e4m3_idesc(kGemmBM, MP);
      long long it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < a.n_tiles && ok; t += gridDim.x)
        for (int kb = 0; kb < a.nkb; ++kb, ++it) {
          const int s = (int)(it % STAGES), acc = (int)(it % kAcc);
          if (!mbar_wait(&tempty[acc], ((uint32_t)(it / kAcc) & 1u) ^ 1u) ||
              !mbar_wait(&full_bar[s], (uint32_t)(it / STAGES) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t wd = sw128_desc(smem_u32(sW + s * Sm::kW));
          const uint64_t ad = sw128_desc(smem_u32(sA + s * Sm::kA));
#pragma unroll
          for (int k = 0; k < kGemmBK / 32; ++k)
            mma_e4m3(tmem_base + (uint32_t)(acc * MP), wd + (uint64_t)(2 * k),
                     ad + (uint64_t)(2 * k), idesc, k > 0 ? 1u : 0u);
          mma_commit(&empty_bar[s]);
          mma_commit(&tfull[acc]);
        }
      mma_commit(drain_bar);
      mbar_drain(drain_bar, 0);
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) / 4, et = threadIdx.x - 64;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * kCols);
    const float *pa = a.s_a + min((long long)et, a.M - 1) * a.nkb;  // thread et < MP: column et
    long long it = 0;
    bool ok = true;
    // after a failed wait a warp skips its work but still meets the others at
    // every block's barrier
    for (int t = blockIdx.x; t < a.n_tiles; t += gridDim.x) {
      const float *pw = a.s_w + (long long)t * a.nkb;
      unsigned long long acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
      float ca = et < MP ? pa[0] : 0.0f, cw = pw[0];
      for (int kb = 0; kb < a.nkb; ++kb, ++it) {
        const int buf = (int)(it % kAcc);
        // this block's factors; the buffer was last read two blocks ago, before
        // every warp passed the previous block's barrier
        float *cf = coef + (it & 1) * MP;
        if (et < MP) cf[et] = __fmul_rn(ca, cw);
        if (kb + 1 < a.nkb) {
          if (et < MP) ca = pa[kb + 1];
          cw = pw[kb + 1];
        }
        asm volatile("bar.sync 1, %0;" ::"r"(32 * kEpi) : "memory");
        if (ok) ok = mbar_wait(&tfull[buf], (uint32_t)(it / kAcc) & 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        tc_fence_after();
        const unsigned long long *cf2 =
            reinterpret_cast<const unsigned long long *>(cf + part * kCols);
#pragma unroll
        for (int q = 0; q < kCols / kLd; ++q) {
          uint32_t r[32];
          if constexpr (kLd == 32) {
            tmem_ld32_issue(lane_base + (uint32_t)(buf * MP + 32 * q), r);
            tmem_ld_wait(r);
          } else {
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                "tcgen05.wait::ld.sync.aligned;"
                : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                  "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                  "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                : "r"(lane_base + (uint32_t)(buf * MP))
                : "memory");
          }
          if (q + 1 == kCols / kLd) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[buf]);
          }
#pragma unroll
          for (int j = 0; j < kLd / 2; ++j)
            ffma2(acc[kLd / 2 * q + j], r[2 * j], r[2 * j + 1], cf2[kLd / 2 * q + j]);
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
