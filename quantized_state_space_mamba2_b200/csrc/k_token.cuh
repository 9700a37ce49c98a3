// k_token.cuh -- row-wise kernels of the token loop around a stack: residual
// addition + RMSNorm + 8-bit codes, embedding rows, and the reordering of
// carried states after a beam selection.  All three are bound by memory.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <type_traits>
#include "fm_common.cuh"

namespace fm {

// ------------------------------------------------------------ fp8 helpers
// two fp32 -> two e4m3 codes (round to nearest even, saturating): lo in bits 0-7
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// four e4m3 codes -> fp32 (exact)
__device__ __forceinline__ float4 e4m3x4_f32(uint32_t c) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(c));
  const float2 lo = __half22float2(*reinterpret_cast<__half2 *>(&a));
  const float2 hi = __half22float2(*reinterpret_cast<__half2 *>(&b));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// four consecutive elements as fp32
__device__ __forceinline__ float4 load4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}

// ------------------------------------------------------------ add + norm + codes
// r = fl(x + residual); y = r w / sqrt(mean(r^2) + eps); codes q = nearest(y / s)
// with s = fl(max|y| / 448) per 128 columns (e4m3) or fl(max|y| / 127) per row
// (int8).  The codes are those of the exact quotient (64-bit sums and
// statistics; an fp32 product decides a code unless it lies so near the middle
// between two codes that its rounding could, and that element is then redone
// in 64 bits), so they do not depend on the order of any fp32 sum.
//
// A CTA walks rows, one warp per 512 columns: 8 lanes hold a 128-column block,
// lane l of them the four groups of 4 columns at 4 l + 32 j, so every load of
// the 8 lanes is one run of 128 bytes (fp32) and a block's maximum takes three
// shuffles.  A row stays in registers: one read of x and residual, one write of
// the sum, the codes and the scales; the weights are read once per CTA.
//
// Up to kNormAheadK columns the next row is on its way while this one is computed:
// 8192 x 2560 fp32 with residual 51 us, 5.3 TB/s, bound by instruction issue.  Wider
// rows, whose 11 to 32 warps leave no registers for a second row, take the variant
// with one CTA per row, which waits for its loads (2048 x 8192: 49 us, 4.4 TB/s;
// 1024 x 16384: 60 us, 3.7 TB/s; 64 registers, 40 bytes of them spilled).  At
// widths that both can run (fp32 with residual to e4m3): 4096 x 5120 47.5 us ahead,
// 57.2 one per row; 4096 x 2560 25.9 and 28.2; 64 x 2560 3.2 and 3.4.  Rows of one
// or two warps, a row or two per CTA, are bound by the chain of a row (loads,
// barriers) either way: 2049 x 768 bf16 to int8 6.7 and 6.5 us.
constexpr int kNormCols = 512;   // columns per warp
constexpr int kNormMaxK = 32 * kNormCols;
constexpr int kNormAheadWarps = 10, kNormAheadK = kNormAheadWarps * kNormCols;
constexpr float kNormTiny = 7.888609052210118e-31f;  // 2^-100: a smaller max|y| counts as zero

__device__ __forceinline__ uint32_t group8_max(uint32_t v) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float group8_max(float v) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// v rounded to fp32 towards zero with the lost bits kept as a last 1: a later
// rounding to fewer than 22 bits is then that of v itself
__device__ __forceinline__ float sticky(double v) {
  float f = __double2float_rz(v);
  if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// Whether t, within 4 ulp of y / s, may round to another code than it does:
// e4m3: a tie of two codes has the low 20 of its 23 fraction bits at 0x80000;
// below the normal codes (|t| < 2^-6) and not under half the smallest one
// (2^-10) the spacing is fixed, and the few values there are always redone.
__device__ __forceinline__ bool e4m3_near(float t) {
  const uint32_t a = __float_as_uint(t) & 0x7FFFFFFFu;
  return (a & 0xFFFFFu) - 0x7FFF8u <= 16u || a - 0x3A7FF000u < 0x3C800000u - 0x3A7FF000u;
}
// int8: |y / s| <= 127, so t is within 127 * 4 * 2^-24 < 2^-15 of it
__device__ __forceinline__ bool int8_near(float t) {
  return fabsf(__fsub_rn(t, rintf(t))) > 0.5f - 0x1p-14f;
}

// four elements of a row in their stored type
struct NormRaw4f {
  float4 v;
  __device__ __forceinline__ void load(const float *p) { v = load4(p); }
  __device__ __forceinline__ float4 f32() const { return v; }
};
struct NormRaw4b {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    u = *reinterpret_cast<const uint2 *>(p);
  }
  __device__ __forceinline__ float4 f32() const {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
  }
};
template <typename TX>
using NormRaw = std::conditional_t<sizeof(TX) == 4, NormRaw4f, NormRaw4b>;

template <typename TX, bool E4M3, bool kAhead>
__global__ void __launch_bounds__(kAhead ? 32 * kNormAheadWarps : 1024, kAhead ? 2 : 1)
    k_add_norm_quant(const TX *x, long long ldx, const float *residual, long long ldr, long long M,
                     int K, double inv_k, const float *__restrict__ norm_w, double eps,
                     uint8_t *__restrict__ q, float *__restrict__ s, float *sum_out,
                     long long lds) {
  pdl_wait();
  pdl_trigger();
  // by the row's parity: a warp is never more than one row ahead of another
  __shared__ double s_ss[2][32];
  __shared__ uint32_t s_max[2][32];
  __shared__ float s_rem[2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int col0 = warp * kNormCols + (lane >> 3) * 128 + (lane & 7) * 4;
  float w[16];
  if constexpr (kAhead) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = col0 + 32 * j;
      const float4 g = c < K ? load4(norm_w + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      w[4 * j] = g.x; w[4 * j + 1] = g.y; w[4 * j + 2] = g.z; w[4 * j + 3] = g.w;
    }
  }
  NormRaw<TX> nx[4];
  float4 nr[4];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = col0 + 32 * j;
      if (c < K) {
        nx[j].load(x + row * ldx + c);
        if (residual) nr[j] = load4(residual + row * ldr + c);
      } else {
        nx[j] = {};
        nr[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  };
  if (kAhead) fetch(blockIdx.x);
  int odd = 0;
  for (long long row = blockIdx.x; row < M; row += gridDim.x, odd ^= 1) {
    if (!kAhead) fetch(row);
    float r[16];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 v = nx[j].f32();
      if (residual) {
        v.x = __fadd_rn(v.x, nr[j].x); v.y = __fadd_rn(v.y, nr[j].y);
        v.z = __fadd_rn(v.z, nr[j].z); v.w = __fadd_rn(v.w, nr[j].w);
      }
      const int c = col0 + 32 * j;
      if (sum_out && c < K) *reinterpret_cast<float4 *>(sum_out + row * lds + c) = v;
      r[4 * j] = v.x; r[4 * j + 1] = v.y; r[4 * j + 2] = v.z; r[4 * j + 3] = v.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __fma_rn((double)r[4 * j + i], (double)r[4 * j + i], ss);
      if constexpr (!kAhead) {
        const float4 g = c < K ? load4(norm_w + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        w[4 * j] = g.x; w[4 * j + 1] = g.y; w[4 * j + 2] = g.z; w[4 * j + 3] = g.w;
      }
    }
    if (kAhead && row + gridDim.x < M) fetch(row + gridDim.x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss = __dadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
    if (lane == 0) s_ss[odd][warp] = ss;
    __syncthreads();
    ss = s_ss[odd][0];
    for (int i = 1; i < nw; ++i) ss = __dadd_rn(ss, s_ss[odd][i]);
    if (!(ss <= 1.7e308) && threadIdx.x == 0) raise_error(kErrNonfinite);
    const double rstd = rsqrt(__fma_rn(ss, inv_k, eps));
    // rstd = rs 2^e with rs in [1, 2): r 2^e is exact and at most about sqrt(K),
    // so the products below cannot overflow whatever the row's magnitude
    const long long rb = __double_as_longlong(rstd);
    const int e = (int)((rb >> 52) & 0x7FF) - 1023;
    const double rs = __longlong_as_double((rb & 0xFFFFFFFFFFFFFll) | 0x3FF0000000000000ll);
    const float pe = e >= -126 && e <= 127 ? __int_as_float((127 + e) << 23) : ldexpf(1.0f, e);
    float p[16];
    uint32_t mb = 0;  // bits of the largest |p|: ordered as the values, NaN above all
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      r[i] = __fmul_rn(r[i], pe);
      p[i] = __fmul_rn(r[i], w[i]);
      mb = max(mb, __float_as_uint(p[i]) & 0x7FFFFFFFu);
    }
    // max|r w| exactly: the largest fp32 product plus the largest exact
    // remainder among the elements that round to it
    mb = group8_max(mb);
    if (!E4M3) {
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 8));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 16));
      if (lane == 0) s_max[odd][warp] = mb;
      __syncthreads();
      mb = s_max[odd][0];
      for (int i = 1; i < nw; ++i) mb = max(mb, s_max[odd][i]);
    }
    if (mb >= 0x7F800000u) raise_error(kErrNonfinite);
    const float m = __uint_as_float(mb);
    float rem = -3.0e38f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (fabsf(p[i]) == m) rem = fmaxf(rem, __fmaf_rn(fabsf(r[i]), fabsf(w[i]), -m));
    rem = group8_max(rem);
    if (!E4M3) {
      rem = fmaxf(rem, __shfl_xor_sync(0xffffffffu, rem, 8));
      rem = fmaxf(rem, __shfl_xor_sync(0xffffffffu, rem, 16));
      if (lane == 0) s_rem[odd][warp] = rem;
      __syncthreads();
      rem = s_rem[odd][0];
      for (int i = 1; i < nw; ++i) rem = fmaxf(rem, s_rem[odd][i]);
    }
    double amax = __dmul_rn(__dadd_rn((double)m, (double)rem), rs);
    // below 2^-100 (which covers every p that lost bits to underflow): zeros
    if (!(m > 0.0f) || amax < (double)kNormTiny) amax = 0.0;
    const float sc = (float)__dmul_rn(amax, E4M3 ? 1.0 / 448.0 : 1.0 / 127.0);
    const float cf = sc > 0.0f ? __fdiv_rn((float)rs, sc) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = col0 + 32 * j;
      float t[4];
      bool near = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[i] = __fmul_rn(p[4 * j + i], cf);
        near = near || (E4M3 ? e4m3_near(t[i]) : int8_near(t[i]));
      }
      if (near && sc > 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t[i] = sticky(__ddiv_rn(
              __dmul_rn(__dmul_rn((double)r[4 * j + i], (double)w[4 * j + i]), rs), (double)sc));
      }
      uint32_t o;
      if constexpr (E4M3) {
        o = e4m3x2(t[0], t[1]) | (e4m3x2(t[2], t[3]) << 16);
      } else {
        o = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) o |= (uint32_t)(quant127(t[i]) & 0xFF) << (8 * i);
      }
      if (col < K) *reinterpret_cast<uint32_t *>(q + row * K + col) = o;
    }
    if constexpr (E4M3) {
      const int nb = (K + 127) / 128, b = warp * 4 + (lane >> 3);
      if ((lane & 7) == 0 && b < nb) s[row * nb + b] = sc;
    } else {
      if (threadIdx.x == 0) s[row] = sc;
    }
  }
}

// Offline: W [N, K] fp32 -> e4m3 codes and one scale per 128 x 128 block,
// s = fl(max|W| / 448), code = nearest(W / s).  One CTA of 256 threads per block,
// which reads it twice (50000 x 2560: 211 us, 3.0 TB/s of weights and codes).
__global__ void __launch_bounds__(256) k_prepare_linear_fp8(const float *__restrict__ W, long long N,
                                                            int K, uint8_t *__restrict__ Wq,
                                                            float *__restrict__ s_w) {
  pdl_wait();
  __shared__ float s_red[8];
  const int k0 = blockIdx.x * 128;
  const long long n0 = (long long)blockIdx.y * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = k0 + 4 * lane;
  uint32_t a_bits = 0;  // of the largest |W|: ordered as the values, NaN above all
  for (int i = warp; i < 128; i += 8)
    if (n0 + i < N && k < K) {
      const float4 v = load4(W + (n0 + i) * K + k);
      a_bits = max(a_bits, max(max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu),
                               max(__float_as_uint(v.z) & 0x7FFFFFFFu, __float_as_uint(v.w) & 0x7FFFFFFFu)));
    }
  if (a_bits >= 0x7F800000u) raise_error(kErrNonfinite);
  float a = warp_max(__uint_as_float(a_bits));
  if (lane == 0) s_red[warp] = a;
  __syncthreads();
  a = warp_max(lane < 8 ? s_red[lane] : 0.0f);
  if (a < kNormTiny) a = 0.0f;
  const float s = (float)__ddiv_rn((double)a, 448.0);
  // A quotient in 64 bits is on the tie's side that W / s is on: a tie has 5 bits
  // and s 24, so W / s is a tie exactly, or off by more than 2^-30 of it.  (A
  // product with 1 / s can miss an exact tie.)
  auto arg = [s](float v) { return s > 0.0f ? sticky(__ddiv_rn((double)v, (double)s)) : 0.0f; };
  for (int i = warp; i < 128; i += 8)
    if (n0 + i < N && k < K) {
      const float4 v = load4(W + (n0 + i) * K + k);
      *reinterpret_cast<uint32_t *>(Wq + (n0 + i) * K + k) =
          e4m3x2(arg(v.x), arg(v.y)) | (e4m3x2(arg(v.z), arg(v.w)) << 16);
    }
  if (threadIdx.x == 0) s_w[(long long)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// ------------------------------------------------------------ embedding rows
// x[m] = scale * table[ids[m]]; an id of -1 (padding) gives zeros, any other id
// outside [0, V) zeros and the device error word.  One warp per 512 columns of a
// row, all their loads on their way at once: bound by memory, two thirds of the
// bytes of a bf16 table's rows being written (8192 x 2560 from bf16: 20.8 us, 6.1
// TB/s; 24.4 before), and by one load's latency where there are few rows (a warp per row, a
// load per 128 columns after another: 5.1 us for 64 x 2560 in a graph).
// TYPE 0: fp32 table, 1: bf16, 2: e4m3 codes with a scale per 128 x 128 block.
constexpr int kEmbedCols = 512;  // columns per warp

template <int TYPE>
__global__ void __launch_bounds__(128) k_embed_rows(const int32_t *__restrict__ ids, long long M,
                                                    const void *__restrict__ table,
                                                    const float *__restrict__ table_s, long long V,
                                                    int K, int pieces, float scale,
                                                    float *__restrict__ x, long long ldx) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long row = w / pieces;
  if (row >= M) return;
  const int c0 = (int)(w - row * pieces) * kEmbedCols + 4 * lane;
  const long long id = ids[row];
  const bool live = id >= 0 && id < V;
  if (!live && id != -1 && c0 == 0) raise_error(kErrIndex);
  const int nb = (K + 127) / 128;
  float4 v[kEmbedCols / 128];
#pragma unroll
  for (int j = 0; j < kEmbedCols / 128; ++j) {
    const int c = c0 + 128 * j;
    v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && c < K) {
      if constexpr (TYPE == 0) v[j] = load4((const float *)table + id * K + c);
      if constexpr (TYPE == 1) v[j] = load4((const __nv_bfloat16 *)table + id * K + c);
      if constexpr (TYPE == 2) {
        v[j] = e4m3x4_f32(*reinterpret_cast<const uint32_t *>((const uint8_t *)table + id * K + c));
        const float s = table_s[(id >> 7) * nb + (c >> 7)];
        v[j].x = __fmul_rn(v[j].x, s); v[j].y = __fmul_rn(v[j].y, s);
        v[j].z = __fmul_rn(v[j].z, s); v[j].w = __fmul_rn(v[j].w, s);
      }
      v[j].x = __fmul_rn(v[j].x, scale); v[j].y = __fmul_rn(v[j].y, scale);
      v[j].z = __fmul_rn(v[j].z, scale); v[j].w = __fmul_rn(v[j].w, scale);
    }
  }
#pragma unroll
  for (int j = 0; j < kEmbedCols / 128; ++j)
    if (c0 + 128 * j < K) *reinterpret_cast<float4 *>(x + row * ldx + c0 + 128 * j) = v[j];
}

// ------------------------------------------------------------ state reordering
// dst[b, j] = src[b, parent[b, j]] for every buffer, in place where src = dst.
// A thread owns one unit (16 bytes where rows allow it) of a row's columns for
// all the beams of one batch entry: it reads every beam's new value before it
// writes any, so no second buffer and no order between threads is needed.
// In place, a beam that keeps its own state is neither read nor written.  A
// parent outside the source's beams leaves the row as it was and sets the
// device error word.  Like every kernel that writes a carried state it issues no
// early trigger: k_scan_step loads its state before its dependency wait.
// Bound by memory: 64 layers of 4 x 8 beams, 5.4 GB of int32 states, 1.15 ms, 7.0
// TB/s of what has to move (source rows that several beams take come from L2).
constexpr int kReorderBufs = 128;  // buffers per launch
constexpr int kReorderBeams = 32;
constexpr int kReorderThreads = 256;

struct ReorderArgs {
  const void *src[kReorderBufs];
  void *dst[kReorderBufs];
  unsigned first[kReorderBufs + 1];  // first block of each buffer
  unsigned units[kReorderBufs];      // units per row
  int n, src_beams, dst_beams;
  const int32_t *parent;
};

template <typename U, int G>
__global__ void __launch_bounds__(kReorderThreads)
    k_reorder_rows(const __grid_constant__ ReorderArgs a) {
  pdl_wait();
  int lo = 0, hi = a.n;  // the buffer of this block
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const unsigned units = a.units[lo];
  const unsigned col = (blockIdx.x - a.first[lo]) * kReorderThreads + threadIdx.x;
  if (col >= units) return;
  const U *src = (const U *)a.src[lo] + (size_t)blockIdx.y * a.src_beams * units + col;
  U *dst = (U *)a.dst[lo] + (size_t)blockIdx.y * a.dst_beams * units + col;
  const bool same = a.src[lo] == a.dst[lo];
  const int32_t *par = a.parent + (size_t)blockIdx.y * a.dst_beams;
  U v[G];
  unsigned moved = 0;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    if (j < a.dst_beams) {
      const int p = par[j];
      if (p < 0 || p >= a.src_beams) {
        if (col == 0) raise_error(kErrIndex);
      } else if (!same || p != j) {
        v[j] = src[(size_t)p * units];
        moved |= 1u << j;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < G; ++j)
    if (moved >> j & 1u) dst[(size_t)j * units] = v[j];
}

}  // namespace fm
