// k_fp8.cuh -- e4m3 matrix product with a scale for each block of 128:
//   Y[m, n] = sum_b s_a[m, b] s_w[n / 128, b] sum_{k in block b} A[m, k] W[n, k].
#pragma once
#include <cuda_bf16.h>
#include "k_gemm.cuh"
#include "k_token.cuh"

namespace fm {

// 64 x 64 outputs per CTA, 4 x 4 per thread, 16 columns of K at a time.
template <typename TY>
__global__ void __launch_bounds__(256)
    k_fp8_gemm_simple(const uint8_t *__restrict__ A, const float *__restrict__ s_a, long long M,
                      const uint8_t *__restrict__ W, const float *__restrict__ s_w, long long N,
                      int K, TY *__restrict__ Y, long long ldy) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sa[64][17], sw[64][17];
  const long long m0 = (long long)blockIdx.y * 64, n0 = (long long)blockIdx.x * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int nb = (K + 127) / 128;
  float acc[4][4] = {}, part[4][4] = {};
  const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 4;
  for (int k0 = 0; k0 < K; k0 += 16) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), w = a;
    if (m0 + lr < M) a = e4m3x4_f32(*(const uint32_t *)(A + (m0 + lr) * K + k0 + lc));
    if (n0 + lr < N) w = e4m3x4_f32(*(const uint32_t *)(W + (n0 + lr) * K + k0 + lc));
    __syncthreads();
    sa[lr][lc] = a.x; sa[lr][lc + 1] = a.y; sa[lr][lc + 2] = a.z; sa[lr][lc + 3] = a.w;
    sw[lr][lc] = w.x; sw[lr][lc + 1] = w.y; sw[lr][lc + 2] = w.z; sw[lr][lc + 3] = w.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part[i][j] = __fmaf_rn(sa[ty + 16 * i][k], sw[tx + 16 * j][k], part[i][j]);
    if ((k0 & 127) == 112 || k0 + 16 >= K) {
      const int b = k0 >> 7;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
          if (m < M && n < N)
            acc[i][j] = __fmaf_rn(__fmul_rn(s_a[m * nb + b], s_w[(n >> 7) * nb + b]), part[i][j],
                                  acc[i][j]);
          part[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < M && n < N) Y[m * ldy + n] = (TY)acc[i][j];
    }
}

}  // namespace fm
