// k_beam.cuh -- selection over beams and vocabulary.
//
// With lse[k] = log sum_v exp(l[k, v]) a candidate (k, v) is worth
//   c[k, v] = score[k] + l[k, v] - lse[k],
// and the n best of a batch entry are taken, ties to the lowest k V + v.
// Within a beam the order of c is that of l, so each beam's n largest logits
// are enough: k_beam_rows finds them and lse, k_beam_merge the n best of the
// beams' lists, by c in 64 bits.
#pragma once
#include <cuda_bf16.h>
#include "fm_common.cuh"

namespace fm {

constexpr int kBeamMax = 32;  // beams and n_out
constexpr int kBeamThreads = 256;

// One candidate as a 64-bit key whose order is (larger logit, lower index):
// the fp32 bits made monotone above the complement of the index.  0: none.
__device__ __forceinline__ unsigned long long beam_key(float l, unsigned v) {
  const unsigned b = __float_as_uint(l);
  const unsigned m = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((unsigned long long)m << 32) | (0xFFFFFFFFu - v);
}
__device__ __forceinline__ float beam_key_logit(unsigned long long k) {
  const unsigned m = (unsigned)(k >> 32);
  return __uint_as_float(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
}
__device__ __forceinline__ unsigned beam_key_index(unsigned long long k) {
  return 0xFFFFFFFFu - (unsigned)k;
}

// NaN counts as -inf, +inf as the largest finite value; -0 as 0 (equal values
// must tie)
__device__ __forceinline__ float beam_logit(float l) {
  return fminf(fmaxf(l, -INFINITY), 3.402823466e38f) + 0.0f;
}
__device__ __forceinline__ float beam_load(const float *p) { return beam_logit(*p); }
__device__ __forceinline__ float beam_load(const __nv_bfloat16 *p) {
  return beam_logit(__bfloat162float(*p));
}

__device__ __forceinline__ unsigned long long cta_max_key(unsigned long long k,
                                                          unsigned long long *s_red) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long x = __shfl_xor_sync(0xffffffffu, k, o);
    k = x > k ? x : k;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = k;
  __syncthreads();
  k = s_red[0];
  for (int i = 1; i < kBeamThreads / 32; ++i) k = s_red[i] > k ? s_red[i] : k;
  return k;
}

// Workspace: keys [rows, n_out] (descending, 0 where there is none), lse [rows].
template <typename T>
__global__ void __launch_bounds__(kBeamThreads)
    k_beam_rows(const T *__restrict__ logits, long long ld, unsigned V, int n_out,
                unsigned long long *__restrict__ keys, double *__restrict__ lse) {
  pdl_wait();
  pdl_trigger();
  __shared__ unsigned long long s_key[kBeamThreads / 32];
  __shared__ double s_sum[kBeamThreads / 32];
  const T *row = logits + blockIdx.x * ld;
  unsigned long long last = ~0ull;
  float top = 0.0f;
  for (int n = 0; n < n_out; ++n) {
    unsigned long long best = 0;
    for (unsigned v = threadIdx.x; v < V; v += kBeamThreads) {
      const float l = beam_load(row + v);
      const unsigned long long k = l > -INFINITY ? beam_key(l, v) : 0;
      if (k < last && k > best) best = k;
    }
    best = cta_max_key(best, s_key);
    if (n == 0) top = beam_key_logit(best);
    if (threadIdx.x == 0) keys[(size_t)blockIdx.x * n_out + n] = best;
    last = best;
  }
  double sum = 0.0;
  for (unsigned v = threadIdx.x; v < V; v += kBeamThreads)
    sum += (double)expf(beam_load(row + v) - top);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kBeamThreads / 32; ++i) sum += s_sum[i];
    lse[blockIdx.x] = (double)top + log(sum);
  }
}

// One warp per batch entry: lane k walks beam k's list.
__global__ void __launch_bounds__(32)
    k_beam_merge(const unsigned long long *__restrict__ keys, const double *__restrict__ lse,
                 int beams, const float *scores, const uint8_t *finished, int eos, int n_out,
                 float *out_scores, int32_t *parent, int32_t *token, uint8_t *out_finished) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x;
  const long long row = (long long)blockIdx.x * beams + lane;
  const bool live = lane < beams;
  const float sc = live ? scores[row] : -INFINITY;
  const bool done = live && finished && finished[row];
  const bool dead = !(sc > -INFINITY);
  const double base = live && !done ? lse[row] : 0.0;
  int at = 0;
  auto value = [&](unsigned &v) -> double {
    if (dead || !live) return -INFINITY;
    if (done) {
      v = (unsigned)eos;
      return at == 0 ? (double)sc : -INFINITY;
    }
    const unsigned long long k = at < n_out ? keys[row * n_out + at] : 0;
    if (!k) return -INFINITY;
    v = beam_key_index(k);
    return ((double)beam_key_logit(k) - base) + (double)sc;
  };
  unsigned v = 0;
  double c = value(v);
  __syncwarp();
  for (int n = 0; n < n_out; ++n) {
    // the lane with the largest c (the lowest lane of equal ones: beams are in
    // lane order, so that is the lowest k V + v)
    double m = c;
    int who = lane;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      const double mo = __shfl_xor_sync(0xffffffffu, m, o);
      const int wo = __shfl_xor_sync(0xffffffffu, who, o);
      if (mo > m || (mo == m && wo < who)) {
        m = mo;
        who = wo;
      }
    }
    const long long o = (long long)blockIdx.x * n_out + n;
    const bool none = !(m > -INFINITY);
    if (none) {
      if (lane == 0) {
        out_scores[o] = -INFINITY;
        parent[o] = n % beams;
        token[o] = -1;
        if (out_finished) out_finished[o] = 0;
      }
    } else if (lane == who) {
      out_scores[o] = fmaxf((float)c, -3.402823466e38f);
      parent[o] = who;
      token[o] = (int32_t)v;
      if (out_finished) out_finished[o] = done || (int)v == eos;
      ++at;
      c = value(v);
    }
    __syncwarp();
  }
}

}  // namespace fm
