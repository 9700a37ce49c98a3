// k_beam.cuh -- selection over beams and vocabulary.
//
// With lse[k] = log sum_v exp(l[k, v]) a candidate (k, v) is worth
//   c[k, v] = score[k] + l[k, v] - lse[k],
// and the n best of a batch entry are taken, ties to the lowest k V + v.
// Within a beam the order of c is that of l, so each beam's n largest logits
// are enough.  k_beam_chunks reads the logits once: a CTA holds a chunk of one
// beam's row in registers and leaves its maximum, its sum of exponentials and
// its n largest logits; k_beam_merge joins the chunks' sums and lists and takes
// the n best of the beams' lists by c, whose log sums it forms again in 64 bits
// where the fp32 exponentials do not tell which candidate is worth more.
//
// What bounds it is the chain of each chunk (its loads, the maxima, the sum, the
// few candidates), so an SM holds as many chunks as its 64 warps allow: 16
// logits per thread, 8 CTAs (32 registers per thread; 56 bytes of a bf16 thread's
// and 88 of an fp32 one's do not fit and are spilled).  64 x 8 x 100003 bf16, a
// fifth of the beams finished and so not read: 53.6 us for the 80 MB of the others,
// 1.5 TB/s (32 per thread, 4 CTAs: 61.7; 8 per thread: 88; a warp by itself over a
// span of the row, without barriers: 73, its code and registers too large).
// The n largest of a chunk are found without
// sorting it: the n-th largest of 32 group maxima (groups of 8 threads) is not
// above the chunk's n-th largest value, so few values reach it; they are
// collected and ranked against each other.  Where ties or masks let more than
// kBeamCap through, n rounds of a maximum over the registers find them instead.
#pragma once
#include <cuda_bf16.h>
#include "fm_common.cuh"

namespace fm {

constexpr int kBeamMax = 32;  // beams and n_out
constexpr int kBeamThreads = 256;

// One candidate as a 64-bit key whose order is (larger logit, lower index):
// the fp32 bits made monotone above the complement of the index.  0: none.  (l
// is not -0: the caller adds 0, so that equal values tie.)
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

// NaN counts as -inf, +inf as the largest finite value
__device__ __forceinline__ float beam_logit(float l) {
  return fminf(fmaxf(l, -INFINITY), 3.402823466e38f);
}
constexpr int kBeamCap = 512;

// A thread's E elements of a row's chunk: groups of 16 bytes, 256 threads side
// by side.  Which thread holds an element does not depend on where the row lies
// in memory, so equal rows have equal sums and their ties stay ties.  In a row
// that is not 16-byte aligned a group is cut from the two aligned vectors that
// cover it (the second is the neighbour's first, in L1).  Elements behind the
// row are -inf.
template <typename T, int E>
struct BeamChunk {
  static constexpr int kVec = 16 / (int)sizeof(T);  // elements per group
  float v[E];
  unsigned first;
  __device__ __forceinline__ unsigned at(int i) const {  // the element's index
    return first + (unsigned)(i / kVec * (kBeamThreads * kVec) + i % kVec);
  }
  __device__ __forceinline__ void load(const T *row, unsigned V, unsigned chunk) {
    const unsigned skew = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u);  // bytes
    first = chunk * (unsigned)(kBeamThreads * E) + threadIdx.x * kVec;
#pragma unroll
    for (int j = 0; j < E / kVec; ++j) {
      const unsigned p = first + j * (kBeamThreads * kVec);  // V < 2^31
      if (p + 2 * kVec <= V) {
        const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(row + p) - skew);
        const uint4 x = q[0];
        uint32_t w[8] = {x.x, x.y, x.z, x.w, 0, 0, 0, 0};
        if (skew) {  // the same for the whole CTA
          const uint4 y = q[1];
          w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
          if (skew & 8) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
          }
          if (skew & 4) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
          }
          if (sizeof(T) == 2 && (skew & 2)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 4) {
            v[4 * j + i] = __uint_as_float(w[i]);
          } else {
            v[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          v[kVec * j + i] = p + i < V ? (float)row[p + i] : -INFINITY;
      }
    }
  }
};

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

// One CTA per chunk of 256 E logits, S chunks per row.
// Workspace: keys [rows, S, n_out] (descending, 0 where there is none), top
// [rows, S] (the chunk's maximum) and sum [rows, S] (of exp(l - top)).
// A row that cannot win by its logits -- its beam finished or dead -- is not read.
template <typename T, int E>
__global__ void __launch_bounds__(kBeamThreads, 8)
    k_beam_chunks(const T *__restrict__ logits, long long ld, unsigned V, int S, int n_out,
                  const float *__restrict__ scores, const uint8_t *__restrict__ finished,
                  unsigned long long *__restrict__ keys, float *__restrict__ tops,
                  double *__restrict__ sums) {
  pdl_wait();
  pdl_trigger();
  constexpr int kVec = BeamChunk<T, E>::kVec, kGroups = E / kVec;
  __shared__ float4 s_max[kBeamThreads / 4];
  __shared__ double s_sum[kBeamThreads / 32];
  __shared__ unsigned long long s_key[kBeamCap];
  __shared__ float s_bar;
  __shared__ int s_count;
  const unsigned row = blockIdx.x / S, chunk = blockIdx.x - row * S;
  const float score = scores[row];  // both loads on their way at once
  const uint8_t done = finished ? finished[row] : 0;
  if (done | !(score > -INFINITY)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_count = 0;
  BeamChunk<T, E> c;
  c.load(logits + (long long)row * ld, V, chunk);
  float gm[kGroups], top, sum;
  // maxima of the thread's 16-byte groups and of the chunk (NaN counts as
  // nothing there), then the sum
  auto maxima = [&]() {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      gm[j] = c.v[j * kVec];
#pragma unroll
      for (int i = 1; i < kVec; ++i) gm[j] = fmaxf(gm[j], c.v[j * kVec + i]);
      m = fmaxf(m, gm[j]);
    }
    reinterpret_cast<float *>(s_max)[threadIdx.x] = m;
    __syncthreads();
    const float4 x = s_max[2 * lane], y = s_max[2 * lane + 1];
    const float g = fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)),
                          fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)));  // of threads 8 lane .. + 7
    top = warp_max(g);
    return g;
  };
  auto exponentials = [&]() {
    sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        float e;  // exp(l - top), within 2^-22 and the argument's rounding
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((c.v[i] - top) * 1.4426950408889634f));
        sum += e;
      }
    }
  };
  float g = maxima();
  exponentials();
  if (__syncthreads_or(!(sum < INFINITY))) {
    // a NaN, or +inf as the maximum: the values the definition gives them
#pragma unroll
    for (int i = 0; i < E; ++i) c.v[i] = beam_logit(c.v[i]);
    g = maxima();
    exponentials();
  }
  if (warp == 0) {
    // the n-th largest group maximum; values of -inf are no candidates
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, g, j);
      rank += o > g || (o == g && j < lane);
    }
    if (rank == n_out - 1) s_bar = fmaxf(g, -3.402823466e38f);
  }
  double total = (double)sum;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;
  __syncthreads();
  const float bar = s_bar;
#pragma unroll
  for (int j = 0; j < kGroups; ++j)
    if (gm[j] >= bar) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (c.v[j * kVec + i] >= bar) {
          const int at = atomicAdd(&s_count, 1);
          if (at < kBeamCap) s_key[at] = beam_key(c.v[j * kVec + i] + 0.0f, c.at(j * kVec + i));
        }
    }
  __syncthreads();
  unsigned long long *out = keys + (size_t)blockIdx.x * n_out;
  const int count = s_count;
  if (threadIdx.x == 0) {
    total = s_sum[0];
    for (int i = 1; i < kBeamThreads / 32; ++i) total += s_sum[i];
    tops[blockIdx.x] = top;
    sums[blockIdx.x] = total;
  }
  if (count <= kBeamCap) {
    for (int i = threadIdx.x; i < max(count, n_out); i += kBeamThreads) {
      if (i >= count) {
        out[i] = 0;  // fewer values than slots
        continue;
      }
      const unsigned long long k = s_key[i];
      int r = 0;
      for (int j = 0; j < count; ++j) r += s_key[j] > k;
      if (r < n_out) out[r] = k;
    }
    return;
  }
  unsigned long long last = ~0ull;
  for (int n = 0; n < n_out; ++n) {
    unsigned long long best = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const unsigned long long k = c.v[i] > -INFINITY ? beam_key(c.v[i] + 0.0f, c.at(i)) : 0;
      if (k < last && k > best) best = k;
    }
    last = cta_max_key(best, s_key);
    if (threadIdx.x == 0) out[n] = last;
  }
}

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const unsigned long long x = __shfl_xor_sync(0xffffffffu, k, o);
    k = x > k ? x : k;
  }
  return k;
}

// sum_v exp(l[v] - top) of a row in 64 bits, by the whole CTA (its result in
// thread 0): which thread adds an element depends on its index alone.
template <typename T>
__device__ __forceinline__ double beam_exact_sum(const T *__restrict__ row, unsigned V,
                                                 double top, double *s_part) {
  double t = 0.0;
#pragma unroll 1  // four at once need more registers than 32 warps have
  for (unsigned i = threadIdx.x; i < V; i += blockDim.x)
    t += exp((double)beam_logit((float)row[i]) - top);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  __syncthreads();  // s_part's last values have been read
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = t;
  __syncthreads();
  t = 0.0;
  if (threadIdx.x == 0)
    for (unsigned i = 0; i < blockDim.x / 32; ++i) t += s_part[i];
  return t;
}

// One CTA per batch entry, one warp per beam for its log sum and its n largest
// logits (the largest key below the last one, n times over its chunks' lists),
// then one warp, lane k at the head of beam k's list.
//
// The chunks' log sums are off by up to tol each, so the order of two beams'
// candidates that lie within it is not known yet: the log sums of such beams are
// then formed again, in 64 bits from the logits, and the lists merged once more.
// Compared are neighbours in the merged order of different beams (gaps that each
// exceed both beams' errors add up to more than those of the two ends), and the
// last one taken with the head of each list: 0.5 us (1 x 4 x 32001 in a graph 7.3
// us, 6.8 without).  Random logits call for new sums in some 10^-4 of the entries,
// equal rows with equal scores always (64 x 8 x 100003 bf16: 509 us then, 53.6 us
// on random logits; 1760 us with 8 warps per CTA).  More warps than beams are there
// for that work alone.

template <typename T>
__global__ void __launch_bounds__(32 * kBeamMax)
    k_beam_merge(const unsigned long long *__restrict__ keys, const float *__restrict__ tops,
                 const double *__restrict__ sums, int S, int beams, const T *__restrict__ logits,
                 long long ld, unsigned V, double tol, const float *scores, const uint8_t *finished,
                 int eos, int n_out, float *out_scores, int32_t *parent, int32_t *token,
                 uint8_t *out_finished) {
  pdl_wait();
  pdl_trigger();
  __shared__ unsigned long long s_list[kBeamMax][kBeamMax];
  __shared__ double s_lse[kBeamMax], s_part[kBeamMax];
  __shared__ float s_score[kBeamMax], s_top[kBeamMax];
  __shared__ uint8_t s_done[kBeamMax];
  __shared__ unsigned s_redo;
  const int lane = threadIdx.x & 31, beam = threadIdx.x >> 5;
  if (beam < beams) {
    const long long row = (long long)blockIdx.x * beams + beam;
    // every first load on its way at once (what a row that was not read left in
    // the workspace is loaded too, and not used)
    const float score = scores[row];
    const uint8_t flag = finished ? finished[row] : 0;
    const float *tp = tops + row * S;
    const double *sp = sums + row * S;
    const unsigned long long *kp = keys + row * S * n_out;
    const int all = S * n_out;
    constexpr int kHold = 8;  // keys per lane held in registers
    unsigned long long own[kHold], last = ~0ull;
#pragma unroll
    for (int i = 0; i < kHold; ++i) own[i] = 32 * i + lane < all ? kp[32 * i + lane] : 0;
    const float top = lane < S ? tp[lane] : -INFINITY;
    const double sum = lane < S ? sp[lane] : 0.0;
    const bool finish = flag != 0, dead = !(score > -INFINITY);
    if (lane == 0) {
      s_score[beam] = score;
      s_done[beam] = finish;
    }
    if (!finish && !dead) {
      float m = top;
      for (int i = 32 + lane; i < S; i += 32) m = fmaxf(m, tp[i]);
      m = warp_max(m);
      double t = sum > 0.0 ? sum * exp((double)top - (double)m) : 0.0;
      for (int i = 32 + lane; i < S; i += 32)
        if (sp[i] > 0.0) t += sp[i] * exp((double)tp[i] - (double)m);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) {
        s_lse[beam] = (double)m + log(t);
        s_top[beam] = m;
      }
      for (int n = 0; n < n_out; ++n) {
        unsigned long long best = 0;
#pragma unroll
        for (int i = 0; i < kHold; ++i)
          if (own[i] < last && own[i] > best) best = own[i];
        for (int i = 32 * kHold + lane; i < all; i += 32)
          if (kp[i] < last && kp[i] > best) best = kp[i];
        last = warp_max_key(best);
        if (lane == 0) s_list[beam][n] = last;
        if (last == 0) {
          for (int j = n + 1 + lane; j < n_out; j += 32) s_list[beam][j] = 0;
          break;
        }
      }
    }
  }
  __syncthreads();
  unsigned rough = 0;  // beams whose log sum is the chunks' (warp 0)
  for (bool first = true;; first = false) {
    if (beam == 0) {
      const bool live = lane < beams && s_score[lane < beams ? lane : 0] > -INFINITY;
      const double sc = live ? (double)s_score[lane] : 0.0;
      const bool done = live && s_done[lane];
      const double base = live && !done ? s_lse[lane] : 0.0;
      if (first) rough = __ballot_sync(0xffffffffu, live && !done);
      int at = 0;
      auto value = [&](unsigned &v) -> double {
        if (!live) return -INFINITY;
        if (done) {
          v = (unsigned)eos;
          return at == 0 ? sc : -INFINITY;
        }
        const unsigned long long k = at < n_out ? s_list[lane][at] : 0;
        if (!k) return -INFINITY;
        v = beam_key_index(k);
        return ((double)beam_key_logit(k) - base) + sc;
      };
      unsigned v = 0;
      double c = value(v), taken = 0.0;  // lane n: what slot n took, and whose
      int from = -1;
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
        if (!(m > -INFINITY)) {
          if (lane == 0) {
            out_scores[o] = -INFINITY;
            parent[o] = n % beams;
            token[o] = -1;
            if (out_finished) out_finished[o] = 0;
          }
        } else {
          if (lane == n) {
            taken = m;
            from = who;
          }
          if (lane == who) {
            out_scores[o] = fmaxf((float)c, -3.402823466e38f);
            parent[o] = who;
            token[o] = (int32_t)v;
            if (out_finished) out_finished[o] = done || (int)v == eos;
            ++at;
            c = value(v);
          }
        }
        __syncwarp();
      }
      // the rough ones of beams a and b, worth ca >= cb, where the two lie too close
      auto close = [&](int a, double ca, int b, double cb) {
        const unsigned pair = rough & (1u << a | 1u << b);
        return a != b && pair && ca - cb <= (pair & (pair - 1) ? 2.0 * tol : tol) ? pair : 0u;
      };
      unsigned redo = 0;
      if (rough && beams > 1) {  // the same for the warp
        const double before = __shfl_up_sync(0xffffffffu, taken, 1);
        const int whose = __shfl_up_sync(0xffffffffu, from, 1);
        const double least = __shfl_sync(0xffffffffu, taken, n_out - 1);
        const int last = __shfl_sync(0xffffffffu, from, n_out - 1);
        if (lane > 0 && from >= 0) redo = close(whose, before, from, taken);
        if (last >= 0 && c > -INFINITY) redo |= close(last, least, lane, c);
        redo = __reduce_or_sync(0xffffffffu, redo);
      }
      rough &= ~redo;
      if (lane == 0) s_redo = redo;
    }
    __syncthreads();
    const unsigned redo = s_redo;
    if (__builtin_expect(redo == 0, 1)) return;
    for (unsigned r = redo; r; r &= r - 1) {
      const int k = __ffs(r) - 1;
      const double top = (double)s_top[k];
      const double t =
          beam_exact_sum(logits + ((long long)blockIdx.x * beams + k) * ld, V, top, s_part);
      if (threadIdx.x == 0) s_lse[k] = top + log(t);
    }
    __syncthreads();
  }
}

}  // namespace fm
