// fm_token_api.cuh -- host side of the token-loop entry points (included at the
// end of fm_lib.cu: argument checks, workspace carving and launches).

static bool dtype_in(fm_dtype t, fm_dtype a, fm_dtype b, fm_dtype c) {
  return t == a || t == b || t == c;
}

// ------------------------------------------------------------------ add + norm + codes
template <typename TX>
static fm_status launch_add_norm(const void *x, int64_t ldx, const float *residual, int64_t ldr,
                                 int64_t M, int K, const float *w, double eps, bool e4m3, void *q,
                                 float *s, float *sum, int64_t lds, cudaStream_t st) {
  const int threads = 32 * ((K + kNormCols - 1) / kNormCols);
  const bool ahead = K <= kNormAheadK;
  auto kern = ahead ? (e4m3 ? k_add_norm_quant<TX, true, true> : k_add_norm_quant<TX, false, true>)
                    : (e4m3 ? k_add_norm_quant<TX, true, false> : k_add_norm_quant<TX, false, false>);
  // as many CTAs as an SM holds (the kernel that fetches ahead: 640 threads'
  // registers), each with a row ahead, or one per row
  const int64_t grid = ahead ? std::min<int64_t>(M, (int64_t)sm_count() *
                                                        std::min(32, 640 / threads))
                             : M;
  FM_TRY(launch_ex("k_add_norm_quant", kern, (unsigned)grid, threads, 0, st, (const TX *)x,
                   (long long)ldx, residual, (long long)ldr, (long long)M, K, 1.0 / (double)K, w, eps,
                   (uint8_t *)q, s, sum, (long long)lds));
  return launched("k_add_norm_quant");
}

extern "C" fm_status fm_add_norm_quant(const void *x, fm_dtype x_type, int64_t ldx,
                                       const float *residual, int64_t ldr, int64_t M, int64_t K,
                                       const float *norm_w, double eps, fm_dtype q_type, void *q,
                                       float *s, float *sum_out, int64_t lds, fm_stream stream) {
  if (x_type != FM_F32 && x_type != FM_BF16)
    return fail(FM_ERR_INVALID_ARG, "%s: x must be fp32 or bf16", __func__);
  if (q_type != FM_I8 && q_type != FM_E4M3)
    return fail(FM_ERR_INVALID_ARG, "%s: q must be int8 or e4m3", __func__);
  if (!(eps >= 1e-30 && eps <= 1e30))  // the kernel's 2^e = 2^exponent(rstd) stays an fp32 number
    return fail(FM_ERR_INVALID_ARG, "%s: eps must lie in [1e-30, 1e30]", __func__);
  if (M < 0 || M > 0x7FFFFFFF || K <= 0 || K % 16 || K > kNormMaxK)
    return fail(FM_ERR_SHAPE, "%s: need 0 <= M < 2^31 and K a multiple of 16, <= %d", __func__,
                kNormMaxK);
  if (ldx < K || ldx % 4 || (residual && (ldr < K || ldr % 4)) || (sum_out && (lds < K || lds % 4)))
    return fail(FM_ERR_SHAPE, "%s: row strides must be multiples of 4, at least K", __func__);
  if (M == 0) return FM_OK;
  // a sum written over an input must fall on the element that it is the sum of
  if (sum_out && ((sum_out == x && (x_type != FM_F32 || (M > 1 && lds != ldx))) ||
                  (sum_out == residual && M > 1 && lds != ldr)))
    return fail(FM_ERR_INVALID_ARG, "%s: sum_out replaces an input of another type or row stride",
                __func__);
  NEED(x);
  OPT(residual);
  NEED(norm_w);
  NEED(q);
  NEED(s);
  OPT(sum_out);
  auto go = x_type == FM_F32 ? launch_add_norm<float> : launch_add_norm<__nv_bfloat16>;
  return go(x, ldx, residual, ldr, M, (int)K, norm_w, eps, q_type == FM_E4M3, q, s, sum_out, lds,
            (cudaStream_t)stream);
}

// ------------------------------------------------------------------ block-scaled e4m3 product
extern "C" fm_status fm_prepare_linear_fp8(const float *W, int64_t N, int64_t K, void *Wq,
                                           float *s_w, fm_stream stream) {
  if (N <= 0 || K <= 0 || K % 16 || K > 0x7FFFFFFF || (N + 127) / 128 > 65535)
    return fail(FM_ERR_SHAPE, "%s: need N in [1, 65535 * 128] and K a positive multiple of 16",
                __func__);
  NEED(W);
  NEED(Wq);
  NEED(s_w);
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)((N + 127) / 128));
  FM_TRY(launch_ex("k_prepare_linear_fp8", k_prepare_linear_fp8, grid, 256, 0, (cudaStream_t)stream,
                   W, (long long)N, (int)K, (uint8_t *)Wq, s_w));
  return launched("k_prepare_linear_fp8");
}

// Output map of the large kernel's TMA stores: N columns, rows ldy elements
// apart, boxes of 32 rows x 128 bytes in the staging buffers' 128-byte swizzle.
static fm_status make_tmap_rows(CUtensorMap *tm, void *Y, bool f32, long long N, long long M,
                                long long ldy) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FM_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled entry point unavailable");
  const cuuint32_t es = f32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  cuuint64_t strides[1] = {(cuuint64_t)ldy * es};
  cuuint32_t box[2] = {128 / es, 32};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, Y,
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FM_ERR_CUDA, "cuTensorMapEncodeTiled (output) failed (%d)", (int)r);
  return FM_OK;
}

template <int BN, int STAGES, typename TY>
static fm_status launch_fp8_large(const void *A, const void *W, long long K, Fp8Args a,
                                  cudaStream_t st) {
  using Sm = Fp8Smem<BN, STAGES>;
  static_assert(Sm::kBytes <= 227 * 1024, "shared memory per CTA");
  CUtensorMap ta, tb, ty;
  FM_TRY(make_tmap(&ta, (const int8_t *)A, a.M, K, kGemmBM));
  FM_TRY(make_tmap(&tb, (const int8_t *)W, a.N, K, BN));
  ty = ta;
  // the TMA unit clips rows in units of 16 bytes: a row that ends inside one
  // would have what lies behind it overwritten
  a.tma_store = a.ldy * (long long)sizeof(TY) % 16 == 0 && a.N * (long long)sizeof(TY) % 16 == 0;
  if (a.tma_store) FM_TRY(make_tmap_rows(&ty, a.Y, sizeof(TY) == 4, a.N, a.M, a.ldy));
  const long long mt = (a.M + kGemmBM - 1) / kGemmBM, nt = (a.N + BN - 1) / BN;
  if (mt * nt > 0x7FFFFFFF) return fail(FM_ERR_SHAPE, "fm_fp8_gemm: too many output tiles");
  a.m_tiles = (int)mt;
  a.n_tiles = (int)nt;
  auto kern = k_fp8_gemm_tc<BN, STAGES, TY>;
  // the warpgroups' register shares must fit what the block is launched with
  // (a share that does not would wait for ever)
  static std::atomic<int> known{0};  // of this variant; a query that failed is made again
  int regs = known.load(std::memory_order_relaxed);
  if (!regs) {
    cudaFuncAttributes fa;
    FM_CHECK_CUDA(cudaFuncGetAttributes(&fa, kern));
    known.store(regs = fa.numRegs, std::memory_order_relaxed);
  }
  if (regs * kFp8Threads < 128 * kFp8RegsLoad + (kFp8Threads - 128) * kFp8RegsAcc)
    return fail(FM_ERR_UNSUPPORTED, "k_fp8_gemm_tc: built with %d registers per thread", regs);
  FM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes));
  const unsigned grid = (unsigned)(mt * nt < sm_count() ? mt * nt : sm_count());
  FM_TRY(launch_ex("k_fp8_gemm_tc", kern, grid, kFp8Threads, Sm::kBytes, st, ta, tb, ty, a));
  return launched("k_fp8_gemm_tc");
}

template <int MP, int STAGES, typename TY>
static fm_status launch_fp8_small(const void *A, const void *W, long long K, Fp8Args a,
                                  cudaStream_t st) {
  using Sm = Fp8SmallSmem<MP, STAGES>;
  static_assert(Sm::kBytes <= 227 * 1024, "shared memory per CTA");
  CUtensorMap ta, tw;
  FM_TRY(make_tmap(&ta, (const int8_t *)A, a.M, K, MP));
  FM_TRY(make_tmap(&tw, (const int8_t *)W, a.N, K, kGemmBM));
  a.n_tiles = (int)((a.N + kGemmBM - 1) / kGemmBM);
  auto kern = k_fp8_gemm_small<MP, STAGES, TY>;
  FM_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes));
  const unsigned grid = (unsigned)(a.n_tiles < sm_count() ? a.n_tiles : sm_count());
  FM_TRY(launch_ex("k_fp8_gemm_small", kern, grid, 64 + 32 * Sm::kEpi, Sm::kBytes, st, tw, ta, a));
  return launched("k_fp8_gemm_small");
}

template <typename TY>
static fm_status launch_fp8(const void *A, const void *W, long long K, const Fp8Args &a,
                            cudaStream_t st) {
  if (a.M <= 16) return launch_fp8_small<16, 11, TY>(A, W, K, a, st);
  if (a.M <= 32) return launch_fp8_small<32, 10, TY>(A, W, K, a, st);
  if (a.M <= 64) return launch_fp8_small<64, 8, TY>(A, W, K, a, st);
  if (a.M <= 128) return launch_fp8_small<128, 5, TY>(A, W, K, a, st);
  // 256 columns per tile halve the traffic of A; narrower tiles where those
  // would leave SMs idle
  if ((a.M + kGemmBM - 1) / kGemmBM * ((a.N + 255) / 256) >= sm_count())
    return launch_fp8_large<256, 4, TY>(A, W, K, a, st);
  return launch_fp8_large<128, 6, TY>(A, W, K, a, st);
}

extern "C" fm_status fm_fp8_gemm(const void *A, const float *s_a, int64_t M, const void *W,
                                 const float *s_w, int64_t N, int64_t K, void *Y, fm_dtype y_type,
                                 int64_t ldy, fm_stream stream) {
  if (y_type != FM_F32 && y_type != FM_BF16)
    return fail(FM_ERR_INVALID_ARG, "%s: Y must be fp32 or bf16", __func__);
  if (M < 0 || N < 0 || M > 0x7FFFFF00 || N > 0x7FFFFF00 || K <= 0 || K % 16 || K > 0x7FFFFF00)
    return fail(FM_ERR_SHAPE, "%s: need M, N, K <= 2^31 - 256, M, N >= 0 and K a positive multiple of 16",
                __func__);
  if (ldy < N || ldy > (int64_t)1 << 36)
    return fail(FM_ERR_SHAPE, "%s: ldy is less than N or above 2^36", __func__);
  if (M == 0 || N == 0) return FM_OK;
  NEED(A);
  NEED(s_a);
  NEED(W);
  NEED(s_w);
  NEED(Y);
  Fp8Args a = {};
  a.s_a = s_a;
  a.s_w = s_w;
  a.M = M;
  a.N = N;
  a.ldy = ldy;
  a.Y = Y;
  a.nkb = (int)((K + kGemmBK - 1) / kGemmBK);
  return y_type == FM_F32 ? launch_fp8<float>(A, W, K, a, (cudaStream_t)stream)
                          : launch_fp8<__nv_bfloat16>(A, W, K, a, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ beam selection
// Logits per thread of a chunk: 16, or 8 for the latency of selections that
// would give an SM less than two chunks of 16.
static int64_t beam_chunks_of(int elems, int64_t V) {
  return (V + kBeamThreads * elems - 1) / (kBeamThreads * elems);
}
static int beam_elems(int64_t rows, int64_t V) {
  return rows * beam_chunks_of(16, V) >= 2 * sm_count() ? 16 : 8;
}
// The most chunks that a selection of up to `rows` rows and V logits has: more rows
// can have fewer of them, where they change from 8 to 16 logits per thread.  With 8
// there are at most twice as many as there would be of 16, which is less than 2
// per SM.
static int64_t beam_most_chunks(int64_t rows, int64_t V) {
  return std::max(rows * beam_chunks_of(16, V),
                  std::min<int64_t>(rows * beam_chunks_of(8, V), 2 * (2 * sm_count() - 1)));
}
static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

static bool beam_sizes_ok(int B, int beams, int64_t V, int n_out) {
  return B >= 0 && beams >= 1 && beams <= kBeamMax && n_out >= 1 && n_out <= kBeamMax && V >= 1 &&
         V <= 0x7FFFFFFF && (int64_t)B * beams <= 0x7FFFFFFF &&
         beam_most_chunks((int64_t)B * beams, V) <= 0x7FFFFFFF;
}

extern "C" size_t fm_beam_workspace_bytes(int B, int beams, int64_t V, int n_out) {
  if (!beam_sizes_ok(B, beams, V, n_out)) return 0;
  const size_t chunks = (size_t)beam_most_chunks((int64_t)B * beams, V);
  return round256(chunks * n_out * 8) + round256(chunks * 8) + round256(chunks * 4);
}

extern "C" fm_status fm_beam_select(const void *logits, fm_dtype type, int64_t ld, int B, int beams,
                                    int64_t V, const float *scores, const uint8_t *finished,
                                    int eos, int n_out, float *out_scores, int32_t *parent,
                                    int32_t *token, uint8_t *out_finished, void *ws,
                                    size_t ws_bytes, fm_stream stream) {
  if (type != FM_F32 && type != FM_BF16)
    return fail(FM_ERR_INVALID_ARG, "%s: logits must be fp32 or bf16", __func__);
  if (!beam_sizes_ok(B, beams, V, n_out))
    return fail(FM_ERR_SHAPE, "%s: need beams and n_out in [1, %d], V in [1, 2^31) and B * beams < 2^31",
                __func__, kBeamMax);
  if (ld < V) return fail(FM_ERR_SHAPE, "%s: ld is less than V", __func__);
  if (eos < -1 || eos >= V || (finished && eos < 0))
    return fail(FM_ERR_INVALID_ARG, "%s: eos must be a token (or -1 where no beam is finished)",
                __func__);
  if (B == 0) return FM_OK;
  NEED(logits);
  NEED(scores);
  OPT(finished);
  NEED(out_scores);
  NEED(parent);
  NEED(token);
  OPT(out_finished);
  if ((out_scores == scores || (finished && out_finished == finished)) && n_out != beams)
    return fail(FM_ERR_INVALID_ARG, "%s: outputs may replace the inputs only where n_out = beams",
                __func__);
  const size_t need = fm_beam_workspace_bytes(B, beams, V, n_out);
  if (!ws || ws_bytes < need)
    return fail(FM_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", __func__, need);
  NEED(ws);
  const int64_t rows = (int64_t)B * beams;
  const int E = beam_elems(rows, V), S = (int)beam_chunks_of(E, V);
  const size_t chunks = (size_t)rows * S;
  unsigned long long *keys = (unsigned long long *)ws;
  double *sums = (double *)((char *)ws + round256(chunks * n_out * 8));
  float *tops = (float *)((char *)sums + round256(chunks * 8));
  cudaStream_t st = (cudaStream_t)stream;
  auto go = [&](auto t) -> fm_status {
    using T = decltype(t);
    auto kern = E == 16 ? k_beam_chunks<T, 16> : k_beam_chunks<T, 8>;
    return launch_ex("k_beam_chunks", kern, (unsigned)chunks, kBeamThreads, 0, st,
                     (const T *)logits, (long long)ld, (unsigned)V, S, n_out, scores, finished, keys,
                     tops, sums);
  };
  FM_TRY(type == FM_F32 ? go(float()) : go(__nv_bfloat16()));
  FM_TRY(launched("k_beam_chunks"));
  // How far a log sum of k_beam_chunks may be off.  With d = top - l, the argument
  // of an exponential is d log2(e) with three relative errors (the difference, the
  // constant, the product: 2^-24 + 2^-26 + 2^-24), the exponential has 2^-22, and
  // up to 16 of them are added in fp32 (15 roundings), the rest in 64 bits.  The
  // mean of d under the softmax is its entropy less the log sum, so at most ln V.
  const double tol = (2.25 * std::log((double)V) + 20.0) * 0x1p-24;
  // an SM holds 32 warps of the merge: as many each as lets its entries run side by
  // side (one beam has no other to be close to)
  const int64_t per_sm = ((int64_t)B + sm_count() - 1) / sm_count();
  const int warps = beams == 1 ? 1 : std::max(beams, (int)(32 / per_sm));
  auto merge = [&](auto t) -> fm_status {
    using T = decltype(t);
    return launch_ex("k_beam_merge", k_beam_merge<T>, (unsigned)B, 32 * warps, 0, st, (const unsigned long long *)keys,
                     (const float *)tops, (const double *)sums, S, beams, (const T *)logits,
                     (long long)ld, (unsigned)V, tol, scores, finished, eos, n_out, out_scores, parent,
                     token, out_finished);
  };
  FM_TRY(type == FM_F32 ? merge(float()) : merge(__nv_bfloat16()));
  return launched("k_beam_merge");
}

// ------------------------------------------------------------------ state reordering
template <typename U>
static fm_status launch_reorder(const ReorderArgs &a, unsigned blocks, int B, cudaStream_t st) {
  auto kern = a.dst_beams <= 4    ? k_reorder_rows<U, 4>
              : a.dst_beams <= 8  ? k_reorder_rows<U, 8>
              : a.dst_beams <= 16 ? k_reorder_rows<U, 16>
                                  : k_reorder_rows<U, 32>;
  FM_TRY(launch_ex("k_reorder_rows", kern, dim3(blocks, (unsigned)B), kReorderThreads, 0, st, a));
  return launched("k_reorder_rows");
}

// Bytes that a thread moves of a row at once: 16 where the rows are multiples of
// 16 (every state of the library), else 4 or 1.
static int reorder_unit(int64_t row_bytes) {
  return row_bytes % 16 == 0 ? 16 : row_bytes % 4 == 0 ? 4 : 1;
}

extern "C" fm_status fm_reorder_rows(const void *const *src, void *const *dst,
                                     const int64_t *row_bytes, int n_bufs, int B, int src_beams,
                                     int dst_beams, const int32_t *parent, fm_stream stream) {
  if (n_bufs < 0 || (n_bufs > 0 && (!src || !dst || !row_bytes)))
    return fail(FM_ERR_INVALID_ARG, "%s: src, dst or row_bytes is null", __func__);
  if (B < 0 || B > 65535 || src_beams < 1 || src_beams > kReorderBeams || dst_beams < 1 ||
      dst_beams > kReorderBeams)
    return fail(FM_ERR_SHAPE, "%s: need B <= 65535 and beams in [1, %d]", __func__, kReorderBeams);
  if (B == 0 || n_bufs == 0) return FM_OK;
  NEED(parent);
  for (int i = 0; i < n_bufs; ++i) {
    // a launch counts a row's units in 32 bits
    if (row_bytes[i] < 0 || row_bytes[i] / reorder_unit(row_bytes[i]) > 0xFFFFFFFFll)
      return fail(FM_ERR_SHAPE, "%s: row_bytes[%d] is negative or too long", __func__, i);
    if (row_bytes[i] && (!src[i] || !dst[i]))
      return fail(FM_ERR_INVALID_ARG, "%s: buffer %d is null", __func__, i);
    if (!aligned16(src[i]) || !aligned16(dst[i]))
      return fail(FM_ERR_ALIGNMENT, "%s: buffer %d is not 16-byte aligned", __func__, i);
    const uintptr_t s0 = (uintptr_t)src[i], d0 = (uintptr_t)dst[i];
    if (s0 == d0) {
      if (src_beams != dst_beams)
        return fail(FM_ERR_INVALID_ARG, "%s: buffer %d in place needs src_beams = dst_beams",
                    __func__, i);
    } else if (s0 < d0 + (uintptr_t)(row_bytes[i] * B * dst_beams) &&
               d0 < s0 + (uintptr_t)(row_bytes[i] * B * src_beams)) {
      return fail(FM_ERR_INVALID_ARG, "%s: src and dst of buffer %d overlap", __func__, i);
    }
    // the parents are read by every block, before and after others have written
    const uintptr_t p0 = (uintptr_t)parent;
    if (row_bytes[i] && d0 < p0 + (uintptr_t)B * dst_beams * 4 &&
        p0 < d0 + (uintptr_t)(row_bytes[i] * B * dst_beams))
      return fail(FM_ERR_INVALID_ARG, "%s: buffer %d overlaps the parents", __func__, i);
  }
  // one launch per 128 buffers of the same unit
  for (int unit : {16, 4, 1}) {
    ReorderArgs a = {};
    a.src_beams = src_beams;
    a.dst_beams = dst_beams;
    a.parent = parent;
    int64_t blocks = 0;
    auto flush = [&]() -> fm_status {
      if (a.n == 0) return FM_OK;
      a.first[a.n] = (unsigned)blocks;
      fm_status st = unit == 16  ? launch_reorder<uint4>(a, (unsigned)blocks, B, (cudaStream_t)stream)
                     : unit == 4 ? launch_reorder<uint32_t>(a, (unsigned)blocks, B, (cudaStream_t)stream)
                                 : launch_reorder<uint8_t>(a, (unsigned)blocks, B, (cudaStream_t)stream);
      a.n = 0;
      blocks = 0;
      return st;
    };
    for (int i = 0; i < n_bufs; ++i) {
      const int64_t rb = row_bytes[i];
      if (rb == 0 || unit != reorder_unit(rb)) continue;
      const int64_t units = rb / unit, nb = (units + kReorderThreads - 1) / kReorderThreads;
      if (a.n == kReorderBufs || blocks + nb > 0x7FFFFFFFll) FM_TRY(flush());
      a.src[a.n] = src[i];
      a.dst[a.n] = dst[i];
      a.first[a.n] = (unsigned)blocks;
      a.units[a.n] = (unsigned)units;
      ++a.n;
      blocks += nb;
    }
    FM_TRY(flush());
  }
  return FM_OK;
}

// ------------------------------------------------------------------ embedding rows
extern "C" fm_status fm_embed_rows(const int32_t *ids, int64_t M, const void *table, fm_dtype type,
                                   const float *table_s, int64_t V, int64_t K, float scale,
                                   float *x, int64_t ldx, fm_stream stream) {
  if (!dtype_in(type, FM_F32, FM_BF16, FM_E4M3))
    return fail(FM_ERR_INVALID_ARG, "%s: the table must be fp32, bf16 or e4m3", __func__);
  if (M < 0 || V < 1 || V > 0x7FFFFFFF || K <= 0 || K % 16 || K > 0x7FFFFF00)
    return fail(FM_ERR_SHAPE, "%s: need V in [1, 2^31) and K a positive multiple of 16", __func__);
  const int64_t pieces = (K + kEmbedCols - 1) / kEmbedCols;
  if (M > 0x7FFFFFFF / pieces)
    return fail(FM_ERR_SHAPE, "%s: M=%lld rows of %lld columns are too many", __func__, (long long)M,
                (long long)K);
  if (ldx < K || ldx % 4)
    return fail(FM_ERR_SHAPE, "%s: ldx must be a multiple of 4, at least K", __func__);
  if (M == 0) return FM_OK;
  NEED(ids);
  NEED(table);
  if (type == FM_E4M3) NEED(table_s);
  NEED(x);
  auto kern = type == FM_F32 ? k_embed_rows<0> : type == FM_BF16 ? k_embed_rows<1> : k_embed_rows<2>;
  FM_TRY(launch_ex("k_embed_rows", kern, (unsigned)((M * pieces + 3) / 4), 128, 0,
                   (cudaStream_t)stream, ids, (long long)M, table, table_s, (long long)V, (int)K,
                   (int)pieces, scale, x, (long long)ldx));
  return launched("k_embed_rows");
}
