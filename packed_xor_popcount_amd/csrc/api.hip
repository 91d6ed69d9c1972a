// api.hip -- the C-ABI of libbnn.so: host-side validation, kernel choice and
// status codes.  Every check runs before anything is enqueued, so an invalid
// call writes nothing and launches nothing.  No allocation, no
// synchronization, no state.
#include "../../include/bnn.h"
#include "bnn_internal.h"
#include "f8.h"
#include "operators.h"

#include <float.h>

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;  // M, N, K, rows and ld limits
constexpr int64_t kGemvMaxM = 8;               // AUTO picks the GEMV kernel up to here
constexpr int64_t kMaxGroups = int64_t(1) << 20;  // experts of a grouped product

bool misaligned(const void *p, uintptr_t a) { return ((uintptr_t)p) % a != 0; }

bnn_status launch_status(hipError_t e) { return e == hipSuccess ? BNN_OK : BNN_E_LAUNCH; }

// Shared checks of the packed products; `epilogue` may be the internal
// threshold repack, whose operands `ep.thr` / `ep.flip` are checked here too.
bnn_status check_gemm(const uint64_t *xp, const uint64_t *wp, const bnn::EpiParams &ep,
                      const void *y, int64_t M, int64_t N, int64_t K, int epilogue, int algo) {
  if (epilogue < BNN_EPI_I32 || epilogue > bnn::kEpiRepackThr) return BNN_E_ARG;
  if (algo < BNN_ALGO_AUTO || algo > BNN_ALGO_MFMA) return BNN_E_ARG;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return BNN_E_SHAPE;
  if (algo == BNN_ALGO_MFMA && K > bnn::kMfmaMaxK) return BNN_E_SHAPE;
  const int64_t kw = bnn_words(K);
  if ((M * kw > 0 && !xp) || (N * kw > 0 && !wp) || (M * N > 0 && !y)) return BNN_E_NULL;
  if (epilogue == BNN_EPI_SCALED && M * N > 0 && !ep.alpha) return BNN_E_NULL;
  if (epilogue == bnn::kEpiRepackThr && M * N > 0 && !ep.thr) return BNN_E_NULL;
  if (misaligned(xp, 8) || misaligned(wp, 8)) return BNN_E_ALIGN;
  if (misaligned(y, bnn::is_repack(epilogue) ? 8 : 4)) return BNN_E_ALIGN;
  if (epilogue == BNN_EPI_SCALED && misaligned(ep.alpha, 4)) return BNN_E_ALIGN;
  if (epilogue == bnn::kEpiRepackThr && (misaligned(ep.thr, 4) || misaligned(ep.flip, 8)))
    return BNN_E_ALIGN;
  return BNN_OK;
}

// Kernel choice and launch of a validated product.
bnn_status run_gemm(const uint64_t *xp, const uint64_t *wp, const bnn::EpiParams &ep, void *y,
                    int64_t M, int64_t N, int64_t K, int epilogue, int algo, hipStream_t s) {
  if (M == 0 || N == 0) return BNN_OK;
  if (algo == BNN_ALGO_AUTO) {
    if (K == 0)
      algo = BNN_ALGO_TILED;  // no K loop: the smallest kernel writes the constant result
    else if (M <= kGemvMaxM)
      algo = BNN_ALGO_GEMV;  // weight-streaming: HBM-bound
    else if (K <= bnn::kMfmaMaxK)
      algo = BNN_ALGO_MFMA;  // matrix cores: ~8x the VALU popcount rate
    else
      algo = BNN_ALGO_TILED;
  }
  if (algo == BNN_ALGO_GEMV)
    return launch_status(bnn::launch_gemv(xp, wp, ep, y, M, N, K, epilogue, s));
  if (algo == BNN_ALGO_MFMA)
    return launch_status(bnn::launch_gemm_mfma(xp, wp, ep, y, M, N, K, epilogue, s));
  return launch_status(bnn::launch_gemm_tiled(xp, wp, ep, y, M, N, K, epilogue, s));
}

// Checks and launch of both 8-bit products.
bnn_status run_gemm_f8(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       void *y, int dtype, bool fast, int64_t M, int64_t N, int64_t K,
                       void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxDim || N >= kMaxDim || K > bnn::kF8MaxK)
    return BNN_E_SHAPE;
  if ((M * K > 0 && (!xq || !xs)) || (N * K > 0 && (!wq || !ws)) || (M * N > 0 && !y))
    return BNN_E_NULL;
  if (misaligned(xq, 16) || misaligned(wq, 16) || misaligned(xs, 4) || misaligned(ws, 4) ||
      misaligned(y, dtype == BNN_FP32 ? 4 : 2))
    return BNN_E_ALIGN;
  if (M == 0 || N == 0) return BNN_OK;
  return launch_status(bnn::launch_gemm_f8(xq, xs, wq, ws, y, dtype, fast, M, N, K,
                                           static_cast<hipStream_t>(stream)));
}

// Sizes of the router, of the sum behind the experts and of the adapters.
bool route_sizes_ok(int64_t T, int64_t E, int64_t k) {
  return T >= 0 && T < kMaxDim && E >= 1 && E <= bnn::kRouteMaxExperts && k >= 1 && k <= E &&
         k <= bnn::kRouteMaxK && T * k < kMaxDim;
}
bool combine_sizes_ok(int64_t R, int64_t T, int64_t N, int64_t k) {
  return R >= 0 && R < kMaxDim && T >= 0 && T < kMaxDim && N >= 0 && N < kMaxDim && k >= 1 &&
         k < kMaxDim && T * k < kMaxDim;
}
bool adapter_sizes_ok(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t L) {
  return T >= 0 && T < bnn::kAdapterMaxRows && K >= 0 && K < kMaxDim && N >= 0 && N < kMaxDim &&
         rank >= 1 && rank <= bnn::kAdapterMaxRank && L >= 0 && L < kMaxGroups;
}

}  // namespace

extern "C" {

int64_t bnn_words(int64_t k) { return k <= 0 ? 0 : (k + 63) / 64; }

const char *bnn_status_str(int status) {
  switch (status) {
    case BNN_OK: return "ok";
    case BNN_E_NULL: return "null pointer for a non-empty buffer";
    case BNN_E_SHAPE: return "invalid shape (negative, too large, or ld < k)";
    case BNN_E_DTYPE: return "unknown element type";
    case BNN_E_ALIGN: return "pointer not aligned to its element size";
    case BNN_E_LAUNCH: return "kernel launch failed";
    case BNN_E_ARG: return "unknown epilogue or algorithm selector";
    default: return "unknown status";
  }
}

const char *bnn_version(void) { return "bnn-mi355x 0.1 (gfx950)"; }

bnn_status bnn_pack_signs(const void *src, int dtype, int64_t rows, int64_t k, int64_t ld_src,
                          uint64_t *dst, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (rows < 0 || k < 0 || ld_src < k || rows >= kMaxDim || ld_src >= kMaxDim) return BNN_E_SHAPE;
  if (rows * k > 0 && !src) return BNN_E_NULL;
  if (rows * bnn_words(k) > 0 && !dst) return BNN_E_NULL;
  if (misaligned(src, dtype == BNN_FP32 ? 4 : 2) || misaligned(dst, 8)) return BNN_E_ALIGN;
  if (rows == 0 || k == 0) return BNN_OK;
  return launch_status(
      bnn::launch_pack(src, dtype, rows, k, ld_src, dst, static_cast<hipStream_t>(stream)));
}

bnn_status bnn_gemm_ex(const uint64_t *xp, const uint64_t *wp, const float *alpha, void *y,
                       int64_t M, int64_t N, int64_t K, int epilogue, int algo, void *stream) {
  if (epilogue < BNN_EPI_I32 || epilogue > BNN_EPI_REPACK) return BNN_E_ARG;
  const bnn::EpiParams ep{alpha, nullptr, nullptr};
  const bnn_status st = check_gemm(xp, wp, ep, y, M, N, K, epilogue, algo);
  if (st != BNN_OK) return st;
  return run_gemm(xp, wp, ep, y, M, N, K, epilogue, algo, static_cast<hipStream_t>(stream));
}

bnn_status bnn_gemm_sign_repack_thr(const uint64_t *xp, const uint64_t *wp, const int32_t *thr,
                                    const uint64_t *flip, uint64_t *yp, int64_t M, int64_t N,
                                    int64_t K, int algo, void *stream) {
  const bnn::EpiParams ep{nullptr, thr, flip};
  const bnn_status st = check_gemm(xp, wp, ep, yp, M, N, K, bnn::kEpiRepackThr, algo);
  if (st != BNN_OK) return st;
  return run_gemm(xp, wp, ep, yp, M, N, K, bnn::kEpiRepackThr, algo,
                  static_cast<hipStream_t>(stream));
}

bnn_status bnn_gemv_act(const void *x, int dtype, int64_t ldx, const uint64_t *wp,
                        const float *alpha, void *y, int64_t M, int64_t N, int64_t K, int epilogue,
                        void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (epilogue < BNN_EPI_I32 || epilogue > BNN_EPI_REPACK) return BNN_E_ARG;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim || ldx < K ||
      ldx >= kMaxDim)
    return BNN_E_SHAPE;
  const int64_t kw = bnn_words(K);
  if ((M * K > 0 && !x) || (N * kw > 0 && !wp) || (M * N > 0 && !y)) return BNN_E_NULL;
  if (epilogue == BNN_EPI_SCALED && M * N > 0 && !alpha) return BNN_E_NULL;
  if (misaligned(x, dtype == BNN_FP32 ? 4 : 2) || misaligned(wp, 8)) return BNN_E_ALIGN;
  if (misaligned(y, epilogue == BNN_EPI_REPACK ? 8 : 4)) return BNN_E_ALIGN;
  if (epilogue == BNN_EPI_SCALED && misaligned(alpha, 4)) return BNN_E_ALIGN;
  if (M == 0 || N == 0) return BNN_OK;
  const bnn::EpiParams ep{alpha, nullptr, nullptr};
  return launch_status(bnn::launch_gemv_act(x, dtype, ldx, wp, ep, y, M, N, K, epilogue,
                                            static_cast<hipStream_t>(stream)));
}

bnn_status bnn_gemm_signw_bf16(const void *x, int64_t ldx, const uint64_t *wp, const float *alpha,
                               float *y, int64_t M, int64_t N, int64_t K, int algo, void *stream) {
  if (algo != BNN_ALGO_AUTO && algo != BNN_ALGO_GEMV && algo != BNN_ALGO_MFMA) return BNN_E_ARG;
  if (M < 0 || N < 0 || K < 0 || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim || ldx < K ||
      ldx >= kMaxDim)
    return BNN_E_SHAPE;
  const int64_t kw = bnn_words(K);
  if ((M * K > 0 && !x) || (N * kw > 0 && !wp) || (M * N > 0 && !y)) return BNN_E_NULL;
  if (misaligned(x, 2) || misaligned(wp, 8) || misaligned(y, 4) || misaligned(alpha, 4))
    return BNN_E_ALIGN;
  if (M == 0 || N == 0) return BNN_OK;
  const bool gemv_ok = bnn::signw_gemv_fits(M, K);
  if (algo == BNN_ALGO_GEMV && !gemv_ok) return BNN_E_SHAPE;
  if (algo == BNN_ALGO_AUTO) algo = gemv_ok ? BNN_ALGO_GEMV : BNN_ALGO_MFMA;
  const uint16_t *xb = static_cast<const uint16_t *>(x);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (algo == BNN_ALGO_GEMV)
    return launch_status(bnn::launch_signw_gemv(xb, ldx, wp, alpha, y, M, N, K, s));
  return launch_status(bnn::launch_signw_mfma(xb, ldx, wp, alpha, y, M, N, K, s));
}

bnn_status bnn_chain3(const void *x, int dtype, int64_t ldx, const uint64_t *w1,
                      const int32_t *thr1, const uint64_t *flip1, const uint64_t *w2,
                      const int32_t *thr2, const uint64_t *flip2, const uint64_t *w3,
                      const float *alpha3, float *y, int64_t M, int64_t K0, int64_t N1, int64_t N2,
                      int64_t N3, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (M < 0 || M >= kMaxDim || ldx < K0 || ldx >= kMaxDim ||
      !bnn::chain3_dims_ok(K0, N1, N2, N3))
    return BNN_E_SHAPE;
  if ((M > 0 && (!x || !y)) || !w1 || !w2 || !w3) return BNN_E_NULL;
  if (misaligned(x, dtype == BNN_FP32 ? 4 : 2) || misaligned(w1, 8) || misaligned(w2, 8) ||
      misaligned(w3, 8) || misaligned(y, 4) || misaligned(alpha3, 4) || misaligned(thr1, 4) ||
      misaligned(thr2, 4) || misaligned(flip1, 8) || misaligned(flip2, 8))
    return BNN_E_ALIGN;
  if (M == 0) return BNN_OK;
  const bnn::Chain3Repack rp{thr1, flip1, thr2, flip2};
  return launch_status(bnn::launch_chain3(x, dtype, ldx, w1, w2, w3, alpha3, y, M, K0, N1, N2, N3,
                                          rp, static_cast<hipStream_t>(stream)));
}

bnn_status bnn_layernorm_fwd(const void *x, int dtype, int64_t ldx, const float *gamma,
                             const float *beta, void *y, int64_t ldy, float *mean, float *rstd,
                             int64_t M, int64_t N, float eps, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (M < 0 || N < 0 || M >= kMaxDim || N >= kMaxDim || ldx < N || ldy < N || ldx >= kMaxDim ||
      ldy >= kMaxDim || (N == 0 && M > 0))
    return BNN_E_SHAPE;
  if (!(eps >= 0.0f) || eps > FLT_MAX) return BNN_E_ARG;
  if (M > 0 && (!x || !y)) return BNN_E_NULL;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(x, es) || misaligned(y, es) || misaligned(gamma, 4) || misaligned(beta, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return BNN_E_ALIGN;
  if (M == 0) return BNN_OK;
  return launch_status(bnn::launch_layernorm_fwd(x, dtype, ldx, gamma, beta, y, ldy, mean, rstd, M,
                                                 N, eps, static_cast<hipStream_t>(stream)));
}

int64_t bnn_layernorm_bwd_workspace(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0 || M >= kMaxDim || N >= kMaxDim) return 0;
  return bnn::layernorm_bwd_partials(M, N) * 2 * N * (int64_t)sizeof(float);
}

bnn_status bnn_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx, int dtype,
                             const float *gamma, const float *mean, const float *rstd, void *dx,
                             int64_t lddx, float *dgamma, float *dbeta, void *workspace,
                             int64_t ws_bytes, int64_t M, int64_t N, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (M < 0 || N < 0 || M >= kMaxDim || N >= kMaxDim || lddy < N || ldx < N || lddx < N ||
      lddy >= kMaxDim || ldx >= kMaxDim || lddx >= kMaxDim || (N == 0 && M > 0))
    return BNN_E_SHAPE;
  if (M > 0 && (!dy || !x || !mean || !rstd || !dx)) return BNN_E_NULL;
  if (!dgamma != !dbeta) return BNN_E_NULL;
  const int64_t need = dgamma ? bnn_layernorm_bwd_workspace(M, N) : 0;
  if (need > 0 && !workspace) return BNN_E_NULL;
  if (ws_bytes < need) return BNN_E_SHAPE;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(dy, es) || misaligned(x, es) || misaligned(dx, es) || misaligned(gamma, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dgamma, 4) ||
      misaligned(dbeta, 4) || misaligned(workspace, 16))
    return BNN_E_ALIGN;
  if (N == 0 || (M == 0 && !dgamma)) return BNN_OK;
  return launch_status(bnn::launch_layernorm_bwd(dy, lddy, x, ldx, dtype, gamma, mean, rstd, dx,
                                                 lddx, dgamma, dbeta,
                                                 static_cast<float *>(workspace), M, N,
                                                 static_cast<hipStream_t>(stream)));
}

int64_t bnn_f8_row_bytes(int64_t k) { return k <= 0 ? 0 : bnn::f8_row_bytes(k); }

int64_t bnn_f8_scale_bytes(int64_t k) { return k <= 0 ? 0 : bnn::f8_scale_bytes(k); }

bnn_status bnn_quant_f8(const void *src, int dtype, int64_t rows, int64_t k, int64_t ld_src,
                        int transpose, uint8_t *q, uint8_t *s, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (transpose != 0 && transpose != 1) return BNN_E_ARG;
  if (rows < 0 || k < 0 || ld_src < k || rows >= kMaxDim || k >= kMaxDim || ld_src >= kMaxDim)
    return BNN_E_SHAPE;
  if (rows * k > 0 && (!src || !q || !s)) return BNN_E_NULL;
  if (misaligned(src, dtype == BNN_FP32 ? 4 : 2) || misaligned(q, 16) || misaligned(s, 4))
    return BNN_E_ALIGN;
  if (rows == 0 || k == 0) return BNN_OK;
  return launch_status(bnn::launch_quant_f8(src, dtype, rows, k, ld_src, transpose != 0, q, s,
                                            static_cast<hipStream_t>(stream)));
}

bnn_status bnn_gemm_f8(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                       void *y, int dtype, int64_t M, int64_t N, int64_t K, void *stream) {
  return run_gemm_f8(xq, xs, wq, ws, y, dtype, false, M, N, K, stream);
}

bnn_status bnn_gemm_f8_fast(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                            const uint8_t *ws, void *y, int64_t M, int64_t N, int64_t K,
                            void *stream) {
  return run_gemm_f8(xq, xs, wq, ws, y, BNN_BF16, true, M, N, K, stream);
}

bnn_status bnn_gemm_signw_grouped(const void *x, int64_t ldx, int64_t xrows, const int32_t *rows,
                                  const int32_t *offsets, const uint64_t *wp, const float *alpha,
                                  const float *row_scale, void *y, int dtype, int64_t R, int64_t E,
                                  int64_t N, int64_t K, int algo, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (algo != BNN_ALGO_AUTO && algo != BNN_ALGO_GEMV && algo != BNN_ALGO_MFMA) return BNN_E_ARG;
  if (R < 0 || E < 0 || N < 0 || K < 0 || xrows < 0 || R >= kMaxDim || N >= kMaxDim ||
      K >= kMaxDim || xrows >= kMaxDim || E >= kMaxGroups || ldx < K || ldx >= kMaxDim ||
      (!rows && xrows < R) || (xrows == 0 && R > 0))
    return BNN_E_SHAPE;
  const int64_t kw = bnn_words(K);
  const bool any = R > 0 && E > 0 && N > 0;
  if (any && (!offsets || !y || (K > 0 && !x) || (kw > 0 && !wp))) return BNN_E_NULL;
  if (misaligned(x, 2) || misaligned(rows, 4) || misaligned(offsets, 4) || misaligned(wp, 8) ||
      misaligned(alpha, 4) || misaligned(row_scale, 4) ||
      misaligned(y, dtype == BNN_FP32 ? 4 : 2))
    return BNN_E_ALIGN;
  if (!any) return BNN_OK;
  return launch_status(bnn::launch_signw_grouped(static_cast<const uint16_t *>(x), ldx, xrows, rows,
                                                 offsets, wp, alpha, row_scale, y, dtype, R, E, N,
                                                 K, algo, static_cast<hipStream_t>(stream)));
}

int64_t bnn_route_fwd_workspace(int64_t T, int64_t E, int64_t k) {
  if (T <= 0 || T >= kMaxDim || E <= 0 || E > bnn::kRouteMaxExperts || k <= 0) return 0;
  return bnn::route_fwd_workspace(T, E, k);
}

bnn_status bnn_route_fwd(const void *z, int dtype, int64_t ldz, const uint8_t *valid,
                         int32_t *experts, float *weights, int32_t *place, int32_t *rows,
                         int32_t *offsets, int32_t *counts, float *stats, float *slope,
                         float *loss, void *workspace, int64_t ws_bytes, int64_t T, int64_t E,
                         int64_t k, int normalise, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (normalise != 0 && normalise != 1) return BNN_E_ARG;
  if (!route_sizes_ok(T, E, k) || ldz < E || ldz >= kMaxDim) return BNN_E_SHAPE;
  if (T > 0 && (!z || !experts || !weights || !place || !rows || !stats)) return BNN_E_NULL;
  if (!offsets || !counts || !slope != !loss) return BNN_E_NULL;
  const int64_t need = bnn_route_fwd_workspace(T, E, k);
  if (need > 0 && !workspace) return BNN_E_NULL;
  if (ws_bytes < need) return BNN_E_SHAPE;
  if (misaligned(z, dtype == BNN_FP32 ? 4 : 2) || misaligned(experts, 4) ||
      misaligned(weights, 4) || misaligned(place, 4) || misaligned(rows, 4) ||
      misaligned(offsets, 4) || misaligned(counts, 4) || misaligned(stats, 4) ||
      misaligned(slope, 4) || misaligned(loss, 4) || misaligned(workspace, 16))
    return BNN_E_ALIGN;
  const bnn::RouteOut out = {experts, weights, place, rows, offsets, counts, stats, slope, loss};
  return launch_status(bnn::launch_route_fwd(z, dtype, ldz, valid, out, workspace, T, (int)E,
                                             (int)k, normalise != 0,
                                             static_cast<hipStream_t>(stream)));
}

bnn_status bnn_route_bwd(const void *z, int dtype, int64_t ldz, const int32_t *experts,
                         const float *weights, const float *stats, const float *slope,
                         const float *dweights, const float *dloss, void *dz, int64_t lddz,
                         int64_t T, int64_t E, int64_t k, int normalise, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (normalise != 0 && normalise != 1) return BNN_E_ARG;
  if (!route_sizes_ok(T, E, k) || ldz < E || ldz >= kMaxDim || lddz < E || lddz >= kMaxDim)
    return BNN_E_SHAPE;
  if (T > 0 && (!z || !stats || !dz || (dweights && (!experts || !weights)))) return BNN_E_NULL;
  if (!slope != !dloss) return BNN_E_NULL;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(z, es) || misaligned(dz, es) || misaligned(experts, 4) ||
      misaligned(weights, 4) || misaligned(stats, 4) || misaligned(slope, 4) ||
      misaligned(dweights, 4) || misaligned(dloss, 4))
    return BNN_E_ALIGN;
  if (T == 0) return BNN_OK;
  return launch_status(bnn::launch_route_bwd(z, dtype, ldz, experts, weights, stats, slope,
                                             dweights, dloss, dz, lddz, T, (int)E, (int)k,
                                             normalise != 0, static_cast<hipStream_t>(stream)));
}

bnn_status bnn_combine_fwd(const void *y, int ydtype, int64_t ldy, int64_t R,
                           const int32_t *place, const float *weights, const void *residual,
                           int64_t ldr, void *out, int dtype, int64_t ldo, int64_t T, int64_t N,
                           int64_t k, void *stream) {
  if ((dtype != BNN_FP32 && dtype != BNN_BF16) || (ydtype != BNN_FP32 && ydtype != BNN_BF16))
    return BNN_E_DTYPE;
  if (!combine_sizes_ok(R, T, N, k) || ldy < N || ldy >= kMaxDim || ldo < N || ldo >= kMaxDim ||
      (residual && (ldr < N || ldr >= kMaxDim)) || (residual && residual == out && ldr != ldo))
    return BNN_E_SHAPE;
  if (T > 0 && N > 0 && (!place || !out || (R > 0 && !y))) return BNN_E_NULL;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(y, ydtype == BNN_FP32 ? 4 : 2) || misaligned(out, es) ||
      misaligned(residual, es) || misaligned(place, 4) || misaligned(weights, 4))
    return BNN_E_ALIGN;
  if (T == 0 || N == 0) return BNN_OK;
  return launch_status(bnn::launch_combine_fwd(y, ydtype, ldy, R, place, weights, residual, ldr,
                                               out, dtype, ldo, T, N, (int)k,
                                               static_cast<hipStream_t>(stream)));
}

bnn_status bnn_combine_bwd(const void *dout, int dtype, int64_t lddo, const void *y,
                           const uint8_t *ys, int ydtype, int64_t ldy, int64_t R,
                           const int32_t *place, const float *weights, void *dy, int dydtype,
                           int64_t lddy, float *dweights, int64_t T, int64_t N, int64_t k,
                           void *stream) {
  if ((dtype != BNN_FP32 && dtype != BNN_BF16) || (dydtype != BNN_FP32 && dydtype != BNN_BF16) ||
      (ydtype != BNN_FP32 && ydtype != BNN_BF16 && ydtype != BNN_F8))
    return BNN_E_DTYPE;
  if (!combine_sizes_ok(R, T, N, k) || lddo < N || lddo >= kMaxDim ||
      (dy && (lddy < N || lddy >= kMaxDim)) ||
      (y && ydtype != BNN_F8 && (ldy < N || ldy >= kMaxDim)))
    return BNN_E_SHAPE;
  if (T > 0 && !place) return BNN_E_NULL;
  if (T > 0 && N > 0 && !dout) return BNN_E_NULL;
  if (dweights && R > 0 && N > 0 && (!y || (ydtype == BNN_F8 && !ys))) return BNN_E_NULL;
  if (misaligned(dout, dtype == BNN_FP32 ? 4 : 2) || misaligned(dy, dydtype == BNN_FP32 ? 4 : 2) ||
      misaligned(y, ydtype == BNN_F8 ? 16 : ydtype == BNN_FP32 ? 4 : 2) || misaligned(ys, 4) ||
      misaligned(place, 4) || misaligned(weights, 4) || misaligned(dweights, 4))
    return BNN_E_ALIGN;
  if (T == 0 || (!dy && !dweights) || (N == 0 && !dweights)) return BNN_OK;
  return launch_status(bnn::launch_combine_bwd(dout, dtype, lddo, y, ys, ydtype, ldy, R, place,
                                               weights, dy, dydtype, lddy, dweights, T, N, (int)k,
                                               static_cast<hipStream_t>(stream)));
}

int64_t bnn_adapter_fwd_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t L) {
  if (!adapter_sizes_ok(T, K, N, rank, L) || T == 0) return 0;
  return bnn::adapter_fwd_workspace(T, N, rank, L);
}

bnn_status bnn_adapter_fwd(const void *x, int64_t ldx, const int32_t *ids, const void *a,
                           const void *b, const float *scale, const void *base, int64_t ldb,
                           void *out, int64_t ldo, int dtype, float *u, void *workspace,
                           int64_t ws_bytes, int64_t T, int64_t K, int64_t N, int64_t rank,
                           int64_t L, void *stream) {
  if (dtype != BNN_FP32 && dtype != BNN_BF16) return BNN_E_DTYPE;
  if (!adapter_sizes_ok(T, K, N, rank, L) || ldx < K || ldx >= kMaxDim || ldo < N ||
      ldo >= kMaxDim || (base && (ldb < N || ldb >= kMaxDim)) || (base == out && base && ldb != ldo))
    return BNN_E_SHAPE;
  if (T > 0 && (!ids || !u || (K > 0 && !x) || (N > 0 && !out))) return BNN_E_NULL;
  if (T > 0 && L > 0 && ((K > 0 && !a) || (N > 0 && !b))) return BNN_E_NULL;
  const int64_t need = bnn_adapter_fwd_workspace(T, K, N, rank, L);
  if (need > 0 && !workspace) return BNN_E_NULL;
  if (ws_bytes < need) return BNN_E_SHAPE;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(x, 2) || misaligned(a, 2) || misaligned(b, 2) || misaligned(ids, 4) ||
      misaligned(scale, 4) || misaligned(base, es) || misaligned(out, es) || misaligned(u, 4) ||
      misaligned(workspace, 16))
    return BNN_E_ALIGN;
  if (T == 0) return BNN_OK;
  return launch_status(bnn::launch_adapter_fwd(
      static_cast<const uint16_t *>(x), ldx, ids, static_cast<const uint16_t *>(a),
      static_cast<const uint16_t *>(b), scale, base, ldb, out, ldo, dtype, u, workspace, T, K, N,
      (int)rank, (int)L, static_cast<hipStream_t>(stream)));
}

int64_t bnn_adapter_bwd_workspace(int64_t T, int64_t K, int64_t N, int64_t rank, int64_t L) {
  if (!adapter_sizes_ok(T, K, N, rank, L) || L > bnn::kRouteMaxExperts) return 0;
  return bnn::adapter_bwd_workspace(T, K, N, rank, L);
}

bnn_status bnn_adapter_bwd(const void *dy, int64_t lddy, const void *x, const uint8_t *xs,
                           int xdtype, int64_t ldx, const float *u, const int32_t *ids,
                           const void *a, const void *b, const float *scale, const void *base,
                           int64_t ldb, void *dx, int64_t lddx, int dtype, float *da, float *db,
                           void *workspace, int64_t ws_bytes, int64_t T, int64_t K, int64_t N,
                           int64_t rank, int64_t L, void *stream) {
  if ((dtype != BNN_FP32 && dtype != BNN_BF16) || (xdtype != BNN_BF16 && xdtype != BNN_F8))
    return BNN_E_DTYPE;
  if (!adapter_sizes_ok(T, K, N, rank, L) || L > bnn::kRouteMaxExperts || lddy < N ||
      lddy >= kMaxDim || ((da || db) && xdtype == BNN_BF16 && (ldx < K || ldx >= kMaxDim)) ||
      (dx && (lddx < K || lddx >= kMaxDim)) || (dx && base && (ldb < K || ldb >= kMaxDim)) ||
      (dx && base == dx && ldb != lddx))
    return BNN_E_SHAPE;
  const bool params = da || db;
  if (params && L > 0 && ((K > 0 && !da) || (N > 0 && !db))) return BNN_E_NULL;
  if (T > 0 && (!ids || (N > 0 && !dy))) return BNN_E_NULL;
  if (T > 0 && L > 0 && ((dx && K > 0 && !a) || (N > 0 && !b))) return BNN_E_NULL;
  if (params && T > 0 && (!u || (K > 0 && (!x || (xdtype == BNN_F8 && !xs))))) return BNN_E_NULL;
  const int64_t need = bnn_adapter_bwd_workspace(T, K, N, rank, L);
  if (need > 0 && !workspace) return BNN_E_NULL;
  if (ws_bytes < need) return BNN_E_SHAPE;
  const uintptr_t es = dtype == BNN_FP32 ? 4 : 2;
  if (misaligned(dy, 2) || misaligned(x, xdtype == BNN_F8 ? 16 : 2) || misaligned(xs, 4) ||
      misaligned(u, 4) || misaligned(ids, 4) || misaligned(a, 2) || misaligned(b, 2) ||
      misaligned(scale, 4) || misaligned(base, es) || misaligned(dx, es) || misaligned(da, 4) ||
      misaligned(db, 4) || misaligned(workspace, 16))
    return BNN_E_ALIGN;
  if (K == 0) dx = nullptr;
  const bool sums = params && L > 0 && K + N > 0;
  if (!sums && (!dx || T == 0)) return BNN_OK;
  const bnn::AdapterGrad g = {static_cast<const uint16_t *>(dy),
                              lddy,
                              x,
                              xdtype == BNN_F8 ? xs : nullptr,
                              ldx,
                              u,
                              ids,
                              static_cast<const uint16_t *>(a),
                              static_cast<const uint16_t *>(b),
                              scale,
                              base,
                              ldb,
                              dx,
                              lddx,
                              dtype,
                              sums,
                              da,
                              db};
  return launch_status(bnn::launch_adapter_bwd(g, workspace, T, K, N, (int)rank, (int)L,
                                               static_cast<hipStream_t>(stream)));
}

bnn_status bnn_gemm_u64(const uint64_t *xp, const uint64_t *wp, int32_t *y, int64_t M, int64_t N,
                        int64_t K, void *stream) {
  return bnn_gemm_ex(xp, wp, nullptr, y, M, N, K, BNN_EPI_I32, BNN_ALGO_AUTO, stream);
}

bnn_status bnn_gemm_u64_scaled(const uint64_t *xp, const uint64_t *wp, const float *alpha,
                               float *y, int64_t M, int64_t N, int64_t K, void *stream) {
  return bnn_gemm_ex(xp, wp, alpha, y, M, N, K, BNN_EPI_SCALED, BNN_ALGO_AUTO, stream);
}

bnn_status bnn_gemm_sign_repack(const uint64_t *xp, const uint64_t *wp, uint64_t *yp, int64_t M,
                                int64_t N, int64_t K, void *stream) {
  return bnn_gemm_ex(xp, wp, nullptr, yp, M, N, K, BNN_EPI_REPACK, BNN_ALGO_AUTO, stream);
}

}  // extern "C"
