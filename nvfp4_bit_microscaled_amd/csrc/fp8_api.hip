// fp8_api.hip -- the extern "C" surface declared in include/nvfp4_amd_fp8.h: argument
// checks (all before any enqueue), then the launchers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.hpp"

namespace {

using nvfp4::fp8::ceil_div;
using nvfp4::fp8::kBlock;

// A row is a workgroup in the norm kernels, and a launch holds fewer than 2^32 threads.
constexpr int64_t kMaxDim = 16776960;

fp4_status from_hip(hipError_t e) { return e == hipSuccess ? FP4_OK : FP4_ERR_HIP; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known(fp4_dtype d) { return d == FP4_BF16 || d == FP4_FP32; }
uintptr_t size_of(fp4_dtype d) { return d == FP4_BF16 ? 2 : 4; }

fp4_status check_dims(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > kMaxDim || cols > kMaxDim) return FP4_ERR_SHAPE;
  // tiles of 128 x 128, one 256-thread workgroup each
  if (ceil_div(rows, kBlock) * ceil_div(cols, kBlock) > kMaxDim) return FP4_ERR_SHAPE;
  return FP4_OK;
}

fp4_status check_tensor(const fp8_tensor *t, int64_t rows, int64_t cols) {
  if (!t) return FP4_ERR_NULL;
  if (t->rows != rows || t->cols != cols) return FP4_ERR_MISMATCH;
  if (rows > 0 && cols > 0 && (!t->codes || !t->scales)) return FP4_ERR_NULL;
  if (!aligned(t->codes, 16) || !aligned(t->scales, 16)) return FP4_ERR_ALIGN;
  return FP4_OK;
}

fp4_status check_tensor(const fp8_tensor *t, int64_t rows, int64_t cols, bool two_d) {
  const fp4_status s = check_tensor(t, rows, cols);
  return s != FP4_OK ? s : (t->two_d != 0) != two_d ? FP4_ERR_MISMATCH : FP4_OK;
}

// a dense or strided tensor of the caller
fp4_status check_array(const void *p, fp4_dtype dtype, int64_t rows, int64_t cols, int64_t ld) {
  if (ld < cols) return FP4_ERR_SHAPE;
  if (!p && rows > 0 && cols > 0) return FP4_ERR_NULL;
  return aligned(p, size_of(dtype)) ? FP4_OK : FP4_ERR_ALIGN;
}

fp4_status check_ws(const void *ws, size_t ws_bytes) {
  if (ws_bytes > 0 && !ws) return FP4_ERR_NULL;
  return ws_bytes > 0 && !aligned(ws, 16) ? FP4_ERR_ALIGN : FP4_OK;
}

fp4_status check_drop(const fp8_dropout_config *d) {
  if (!d) return FP4_ERR_NULL;
  if (!(d->p >= 0.0 && d->p * 65536.0 + 0.5 < 65536.0)) return FP4_ERR_SHAPE;
  return aligned(d->step, 8) ? FP4_OK : FP4_ERR_ALIGN;
}

// Adapters' ranks, and how many elements all of them may have (a launch holds fewer than
// 2^32 threads).
constexpr int32_t kMaxRank = 128, kMaxAdapters = 65535;
constexpr int64_t kMaxAdapterElements = int64_t(1) << 32;
constexpr uint32_t kLoraFlags = FP8_GEMM_FAST | FP8_LORA_MIXED;

fp4_status check_lora_sizes(int64_t N, int64_t lda, int32_t rank, int32_t count) {
  if (rank <= 0 || rank > kMaxRank || rank % 8 != 0 || count <= 0 || count > kMaxAdapters) return FP4_ERR_SHAPE;
  if (lda < 0 || lda > kMaxDim + 8 || lda % 8 != 0) return FP4_ERR_SHAPE;
  return int64_t(rank) * count * (lda + N) > kMaxAdapterElements ? FP4_ERR_SHAPE : FP4_OK;
}

fp4_status check_lora(const fp8_lora *l, int64_t N, int64_t K, const int32_t *index) {
  if (!l) return FP4_ERR_NULL;
  if (l->lda < K) return FP4_ERR_SHAPE;
  const fp4_status s = check_lora_sizes(N, l->lda, l->rank, l->count);
  if (s != FP4_OK) return s;
  if ((!l->a && l->lda > 0) || (!l->b && N > 0) || !l->scale) return FP4_ERR_NULL;
  return aligned(l->a, 16) && aligned(l->b, 16) && aligned(l->scale, 4) && aligned(index, 4) ? FP4_OK : FP4_ERR_ALIGN;
}

int64_t kblocks(int64_t k) { return ceil_div(k, kBlock); }
size_t larger(size_t a, size_t b) { return a > b ? a : b; }

// The block's workspaces.  Every step may use all of it: the first half's partials
// (forward) or dh (backward) are read before a later product's partials are written.
size_t fprop_ws(int64_t M, int64_t K, int64_t F, bool keep, bool fast) {
  namespace f = nvfp4::fp8;
  return larger(f::act_ws_bytes(M, F, kblocks(K), fast, keep), f::gemm_ws_bytes(M, K, kblocks(F), fast));
}

// vec: g and u are aligned to 16 bytes
size_t backward_ws(int64_t M, int64_t K, int64_t F, bool vec, bool fast) {
  namespace f = nvfp4::fp8;
  return larger(larger(f::dact_ws_bytes(M, F, kblocks(K), vec, fast), f::gemm_ws_bytes(M, K, 2 * kblocks(F), fast)),
                f::gemm_group_ws_bytes(F, K, kblocks(M), 3, fast));
}

size_t ffn_ws(int64_t M, int64_t K, int64_t F) {
  size_t n = 0;
  for (const bool fast : {false, true})
    for (const bool other : {false, true})
      n = larger(n, larger(fprop_ws(M, K, F, other, fast), backward_ws(M, K, F, other, fast)));
  return n;
}

#define FP8_TRY(expr)                        \
  do {                                       \
    const fp4_status s_ = (expr);            \
    if (s_ != FP4_OK) return s_;             \
  } while (0)

#define FP8_RUN(expr)                                \
  do {                                               \
    if ((expr) != hipSuccess) return FP4_ERR_HIP;    \
  } while (0)

fp4_status check_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype, int64_t rows,
                      int64_t cols, const float *weight, float eps, void *h, int64_t ldh, const fp8_tensor *yq,
                      const fp8_tensor *yq_t, const float *rstd) {
  if (!known(dtype)) return FP4_ERR_DTYPE;
  FP8_TRY(check_dims(rows, cols));
  if (!(eps > 0.0f)) return FP4_ERR_SHAPE;
  FP8_TRY(check_array(x, dtype, rows, cols, ldx));
  if ((residual != nullptr) != (h != nullptr) && rows > 0 && cols > 0) return FP4_ERR_NULL;
  if (residual) {
    FP8_TRY(check_array(residual, dtype, rows, cols, ldr));
    FP8_TRY(check_array(h, dtype, rows, cols, ldh));
  }
  FP8_TRY(check_array(weight, FP4_FP32, 1, cols, cols));
  FP8_TRY(check_tensor(yq, rows, cols));
  if (yq->two_d) return FP4_ERR_MODE;
  if (yq_t) {
    FP8_TRY(check_tensor(yq_t, cols, rows));
    if (yq_t->two_d) return FP4_ERR_MODE;
    if (!rstd && rows > 0) return FP4_ERR_NULL;
  }
  return aligned(rstd, 4) ? FP4_OK : FP4_ERR_ALIGN;
}

fp4_status check_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                               int64_t cols, const float *weight, const float *rstd, const void *dx,
                               const float *dweight, const void *ws, size_t ws_bytes) {
  if (!known(dtype)) return FP4_ERR_DTYPE;
  FP8_TRY(check_dims(rows, cols));
  FP8_TRY(check_array(dy, dtype, rows, cols, cols));
  FP8_TRY(check_array(h, dtype, rows, cols, cols));
  FP8_TRY(check_array(dx, dtype, rows, cols, cols));
  if (dh) FP8_TRY(check_array(dh, dtype, rows, cols, cols));
  FP8_TRY(check_array(weight, FP4_FP32, 1, cols, cols));
  FP8_TRY(check_array(rstd, FP4_FP32, 1, rows, rows));
  FP8_TRY(check_array(dweight, FP4_FP32, 1, cols, cols));
  FP8_TRY(check_ws(ws, ws_bytes));
  return ws_bytes < nvfp4::fp8::rms_norm_ws_bytes(rows, cols) ? FP4_ERR_WORKSPACE : FP4_OK;
}

// either: the workspace of either call (fp8_ffn_ws_bytes) is asked for, else this call's own
fp4_status ffn_fprop(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, const fp8_tensor *wd,
                     const fp8_tensor *hq, void *g, void *u, void *y, int64_t ldy, bool fast, bool either, void *ws,
                     size_t ws_bytes, hipStream_t stream) {
  if (!xq || !wg || !wu || !wd || !hq) return FP4_ERR_NULL;
  const int64_t M = xq->rows, K = xq->cols, F = wg->rows;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, F));
  FP8_TRY(check_dims(F, K));
  FP8_TRY(check_tensor(xq, M, K, false));
  FP8_TRY(check_tensor(wg, F, K, true));
  FP8_TRY(check_tensor(wu, F, K, true));
  FP8_TRY(check_tensor(wd, K, F, true));
  FP8_TRY(check_tensor(hq, M, F, false));
  if ((g != nullptr) != (u != nullptr) && M > 0 && F > 0) return FP4_ERR_NULL;
  if (!aligned(g, 2) || !aligned(u, 2)) return FP4_ERR_ALIGN;
  FP8_TRY(check_array(y, FP4_BF16, M, K, ldy));
  FP8_TRY(check_ws(ws, ws_bytes));
  if (ws_bytes < (either ? ffn_ws(M, K, F) : fprop_ws(M, K, F, g != nullptr, fast))) return FP4_ERR_WORKSPACE;
  FP8_RUN(nvfp4::fp8::launch_gemm_act(xq, wg, wu, static_cast<uint16_t *>(g), static_cast<uint16_t *>(u), hq, fast,
                                      ws, ws_bytes, stream));
  return from_hip(nvfp4::fp8::launch_gemm(hq, wd, y, FP4_BF16, ldy, fast, ws, ws_bytes, stream));
}

fp4_status ffn_backward(const fp8_tensor *dyq, const fp8_tensor *dyq_t, const fp8_tensor *xq_t, const fp8_tensor *wg_t,
                        const fp8_tensor *wu_t, const fp8_tensor *wd_t, const void *g, const void *u,
                        const fp8_ffn_buffers *bufs, void *dx, void *dwg, void *dwu, void *dwd, bool fast, bool either,
                        void *ws, size_t ws_bytes, hipStream_t stream) {
  if (!dyq || !dyq_t || !xq_t || !wg_t || !wu_t || !wd_t || !bufs) return FP4_ERR_NULL;
  const int64_t M = dyq->rows, K = dyq->cols, F = wd_t->rows;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, F));
  FP8_TRY(check_dims(F, K));
  FP8_TRY(check_tensor(dyq, M, K, false));
  FP8_TRY(check_tensor(dyq_t, K, M, false));
  FP8_TRY(check_tensor(xq_t, K, M, false));
  FP8_TRY(check_tensor(wg_t, K, F, true));
  FP8_TRY(check_tensor(wu_t, K, F, true));
  FP8_TRY(check_tensor(wd_t, F, K, true));
  FP8_TRY(check_tensor(&bufs->dgq, M, F, false));
  FP8_TRY(check_tensor(&bufs->duq, M, F, false));
  FP8_TRY(check_tensor(&bufs->dgq_t, F, M, false));
  FP8_TRY(check_tensor(&bufs->duq_t, F, M, false));
  FP8_TRY(check_tensor(&bufs->hq_t, F, M, false));
  FP8_TRY(check_array(g, FP4_BF16, M, F, F));
  FP8_TRY(check_array(u, FP4_BF16, M, F, F));
  FP8_TRY(check_array(dx, FP4_BF16, M, K, K));
  FP8_TRY(check_array(dwg, FP4_BF16, F, K, K));
  FP8_TRY(check_array(dwu, FP4_BF16, F, K, K));
  FP8_TRY(check_array(dwd, FP4_BF16, K, F, F));
  FP8_TRY(check_ws(ws, ws_bytes));
  const bool vec = aligned(g, 16) && aligned(u, 16);
  if (ws_bytes < (either ? ffn_ws(M, K, F) : backward_ws(M, K, F, vec, fast))) return FP4_ERR_WORKSPACE;
  FP8_RUN(nvfp4::fp8::launch_gemm_dact(dyq, wd_t, static_cast<const uint16_t *>(g), static_cast<const uint16_t *>(u),
                                       bufs, fast, ws, stream));
  FP8_RUN(nvfp4::fp8::launch_gemm_sum(&bufs->dgq, wg_t, &bufs->duq, wu_t, dx, FP4_BF16, K, fast, ws, ws_bytes, stream));
  const nvfp4::fp8::GemmCall grads[3] = {{&bufs->dgq_t, xq_t, dwg, FP4_BF16, K},
                                         {&bufs->duq_t, xq_t, dwu, FP4_BF16, K},
                                         {dyq_t, &bufs->hq_t, dwd, FP4_BF16, F}};
  return from_hip(nvfp4::fp8::launch_gemm_group(grads, 3, fast, ws, ws_bytes, stream));
}

}  // namespace

extern "C" {

fp4_status fp8_tensor_bytes(int64_t rows, int64_t cols, int32_t two_d, size_t *codes_bytes, size_t *scales_bytes) {
  if (!codes_bytes || !scales_bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(rows, cols));
  *codes_bytes = size_t(rows) * size_t(nvfp4::fp8::padded_cols(cols));
  *scales_bytes = size_t(kblocks(cols)) * size_t(nvfp4::fp8::scale_row(rows, two_d != 0));
  return FP4_OK;
}

fp4_status fp8_quantize(const void *x, fp4_dtype dtype, int64_t rows, int64_t cols, int64_t ld, const fp8_tensor *q,
                        const fp8_tensor *q_t, hipStream_t stream) {
  if (!known(dtype)) return FP4_ERR_DTYPE;
  if (!q && !q_t) return FP4_ERR_NULL;
  FP8_TRY(check_dims(rows, cols));
  FP8_TRY(check_array(x, dtype, rows, cols, ld));
  if (q) FP8_TRY(check_tensor(q, rows, cols));
  if (q_t) FP8_TRY(check_tensor(q_t, cols, rows));
  if (q && q_t && (q->two_d != 0) != (q_t->two_d != 0)) return FP4_ERR_MISMATCH;
  return from_hip(nvfp4::fp8::launch_quantize(x, dtype, rows, cols, ld, q, q_t, stream));
}

fp4_status fp8_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype, int64_t rows,
                        int64_t cols, const float *weight, float eps, void *h, int64_t ldh, const fp8_tensor *yq,
                        const fp8_tensor *yq_t, float *rstd, hipStream_t stream) {
  FP8_TRY(check_norm(x, ldx, residual, ldr, dtype, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd));
  return from_hip(nvfp4::fp8::launch_rms_norm(x, ldx, residual, ldr, dtype, rows, cols, weight, eps, h, ldh, yq, yq_t,
                                              rstd, stream));
}

fp4_status fp8_dropout_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                                int64_t rows, int64_t cols, const fp8_dropout_config *drop, const float *weight,
                                float eps, void *h, int64_t ldh, const fp8_tensor *yq, const fp8_tensor *yq_t,
                                float *rstd, hipStream_t stream) {
  FP8_TRY(check_norm(x, ldx, residual, ldr, dtype, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd));
  FP8_TRY(check_drop(drop));
  if (!residual && rows > 0 && cols > 0) return FP4_ERR_NULL;
  return from_hip(nvfp4::fp8::launch_dropout_rms_norm(x, ldx, residual, ldr, dtype, rows, cols,
                                                      nvfp4::fp8::drop_of(drop), weight, eps, h, ldh, yq, yq_t, rstd,
                                                      stream));
}

fp4_status fp8_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype, int64_t rows,
                       int64_t cols, const fp8_dropout_config *drop, void *y, int64_t ldy, hipStream_t stream) {
  if (!known(dtype)) return FP4_ERR_DTYPE;
  FP8_TRY(check_dims(rows, cols));
  FP8_TRY(check_drop(drop));
  FP8_TRY(check_array(x, dtype, rows, cols, ldx));
  if (residual) FP8_TRY(check_array(residual, dtype, rows, cols, ldr));
  FP8_TRY(check_array(y, dtype, rows, cols, ldy));
  return from_hip(nvfp4::fp8::launch_dropout(x, ldx, residual, ldr, dtype, rows, cols, nvfp4::fp8::drop_of(drop), y, ldy,
                                             stream));
}

fp4_status fp8_rms_norm_ws_bytes(int64_t rows, int64_t cols, size_t *bytes) {
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(rows, cols));
  *bytes = nvfp4::fp8::rms_norm_ws_bytes(rows, cols);
  return FP4_OK;
}

fp4_status fp8_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                                 int64_t cols, const float *weight, const float *rstd, void *dx, float *dweight,
                                 void *ws, size_t ws_bytes, hipStream_t stream) {
  FP8_TRY(check_norm_backward(dy, h, dh, dtype, rows, cols, weight, rstd, dx, dweight, ws, ws_bytes));
  return from_hip(nvfp4::fp8::launch_rms_norm_backward(dy, h, dh, dtype, rows, cols, weight, rstd, dx, dweight,
                                                       static_cast<float *>(ws), stream));
}

fp4_status fp8_dropout_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                                         int64_t cols, const fp8_dropout_config *drop, const float *weight,
                                         const float *rstd, void *dx, void *dresidual, float *dweight, void *ws,
                                         size_t ws_bytes, hipStream_t stream) {
  FP8_TRY(check_norm_backward(dy, h, dh, dtype, rows, cols, weight, rstd, dx, dweight, ws, ws_bytes));
  FP8_TRY(check_drop(drop));
  FP8_TRY(check_array(dresidual, dtype, rows, cols, cols));
  return from_hip(nvfp4::fp8::launch_dropout_rms_norm_backward(dy, h, dh, dtype, rows, cols, nvfp4::fp8::drop_of(drop),
                                                               weight, rstd, dx, dresidual, dweight,
                                                               static_cast<float *>(ws), stream));
}

fp4_status fp8_lora_fprop_ws_bytes(int64_t M, int64_t N, int64_t K, int32_t rank, uint32_t flags, size_t *bytes) {
  if (flags & ~kLoraFlags) return FP4_ERR_MODE;
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, N));
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(N, K));
  FP8_TRY(check_lora_sizes(N, 0, rank, 1));
  *bytes = nvfp4::fp8::lora_fprop_ws_bytes(M, N, K, rank, flags & FP8_LORA_MIXED, flags & FP8_GEMM_FAST);
  return FP4_OK;
}

fp4_status fp8_lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t count, uint32_t flags,
                                      size_t *bytes) {
  if (flags & ~kLoraFlags) return FP4_ERR_MODE;
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, N));
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(N, K));
  FP8_TRY(check_lora_sizes(N, ceil_div(K, 8) * 8, rank, count));
  *bytes = nvfp4::fp8::lora_backward_ws_bytes(M, N, K, rank, count, flags & FP8_LORA_MIXED, flags & FP8_GEMM_FAST);
  return FP4_OK;
}

fp4_status fp8_lora_fprop(const fp8_tensor *xq, const fp8_tensor *wq, const fp8_lora *lora, const int32_t *index,
                          const fp8_dropout_config *drop, void *y, int64_t ldy, uint32_t flags, void *ws,
                          size_t ws_bytes, hipStream_t stream) {
  if (flags & ~kLoraFlags) return FP4_ERR_MODE;
  if (!xq || !wq) return FP4_ERR_NULL;
  const bool fast = flags & FP8_GEMM_FAST, mixed = flags & FP8_LORA_MIXED;
  const int64_t M = xq->rows, K = xq->cols, N = wq->rows;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, N));
  FP8_TRY(check_dims(N, K));
  FP8_TRY(check_tensor(xq, M, K, false));
  FP8_TRY(check_tensor(wq, N, K, true));
  FP8_TRY(check_lora(lora, N, K, index));
  if (drop) FP8_TRY(check_drop(drop));
  FP8_TRY(check_array(y, FP4_BF16, M, N, ldy));
  FP8_TRY(check_ws(ws, ws_bytes));
  if (ws_bytes < nvfp4::fp8::lora_fprop_ws_bytes(M, N, K, lora->rank, mixed, fast)) return FP4_ERR_WORKSPACE;
  return from_hip(nvfp4::fp8::launch_lora_fprop(xq, wq, lora, index, nvfp4::fp8::drop_of(drop), y, ldy, mixed, fast, ws,
                                                ws_bytes, stream));
}

fp4_status fp8_lora_backward(const fp8_tensor *dyq, const fp8_tensor *wq_t, const fp8_tensor *xq, const fp8_lora *lora,
                             const int32_t *index, const fp8_dropout_config *drop, void *dx, int64_t lddx, float *da,
                             float *db, uint32_t flags, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (flags & ~kLoraFlags) return FP4_ERR_MODE;
  if (!dyq || !wq_t || !xq) return FP4_ERR_NULL;
  const bool fast = flags & FP8_GEMM_FAST, mixed = flags & FP8_LORA_MIXED;
  const int64_t M = dyq->rows, N = dyq->cols, K = xq->cols;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, N));
  FP8_TRY(check_dims(N, K));
  FP8_TRY(check_tensor(dyq, M, N, false));
  FP8_TRY(check_tensor(wq_t, K, N, true));
  FP8_TRY(check_tensor(xq, M, K, false));
  FP8_TRY(check_lora(lora, N, K, index));
  if (drop) FP8_TRY(check_drop(drop));
  FP8_TRY(check_array(dx, FP4_BF16, M, K, lddx));
  if ((!da && lora->lda > 0) || (!db && N > 0)) return FP4_ERR_NULL;
  if (!aligned(da, 16) || !aligned(db, 16)) return FP4_ERR_ALIGN;
  FP8_TRY(check_ws(ws, ws_bytes));
  if (ws_bytes < nvfp4::fp8::lora_backward_ws_bytes(M, N, K, lora->rank, lora->count, mixed, fast)) return FP4_ERR_WORKSPACE;
  return from_hip(nvfp4::fp8::launch_lora_backward(dyq, wq_t, xq, lora, index, nvfp4::fp8::drop_of(drop), dx, lddx, da,
                                                   db, mixed, fast, ws, ws_bytes, stream));
}

fp4_status fp8_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes) {
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, N));
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(N, K));
  *bytes = larger(nvfp4::fp8::gemm_ws_bytes(M, N, kblocks(K), true), nvfp4::fp8::gemm_ws_bytes(M, N, kblocks(K), false));
  return FP4_OK;
}

fp4_status fp8_gemm(const fp8_tensor *a, const fp8_tensor *b, void *c, fp4_dtype c_dtype, int64_t ldc, uint32_t flags,
                    void *ws, size_t ws_bytes, hipStream_t stream) {
  if (flags & ~FP8_GEMM_FAST) return FP4_ERR_MODE;
  if (!a || !b) return FP4_ERR_NULL;
  if (!known(c_dtype)) return FP4_ERR_DTYPE;
  if (a->cols != b->cols) return FP4_ERR_MISMATCH;
  FP8_TRY(check_dims(a->rows, a->cols));
  FP8_TRY(check_dims(b->rows, b->cols));
  FP8_TRY(check_dims(a->rows, b->rows));
  FP8_TRY(check_tensor(a, a->rows, a->cols));
  FP8_TRY(check_tensor(b, b->rows, b->cols));
  FP8_TRY(check_array(c, c_dtype, a->rows, b->rows, ldc));
  FP8_TRY(check_ws(ws, ws_bytes));
  return from_hip(nvfp4::fp8::launch_gemm(a, b, c, c_dtype, ldc, flags & FP8_GEMM_FAST, ws, ws_bytes, stream));
}

fp4_status fp8_ffn_ws_bytes(int64_t M, int64_t K, int64_t F, size_t *bytes) {
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, F));
  FP8_TRY(check_dims(F, K));
  *bytes = ffn_ws(M, K, F);
  return FP4_OK;
}

fp4_status fp8_ffn_fprop_ws_bytes(int64_t M, int64_t K, int64_t F, int32_t keep, uint32_t flags, size_t *bytes) {
  if (flags & ~FP8_GEMM_FAST) return FP4_ERR_MODE;
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, F));
  FP8_TRY(check_dims(F, K));
  *bytes = fprop_ws(M, K, F, keep != 0, flags & FP8_GEMM_FAST);
  return FP4_OK;
}

fp4_status fp8_ffn_backward_ws_bytes(int64_t M, int64_t K, int64_t F, uint32_t flags, size_t *bytes) {
  if (flags & ~FP8_GEMM_FAST) return FP4_ERR_MODE;
  if (!bytes) return FP4_ERR_NULL;
  FP8_TRY(check_dims(M, K));
  FP8_TRY(check_dims(M, F));
  FP8_TRY(check_dims(F, K));
  *bytes = backward_ws(M, K, F, true, flags & FP8_GEMM_FAST);
  return FP4_OK;
}

fp4_status fp8_ffn_fprop(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, const fp8_tensor *wd,
                         const fp8_tensor *hq, void *g, void *u, void *y, int64_t ldy, void *ws, size_t ws_bytes,
                         hipStream_t stream) {
  return ffn_fprop(xq, wg, wu, wd, hq, g, u, y, ldy, false, true, ws, ws_bytes, stream);
}

fp4_status fp8_ffn_fprop_flags(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, const fp8_tensor *wd,
                               const fp8_tensor *hq, void *g, void *u, void *y, int64_t ldy, uint32_t flags, void *ws,
                               size_t ws_bytes, hipStream_t stream) {
  if (flags & ~FP8_GEMM_FAST) return FP4_ERR_MODE;
  return ffn_fprop(xq, wg, wu, wd, hq, g, u, y, ldy, flags & FP8_GEMM_FAST, false, ws, ws_bytes, stream);
}

fp4_status fp8_ffn_backward(const fp8_tensor *dyq, const fp8_tensor *dyq_t, const fp8_tensor *xq_t,
                            const fp8_tensor *wg_t, const fp8_tensor *wu_t, const fp8_tensor *wd_t, const void *g,
                            const void *u, const fp8_ffn_buffers *bufs, void *dx, void *dwg, void *dwu, void *dwd,
                            void *ws, size_t ws_bytes, hipStream_t stream) {
  return ffn_backward(dyq, dyq_t, xq_t, wg_t, wu_t, wd_t, g, u, bufs, dx, dwg, dwu, dwd, false, true, ws, ws_bytes,
                      stream);
}

fp4_status fp8_ffn_backward_flags(const fp8_tensor *dyq, const fp8_tensor *dyq_t, const fp8_tensor *xq_t,
                                  const fp8_tensor *wg_t, const fp8_tensor *wu_t, const fp8_tensor *wd_t,
                                  const void *g, const void *u, const fp8_ffn_buffers *bufs, void *dx, void *dwg,
                                  void *dwu, void *dwd, uint32_t flags, void *ws, size_t ws_bytes,
                                  hipStream_t stream) {
  if (flags & ~FP8_GEMM_FAST) return FP4_ERR_MODE;
  return ffn_backward(dyq, dyq_t, xq_t, wg_t, wu_t, wd_t, g, u, bufs, dx, dwg, dwu, dwd, flags & FP8_GEMM_FAST, false,
                      ws, ws_bytes, stream);
}

}  // extern "C"
