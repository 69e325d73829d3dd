// fp8.hpp -- device helpers and launchers of the 8-bit operators (E4M3 codes with one
// power-of-two scale per block of 128; the definitions are in include/nvfp4_amd_fp8.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_amd_fp8.h"
#include "device.hpp"
#include "fp8_plan.hpp"
#include "internal.hpp"

namespace nvfp4 {
namespace fp8 {

inline int64_t padded_cols(int64_t cols) { return ceil_div(cols, kBlock) * kBlock; }
// bytes of one K block's scales
inline int64_t scale_row(int64_t rows, bool two_d) {
  return two_d ? ceil_div(rows, kBlock) : ceil_div(rows, 16) * 16;
}

// A quantized output as the kernels write it.
struct Out {
  uint8_t *codes, *scales;  // codes null: this layout is not wanted
  int64_t rows, cols_p, srow;
};

inline Out out_of(const fp8_tensor *t) {
  if (!t) return Out{};
  return Out{t->codes, t->scales, t->rows, padded_cols(t->cols), scale_row(t->rows, t->two_d != 0)};
}

// The five tensors of the gated block's backward element-wise step.
struct DactOut {
  Out dg, du, dg_t, du_t, h_t;
};

inline DactOut dact_out(const fp8_ffn_buffers *b) {
  return DactOut{out_of(&b->dgq), out_of(&b->duq), out_of(&b->dgq_t), out_of(&b->duq_t), out_of(&b->hq_t)};
}

// E8M0 byte of the smallest 2^e with amax <= 448 * 2^e, from the bits of the
// non-negative amax = m * 2^x, 1 <= m < 2: 448 = 1.75 * 2^8, so e = x - 8, plus 1 when
// m > 1.75 (adding 0x1FFFFF to the mantissa then carries).  Clamped to [1, 254]; a
// block of zeros takes the scale 1.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = int((b + 0x1FFFFFu) >> 23) - 8;
  return b == 0u ? 127u : uint32_t(max(1, min(254, e)));
}

// The scale itself, 2^(byte - 127).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four values over their scale (at most 448 in magnitude) to E4M3, nearest-even.
// gfx950's scaled converter divides by the power of two and rounds once: the same codes,
// over all values and at every tie and its neighbours, as a product with the inverse
// and the plain converter, without the products.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float scale) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, w);
}

// Rotation by N lanes within each row of 16.
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}

// Maximum over the 16 lanes of a row, in every lane.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  return fmaxf(v, row_ror<1>(v));
}

// The same of non-negative floats by their bits, which order alike: one instruction a
// step, where a float maximum of a shuffled value first makes it canonical.
template <int N>
__device__ __forceinline__ uint32_t row_ror_bits(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t row16_max_bits(uint32_t v) {
  v = max(v, row_ror_bits<8>(v));
  v = max(v, row_ror_bits<4>(v));
  v = max(v, row_ror_bits<2>(v));
  return max(v, row_ror_bits<1>(v));
}

// sigmoid(g).  exp(-g) = 2^(-g log2 e): the product's rounding shifts the result by at
// most |g| * 2^-24 relative, below a bf16 or E4M3 step for every g whose sigmoid is not
// itself negligible; the hardware's exp2 and reciprocal are within one ulp.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// silu'(g) from s = sigmoid(g) and silu = g * s: s + silu * (1 - s).
__device__ __forceinline__ float dsilu(float s, float silu) { return __builtin_fmaf(silu, 1.0f - s, s); }

// ---- launchers (arguments already checked)

hipError_t launch_quantize(const void *x, fp4_dtype dtype, int64_t rows, int64_t cols, int64_t ld, const fp8_tensor *q,
                           const fp8_tensor *q_t, hipStream_t stream);
hipError_t launch_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                           int64_t rows, int64_t cols, const float *weight, float eps, void *h, int64_t ldh,
                           const fp8_tensor *yq, const fp8_tensor *yq_t, float *rstd, hipStream_t stream);
hipError_t launch_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                                    int64_t cols, const float *weight, const float *rstd, void *dx, float *dweight,
                                    float *ws, hipStream_t stream);
size_t rms_norm_ws_bytes(int64_t rows, int64_t cols);

// hq = Q(silu(g) * u) from g and u of row stride ld
hipError_t launch_act_quantize(const uint16_t *g, const uint16_t *u, int64_t ld, const fp8_tensor *hq,
                               hipStream_t stream);
// the backward's element-wise step: dh binary32 [M][F] -> the five tensors of bufs
hipError_t launch_dact_quantize(const float *dh, int64_t ld, const uint16_t *g, const uint16_t *u,
                                const fp8_ffn_buffers *bufs, hipStream_t stream);

// fast: by the 8-bit matrix instruction, else by the bf16 one (FP8_GEMM_FAST)
hipError_t launch_gemm(const fp8_tensor *a, const fp8_tensor *b, void *c, fp4_dtype c_dtype, int64_t ldc, bool fast,
                       void *ws, size_t ws_bytes, hipStream_t stream);
// C = a1 b1^T + a2 b2^T, one accumulation over both
hipError_t launch_gemm_sum(const fp8_tensor *a1, const fp8_tensor *b1, const fp8_tensor *a2, const fp8_tensor *b2,
                           void *c, fp4_dtype c_dtype, int64_t ldc, bool fast, void *ws, size_t ws_bytes,
                           hipStream_t stream);
size_t gemm_ws_bytes(int64_t M, int64_t N, int64_t KB, bool fast);  // KB: 128-wide K stages in all

// Up to three independent products, fast ones in one launch where all are large.
struct GemmCall {
  const fp8_tensor *a, *b;
  void *c;
  fp4_dtype c_dtype;
  int64_t ldc;
};
hipError_t launch_gemm_group(const GemmCall *calls, int n, bool fast, void *ws, size_t ws_bytes, hipStream_t stream);
// of n products whose tile grids are M x N or N x M
size_t gemm_group_ws_bytes(int64_t M, int64_t N, int64_t KB, int n, bool fast);

// The gated block's projections, activation and quantization: hq = Q(silu(g) * u), g = x
// wg^T and u = x wu^T in bf16, written where not null.  ws: act_ws_bytes, keep where they are.
size_t act_ws_bytes(int64_t M, int64_t F, int64_t KB, bool fast, bool keep);
hipError_t launch_gemm_act(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, uint16_t *g, uint16_t *u,
                           const fp8_tensor *hq, bool fast, void *ws, size_t ws_bytes, hipStream_t stream);
// The backward pass's dh = dy wd and its element-wise step.  ws: dact_ws_bytes, vec where g
// and u are aligned to 16 bytes.
size_t dact_ws_bytes(int64_t M, int64_t F, int64_t KB, bool vec, bool fast);
hipError_t launch_gemm_dact(const fp8_tensor *dyq, const fp8_tensor *wd_t, const uint16_t *g, const uint16_t *u,
                            const fp8_ffn_buffers *bufs, bool fast, void *ws, hipStream_t stream);

}  // namespace fp8
}  // namespace nvfp4
