// fp8.hpp -- device helpers and launchers of the 8-bit operators (E4M3 codes with one
// power-of-two scale per block of 128; the definitions are in include/nvfp4_amd_fp8.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "../../include/nvfp4_amd_fp8.h"
#include "device.hpp"
#include "fp8_plan.hpp"
#include "internal.hpp"

namespace nvfp4 {
namespace fp8 {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

template <class F, int... Is>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// K step Q (8 of a lane's 32 codes) as bf16 values with their block's scale applied;
// the converter takes the scale as a binary32 power of two.
template <int Q>
__device__ __forceinline__ bf16x8 widen8(const i32x8 &v, float scale) {
  const uint32_t lo = uint32_t(v[2 * Q]), hi = uint32_t(v[2 * Q + 1]);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

constexpr float kInfinity = __builtin_huge_valf();

// f as the sum of N bf16, each the nearest to what is left of it: three hold all of a binary32.
// A finite f has finite parts (the first is the largest bf16 where f would round to an
// infinity); an infinity or NaN is the first part, and the others are zeros, as inf - inf is a NaN.
template <int N>
__device__ __forceinline__ void split_bf16(float f, uint16_t (&w)[N]) {
  constexpr float kMost = 3.38953139e38f;  // (2 - 2^-7) 2^127
  const bool finite = __builtin_fabsf(f) < kInfinity;
  float left = f;
#pragma unroll
  for (int s = 0; s < N; ++s) {
    const float top = s == 0 && finite ? fminf(fmaxf(left, -kMost), kMost) : left;
    const __bf16 h = static_cast<__bf16>(top);
    w[s] = __builtin_bit_cast(uint16_t, h);
    left = finite ? left - static_cast<float>(h) : 0.0f;
  }
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

// Dropout (the definitions are in the header): thr = T, 0 for none, gain = q.
struct Drop {
  uint32_t thr;
  float gain;
  uint64_t seed, offset;
  const uint64_t *step;
};

inline Drop drop_of(const fp8_dropout_config *d) {
  if (!d) return Drop{0u, 1.0f, 0u, 0u, nullptr};
  const uint32_t t = uint32_t(d->p * 65536.0 + 0.5);
  return Drop{t, float(65536.0 / double(65536u - t)), d->seed, d->offset, d->step};
}

// The generator's state of a kernel, in scalar registers.
struct Mask {
  uint32_t thr, k0, k1, o0, o1;
  __device__ __forceinline__ explicit Mask(const Drop &d) : thr(d.thr), k0(uint32_t(d.seed)), k1(uint32_t(d.seed >> 32)) {
    const uint64_t o = d.offset + (d.step ? *d.step : 0u);
    o0 = uint32_t(o);
    o1 = uint32_t(o >> 32);
  }
  // half-word j (16 bits) for element j of group g
  __device__ __forceinline__ Philox4 draw(uint64_t g) const {
    return philox4x32_10(uint32_t(g), uint32_t(g >> 32), o0, o1, k0, k1);
  }
  // half-word j is all ones where element j of group g is kept, else 0: T - u saturates at 0
  // for the bits u of a kept element, and min(., 1) - 1 makes masks of it, two at a time
  __device__ __forceinline__ uint4 halves(uint64_t g) const {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const Philox4 r = draw(g);
    const u16x2 t = {uint16_t(thr), uint16_t(thr)}, one = {1, 1};
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u16x2 under = __builtin_elementwise_sub_sat(t, __builtin_bit_cast(u16x2, r.v[j]));
      w[j] = __builtin_bit_cast(uint32_t, u16x2(__builtin_elementwise_min(under, one) - one));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the same as bytes
  __device__ __forceinline__ uint2 bytes(uint64_t g) const {
    const uint4 w = halves(g);
    return make_uint2(__builtin_amdgcn_perm(w.y, w.x, 0x06040200u), __builtin_amdgcn_perm(w.w, w.z, 0x06040200u));
  }
  // bit j: element j of group g is kept
  __device__ __forceinline__ uint32_t bits(uint64_t g) const {
    const Philox4 r = draw(g);
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b |= ((r.v[j] & 0xFFFFu) >= thr ? 1u << (2 * j) : 0u) | ((r.v[j] >> 16) >= thr ? 2u << (2 * j) : 0u);
    return b;
  }
};

// What low-rank adapters add to a product, row m of which has adapter i = index[m]: coef[m]
// b_i^T, coef[m] the sum of the bf16 rows coef[m][0] .. coef[m][parts - 1], kept where the
// dropout of the result keeps.
struct LoraAdd {
  const uint16_t *coef;  // [M][parts][rank] bf16, of rows that have an adapter
  const uint16_t *b;     // [count][N][rank] bf16
  const int32_t *index;  // null: all 0
  int count, rank, parts;
  Drop drop;
};
// The bf16 of a coefficient: all of binary32, or with the 8-bit instruction, whose own sums keep
// fewer bits, 16 of its 24.
inline int lora_parts(bool fast) { return fast ? 2 : 3; }

// ---- launchers (arguments already checked)

hipError_t launch_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype, int64_t rows,
                          int64_t cols, const Drop &drop, void *y, int64_t ldy, hipStream_t stream);
// the norm with x dropped out before the residual's addition, and its gradient
hipError_t launch_dropout_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                                   int64_t rows, int64_t cols, const Drop &drop, const float *weight, float eps,
                                   void *h, int64_t ldh, const fp8_tensor *yq, const fp8_tensor *yq_t, float *rstd,
                                   hipStream_t stream);
hipError_t launch_dropout_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype,
                                            int64_t rows, int64_t cols, const Drop &drop, const float *weight,
                                            const float *rstd, void *dx, void *dresidual, float *dweight, float *ws,
                                            hipStream_t stream);

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
// The product's partial sums alone, [ksplit][M][ld] binary32 in ws.
struct Partials {
  int config, ksplit;
  int64_t ld;
  size_t bytes;
};
Partials gemm_partials(int64_t M, int64_t N, int64_t KB, bool fast);
hipError_t launch_gemm_partials(const fp8_tensor *a, const fp8_tensor *b, bool fast, float *ws, hipStream_t stream);
// C = a b^T and what `lora` adds, bf16, of more than 64 rows
hipError_t launch_gemm_lora(const fp8_tensor *a, const fp8_tensor *b, const LoraAdd &lora, void *c, int64_t ldc, bool fast,
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

// Low-rank adapters beside a projection (fp8_lora.hip).
// mixed: the caller's word that neighbouring tokens have different adapters.
size_t lora_fprop_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, bool mixed, bool fast);
hipError_t launch_lora_fprop(const fp8_tensor *xq, const fp8_tensor *wq, const fp8_lora *lora, const int32_t *index,
                             const Drop &drop, void *y, int64_t ldy, bool mixed, bool fast, void *ws, size_t ws_bytes,
                             hipStream_t stream);
size_t lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, int count, bool mixed, bool fast);
hipError_t launch_lora_backward(const fp8_tensor *dyq, const fp8_tensor *wq_t, const fp8_tensor *xq, const fp8_lora *lora,
                                const int32_t *index, const Drop &drop, void *dx, int64_t lddx, float *da, float *db,
                                bool mixed, bool fast, void *ws, size_t ws_bytes, hipStream_t stream);

}  // namespace fp8
}  // namespace nvfp4
