// fp8_quant.hip -- the memory-bound kernels of the 8-bit operators: quantization in
// both layouts, the RMS norm with its residual and its gradient, and the gated
// block's element-wise steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.hpp"

namespace nvfp4 {
namespace fp8 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void load8_vec(const uint16_t *p, float v[8]) {
  const uint4 q = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load8_vec(const float *p, float v[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  const float4 b = *reinterpret_cast<const float4 *>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ float widen(uint16_t b) { return bf16_to_f32(b); }
__device__ __forceinline__ float widen(float f) { return f; }

// Nearest-even bf16 that keeps a NaN a NaN (adding to a NaN's bits could carry into an
// infinity or past the sign).
__device__ __forceinline__ uint16_t to_bf16(float f) {
  return f != f ? uint16_t(0x7FC0u) : f32_to_bf16(f);
}

// v rounded to T's type and back
__device__ __forceinline__ float rounded(float v, uint16_t) { return bf16_to_f32(to_bf16(v)); }
__device__ __forceinline__ float rounded(float v, float) { return v; }

__device__ __forceinline__ void store8_vec(uint16_t *p, const float v[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = uint32_t(to_bf16(v[2 * j])) | (uint32_t(to_bf16(v[2 * j + 1])) << 16);
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8_vec(float *p, const float v[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = to_bf16(v); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// 8 elements as loaded, widened when they are used: a load in flight then holds 4 (bf16)
// or 8 (binary32) registers.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void set(int j, uint16_t b) {
    uint32_t &x = j >> 1 == 0 ? w.x : j >> 1 == 1 ? w.y : j >> 1 == 2 ? w.z : w.w;
    x |= uint32_t(b) << (16 * (j & 1));
  }
  __device__ __forceinline__ float at(int j) const {
    const uint32_t x = j >> 1 == 0 ? w.x : j >> 1 == 1 ? w.y : j >> 1 == 2 ? w.z : w.w;
    return __uint_as_float((j & 1) ? (x & 0xFFFF0000u) : (x << 16));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void set(int j, float v) {
    (j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : j == 3 ? a.w : j == 4 ? b.x : j == 5 ? b.y : j == 6 ? b.z : b.w) = v;
  }
  __device__ __forceinline__ float at(int j) const {
    return j == 0 ? a.x : j == 1 ? a.y : j == 2 ? a.z : j == 3 ? a.w : j == 4 ? b.x : j == 5 ? b.y : j == 6 ? b.z : b.w;
  }
};

// A row's group of 8 from column c on, zeros past `cols`.  VEC: cols is a multiple of 8
// and groups are 16-byte aligned, so a group is inside or outside as a whole and no
// element-wise path stands between one load and the next.  Otherwise an access's lanes
// are 8 elements apart, and rows that take no 16-byte loads cost two to three times as
// much: 8192x4095 bf16 quantized in 45 us (8192x4096: 23), the norm's rows of 16384x5117
// in 375 (5120 columns: 111).
template <bool VEC, typename T>
__device__ __forceinline__ Raw8<T> fetch8(const T *row, int64_t c, int64_t cols) {
  Raw8<T> r;
  r.zero();
  if constexpr (VEC) {
    if (c < cols) r.load(row + c);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) r.set(j, row[c + j]);
  }
  return r;
}

template <bool VEC, typename T>
__device__ __forceinline__ void put8(T *row, int64_t c, int64_t cols, const float v[8]) {
  if constexpr (VEC) {
    if (c < cols) store8_vec(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) store1(row + c + j, v[j]);
  }
}

// 8 elements of a row from column c on, zeros past `cols`; vec: whole groups are
// 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, bool vec, float v[8]) {
  if (vec && c + 8 <= cols) {
    load8_vec(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? widen(row[c + j]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *row, int64_t c, int64_t cols, bool vec, const float v[8]) {
  if (vec && c + 8 <= cols) {
    store8_vec(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) store1(row + c + j, v[j]);
  }
}

// ---------------------------------------------------------------------------
// A 128 x 128 tile in a workgroup's registers: thread t holds rows 8 (t / 16) + p and
// columns 8 (t % 16) + j as v[p][j], zeros outside the tensor.  Loads of a tile's row
// are 16 lanes x 8 elements; a thread's 8 x 8 block gives 8 codes side by side in both
// layouts.  Row maxima stay in 16 lanes; column maxima join the 16 thread rows through
// LDS; the transposed codes pass through LDS so that both layouts leave as whole
// 128-byte runs.
struct TileLds {
  float col[4][kBlock];
  float all[4];
  alignas(16) uint8_t codes[kBlock * kBlock];
};

__device__ __forceinline__ void tile_rows_out(const float (&v)[8][8], const Out &o, int64_t r0, int64_t c0,
                                              const uint32_t (&sb)[8], int cg, int rg) {
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = r0 + 8 * rg + p;
    if (r < o.rows) {
      const float m = scale_of(sb[p]);
      uint2 w;
      w.x = encode4(v[p][0], v[p][1], v[p][2], v[p][3], m);
      w.y = encode4(v[p][4], v[p][5], v[p][6], v[p][7], m);
      *reinterpret_cast<uint2 *>(o.codes + r * o.cols_p + c0 + 8 * cg) = w;
    }
  }
}

__device__ __forceinline__ void tile_cols_out(const float (&v)[8][8], const Out &o, int64_t r0, int64_t c0,
                                              const uint32_t (&sb)[8], int cg, int rg, TileLds &lds) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = scale_of(sb[j]);
    uint2 w;
    w.x = encode4(v[0][j], v[1][j], v[2][j], v[3][j], m);
    w.y = encode4(v[4][j], v[5][j], v[6][j], v[7][j], m);
    // 8-byte slot rg of column 8 cg + j, XOR-swizzled by cg against bank conflicts
    *reinterpret_cast<uint2 *>(lds.codes + (8 * cg + j) * kBlock + ((rg ^ cg) << 3)) = w;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int u = k * kThreads + threadIdx.x, col = u >> 3, q = u & 7, s = col >> 3;
    const uint2 a = *reinterpret_cast<const uint2 *>(lds.codes + col * kBlock + (((2 * q) ^ s) << 3));
    const uint2 b = *reinterpret_cast<const uint2 *>(lds.codes + col * kBlock + (((2 * q + 1) ^ s) << 3));
    if (c0 + col < o.rows)
      *reinterpret_cast<uint4 *>(o.codes + (c0 + col) * o.cols_p + r0 + 16 * q) = make_uint4(a.x, a.y, b.x, b.y);
  }
}

// 8 scale bytes from `at` on, clipped at the padded row count.
__device__ __forceinline__ void store_scales8(uint8_t *row, int64_t at, int64_t srow, const uint32_t (&sb)[8]) {
  if (at >= srow) return;  // srow is a multiple of 16 and `at` of 8
  uint2 w;
  w.x = sb[0] | (sb[1] << 8) | (sb[2] << 16) | (sb[3] << 24);
  w.y = sb[4] | (sb[5] << 8) | (sb[6] << 16) | (sb[7] << 24);
  *reinterpret_cast<uint2 *>(row + at) = w;
}

// Quantizes the tile at (r0, c0) into the wanted layouts.  Every thread calls it; the
// caller syncs before the LDS is used again.
__device__ __forceinline__ void tile_quantize(const float (&v)[8][8], const Out &q, const Out &qt, bool two_d,
                                              int64_t r0, int64_t c0, TileLds &lds) {
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4;
  uint32_t sb[8];
  if (two_d) {
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, __builtin_fabsf(v[p][j]));
    m = row16_max(m);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    if ((t & 63) == 0) lds.all[t >> 6] = m;
    __syncthreads();
    const uint32_t s = scale_byte(fmaxf(fmaxf(lds.all[0], lds.all[1]), fmaxf(lds.all[2], lds.all[3])));
#pragma unroll
    for (int p = 0; p < 8; ++p) sb[p] = s;
    if (t == 0) {
      if (q.codes) q.scales[(c0 / kBlock) * q.srow + r0 / kBlock] = uint8_t(s);
      if (qt.codes) qt.scales[(r0 / kBlock) * qt.srow + c0 / kBlock] = uint8_t(s);
    }
    if (q.codes) tile_rows_out(v, q, r0, c0, sb, cg, rg);
    if (qt.codes) tile_cols_out(v, qt, r0, c0, sb, cg, rg, lds);
    return;
  }
  if (q.codes) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, __builtin_fabsf(v[p][j]));
      sb[p] = scale_byte(row16_max(m));
    }
    if (cg == 0) store_scales8(q.scales + (c0 / kBlock) * q.srow, r0 + 8 * rg, q.srow, sb);
    tile_rows_out(v, q, r0, c0, sb, cg, rg);
  }
  if (qt.codes) {
    float m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0.0f;
#pragma unroll
      for (int p = 0; p < 8; ++p) m[j] = fmaxf(m[j], __builtin_fabsf(v[p][j]));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 16, 64));
      m[j] = fmaxf(m[j], __shfl_xor(m[j], 32, 64));
    }
    if ((t & 48) == 0) {  // one thread row of each wave
#pragma unroll
      for (int j = 0; j < 8; ++j) lds.col[t >> 6][8 * cg + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = 8 * cg + j;
      sb[j] = scale_byte(fmaxf(fmaxf(lds.col[0][c], lds.col[1][c]), fmaxf(lds.col[2][c], lds.col[3][c])));
    }
    if (rg == 0) store_scales8(qt.scales + (r0 / kBlock) * qt.srow, c0 + 8 * cg, qt.srow, sb);
    tile_cols_out(v, qt, r0, c0, sb, cg, rg, lds);
  }
}

// Tile index -> (row block, column block), column blocks innermost.
__device__ __forceinline__ void tile_pos(int64_t cblocks, int64_t &r0, int64_t &c0) {
  const int64_t b = blockIdx.x;
  r0 = (b / cblocks) * kBlock;
  c0 = (b % cblocks) * kBlock;
}

// A thread's 8 x 8 of the tile at (r0, c0) as loaded.  A tile inside the tensor issues its
// eight loads without a test between them.
template <typename T>
__device__ __forceinline__ void tile_fetch(const T *x, int64_t rows, int64_t cols, int64_t ld, bool vec, int64_t r0,
                                           int64_t c0, int cg, int rg, Raw8<T> (&v)[8]) {
  const int64_t r = r0 + 8 * rg, c = c0 + 8 * cg;
  if (vec && r0 + kBlock <= rows && c0 + kBlock <= cols) {
    const T *at = x + r * ld + c;
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p].load(at + p * ld);
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) v[p] = fetch8<false>(x + (r + p < rows ? r + p : 0) * ld, c, r + p < rows ? cols : 0);
  }
}

// Both layouts of a 128 x 128 tile from one read of it: a thread holds 8 x 8 elements, so
// a row's block maximum joins 16 lanes and a column's joins 16 threads of four waves, and
// the codes leave in whole 128-byte rows of either layout.  HBM bounds it: 20480 x 5120
// fp32 in both layouts, 629 MB, 118 us (5.3 TB/s; a copy runs at 4.8 to 4.9); 8192 x 4096
// bf16, 22.6 us.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T *x, int64_t rows, int64_t cols, int64_t ld,
                                                            int64_t cblocks, int vec, Out q, Out qt, int two_d) {
  __shared__ TileLds lds;
  int64_t r0, c0;
  tile_pos(cblocks, r0, c0);
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  Raw8<T> raw[8];
  tile_fetch(x, rows, cols, ld, vec, r0, c0, cg, rg, raw);
  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[p][j] = raw[p].at(j);
  tile_quantize(v, q, qt, two_d, r0, c0, lds);
}

// ---------------------------------------------------------------------------
// The norm's row pass: TPR threads own a row, each NCH groups of 8 columns held in
// registers between the sum of squares and the output, so x and the residual are read
// once.  A 128-column block is 16 neighbouring lanes.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S s, S *part) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the last row's sums have been read
    if ((threadIdx.x & 63) == 0) part[w] = s;
    __syncthreads();
    s = (part[0] + part[1]) + (part[2] + part[3]);
  }
  return s;
}

// (sum / cols + eps)^-1/2, rounded once: a Newton step in binary64 on the binary32 value.
// A block's scale and a code's rounding are steps in y, so what is left of y's error
// decides how often they fall on the other side of one; the time is the same.
__device__ __forceinline__ float inv_rms(double sum, int64_t cols, float eps) {
  const double m = sum * (1.0 / double(cols)) + double(eps);
  const float y = 1.0f / __fsqrt_rn(float(m));
  const double e = __builtin_fma(-m * double(y), double(y), 1.0);
  // out of binary32's range (y is 0 or infinite) there is no step to take
  return __builtin_fabs(e) < 1.0 ? float(double(y) + 0.5 * double(y) * e) : y;
}
// h * rs * w, rounded once but for second-order terms
__device__ __forceinline__ float normed(float h, float rs, float w) {
  const float p = h * rs;
  return __builtin_fmaf(p, w, __builtin_fmaf(h, rs, -p) * w);
}

template <typename T>
struct NormArgs {
  const T *x, *res;
  T *h;
  int64_t ldx, ldr, ldh, rows, cols;
  const float *weight;
  float eps;
  float *rstd;
  Out y;
  int vec;
  Drop drop;  // of x, where the kernel is one with DROP
};

// v[j] = x[j] dropped out: times gain where bit j is set, else 0 (whatever x[j] is)
__device__ __forceinline__ float dropped(float x, uint32_t bits, int j, float gain) {
  return (bits >> j) & 1u ? x * gain : 0.0f;
}
__host__ __device__ __forceinline__ int64_t drop_groups(int64_t cols) { return (cols + 7) >> 3; }

// The norm of rows that fit in registers: TPR threads to a row, 8 NCH elements each, in
// one pass; a workgroup of 256 takes 256 / TPR rows.  The 16 lanes of a block of 128 find
// its maximum without LDS.  HBM bounds it: 16384 x 5120 bf16 with the residual, 587 MB,
// 109 us (5.4 TB/s); one row of 5120 takes 4.2 us, the launch and two round trips to memory.
// DROP: x is dropped out before the residual is added; a thread's 8 columns are one group of
// the generator (114 us: the generator runs while the loads are on their way).
template <typename T, int TPR, int NCH, bool VEC, bool DROP>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs<T> p) {
  __shared__ double part[4];
  const int lt = threadIdx.x % TPR;
  const int64_t r = int64_t(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (TPR < kThreads && r >= p.rows) return;  // whole waves; no barrier follows when TPR is a wave
  const T *xr = p.x + r * p.ldx;
  const T *rr = p.res ? p.res + r * p.ldr : nullptr;
  T *hr = p.res ? p.h + r * p.ldh : nullptr;
  Raw8<T> x[NCH], r2[NCH];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int64_t c = 8 * int64_t(lt + k * TPR);
    x[k] = fetch8<VEC>(xr, c, p.cols);
    if (rr) r2[k] = fetch8<VEC>(rr, c, p.cols);
  }
  // the weights' loads are behind the row's, and there when the sum is
  Raw8<float> w[NCH];
#pragma unroll
  for (int k = 0; k < NCH; ++k) w[k] = fetch8<VEC>(p.weight, 8 * int64_t(lt + k * TPR), p.cols);
  uint32_t kept[NCH];
  if constexpr (DROP) {
    const Mask mask(p.drop);
#pragma unroll
    for (int k = 0; k < NCH; ++k) kept[k] = mask.bits(uint64_t(r) * drop_groups(p.cols) + (lt + k * TPR));
  }
  float v[NCH][8];
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (DROP) v[k][j] = rounded(dropped(x[k].at(j), kept[k], j, p.drop.gain) + r2[k].at(j), T());
      else v[k][j] = rr ? rounded(x[k].at(j) + r2[k].at(j), T()) : x[k].at(j);
      s = __builtin_fmaf(v[k][j], v[k][j], s);
    }
    if (rr) put8<VEC>(hr, 8 * int64_t(lt + k * TPR), p.cols, v[k]);
  }
  const float rs = inv_rms(row_sum<TPR>(double(s), part), p.cols, p.eps);
  if (lt == 0 && p.rstd) p.rstd[r] = rs;
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int64_t c = 8 * int64_t(lt + k * TPR);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // zeros past the width also where rstd is a NaN
      v[k][j] = normed(v[k][j], (VEC ? c : c + j) < p.cols ? rs : 0.0f, w[k].at(j));
      m = fmaxf(m, __builtin_fabsf(v[k][j]));
    }
    const uint32_t sb = scale_byte(row16_max(m));
    if (c < p.y.cols_p) {
      const float sc = scale_of(sb);
      uint2 o;
      o.x = encode4(v[k][0], v[k][1], v[k][2], v[k][3], sc);
      o.y = encode4(v[k][4], v[k][5], v[k][6], v[k][7], sc);
      *reinterpret_cast<uint2 *>(p.y.codes + r * p.y.cols_p + c) = o;
      if ((lt & 15) == 0) p.y.scales[(c / kBlock) * p.y.srow + r] = uint8_t(sb);
    }
  }
}

// Rows too wide for registers: the same with h read again (from h, or x without a
// residual) for the output; each thread re-reads what it wrote itself.
template <typename T, bool DROP>
__global__ __launch_bounds__(kThreads) void norm_wide_kernel(NormArgs<T> p) {
  __shared__ double part[4];
  const int64_t r = blockIdx.x;
  const T *xr = p.x + r * p.ldx;
  const T *rr = p.res ? p.res + r * p.ldr : nullptr;
  T *hr = p.res ? p.h + r * p.ldh : nullptr;
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kThreads) {
    float v[8], w[8];
    load8(xr, c, p.cols, p.vec, v);
    if constexpr (DROP) {
      const uint32_t kept = Mask(p.drop).bits(uint64_t(r) * drop_groups(p.cols) + (c >> 3));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = dropped(v[j], kept, j, p.drop.gain);
    }
    if (rr) {
      load8(rr, c, p.cols, p.vec, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = rounded(v[j] + w[j], T());
      store8(hr, c, p.cols, p.vec, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[j], v[j], s);
  }
  const float rs = inv_rms(row_sum<kThreads>(double(s), part), p.cols, p.eps);
  if (threadIdx.x == 0 && p.rstd) p.rstd[r] = rs;
  const T *src = p.res ? hr : xr;
  for (int64_t c = 8 * threadIdx.x; c < p.y.cols_p; c += 8 * kThreads) {  // whole groups of 16 lanes
    float v[8], w[8], m = 0.0f;
    load8(src, c, p.cols, p.vec, v);
    load8(p.weight, c, p.cols, p.vec, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = normed(v[j], c + j < p.cols ? rs : 0.0f, w[j]);
      m = fmaxf(m, __builtin_fabsf(v[j]));
    }
    const uint32_t sb = scale_byte(row16_max(m));
    const float sc = scale_of(sb);
    uint2 o;
    o.x = encode4(v[0], v[1], v[2], v[3], sc);
    o.y = encode4(v[4], v[5], v[6], v[7], sc);
    *reinterpret_cast<uint2 *>(p.y.codes + r * p.y.cols_p + c) = o;
    if ((threadIdx.x & 15) == 0) p.y.scales[(c / kBlock) * p.y.srow + r] = uint8_t(sb);
  }
}

// y^T of the norm, from h and rstd: the quantizer's tiles, scaled by rstd and weight.  Its
// blocks run down 128 rows, which no workgroup of norm_kernel holds (128 rows of 5120
// bf16 are 1.3 MB), so it reads h again: 16384 x 5120, 252 MB, 52 us (4.9 TB/s).
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_cols_kernel(const T *h, int64_t ld, int64_t rows, int64_t cols,
                                                             const float *weight, const float *rstd, int64_t cblocks,
                                                             int vec, Out qt) {
  __shared__ TileLds lds;
  int64_t r0, c0;
  tile_pos(cblocks, r0, c0);
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  Raw8<T> raw[8];
  tile_fetch(h, rows, cols, ld, vec, r0, c0, cg, rg, raw);
  float w[8], rs[8], v[8][8];
  load8(weight, c0 + 8 * cg, cols, vec, w);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int64_t r = r0 + 8 * rg + p;
    rs[p] = r < rows ? rstd[r] : 0.0f;  // rows past the end hold zeros, whatever the last one's is
  }
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[p][j] = normed(raw[p].at(j), rs[p], w[j]);
  tile_quantize(v, Out{}, qt, false, r0, c0, lds);
}

// ---------------------------------------------------------------------------
// The norm's gradient: a workgroup walks rows blockIdx, + gridDim, ... and keeps its
// sums of dy * hhat per column in registers (at most rows / gridDim terms in binary32);
// they go to partial[blockIdx] and a second kernel joins the partials in binary64.
template <typename T>
struct NormGradArgs {
  const T *dy, *h, *dh;
  T *dx;
  int64_t rows, cols;
  const float *weight, *rstd;
  float *partial;
  int vec;
  T *dres;    // with DROP: the residual's gradient, dx being x's
  Drop drop;
};

// Thread lt's groups k of 8 columns: whole 16-byte groups where rows allow it (VEC), else
// columns TPR apart, so that the lanes of each element-wise access are neighbours.
template <int TPR, bool VEC, typename T>
__device__ __forceinline__ Raw8<T> fetch_cols(const T *row, int lt, int k, int64_t cols) {
  if constexpr (VEC) return fetch8<true>(row, 8 * int64_t(lt + k * TPR), cols);
  Raw8<T> r;
  r.zero();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t c = int64_t(8 * k + j) * TPR + lt;
    if (c < cols) r.set(j, row[c]);
  }
  return r;
}
template <int TPR, bool VEC, typename T>
__device__ __forceinline__ void put_cols(T *row, int lt, int k, int64_t cols, const float v[8]) {
  if constexpr (VEC) {
    put8<true>(row, 8 * int64_t(lt + k * TPR), cols, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = int64_t(8 * k + j) * TPR + lt;
      if (c < cols) store1(row + c, v[j]);
    }
  }
}

// Which of thread lt's elements of group k, in the places of fetch_cols, row r keeps: bit j.
// Without VEC a wave's 64 columns of each j are 8 of the generator's groups, and its lanes
// draw the 64 groups of all eight j once and hand the bits round.
template <int TPR, bool VEC>
__device__ __forceinline__ uint32_t kept_cols(const Mask &m, uint64_t row_group, int lt, int k) {
  if constexpr (VEC) return m.bits(row_group + uint64_t(lt + k * TPR));
  const int lane = lt & 63, first = lt & ~63;
  const uint32_t mine = m.bits(row_group + uint64_t(((8 * k + (lane >> 3)) * TPR + first) >> 3) + (lane & 7));
  uint32_t b = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) b |= ((uint32_t(__shfl(int(mine), 8 * j + (lane >> 3), 64)) >> (lane & 7)) & 1u) << j;
  return b;
}

// The gradient on rows that fit in registers, one pass: a persistent workgroup walks rows
// with the sums of dy * hhat for its columns in registers and writes them once, as a row
// of `partial`.  The next row's loads are issued before this row's sum is waited for.  HBM
// bounds it: 16384 x 5120 bf16 with dh, 671 MB, 142 us (4.7 TB/s) with 745 workgroups.
// 777 x 2501 fp32 takes 11 us (2.9 TB/s): 389 workgroups of two rows, one after the other,
// on 256 CUs.  bf16 rows that take no 16-byte accesses are written two bytes a lane:
// 16384 x 5117 706 us.  DROP: dx is dropped out and the residual's gradient written too, 839
// MB, 194 us (4.3 TB/s).
template <typename T, int TPR, int NCH, bool VEC, bool DROP>
__global__ __launch_bounds__(kThreads) void norm_grad_kernel(NormGradArgs<T> p) {
  __shared__ float part[2][4];
  constexpr int RPB = kThreads / TPR;
  const int lt = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t step = int64_t(gridDim.x) * RPB;
  float w[NCH][8], dw[NCH][8];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const Raw8<float> x = fetch_cols<TPR, VEC>(p.weight, lt, k, p.cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[k][j] = x.at(j);
      dw[k][j] = 0.0f;
    }
  }
  // the next row's h and dy are loaded while this row is worked on: with a barrier to a
  // row and two or three workgroups on a CU nothing else hides their latency
  Raw8<T> hn[NCH], yn[NCH];
  float rn = 0.0f;
  auto fetch = [&](int64_t r) {
    rn = p.rstd[r];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      hn[k] = fetch_cols<TPR, VEC>(p.h + r * p.cols, lt, k, p.cols);
      yn[k] = fetch_cols<TPR, VEC>(p.dy + r * p.cols, lt, k, p.cols);
    }
  };
  const Mask mask(p.drop);
  int64_t r = int64_t(blockIdx.x) * RPB + sub;
  if (r < p.rows) fetch(r);
  for (int odd = 0; r < p.rows; r += step, odd ^= 1) {
    Raw8<T> d[NCH];
    if (p.dh) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) d[k] = fetch_cols<TPR, VEC>(p.dh + r * p.cols, lt, k, p.cols);
    }
    const float rs = rn;
    float hh[NCH][8], v[NCH][8], s = 0.0f;
#pragma unroll
    for (int k = 0; k < NCH; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = yn[k].at(j);
        hh[k][j] = hn[k].at(j) * rs;
        dw[k][j] = __builtin_fmaf(y, hh[k][j], dw[k][j]);
        v[k][j] = y * w[k][j];
        s = __builtin_fmaf(v[k][j], hh[k][j], s);
      }
    if (r + step < p.rows) fetch(r + step);
    uint32_t kept[NCH];
    if constexpr (DROP) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) kept[k] = kept_cols<TPR, VEC>(mask, uint64_t(r) * drop_groups(p.cols), lt, k);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    if constexpr (TPR > 64) {
      // two slots in turn: a wave may write the next row's sum while another reads this one's
      if ((threadIdx.x & 63) == 0) part[odd][threadIdx.x >> 6] = s;
      __syncthreads();
      s = (part[odd][0] + part[odd][1]) + (part[odd][2] + part[odd][3]);
    }
    s = s / float(p.cols);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = __builtin_fmaf(rs, v[k][j] - hh[k][j] * s, p.dh ? d[k].at(j) : 0.0f);
      if constexpr (DROP) {
        put_cols<TPR, VEC>(p.dres + r * p.cols, lt, k, p.cols, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = dropped(o[j], kept[k], j, p.drop.gain);
      }
      put_cols<TPR, VEC>(p.dx + r * p.cols, lt, k, p.cols, o);
    }
  }
  float *out = p.partial + (int64_t(blockIdx.x) * RPB + sub) * p.cols;
#pragma unroll
  for (int k = 0; k < NCH; ++k) put_cols<TPR, VEC>(out, lt, k, p.cols, dw[k]);
}

// Rows too wide for registers: each row is read twice, and the sums of dy * hhat are
// left to norm_dw_kernel.
template <typename T, bool DROP>
__global__ __launch_bounds__(kThreads) void norm_grad_wide_kernel(NormGradArgs<T> p) {
  __shared__ float part[4];
  const int64_t r = blockIdx.x;
  const float rs = p.rstd[r];
  const T *hr = p.h + r * p.cols, *dyr = p.dy + r * p.cols;
  float s = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kThreads) {
    float hh[8], v[8], w[8];
    load8(hr, c, p.cols, p.vec, hh);
    load8(dyr, c, p.cols, p.vec, v);
    load8(p.weight, c, p.cols, p.vec, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fmaf(v[j] * w[j], hh[j] * rs, s);
  }
  s = row_sum<kThreads>(s, part) / float(p.cols);
  for (int64_t c = 8 * threadIdx.x; c < p.cols; c += 8 * kThreads) {
    float hh[8], v[8], w[8], d[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    load8(hr, c, p.cols, p.vec, hh);
    load8(dyr, c, p.cols, p.vec, v);
    load8(p.weight, c, p.cols, p.vec, w);
    if (p.dh) load8(p.dh + r * p.cols, c, p.cols, p.vec, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = __builtin_fmaf(rs, v[j] * w[j] - hh[j] * rs * s, d[j]);
    if constexpr (DROP) {
      store8(p.dres + r * p.cols, c, p.cols, p.vec, d);
      const uint32_t kept = Mask(p.drop).bits(uint64_t(r) * drop_groups(p.cols) + (c >> 3));
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = dropped(d[j], kept, j, p.drop.gain);
    }
    store8(p.dx + r * p.cols, c, p.cols, p.vec, d);
  }
}

// partial[b][c] = sum of dy * hhat over rows b, b + parts, ...; a thread owns a column.
// It runs before norm_grad_wide_kernel, which may overwrite dy.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dw_kernel(NormGradArgs<T> p, int parts) {
  const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= p.cols) return;
  float s = 0.0f;
  for (int64_t r = blockIdx.y; r < p.rows; r += parts)
    s = __builtin_fmaf(widen(p.dy[r * p.cols + c]), widen(p.h[r * p.cols + c]) * p.rstd[r], s);
  p.partial[int64_t(blockIdx.y) * p.cols + c] = s;
}

// dweight[c] = the partials' sum in binary64, in a fixed order: a workgroup takes 32
// columns, its 32 thread rows the partials t, t + 32, ..., and the first of them adds the
// 32 sums.  5.9 us after 16384 x 5120, 15 MB.  (64 columns and 4 thread rows, one load
// after another, took 38 us for 512 partials of 5120 columns.)
constexpr int kFinishRows = 32;
__global__ __launch_bounds__(32 * kFinishRows) void norm_dw_finish_kernel(const float *partial, int parts,
                                                                          int64_t cols, float *dweight) {
  __shared__ double sum[kFinishRows][32];
  const int x = threadIdx.x & 31, t = threadIdx.x >> 5;
  const int64_t c = int64_t(blockIdx.x) * 32 + x;
  double s = 0.0;
  if (c < cols) {
    int b = t;
    for (; b + 3 * kFinishRows < parts; b += 4 * kFinishRows) {
      const float v0 = partial[int64_t(b) * cols + c], v1 = partial[int64_t(b + kFinishRows) * cols + c];
      const float v2 = partial[int64_t(b + 2 * kFinishRows) * cols + c];
      const float v3 = partial[int64_t(b + 3 * kFinishRows) * cols + c];
      s += (double(v0) + double(v1)) + (double(v2) + double(v3));
    }
    for (; b < parts; b += kFinishRows) s += double(partial[int64_t(b) * cols + c]);
  }
  sum[t][x] = s;
  __syncthreads();
  if (t == 0 && c < cols) {
    for (int k = 1; k < kFinishRows; ++k) s += sum[k][x];
    dweight[c] = float(s);
  }
}

// ---------------------------------------------------------------------------
// Dropout with the residual's addition.  The mask is drawn where it is used: ten rounds of
// Philox give a thread the 16 bits of each of its 8 elements, some 560 cycles of a wave (its
// 32-bit products run at a quarter of the rate): 16384 x 5120 would take 43 us of them, and
// takes 86 us with the residual, bf16, for its 503 MB (5.8 TB/s).  8 x 5120 2.6 us: the launch.
template <typename T>
struct DropArgs {
  const T *x, *res;
  T *y;
  int64_t ldx, ldr, ldy, rows, cols;
  Drop drop;
};

// Rows that follow each other and whole groups of 8, 16-byte aligned: the tensor is one run
// of groups, and a group's place is its number in the generator.
template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_kernel(DropArgs<T> p, int64_t groups) {
  const Mask mask(p.drop);
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < groups; g += step) {
    Raw8<T> x, r;
    x.load(p.x + 8 * g);
    if constexpr (RES) r.load(p.res + 8 * g);
    const uint32_t kept = mask.bits(uint64_t(g));
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = dropped(x.at(j), kept, j, p.drop.gain);
      if constexpr (RES) v[j] += r.at(j);
    }
    store8_vec(p.y + 8 * g, v);
  }
}

// Any rows: a wave takes 512 columns of one, a lane draws one group of 8 and then handles
// column 64 j + lane for j = 0..7, so that an access's lanes are neighbours.  With the residual
// 16384 x 5117 fp32 187 us (5.4 TB/s), bf16 159 us (3.2 TB/s): a wave's access is 128 bytes.
template <typename T, bool RES>
__global__ __launch_bounds__(kThreads) void dropout_rows_kernel(DropArgs<T> p, int64_t chunks) {
  const Mask mask(p.drop);
  const int lane = threadIdx.x & 63;
  const int64_t waves = p.rows * chunks, step = int64_t(gridDim.x) * (kThreads / 64);
  for (int64_t w = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); w < waves; w += step) {
    const int64_t row = w / chunks, c0 = (w % chunks) * 512;
    const T *xr = p.x + row * p.ldx + c0 + lane, *rr = p.res + row * p.ldr + c0 + lane;
    T *yr = p.y + row * p.ldy + c0 + lane;
    const int left = int(p.cols - c0 < 512 ? p.cols - c0 : 512) - lane;  // column 64 j + lane is inside: 64 j < left
    T x[8] = {}, r[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (64 * j < left) {
        x[j] = xr[64 * j];
        if constexpr (RES) r[j] = rr[64 * j];
      }
    const uint32_t mine = mask.bits(uint64_t(row) * drop_groups(p.cols) + (c0 >> 3) + lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t kept = uint32_t(__shfl(int(mine), 8 * j + (lane >> 3), 64));
      float v = dropped(widen(x[j]), kept, lane & 7, p.drop.gain);
      if constexpr (RES) v += widen(r[j]);
      if (64 * j < left) store1(yr + 64 * j, v);
    }
  }
}

// ---------------------------------------------------------------------------
// The gated block's activation of binary32-sum products, which leave g and u in memory:
// hq = Q(silu(g) * u).  The quantizer's tiles, bound by the bytes as it is: 4096 x 20480,
// 422 MB, 78 us (5.4 TB/s).
__global__ __launch_bounds__(kThreads) void act_kernel(const uint16_t *g, const uint16_t *u, int64_t ld, int64_t rows,
                                                       int64_t cols, int64_t cblocks, int vec, Out h) {
  __shared__ TileLds lds;
  int64_t r0, c0;
  tile_pos(cblocks, r0, c0);
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  Raw8<uint16_t> a[8], b[8];
  tile_fetch(g, rows, cols, ld, vec, r0, c0, cg, rg, a);
  tile_fetch(u, rows, cols, ld, vec, r0, c0, cg, rg, b);
  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[p].at(j);
      v[p][j] = x * sigmoid(x) * b[p].at(j);
    }
  tile_quantize(v, h, Out{}, false, r0, c0, lds);
}

// The gated block's backward element-wise step on 128 x 128 tiles.
// Output W of a tile (dg, du or h, in its layouts).
template <int W>
__device__ __forceinline__ void dact_part(const Raw8<uint16_t> (&a)[8], const Raw8<uint16_t> (&b)[8],
                                          const Raw8<float> (&d)[8], const Out &q, const Out &qt, int64_t r0, int64_t c0,
                                          TileLds &lds) {
  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[p].at(j), y = b[p].at(j), s = sigmoid(x), silu = x * s;
      v[p][j] = W == 0 ? d[p].at(j) * y * dsilu(s, silu) : W == 1 ? d[p].at(j) * silu : silu * y;
    }
  tile_quantize(v, q, qt, false, r0, c0, lds);
}

// A workgroup writes all three outputs, or (gridDim.y = 3: few tiles) one of them.
// 4096 x 20480: 1.1 GB, 248 us (4.4 TB/s).
__global__ __launch_bounds__(kThreads, 2) void dact_kernel(const float *dh, int64_t ld, const uint16_t *g,
                                                           const uint16_t *u, int64_t rows, int64_t cols,
                                                           int64_t cblocks, int vec, int dh_vec, DactOut o) {
  __shared__ TileLds lds;
  int64_t r0, c0;
  tile_pos(cblocks, r0, c0);
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
  Raw8<uint16_t> a[8], b[8];
  Raw8<float> d[8];
  tile_fetch(g, rows, cols, cols, vec, r0, c0, cg, rg, a);
  tile_fetch(u, rows, cols, cols, vec, r0, c0, cg, rg, b);
  tile_fetch(dh, rows, cols, ld, dh_vec, r0, c0, cg, rg, d);
  const bool all = gridDim.y == 1;
  if (all || blockIdx.y == 0) dact_part<0>(a, b, d, o.dg, o.dg_t, r0, c0, lds);
  if (all) __syncthreads();
  if (all || blockIdx.y == 1) dact_part<1>(a, b, d, o.du, o.du_t, r0, c0, lds);
  if (all) __syncthreads();
  if (all || blockIdx.y == 2) dact_part<2>(a, b, d, Out{}, o.h_t, r0, c0, lds);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// whole groups of 8 elements are 16-byte aligned in every row
template <typename T>
bool vec_ok(const void *p, int64_t ld) {
  return aligned16(p) && (ld * int64_t(sizeof(T))) % 16 == 0;
}

template <typename T>
hipError_t quantize_t(const void *x, int64_t rows, int64_t cols, int64_t ld, const fp8_tensor *q, const fp8_tensor *qt,
                      hipStream_t stream) {
  const int64_t cb = ceil_div(cols, kBlock), tiles = cb * ceil_div(rows, kBlock);
  const bool two_d = (q ? q : qt)->two_d != 0;
  return launch(quantize_kernel<T>, dim3(unsigned(tiles)), dim3(kThreads), stream, static_cast<const T *>(x), rows,
                cols, ld, cb, int(vec_ok<T>(x, ld)), out_of(q), out_of(qt), int(two_d));
}

// w: the width with its padding (whose codes are written too)
template <typename T, bool VEC, bool DROP>
hipError_t launch_norm_rows(const NormArgs<T> &a, int64_t w, unsigned by1, unsigned by4, hipStream_t stream) {
  const dim3 blk(kThreads);
  if (w <= 512) return launch(norm_kernel<T, 64, 1, VEC, DROP>, dim3(by4), blk, stream, a);
  if (w <= 1024) return launch(norm_kernel<T, 64, 2, VEC, DROP>, dim3(by4), blk, stream, a);
  if (w <= 2048) return launch(norm_kernel<T, 256, 1, VEC, DROP>, dim3(by1), blk, stream, a);
  if (w <= 4096) return launch(norm_kernel<T, 256, 2, VEC, DROP>, dim3(by1), blk, stream, a);
  if (w <= 6144) return launch(norm_kernel<T, 256, 3, VEC, DROP>, dim3(by1), blk, stream, a);
  return launch(norm_kernel<T, 256, 4, VEC, DROP>, dim3(by1), blk, stream, a);
}

template <typename T, bool DROP>
hipError_t norm_t(const void *x, int64_t ldx, const void *res, int64_t ldr, int64_t rows, int64_t cols,
                  const float *weight, float eps, void *h, int64_t ldh, const fp8_tensor *yq, const fp8_tensor *yq_t,
                  float *rstd, const Drop &drop, hipStream_t stream) {
  NormArgs<T> a{static_cast<const T *>(x), static_cast<const T *>(res), static_cast<T *>(h), ldx, ldr, ldh, rows, cols,
                weight, eps, rstd, out_of(yq), 0, drop};
  a.vec = vec_ok<T>(x, ldx) && (!res || (vec_ok<T>(res, ldr) && vec_ok<T>(h, ldh))) && aligned16(weight);
  const dim3 blk(kThreads);
  const unsigned by4 = unsigned(ceil_div(rows, 4)), by1 = unsigned(rows);
  const int64_t w = padded_cols(cols);
  hipError_t e;
  if (w > 8192) e = launch(norm_wide_kernel<T, DROP>, dim3(by1), blk, stream, a);
  else if (a.vec && cols % 8 == 0) e = launch_norm_rows<T, true, DROP>(a, w, by1, by4, stream);
  else e = launch_norm_rows<T, false, DROP>(a, w, by1, by4, stream);
  if (e != hipSuccess || !yq_t) return e;
  const T *src = res ? static_cast<const T *>(h) : static_cast<const T *>(x);
  const int64_t ld = res ? ldh : ldx, cb = ceil_div(cols, kBlock);
  return launch(norm_cols_kernel<T>, dim3(unsigned(cb * ceil_div(rows, kBlock))), blk, stream, src, ld, rows, cols,
                weight, rstd, cb, int(vec_ok<T>(src, ld) && aligned16(weight)), out_of(yq_t));
}

template <typename T>
hipError_t dropout_t(const void *x, int64_t ldx, const void *res, int64_t ldr, int64_t rows, int64_t cols,
                     const Drop &drop, void *y, int64_t ldy, hipStream_t stream) {
  const DropArgs<T> a{static_cast<const T *>(x), static_cast<const T *>(res), static_cast<T *>(y),
                      ldx, ldr, ldy, rows, cols, drop};
  const dim3 blk(kThreads);
  constexpr int64_t kMost = 1 << 20;  // workgroups; they walk what is left
  auto grid = [&](int64_t n) { return dim3(unsigned(n < kMost ? n : kMost)); };
  const bool run = ((rows == 1) || (ldx == cols && ldy == cols && (!res || ldr == cols))) && cols % 8 == 0 &&
                   aligned16(x) && aligned16(y) && (!res || aligned16(res));
  if (run) {
    const int64_t groups = rows * (cols / 8);
    return res ? launch(dropout_kernel<T, true>, grid(ceil_div(groups, kThreads)), blk, stream, a, groups)
               : launch(dropout_kernel<T, false>, grid(ceil_div(groups, kThreads)), blk, stream, a, groups);
  }
  const int64_t chunks = ceil_div(cols, 512), wgs = ceil_div(rows * chunks, kThreads / 64);
  return res ? launch(dropout_rows_kernel<T, true>, grid(wgs), blk, stream, a, chunks)
             : launch(dropout_rows_kernel<T, false>, grid(wgs), blk, stream, a, chunks);
}

constexpr int64_t kNormGradMaxCols = 8192;  // wider rows take the wide kernels
constexpr int64_t kNormGradBlocks = 768;
constexpr int64_t kNormDwParts = 64;

int64_t norm_grad_rows_per_block(int64_t cols) { return cols <= 1024 ? 4 : 1; }

int64_t norm_grad_blocks(int64_t rows, int64_t cols) {
  const int64_t n = ceil_div(rows, norm_grad_rows_per_block(cols));
  return n > 0 ? ceil_div(n, ceil_div(n, kNormGradBlocks)) : 0;  // as few as give the same most rows to one
}

int64_t norm_grad_parts(int64_t rows, int64_t cols) {
  if (cols > kNormGradMaxCols) return rows < kNormDwParts ? rows : kNormDwParts;
  return norm_grad_blocks(rows, cols) * norm_grad_rows_per_block(cols);
}

template <typename T, bool VEC, bool DROP>
hipError_t launch_norm_grad_rows(const NormGradArgs<T> &a, unsigned blocks, hipStream_t stream) {
  const dim3 grid(blocks), blk(kThreads);
  if (a.cols <= 512) return launch(norm_grad_kernel<T, 64, 1, VEC, DROP>, grid, blk, stream, a);
  if (a.cols <= 1024) return launch(norm_grad_kernel<T, 64, 2, VEC, DROP>, grid, blk, stream, a);
  if (a.cols <= 2048) return launch(norm_grad_kernel<T, 256, 1, VEC, DROP>, grid, blk, stream, a);
  if (a.cols <= 4096) return launch(norm_grad_kernel<T, 256, 2, VEC, DROP>, grid, blk, stream, a);
  if (a.cols <= 6144) return launch(norm_grad_kernel<T, 256, 3, VEC, DROP>, grid, blk, stream, a);
  return launch(norm_grad_kernel<T, 256, 4, VEC, DROP>, grid, blk, stream, a);
}

template <typename T, bool DROP>
hipError_t norm_grad_t(const void *dy, const void *h, const void *dh, int64_t rows, int64_t cols, const float *weight,
                       const float *rstd, void *dx, void *dres, float *dweight, float *ws, const Drop &drop,
                       hipStream_t stream) {
  NormGradArgs<T> a{static_cast<const T *>(dy), static_cast<const T *>(h), static_cast<const T *>(dh),
                    static_cast<T *>(dx), rows, cols, weight, rstd, ws, 0, static_cast<T *>(dres), drop};
  a.vec = vec_ok<T>(dy, cols) && vec_ok<T>(h, cols) && (!dh || vec_ok<T>(dh, cols)) && vec_ok<T>(dx, cols) &&
          (!DROP || vec_ok<T>(dres, cols)) && aligned16(weight);
  const dim3 blk(kThreads);
  const int parts = int(norm_grad_parts(rows, cols));
  hipError_t e = hipSuccess;
  if (rows > 0) {
    if (cols > kNormGradMaxCols) {
      e = launch(norm_dw_kernel<T>, dim3(unsigned(ceil_div(cols, kThreads)), unsigned(parts)), blk, stream, a, parts);
      if (e == hipSuccess) e = launch(norm_grad_wide_kernel<T, DROP>, dim3(unsigned(rows)), blk, stream, a);
    } else {
      const unsigned blocks = unsigned(norm_grad_blocks(rows, cols));
      e = a.vec && cols % 8 == 0 ? launch_norm_grad_rows<T, true, DROP>(a, blocks, stream)
                                 : launch_norm_grad_rows<T, false, DROP>(a, blocks, stream);
    }
    if (e != hipSuccess) return e;
  }
  return launch(norm_dw_finish_kernel, dim3(unsigned(ceil_div(cols, 32))), dim3(32 * kFinishRows), stream, ws, parts,
                cols, dweight);
}

}  // namespace

hipError_t launch_quantize(const void *x, fp4_dtype dtype, int64_t rows, int64_t cols, int64_t ld, const fp8_tensor *q,
                           const fp8_tensor *q_t, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  return dtype == FP4_BF16 ? quantize_t<uint16_t>(x, rows, cols, ld, q, q_t, stream)
                           : quantize_t<float>(x, rows, cols, ld, q, q_t, stream);
}

hipError_t launch_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                           int64_t rows, int64_t cols, const float *weight, float eps, void *h, int64_t ldh,
                           const fp8_tensor *yq, const fp8_tensor *yq_t, float *rstd, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  return dtype == FP4_BF16
             ? norm_t<uint16_t, false>(x, ldx, residual, ldr, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd, Drop{}, stream)
             : norm_t<float, false>(x, ldx, residual, ldr, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd, Drop{}, stream);
}

hipError_t launch_dropout_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                                   int64_t rows, int64_t cols, const Drop &drop, const float *weight, float eps,
                                   void *h, int64_t ldh, const fp8_tensor *yq, const fp8_tensor *yq_t, float *rstd,
                                   hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  return dtype == FP4_BF16
             ? norm_t<uint16_t, true>(x, ldx, residual, ldr, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd, drop, stream)
             : norm_t<float, true>(x, ldx, residual, ldr, rows, cols, weight, eps, h, ldh, yq, yq_t, rstd, drop, stream);
}

size_t rms_norm_ws_bytes(int64_t rows, int64_t cols) {
  return size_t(norm_grad_parts(rows, cols)) * size_t(cols) * sizeof(float);
}

hipError_t launch_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                                    int64_t cols, const float *weight, const float *rstd, void *dx, float *dweight,
                                    float *ws, hipStream_t stream) {
  if (cols == 0) return hipSuccess;
  return dtype == FP4_BF16
             ? norm_grad_t<uint16_t, false>(dy, h, dh, rows, cols, weight, rstd, dx, nullptr, dweight, ws, Drop{}, stream)
             : norm_grad_t<float, false>(dy, h, dh, rows, cols, weight, rstd, dx, nullptr, dweight, ws, Drop{}, stream);
}

hipError_t launch_dropout_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype,
                                            int64_t rows, int64_t cols, const Drop &drop, const float *weight,
                                            const float *rstd, void *dx, void *dresidual, float *dweight, float *ws,
                                            hipStream_t stream) {
  if (cols == 0) return hipSuccess;
  return dtype == FP4_BF16
             ? norm_grad_t<uint16_t, true>(dy, h, dh, rows, cols, weight, rstd, dx, dresidual, dweight, ws, drop, stream)
             : norm_grad_t<float, true>(dy, h, dh, rows, cols, weight, rstd, dx, dresidual, dweight, ws, drop, stream);
}

hipError_t launch_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype, int64_t rows,
                          int64_t cols, const Drop &drop, void *y, int64_t ldy, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  return dtype == FP4_BF16 ? dropout_t<uint16_t>(x, ldx, residual, ldr, rows, cols, drop, y, ldy, stream)
                           : dropout_t<float>(x, ldx, residual, ldr, rows, cols, drop, y, ldy, stream);
}

hipError_t launch_act_quantize(const uint16_t *g, const uint16_t *u, int64_t ld, const fp8_tensor *hq,
                               hipStream_t stream) {
  const int64_t rows = hq->rows, cols = hq->cols, cb = ceil_div(cols, kBlock), tiles = cb * ceil_div(rows, kBlock);
  if (tiles == 0) return hipSuccess;
  return launch(act_kernel, dim3(unsigned(tiles)), dim3(kThreads), stream, g, u, ld, rows, cols, cb,
                int(vec_ok<uint16_t>(g, ld) && vec_ok<uint16_t>(u, ld)), out_of(hq));
}

hipError_t launch_dact_quantize(const float *dh, int64_t ld, const uint16_t *g, const uint16_t *u,
                                const fp8_ffn_buffers *b, hipStream_t stream) {
  const int64_t rows = b->dgq.rows, cols = b->dgq.cols;
  const int64_t cb = ceil_div(cols, kBlock), tiles = cb * ceil_div(rows, kBlock);
  if (tiles == 0) return hipSuccess;
  const int vec = vec_ok<uint16_t>(g, cols) && vec_ok<uint16_t>(u, cols), dh_vec = vec_ok<float>(dh, ld);
  const DactOut o = dact_out(b);
  // 125 tiles: 22 us with a workgroup per output, 24 with one for all three
  return launch(dact_kernel, dim3(unsigned(tiles), tiles < 512 ? 3u : 1u), dim3(kThreads), stream, dh, ld, g, u, rows,
                cols, cb, vec, dh_vec, o);
}

}  // namespace fp8
}  // namespace nvfp4
