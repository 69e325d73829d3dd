// fp8_lora.hip -- low-rank adapters beside a projection: the kernels next to the product
// itself (fp8_gemm.hip adds the adapters' part where it stores its results).
//
//   forward   down_kernel   t = dropout(x) a_i^T             [M][rank], binary32
//             product       y = x W^T + c_i t b_i^T          c_i = scale_i times dropout's gain
//   backward  order_kernel  the tokens in the order of their adapters; a and b transposed
//             down_kernel   t again and dt = dy b_i
//             product       dx = dy W + c_i dropout mask (dt a_i)
//             outer_kernel  dt^T dropout(x) and dy^T t, summed over runs of tokens
//             join_kernel   da and db: c_i times the runs' sums
// t is a fraction rank / N of what the product reads and writes, so recomputing it costs the
// backward pass one read of x's codes and the forward pass nothing to keep.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8.hpp"

namespace nvfp4 {
namespace fp8 {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;  // of a step of outer_kernel

// The rows that a kernel here reads: E4M3 with one scale per 1 x 128 block.
struct Source {
  const uint8_t *codes, *scales;
  int64_t ld, srow, cols;
  int blocks;
  Drop drop;  // of its values
};

Source source_of(const fp8_tensor *t, const Drop &drop) {
  return Source{t->codes, t->scales, padded_cols(t->cols), scale_row(t->rows, false), t->cols,
                int(ceil_div(t->cols, kBlock)), drop};
}

// The adapter of token m, -1 for none.
__device__ __forceinline__ int adapter_of(const int32_t *index, int64_t m, int count) {
  const int i = index ? index[m] : 0;
  return i < count ? i : -1;
}

// ANDed with a group's 8 codes: a dropped element's byte becomes 0.
__device__ __forceinline__ uint2 code_mask(uint32_t bits) {
  // bit j of a nibble to the low bit of byte j, times 255
  const uint32_t lo = ((bits & 0xFu) * 0x00204081u) & 0x01010101u, hi = ((bits >> 4) * 0x00204081u) & 0x01010101u;
  return make_uint2(lo * 0xFFu, hi * 0xFFu);
}

// ---------------------------------------------------------------------------
// t[m] = v[m] a_i^T: a workgroup takes 16 rows, one part of the contraction and, in turn,
// the adapters of its rows that fall to its slot; its four waves take blocks of 128 in turn
// and join their sums.  A lane holds 32 neighbouring values of a row and the 64 bytes of a
// that they meet, so operands come from memory as the matrix instruction wants them (any
// assignment of the contraction to lane groups will do) and nothing passes through LDS but
// the sums.  Rows with another adapter, or none, are left as they are: nothing reads them.
struct DownSide {
  Source v;
  const uint16_t *a;  // [count][rank][lda]
  int64_t lda;
  float *t;  // [parts][M][rank]
  int parts;
};

struct DownArgs {
  DownSide side[2];
  int first;  // workgroups of side 0
  int slots;
  int64_t M;
  const int32_t *index;
  int count, rank;
};

// NR tiles of 16 of the rank
template <int NR>
__global__ __launch_bounds__(kThreads) void down_kernel(DownArgs p) {
  __shared__ __attribute__((aligned(16))) float sums[4][16][16 * NR];
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const bool second = int(blockIdx.x) >= p.first;
  const DownSide &side = p.side[second ? 1 : 0];
  const Source &v = side.v;
  int wg = int(blockIdx.x) - (second ? p.first : 0);
  const int part = __builtin_amdgcn_readfirstlane(wg % side.parts);
  wg = __builtin_amdgcn_readfirstlane(wg / side.parts);
  const int slot = __builtin_amdgcn_readfirstlane(wg % p.slots);
  const int64_t m0 = int64_t(__builtin_amdgcn_readfirstlane(wg / p.slots)) * 16;
  const int64_t m = m0 + lr, row = m < p.M ? m : p.M - 1;
  const int idx = m < p.M ? adapter_of(p.index, m, p.count) : -1;
  const int b_begin = int(int64_t(v.blocks) * part / side.parts), b_end = int(int64_t(v.blocks) * (part + 1) / side.parts);
  const Mask mask(v.drop);
  const uint64_t row_group = uint64_t(row) * uint64_t((v.cols + 7) >> 3);

  bool pending = idx >= 0;
  for (int turn = 0;; ++turn) {
    const uint64_t some = __ballot(pending);
    if (some == 0) return;  // the same for every wave: all hold the tile's rows
    const int cur = __builtin_amdgcn_readlane(idx, __builtin_ctzll(some));
    pending = pending && idx != cur;
    if (turn % p.slots != slot) continue;

    f32x4 acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t *a_row[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {  // past the rank: some row, whose sums are not stored
      const int r = 16 * n + lr < p.rank ? 16 * n + lr : 0;
      a_row[n] = side.a + (int64_t(cur) * p.rank + r) * side.lda;
    }
    for (int b = b_begin + wave; b < b_end; b += 4) {
      const int64_t k = int64_t(b) * kBlock + 32 * lg;
      const uint4 *src = reinterpret_cast<const uint4 *>(v.codes + row * v.ld + k);
      const uint4 x = src[0], y = src[1];
      const uint32_t sb = v.scales[int64_t(b) * v.srow + row];
      bf16x8 fa[NR][4];
      if (int64_t(b + 1) * kBlock <= v.cols) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) fa[n][q] = *reinterpret_cast<const bf16x8 *>(a_row[n] + k + 8 * q);
      } else {  // lda is a multiple of 8: a group is readable where it begins inside
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            bf16x8 w = bf16x8{};
            if (k + 8 * q < v.cols) w = *reinterpret_cast<const bf16x8 *>(a_row[n] + k + 8 * q);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = k + 8 * q + j < v.cols ? w[j] : __bf16(0.0f);
            fa[n][q] = w;
          }
      }
      i32x8 codes{int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
      if (mask.thr) {
        static_for<4>([&](auto qc) {
          constexpr int q = decltype(qc)::value;
          const uint2 keep = code_mask(mask.bits(row_group + uint64_t((k >> 3) + q)));
          codes[2 * q] &= int(keep.x);
          codes[2 * q + 1] &= int(keep.y);
        });
      }
      const float scale = scale_of(sb);
      static_for<4>([&](auto qc) {
        constexpr int q = decltype(qc)::value;
        const bf16x8 fv = widen8<q>(codes, scale);
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[n][q], fv, acc[n], 0, 0, 0);
      });
    }
    // lane (lr, lg): row lr's products with a's rows 16 n + 4 lg + 0..3
#pragma unroll
    for (int n = 0; n < NR; ++n)
      *reinterpret_cast<float4 *>(&sums[wave][lr][16 * n + 4 * lg]) = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    __syncthreads();
    for (int e = t; e < 16 * (p.rank / 4); e += kThreads) {
      const int tok = e & 15, r = 4 * (e >> 4);
      const int64_t mt = m0 + tok;
      if (mt >= p.M || adapter_of(p.index, mt, p.count) != cur) continue;
      float4 s = *reinterpret_cast<const float4 *>(&sums[0][tok][r]);
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float4 o = *reinterpret_cast<const float4 *>(&sums[w][tok][r]);
        s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
      }
      *reinterpret_cast<float4 *>(side.t + (int64_t(part) * p.M + mt) * p.rank + r) = s;
    }
    __syncthreads();  // the sums have been read
  }
}

// ---------------------------------------------------------------------------
// Before the backward pass's products.  Workgroups 0 .. count - 1: adapter i's tokens in
// their order, perm[start[i]] .. perm[start[i + 1] - 1], where start[i] counts the tokens of
// the adapters before it; each thread takes a run of tokens and a scan places its finds.  The
// others transpose: a [rank][lda] to at [K][rank] and b [N][rank] to bt [rank][ldb], zeros
// from N on, 64 rows or columns each.
struct OrderArgs {
  const int32_t *index;
  int64_t M;
  int count, rank;
  int32_t *perm, *start;
  const uint16_t *a, *b;
  int64_t K, N, lda, ldb;
  uint16_t *at, *bt;
  int a_tiles, b_tiles;  // of 64, to an adapter
};

__global__ __launch_bounds__(kThreads) void order_kernel(OrderArgs p) {
  __shared__ int32_t scan[2][kThreads];
  __shared__ uint16_t tile[128][65];
  const int t = threadIdx.x;
  if (int(blockIdx.x) < p.count) {
    const int me = blockIdx.x;
    const int64_t run = (p.M + kThreads - 1) / kThreads, first = t * run, last = first + run < p.M ? first + run : p.M;
    int mine = 0, before = 0;
    for (int64_t m = first; m < last; ++m) {
      const int i = adapter_of(p.index, m, p.count);
      mine += i == me;
      before += i >= 0 && i < me;
    }
    scan[0][t] = mine;
    scan[1][t] = before;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
      const int x = t >= o ? scan[0][t - o] : 0, y = t >= o ? scan[1][t - o] : 0;
      __syncthreads();
      scan[0][t] += x;
      scan[1][t] += y;
      __syncthreads();
    }
    const int base = scan[1][kThreads - 1];
    int at = base + scan[0][t] - mine;
    for (int64_t m = first; m < last; ++m)
      if (adapter_of(p.index, m, p.count) == me) p.perm[at++] = int32_t(m);
    if (t == 0) p.start[me] = base;
    if (t == 0 && me == p.count - 1) p.start[p.count] = base + scan[0][kThreads - 1];
    return;
  }
  int w = int(blockIdx.x) - p.count;
  const bool of_b = w >= p.count * p.a_tiles;
  if (of_b) w -= p.count * p.a_tiles;
  const int tiles = of_b ? p.b_tiles : p.a_tiles;
  const int64_t i = w / tiles, c0 = int64_t(w % tiles) * 64;
  if (!of_b) {
    const uint16_t *src = p.a + i * p.rank * p.lda;
    for (int e = t; e < p.rank * 64; e += kThreads) {
      const int r = e >> 6, c = e & 63;
      if (c0 + c < p.K) tile[r][c] = src[r * p.lda + c0 + c];
    }
    __syncthreads();
    uint16_t *dst = p.at + (i * p.K + c0) * p.rank;
    for (int e = t; e < p.rank * 64; e += kThreads) {
      const int c = e / p.rank, r = e % p.rank;
      if (c0 + c < p.K) dst[e] = tile[r][c];
    }
  } else {
    const uint16_t *src = p.b + (i * p.N + c0) * p.rank;
    for (int e = t; e < p.rank * 64; e += kThreads) {
      const int c = e / p.rank, r = e % p.rank;
      tile[r][c] = c0 + c < p.N ? src[e] : uint16_t(0);
    }
    __syncthreads();
    uint16_t *dst = p.bt + i * p.rank * p.ldb;
    for (int e = t; e < p.rank * 64; e += kThreads) {
      const int r = e >> 6, c = e & 63;
      if (c0 + c < p.ldb) dst[r * p.ldb + c0 + c] = tile[r][c];
    }
  }
}

// ---------------------------------------------------------------------------
// sum over tokens of coef[m]^T v[m] for 128 columns of v, over a run of `chunk` of the
// ordered tokens, one sum for every adapter that has some of them.  The contraction runs over
// tokens, so both operands are wanted transposed: v's codes as they are and the coefficients
// as three bf16 each (a binary32 whole) lie in LDS by tokens, and gfx950's transposing LDS
// reads hand a lane 8 tokens of a column.  A block's scale multiplies its token's coefficient.
struct OuterSide {
  Source v;
  const float *coef;  // [parts][M][rank]
  int parts;
  float *out;  // [piece][rank][128 blocks], or with by_col [piece][128 blocks][rank]
  int by_col;
};

struct OuterArgs {
  OuterSide side[2];
  int64_t M;
  int64_t chunk;
  const int32_t *index, *perm, *start;
  int count, rank;
};

// Adapters before `a` that have tokens: the pieces of chunk c are c + that, one more at each
// step to the next chunk or adapter.
__device__ __forceinline__ int used_before(const int32_t *start, int a) {
  int n = 0;
  for (int i = int(threadIdx.x & 63); i < a; i += 64) n += start[i + 1] > start[i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
  return __builtin_amdgcn_readfirstlane(n);
}

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

template <int NR>
__global__ __launch_bounds__(kThreads) void outer_kernel(OuterArgs p) {
  // 16 bytes of padding: the 32 rows of 16 bytes that one transposing read of a wave takes
  // cover the banks evenly
  constexpr int kRow = kBlock + 16;
  constexpr int RP = 16 * NR;
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTokens * kRow];
  __shared__ __attribute__((aligned(16))) uint16_t coefs[3][kTokens][RP];
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const bool second = int(blockIdx.x) >= p.side[0].v.blocks;
  const OuterSide &side = p.side[second ? 1 : 0];
  const Source &v = side.v;
  const int blk = int(blockIdx.x) - (second ? p.side[0].v.blocks : 0);
  const int64_t c0 = int64_t(blk) * kBlock;
  const int64_t total = p.start[p.count], first = int64_t(blockIdx.y) * p.chunk;
  if (first >= total) return;
  const int64_t last = first + p.chunk < total ? first + p.chunk : total;
  const Mask mask(v.drop);
  const int64_t groups = (v.cols + 7) >> 3;

  int a = __builtin_amdgcn_readfirstlane(adapter_of(p.index, p.perm[first], p.count));
  int piece = int(blockIdx.y) + used_before(p.start, a);
  for (int64_t at = first; at < last; ++a) {
    const int64_t stop = p.start[a + 1] < last ? p.start[a + 1] : last;
    if (stop <= at) continue;  // no token
    f32x4 acc[2][NR];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < NR; ++n) acc[f][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (; at < stop; at += kTokens) {
      // a thread takes 32 codes of a token and, of its coefficients, every fourth four
      const int tok = t >> 2, quarter = t & 3;
      const bool live = at + tok < stop;
      const int64_t m = live ? p.perm[at + tok] : 0;
      uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
      float scale = 0.0f;
      if (live) {
        const uint4 *src = reinterpret_cast<const uint4 *>(v.codes + m * v.ld + c0 + 32 * quarter);
        x = src[0];
        y = src[1];
        scale = scale_of(v.scales[int64_t(blk) * v.srow + m]);
      }
      float4 cf[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int r = 16 * n + 4 * quarter;
        cf[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!live || r >= p.rank) continue;
        const float *src = side.coef + m * p.rank + r;
        for (int s = 0; s < side.parts; ++s) {
          const float4 o = *reinterpret_cast<const float4 *>(src + int64_t(s) * p.M * p.rank);
          cf[n].x += o.x; cf[n].y += o.y; cf[n].z += o.z; cf[n].w += o.w;
        }
      }
      if (mask.thr) {
        const uint64_t g = uint64_t(m) * uint64_t(groups) + uint64_t((c0 >> 3) + 4 * quarter);
        const uint2 k0 = code_mask(mask.bits(g)), k1 = code_mask(mask.bits(g + 1));
        const uint2 k2 = code_mask(mask.bits(g + 2)), k3 = code_mask(mask.bits(g + 3));
        x.x &= k0.x; x.y &= k0.y; x.z &= k1.x; x.w &= k1.y;
        y.x &= k2.x; y.y &= k2.y; y.z &= k3.x; y.w &= k3.y;
      }
      __syncthreads();  // the last step's operands have been read
      *reinterpret_cast<uint4 *>(codes + tok * kRow + 32 * quarter) = x;
      *reinterpret_cast<uint4 *>(codes + tok * kRow + 32 * quarter + 16) = y;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float f[4] = {cf[n].x * scale, cf[n].y * scale, cf[n].z * scale, cf[n].w * scale};
        s16x4 w[3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float left = f[j];
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            const __bf16 h = static_cast<__bf16>(left);
            w[s][j] = __builtin_bit_cast(short, h);
            left -= static_cast<float>(h);
          }
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) *reinterpret_cast<s16x4 *>(&coefs[s][tok][16 * n + 4 * quarter]) = w[s];
      }
      __syncthreads();
      // the lane's place in a transposing read: 8 tokens of 16 codes, 4 tokens of 16 bf16
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k8 = 32 * half + 8 * lg;
        bf16x8 fv[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint8_t *from = codes + (k8 + (lr >> 1)) * kRow + 32 * wave + 16 * f + 8 * (lr & 1);
          const i32x2 c = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2 *)const_cast<uint8_t *>(from));
          fv[f] = widen8<0>(i32x8{c[0], c[1], 0, 0, 0, 0, 0, 0}, 1.0f);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            s16x8 w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint16_t *from = &coefs[s][k8 + 4 * h + (lr >> 2)][16 * n + 4 * (lr & 3)];
              const s16x4 c = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(from));
#pragma unroll
              for (int j = 0; j < 4; ++j) w[4 * h + j] = c[j];
            }
            const bf16x8 fc = __builtin_bit_cast(bf16x8, w);
#pragma unroll
            for (int f = 0; f < 2; ++f) acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fc, fv[f], acc[f][n], 0, 0, 0);
          }
      }
    }
    at = stop;
    // lane (lr, lg): column lr of its tile f, a's rows or b's columns 16 n + 4 lg + 0..3
    const int64_t wide = int64_t(v.blocks) * kBlock;
    float *out = side.out + int64_t(piece) * wide * p.rank;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int r = 16 * n + 4 * lg;
        const int64_t c = c0 + 32 * wave + 16 * f + lr;
        if (r >= p.rank) continue;
        if (side.by_col) {
          *reinterpret_cast<float4 *>(out + c * p.rank + r) =
              make_float4(acc[f][n][0], acc[f][n][1], acc[f][n][2], acc[f][n][3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) out[(r + j) * wide + c] = acc[f][n][j];
        }
      }
    ++piece;
  }
}

// da [count][rank][lda] and db [count][N][rank] from the pieces in their order; an adapter
// without tokens, and da's padding, take zeros.  Four elements to a thread.
struct JoinArgs {
  const float *pa, *pb;  // the pieces of either
  float *da, *db;
  int64_t K, N, lda, wide_a, wide_b, chunk;
  const float *scale;
  float gain;
  const int32_t *start;
  int rank;
  int a_wgs, wgs;  // workgroups of an adapter: da's, both
};

__global__ __launch_bounds__(kThreads) void join_kernel(JoinArgs p) {
  const int a = int(blockIdx.x) / p.wgs, w = int(blockIdx.x) % p.wgs;
  const bool of_b = w >= p.a_wgs;
  const int64_t e = 4 * (int64_t(w - (of_b ? p.a_wgs : 0)) * kThreads + threadIdx.x);
  const int64_t size = p.rank * (of_b ? p.N : p.lda);
  const int64_t begin = p.start[a], end = p.start[a + 1];
  const int64_t used = used_before(p.start, a);
  if (e >= size) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t k = of_b ? -1 : e % p.lda;
  if (end > begin && k < p.K) {  // lda may pass the pieces' rows
    const float *src = of_b ? p.pb + e : p.pa + (e / p.lda) * p.wide_a + k;
    const int64_t piece = p.rank * (of_b ? p.wide_b : p.wide_a);
    for (int64_t c = begin / p.chunk; c <= (end - 1) / p.chunk; ++c) {
      const float4 o = *reinterpret_cast<const float4 *>(src + (c + used) * piece);
      v[0] += o.x; v[1] += o.y; v[2] += o.z; v[3] += o.w;
    }
    const float f = p.scale[a] * p.gain;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = k + j < p.K || of_b ? v[j] * f : 0.0f;
  }
  float *dst = of_b ? p.db + a * size + e : p.da + a * size + e;
  *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------------------

// How the contraction over `blocks` blocks of 128 is split and how many workgroups share a
// tile's adapters: enough workgroups to fill the card, at least four blocks (one to a wave)
// to a part.
struct DownPlan {
  int parts, slots;
};
DownPlan down_plan(int64_t M, int64_t blocks, int count) {
  const int64_t tiles = ceil_div(M, 16);
  int64_t slots = 64 / tiles;
  slots = slots < 1 ? 1 : slots > 16 ? 16 : slots;
  if (slots > count) slots = count;
  if (slots > M) slots = M;
  int64_t parts = ceil_div(2 * cu_count(), tiles * slots);
  const int64_t most = ceil_div(blocks, 4) < 16 ? ceil_div(blocks, 4) : 16;
  parts = parts < most ? parts : most;
  return DownPlan{int(parts < 1 ? 1 : parts), int(slots)};
}

// Tokens of a run of outer_kernel: four workgroups to a CU where there are tokens enough.
int64_t outer_chunk(int64_t M, int64_t blocks) {
  const int64_t want = ceil_div(4 * cu_count(), blocks);
  const int64_t c = ceil_div(ceil_div(M, want), kTokens) * kTokens;
  return c < kTokens ? kTokens : c;
}

hipError_t launch_down(const DownArgs &a, int64_t wgs, hipStream_t stream) {
  const dim3 grid{unsigned(wgs)}, blk{kThreads};
  if (a.rank <= 16) return launch(down_kernel<1>, grid, blk, stream, a);
  if (a.rank <= 32) return launch(down_kernel<2>, grid, blk, stream, a);
  if (a.rank <= 64) return launch(down_kernel<4>, grid, blk, stream, a);
  return launch(down_kernel<8>, grid, blk, stream, a);
}

hipError_t launch_outer(const OuterArgs &a, dim3 grid, hipStream_t stream) {
  const dim3 blk{kThreads};
  if (a.rank <= 16) return launch(outer_kernel<1>, grid, blk, stream, a);
  if (a.rank <= 32) return launch(outer_kernel<2>, grid, blk, stream, a);
  if (a.rank <= 64) return launch(outer_kernel<4>, grid, blk, stream, a);
  return launch(outer_kernel<8>, grid, blk, stream, a);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// The backward pass's workspace, in bytes from its beginning.
struct BackwardPlan {
  DownPlan x, dy;
  int64_t chunk, chunks, pieces, ldb;
  size_t t, dt, perm, start, at, bt, rest, rest_bytes;
};
BackwardPlan backward_plan(int64_t M, int64_t N, int64_t K, int rank, int64_t count, bool fast) {
  BackwardPlan p{};
  const int64_t kb = ceil_div(K, kBlock), nb = ceil_div(N, kBlock);
  p.x = down_plan(M, kb, int(count));
  p.dy = down_plan(M, nb, int(count));
  p.chunk = outer_chunk(M, kb + nb);
  p.chunks = ceil_div(M, p.chunk);
  p.pieces = p.chunks + (count < M ? count : M) - 1;
  p.ldb = ceil_div(N, 8) * 8;
  size_t n = 0;
  auto place = [&](size_t bytes) {
    const size_t at = n;
    n += up16(bytes);
    return at;
  };
  p.t = place(size_t(p.x.parts) * M * rank * 4);
  p.dt = place(size_t(p.dy.parts) * M * rank * 4);
  p.perm = place(size_t(M) * 4);
  p.start = place(size_t(count + 1) * 4);
  p.at = place(size_t(count) * K * rank * 2);
  p.bt = place(size_t(count) * rank * p.ldb * 2);
  p.rest = n;  // the product's partials, and after it the sums' pieces
  const size_t gemm = gemm_ws_bytes(M, K, nb, fast), outer = size_t(p.pieces) * size_t(kb + nb) * kBlock * rank * 4;
  p.rest_bytes = up16(gemm > outer ? gemm : outer);
  return p;
}

}  // namespace

size_t lora_fprop_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, bool fast) {
  if (M == 0 || N == 0) return 0;
  const int64_t kb = ceil_div(K, kBlock);
  // the most parts are those of one adapter to a tile
  return up16(size_t(down_plan(M, kb, 1).parts) * M * rank * 4) + gemm_ws_bytes(M, N, kb, fast);
}

hipError_t launch_lora_fprop(const fp8_tensor *xq, const fp8_tensor *wq, const fp8_lora *lora, const int32_t *index,
                             const Drop &drop, void *y, int64_t ldy, bool fast, void *ws, size_t ws_bytes,
                             hipStream_t stream) {
  const int64_t M = xq->rows, N = wq->rows;
  if (M == 0 || N == 0) return hipSuccess;
  const DownPlan pl = down_plan(M, ceil_div(xq->cols, kBlock), lora->count);
  float *t = static_cast<float *>(ws);
  DownArgs d{};
  d.side[0] = DownSide{source_of(xq, drop), static_cast<const uint16_t *>(lora->a), lora->lda, t, pl.parts};
  d.slots = pl.slots;
  d.M = M;
  d.index = index;
  d.count = lora->count;
  d.rank = lora->rank;
  const int64_t wgs = ceil_div(M, 16) * pl.slots * pl.parts;
  d.first = int(wgs);
  const hipError_t e = launch_down(d, wgs, stream);
  if (e != hipSuccess) return e;
  const LoraAdd add{t, M * lora->rank, static_cast<const uint16_t *>(lora->b), lora->scale, index, pl.parts, lora->count,
                    lora->rank, drop.gain, Drop{}};
  const size_t used = up16(size_t(pl.parts) * M * lora->rank * 4);
  return launch_gemm_lora(xq, wq, add, y, ldy, fast, static_cast<uint8_t *>(ws) + used, ws_bytes - used, stream);
}

size_t lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, int count, bool fast) {
  if (M == 0 || N == 0 || K == 0) return up16(size_t(count + 1) * 4);
  const BackwardPlan p = backward_plan(M, N, K, rank, count, fast);
  return p.rest + p.rest_bytes;
}

hipError_t launch_lora_backward(const fp8_tensor *dyq, const fp8_tensor *wq_t, const fp8_tensor *xq, const fp8_lora *lora,
                                const int32_t *index, const Drop &drop, void *dx, int64_t lddx, float *da, float *db,
                                bool fast, void *ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t M = dyq->rows, N = dyq->cols, K = xq->cols;
  const int rank = lora->rank, count = lora->count;
  uint8_t *base = static_cast<uint8_t *>(ws);
  JoinArgs j{};
  j.da = da;
  j.db = db;
  j.K = K;
  j.N = N;
  j.lda = lora->lda;
  j.scale = lora->scale;
  j.gain = drop.gain;
  j.rank = rank;
  j.a_wgs = int(ceil_div(rank * lora->lda, 4 * kThreads));
  j.wgs = j.a_wgs + int(ceil_div(rank * N, 4 * kThreads));
  j.chunk = 1;
  OrderArgs o{};
  o.index = index;
  o.M = M;
  o.count = count;
  o.rank = rank;
  hipError_t e;
  if (M == 0 || N == 0 || K == 0) {  // no product: the gradients are zeros
    o.M = 0;
    o.start = reinterpret_cast<int32_t *>(base);
    e = launch(order_kernel, dim3(unsigned(count)), dim3(kThreads), stream, o);
    if (e != hipSuccess) return e;
    if (M > 0 && K > 0) {  // N = 0: dx is a product over nothing
      e = launch_gemm(dyq, wq_t, dx, FP4_BF16, lddx, fast, nullptr, 0, stream);
      if (e != hipSuccess) return e;
    }
    j.start = o.start;
    return j.wgs == 0 ? hipSuccess : launch(join_kernel, dim3(unsigned(count * int64_t(j.wgs))), dim3(kThreads), stream, j);
  }
  const BackwardPlan p = backward_plan(M, N, K, rank, count, fast);
  float *t = reinterpret_cast<float *>(base + p.t), *dt = reinterpret_cast<float *>(base + p.dt);
  o.perm = reinterpret_cast<int32_t *>(base + p.perm);
  o.start = reinterpret_cast<int32_t *>(base + p.start);
  o.a = static_cast<const uint16_t *>(lora->a);
  o.b = static_cast<const uint16_t *>(lora->b);
  o.K = K;
  o.N = N;
  o.lda = lora->lda;
  o.ldb = p.ldb;
  o.at = reinterpret_cast<uint16_t *>(base + p.at);
  o.bt = reinterpret_cast<uint16_t *>(base + p.bt);
  o.a_tiles = int(ceil_div(K, 64));
  o.b_tiles = int(ceil_div(N, 64));
  e = launch(order_kernel, dim3(unsigned(count * int64_t(1 + o.a_tiles + o.b_tiles))), dim3(kThreads), stream, o);
  if (e != hipSuccess) return e;

  DownArgs d{};
  d.side[0] = DownSide{source_of(xq, drop), o.a, lora->lda, t, p.x.parts};
  d.side[1] = DownSide{source_of(dyq, Drop{}), o.bt, p.ldb, dt, p.dy.parts};
  d.slots = p.x.slots;
  d.M = M;
  d.index = index;
  d.count = count;
  d.rank = rank;
  const int64_t tiles = ceil_div(M, 16) * d.slots;
  d.first = int(tiles * p.x.parts);
  e = launch_down(d, tiles * (p.x.parts + p.dy.parts), stream);
  if (e != hipSuccess) return e;

  const LoraAdd add{dt, M * rank, o.at, lora->scale, index, p.dy.parts, count, rank, drop.gain, drop};
  e = launch_gemm_lora(dyq, wq_t, add, dx, lddx, fast, base + p.rest, ws_bytes - p.rest, stream);
  if (e != hipSuccess) return e;

  const int64_t kb = ceil_div(K, kBlock), nb = ceil_div(N, kBlock);
  float *pieces = reinterpret_cast<float *>(base + p.rest);
  OuterArgs u{};
  u.side[0] = OuterSide{source_of(xq, drop), dt, p.dy.parts, pieces, 0};
  u.side[1] = OuterSide{source_of(dyq, Drop{}), t, p.x.parts, pieces + p.pieces * kb * kBlock * rank, 1};
  u.M = M;
  u.chunk = p.chunk;
  u.index = index;
  u.perm = o.perm;
  u.start = o.start;
  u.count = count;
  u.rank = rank;
  e = launch_outer(u, dim3(unsigned(kb + nb), unsigned(p.chunks)), stream);
  if (e != hipSuccess) return e;
  j.pa = u.side[0].out;
  j.pb = u.side[1].out;
  j.wide_a = kb * kBlock;
  j.wide_b = nb * kBlock;
  j.chunk = p.chunk;
  j.start = o.start;
  return launch(join_kernel, dim3(unsigned(count * int64_t(j.wgs))), dim3(kThreads), stream, j);
}

}  // namespace fp8
}  // namespace nvfp4
