// fp8_lora.hip -- low-rank adapters beside a projection: the kernels next to the product
// itself (fp8_gemm.hip adds the adapters' part where it stores its results).
//
//   forward   down_kernel   t = dropout(x) a_i^T, passed on as c_i t in two or three bf16
//             product       y = x W^T + c_i t b_i^T          c_i = scale_i times dropout's gain
//             or of few tokens the product's partial sums, and
//             up_kernel     y = their sum + c_i t b_i^T      in binary32
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
constexpr int kDirectTokens = 512;  // the most that outer_kernel takes in one run

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

// ---------------------------------------------------------------------------
// t[m] = v[m] a_i^T: a workgroup takes 16 rows, 16 NR of the rank and, in turn, the adapters
// of its rows that fall to its slot; its waves take blocks of 128 in turn and join their
// sums.  Operands come from memory as the matrix instruction wants them, any assignment of
// the contraction to lane groups doing: lane group g's step 2 h + s is the 8 values from 64 h
// + 16 g + 8 s on, so that one load of a wave covers 64 or 128 neighbouring bytes of 16 rows.
// Nothing passes through LDS but the sums.  Rows with another adapter, or none, are left as
// they are: nothing reads them.  Of few tokens a's bytes bound it (8 tokens, eight adapters of
// 16 x 5120, 1.3 MB: 5.4 us, most of it the launch and three trips to memory); of many the
// lines of a that every workgroup reads again: 4096 tokens, rank 64 of 5120 with dropout, 27.5
// us for 21 MB of codes and 168 MB of a from L2; x (dropped out) and dy of 4096 tokens, 5120
// and 20480, rank 16, 43.5 us, 105 MB of codes.
struct DownSide {
  Source v;
  const uint16_t *a;  // [count][rank][lda]
  int64_t lda;
  float *t;        // [parts][M][rank], or null
  uint16_t *coef;  // [M][coef_parts][rank]: c_i t as the sum of as many bf16, or null
};

struct DownArgs {
  DownSide side[2];
  int first;  // workgroups of side 0
  int slots, rank_tiles, parts;
  int64_t M;
  const int32_t *index;
  const float *scale;
  float gain;
  int count, rank, coef_parts;
};

// U: blocks of a wave whose loads are in flight together
template <int NR, int WAVES, int U, bool DROP>
__global__ __launch_bounds__(64 * WAVES) void down_kernel(DownArgs p) {
  constexpr int RP = 16 * NR;
  __shared__ __attribute__((aligned(16))) float sums[WAVES][16][RP];
  __shared__ int ids[16];
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const bool second = int(blockIdx.x) >= p.first;
  const DownSide &side = p.side[second ? 1 : 0];
  const Source &v = side.v;
  int wg = int(blockIdx.x) - (second ? p.first : 0);
  const int r0 = RP * __builtin_amdgcn_readfirstlane(wg % p.rank_tiles);
  wg = __builtin_amdgcn_readfirstlane(wg / p.rank_tiles);
  const int part = __builtin_amdgcn_readfirstlane(wg % p.parts);
  wg = __builtin_amdgcn_readfirstlane(wg / p.parts);
  const int slot = __builtin_amdgcn_readfirstlane(wg % p.slots);
  const int64_t m0 = int64_t(__builtin_amdgcn_readfirstlane(wg / p.slots)) * 16;
  const int64_t m = m0 + lr, row = m < p.M ? m : p.M - 1;
  const int idx = m < p.M ? adapter_of(p.index, m, p.count) : -1;
  const int b_begin = int(int64_t(v.blocks) * part / p.parts), b_end = int(int64_t(v.blocks) * (part + 1) / p.parts);
  if (t < 16) ids[t] = idx;
  const Mask mask(v.drop);
  const uint64_t row_group = uint64_t(row) * uint64_t((v.cols + 7) >> 3) + 2 * lg;
  const uint8_t *codes_row = v.codes + row * v.ld + 16 * lg;

  bool pending = idx >= 0;
  for (int turn = 0;; ++turn) {
    const uint64_t some = __ballot(pending);
    if (some == 0) return;  // the same for every wave: all hold the tile's rows
    const int cur = __builtin_amdgcn_readlane(idx, __builtin_ctzll(some));
    pending = pending && idx != cur;
    if (turn % p.slots != slot) continue;

    const float c = p.scale[cur] * p.gain;
    f32x4 acc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t *a_row[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {  // past the rank: some row, whose sums are not stored
      const int r = r0 + 16 * n + lr < p.rank ? r0 + 16 * n + lr : 0;
      a_row[n] = side.a + (int64_t(cur) * p.rank + r) * side.lda + 16 * lg;
    }
    for (int b0 = b_begin + wave; b0 < b_end; b0 += U * WAVES) {
      uint4 x[U][2];
      uint32_t sb[U];
      bf16x8 fa[U][NR][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + u * WAVES;
        if (b >= b_end) break;
        const int64_t k = int64_t(b) * kBlock;
        x[u][0] = *reinterpret_cast<const uint4 *>(codes_row + k);
        x[u][1] = *reinterpret_cast<const uint4 *>(codes_row + k + 64);
        sb[u] = v.scales[int64_t(b) * v.srow + row];
        // lda is a multiple of 8: a group is readable where it begins inside
        const int inside = v.cols - k < kBlock ? int(v.cols - k) - 16 * lg : kBlock;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int at = 64 * (q >> 1) + 8 * (q & 1);
            fa[u][n][q] = at < inside ? *reinterpret_cast<const bf16x8 *>(a_row[n] + k + at) : bf16x8{};
          }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + u * WAVES;
        if (b >= b_end) break;
        const int64_t k = int64_t(b) * kBlock;
        if (k + kBlock > v.cols) {  // what follows a's rows is not read for a result
          const int left = int(v.cols - k) - 16 * lg;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int inside = left - 64 * (q >> 1) - 8 * (q & 1);  // elements of the group
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const uint32_t keep = inside >= 2 * d + 2 ? ~0u : inside == 2 * d + 1 ? 0xFFFFu : 0u;
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                u32x4 w = __builtin_bit_cast(u32x4, fa[u][n][q]);
                w[d] &= keep;
                fa[u][n][q] = __builtin_bit_cast(bf16x8, w);
              }
            }
          }
        }
        i32x8 codes{int(x[u][0].x), int(x[u][0].y), int(x[u][0].z), int(x[u][0].w),
                    int(x[u][1].x), int(x[u][1].y), int(x[u][1].z), int(x[u][1].w)};
        if constexpr (DROP) {
          if (mask.thr) {  // not of a gradient's rows
            static_for<4>([&](auto qc) {
              constexpr int q = decltype(qc)::value;
              const uint2 keep = mask.bytes(row_group + uint64_t((k >> 3) + 8 * (q >> 1) + (q & 1)));
              codes[2 * q] &= int(keep.x);
              codes[2 * q + 1] &= int(keep.y);
            });
          }
        }
        const float scale = scale_of(sb[u]);
        static_for<4>([&](auto qc) {
          constexpr int q = decltype(qc)::value;
          const bf16x8 fv = widen8<q>(codes, scale);
#pragma unroll
          for (int n = 0; n < NR; ++n)
            acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[u][n][q], fv, acc[n], 0, 0, 0);
        });
      }
    }
    // lane (lr, lg): row lr's products with a's rows 16 n + 4 lg + 0..3
#pragma unroll
    for (int n = 0; n < NR; ++n)
      *reinterpret_cast<float4 *>(&sums[wave][lr][16 * n + 4 * lg]) = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    __syncthreads();
    for (int e = t; e < 16 * RP; e += 64 * WAVES) {
      const int tok = e / RP, r = e % RP;
      const int64_t mt = m0 + tok;
      float s = sums[0][tok][r];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) s += sums[w][tok][r];
      if (r0 + r >= p.rank || ids[tok] != cur) continue;
      if (side.t) side.t[(int64_t(part) * p.M + mt) * p.rank + r0 + r] = s;
      if (side.coef) {
        uint16_t *to = side.coef + mt * p.coef_parts * p.rank + r0 + r;
        uint16_t w[3];
        split_bf16(s * c, w);
        to[0] = w[0];
        to[p.rank] = w[1];
        if (p.coef_parts == 3) to[2 * p.rank] = w[2];
      }
    }
    __syncthreads();  // the sums have been read
  }
}

// ---------------------------------------------------------------------------
// The result of few tokens, or of more with mixed adapters: the product's partial sums in their
// order and, by plain binary32 products, what the row's adapter adds.  A workgroup takes 256
// columns of a row.  b is read once for each token that has it, as few tokens leave nothing to
// share, by as many compute units as there are columns and tokens; inside the product a tile's
// adapters come one after the other, each with a wait for memory.  8 x 20480, eight adapters of
// 16: 4.0 us, 6.2 MB.
struct UpArgs {
  const float *base;  // [base_parts][M][base_ld]
  int base_parts;
  int64_t base_ld;
  const float *t;  // [parts][M][rank]
  int parts;
  const float *scale;
  float gain;
  const int32_t *index;
  int count, rank;
  const uint16_t *b;  // [count][N][rank], or with ldb > 0 the transpose [count][rank][ldb]
  int64_t ldb;
  int64_t M, N;
  uint16_t *y;
  int64_t ldy;
  Drop drop;  // of what the adapter adds
};

__global__ __launch_bounds__(kThreads) void up_kernel(UpArgs p) {
  __shared__ __attribute__((aligned(16))) float coef[128];
  const int t = threadIdx.x;
  const int64_t wide = (p.N + kThreads - 1) / kThreads;
  const int64_t m = int64_t(blockIdx.x) / wide, n = int64_t(blockIdx.x) % wide * kThreads + t;
  const int i = adapter_of(p.index, m, p.count);
  float v = 0.0f;
  if (n < p.N) {
    const float *src = p.base + m * p.base_ld + n;
#pragma unroll 4
    for (int s = 0; s < p.base_parts; ++s) v += src[int64_t(s) * p.M * p.base_ld];
  }
  if (i >= 0) {  // the same for the whole workgroup
    if (t < p.rank) {
      const float *src = p.t + m * p.rank + t;
      float s = 0.0f;
#pragma unroll 4
      for (int k = 0; k < p.parts; ++k) s += src[int64_t(k) * p.M * p.rank];
      coef[t] = s * (p.scale[i] * p.gain);
    }
    __syncthreads();
    float low = 0.0f;
    if (n < p.N) {
      if (p.ldb == 0) {
        const uint4 *row = reinterpret_cast<const uint4 *>(p.b + (int64_t(i) * p.N + n) * p.rank);
#pragma unroll 2
        for (int r = 0; r < p.rank; r += 8) {
          const uint4 w = row[r >> 3];
          const float4 c0 = *reinterpret_cast<const float4 *>(coef + r), c1 = *reinterpret_cast<const float4 *>(coef + r + 4);
          low = __builtin_fmaf(c0.x, __uint_as_float(w.x << 16), low);
          low = __builtin_fmaf(c0.y, __uint_as_float(w.x & 0xFFFF0000u), low);
          low = __builtin_fmaf(c0.z, __uint_as_float(w.y << 16), low);
          low = __builtin_fmaf(c0.w, __uint_as_float(w.y & 0xFFFF0000u), low);
          low = __builtin_fmaf(c1.x, __uint_as_float(w.z << 16), low);
          low = __builtin_fmaf(c1.y, __uint_as_float(w.z & 0xFFFF0000u), low);
          low = __builtin_fmaf(c1.z, __uint_as_float(w.w << 16), low);
          low = __builtin_fmaf(c1.w, __uint_as_float(w.w & 0xFFFF0000u), low);
        }
      } else {
        const uint16_t *col = p.b + int64_t(i) * p.rank * p.ldb + n;
#pragma unroll 8
        for (int r = 0; r < p.rank; ++r) low = __builtin_fmaf(coef[r], bf16_to_f32(col[r * p.ldb]), low);
      }
      if (p.drop.thr) {
        const uint32_t kept = Mask(p.drop).bits(uint64_t(m) * uint64_t((p.N + 7) >> 3) + uint64_t(n >> 3));
        low = (kept >> (n & 7)) & 1u ? low : 0.0f;
      }
      v += low;
    }
  }
  if (n < p.N) p.y[m * p.ldy + n] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// ---------------------------------------------------------------------------
// Before the backward pass's products.  Workgroups 0 .. count - 1: adapter i's tokens in
// their order, perm[start[i]] .. perm[start[i + 1] - 1], where start[i] counts the tokens of
// the adapters before it; each thread takes a run of tokens and a scan places its finds.  The
// others transpose: a [rank][lda] to at [K][rank] and b [N][rank] to bt [rank][ldb], zeros
// from N on, 64 rows or columns each.  10 us for 4096 tokens and an adapter of 16 x (5120 +
// 20480): the two passes over the tokens and the scan, one wait after the other.
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
    // eight loads at a time: the stores between them would keep them apart
    auto each = [&](auto &&take) {
      for (int64_t m = first; m < last; m += 8) {
        int i[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) i[k] = m + k < last ? adapter_of(p.index, m + k, p.count) : -1;
#pragma unroll
        for (int k = 0; k < 8; ++k) take(i[k], m + k);
      }
    };
    int mine = 0, before = 0;
    each([&](int i, int64_t) {
      mine += i == me;
      before += i >= 0 && i < me;
    });
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
    each([&](int i, int64_t m) {
      if (i == me) p.perm[at++] = int32_t(m);
    });
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
// Of few tokens (`direct`) a workgroup takes all of one adapter's and writes the gradient
// itself, zeros where it has none.  4096 tokens, 5120 and 20480 columns, rank 16 with dropout:
// 42 us for 105 MB (2.5 TB/s): a workgroup's rows are 128 bytes of every 5 or 20 KB.  Steps
// of 128 tokens took 1.5 us more there and 15 us instead of 11 for 777 x (2501 + 1030) of rank 32.
struct OuterSide {
  Source v;
  const float *coef;  // [M][rank]
  float *out;   // [piece][rank][wide], or with by_col [piece][wide][rank]; direct: an adapter a piece
  int64_t wide, limit;  // columns from v.cols on up to `limit` are written as zeros
  int by_col;
};

struct OuterArgs {
  OuterSide side[2];
  int64_t chunk;  // 0: direct
  const int32_t *index, *perm, *start;
  const float *scale;  // direct
  float gain;
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

// A token's coefficient with its block's scale.  Past binary32 it is the largest value there is:
// the block of an infinity or NaN has a scale of 2^120 and codes of zero (or a mask's zeros),
// which an infinite coefficient would make NaNs of.
__device__ __forceinline__ float scaled(float coef, float scale) {
  constexpr float kMost = 3.40282347e38f;
  const float f = coef * scale;
  return __builtin_fabsf(coef) < kInfinity ? fminf(fmaxf(f, -kMost), kMost) : f;
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
  // the waves share the rank's tiles before they share the columns': a coefficient's three
  // parts are read by as few waves as can be
  constexpr int WN = NR < 4 ? NR : 4, WF = 4 / WN, TN = NR / WN, TF = 8 / WF;
  __shared__ __attribute__((aligned(16))) uint8_t codes[kTokens * kRow];
  __shared__ __attribute__((aligned(16))) uint16_t coefs[3][kTokens][RP];
  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n_first = (wave % WN) * TN, f_first = (wave / WN) * TF;
  const bool second = int(blockIdx.x) >= p.side[0].v.blocks;
  const OuterSide &side = p.side[second ? 1 : 0];
  const Source &v = side.v;
  const int blk = int(blockIdx.x) - (second ? p.side[0].v.blocks : 0);
  const int64_t c0 = int64_t(blk) * kBlock;
  const bool direct = p.chunk == 0;
  const int64_t total = p.start[p.count], first = direct ? p.start[blockIdx.y] : int64_t(blockIdx.y) * p.chunk;
  if (!direct && first >= total) return;
  const int64_t last = direct ? p.start[blockIdx.y + 1] : first + p.chunk < total ? first + p.chunk : total;
  const Mask mask(v.drop);
  const int64_t groups = (v.cols + 7) >> 3;

  // a thread takes 32 codes of a token of a step and, of its coefficients, every fourth four
  const int tok = t >> 2, quarter = t & 3;
  const uint8_t *codes_at = v.codes + c0 + 32 * quarter, *scales_at = v.scales + int64_t(blk) * v.srow;
  const float *coef_at = side.coef + 4 * quarter;
  struct Step {
    uint4 x, y;
    uint32_t scale;
    float4 cf[NR];
    int64_t m;  // -1: no token
  };
  auto token = [&](int64_t at, int64_t stop) { return at + tok < stop ? int64_t(p.perm[at + tok]) : int64_t(-1); };
  auto fetch = [&](Step &s, int64_t m) {
    s.m = m;
    s.x = s.y = make_uint4(0u, 0u, 0u, 0u);
    s.scale = 0;
#pragma unroll
    for (int n = 0; n < NR; ++n) s.cf[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (m < 0) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(codes_at + m * v.ld);
    s.x = src[0];
    s.y = src[1];
    s.scale = scales_at[m];
#pragma unroll
    for (int n = 0; n < NR; ++n)
      if (16 * n + 4 * quarter < p.rank) s.cf[n] = *reinterpret_cast<const float4 *>(coef_at + m * p.rank + 16 * n);
  };

  int a = direct ? int(blockIdx.y) : __builtin_amdgcn_readfirstlane(adapter_of(p.index, p.perm[first], p.count));
  int piece = direct ? a : int(blockIdx.y) + used_before(p.start, a);
  const float c = !direct ? 1.0f : last > first ? p.scale[a] * p.gain : 0.0f;
  int64_t at = first;
  do {
    const int64_t stop = p.start[a + 1] < last ? p.start[a + 1] : last;
    ++a;
    if (stop <= at && !direct) continue;  // no token
    f32x4 acc[TF][TN];
#pragma unroll
    for (int f = 0; f < TF; ++f)
#pragma unroll
      for (int n = 0; n < TN; ++n) acc[f][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // the next step's operands are on their way while this one's are multiplied, and the
    // place of the one after
    Step now;
    fetch(now, token(at, stop));
    int64_t next = token(at + kTokens, stop);
    for (; at < stop; at += kTokens) {
      uint4 x = now.x, y = now.y;
      if (mask.thr) {
        const uint64_t g = uint64_t(now.m < 0 ? 0 : now.m) * uint64_t(groups) + uint64_t((c0 >> 3) + 4 * quarter);
        const uint2 k0 = mask.bytes(g), k1 = mask.bytes(g + 1), k2 = mask.bytes(g + 2), k3 = mask.bytes(g + 3);
        x.x &= k0.x; x.y &= k0.y; x.z &= k1.x; x.w &= k1.y;
        y.x &= k2.x; y.y &= k2.y; y.z &= k3.x; y.w &= k3.y;
      }
      const float scale = scale_of(now.scale);
      __syncthreads();  // the last step's operands have been read
      *reinterpret_cast<uint4 *>(codes + tok * kRow + 32 * quarter) = x;
      *reinterpret_cast<uint4 *>(codes + tok * kRow + 32 * quarter + 16) = y;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float f[4] = {scaled(now.cf[n].x, scale), scaled(now.cf[n].y, scale), scaled(now.cf[n].z, scale),
                            scaled(now.cf[n].w, scale)};
        s16x4 w[3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint16_t part[3];
          split_bf16(f[j], part);
#pragma unroll
          for (int s = 0; s < 3; ++s) w[s][j] = short(part[s]);
        }
#pragma unroll
        for (int s = 0; s < 3; ++s) *reinterpret_cast<s16x4 *>(&coefs[s][tok][16 * n + 4 * quarter]) = w[s];
      }
      fetch(now, next);
      next = token(at + 2 * kTokens, stop);
      __syncthreads();
      // the lane's place in a transposing read: 8 tokens of 16 codes, 4 tokens of 16 bf16
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k8 = 32 * half + 8 * lg;
        bf16x8 fv[TF];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
          const uint8_t *from = codes + (k8 + (lr >> 1)) * kRow + 16 * (f_first + f) + 8 * (lr & 1);
          const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (__attribute__((address_space(3))) i32x2 *)const_cast<uint8_t *>(from));
          fv[f] = widen8<0>(i32x8{w[0], w[1], 0, 0, 0, 0, 0, 0}, 1.0f);
        }
#pragma unroll
        for (int n = 0; n < TN; ++n)
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            s16x8 w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint16_t *from = &coefs[s][k8 + 4 * h + (lr >> 2)][16 * (n_first + n) + 4 * (lr & 3)];
              const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4 *)const_cast<uint16_t *>(from));
#pragma unroll
              for (int j = 0; j < 4; ++j) w[4 * h + j] = q[j];
            }
            const bf16x8 fc = __builtin_bit_cast(bf16x8, w);
#pragma unroll
            for (int f = 0; f < TF; ++f) acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fc, fv[f], acc[f][n], 0, 0, 0);
          }
      }
    }
    at = stop;
    // lane (lr, lg): column lr of its tile f, a's rows or b's columns 16 n + 4 lg + 0..3
    float *out = side.out + int64_t(piece) * side.wide * p.rank;
    auto put = [&](int64_t col, int r, const f32x4 &w) {
      const bool in = col < v.cols;
      const float4 o = in ? make_float4(w[0] * c, w[1] * c, w[2] * c, w[3] * c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (side.by_col) {
        *reinterpret_cast<float4 *>(out + col * p.rank + r) = o;
      } else {
        out[r * side.wide + col] = o.x;
        out[(r + 1) * side.wide + col] = o.y;
        out[(r + 2) * side.wide + col] = o.z;
        out[(r + 3) * side.wide + col] = o.w;
      }
    };
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      const int r = 16 * (n_first + n) + 4 * lg;
      if (r >= p.rank) continue;
#pragma unroll
      for (int f = 0; f < TF; ++f) {
        const int64_t col = c0 + 16 * (f_first + f) + lr;
        if (col < side.limit) put(col, r, acc[f][n]);
      }
      // what lies past the last block of 128
      if (blk == v.blocks - 1)
        for (int64_t col = c0 + kBlock + 16 * (wave / WN) + lr; col < side.limit; col += 16 * WF)
          put(col, r, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
    }
    ++piece;
  } while (at < last);
}

// da [count][rank][lda] and db [count][N][rank] from the pieces in their order; an adapter
// without tokens, and da's padding, take zeros.  Four elements to a thread: 5.8 us for six
// pieces of 16 x 25600.
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

// How many workgroups share a tile: with few tiles up to 16 take its adapters in turn, one
// each 16 of the rank and, where the caller takes parts, up to 8 a part of the contraction,
// one block or two to a wave.  A CU alone reads from memory at some 30 GB/s: an adapter of 16
// x 5120 took one workgroup 8 us, five of them 4.  The order of a sum's terms, which the waves
// and parts give, does not depend on how many adapters there are.
struct DownPlan {
  int slots, rank_tiles, parts;
  int64_t wgs;  // of a side
};
DownPlan down_plan(int64_t M, int64_t blocks, int rank, int count, bool in_parts) {
  const int64_t tiles = ceil_div(M, 16), full = 2 * cu_count();
  int64_t slots = 64 / tiles;
  slots = slots < 1 ? 1 : slots > 16 ? 16 : slots;
  if (slots > count) slots = count;
  if (slots > M) slots = M;
  int64_t rank_tiles = ceil_div(rank, 16), parts = 1;
  if (in_parts && tiles * rank_tiles < cu_count()) {
    parts = full / (tiles * rank_tiles);
    const int64_t most = ceil_div(blocks, 8) < 8 ? ceil_div(blocks, 8) : 8;
    parts = parts < most ? parts : most;
  }
  if (parts <= 1) {
    parts = 1;
    if (tiles * slots > cu_count() / 4) rank_tiles = 1;
  }
  return DownPlan{int(slots), int(rank_tiles), int(parts), tiles * slots * rank_tiles * parts};
}

// Whether the product's partial sums and up_kernel run, or the product that begins with the
// adapters.  The first reads b once a token, the second takes a tile's adapters one after the
// other: 64 tokens and fewer take the first, and more where the caller says that their adapters
// are mixed.  How many adapters are loaded says neither, nor may it change a token's last bits.
// Forward calls by the product and by the partial sums, us, rank 16, of tokens with one adapter,
// eight and 64 mixed: 65 x 5120 x 5120 28 and 24, 39 and 25, 70 and 28; 128 x 5120 x 5120 31 and
// 31, 38 and 33, 64 and 38; 128 x 2048 x 512 12 and 15, 19 and 16, 38 and 17; 512 x 20480 x 5120
// 71 and 147, 106 and 150, 249 and 165; 256 x 5120 x 20480 86 and 69, 118 and 78, 200 and 93.
// A launch holds fewer than 2^32 threads: what would pass that takes the product.
constexpr int64_t kFewTokens = 64, kMixedTokens = 512, kMaxGroups = 16776960;
bool few_tokens(int64_t M, int64_t width, bool mixed) {
  return M <= kFewTokens || (mixed && M <= kMixedTokens && M * ceil_div(width, kThreads) <= kMaxGroups);
}

hipError_t launch_up(const fp8_tensor *a, const fp8_tensor *w, bool fast, UpArgs &u, void *ws, hipStream_t stream) {
  const Partials pl = gemm_partials(a->rows, w->rows, ceil_div(a->cols, kBlock), fast);
  const hipError_t e = launch_gemm_partials(a, w, fast, static_cast<float *>(ws), stream);
  if (e != hipSuccess) return e;
  u.base = static_cast<const float *>(ws);
  u.base_parts = pl.ksplit;
  u.base_ld = pl.ld;
  u.M = a->rows;
  u.N = w->rows;
  return launch(up_kernel, dim3(unsigned(u.M * ceil_div(u.N, kThreads))), dim3(kThreads), stream, u);
}

// Tokens of a run of outer_kernel: four workgroups to a CU where there are tokens enough; 0
// where there are so few that a workgroup goes through all of an adapter's.
int64_t outer_chunk(int64_t M, int64_t blocks) {
  if (M <= kDirectTokens) return 0;
  const int64_t want = ceil_div(4 * cu_count(), blocks);
  const int64_t c = ceil_div(ceil_div(M, want), kTokens) * kTokens;
  return c < kTokens ? kTokens : c;
}

// As many waves to a workgroup as its registers leave room for: up to 4096 tokens it is the
// only one on its CU.
template <bool DROP>
hipError_t launch_down_as(const DownArgs &a, dim3 grid, hipStream_t stream) {
  if (a.parts > 1) return launch(down_kernel<1, 4, 2, DROP>, grid, dim3(256), stream, a);
  if (a.rank <= 16 || a.rank_tiles > 1) return launch(down_kernel<1, 16, DROP ? 1 : 2, DROP>, grid, dim3(1024), stream, a);
  if (a.rank <= 32) return launch(down_kernel<2, 16, 1, DROP>, grid, dim3(1024), stream, a);
  if (a.rank <= 64) return launch(down_kernel<4, 8, 1, DROP>, grid, dim3(512), stream, a);
  return launch(down_kernel<8, 4, 1, DROP>, grid, dim3(256), stream, a);
}

hipError_t launch_down(DownArgs &a, int sides, const DownPlan &pl, hipStream_t stream) {
  a.slots = pl.slots;
  a.rank_tiles = pl.rank_tiles;
  a.parts = pl.parts;
  a.first = int(pl.wgs);
  const dim3 grid{unsigned(sides * pl.wgs)};
  return a.side[0].v.drop.thr ? launch_down_as<true>(a, grid, stream) : launch_down_as<false>(a, grid, stream);
}

hipError_t launch_outer(const OuterArgs &a, dim3 grid, hipStream_t stream) {
  const dim3 blk{kThreads};
  if (a.rank <= 16) return launch(outer_kernel<1>, grid, blk, stream, a);
  if (a.rank <= 32) return launch(outer_kernel<2>, grid, blk, stream, a);
  if (a.rank <= 64) return launch(outer_kernel<4>, grid, blk, stream, a);
  return launch(outer_kernel<8>, grid, blk, stream, a);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// What the product with the weight takes.
size_t product_bytes(int64_t M, int64_t N, int64_t blocks, bool few, bool fast) {
  return up16(few ? gemm_partials(M, N, blocks, fast).bytes : gemm_ws_bytes(M, N, blocks, fast));
}

// The backward pass's workspace, in bytes from its beginning.
struct BackwardPlan {
  int64_t chunk, chunks, pieces, ldb;
  size_t t, dt, coef, perm, start, at, bt, rest, rest_bytes;
};
BackwardPlan backward_plan(int64_t M, int64_t N, int64_t K, int rank, int64_t count, bool few, bool fast) {
  BackwardPlan p{};
  const int64_t kb = ceil_div(K, kBlock), nb = ceil_div(N, kBlock);
  p.chunk = outer_chunk(M, kb + nb);
  p.chunks = p.chunk ? ceil_div(M, p.chunk) : count;
  p.pieces = p.chunk ? p.chunks + (count < M ? count : M) - 1 : 0;
  p.ldb = ceil_div(N, 8) * 8;
  size_t n = 0;
  auto place = [&](size_t bytes) {
    const size_t at = n;
    n += up16(bytes);
    return at;
  };
  p.t = place(size_t(M) * rank * 4);
  p.dt = place(size_t(M) * rank * 4);
  p.coef = place(few ? 0 : size_t(lora_parts(fast)) * M * rank * 2);
  p.perm = place(size_t(M) * 4);
  p.start = place(size_t(count + 1) * 4);
  p.at = place(few ? 0 : size_t(count) * K * rank * 2);
  p.bt = place(size_t(count) * rank * p.ldb * 2);
  p.rest = n;  // the product's partials, and after it the sums' pieces
  const size_t gemm = product_bytes(M, K, nb, few, fast), outer = size_t(p.pieces) * size_t(kb + nb) * kBlock * rank * 4;
  p.rest_bytes = up16(gemm > outer ? gemm : outer);
  return p;
}

}  // namespace

// t in parts, or as bf16.
size_t coef_bytes(int64_t M, int64_t blocks, int rank, bool few, bool fast) {
  const size_t each = few ? size_t(down_plan(M, blocks, rank, 1, few).parts) * 4 : size_t(lora_parts(fast)) * 2;
  return up16(each * M * rank);
}

size_t lora_fprop_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, bool mixed, bool fast) {
  if (M == 0 || N == 0) return 0;
  const int64_t kb = ceil_div(K, kBlock);
  const bool few = few_tokens(M, N, mixed);
  return coef_bytes(M, kb, rank, few, fast) + product_bytes(M, N, kb, few, fast);
}

hipError_t launch_lora_fprop(const fp8_tensor *xq, const fp8_tensor *wq, const fp8_lora *lora, const int32_t *index,
                             const Drop &drop, void *y, int64_t ldy, bool mixed, bool fast, void *ws, size_t ws_bytes,
                             hipStream_t stream) {
  const int64_t M = xq->rows, N = wq->rows, kb = ceil_div(xq->cols, kBlock);
  if (M == 0 || N == 0) return hipSuccess;
  const int rank = lora->rank, count = lora->count;
  const bool few = few_tokens(M, N, mixed);
  const DownPlan pl = down_plan(M, kb, rank, count, few);
  const uint16_t *b = static_cast<const uint16_t *>(lora->b);
  float *t = static_cast<float *>(ws);
  uint16_t *coef = static_cast<uint16_t *>(ws);
  const size_t used = coef_bytes(M, kb, rank, few, fast);
  void *rest = static_cast<uint8_t *>(ws) + used;
  DownArgs d{};
  d.side[0] = DownSide{source_of(xq, drop), static_cast<const uint16_t *>(lora->a), lora->lda, few ? t : nullptr,
                       few ? nullptr : coef};
  d.M = M;
  d.index = index;
  d.scale = lora->scale;
  d.gain = drop.gain;
  d.count = count;
  d.rank = rank;
  d.coef_parts = lora_parts(fast);
  const hipError_t e = launch_down(d, 1, pl, stream);
  if (e != hipSuccess) return e;
  if (few) {
    UpArgs u{};
    u.t = t;
    u.parts = pl.parts;
    u.scale = lora->scale;
    u.gain = drop.gain;
    u.index = index;
    u.count = count;
    u.rank = rank;
    u.b = b;
    u.y = static_cast<uint16_t *>(y);
    u.ldy = ldy;
    return launch_up(xq, wq, fast, u, rest, stream);
  }
  const LoraAdd add{coef, b, index, count, rank, d.coef_parts, Drop{}};
  return launch_gemm_lora(xq, wq, add, y, ldy, fast, rest, ws_bytes - used, stream);
}

size_t lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int rank, int count, bool mixed, bool fast) {
  if (M == 0 || N == 0 || K == 0) return up16(size_t(count + 1) * 4);
  const BackwardPlan p = backward_plan(M, N, K, rank, count, few_tokens(M, K, mixed), fast);
  return p.rest + p.rest_bytes;
}

hipError_t launch_lora_backward(const fp8_tensor *dyq, const fp8_tensor *wq_t, const fp8_tensor *xq, const fp8_lora *lora,
                                const int32_t *index, const Drop &drop, void *dx, int64_t lddx, float *da, float *db,
                                bool mixed, bool fast, void *ws, size_t ws_bytes, hipStream_t stream) {
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
  const bool few = few_tokens(M, K, mixed);
  const BackwardPlan p = backward_plan(M, N, K, rank, count, few, fast);
  float *t = reinterpret_cast<float *>(base + p.t), *dt = reinterpret_cast<float *>(base + p.dt);
  uint16_t *coef = reinterpret_cast<uint16_t *>(base + p.coef);
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
  o.a_tiles = few ? 0 : int(ceil_div(K, 64));  // a as it is does
  o.b_tiles = int(ceil_div(N, 64));
  e = launch(order_kernel, dim3(unsigned(count * int64_t(1 + o.a_tiles + o.b_tiles))), dim3(kThreads), stream, o);
  if (e != hipSuccess) return e;

  DownArgs d{};
  d.side[0] = DownSide{source_of(xq, drop), o.a, lora->lda, t, nullptr};
  d.side[1] = DownSide{source_of(dyq, Drop{}), o.bt, p.ldb, dt, few ? nullptr : coef};
  d.M = M;
  d.index = index;
  d.scale = lora->scale;
  d.gain = drop.gain;
  d.count = count;
  d.rank = rank;
  d.coef_parts = lora_parts(fast);
  e = launch_down(d, 2, down_plan(M, 0, rank, count, false), stream);
  if (e != hipSuccess) return e;

  if (few) {
    UpArgs u{};
    u.t = dt;
    u.parts = 1;
    u.scale = lora->scale;
    u.gain = drop.gain;
    u.index = index;
    u.count = count;
    u.rank = rank;
    u.b = o.a;
    u.ldb = lora->lda;
    u.y = static_cast<uint16_t *>(dx);
    u.ldy = lddx;
    u.drop = drop;
    e = launch_up(dyq, wq_t, fast, u, base + p.rest, stream);
  } else {
    const LoraAdd add{coef, o.at, index, count, rank, d.coef_parts, drop};
    e = launch_gemm_lora(dyq, wq_t, add, dx, lddx, fast, base + p.rest, ws_bytes - p.rest, stream);
  }
  if (e != hipSuccess) return e;

  const int64_t kb = ceil_div(K, kBlock), nb = ceil_div(N, kBlock);
  float *pieces = reinterpret_cast<float *>(base + p.rest);
  OuterArgs u{};
  const bool direct = p.chunk == 0;
  u.side[0] = OuterSide{source_of(xq, drop), dt, direct ? da : pieces, direct ? lora->lda : kb * kBlock,
                        direct ? lora->lda : kb * kBlock, 0};
  u.side[1] = OuterSide{source_of(dyq, Drop{}), t, direct ? db : pieces + p.pieces * kb * kBlock * rank,
                        direct ? N : nb * kBlock, direct ? N : nb * kBlock, 1};
  u.chunk = p.chunk;
  u.index = index;
  u.perm = o.perm;
  u.start = o.start;
  u.scale = lora->scale;
  u.gain = drop.gain;
  u.count = count;
  u.rank = rank;
  e = launch_outer(u, dim3(unsigned(kb + nb), unsigned(p.chunks)), stream);
  if (e != hipSuccess || direct) return e;
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
