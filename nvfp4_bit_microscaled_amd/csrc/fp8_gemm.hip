// fp8_gemm.hip -- products of two E4M3 tensors with a power-of-two scale per block of
// 128: C = deq(A) . deq(B)^T, FP32 accumulation.
//
// FAST: the 128-wide blocks meet gfx950's block-scaled matrix instruction exactly:
// v_mfma_scale_f32_16x16x128_f8f6f4 takes one E8M0 scale per row and 32 K values, and
// all four 32-groups of a K block share the block's scale byte, so one instruction is
// one K block of a 16 x 16 tile and operands go from memory to LDS to the matrix core
// as they are.  What that gives up: the instruction adds the products of 8 consecutive
// bytes of a lane after cutting each off at 2^-13 of the group's largest power of two
// (measured here with pairs of powers of two; so do the unscaled 8-bit instructions);
// everything after that is binary32.  On normal operands C is 1.5e-5 off (relative
// 2-norm), far below a bf16 result's own rounding, and not what a binary32 C promises.
// Otherwise the lane's codes are converted to bf16 with their scale applied (E4M3 times
// a power of two is exact in bf16) and v_mfma_f32_16x16x32_bf16 keeps every product:
// 3.6e-8 off, at half the matrix rate and one conversion per two elements.
//
// MFMA operand mapping: lane l supplies row l % 16 of its operand and 32 of its 128 K
// values (any assignment of K values to lane groups works, since A and B use the same
// one and the scale is the same for all).  Rows are dealt so that tile i of a wave
// takes row (l % 16) * T + i of the wave's 16 T rows: a lane's T scales are then T
// neighbouring bytes, and with B as the first operand its outputs are 4 T neighbouring
// columns of each of its rows of C.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8.hpp"

namespace nvfp4 {
namespace fp8 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kGroupM = 8;

// One operand: its rows, bytes per row of codes, bytes per K block of scales.
struct Operand {
  const uint8_t *codes, *scales;
  int64_t rows, ld, srow;
  int two_d;
};

struct GemmParams {
  Operand a[2], b[2];  // stages [0, kb) read pair 0, [kb, 2 kb) pair 1
  int64_t M, N;
  int kb;              // K blocks of a pair
  int stages;          // in all
  void *c;
  int64_t ldc;
  int c_bf16, c_vec;   // c_vec: 16-byte stores of whole groups are aligned
  int ksplit;
  float *ws;           // ksplit > 1: raw partials [ksplit][M][ws_ld]
  int64_t ws_ld;
};

__device__ __forceinline__ u32x4 make_rsrc(const void *p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return u32x4{uint32_t(a), uint32_t(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// DMA from a buffer into LDS: lane l reads voffset + soffset (zeros where voffset is at
// or past the buffer's range) and writes its 16, 4 or (zero-extended to 4) 1 bytes at
// dst + l * that size.  Inline assembly so that the compiler does not stall later LDS
// reads of other buffers on these loads; the kernels wait with vmcnt themselves before
// the barrier that precedes the first read.  M0 carries dst; no other instruction of
// this file uses M0 (tests/test_fp8_abi.py checks the assembly), and its write needs
// one wait state before the DMA reads it.
__device__ __forceinline__ void dma16(const u32x4 &rsrc, void *dst, uint32_t voffset, uint32_t soffset) {
  const uint32_t a = uint32_t(reinterpret_cast<uintptr_t>(dst));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(a), "v"(voffset), "s"(rsrc), "s"(soffset));
}
__device__ __forceinline__ void dma4(const u32x4 &rsrc, void *dst, uint32_t voffset, uint32_t soffset) {
  const uint32_t a = uint32_t(reinterpret_cast<uintptr_t>(dst));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(a), "v"(voffset), "s"(rsrc), "s"(soffset));
}
__device__ __forceinline__ void dma1(const u32x4 &rsrc, void *dst, uint32_t voffset, uint32_t soffset) {
  const uint32_t a = uint32_t(reinterpret_cast<uintptr_t>(dst));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, %3 offen lds"
               :
               : "s"(a), "v"(voffset), "s"(rsrc), "s"(soffset));
}

// Workgroup -> tile: consecutive workgroups go to different XCDs, so ids are renumbered
// to give each XCD a contiguous range, walked in groups of kGroupM tile rows so that
// neighbours share A rows and B rows in that XCD's L2.
__device__ __forceinline__ void tile_of(int pid, int total, int num_m, int num_n, int &tm, int &tn) {
  if ((total & 7) == 0) pid = (pid & 7) * (total >> 3) + (pid >> 3);
  const int per_group = kGroupM * num_n;
  const int grp = pid / per_group, first = grp * kGroupM;
  const int gsz = min(num_m - first, kGroupM);
  tm = first + (pid % per_group) % gsz;
  tn = (pid % per_group) / gsz;
}

// T scale bytes of a lane (T = 1, 2, 4, 8) for the tiles i = 0..T-1: byte i & 3 of word i >> 2.
template <int T>
__device__ __forceinline__ void read_scales(const uint8_t *p, uint32_t (&w)[(T + 3) / 4]) {
  if constexpr (T == 8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else if constexpr (T == 4) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (T == 2) {
    w[0] = *reinterpret_cast<const uint16_t *>(p);
  } else {
    w[0] = *p;
  }
}

template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma(i32x8 a, i32x8 b, f32x4 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, SA, int(sa), SB, int(sb));
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

__device__ __forceinline__ float scale_value(uint32_t word, int byte) {
  return __uint_as_float(((word >> (8 * byte)) & 0xFFu) << 23);
}

template <class F, int... Is>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// One output row's 4 * T neighbouring columns n0 .. of this lane.
template <int NV>
__device__ __forceinline__ void store_run(const GemmParams &p, void *c, int64_t ldc, bool bf16, bool vec, int64_t m,
                                          int64_t n0, const float (&v)[NV]) {
  if (bf16) {
    uint16_t *dst = reinterpret_cast<uint16_t *>(c) + m * ldc + n0;
    constexpr int W = NV < 8 ? NV : 8;
#pragma unroll
    for (int k = 0; k < NV; k += W) {
      if (vec && W == 8 && n0 + k + 8 <= p.N) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = uint32_t(f32_to_bf16(v[k + (2 * j) % W])) | (uint32_t(f32_to_bf16(v[k + (2 * j + 1) % W])) << 16);
        *reinterpret_cast<uint4 *>(dst + k) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (n0 + k + j < p.N) dst[k + j] = f32_to_bf16(v[k + j]);
      }
    }
  } else {
    float *dst = reinterpret_cast<float *>(c) + m * ldc + n0;
#pragma unroll
    for (int k = 0; k < NV; k += 4) {
      if (vec && n0 + k + 4 <= p.N) {
        *reinterpret_cast<float4 *>(dst + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + k + j < p.N) dst[k + j] = v[k + j];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The general kernel: a BM x BN tile, WAVES_M x WAVES_N waves, NBUF stages of 128 K in
// LDS.  Stage layout: A codes [BM][128 B], B codes [BN][128 B], 256 B of A scales,
// 256 B of B scales.  A row's eight 16-byte chunks sit at chunk ^ (row / T) % 8 with T
// the operand's tiles per wave: the 16 lanes that read one chunk of rows T apart then
// spread over all chunk positions.  Rows past the matrix come back as zeros (the
// buffer's range check) and their outputs are not stored.
template <int BM, int BN, int WAVES_M, int WAVES_N, int NBUF, bool FAST>
__global__ __launch_bounds__(64 * WAVES_M *WAVES_N) void gemm_kernel(GemmParams p) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 16, TN = WN / 16;
  // DMA instructions (8 rows each) per wave; a tile with fewer rows than waves * 8 is
  // loaded by several waves, which write the same bytes
  constexpr int JA = BM > 8 * NW ? BM / (8 * NW) : 1, JB = BN > 8 * NW ? BN / (8 * NW) : 1;
  constexpr int S_OFF = (BM + BN) * kBlock, STAGE = S_OFF + 512;
  constexpr int NDMA = JA + JB + 1;
  static_assert(NW % 2 == 0 && BM <= 256 && BN <= 256, "scale DMA: one dword per lane covers 256 rows");
  static_assert((NBUF - 2) * NDMA < 63, "vmcnt");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * STAGE];

  const int t = threadIdx.x, lane = t & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int num_m = int((p.M + BM - 1) / BM), num_n = int((p.N + BN - 1) / BN);
  int tm, tn;
  const int split = int(blockIdx.x) % p.ksplit;
  tile_of(int(blockIdx.x) / p.ksplit, int(gridDim.x) / p.ksplit, num_m, num_n, tm, tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int s_begin = int(int64_t(p.stages) * split / p.ksplit);
  const int s_end = int(int64_t(p.stages) * (split + 1) / p.ksplit);

  // row (within the tile) of DMA instruction j of this wave
  auto dma_row = [&](int j, int rows) { return ((j * NW + wave) * 8) % rows; };
  auto chunk_of = [&](int row, int T) { return uint32_t(((lane & 7) ^ ((row / T) & 7)) << 4); };
  // rows of a tile: base of 8 rows, range = the rows that exist
  auto rsrc_of = [&](const Operand &o, int64_t row, bool live) {
    const int64_t left = o.rows - row;
    const uint32_t n = !live || left <= 0 ? 0u : uint32_t(left < 8 ? left : 8);
    return make_rsrc(o.codes + (n ? row * o.ld : 0), n * uint32_t(o.ld));
  };
  auto issue = [&](int s, int buf) {
    const bool live = s < s_end;
    const int pair = s >= p.kb ? 1 : 0;
    const uint32_t kt = uint32_t(s - pair * p.kb);
    const Operand &a = p.a[pair], &b = p.b[pair];
    uint8_t *base = lds + buf * STAGE;
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const int row = dma_row(j, BM);
      const uint32_t v = uint32_t(lane >> 3) * uint32_t(a.ld) + chunk_of(row + (lane >> 3), TM);
      dma16(rsrc_of(a, m0 + row, live), base + row * kBlock, v, live ? kt * kBlock : 0u);
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int row = dma_row(j, BN);
      const uint32_t v = uint32_t(lane >> 3) * uint32_t(b.ld) + chunk_of(row + (lane >> 3), TN);
      dma16(rsrc_of(b, n0 + row, live), base + (BM + row) * kBlock, v, live ? kt * kBlock : 0u);
    }
    // scales: even waves A's, odd waves B's (several waves write the same bytes).  1D:
    // lane l the dword of rows 4 l .. 4 l + 3; 2D: lane l the byte of tile l.
    const Operand &o = (wave & 1) ? b : a;
    const int64_t r0 = (wave & 1) ? n0 : m0;
    const int64_t first = o.two_d ? r0 / kBlock : r0;
    const int64_t left = o.srow - first;
    const u32x4 rs = make_rsrc(o.scales + (live ? int64_t(kt) * o.srow + first : 0),
                               live && left > 0 ? uint32_t(left) : 0u);
    uint8_t *dst = base + S_OFF + 256 * (wave & 1);
    if (o.two_d) dma1(rs, dst, uint32_t(lane), 0u);
    else dma4(rs, dst, uint32_t(lane) * 4u, 0u);
  };

  const int wm = (wave / WAVES_N) * WM, wn = (wave % WAVES_N) * WN;
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int s = 0; s < NBUF - 1; ++s) issue(s_begin + s, s);
  int buf = 0;
  for (int s = s_begin; s < s_end; ++s) {
    // stage s has landed for this wave, and its reads of the buffer that is refilled
    // next are done; past the barrier both hold for every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * NDMA) : "memory");
    __syncthreads();
    issue(s + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
    const uint8_t *base = lds + buf * STAGE;
    auto frag = [&](int row) {
      const uint8_t *r = base + row * kBlock;
      const uint4 x = *reinterpret_cast<const uint4 *>(r + ((lg ^ (lr & 7)) << 4));
      const uint4 y = *reinterpret_cast<const uint4 *>(r + (((lg + 4) ^ (lr & 7)) << 4));
      return i32x8{int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
    };
    uint32_t sa[(TM + 3) / 4], sb[(TN + 3) / 4];
    const int pair = s >= p.kb ? 1 : 0;
    if (p.a[pair].two_d) {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(base + S_OFF + 4 * (wm / kBlock)) * 0x01010101u;
#pragma unroll
      for (int i = 0; i < (TM + 3) / 4; ++i) sa[i] = v;
    } else {
      read_scales<TM>(base + S_OFF + wm + lr * TM, sa);
    }
    if (p.b[pair].two_d) {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(base + S_OFF + 256 + 4 * (wn / kBlock)) * 0x01010101u;
#pragma unroll
      for (int i = 0; i < (TN + 3) / 4; ++i) sb[i] = v;
    } else {
      read_scales<TN>(base + S_OFF + 256 + wn + lr * TN, sb);
    }
    i32x8 fb[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = frag(BM + wn + lr * TN + j);
    if constexpr (!FAST) {
      i32x8 fa[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = frag(wm + lr * TM + i);
      static_for<4>([&](auto qc) {
        constexpr int q = decltype(qc)::value;
        bf16x8 wb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) wb[j] = widen8<q>(fb[j], scale_value(sb[j >> 2], j & 3));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const bf16x8 wa = widen8<q>(fa[i], scale_value(sa[i >> 2], i & 3));
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
        }
      });
    } else static_for<TM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      const i32x8 fa = frag(wm + lr * TM + i);
      static_for<TN>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        acc[i][j] = mfma<(j & 3), (i & 3)>(fb[j], fa, acc[i][j], sb[j >> 2], sa[i >> 2]);
      });
    });
    buf = buf + 1 == NBUF ? 0 : buf + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no DMA into LDS outlives the workgroup

  const bool raw = p.ksplit > 1;
  void *c = raw ? static_cast<void *>(p.ws + int64_t(split) * p.M * p.ws_ld) : p.c;
  const int64_t ldc = raw ? p.ws_ld : p.ldc;
  const int64_t n = n0 + wn + 4 * lg * TN;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t m = m0 + wm + lr * TM + i;
    float v[4 * TN];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < TN; ++j) v[r * TN + j] = acc[i][j][r];
    if (m < p.M) store_run<4 * TN>(p, c, ldc, !raw && p.c_bf16, raw || p.c_vec, m, n, v);
  }
}

// C = the partials' sum in split order.
__global__ __launch_bounds__(256) void reduce_kernel(GemmParams p) {
  const int64_t groups = p.ws_ld / 4;
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = e / groups, n = (e % groups) * 4;
  if (m >= p.M) return;
  const float *src = p.ws + m * p.ws_ld + n;
  float4 v = *reinterpret_cast<const float4 *>(src);
  for (int s = 1; s < p.ksplit; ++s) {
    const float4 w = *reinterpret_cast<const float4 *>(src + int64_t(s) * p.M * p.ws_ld);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n + j >= p.N) break;
    if (p.c_bf16) reinterpret_cast<uint16_t *>(p.c)[m * p.ldc + n + j] = f32_to_bf16(r[j]);
    else reinterpret_cast<float *>(p.c)[m * p.ldc + n + j] = r[j];
  }
}

int cu_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0)
      v = 256;
    return v;
  }();
  return n;
}

struct Plan {
  int bm, ksplit;
};

// Tile height by M; K split until the launch has two workgroups per CU, with at least
// four stages to a part.
Plan plan_of(int64_t M, int64_t N, int64_t stages) {
  Plan pl;
  pl.bm = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = ceil_div(M, pl.bm) * ceil_div(N, kBlock);
  int64_t s = tiles > 0 ? 2 * cu_count() / tiles : 1;
  s = s < stages / 4 ? s : stages / 4;
  pl.ksplit = int(s < 1 ? 1 : s > 16 ? 16 : s);
  return pl;
}

int64_t ws_ld_of(int64_t N) { return ceil_div(N, 4) * 4; }
size_t plan_bytes(const Plan &pl, int64_t M, int64_t N) {
  return pl.ksplit > 1 ? size_t(pl.ksplit) * size_t(M) * size_t(ws_ld_of(N)) * sizeof(float) : 0;
}

Operand operand_of(const fp8_tensor *t) {
  return Operand{t->codes, t->scales, t->rows, padded_cols(t->cols), scale_row(t->rows, t->two_d), t->two_d != 0};
}

template <bool FAST>
hipError_t run(GemmParams &p, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  Plan pl = plan_of(p.M, p.N, p.stages);
  if (plan_bytes(pl, p.M, p.N) > ws_bytes) pl.ksplit = 1;
  p.ksplit = pl.ksplit;
  p.ws = static_cast<float *>(ws);
  p.ws_ld = ws_ld_of(p.N);
  const int64_t esz = p.c_bf16 ? 2 : 4;
  p.c_vec = (reinterpret_cast<uintptr_t>(p.c) & 15u) == 0 && (p.ldc * esz) % 16 == 0;
  const dim3 grid(unsigned(ceil_div(p.M, pl.bm) * ceil_div(p.N, kBlock) * pl.ksplit)), blk(256);
  hipError_t e;
  if (pl.bm == 16) e = launch(gemm_kernel<16, 128, 1, 4, 4, FAST>, grid, blk, stream, p);
  else if (pl.bm == 32) e = launch(gemm_kernel<32, 128, 1, 4, 4, FAST>, grid, blk, stream, p);
  else if (pl.bm == 64) e = launch(gemm_kernel<64, 128, 1, 4, 3, FAST>, grid, blk, stream, p);
  else e = launch(gemm_kernel<128, 128, 2, 2, 2, FAST>, grid, blk, stream, p);
  if (e != hipSuccess || pl.ksplit == 1) return e;
  return launch(reduce_kernel, dim3(unsigned(ceil_div(p.M * (p.ws_ld / 4), 256))), blk, stream, p);
}

}  // namespace

size_t gemm_ws_bytes(int64_t M, int64_t N, int64_t stages) { return plan_bytes(plan_of(M, N, stages), M, N); }

hipError_t launch_gemm(const fp8_tensor *a, const fp8_tensor *b, void *c, fp4_dtype c_dtype, int64_t ldc, bool fast,
                       void *ws, size_t ws_bytes, hipStream_t stream) {
  GemmParams p{};
  p.a[0] = p.a[1] = operand_of(a);
  p.b[0] = p.b[1] = operand_of(b);
  p.M = a->rows;
  p.N = b->rows;
  p.kb = p.stages = int(ceil_div(a->cols, kBlock));
  p.c = c;
  p.ldc = ldc;
  p.c_bf16 = c_dtype == FP4_BF16;
  return fast ? run<true>(p, ws, ws_bytes, stream) : run<false>(p, ws, ws_bytes, stream);
}

hipError_t launch_gemm_sum(const fp8_tensor *a1, const fp8_tensor *b1, const fp8_tensor *a2, const fp8_tensor *b2,
                           void *c, fp4_dtype c_dtype, int64_t ldc, void *ws, size_t ws_bytes, hipStream_t stream) {
  GemmParams p{};
  p.a[0] = operand_of(a1);
  p.a[1] = operand_of(a2);
  p.b[0] = operand_of(b1);
  p.b[1] = operand_of(b2);
  p.M = a1->rows;
  p.N = b1->rows;
  p.kb = int(ceil_div(a1->cols, kBlock));
  p.stages = 2 * p.kb;
  p.c = c;
  p.ldc = ldc;
  p.c_bf16 = c_dtype == FP4_BF16;
  return run<true>(p, ws, ws_bytes, stream);
}

}  // namespace fp8
}  // namespace nvfp4
