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
#include <stddef.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "fp8.hpp"

namespace nvfp4 {
namespace fp8 {

namespace {

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
  int64_t m_first;     // this launch's tiles begin at row m_first, num_m rows of them
  int num_m;
  int kb;              // K blocks of a pair
  int stages;          // in all
  void *c;
  int64_t ldc;
  int c_bf16, c_vec;   // c_vec: 16-byte stores of whole groups are aligned
  int ksplit;
  int raw;             // the results go to ws: raw partials [ksplit][M][ws_ld]
  int dual;            // > 0: tile columns from `dual` on read b[1] (not a second pair) and
                       // their partials follow b[0]'s: the gated block's two projections
  float *ws;
  int64_t ws_ld;
  LoraAdd lora;        // the kernels with LORA
};

// A raw buffer's descriptor from wave-uniform values, which the compiler may hold in vector
// registers.
__device__ __forceinline__ u32x4 uniform_rsrc(uint64_t a, uint32_t bytes) {
  return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a))),
               uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a >> 32))) & 0xFFFFu,
               uint32_t(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
}

// Buffer of `bytes` bytes at the wave-uniform p for the epilogues' loads and stores:
// accesses past it (offset and scalar offset together) read zeros and write nothing, so
// a tile that sticks out of a tensor needs no tests of its rows.  The sum of a caller's
// offset and scalar offset stays below kOutside; kOutside in the offset's place comes with
// a scalar offset below 2^30, so that it is past every buffer and the sum does not wrap.
constexpr uint32_t kOutside = 0xC0000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(a)), hi = __builtin_amdgcn_readfirstlane(uint32_t(a >> 32));
  const int64_t most = kOutside - 1u;
  const int n = __builtin_amdgcn_readfirstlane(int(uint32_t(bytes < 0 ? 0 : bytes < most ? bytes : most)));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>((uint64_t(hi) << 32) | lo), short(0), n, 0x00020000);
}
__device__ __forceinline__ uint4 buf_load16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, int(voff), int(soff), 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void buf_store16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, const uint4 &w) {
  __builtin_amdgcn_raw_buffer_store_b128(u32x4{w.x, w.y, w.z, w.w}, r, int(voff), int(soff), 0);
}

// DMA from a buffer into LDS: lane l reads voffset + soffset (zeros where that sum is at
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

// A wave-uniform value in a scalar register: integer division runs on the vector unit,
// and what is computed from its result would stay there.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// An address in scalar registers for good: the compiler would load the kernel's arguments
// again in every stage, and wait for them together with the LDS reads.
__device__ __forceinline__ uint64_t base_of(const uint8_t *ptr) {
  const uint64_t a = reinterpret_cast<uint64_t>(ptr);
  uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(a)), hi = __builtin_amdgcn_readfirstlane(uint32_t(a >> 32));
  asm volatile("" : "+s"(lo), "+s"(hi));
  return (uint64_t(hi) << 32) | lo;
}
__device__ __forceinline__ uint64_t pick(bool second, uint64_t x, uint64_t y) { return second ? y : x; }

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

__device__ __forceinline__ float scale_value(uint32_t word, int byte) {
  return __uint_as_float(((word >> (8 * byte)) & 0xFFu) << 23);
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
// Low-rank adapters: row m gets coef[m] b_i^T, i its adapter, the two or three bf16 of each
// coefficient side by side along the contraction (with two a rank of 16 is one 16 x 16 x 32
// matrix instruction a tile).  They are what the accumulators begin with, while
// the first stages are on their way to LDS: the registers of the operands are still free and
// the main loop and its epilogue are those without adapters.  (Added to the results at their
// end, next to 256 accumulators, they took 16 us a 256 x 256 tile where the registers
// sufficed, and 50 where they did not.)  A dropout of the adapters' part is then one of the
// accumulators.
//
// A wave goes through the adapters of its rows, first come first, and takes the other rows'
// coefficients as zeros.  An infinity or NaN in b must not meet those zeros: unless all of
// the wave's rows have the adapter, such elements are taken as zeros too, and the columns that
// had one get an infinity in the adapter's rows, 3e38 * 3e38, at the end.

__device__ __forceinline__ int lora_index(const LoraAdd &o, int64_t m, int64_t M) {
  const int i = m >= M ? -1 : o.index ? o.index[m] : 0;
  return i < o.count ? i : -1;
}

__device__ __forceinline__ f32x4 lora_mfma(const bf16x8 &b, const bf16x8 &a, const f32x4 &c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 lora_mfma(const bf16x8 &b, const bf16x8 &a, const f32x16 &c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
}

// w without its infinities and NaNs; whether there were any
__device__ __forceinline__ bool lora_finite(bf16x8 &w) {
  u32x4 v = __builtin_bit_cast(u32x4, w);
  bool some = false;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const bool lo = (v[d] & 0x7F80u) == 0x7F80u, hi = (v[d] & 0x7F800000u) == 0x7F800000u;
    v[d] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
    some = some || lo || hi;
  }
  w = __builtin_bit_cast(bf16x8, v);
  return some;
}

// acc[i][j] += what the adapters idx[i] of the rows add.  V is a tile's accumulator (f32x4: 16
// x 16, contraction 32; f32x16: 32 x 32, contraction 16); the lane has rows m0 + i of the
// result, supplies rows n_row + j of b and, of each step of the contraction, the values from
// 8 kg on; its elements 4 t + r of tiles j are columns n_col + 8 TN t + r TN + j.  U steps have
// their loads in flight together.  No branch stands around a change of the accumulators, which
// would be copied where its sides meet: what is past the end is multiplied as zeros.  DROP:
// the accumulators, the adapters' part alone, are then dropped out.  Measured, us with and
// without adapters: 4096 x 20480 x 5120 by the 8-bit instruction 374 and 322 (rank 64), with
// the dropout 4096 x 5120 x 20480 365 and 319 (rank 16); 333 x 4100 x 4090 binary32, five
// adapters of 24, 37.8 and 31.8.  The adapters of a tile's rows come one after the other: an
// adapter's tokens belong next to each other (the call on 4096 tokens beside 20480 x 5120 with
// 16 adapters of 64: 459 us in runs, 1227 mixed).
template <int U, bool DROP, int TM, int TN, class V>
__device__ __forceinline__ void lora_add(const LoraAdd &o, int64_t M, int64_t N, int64_t m0, int64_t n_row,
                                         int64_t n_col, int kg, const int (&idx)[TM], V (&acc)[TM][TN]) {
  constexpr int kStep = sizeof(V) == 16 ? 32 : 16;
  uint32_t inside = 0, pending = 0;
  static_for<TM>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    inside |= m0 + i < M ? 1u << i : 0u;
    pending |= idx[i] >= 0 ? 1u << i : 0u;
  });
  for (;;) {
    const uint64_t some = __ballot(pending != 0);
    if (some == 0) break;
    int mine = 0;
    static_for<TM>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = TM - 1 - decltype(ic)::value;
      if ((pending >> i) & 1u) mine = idx[i];
    });
    const int cur = __builtin_amdgcn_readlane(mine, __builtin_ctzll(some));
    uint32_t match = 0;
    static_for<TM>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      match |= idx[i] == cur ? 1u << i : 0u;
    });
    pending &= ~match;
    const bool whole = __all(match == inside);
    uint32_t bad = 0;  // bit j: row n_row + j of the adapter's b holds an infinity or NaN
    const uint16_t *rows = o.b + (int64_t(cur) * N + n_row) * o.rank;
    const int width = o.parts * o.rank;
    for (int e0 = 0; e0 < width; e0 += U * kStep) {
      bf16x8 fa[U][TM], fb[U][TN];
      static_for<U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        const int e = e0 + u * kStep + 8 * kg, off = e < o.rank ? e : e < 2 * o.rank ? e - o.rank : e - 2 * o.rank;
        const bool live = e < width;
        static_for<TM>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          fa[u][i] = live && ((match >> i) & 1u)
                         ? *reinterpret_cast<const bf16x8 *>(o.coef + (m0 + i) * width + e) : bf16x8{};
        });
        static_for<TN>([&](auto jc) __attribute__((always_inline)) {
          constexpr int j = decltype(jc)::value;
          fb[u][j] = live && n_row + j < N ? *reinterpret_cast<const bf16x8 *>(rows + j * o.rank + off) : bf16x8{};
        });
      });
      if (!whole) {
        static_for<U>([&](auto uc) __attribute__((always_inline)) {
          static_for<TN>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            bad |= lora_finite(fb[decltype(uc)::value][j]) ? 1u << j : 0u;
          });
        });
      }
      static_for<U>([&](auto uc) __attribute__((always_inline)) {
        constexpr int u = decltype(uc)::value;
        static_for<TM>([&](auto ic) __attribute__((always_inline)) {
          constexpr int i = decltype(ic)::value;
          static_for<TN>([&](auto jc) __attribute__((always_inline)) {
            constexpr int j = decltype(jc)::value;
            acc[i][j] = lora_mfma(fb[u][j], fa[u][i], acc[i][j]);
          });
        });
      });
    }
    // every lane of a row of b knows what the others saw of it
    if constexpr (sizeof(V) == 16) bad |= uint32_t(__shfl_xor(int(bad), 16, 64));
    bad |= uint32_t(__shfl_xor(int(bad), 32, 64));
    const bf16x8 huge = kg == 0 ? bf16x8{__bf16(3e38f), 0, 0, 0, 0, 0, 0, 0} : bf16x8{};
    static_for<TM>([&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      const bf16x8 a = (match >> i) & 1u ? huge : bf16x8{};
      static_for<TN>([&](auto jc) __attribute__((always_inline)) {
        constexpr int j = decltype(jc)::value;
        acc[i][j] = lora_mfma((bad >> j) & 1u ? huge : bf16x8{}, a, acc[i][j]);
      });
    });
  }
  if constexpr (!DROP) return;
  const Mask mask(o.drop);
  static_for<TM>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    static_for<int(sizeof(V)) / 16>([&](auto tc) __attribute__((always_inline)) {
      constexpr int t = decltype(tc)::value;
      // 4 TN neighbouring columns are one or two of the generator's groups
      const uint64_t at = uint64_t(m0 + i) * uint64_t((N + 7) >> 3) + uint64_t((n_col + 8 * TN * t) >> 3);
      uint32_t kept = mask.bits(at);
      if constexpr (TN == 4) kept |= mask.bits(at + 1) << 8;
      static_for<TN>([&](auto jc) __attribute__((always_inline)) {
        constexpr int j = decltype(jc)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][4 * t + r] = (kept >> (r * TN + j)) & 1u ? acc[i][j][4 * t + r] : 0.0f;
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// The same with a dropout of the adapters' part, for accumulators that are zeros and too many
// to be changed one by one: a tile of rows at a time beside them, b read again for each.
template <int U, int TM, int TN, class V>
__device__ __forceinline__ void lora_rows(const LoraAdd &o, int64_t M, int64_t N, int64_t m0, int64_t n_row,
                                          int64_t n_col, int kg, const int (&idx)[TM], V (&acc)[TM][TN]) {
  static_for<TM>([&](auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    const int one[1] = {idx[i]};
    V more[1][TN];
    static_for<TN>([&](auto jc) __attribute__((always_inline)) { more[0][decltype(jc)::value] = V{}; });
    lora_add<U, true>(o, M, N, m0 + i, n_row, n_col, kg, one, more);
    static_for<TN>([&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      acc[i][j] = more[0][j];
    });
    __builtin_amdgcn_sched_barrier(0);
  });
}

// ---------------------------------------------------------------------------
// The general kernel: a BM x BN tile, WAVES_M x WAVES_N waves, NBUF stages of 128 K in
// LDS.  Stage layout: A codes [BM][128 B], B codes [BN][128 B], 256 B of A scales,
// 256 B of B scales.  LDS position P = 16 i + r of a wave's 16 T rows holds row T r + i:
// the 16 lanes that read tile i read neighbouring positions, and with chunk c at
// c ^ (P / 2) % 8 they cover all 64 banks.  Rows past the matrix come back as zeros (the
// buffer's range check) and their outputs are not stored.  All of a load's address but
// the lane's own row and chunk is scalar: with the tile's coordinates left in vector
// registers by the integer divisions, each load's descriptor was computed there, and a
// stage of 64 x 128 took 1.2 us.
// Few rows are bound by B's bytes: 4 x 20480 x 5120 17.6 us, 105 MB (6.0 TB/s; the operands
// partly in the last-level cache).  The binary32 sums of many rows by the matrix cores and
// the conversions between their instructions: 8192^3 1370 to 1420 TFLOP/s, the cores busy
// 57% of cycles at 1.95 GHz (a bf16 library product: 1330 to 1410 TFLOP/s).  Middle sizes
// run 7 us and about 0.46 us a stage: 333 x 4100 x 4090 21.7 us with 64 x 128 tiles, one
// workgroup to a CU and two stages of 24.5 KB on the way.
// LORA: 1 with low-rank adapters, in the first K part; 2 and a dropout of their part.
template <int BM, int BN, int WAVES_M, int WAVES_N, int NBUF, bool FAST, int LORA>
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
  const int num_m = p.num_m, num_n = p.dual ? 2 * p.dual : int((p.N + BN - 1) / BN);
  int tm, tn;
  const int split = scalar(int(blockIdx.x) % p.ksplit);
  tile_of(scalar(int(blockIdx.x) / p.ksplit), scalar(int(gridDim.x) / p.ksplit), num_m, num_n, tm, tn);
  tm = scalar(tm);
  tn = scalar(tn);
  const bool other = p.dual && tn >= p.dual;
  if (other) tn -= p.dual;
  const int64_t m0 = p.m_first + int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  const int s_begin = scalar(p.stages * split / p.ksplit), s_end = scalar(p.stages * (split + 1) / p.ksplit);

  // DMA instruction j of a wave fills the 8 positions from 8 (NW j + wave) on (modulo the
  // tile): P = 16 T w + 16 i + r of wave row w, whose row 16 T w + T r + i goes into the
  // scalar offset but for lane / 8 of r.  NW is even, so r / 8 is the wave's parity.
  const uint32_t ld = uint32_t(p.a[0].ld);
  auto row_of = [&](int j, int rows, int T) {
    const int P = ((j * NW + wave) * 8) % rows;
    return (P / (16 * T)) * 16 * T + ((P >> 4) % T) + (P & 8) * T;
  };
  const uint32_t chunk = uint32_t(((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) << 4);
  const uint32_t voff_a = uint32_t(lane >> 3) * uint32_t(TM) * ld + chunk;
  const uint32_t voff_b = uint32_t(lane >> 3) * uint32_t(TN) * ld + chunk;
  auto range_of = [&](int64_t rows, int64_t first, int most) {
    const int64_t left = rows - first;
    return uint32_t(left < most ? left : most) * ld;
  };
  const uint32_t a_range = range_of(p.a[0].rows, m0, BM), b_range = range_of(p.b[0].rows, n0, BN);
  // scales: even waves load A's, odd waves B's (several waves write the same bytes).  1D:
  // lane l the dword of rows 4 l .. 4 l + 3; 2D: lane l the byte of tile l.
  const bool sc_b = wave & 1;
  const int sc_2d = sc_b ? p.b[0].two_d : p.a[0].two_d;
  const int64_t sc_row = sc_b ? p.b[0].srow : p.a[0].srow;
  const int64_t sc_first = sc_2d ? (sc_b ? n0 : m0) / kBlock : (sc_b ? n0 : m0);
  const int64_t sc_left = sc_row - sc_first;
  const uint32_t sc_range = uint32_t(sc_left < 256 ? sc_left : 256), sc_step = uint32_t(sc_row);
  const uint64_t a0 = base_of(p.a[0].codes + m0 * int64_t(ld)), a1 = base_of(p.a[1].codes + m0 * int64_t(ld));
  const uint64_t b0 = base_of((other ? p.b[1].codes : p.b[0].codes) + n0 * int64_t(ld));
  const uint64_t b1 = base_of(p.b[1].codes + n0 * int64_t(ld));
  const uint64_t c0 = base_of((sc_b ? (other ? p.b[1].scales : p.b[0].scales) : p.a[0].scales) + sc_first);
  const uint64_t c1 = base_of((sc_b ? p.b[1].scales : p.a[1].scales) + sc_first);
  const int kb = p.kb, a2d = p.a[0].two_d, b2d = p.b[0].two_d;
  auto issue = [&](int s, int buf) {
    const bool live = s < s_end, second = s >= kb;
    const uint32_t kt = live ? uint32_t(s - (second ? kb : 0)) : 0u;
    uint8_t *base = lds + buf * STAGE;
    const u32x4 ra = uniform_rsrc(pick(second, a0, a1), live ? a_range : 0u);
    const u32x4 rb = uniform_rsrc(pick(second, b0, b1), live ? b_range : 0u);
#pragma unroll
    for (int j = 0; j < JA; ++j)
      dma16(ra, base + ((j * NW + wave) * 8) % BM * kBlock, voff_a, kt * kBlock + uint32_t(row_of(j, BM, TM)) * ld);
#pragma unroll
    for (int j = 0; j < JB; ++j)
      dma16(rb, base + (BM + ((j * NW + wave) * 8) % BN) * kBlock, voff_b,
            kt * kBlock + uint32_t(row_of(j, BN, TN)) * ld);
    const uint32_t at = kt * sc_step;
    const u32x4 rs = uniform_rsrc(pick(second, c0, c1), live ? at + sc_range : 0u);
    uint8_t *dst = base + S_OFF + 256 * (wave & 1);
    if (sc_2d) dma1(rs, dst, uint32_t(lane), at);
    else dma4(rs, dst, uint32_t(lane) * 4u, at);
  };

  const int wm = (wave / WAVES_N) * WM, wn = (wave % WAVES_N) * WN;
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int s = 0; s < NBUF - 1; ++s) issue(s_begin + s, s);
  if constexpr (LORA != 0) {
    if (split == 0) {
      int ids[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) ids[i] = lora_index(p.lora, m0 + wm + lr * TM + i, p.M);
      lora_add<BM <= 64 || (BM == 128 && LORA == 1) ? 2 : 1, LORA == 2>(p.lora, p.M, p.N, m0 + wm + lr * TM, n0 + wn + lr * TN,
                                             n0 + wn + 4 * lg * TN, lg, ids, acc);
    }
  }
  int buf = 0;
  for (int s = s_begin; s < s_end; ++s) {
    // stage s has landed for this wave, and its reads of the buffer that is refilled
    // next are done; past the barrier both hold for every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * NDMA) : "memory");
    __syncthreads();
    issue(s + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
    const uint8_t *base = lds + buf * STAGE;
    auto frag = [&](int tile) {  // the wave's tile that starts at position `tile`
      const uint8_t *r = base + (tile + lr) * kBlock;
      const uint4 x = *reinterpret_cast<const uint4 *>(r + ((lg ^ (lr >> 1)) << 4));
      const uint4 y = *reinterpret_cast<const uint4 *>(r + (((lg + 4) ^ (lr >> 1)) << 4));
      return i32x8{int(x.x), int(x.y), int(x.z), int(x.w), int(y.x), int(y.y), int(y.z), int(y.w)};
    };
    uint32_t sa[(TM + 3) / 4], sb[(TN + 3) / 4];
    if (a2d) {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(base + S_OFF + 4 * (wm / kBlock)) * 0x01010101u;
#pragma unroll
      for (int i = 0; i < (TM + 3) / 4; ++i) sa[i] = v;
    } else {
      read_scales<TM>(base + S_OFF + wm + lr * TM, sa);
    }
    if (b2d) {
      const uint32_t v = *reinterpret_cast<const uint32_t *>(base + S_OFF + 256 + 4 * (wn / kBlock)) * 0x01010101u;
#pragma unroll
      for (int i = 0; i < (TN + 3) / 4; ++i) sb[i] = v;
    } else {
      read_scales<TN>(base + S_OFF + 256 + wn + lr * TN, sb);
    }
    i32x8 fb[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = frag(BM + wn + 16 * j);
    if constexpr (!FAST) {
      i32x8 fa[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = frag(wm + 16 * i);
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
      const i32x8 fa = frag(wm + 16 * i);
      static_for<TN>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        acc[i][j] = mfma<(j & 3), (i & 3)>(fb[j], fa, acc[i][j], sb[j >> 2], sa[i >> 2]);
      });
    });
    buf = buf + 1 == NBUF ? 0 : buf + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no DMA into LDS outlives the workgroup

  const bool raw = p.raw;
  void *c = raw ? static_cast<void *>(p.ws + int64_t((other ? p.ksplit : 0) + split) * p.M * p.ws_ld) : p.c;
  const int64_t ldc = raw ? p.ws_ld : p.ldc;
  if (raw || p.c_vec) {
    const int64_t n = n0 + wn + 4 * lg * TN;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int64_t m = m0 + wm + lr * TM + i;
      float v[4 * TN];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < TN; ++j) v[r * TN + j] = acc[i][j][r];
      if (m < p.M) store_run<4 * TN>(p, c, ldc, !raw && p.c_bf16, true, m, n, v);
    }
    return;
  }
  // Rows of C that take no 16-byte stores: through LDS, so that an instruction's lanes
  // write neighbouring elements of a row (element by element from the registers, 64 lanes
  // wrote 64 places at a time).  A wave's results, binary32, in a region of its own and in
  // as many passes as fit there: pass x holds rows TM l + i of the TP values i from TP x
  // on, as rows TP l + i % TP, chunk c at c ^ l.
  constexpr int kPasses = (NW * WM * WN * 4 + NBUF * STAGE - 1) / (NBUF * STAGE), TP = TM / kPasses;
  static_assert(TM % kPasses == 0, "whole tiles to a pass");
  float *region = reinterpret_cast<float *>(lds) + wave * (WM / kPasses) * WN;
  constexpr int kChunks = WN / 4;
  const int col = lane % WN;
  static_for<kPasses>([&](auto pc) {
    constexpr int i0 = decltype(pc)::value * TP;
    __syncthreads();  // every wave's DMA has landed and its operands are read
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int k = 0; k < TN; ++k) {  // 4 of the lane's 4 TN neighbouring columns
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i0 + i][(4 * k + e) % TN][(4 * k + e) / TN];
        *reinterpret_cast<float4 *>(region + (lr * TP + i) * WN + (((lg * TN + k) ^ (lr & (kChunks - 1))) << 2)) =
            make_float4(v[0], v[1], v[2], v[3]);
      }
#pragma unroll 4
    for (int row = lane / WN; row < WM / kPasses; row += 64 / WN) {
      const int l = row / TP;
      const int64_t m = m0 + wm + l * TM + i0 + row % TP, n = n0 + wn + col;
      const float v = region[row * WN + ((((col >> 2) ^ (l & (kChunks - 1))) << 2) | (col & 3))];
      if (m < p.M && n < p.N) {
        if (p.c_bf16) reinterpret_cast<uint16_t *>(c)[m * ldc + n] = f32_to_bf16(v);
        else reinterpret_cast<float *>(c)[m * ldc + n] = v;
      }
    }
  });
}

// ---------------------------------------------------------------------------
// The main kernel: a 256 x 256 tile, four waves of 128 x 128, two stages of 128 K in
// LDS, and the 32 x 32 x 64 form of the instruction (4 x 4 tiles fill all 256
// accumulator registers; the 16 x 16 form's 64 small tuples did not fit the register
// allocator).  Lane l supplies row l % 32 and 32 of the 64 K values; tile i of a wave
// takes rows 4 (l % 32) + i, so a lane's four scales are one dword.  A wave's stage is
// four quarters,
//   Q0 = A0 B0,  Q1 = A0 B1,  Q2 = A1 B1,  Q3 = A1 B0   (A0 = its A tiles 0, 1, ...),
// of 8 MFMAs each.  Every quarter reads one half operand for a later one into registers
// that the quarter before it has freed (B1 of this stage during Q0, A1 during Q1, the
// next stage's A0 during Q2 and B0 during Q3, in B1's registers: B's two register sets
// swap roles from stage to stage), so 128 registers hold the operands of a pipeline
// that does not wait for LDS, and the LDS reads are spread evenly.  A half operand's
// 16 KB of LDS are refilled, for the stage after next, in the quarter after the one that
// read them: a barrier between quarters, and seven quarters for a load to arrive.  (One
// barrier a stage, with the whole buffer refilled after it, left four: 8192^3 ran at
// 2200 TFLOP/s and, with the loads taken out, at 2770.)
struct Problem {
  Operand a[2], b[2];  // stages [0, kb) read pair 0, [kb, 2 kb) pair 1
  int64_t M, N;
  int kb, stages;
  void *c;
  int64_t ldc;
  int c_bf16, c_vec;
  int num_m, num_n;
  int tile0;  // the problem's first tile in the launch's sequence
};

// The gated block's first half in one launch (kAct): B rows of a tile are 128 of wg
// (pair 0) and the same 128 of wu (pair 1), and the epilogue writes silu(g) * u
// quantized, and g and u where they are wanted.
struct ActOut {
  uint16_t *g, *u;  // bf16 [M][F], or null
  int vec;          // their rows take 16-byte stores
  uint8_t *codes, *scales;
  int64_t cols_p, srow;
};

// The gated block's backward: dh stays in the accumulators, and the epilogue (kDact)
// quantizes dg, du and h in both layouts.
struct DactArgs {
  const uint16_t *g, *u;  // bf16 [M][F], 16-byte aligned rows
  DactOut out;
};

// kLora: kStore with low-rank adapters; kLoraDrop: and a dropout of their part.
enum Epilogue { kStore, kAct, kDact, kLora, kLoraDrop };

struct BigParams {
  ActOut act;
  DactArgs dact;
  LoraAdd lora;
  Problem prob[kMaxProblems];
  int problems;
  int whole;   // tiles [0, whole) run unsplit, the others in `split` K parts
  int split;
  float *ws;   // raw partial tiles [256][256], item (tile - whole) * split + part
};

// Problem k of a kernel whose only argument is a BigParams, read from the kernel's
// arguments by address: an index into the argument itself would copy them all to private
// memory, and what is read back from there is not scalar.
typedef const __attribute__((address_space(4))) Problem ConstProblem;
__device__ __forceinline__ ConstProblem &problem_at(int k) {
  const auto args = (const __attribute__((address_space(4))) char *)__builtin_amdgcn_kernarg_segment_ptr();
  return reinterpret_cast<ConstProblem *>(args + offsetof(BigParams, prob))[k];
}

// tile of the launch's sequence -> problem, tile coordinates
__device__ __forceinline__ int big_tile(const BigParams &p, int tile, int &tm, int &tn) {
  int k = 0;
  if (p.problems > 1 && tile >= p.prob[1].tile0) k = 1;
  if (p.problems > 2 && tile >= p.prob[2].tile0) k = 2;
  auto of_problem = [&](int x, int y, int z) { return k == 0 ? x : k == 1 ? y : z; };
  const int l = tile - of_problem(p.prob[0].tile0, p.prob[1].tile0, p.prob[2].tile0);
  const int num_m = of_problem(p.prob[0].num_m, p.prob[1].num_m, p.prob[2].num_m);
  const int num_n = of_problem(p.prob[0].num_n, p.prob[1].num_n, p.prob[2].num_n);
  const int per_group = kGroupM * num_n;
  const int grp = l / per_group, first = grp * kGroupM;
  const int gsz = min(num_m - first, kGroupM);
  tm = first + (l % per_group) % gsz;
  tn = (l % per_group) / gsz;
  return k;
}

// 8 values to bf16, nearest-even, by the hardware's packed conversion (four instructions;
// rounding on the bits took five times as many).
__device__ __forceinline__ uint4 pack_bf16(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 x = {v[2 * j], v[2 * j + 1]};
    w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float bf16_at(const uint4 &w, int j) {
  const uint32_t v = (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w;
  return __uint_as_float((j & 1) ? (v & 0xFFFF0000u) : (v << 16));
}

// One accumulator into a vector register.  An explicit move, so that the epilogues read
// the 256 accumulators one by one as they use them: left to the compiler, they were
// moved (and spilled) wherever an epilogue branches.  The compiler does not see that the
// register was written by a matrix instruction: acc_settle comes first.
__device__ __forceinline__ float acc_read(const f32x16 &a, int r) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a[r]));
  return v;
}
// At least the 19 wait states from a 16-pass matrix instruction to a read of its result.
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// bf16 results leave through LDS, a wave's 128 rows of 256 bytes in a region of its own:
// a lane's 16-byte pieces of a row lie 32 or 64 bytes apart, and stored straight from the
// registers every instruction wrote 32 partial lines (kAct's g and u alone took 100 of
// 860 us at 4096x5120x20480).  16-byte chunk c of row 4 l + i sits at
// c ^ (l % 16) ^ 8 (i % 2): writes (16 lanes of one i) and reads (whole rows, or two halves
// of neighbouring rows) both cover all 64 banks.
__device__ __forceinline__ uint4 *staged(uint8_t *region, int l, int i, int c) {
  return reinterpret_cast<uint4 *>(region + (4 * l + i) * 256 + ((c ^ (l & 15) ^ ((i & 1) << 3)) << 4));
}
constexpr int kRegion = 128 * 256;
// A wave's staged rows to its 128 columns of the result, `inside` of them in it, rows cld
// bytes apart.
__device__ __forceinline__ void store_staged(uint8_t *region, __amdgpu_buffer_rsrc_t rc, uint32_t cld, int inside,
                                             bool vec, int lane) {
  if (!vec) {  // rows that take no 16-byte stores: half a row an instruction
    const uint32_t v0 = lane < inside ? 2u * lane : kOutside, v1 = 64 + lane < inside ? 2u * lane + 128u : kOutside;
#pragma unroll 4
    for (int row = 0; row < 128; ++row) {
      const int e = lane & 7, c = lane >> 3;
      const uint16_t x = reinterpret_cast<const uint16_t *>(staged(region, row >> 2, row & 3, c))[e];
      const uint16_t y = reinterpret_cast<const uint16_t *>(staged(region, row >> 2, row & 3, 8 + c))[e];
      __builtin_amdgcn_raw_buffer_store_b16(x, rc, int(v0), int(uint32_t(row) * cld), 0);
      __builtin_amdgcn_raw_buffer_store_b16(y, rc, int(v1), int(uint32_t(row) * cld), 0);
    }
    return;
  }
  // 4 rows of 256 bytes an instruction
  const int c = lane & 15, row = lane >> 4;
  const uint32_t v = 8 * c < inside ? uint32_t(row) * cld + 16u * c : kOutside;
#pragma unroll
  for (int k = 0; k < 32; ++k) buf_store16(rc, v, uint32_t(4 * k) * cld, *staged(region, k, row, c));
}

// kAct's epilogue.  Lane (l32, g) of wave column h holds rows m0 + wm + 4 l32 + i and, of
// each, columns n0 + 64 h + 16 t + 8 g + 2 r + j: gate in acc[i][j][4 t + r], up in
// acc[i][2 + j][4 t + r].  g and u are rounded to bf16 before silu, as the backward pass
// reads them.  A row's block maximum joins two lanes and, through LDS, two waves.
__device__ __forceinline__ void act_store(const ActOut &o, int64_t M, int64_t F, int64_t m0, int64_t n0, int wm, int h,
                                          int l32, int g, f32x16 (&acc)[4][4], uint8_t *region,
                                          float *lds) {
  const int64_t mw = m0 + wm, mb = mw + 4 * l32, nb = n0 + 64 * h;
  const uint32_t ld = uint32_t(F) * 2u, cld = uint32_t(o.cols_p);
  const int64_t left = M - mw;
  const __amdgpu_buffer_rsrc_t rg = buffer_of(o.g + mw * F + nb, o.g ? left * F * 2 - nb * 2 : 0);
  const __amdgpu_buffer_rsrc_t ru = buffer_of(o.u + mw * F + nb, o.g ? left * F * 2 - nb * 2 : 0);
  const __amdgpu_buffer_rsrc_t rc = buffer_of(o.codes + mw * o.cols_p + nb, left * o.cols_p - nb);
  const uint32_t code_at = uint32_t(4 * l32) * cld + 8u * g;
  // columns of the lane's that lie inside; past F a token with a NaN has NaNs, not zeros
  const int inside = int(F - nb < kBlock ? F - nb : int64_t(kBlock)) - 8 * g;
  uint32_t sb[4];
  // a row at a time: all four at once held 128 values across the exchange and made the
  // main loop spill
  static_for<4>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    float hv[4][8], mx = 0.0f;
    static_for<4>([&](auto tc) {
      constexpr int t = decltype(tc)::value;
      float a[8], b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = acc_read(acc[i][e & 1], 4 * t + (e >> 1));
        b[e] = acc_read(acc[i][2 + (e & 1)], 4 * t + (e >> 1));
      }
      const uint4 ga = pack_bf16(a), ub = pack_bf16(b);
      // columns 16 t + 8 g .. of the wave's 64: chunk 2 t + g of g's half, then u's
      *staged(region, l32, i, 2 * t + g) = ga;
      *staged(region, l32, i, 8 + 2 * t + g) = ub;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float gv = bf16_at(ga, e);
        const float x = gv * sigmoid(gv) * bf16_at(ub, e);
        hv[t][e] = 16 * t + e < inside ? x : 0.0f;
        mx = fmaxf(mx, __builtin_fabsf(hv[t][e]));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    // [row i][wave column][a value per lane of the tile's two wave rows]
    float *const slot = lds + 128 * i + (wm >> 2) + l32;
    if (g == 0) slot[64 * h] = mx;
    __syncthreads();
    sb[i] = scale_byte(fmaxf(mx, slot[64 * (h ^ 1)]));
    const float m = scale_of(sb[i]);
    static_for<4>([&](auto tc) {
      constexpr int t = decltype(tc)::value;
      const float (&x)[8] = hv[t];
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{encode4(x[0], x[1], x[2], x[3], m), encode4(x[4], x[5], x[6], x[7], m)},
                                            rc, int(code_at), int(uint32_t(i) * cld + 16u * t), 0);
    });
    __builtin_amdgcn_sched_barrier(0);
  });
  if (h == 0 && g == 0 && mb < o.srow)  // srow is a multiple of 16
    *reinterpret_cast<uint32_t *>(o.scales + (n0 / kBlock) * o.srow + mb) =
        sb[0] | (sb[1] << 8) | (sb[2] << 16) | (sb[3] << 24);
  const int lane = l32 + 32 * g;
  if (o.g && !o.vec) {
    // rows that take no 16-byte stores: a row of 64 columns an instruction
    const uint32_t v = nb + lane < F ? 2u * lane : kOutside;
#pragma unroll 4
    for (int row = 0; row < 128; ++row) {
      const int e = lane & 7;
      const uint16_t gv = reinterpret_cast<const uint16_t *>(staged(region, row >> 2, row & 3, lane >> 3))[e];
      const uint16_t uv = reinterpret_cast<const uint16_t *>(staged(region, row >> 2, row & 3, 8 + (lane >> 3)))[e];
      __builtin_amdgcn_raw_buffer_store_b16(gv, rg, int(v), int(uint32_t(row) * ld), 0);
      __builtin_amdgcn_raw_buffer_store_b16(uv, ru, int(v), int(uint32_t(row) * ld), 0);
    }
  } else if (o.g) {
    // 8 rows of 128 bytes an instruction; columns past F (a multiple of 8) would be the
    // next row's
    const int c = lane & 7;
    const uint32_t v = nb + 8 * c < F ? uint32_t(lane >> 3) * ld + 16u * c : kOutside;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int row = 8 * q + (lane >> 3);
      buf_store16(rg, v, uint32_t(8 * q) * ld, *staged(region, row >> 2, row & 3, c));
      buf_store16(ru, v, uint32_t(8 * q) * ld, *staged(region, row >> 2, row & 3, 8 + c));
    }
  }
}

// kDact's epilogue.  A wave's 128 x 128 of dh are whole blocks of both layouts.  Lane
// (l32, g) holds rows m = 4 l32 + i and columns n = 32 t + 16 g + 4 r + j of them in
// acc[i][j][4 t + r].  First the layout along F, a row at a time (its block is the lane's
// 64 columns and those of lane ^ 32); then the one along M, 8 columns at a time (a
// column's block is 4 rows of 32 lanes, so its codes leave as one dword a lane, 128
// bytes a column).  g and u are read, and silu taken, once for each: both layouts at
// once would need the three products of a whole tile in registers.  With one wave to a
// SIMD nothing else covers the loads, so each 16 bytes of g and u are replaced by those
// of the next row (the next columns) as soon as they are used.
// F is a multiple of 8.  Past F what is read of g and u is the next row's, whose infinities
// and NaNs times a dh of 0 are not 0: the codes there are set to 0 (a NaN does not enter
// the block's maximum), and in the other layout they go to rows that do not exist.
__device__ __forceinline__ void dact_store(const DactArgs &p, int64_t M, int64_t F, int64_t mb, int64_t nb, int l32,
                                           int g, f32x16 (&acc)[4][4]) {
  const DactOut &o = p.out;
  const int64_t left = M - mb;
  const uint32_t ld = uint32_t(F) * 2u, cld = uint32_t(o.dg.cols_p), tld = uint32_t(o.dg_t.cols_p);
  const __amdgpu_buffer_rsrc_t rg = buffer_of(p.g + mb * F + nb, left * F * 2 - nb * 2);
  const __amdgpu_buffer_rsrc_t ru = buffer_of(p.u + mb * F + nb, left * F * 2 - nb * 2);
  const uint32_t gu_at = uint32_t(4 * l32) * ld + 32u * g;
  // 8 columns 32 (h / 2) + 16 g + 8 (h % 2) of row i
  auto soff = [&](int i, int h) { return uint32_t(i) * ld + uint32_t(64 * (h >> 1) + 16 * (h & 1)); };
  uint32_t sg[4], su[4];
  {
    const __amdgpu_buffer_rsrc_t rdg = buffer_of(o.dg.codes + mb * o.dg.cols_p + nb, left * o.dg.cols_p - nb);
    const __amdgpu_buffer_rsrc_t rdu = buffer_of(o.du.codes + mb * o.dg.cols_p + nb, left * o.dg.cols_p - nb);
    const uint32_t at = uint32_t(4 * l32) * cld + 16u * g;
    uint4 ga[8], ua[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      ga[h] = buf_load16(rg, gu_at, soff(0, h));
      ua[h] = buf_load16(ru, gu_at, soff(0, h));
    }
    static_for<4>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      float dg[64], du[64], tg = 0.0f, tu = 0.0f;
      static_for<8>([&](auto hc) {
        constexpr int h = decltype(hc)::value, t = h >> 1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = acc_read(acc[i][e & 3], 4 * t + 2 * (h & 1) + (e >> 2)), gv = bf16_at(ga[h], e), s = sigmoid(gv);
          const float silu = gv * s;
          dg[8 * h + e] = d * bf16_at(ua[h], e) * dsilu(s, silu);
          du[8 * h + e] = d * silu;
          tg = fmaxf(tg, __builtin_fabsf(dg[8 * h + e]));
          tu = fmaxf(tu, __builtin_fabsf(du[8 * h + e]));
        }
        if constexpr (i < 3) {
          ga[h] = buf_load16(rg, gu_at, soff(i + 1, h));
          ua[h] = buf_load16(ru, gu_at, soff(i + 1, h));
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      sg[i] = scale_byte(fmaxf(tg, __shfl_xor(tg, 32, 64)));
      su[i] = scale_byte(fmaxf(tu, __shfl_xor(tu, 32, 64)));
      const float mg = scale_of(sg[i]), mu = scale_of(su[i]);
      static_for<4>([&](auto tc) {
        constexpr int t = decltype(tc)::value;
        uint32_t w[4], v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float *x = dg + 16 * t + 4 * e, *y = du + 16 * t + 4 * e;
          const bool inside = nb + 32 * t + 16 * g + 8 * (e >> 1) < F;
          w[e] = inside ? encode4(x[0], x[1], x[2], x[3], mg) : 0u;
          v[e] = inside ? encode4(y[0], y[1], y[2], y[3], mu) : 0u;
        }
        buf_store16(rdg, at, uint32_t(i) * cld + 32u * t, make_uint4(w[0], w[1], w[2], w[3]));
        buf_store16(rdu, at, uint32_t(i) * cld + 32u * t, make_uint4(v[0], v[1], v[2], v[3]));
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  if (g == 0 && mb + 4 * l32 < o.dg.srow) {  // srow is a multiple of 16
    const int64_t at = (nb / kBlock) * o.dg.srow + mb + 4 * l32;
    *reinterpret_cast<uint32_t *>(o.dg.scales + at) = sg[0] | (sg[1] << 8) | (sg[2] << 16) | (sg[3] << 24);
    *reinterpret_cast<uint32_t *>(o.du.scales + at) = su[0] | (su[1] << 8) | (su[2] << 16) | (su[3] << 24);
  }
  const int64_t t_base = nb * int64_t(tld) + mb, t_left = F * int64_t(tld) - t_base;
  const int64_t ts_base = (mb / kBlock) * o.dg_t.srow + nb;
  const __amdgpu_buffer_rsrc_t rt[3] = {buffer_of(o.dg_t.codes + t_base, t_left), buffer_of(o.du_t.codes + t_base, t_left),
                                        buffer_of(o.h_t.codes + t_base, t_left)};
  uint8_t *const ts[3] = {o.dg_t.scales + ts_base, o.du_t.scales + ts_base, o.h_t.scales + ts_base};
  const uint32_t t_at = 16u * g * tld + 4u * l32;
  // Rows past M count as 0: their codes read as zeros, but their scales are whatever the
  // caller's padding holds, and one that means NaN makes their dh NaN.
  // 8 columns of tensor T: v[e][i] the values of column 32 (h / 2) + 16 g + 8 (h % 2) + e
  auto columns = [&](auto tc, int h, const float (&v)[8][4]) {
    constexpr int T = decltype(tc)::value;
    uint32_t sb[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // from 0 on, so that four NaNs count as nothing: their bits are above every number's
      const float top = fmaxf(fmaxf(fmaxf(0.0f, __builtin_fabsf(v[e][0])), __builtin_fabsf(v[e][1])),
                              fmaxf(__builtin_fabsf(v[e][2]), __builtin_fabsf(v[e][3])));
      uint32_t x = row16_max_bits(__float_as_uint(top));
      x = max(x, uint32_t(__builtin_amdgcn_ds_swizzle(int(x), 0x401F)));  // lane ^ 16
      sb[e] = scale_byte(__uint_as_float(x));
    }
    const int n = 32 * (h >> 1) + 8 * (h & 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      __builtin_amdgcn_raw_buffer_store_b32(encode4(v[e][0], v[e][1], v[e][2], v[e][3], scale_of(sb[e])), rt[T],
                                            int(t_at), int(uint32_t(n + e) * tld), 0);
    }
    if (l32 == 0 && nb + n + 16 * g < o.dg_t.srow)
      *reinterpret_cast<uint2 *>(ts[T] + n + 16 * g) = make_uint2(sb[0] | (sb[1] << 8) | (sb[2] << 16) | (sb[3] << 24),
                                                                 sb[4] | (sb[5] << 8) | (sb[6] << 16) | (sb[7] << 24));
  };
  // 16 neighbouring columns at a time, so that a 32-byte piece of a row is read by loads
  // that follow one another
  uint4 ga[4][2], ua[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ga[i][k] = buf_load16(rg, gu_at, soff(i, k));
      ua[i][k] = buf_load16(ru, gu_at, soff(i, k));
    }
  static_for<8>([&](auto hc) {
    constexpr int h = decltype(hc)::value, t = h >> 1;
    float dg[8][4], du[8][4], hv[8][4];
    static_for<4>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float acc_v = acc_read(acc[i][e & 3], 4 * t + 2 * (h & 1) + (e >> 2));
        const float d = 4 * l32 + i < left ? acc_v : 0.0f;
        const float gv = bf16_at(ga[i][h & 1], e), uv = bf16_at(ua[i][h & 1], e);
        const float s = sigmoid(gv), silu = gv * s;
        dg[e][i] = d * uv * dsilu(s, silu);
        du[e][i] = d * silu;
        hv[e][i] = silu * uv;
      }
      if constexpr ((h & 1) && h < 7) {
        ga[i][0] = buf_load16(rg, gu_at, soff(i, h + 1));
        ga[i][1] = buf_load16(rg, gu_at, soff(i, h + 2));
        ua[i][0] = buf_load16(ru, gu_at, soff(i, h + 1));
        ua[i][1] = buf_load16(ru, gu_at, soff(i, h + 2));
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    columns(std::integral_constant<int, 0>{}, h, dg);
    columns(std::integral_constant<int, 1>{}, h, du);
    columns(std::integral_constant<int, 2>{}, h, hv);
    __builtin_amdgcn_sched_barrier(0);
  });
}

// Measured (TFLOP/s): kStore 2580 at 8192^3, 2700 at 4096 x 20480 x 5120; three weight
// gradients in one launch 2430 (4096 tokens, 5120, 20480), the matrix cores busy 65% of
// cycles at 1.67 GHz, a clock that the power limit sets.  kAct 2260 to 2320 there, 742 to 761
// us.  kDact 603 us of which the product is 305: its epilogue reads and writes 756 MB with
// one wave to a SIMD, and the matrix cores wait.
template <Epilogue EPI>
__global__ __launch_bounds__(256) void gemm256_kernel(BigParams p) {
  constexpr bool ACT = EPI == kAct;
  constexpr int kTileN = ACT ? kBig / 2 : kBig;  // columns of the result per tile
  // a stage: codes; 256 B each of A's and B's 1 x 128 scales, of A's and B's tile
  // scales and (kAct) of wu's
  constexpr int S_OFF = 2 * kBig * kBlock, STAGE = S_OFF + 1280;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);

  // consecutive workgroups go to different XCDs: each XCD takes a contiguous run
  int item = int(blockIdx.x), part = 0, parts = 1, tile;
  if (item < p.whole) {
    tile = (p.whole & 7) == 0 ? (item & 7) * (p.whole >> 3) + (item >> 3) : item;
  } else {
    const int n = int(gridDim.x) - p.whole;
    item -= p.whole;
    if ((n & 7) == 0) item = (item & 7) * (n >> 3) + (item >> 3);
    parts = p.split;
    part = scalar(item % parts);
    tile = p.whole + scalar(item / parts);
  }
  int tm, tn;
  const int k = scalar(big_tile(p, tile, tm, tn));
  tm = scalar(tm);
  tn = scalar(tn);
  const ConstProblem &q = problem_at(k);
  const int64_t m0 = int64_t(tm) * kBig, n0 = int64_t(tn) * kTileN;
  const int kb = q.kb;
  const int s_begin = int(int64_t(q.stages) * part / parts), s_end = int(int64_t(q.stages) * (part + 1) / parts);

  // LDS position P = 128 h + 32 i + l of an operand holds row 128 h + 4 l + i, so that
  // the 32 lanes that read tile i of half h read neighbouring positions: both parities
  // of the 128-byte rows and, with chunk c at c ^ (P / 2) % 8, all 64 banks.  DMA
  // instruction j of a wave fills positions 32 j + 8 wave + lane / 8, 16 bytes a lane;
  // the row of i and h goes into the scalar offset.  Rows past the operand read as zeros
  // (the range check is on the whole offset).
  // kAct: B's position 128 h + 32 i + l holds row 64 h + 2 l + i % 2 of wg (i < 2) or wu.
  const uint32_t ld = uint32_t(q.a[0].ld);
  const int dl = 8 * wave + (lane >> 3);  // position within a tile
  const uint32_t chunk = uint32_t(((lane & 7) ^ ((dl >> 1) & 7)) << 4);
  const uint32_t voff_a = uint32_t(4 * dl) * ld + chunk, voff_b = uint32_t((ACT ? 2 : 4) * dl) * ld + chunk;
  const int64_t am = q.a[0].rows - m0, bn = q.b[0].rows - n0;
  const uint32_t a_range = uint32_t(am < kBig ? am : kBig) * ld, b_range = uint32_t(bn < kTileN ? bn : kTileN) * ld;
  // scales: even waves load A's, odd waves B's (two waves write the same bytes)
  const bool sc_b = wave & 1;
  const int sc_2d = sc_b ? q.b[0].two_d : q.a[0].two_d;
  const int64_t sc_row = sc_b ? q.b[0].srow : q.a[0].srow;
  const int64_t sc_first = sc_2d ? (sc_b ? n0 : m0) / kBlock : (sc_b ? n0 : m0);
  const int64_t sc_left = sc_row - sc_first;
  const uint64_t a_base0 = base_of(q.a[0].codes + m0 * int64_t(ld)), a_base1 = base_of(q.a[1].codes + m0 * int64_t(ld));
  const uint64_t b_base0 = base_of(q.b[0].codes + n0 * int64_t(ld)), b_base1 = base_of(q.b[1].codes + n0 * int64_t(ld));
  const uint64_t s_base0 = base_of((sc_b ? q.b[ACT && wave == 3 ? 1 : 0].scales : q.a[0].scales) + sc_first);
  const uint64_t s_base1 = base_of((sc_b ? q.b[1].scales : q.a[1].scales) + sc_first);
  const uint32_t sc_range = uint32_t(sc_left < kBig ? sc_left : kBig), sc_step = uint32_t(sc_row);
  // K block and pair of stage s; past the end the DMA reads an empty range (zeros)
  struct Aim {
    uint32_t kt;
    bool live, second;
  };
  auto aim = [&](int s) {
    const bool second = s >= kb, live = s < s_end;
    return Aim{live ? uint32_t(s - (second ? kb : 0)) : 0u, live, second};
  };
  // DMA instruction d = 0..3 of half h of A (or B) into buffer `buf`
  auto dma_a = [&](const Aim &m, int buf, int h, int d) {
    const int j = 4 * (d >> 1) + 2 * h + (d & 1);
    dma16(uniform_rsrc(pick(m.second, a_base0, a_base1), m.live ? a_range : 0u),
          lds + buf * STAGE + (32 * j + 8 * wave) * kBlock, voff_a,
          m.kt * kBlock + uint32_t(128 * (j >> 2) + (j & 3)) * ld);
  };
  auto dma_b = [&](const Aim &m, int buf, int h, int d) {
    const int j = 4 * (d >> 1) + 2 * h + (d & 1);
    dma16(uniform_rsrc(ACT ? (h ? b_base1 : b_base0) : pick(m.second, b_base0, b_base1), m.live ? b_range : 0u),
          lds + buf * STAGE + (kBig + 32 * j + 8 * wave) * kBlock, voff_b,
          m.kt * kBlock + uint32_t(ACT ? 64 * (j >> 2) + (j & 1) : 128 * (j >> 2) + (j & 3)) * ld);
  };
  // scales: a dword a lane of 1 x 128 ones (d = 0) and a byte a lane of tiles' (d = 1); the
  // kind that the operand does not have writes zeros to a place of its own, which costs
  // less than a branch in the loop
  auto dma_s = [&](const Aim &m, int buf, int d) {
    const bool on = m.live && (d == 0) == !sc_2d;
    const uint32_t at = m.kt * sc_step;
    const u32x4 r = uniform_rsrc(pick(m.second, s_base0, s_base1), on ? at + sc_range : 0u);
    uint8_t *dst = lds + buf * STAGE + S_OFF + (sc_b ? 256 : 0);
    if (d == 0) dma4(r, dst, 4u * uint32_t(lane), at);
    else dma1(r, dst + (ACT && wave == 3 ? 768 : 512), uint32_t(lane), at);
  };

  const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128;
  // LDS: read r = 0..3 of a tile (16 of a lane's 64 bytes) takes chunk 2 r + g
  const int l32 = lane & 31, g = lane >> 5;
  uint32_t fa_at[4], fb_at[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint32_t ch = uint32_t(((2 * r + g) ^ ((l32 >> 1) & 7)) << 4);
    fa_at[r] = uint32_t((wm + l32) * kBlock) + ch;
    fb_at[r] = uint32_t((kBig + wn + l32) * kBlock) + ch;
  }
  const int a2d = q.a[0].two_d, b2d = q.b[0].two_d;
  const uint32_t sa_at = S_OFF + (a2d ? uint32_t(512 + 4 * (wm / kBlock)) : uint32_t(wm + 4 * l32));
  const uint32_t sb_at = S_OFF + 256 + (b2d ? uint32_t(512 + 4 * (wn / kBlock)) : uint32_t(wn + 4 * l32));
  const uint32_t sa_mul = a2d ? 0x01010101u : 1u, sb_mul = b2d ? 0x01010101u : 1u;
  const uint32_t sg_at = S_OFF + 768, su_at = S_OFF + 1024;  // kAct: the tile's scales of wg and wu

  // operands of a half: [tile][K step of 64], 8 dwords a lane
  i32x8 fa[2][2][2], fb[2][2][2];
  uint32_t sa[2], sb[2], su[2];  // by the stage's parity; su: kAct
  auto put = [](i32x8 &f, int half, const uint4 &v) {
    f[4 * half] = int(v.x);
    f[4 * half + 1] = int(v.y);
    f[4 * half + 2] = int(v.z);
    f[4 * half + 3] = int(v.w);
  };
  // read x = 0..7 of half h from buffer `buf`: K step x / 4, tile (x / 2) % 2, part x % 2
  auto read_a = [&](int buf, int h, int x) {
    const int st = x >> 2, i = (x >> 1) & 1, part_ = x & 1;
    put(fa[h][i][st], part_, *reinterpret_cast<const uint4 *>(lds + buf * STAGE + fa_at[2 * st + part_] + 32 * (2 * h + i) * kBlock));
  };
  auto read_b = [&](int buf, int h, int set, int x) {
    const int st = x >> 2, i = (x >> 1) & 1, part_ = x & 1;
    put(fb[set][i][st], part_, *reinterpret_cast<const uint4 *>(lds + buf * STAGE + fb_at[2 * st + part_] + 32 * (2 * h + i) * kBlock));
  };
  auto read_scales = [&](int buf) {
    sa[buf] = *reinterpret_cast<const uint32_t *>(lds + buf * STAGE + sa_at);
    if constexpr (ACT) {
      sb[buf] = *reinterpret_cast<const uint32_t *>(lds + buf * STAGE + sg_at);
      su[buf] = *reinterpret_cast<const uint32_t *>(lds + buf * STAGE + su_at);
    } else {
      sb[buf] = *reinterpret_cast<const uint32_t *>(lds + buf * STAGE + sb_at);
    }
  };
  // a byte per tile: a tile scale is every tile's (kAct: wg's for tiles 0, 1, wu's for 2, 3)
  auto spread_scales = [&](int buf) {
    sa[buf] *= sa_mul;
    if constexpr (ACT) sb[buf] = __builtin_amdgcn_perm(su[buf], sb[buf], 0x04040000u);
    else sb[buf] *= sb_mul;
  };

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};

  // 8 MFMAs of A half HA and B half HB (in register set SET) of a stage of parity PAR;
  // slot k also runs extra(k)
  auto quarter = [&](auto hac, auto hbc, auto setc, auto parc, auto &&extra) {
    constexpr int HA = decltype(hac)::value, HB = decltype(hbc)::value, SET = decltype(setc)::value;
    constexpr int PAR = decltype(parc)::value;
    static_for<8>([&](auto kc) {
      constexpr int kk = decltype(kc)::value, st = kk >> 2, i = (kk >> 1) & 1, j = kk & 1;
      acc[2 * HA + i][2 * HB + j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          fb[SET][j][st], fa[HA][i][st], acc[2 * HA + i][2 * HB + j], 0, 0, 2 * HB + j, int(sb[PAR]), 2 * HA + i,
          int(sa[PAR]));
      extra(kc);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  // Between quarters: this wave's LDS reads are done, and of its DMA all but the newest
  // N instructions have landed; past the barrier both hold for every wave.
  auto join = [&](auto nc) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(nc)::value) : "memory");
    __syncthreads();
  };
  // A stage, its data in buffer PAR and its B0 in register set PAR.  DMA per quarter: Q0
  // B0 and the scales (6 instructions), Q1 B1, Q2 A1 (4 each) of stage s + 2, Q3 A0 of
  // stage s + 3; the counts below are those issued after the half that the next quarter
  // reads.
  auto stage = [&](auto parc, int s) {
    constexpr int PAR = decltype(parc)::value;
    using P0 = std::integral_constant<int, PAR>;
    using P1 = std::integral_constant<int, PAR ^ 1>;
    const Aim next = aim(s + 2), after = aim(s + 3);
    quarter(I0{}, I0{}, P0{}, P0{}, [&](auto kc) {
      constexpr int kk = decltype(kc)::value;
      if constexpr (kk < 4) {
        read_b(PAR, 1, PAR ^ 1, 2 * kk);
        read_b(PAR, 1, PAR ^ 1, 2 * kk + 1);
        dma_b(next, PAR, 0, kk);
      } else if constexpr (kk < 6) {
        dma_s(next, PAR, kk - 4);
      }
    });
    join(std::integral_constant<int, 28>{});
    quarter(I0{}, I1{}, P1{}, P0{}, [&](auto kc) {
      constexpr int kk = decltype(kc)::value;
      if constexpr (kk < 4) {
        read_a(PAR, 1, 2 * kk);
        read_a(PAR, 1, 2 * kk + 1);
        dma_b(next, PAR, 1, kk);
      }
    });
    join(std::integral_constant<int, 28>{});
    quarter(I1{}, I1{}, P1{}, P0{}, [&](auto kc) {
      constexpr int kk = decltype(kc)::value;
      if constexpr (kk < 4) {
        read_a(PAR ^ 1, 0, 2 * kk);
        read_a(PAR ^ 1, 0, 2 * kk + 1);
        dma_a(next, PAR, 1, kk);
      }
    });
    join(std::integral_constant<int, 26>{});
    quarter(I1{}, I0{}, P0{}, P0{}, [&](auto kc) {
      constexpr int kk = decltype(kc)::value;
      if constexpr (kk == 0) read_scales(PAR ^ 1);
      if constexpr (kk < 4) {
        read_b(PAR ^ 1, 0, PAR ^ 1, 2 * kk);
        read_b(PAR ^ 1, 0, PAR ^ 1, 2 * kk + 1);
        dma_a(after, PAR ^ 1, 0, kk);
      }
      if constexpr (kk == 6) spread_scales(PAR ^ 1);
    });
    join(std::integral_constant<int, 26>{});
  };

  // stages 0 and 1, and A0 of stage 2 once A0 of stage 0 has been read, in the loop's order
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const Aim m = aim(s_begin + b);
#pragma unroll
    for (int d = 0; d < 4; ++d) dma_a(m, b, 0, d);
#pragma unroll
    for (int d = 0; d < 4; ++d) dma_b(m, b, 0, d);
    dma_s(m, b, 0);
    dma_s(m, b, 1);
#pragma unroll
    for (int d = 0; d < 4; ++d) dma_b(m, b, 1, d);
#pragma unroll
    for (int d = 0; d < 4; ++d) dma_a(m, b, 1, d);
  }
  if constexpr (EPI == kLora || EPI == kLoraDrop) {
    if (part == 0) {
      int ids[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ids[i] = lora_index(p.lora, m0 + wm + 4 * l32 + i, q.M);
      const int64_t m = m0 + wm + 4 * l32, n_row = n0 + wn + 4 * l32, n_col = n0 + wn + 16 * g;
      if constexpr (EPI == kLora) lora_add<2, false>(p.lora, q.M, q.N, m, n_row, n_col, g, ids, acc);
      else lora_rows<2>(p.lora, q.M, q.N, m, n_row, n_col, g, ids, acc);
    }
  }
  join(std::integral_constant<int, 26>{});
  read_scales(0);
#pragma unroll
  for (int x = 0; x < 8; ++x) read_a(0, 0, x);
#pragma unroll
  for (int x = 0; x < 8; ++x) read_b(0, 0, 0, x);
  spread_scales(0);
  join(std::integral_constant<int, 22>{});
  const Aim third = aim(s_begin + 2);
#pragma unroll
  for (int d = 0; d < 4; ++d) dma_a(third, 0, 0, d);
  // stages in pairs: past an odd count, one of zeros (a third copy of the stage for it made
  // the accumulators spill where the copies meet)
  for (int s = s_begin; s < s_end; s += 2) {
    stage(I0{}, s);
    stage(I1{}, s + 1);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no DMA into LDS outlives the workgroup
  acc_settle();

  if constexpr (ACT) {
    __syncthreads();  // every wave's DMA has landed: the LDS is free
    act_store(p.act, q.M, q.N, m0, n0, wm, wave & 1, l32, g, acc, lds + wave * kRegion,
              reinterpret_cast<float *>(lds + 4 * kRegion));
    return;
  }
  if constexpr (EPI == kDact) {
    const int64_t mb = m0 + wm, nb = n0 + wn;
    if (mb >= q.M || nb >= q.N) return;
    dact_store(p.dact, q.M, q.N, mb, nb, l32, g, acc);
    return;
  }
  const bool raw = parts > 1;
  GemmParams o{};
  o.N = raw ? kBig : q.N;
  const int64_t M = raw ? kBig : q.M;
  void *c = raw ? static_cast<void *>(p.ws + int64_t(item) * (kBig * kBig)) : q.c;
  const int64_t ldc = raw ? kBig : q.ldc;
  const int64_t mb = (raw ? 0 : m0) + wm + 4 * l32, nb = (raw ? 0 : n0) + wn + 16 * g;
  const bool bf16 = !raw && q.c_bf16;
  if (raw || q.c_vec || (bf16 && ldc < (int64_t(1) << 21))) {
    // c_vec: whole groups of 16 bytes are inside or outside the result together
    const int64_t mw = (raw ? 0 : m0) + wm, nw = (raw ? 0 : n0) + wn;
    const uint32_t esz = bf16 ? 2u : 4u, cld = uint32_t(ldc) * esz;
    const __amdgpu_buffer_rsrc_t rc = buffer_of(static_cast<uint8_t *>(c) + (mw * ldc + nw) * esz,
                                                ((M - mw - 1) * ldc + o.N - nw) * esz);
    const uint32_t at = uint32_t(4 * l32) * cld + uint32_t(16 * g) * esz;
    auto blocks = [&](auto &&store) {
      static_for<4>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        static_for<4>([&](auto tc) {
          constexpr int tt = decltype(tc)::value;
          float v[16];
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * r + j] = acc_read(acc[i][j], 4 * tt + r);
          store(v, nb + 32 * tt, uint32_t(i) * cld + uint32_t(32 * tt) * esz);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
    };
    if (bf16) {
      __syncthreads();  // every wave's DMA has landed: the LDS is free
      uint8_t *region = lds + wave * kRegion;
      static_for<4>([&](auto ic) {
        constexpr int i = decltype(ic)::value;
        static_for<4>([&](auto tc) {
          constexpr int tt = decltype(tc)::value;
          float lo[8], hi[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            lo[e] = acc_read(acc[i][e & 3], 4 * tt + (e >> 2));
            hi[e] = acc_read(acc[i][e & 3], 4 * tt + 2 + (e >> 2));
          }
          *staged(region, l32, i, 4 * tt + 2 * g) = pack_bf16(lo);
          *staged(region, l32, i, 4 * tt + 2 * g + 1) = pack_bf16(hi);
          __builtin_amdgcn_sched_barrier(0);
        });
      });
      store_staged(region, rc, cld, int(o.N - nw < kBig ? o.N - nw : kBig), q.c_vec, lane);
    } else {
      blocks([&](const float (&v)[16], int64_t n, uint32_t soff) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4)
          buf_store16(rc, n + 4 * k4 < o.N ? at + 16u * k4 : kOutside, soff,
                      make_uint4(__float_as_uint(v[4 * k4]), __float_as_uint(v[4 * k4 + 1]),
                                 __float_as_uint(v[4 * k4 + 2]), __float_as_uint(v[4 * k4 + 3])));
      });
    }
    return;
  }
  // a lane's registers 4 t .. 4 t + 3 of the four tiles j are 16 neighbouring columns
  static_for<4>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    static_for<4>([&](auto tc) {
      constexpr int tt = decltype(tc)::value;
      float v[16];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * r + j] = acc_read(acc[i][j], 4 * tt + r);
      if (mb + i < M) store_run<16>(o, c, ldc, bf16, false, mb + i, nb + 32 * tt, v);
      __builtin_amdgcn_sched_barrier(0);
    });
  });
}

// C of the split tiles: the partial tiles' sum in part order.  A workgroup takes 16 rows
// of a tile, a thread 4 columns of 4 rows.  13 us for 64 tiles in four parts, 75 MB.
__global__ __launch_bounds__(256) void reduce256_kernel(BigParams p) {
  const int tile = p.whole + int(blockIdx.x >> 4);
  int tm, tn;
  const ConstProblem &q = problem_at(big_tile(p, tile, tm, tn));
  const int col = 4 * (threadIdx.x & 63);
  const int64_t n = int64_t(tn) * kBig + col;
  const float *src = p.ws + int64_t(tile - p.whole) * p.split * (kBig * kBig);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 16 * int(blockIdx.x & 15) + 4 * r + int(threadIdx.x >> 6);
    const int64_t m = int64_t(tm) * kBig + row;
    if (m >= q.M || n >= q.N) continue;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.split; ++s) {
      const float4 w = *reinterpret_cast<const float4 *>(src + int64_t(s) * (kBig * kBig) + row * kBig + col);
      v[0] += w.x;
      v[1] += w.y;
      v[2] += w.z;
      v[3] += w.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (n + j >= q.N) break;
      if (q.c_bf16) reinterpret_cast<uint16_t *>(q.c)[m * q.ldc + n + j] = f32_to_bf16(v[j]);
      else reinterpret_cast<float *>(q.c)[m * q.ldc + n + j] = v[j];
    }
  }
}

// C = the partials' sum in split order.  4.6 us for six parts of 8 x 5120: the launch.
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

// The gated block on few tokens: g and u are the dual product's partials, summed in split
// order; a wave takes one 1 x 128 block, two columns to a lane.  hq = Q(silu(g) * u) from
// g and u rounded to bf16, which are written where wanted.  4.7 us for 8 x 20480: the launch.
__global__ __launch_bounds__(256) void reduce_act_kernel(GemmParams p, uint16_t *g, uint16_t *u, Out hq) {
  const int lane = threadIdx.x & 63;
  const int64_t blocks = hq.cols_p / kBlock;
  const int64_t w = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int64_t m = w / blocks, kbk = w % blocks, n = kbk * kBlock + 2 * lane;
  if (m >= p.M) return;
  float v[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
  // ws_ld is a multiple of 4; columns from N up to it were not written, and what is read
  // there is not used
  if (n < p.ws_ld) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int s = 0; s < p.ksplit; ++s) {
        const float2 x =
            *reinterpret_cast<const float2 *>(p.ws + (int64_t(k * p.ksplit + s) * p.M + m) * p.ws_ld + n);
        v[k][0] += x.x;
        v[k][1] += x.y;
      }
  }
  float h[2], top = 0.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint16_t gb = f32_to_bf16(v[0][j]), ub = f32_to_bf16(v[1][j]);
    if (g && n + j < p.N) {
      g[m * p.N + n + j] = gb;
      u[m * p.N + n + j] = ub;
    }
    const float gv = bf16_to_f32(gb);
    h[j] = n + j < p.N ? gv * sigmoid(gv) * bf16_to_f32(ub) : 0.0f;
    top = fmaxf(top, __builtin_fabsf(h[j]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  const uint32_t sb = scale_byte(top);
  *reinterpret_cast<uint16_t *>(hq.codes + m * hq.cols_p + n) =
      uint16_t(encode4(h[0], h[1], 0.0f, 0.0f, scale_of(sb)));
  if (lane == 0) hq.scales[kbk * hq.srow + m] = uint8_t(sb);
}

}  // namespace

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

namespace {

Operand operand_of(const fp8_tensor *t) {
  return Operand{t->codes, t->scales, t->rows, padded_cols(t->cols), scale_row(t->rows, t->two_d), t->two_d != 0};
}

void set_vec(void *c, int64_t ldc, int bf16, int &vec) {
  vec = (reinterpret_cast<uintptr_t>(c) & 15u) == 0 && (ldc * (bf16 ? 2 : 4)) % 16 == 0;
}

// `problems` products in one launch by a plan of the 256 x 256 kernel.
hipError_t run_big(BigParams &p, const Plan &pl, void *ws, hipStream_t stream, int lora = 0) {
  int64_t tiles = 0;
  for (int k = 0; k < p.problems; ++k) {
    Problem &q = p.prob[k];
    q.num_m = int(ceil_div(q.M, kBig));
    q.num_n = int(ceil_div(q.N, kBig));
    q.tile0 = int(tiles);
    tiles += int64_t(q.num_m) * q.num_n;
    set_vec(q.c, q.ldc, q.c_bf16, q.c_vec);
    // buffer offsets of a tile's 256 rows fit in 32 bits, groups do not straddle a row's end
    q.c_vec = q.c_vec && q.ldc < (int64_t(1) << 21) && q.N % (q.c_bf16 ? 8 : 4) == 0;
  }
  p.whole = pl.whole;
  p.split = pl.split;
  p.ws = static_cast<float *>(ws);
  const int rest = int(tiles) - pl.whole;
  const dim3 grid(unsigned(pl.whole + rest * pl.split));
  const auto kernel = lora == 2 ? gemm256_kernel<kLoraDrop> : lora ? gemm256_kernel<kLora> : gemm256_kernel<kStore>;
  const hipError_t e = launch(kernel, grid, dim3(256), stream, p);
  if (e != hipSuccess || rest == 0) return e;
  return launch(reduce256_kernel, dim3(unsigned(rest) * 16u), dim3(256), stream, p);
}

// g and u (nullable) and hq of the gated block, x [M][K] against wg and wu [F][K].
hipError_t run_act(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, uint16_t *g, uint16_t *u,
                   const fp8_tensor *hq, hipStream_t stream) {
  BigParams p{};
  Problem &q = p.prob[0];
  q.a[0] = q.a[1] = operand_of(xq);
  q.b[0] = operand_of(wg);
  q.b[1] = operand_of(wu);
  q.M = xq->rows;
  q.N = wg->rows;
  q.kb = q.stages = int(ceil_div(xq->cols, kBlock));
  q.num_m = int(ceil_div(q.M, kBig));
  q.num_n = int(ceil_div(q.N, kBig / 2));
  p.problems = 1;
  p.split = 1;
  p.whole = q.num_m * q.num_n;
  const uintptr_t at = reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(u);
  p.act = ActOut{g, u, q.N % 8 == 0 && (at & 15u) == 0, hq->codes, hq->scales, padded_cols(hq->cols), scale_row(hq->rows, false)};
  return launch(gemm256_kernel<kAct>, dim3(unsigned(p.whole)), dim3(256), stream, p);
}

hipError_t run_dact(const fp8_tensor *dyq, const fp8_tensor *wd_t, const uint16_t *g, const uint16_t *u,
                    const fp8_ffn_buffers *bufs, hipStream_t stream) {
  BigParams p{};
  Problem &q = p.prob[0];
  q.a[0] = q.a[1] = operand_of(dyq);
  q.b[0] = q.b[1] = operand_of(wd_t);
  q.M = dyq->rows;
  q.N = wd_t->rows;
  q.kb = q.stages = int(ceil_div(dyq->cols, kBlock));
  q.num_m = int(ceil_div(q.M, kBig));
  q.num_n = int(ceil_div(q.N, kBig));
  p.problems = 1;
  p.split = 1;
  p.whole = q.num_m * q.num_n;
  p.dact = DactArgs{g, u, dact_out(bufs)};
  return launch(gemm256_kernel<kDact>, dim3(unsigned(p.whole)), dim3(256), stream, p);
}

Problem problem_of(const GemmParams &g) {
  Problem q{};
  for (int k = 0; k < 2; ++k) {
    q.a[k] = g.a[k];
    q.b[k] = g.b[k];
  }
  q.M = g.M;
  q.N = g.N;
  q.kb = g.kb;
  q.stages = g.stages;
  q.c = g.c;
  q.ldc = g.ldc;
  q.c_bf16 = g.c_bf16;
  return q;
}

// Rows [first, end) of the product, first a multiple of the tile's.
template <bool FAST, int LORA = 0>
hipError_t launch_general(GemmParams &p, int config, int64_t first, int64_t end, hipStream_t stream) {
  const Config &c = kConfigs[config];
  p.m_first = first;
  p.num_m = int(ceil_div(end - first, c.bm));
  const int64_t groups = int64_t(p.num_m) * (p.dual ? 2 * p.dual : ceil_div(p.N, c.bn)) * p.ksplit;
  const dim3 grid{unsigned(groups)}, blk{256};
  if constexpr (!FAST) {
    // eight waves of 128 x 64: a conversion serves more products than in 64 x 64, and half
    // the bytes come from L2 (8192^3: 785-800 us, 128 x 128 tiles 973)
    if (config == 7) return launch(gemm_kernel<256, 256, 2, 4, 2, false, LORA>, grid, dim3(512), stream, p);
  }
  switch (config) {
    case 0:
    case 1:
    case 2:
      if constexpr (LORA != 0) {
        return hipErrorInvalidValue;  // more than 64 rows, and a tail of fewer, take others
      } else {
        if (config == 0) return launch(gemm_kernel<16, 64, 1, 4, 4, FAST, 0>, grid, blk, stream, p);
        if (config == 1) return launch(gemm_kernel<16, 128, 1, 4, 4, FAST, 0>, grid, blk, stream, p);
        return launch(gemm_kernel<32, 128, 1, 4, 4, FAST, 0>, grid, blk, stream, p);
      }
    case 3: return launch(gemm_kernel<64, 64, 2, 2, 3, FAST, LORA>, grid, blk, stream, p);
    case 4: return launch(gemm_kernel<64, 128, 2, 2, 3, FAST, LORA>, grid, blk, stream, p);
    case 5: return launch(gemm_kernel<128, 64, 2, 2, 3, FAST, LORA>, grid, blk, stream, p);
    default:
      if (three_stages(groups)) return launch(gemm_kernel<128, 128, 2, 2, 3, FAST, LORA>, grid, blk, stream, p);
      return launch(gemm_kernel<128, 128, 2, 2, 2, FAST, LORA>, grid, blk, stream, p);
  }
}

constexpr int kLoraTail = 4;  // 64 x 128

template <bool FAST, int LORA = 0>
hipError_t run(GemmParams &p, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  // the plan's split or none: with less than its workspace a caller gets the unsplit sums
  Plan pl = plan_of(p.M, p.N, p.stages, FAST, kNoLimit);
  if (pl.bytes > ws_bytes) pl = plan_of(p.M, p.N, p.stages, FAST, 0);
  if (pl.config < 0) {
    BigParams b{};
    b.prob[0] = problem_of(p);
    b.problems = 1;
    b.lora = p.lora;
    return run_big(b, pl, ws, stream, LORA);
  }
  p.ksplit = pl.ksplit;
  p.raw = pl.ksplit > 1;
  p.ws = static_cast<float *>(ws);
  p.ws_ld = ws_ld_of(p.N);
  set_vec(p.c, p.ldc, p.c_bf16, p.c_vec);
  const Split sp = split_rows(p.M, p.N, p.stages, FAST, pl);
  if (sp.rows > 0) {
    const hipError_t e = launch_general<FAST, LORA>(p, pl.config, 0, sp.rows, stream);
    // the kernels with adapters begin at tiles of 64 rows
    const int tail = LORA != 0 && kConfigs[sp.tail].bm < 64 ? kLoraTail : sp.tail;
    return e != hipSuccess ? e : launch_general<FAST, LORA>(p, tail, sp.rows, p.M, stream);
  }
  const hipError_t e = launch_general<FAST, LORA>(p, pl.config, 0, p.M, stream);
  if (e != hipSuccess || pl.ksplit == 1) return e;
  return launch(reduce_kernel, dim3(unsigned(ceil_div(p.M * (p.ws_ld / 4), 256))), dim3(256), stream, p);
}

}  // namespace

size_t gemm_ws_bytes(int64_t M, int64_t N, int64_t stages, bool fast) {
  return M > 0 && N > 0 ? plan_of(M, N, stages, fast, kNoLimit).bytes : 0;
}

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

Partials gemm_partials(int64_t M, int64_t N, int64_t stages, bool fast) {
  const Plan pl = plan_general(M, N, stages, 1, kNoLimit, fast);
  const int64_t ld = ws_ld_of(N);
  return Partials{pl.config, pl.ksplit, ld, size_t(pl.ksplit) * size_t(M) * size_t(ld) * sizeof(float)};
}

hipError_t launch_gemm_partials(const fp8_tensor *a, const fp8_tensor *b, bool fast, float *ws, hipStream_t stream) {
  GemmParams p{};
  p.a[0] = p.a[1] = operand_of(a);
  p.b[0] = p.b[1] = operand_of(b);
  p.M = a->rows;
  p.N = b->rows;
  p.kb = p.stages = int(ceil_div(a->cols, kBlock));
  const Partials pl = gemm_partials(p.M, p.N, p.stages, fast);
  p.ksplit = pl.ksplit;
  p.raw = 1;
  p.ws = ws;
  p.ws_ld = pl.ld;
  return fast ? launch_general<true>(p, pl.config, 0, p.M, stream) : launch_general<false>(p, pl.config, 0, p.M, stream);
}

hipError_t launch_gemm_lora(const fp8_tensor *a, const fp8_tensor *b, const LoraAdd &lora, void *c, int64_t ldc, bool fast,
                            void *ws, size_t ws_bytes, hipStream_t stream) {
  GemmParams p{};
  p.a[0] = p.a[1] = operand_of(a);
  p.b[0] = p.b[1] = operand_of(b);
  p.M = a->rows;
  p.N = b->rows;
  p.kb = p.stages = int(ceil_div(a->cols, kBlock));
  p.c = c;
  p.ldc = ldc;
  p.c_bf16 = 1;
  p.lora = lora;
  if (lora.drop.thr) return fast ? run<true, 2>(p, ws, ws_bytes, stream) : run<false, 2>(p, ws, ws_bytes, stream);
  return fast ? run<true, 1>(p, ws, ws_bytes, stream) : run<false, 1>(p, ws, ws_bytes, stream);
}

hipError_t launch_gemm_sum(const fp8_tensor *a1, const fp8_tensor *b1, const fp8_tensor *a2, const fp8_tensor *b2,
                           void *c, fp4_dtype c_dtype, int64_t ldc, bool fast, void *ws, size_t ws_bytes,
                           hipStream_t stream) {
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
  return fast ? run<true>(p, ws, ws_bytes, stream) : run<false>(p, ws, ws_bytes, stream);
}

hipError_t launch_gemm_group(const GemmCall *calls, int n, bool fast, void *ws, size_t ws_bytes, hipStream_t stream) {
  int64_t shapes[kMaxProblems][3];
  for (int k = 0; k < n; ++k) {
    shapes[k][0] = calls[k].a->rows;
    shapes[k][1] = calls[k].b->rows;
    shapes[k][2] = ceil_div(calls[k].a->cols, kBlock);
  }
  const Plan pl = fast ? plan_group(shapes, n, ws_bytes) : Plan{-1, 1, 0, 1, -1, 0};
  if (pl.us < 0) {
    for (int k = 0; k < n; ++k) {
      const GemmCall &g = calls[k];
      const hipError_t e = launch_gemm(g.a, g.b, g.c, g.c_dtype, g.ldc, fast, ws, ws_bytes, stream);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  BigParams p{};
  for (int k = 0; k < n; ++k) {
    const GemmCall &g = calls[k];
    Problem &q = p.prob[k];
    q.a[0] = q.a[1] = operand_of(g.a);
    q.b[0] = q.b[1] = operand_of(g.b);
    q.M = g.a->rows;
    q.N = g.b->rows;
    q.kb = q.stages = int(ceil_div(g.a->cols, kBlock));
    q.c = g.c;
    q.ldc = g.ldc;
    q.c_bf16 = g.c_dtype == FP4_BF16;
  }
  p.problems = n;
  return run_big(p, pl, ws, stream);
}

size_t gemm_group_ws_bytes(int64_t M, int64_t N, int64_t stages, int n, bool fast) {
  if (M == 0 || N == 0) return 0;
  const size_t one = gemm_ws_bytes(M, N, stages, fast), other = gemm_ws_bytes(N, M, stages, fast);
  const size_t apart = one > other ? one : other;
  if (!fast) return apart;
  const int64_t shapes[kMaxProblems][3] = {{M, N, stages}, {M, N, stages}, {N, M, stages}};
  const Plan pl = plan_group(shapes, n, kNoLimit);
  return pl.us >= 0 && pl.bytes > apart ? pl.bytes : apart;
}

namespace {

// g and u (nullable) and hq from one dual product into ws and a kernel that sums, activates
// and quantizes.
template <bool FAST>
hipError_t run_act_dual(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, uint16_t *g, uint16_t *u,
                        const fp8_tensor *hq, void *ws, size_t ws_bytes, hipStream_t stream) {
  GemmParams p{};
  p.a[0] = p.a[1] = operand_of(xq);
  p.b[0] = operand_of(wg);
  p.b[1] = operand_of(wu);
  p.M = xq->rows;
  p.N = wg->rows;
  if (p.M == 0 || p.N == 0) return hipSuccess;
  p.kb = p.stages = int(ceil_div(xq->cols, kBlock));
  const Plan pl = plan_general(p.M, p.N, p.stages, 2, ws_bytes, FAST);
  p.ksplit = pl.ksplit;
  p.raw = 1;
  p.dual = int(ceil_div(p.N, kConfigs[pl.config].bn));
  p.ws = static_cast<float *>(ws);
  p.ws_ld = ws_ld_of(p.N);
  const hipError_t e = launch_general<FAST>(p, pl.config, 0, p.M, stream);
  if (e != hipSuccess) return e;
  const int64_t waves = p.M * ceil_div(p.N, kBlock);
  return launch(reduce_act_kernel, dim3(unsigned(ceil_div(waves, 4))), dim3(256), stream, p, g, u, out_of(hq));
}

hipError_t run_act_apart(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, uint16_t *g, uint16_t *u,
                         const fp8_tensor *hq, void *ws, size_t ws_bytes, hipStream_t stream) {
  const int64_t M = xq->rows, F = wg->rows;
  int64_t ld = F;
  if (!g) {
    ld = act_ld(F);
    g = static_cast<uint16_t *>(ws);
    u = g + M * ld;
    ws = u + M * ld;  // a multiple of 16 bytes on
    ws_bytes -= act_held_bytes(M, F);
  }
  hipError_t e = launch_gemm(xq, wg, g, FP4_BF16, ld, false, ws, ws_bytes, stream);
  if (e == hipSuccess) e = launch_gemm(xq, wu, u, FP4_BF16, ld, false, ws, ws_bytes, stream);
  return e != hipSuccess ? e : launch_act_quantize(g, u, ld, hq, stream);
}

}  // namespace

size_t act_ws_bytes(int64_t M, int64_t F, int64_t stages, bool fast, bool keep) {
  if (M == 0 || F == 0 || (fast && act_fused(M, F, stages))) return 0;
  if (!fast && act_apart(M, F, stages)) return gemm_ws_bytes(M, F, stages, false) + (keep ? 0 : act_held_bytes(M, F));
  return plan_general(M, F, stages, 2, kNoLimit, fast).bytes;
}

hipError_t launch_gemm_act(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu, uint16_t *g, uint16_t *u,
                           const fp8_tensor *hq, bool fast, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (xq->rows == 0 || wg->rows == 0) return hipSuccess;
  const int64_t stages = ceil_div(xq->cols, kBlock);
  if (!fast)
    return act_apart(xq->rows, wg->rows, stages) ? run_act_apart(xq, wg, wu, g, u, hq, ws, ws_bytes, stream)
                                                 : run_act_dual<false>(xq, wg, wu, g, u, hq, ws, ws_bytes, stream);
  return act_fused(xq->rows, wg->rows, stages) ? run_act(xq, wg, wu, g, u, hq, stream)
                                               : run_act_dual<true>(xq, wg, wu, g, u, hq, ws, ws_bytes, stream);
}

size_t dact_ws_bytes(int64_t M, int64_t F, int64_t stages, bool vec, bool fast) {
  if (M == 0 || F == 0 || (fast && dact_fused(M, F, stages, vec))) return 0;
  return size_t(M) * size_t(ceil_div(F, 8) * 8) * sizeof(float);
}

hipError_t launch_gemm_dact(const fp8_tensor *dyq, const fp8_tensor *wd_t, const uint16_t *g, const uint16_t *u,
                            const fp8_ffn_buffers *bufs, bool fast, void *ws, hipStream_t stream) {
  const int64_t M = dyq->rows, F = wd_t->rows;
  if (M == 0 || F == 0) return hipSuccess;
  const bool aligned = ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(u)) & 15u) == 0;
  if (fast && dact_fused(M, F, ceil_div(dyq->cols, kBlock), aligned)) return run_dact(dyq, wd_t, g, u, bufs, stream);
  // dh's rows padded to 8, so that they take wide stores and loads (wd_t's rows past F read
  // as zeros)
  GemmParams p{};
  p.a[0] = p.a[1] = operand_of(dyq);
  p.b[0] = p.b[1] = operand_of(wd_t);
  p.M = M;
  p.N = p.ldc = ceil_div(F, 8) * 8;
  p.kb = p.stages = int(ceil_div(dyq->cols, kBlock));
  p.c = ws;
  const hipError_t e = fast ? run<true>(p, nullptr, 0, stream) : run<false>(p, nullptr, 0, stream);
  return e != hipSuccess ? e : launch_dact_quantize(static_cast<const float *>(ws), p.ldc, g, u, bufs, stream);
}

}  // namespace fp8
}  // namespace nvfp4
