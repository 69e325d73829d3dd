// fp8_plan.hpp -- which kernel, tile and K split an 8-bit product or a step of the gated
// block runs on, from its sizes alone.  Plain host code: tests/test_fp8_plan.py builds it
// with the host compiler to check that the tested sizes reach the paths they are for.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {
namespace fp8 {

constexpr int kBlock = 128;
constexpr int kBig = 256;  // the large kernel's tile

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Compute units of the current GPU (256 where there is none).
int cu_count();

// Plans.  A product runs on the kernel, tile and K split whose time is least by this
// model, whose constants were fitted to timings of 20 shapes from 4 x 5120 x 5120 to
// 4096 x 1024 x 8192.  It is there to order the variants of a size.  Of 25 sizes from
// 1 x 5120 x 5120 to 16384 x 20480 x 5120 with bf16 results the calls took 0.66 to 1.31 of
// it (8-bit instruction) and 0.72 to 1.07 (binary32 sums): less where a few us of work are
// added to the 7, more where the power limit lowers the clock.  Binary32 results, whose
// stores it leaves out, took up to 1.6 of it.
//   general kernel   7 us + stages per part * (one workgroup to a CU: t1, two: t2, times
//                    the rounds of two), 4 us and the partials' bytes at 4 TB/s for a split
//   256 x 256 kernel 12 us + 1.27 us a stage and round, 8 us for a last round, 6 us and the
//                    bytes at 5.5 TB/s for its split
// the general one never less than the operands' bytes at 6 TB/s.  Both sides at a few shapes (us):
// 512x4096x4096 64x128 tiles 19.9, 128x128 22.5, 256x256 49.2; 2048x4096x4096 128x128 39,
// 256x256 61; 4000x4000x4000 128x128 78, 256x256 56; 4x5120x20480 in one part 38, in six 25.
// The last entry is the binary32 sums' large tile (times b1, b2), which the 8-bit instruction
// has no use for: its own 256 x 256 kernel is faster.
struct Config {
  int bm, bn;
  double t1, t2;  // us a stage with one and two workgroups to a CU, 8-bit matrix instruction
  double b1, b2;  // and the bf16 one (0: two do not fit; both 0: not used)
};
constexpr Config kConfigs[] = {
    {16, 64, 0.24, 0.43, 0.24, 0.45},  {16, 128, 0.34, 0.90, 0.34, 0.90}, {32, 128, 0.40, 0.95, 0.45, 1.0},
    {64, 64, 0.32, 0.45, 0.45, 0.75},  {64, 128, 0.40, 0.57, 0.70, 1.21}, {128, 64, 0.41, 0.57, 0.70, 1.21},
    {128, 128, 0.66, 1.03, 1.00, 1.80}, {256, 256, 0, 0, 3.20, 0}};

struct Plan {
  int config;  // of kConfigs, or -1: the 256 x 256 kernel
  int ksplit;  // general kernel
  int whole, split;  // 256 x 256 kernel: unsplit tiles, K parts of the others
  double us;
  size_t bytes;
};

// floats of a row of partial results
inline int64_t ws_ld_of(int64_t N) { return ceil_div(N, 4) * 4; }
constexpr size_t kNoLimit = ~size_t(0);

// The general kernel on M x (copies * N): copies = 2 for the dual product, whose results
// are raw also without a split.
inline Plan plan_general(int64_t M, int64_t N, int64_t stages, int copies, size_t limit, bool fast = true) {
  const int cus = cu_count();
  Plan best{};
  best.us = 1e30;
  const double least = double(M + copies * N) * double(stages) * kBlock / 6e6;
  for (int k = 0; k < int(sizeof(kConfigs) / sizeof(kConfigs[0])); ++k) {
    const Config &c = kConfigs[k];
    if (M <= 64 ? c.bm < M || c.bm >= 2 * M + 16 : c.bm < 64) continue;
    const double one = fast ? c.t1 : c.b1, two = fast ? c.t2 : c.b2;
    if (one == 0) continue;
    const int64_t tiles = ceil_div(M, c.bm) * ceil_div(N, c.bn) * copies;
    for (int ks = 1; ks <= 16 && (ks == 1 || ks * 4 <= stages); ++ks) {
      const int64_t groups = tiles * ks;
      if (ks > 1 && groups > 2 * cus) break;
      const size_t bytes = ks > 1 || copies > 1 ? size_t(copies) * ks * size_t(M) * size_t(ws_ld_of(N)) * sizeof(float) : 0;
      if (ks > 1 && bytes > limit) break;
      const double step = groups <= cus ? one : two > 0 ? two * double(ceil_div(groups, 2 * cus)) : one * double(ceil_div(groups, cus));
      double us = 7 + double(ceil_div(stages, ks)) * step;
      if (us < least) us = least;
      if (ks > 1) us += 4 + double(bytes) * 2 / 4e6;
      if (us < best.us) best = Plan{k, ks, 0, 1, us, bytes};
    }
  }
  return best;
}

// The 256 x 256 kernel: whole rounds of tiles unsplit, the rest in as many K parts as fill
// the last round (at least 4 stages to a part), or whole.
inline Plan plan_big(int64_t tiles, int64_t stages, size_t limit) {
  const int cus = cu_count();
  const int64_t rem = tiles % cus;
  Plan best{-1, 1, int(tiles), 1, 12 + 1.27 * double(stages * ceil_div(tiles, cus)) + (tiles > cus && rem ? 8 : 0), 0};
  if (rem > 0) {
    int64_t s = cus / rem;
    s = s < stages / 4 ? s : stages / 4;
    s = s < 16 ? s : 16;
    const size_t bytes = size_t(rem * (s > 0 ? s : 0)) * kBig * kBig * sizeof(float);
    const double us = 12 + 1.27 * double(stages * (tiles / cus) + (s > 1 ? ceil_div(stages, s) : 0)) +
                      (tiles > cus ? 8 : 0) + 6 + double(bytes) * 2 / 5.5e6;
    if (s > 1 && bytes <= limit && us < best.us) best = Plan{-1, 1, int(tiles - rem), int(s), us, bytes};
  }
  return best;
}

inline int64_t big_tiles(int64_t M, int64_t N) { return ceil_div(M, kBig) * ceil_div(N, kBig); }

inline Plan plan_of(int64_t M, int64_t N, int64_t stages, bool fast, size_t limit) {
  const Plan g = plan_general(M, N, stages, 1, limit, fast);
  if (!fast || M <= 128 || N <= 128) return g;
  const Plan b = plan_big(big_tiles(M, N), stages, limit);
  return b.us < g.us ? b : g;
}

// A plan's 128 x 128 tiles: a third stage in flight for a workgroup alone on its CU, two
// workgroups otherwise (128x20480x5120: 35 us against 42; 2048x4096x4096: 53 against 39)
inline bool three_stages(int64_t groups) { return groups <= cu_count(); }

// Whole rounds of 256 x 256 tiles of binary32 sums: rows [0, rows) take them and the rest
// the tile `tail`, where that takes less than a round for a few tiles (20480x5120x16384,
// 6.25 rounds, on one board: 2734 us in one launch, 2635 in two).  rows = 0: one launch.
struct Split {
  int64_t rows;
  int tail;
};
inline Split split_rows(int64_t M, int64_t N, int64_t stages, bool fast, const Plan &pl) {
  if (pl.config < 0 || kConfigs[pl.config].bm != 256 || pl.ksplit != 1) return Split{0, 0};
  const int64_t across = ceil_div(N, 256), tiles = ceil_div(M, 256) * across;
  const int64_t rows = tiles / cu_count() * cu_count() / across * 256;
  if (rows <= 0 || rows >= M) return Split{0, 0};
  const Plan head = plan_general(rows, N, stages, 1, 0, fast), tail = plan_general(M - rows, N, stages, 1, 0, fast);
  if (head.config != pl.config || head.us + tail.us >= pl.us) return Split{0, 0};
  return Split{rows, tail.config};
}

constexpr int kMaxProblems = 3;  // of one launch of the 256 x 256 kernel

// The plan of `n` products in one launch of the 256 x 256 kernel, or one with us < 0 where
// their own launches take less by the model.
inline Plan plan_group(const int64_t (*shapes)[3], int n, size_t limit) {
  int64_t tiles = 0, least = INT64_MAX, most = 0;
  double apart = 0;
  for (int k = 0; k < n; ++k) {
    const int64_t M = shapes[k][0], N = shapes[k][1], st = shapes[k][2];
    if (M <= 128 || N <= 128) return Plan{-1, 1, 0, 1, -1, 0};
    tiles += big_tiles(M, N);
    least = st < least ? st : least;
    most = st > most ? st : most;
    apart += plan_of(M, N, st, true, limit).us;
  }
  Plan pl = plan_big(tiles, least, limit);
  if (least != most || pl.us >= apart) pl.us = -1;
  return pl;
}

// The gated block's first half by the model: the 256 x 256 kernel with its epilogue (12 us
// a tile), or the dual product, its partials (0.95 us a MB: written and read at 2.1 TB/s)
// and the kernel that reads them.  Forward calls with either, us: 65x5120x20480 fused 107,
// dual 106; 128x5120x20480 119, 133 (the model has it the other way round); 256x5120x20480
// 146, 196; 4096x5120x20480 1075, 1700; 300x512x2048 24, 22; 1024x512x2048 26, 40;
// 100x1000x3000 28, 20; 1000x257x1001 25, 24.
inline double act_fused_us(int64_t M, int64_t F, int64_t stages) {
  const int64_t rounds = ceil_div(ceil_div(M, kBig) * ceil_div(F, kBlock), cu_count());
  return 12 + double(rounds) * (1.27 * double(stages) + 12);
}
// F is bounded by the buffer offsets of a tile's rows of g and u.
inline bool act_fused(int64_t M, int64_t F, int64_t stages) {
  if (M <= 64 || F >= (int64_t(1) << 22)) return false;
  const Plan d = plan_general(M, F, stages, 2, kNoLimit);
  return act_fused_us(M, F, stages) < d.us + 6 + double(d.bytes) * 2 / 2.1e6;
}

// Binary32 sums have no kernel with an epilogue of the gated block's: the same dual product
// on few tokens, or both projections to memory in bf16 (to the workspace where the caller
// does not keep them) and a kernel that reads them.  Forward calls with either, us:
// 128x5120x20480 dual 141, apart 154; 256x5120x20480 239, 232; 1024x5120x20480 698, 605;
// 4096x5120x20480 2478, 2059; 300x512x2048 25, 35; 1024x512x2048 41, 34; 1000x257x1001 26, 41.
inline int64_t act_ld(int64_t F) { return ceil_div(F, 8) * 8; }
inline size_t act_held_bytes(int64_t M, int64_t F) { return size_t(M) * size_t(act_ld(F)) * 4; }
inline bool act_apart(int64_t M, int64_t F, int64_t stages) {
  if (M <= 64) return false;
  const Plan d = plan_general(M, F, stages, 2, kNoLimit, false);
  return 2 * plan_of(M, F, stages, false, kNoLimit).us + 8 + double(M) * double(F) * 9 / 4.5e6 <
         d.us + 6 + double(d.bytes) * 2 / 2.1e6;
}

// The backward pass's first half: the same choice.  The fused epilogue takes 50 us a tile;
// apart, dh passes through memory (binary32, written and read) and the element-wise
// kernel moves 13 bytes an element more.  Backward calls with either, us: 256x5120x20480
// fused 431, apart 417; 512x5120x20480 524, 528; 1024x5120x20480 804, 851; 1024x512x2048
// 82, 55; 1024x2048x8192 193, 207 (the model has it the other way round); 1500x2048x8192
// 244, 270.
// aligned: g and u are, to 16 bytes.
inline bool dact_fused(int64_t M, int64_t F, int64_t stages, bool aligned) {
  if (M <= 64 || F % 8 != 0 || F >= (int64_t(1) << 22) || !aligned) return false;
  const int64_t rounds = ceil_div(big_tiles(M, F), cu_count());
  const double fused = 12 + double(rounds) * (1.27 * double(stages) + 50);
  return fused < plan_of(M, F, stages, true, 0).us + 10 + double(M) * double(F) * 21 / 4.5e6;
}

}  // namespace fp8
}  // namespace nvfp4
