/* The plan of the 8-bit products (csrc/fp8_plan.hpp) for a GPU of 256 compute units, for
 * tests/test_fp8_plan.py. */
#include "../../nvfp4_bit_microscaled_amd/csrc/fp8_plan.hpp"

namespace nvfp4 {
namespace fp8 {
int cu_count() { return 256; }
}  // namespace fp8
}  // namespace nvfp4

using namespace nvfp4::fp8;

static void put(const Plan &p, int64_t M, int64_t N, int64_t stages, bool fast, int copies, int64_t *out) {
  out[0] = p.config < 0 ? 256 : kConfigs[p.config].bm;
  out[1] = p.config < 0 ? 256 : kConfigs[p.config].bn;
  out[2] = p.config < 0 ? p.split : p.ksplit;
  const Split s = split_rows(M, N, stages, fast, p);
  out[3] = s.rows;
  out[4] = p.config < 0 ? p.whole : ceil_div(M, out[0]) * ceil_div(N, out[1]) * copies * p.ksplit;
  out[5] = p.config < 0;
}

extern "C" {

/* out: tile rows and columns, K parts, rows of the head launch (0: one launch), workgroups
 * (of the 256 x 256 kernel: unsplit tiles), whether it is the 256 x 256 kernel */
void fp8_plan_product(int64_t M, int64_t N, int64_t stages, int fast, int ws, int64_t *out) {
  put(plan_of(M, N, stages, fast, ws ? kNoLimit : 0), M, N, stages, fast, 1, out);
}

void fp8_plan_dual(int64_t M, int64_t F, int64_t stages, int fast, int64_t *out) {
  put(plan_general(M, F, stages, 2, kNoLimit, fast), M, F, stages, fast, 2, out);
}

/* three weight gradients: 0 apart, else K parts of the last tiles; *whole: the unsplit ones */
int64_t fp8_plan_group(int64_t F, int64_t K, int64_t stages, int64_t *whole) {
  const int64_t shapes[kMaxProblems][3] = {{F, K, stages}, {F, K, stages}, {K, F, stages}};
  const Plan p = plan_group(shapes, kMaxProblems, kNoLimit);
  *whole = p.whole;
  return p.us < 0 ? 0 : p.split;
}

int fp8_plan_act_fused(int64_t M, int64_t F, int64_t stages) { return act_fused(M, F, stages); }
int fp8_plan_act_apart(int64_t M, int64_t F, int64_t stages) { return act_apart(M, F, stages); }
int fp8_plan_dact_fused(int64_t M, int64_t F, int64_t stages) { return dact_fused(M, F, stages, true); }
int fp8_plan_three_stages(int64_t groups) { return three_stages(groups); }
}
