// linear_plan.hip -- what plan_linear and the rules beside it choose for a
// call, for the test that every kernel they can choose is run by a test.
#include "linear_plan.hpp"

using namespace fp4q_dev;

// out: kind (0 few rows, 1..4 tiles of 32, 64, 128, 256 rows), weight format,
// planes, weight-row tiles of the few-row kernel, 64-bit gather, activations
// copied, gathered by the copy, parts of the sum.  rows: x [T, ld_x] is gathered.
extern "C" void fp4q_probe_linear_plan(int grad, int sf, int x_dt, int grouped, int rows, int64_t T, int64_t ld_x,
                                       int64_t R, int64_t N, int64_t K, int E, int32_t* out) {
    const LinearPlan q = plan_linear(grad != 0, sf, x_dt, grouped != 0, R, N, K, E);
    const bool few = q.kind == Kind::kSkinny, gather = rows && q.copy && far_rows(T, q.pitch);
    out[0] = (int)q.kind;
    out[1] = weight_format(sf, x_dt);
    out[2] = q.np;
    out[3] = few ? few_rows_tiles(grouped != 0, R, N, E) : 0;
    out[4] = !few && rows && !q.copy && far_rows(T, ld_x);
    out[5] = q.copy;
    out[6] = gather;
    out[7] = q.splits;
}
