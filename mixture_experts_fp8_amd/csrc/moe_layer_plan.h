// Host-side arithmetic of the operators around the expert step: workspace layouts and argument
// validation.  Plain C++ (no HIP), like moe_plan.h: also built on its own into a CPU test.
#pragma once
#include "moe_plan.h"

namespace moe {

// ---- RMS norm backward: weight-gradient partials, one row of H floats per workgroup
int norm_bwd_parts(int T, int H);   // workgroups (= partial rows) of the backward kernel
size_t norm_bwd_ws_bytes(int T, int H);

// ---- balance loss: workgroup b takes rows [b * chunk, (b + 1) * chunk); the part of sequence s
// in it writes its sums to slot b + s (increasing along the rows, so no two parts share one).
struct BalancePlan {
    bool one;                                // one workgroup, one launch, no parts
    int chunk, nblocks, nslots, stride;      // stride: floats of a slot's row, E rounded up to 4
    size_t probs, hits, z, seq, done, end;   // byte offsets: float [slots][stride], int [slots][stride],
                                             // float [slots], float [S][2], int
};
BalancePlan balance_plan(int T, int E, int S);

namespace host {
int check_add_rmsnorm(const moe_add_rmsnorm_args* a);
int check_add_rmsnorm_backward(const moe_add_rmsnorm_backward_args* a);
int check_linear(const moe_linear_args* a);
int check_balance_loss(const moe_balance_loss_args* a);
int check_route_backward(const moe_route_backward_args* a);
int check_combine_backward(const moe_combine_backward_args* a);
}  // namespace host

}  // namespace moe
