// Host-side arithmetic of the operators around the expert step: workspace layouts and argument
// validation.  Plain C++ (no HIP), like moe_plan.h: also built on its own into a CPU test.
#pragma once
#include "moe_plan.h"

namespace moe {

// ---- RMS norm backward: weight-gradient partials, one row of H floats per workgroup
int norm_bwd_parts(int T, int H);   // workgroups (= partial rows) of the backward kernel
size_t norm_bwd_ws_bytes(int T, int H);
int layernorm_bwd_parts(int T, int H);            // the same for the layer norm,
size_t layernorm_bwd_ws_bytes(int T, int H);      // which has a second set of parts for the bias

// ---- balance loss: workgroup b takes rows [b * chunk, (b + 1) * chunk); the part of sequence s
// in it writes its sums to slot b + s (increasing along the rows, so no two parts share one).
struct BalancePlan {
    bool one;                                // one workgroup, one launch, no parts
    int chunk, nblocks, nslots, stride;      // stride: floats of a slot's row, E rounded up to 4
    size_t probs, hits, z, seq, done, end;   // byte offsets: float [slots][stride], int [slots][stride],
                                             // float [slots], float [S][2], int
};
BalancePlan balance_plan(int T, int E, int S);

// ---- gated block backward: its two bf16 products in one launch
struct ProductPlan {
    int tile;       // of product_plan's table
    int parts[2];   // parts that the sums of dx and dw are split into; 0: not asked for
    int first;      // the product that goes first: 0 dw, 1 dx
};
ProductPlan product_plan(int T, int K, int I, bool dx, bool dw);
// operands of the products, their parts, and partial rows of the bias's gradient
struct GatedBwdPlan {
    int row_blocks, parts;                             // blocks of 64 rows; partial rows [parts][2I] floats
    ProductPlan product;
    size_t part, weights, rows, dgu_packed, join[2], end;   // byte offsets; what is not needed takes nothing
};
GatedBwdPlan gated_bwd_plan(int T, int K, int I, bool dx, bool dw, bool dbias);

// ---- adapters: rows of one sequence in one window are a slot, which has operands of 16 rows x 32 ranks in
// the workspace, each as `split` bf16 parts
struct LoraPlan {
    int window, steps, split;   // rows of a window; operands along the rank; parts
    int64_t slots;
    size_t end;                 // workspace bytes
};
LoraPlan lora_plan(int T, int R, int S, bool bf16);   // S = 0: a sequence per row

namespace host {
int check_add_rmsnorm(const moe_add_rmsnorm_args* a);
int check_add_rmsnorm_backward(const moe_add_rmsnorm_backward_args* a);
int check_add_layernorm(const moe_add_layernorm_args* a);
int check_add_layernorm_backward(const moe_add_layernorm_backward_args* a);
int check_linear(const moe_linear_args* a);
int check_gated_linear(const moe_gated_linear_args* a);
int check_gated_linear_backward(const moe_gated_linear_backward_args* a);
int check_lora(const moe_lora_args* a);
int check_balance_loss(const moe_balance_loss_args* a);
int check_route_backward(const moe_route_backward_args* a);
int check_combine_backward(const moe_combine_backward_args* a);
}  // namespace host

}  // namespace moe
