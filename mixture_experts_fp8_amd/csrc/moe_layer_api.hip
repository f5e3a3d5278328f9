// C ABI of the operators around the expert step: arguments checked by moe_layer_host.cpp, then the
// launches.
#include "../../include/moe_fp8.h"
#include "layer_common.h"

using moe::host::ok;

namespace {

int done(const char* op, hipError_t e) {
    return e == hipSuccess ? ok() : moe::host::fail(MOE_ERR_HIP, "%s: HIP error %d (%s)", op, (int)e, hipGetErrorString(e));
}

}  // namespace

extern "C" {

int moe_add_rmsnorm(const moe_add_rmsnorm_args* a) {
    if (int rc = moe::host::check_add_rmsnorm(a)) return rc;
    const int group = !a->yq ? 0 : a->quant == MOE_QUANT_FP8_BLOCK128 ? 128 : 32;
    const moe::NormArgs n{a->T, a->H, a->x, a->ld_x, a->residual, a->ld_residual, a->weight, a->eps,
                          a->h, a->y, a->yq, a->ys, group, 1.0 / a->H};
    return done("moe_add_rmsnorm", moe::launch_add_rmsnorm(n, static_cast<hipStream_t>(a->stream)));
}

size_t moe_add_rmsnorm_backward_workspace_size(int32_t T, int32_t H) {
    return T < 1 || H < 1 ? 0 : moe::norm_bwd_ws_bytes(T, H);
}

int moe_add_rmsnorm_backward(const moe_add_rmsnorm_backward_args* a) {
    if (int rc = moe::host::check_add_rmsnorm_backward(a)) return rc;
    const moe::NormBwdArgs n{a->T, a->H, a->dy, a->h, a->weight, a->eps, a->dh, a->dx, a->dweight,
                             static_cast<float*>(a->workspace), 1.0 / a->H};
    return done("moe_add_rmsnorm_backward", moe::launch_add_rmsnorm_backward(n, static_cast<hipStream_t>(a->stream)));
}

int moe_add_layernorm(const moe_add_layernorm_args* a) {
    if (int rc = moe::host::check_add_layernorm(a)) return rc;
    const int group = !a->yq ? 0 : a->quant == MOE_QUANT_FP8_BLOCK128 ? 128 : 32;
    const moe::NormArgs n{a->T, a->H, a->x, a->ld_x, a->residual, a->ld_residual, a->weight, a->eps,
                          a->h, a->y, a->yq, a->ys, group, 1.0 / a->H, a->bias};
    return done("moe_add_layernorm", moe::launch_add_layernorm(n, static_cast<hipStream_t>(a->stream)));
}

size_t moe_add_layernorm_backward_workspace_size(int32_t T, int32_t H) {
    return T < 1 || H < 1 ? 0 : moe::layernorm_bwd_ws_bytes(T, H);
}

int moe_add_layernorm_backward(const moe_add_layernorm_backward_args* a) {
    if (int rc = moe::host::check_add_layernorm_backward(a)) return rc;
    float* part = static_cast<float*>(a->workspace);
    const moe::NormBwdArgs n{a->T, a->H, a->dy, a->h, a->weight, a->eps, a->dh, a->dx, a->dweight,
                             part, 1.0 / a->H, a->dbias, part ? part + moe::layernorm_bwd_ws_bytes(a->T, a->H) / 8 : nullptr};
    return done("moe_add_layernorm_backward", moe::launch_add_layernorm_backward(n, static_cast<hipStream_t>(a->stream)));
}

size_t moe_linear_workspace_size(int32_t T, int32_t K, int32_t N, int32_t quant) {
    (void)T, (void)K, (void)N, (void)quant;
    return 0;
}

int moe_linear(const moe_linear_args* a) {
    if (int rc = moe::host::check_linear(a)) return rc;
    const moe::LinArgs l{a->T, a->K, a->N, a->xq, a->xs, a->w, a->w_scale, a->bias, a->residual, a->ld_residual,
                         a->y, a->ld_y, a->activation, a->out_dtype == MOE_DTYPE_BF16, a->quant == MOE_QUANT_MXFP8};
    return done("moe_linear", moe::launch_linear(l, static_cast<hipStream_t>(a->stream)));
}

int moe_gated_linear(const moe_gated_linear_args* a) {
    if (int rc = moe::host::check_gated_linear(a)) return rc;
    moe::LinArgs l{a->T, a->K, 2 * a->I, a->xq, a->xs, a->w, a->w_scale, a->bias, nullptr, 0,
                   a->h, a->I, a->activation, 1, a->quant == MOE_QUANT_MXFP8};
    l.gu = a->gu;
    return done("moe_gated_linear", moe::launch_gated_linear(l, static_cast<hipStream_t>(a->stream)));
}

size_t moe_gated_linear_backward_workspace_size(int32_t T, int32_t K, int32_t I, int32_t with_dx, int32_t with_dw,
                                                int32_t with_dbias) {
    return T < 1 || K < 1 || I < 1 ? 0 : moe::gated_bwd_plan(T, K, I, with_dx, with_dw, with_dbias).end;
}

int moe_gated_linear_backward(const moe_gated_linear_backward_args* a) {
    if (int rc = moe::host::check_gated_linear_backward(a)) return rc;
    const moe::GatedBwdArgs g{a->T, a->K, a->I, a->activation, a->quant == MOE_QUANT_MXFP8, a->dw_dtype == MOE_DTYPE_BF16,
                              a->dh, a->gu, a->xq, a->xs, a->w, a->w_scale, a->dgu, a->dx, a->dw, a->dbias,
                              static_cast<uint8_t*>(a->workspace)};
    return done("moe_gated_linear_backward", moe::launch_gated_backward(g, static_cast<hipStream_t>(a->stream)));
}

size_t moe_lora_workspace_size(int32_t T, int32_t R, int32_t num_seqs, int32_t with_offsets, int32_t out_dtype) {
    return T < 1 || R < 1 || num_seqs < 1 ? 0 : moe::lora_plan(T, R, with_offsets ? num_seqs : 0, out_dtype == MOE_DTYPE_BF16).end;
}

int moe_lora(const moe_lora_args* a) {
    if (int rc = moe::host::check_lora(a)) return rc;
    moe::LoraArgs l{a->T, a->K, a->R, a->num_adapters, a->num_seqs, a->x, a->ld_x, a->a, a->b, a->scale,
                    a->adapter_ids, a->seq_offsets, a->workspace, {}};
    l.out.N = a->N, l.out.res = a->residual, l.out.ldr = a->ld_residual;
    l.out.y = a->y, l.out.ldy = a->ld_y, l.out.out_bf16 = a->out_dtype == MOE_DTYPE_BF16;
    return done("moe_lora", moe::launch_lora(l, static_cast<hipStream_t>(a->stream)));
}

size_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t num_seqs) {
    return T < 1 || E < 1 || num_seqs < 1 ? 0 : moe::balance_plan(T, E, num_seqs).end;
}

int moe_balance_loss(const moe_balance_loss_args* a) {
    if (int rc = moe::host::check_balance_loss(a)) return rc;
    const moe::BalanceArgs b{a->T, a->route->num_experts, a->route->top_k, a->num_seqs, a->route->scoring,
                             a->router_logits, a->topk_ids, a->seq_offsets, a->balance_coef, a->z_coef, a->losses,
                             a->counts, a->mean_probs, static_cast<uint8_t*>(a->workspace)};
    return done("moe_balance_loss", moe::launch_balance_loss(b, static_cast<hipStream_t>(a->stream)));
}

int moe_route_backward(const moe_route_backward_args* a) {
    if (int rc = moe::host::check_route_backward(a)) return rc;
    const moe_route_params* p = a->route;
    const moe::RouteBwdArgs b{a->T, p->num_experts, p->top_k, a->num_seqs, p->scoring, p->renormalize != 0,
                              p->routed_scaling_factor, a->router_logits, a->topk_ids, a->dtopk_weights, a->counts,
                              a->seq_offsets, a->balance_coef, a->z_coef, a->dlogits,
                              (float)p->num_experts / (float)p->top_k};
    return done("moe_route_backward", moe::launch_route_backward(b, static_cast<hipStream_t>(a->stream)));
}

int moe_combine_backward(const moe_combine_backward_args* a) {
    if (int rc = moe::host::check_combine_backward(a)) return rc;
    const moe::CombineBwdArgs c{a->T, a->k, a->H, a->dtype == MOE_DTYPE_BF16, a->T * a->k, a->dy,
                                a->expert_out, a->assign_pos, a->topk_weights, a->dtopk_weights, a->dexpert_out,
                                a->dexpert_out && a->clear_rows};
    return done("moe_combine_backward", moe::launch_combine_backward(c, static_cast<hipStream_t>(a->stream)));
}

}  // extern "C"
