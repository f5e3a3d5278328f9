// Host-side arithmetic of the operators around the expert step (plain C++, no HIP): workspace
// layouts and the validation of every entry point's arguments, which runs before the first launch.
#include "moe_layer_plan.h"

#include <algorithm>
#include <cmath>

namespace moe {

// One workgroup per CU (16384 x 4096 with dweight 91 us, 512 workgroups 99: their partial rows cost more
// than they hide; 4096 x 1024, four rows at a time, 12.7 and 15.5), two where a thread has one vector of a
// row and each workgroup many rows (16384 x 2048: 66 us with one, 52 with two; 1000 x 2048: 10.9 and 12.9;
// 65536 x 512: 64 and 52).
int norm_bwd_parts(int T, int H) {
    if (H <= 1024) return (int)std::min<int64_t>(cdiv(T, 4), H <= 512 && T >= 32768 ? 512 : 256);
    return std::min(T, H <= 2048 && T >= 4096 ? 512 : 256);
}
size_t norm_bwd_ws_bytes(int T, int H) { return (size_t)norm_bwd_parts(T, H) * H * 4; }

// A workgroup takes 32 rows at once (8 above 256 experts) and the sequences in its rows one after the
// other.  Up to four rounds in at most four sequences, one workgroup does everything; beyond that one
// round each, or fewer rows where the sequences are shorter, and more rounds where that would be more than
// 512 workgroups (256 fill the chip; more parts only lengthen the second kernel).
BalancePlan balance_plan(int T, int E, int S) {
    BalancePlan p;
    const int round = E <= 256 ? 32 : 8;
    p.one = T <= 4 * round && S <= 4;
    p.chunk = p.one ? 4 * round : std::max(std::min<int>(round, (int)cdiv(T, S)), (int)cdiv(T, S > 256 || E > 256 ? 512 : 256));
    p.nblocks = (int)cdiv(T, p.chunk);
    p.nslots = p.nblocks + S;
    p.stride = (E + 3) / 4 * 4;
    size_t o = 0;
    auto take = [&](size_t n) {
        const size_t r = o;
        o += align256(n);
        return r;
    };
    const size_t rows = p.one ? 0 : p.nslots;
    p.probs = take(rows * p.stride * 4);
    p.hits = take(rows * p.stride * 4);
    p.z = take(rows * 4);
    p.seq = take((size_t)S * 8);
    p.done = take(4);
    p.end = o;
    return p;
}

namespace host {
namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// [p, p + n bytes) of a call's buffers; NULL pointers hold nothing
struct Span {
    const char* name;
    const void* p;
    uint64_t n;
};
bool meet(const Span& a, const Span& b) {
    return a.p && b.p && (uintptr_t)a.p < (uintptr_t)b.p + b.n && (uintptr_t)b.p < (uintptr_t)a.p + a.n;
}
// outputs may not overlap each other
int check_outputs(const char* op, const Span* out, int n) {
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (meet(out[i], out[j]))
                return fail(MOE_ERR_INVALID, "%s: %s and %s must not overlap", op, out[i].name, out[j].name);
    return MOE_OK;
}
// an output may not overlap an input, unless `same` allows exactly that buffer
int check_io(const char* op, const Span& out, const Span& in, bool same = false) {
    if (meet(out, in) && !(same && out.p == in.p))
        return fail(MOE_ERR_INVALID, "%s: %s must not overlap %s%s", op, out.name, in.name,
                    same ? " (it may be the same buffer with the same row length)" : "");
    return MOE_OK;
}

// buffers of 4-byte elements start at one
int check_words(const char* op, const Span* s, int n) {
    for (int i = 0; i < n; ++i)
        if (!aligned(s[i].p, 4)) return fail(MOE_ERR_INVALID, "%s: %s must be 4-byte aligned", op, s[i].name);
    return MOE_OK;
}

// bytes of a [rows, cols] matrix with rows ld elements apart
uint64_t span2(int64_t rows, int64_t cols, int64_t ld, int size) {
    return ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * size;
}

int check_norm_shape(const char* op, int T, int H, float eps) {
    if (T < 1 || H < 1) return fail(MOE_ERR_INVALID, "%s: T (%d) and H (%d) must be > 0", op, T, H);
    if (H % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H (%d) must be a multiple of 8", op, H);
    if (H > 32768) return fail(MOE_ERR_UNSUPPORTED, "%s: H (%d) must not exceed 32768", op, H);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID, "%s: eps must be finite and >= 0", op);
    return MOE_OK;
}

int check_router(const char* op, const moe_route_params* p, int T, int S, const int32_t* off, const float* logits,
                 float ca, float cz) {
    if (!p) return fail(MOE_ERR_INVALID, "%s: route params must not be NULL", op);
    if (T < 1) return fail(MOE_ERR_INVALID, "%s: T (%d) must be > 0", op, T);
    const int E = p->num_experts;
    if (E < 1) return fail(MOE_ERR_INVALID, "%s: num_experts (%d) must be > 0", op, E);
    if (E > MOE_MAX_EXPERTS)
        return fail(MOE_ERR_UNSUPPORTED, "%s: num_experts (%d) exceeds max %d", op, E, MOE_MAX_EXPERTS);
    if (p->top_k < 1 || p->top_k > E)
        return fail(MOE_ERR_INVALID, "%s: top_k (%d) must be in [1, num_experts=%d]", op, p->top_k, E);
    if (p->scoring != MOE_SCORING_SOFTMAX && p->scoring != MOE_SCORING_SIGMOID)
        return fail(MOE_ERR_INVALID, "%s: scoring (%d) must be 0 (softmax) or 1 (sigmoid)", op, p->scoring);
    if ((int64_t)T * p->top_k >= ((int64_t)1 << 29))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * top_k (%lld) must be below 2^29", op, (long long)T * p->top_k);
    if (S < 1) return fail(MOE_ERR_INVALID, "%s: num_seqs (%d) must be > 0", op, S);
    if (!off && S != 1) return fail(MOE_ERR_INVALID, "%s: num_seqs (%d) must be 1 without seq_offsets", op, S);
    if (S > (1 << 20)) return fail(MOE_ERR_UNSUPPORTED, "%s: num_seqs (%d) exceeds max %d", op, S, 1 << 20);
    if (!logits) return fail(MOE_ERR_INVALID, "%s: router_logits must not be NULL", op);
    if (!aligned(logits, 4) || !aligned(off, 4))
        return fail(MOE_ERR_INVALID, "%s: router_logits and seq_offsets must be 4-byte aligned", op);
    if (!std::isfinite(ca) || !std::isfinite(cz))
        return fail(MOE_ERR_INVALID, "%s: balance_coef and z_coef must be finite", op);
    return MOE_OK;
}

int check_ws(const char* op, const void* ws, size_t have, size_t need) {
    if (!need) return MOE_OK;
    if (!ws || have < need)
        return fail(MOE_ERR_WORKSPACE, "%s: workspace too small: need %zu bytes, have %zu", op, need,
                    ws ? have : (size_t)0);
    if (!aligned(ws, 256)) return fail(MOE_ERR_INVALID, "%s: workspace must be 256-byte aligned", op);
    return MOE_OK;
}

}  // namespace

int check_add_rmsnorm(const moe_add_rmsnorm_args* a) {
    const char* op = "moe_add_rmsnorm";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    int rc = check_norm_shape(op, a->T, a->H, a->eps);
    if (rc) return rc;
    const int T = a->T, H = a->H;
    if (!a->x || !a->weight) return fail(MOE_ERR_INVALID, "%s: x and weight must not be NULL", op);
    if (!a->h && !a->y && !a->yq) return fail(MOE_ERR_INVALID, "%s: one of h, y and yq must be given", op);
    if (!a->yq != !a->ys) return fail(MOE_ERR_INVALID, "%s: yq and ys come together", op);
    int group = 0;
    if (a->yq) {
        if (a->quant == MOE_QUANT_FP8_BLOCK128) group = 128;
        else if (a->quant == MOE_QUANT_MXFP8 || a->quant == MOE_QUANT_W4A8) group = 32;
        else return fail(MOE_ERR_INVALID, "%s: quant (%d) must be a scheme that quantises activations", op, a->quant);
        if (H % group)
            return fail(MOE_ERR_UNSUPPORTED, "%s: H (%d) must be a multiple of %d with codes", op, H, group);
        if (!aligned(a->yq, 8)) return fail(MOE_ERR_UNSUPPORTED, "%s: yq must be 8-byte aligned", op);
    }
    if (a->ld_x < H || (a->residual && a->ld_residual < H))
        return fail(MOE_ERR_INVALID, "%s: ld_x (%lld) and ld_residual (%lld) must be >= H (%d)", op,
                    (long long)a->ld_x, (long long)a->ld_residual, H);
    if (a->ld_x % 8 || (a->residual && a->ld_residual % 8) || !aligned(a->x, 16) || !aligned(a->residual, 16) ||
        !aligned(a->weight, 16) || !aligned(a->h, 16) || !aligned(a->y, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: x, residual, weight, h and y must be 16-byte aligned, rows a multiple of "
                    "8 elements apart", op);
    const Span x{"x", a->x, span2(T, H, a->ld_x, 2)};
    const Span res{"residual", a->residual, a->residual ? span2(T, H, a->ld_residual, 2) : 0};
    const Span w{"weight", a->weight, (uint64_t)H * 4};
    const uint64_t n = (uint64_t)T * H;
    const Span out[4] = {{"h", a->h, n * 2}, {"y", a->y, n * 2}, {"yq", a->yq, n}, {"ys", a->ys, group ? n / group : 0}};
    if ((rc = check_outputs(op, out, 4))) return rc;
    for (int i = 0; i < 4; ++i) {
        if ((rc = check_io(op, out[i], x, i < 2 && a->ld_x == H))) return rc;
        if ((rc = check_io(op, out[i], res, i == 0 && a->ld_residual == H))) return rc;
        if ((rc = check_io(op, out[i], w))) return rc;
    }
    return MOE_OK;
}

int check_add_rmsnorm_backward(const moe_add_rmsnorm_backward_args* a) {
    const char* op = "moe_add_rmsnorm_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    int rc = check_norm_shape(op, a->T, a->H, a->eps);
    if (rc) return rc;
    if (!a->dy || !a->h || !a->weight || !a->dx)
        return fail(MOE_ERR_INVALID, "%s: dy, h, weight and dx must not be NULL", op);
    if (!aligned(a->dy, 16) || !aligned(a->h, 16) || !aligned(a->weight, 16) || !aligned(a->dh, 16) || !aligned(a->dx, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: dy, h, weight, dh and dx must be 16-byte aligned", op);
    if (!aligned(a->dweight, 4)) return fail(MOE_ERR_INVALID, "%s: dweight must be 4-byte aligned", op);
    const size_t need = a->dweight ? norm_bwd_ws_bytes(a->T, a->H) : 0;
    const uint64_t n = (uint64_t)a->T * a->H * 2, nw = (uint64_t)a->H * 4;
    const Span out[3] = {{"dx", a->dx, n}, {"dweight", a->dweight, nw}, {"workspace", need ? a->workspace : nullptr, need}};
    const Span in[4] = {{"dy", a->dy, n}, {"h", a->h, n}, {"dh", a->dh, n}, {"weight", a->weight, nw}};
    if ((rc = check_ws(op, a->workspace, a->workspace_bytes, need))) return rc;
    if ((rc = check_outputs(op, out, 3))) return rc;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 4; ++j)
            if ((rc = check_io(op, out[i], in[j], i == 0 && (j == 0 || j == 2)))) return rc;
    return MOE_OK;
}

int check_linear(const moe_linear_args* a) {
    const char* op = "moe_linear";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    const int T = a->T, K = a->K, N = a->N;
    if (T < 1 || K < 1 || N < 1) return fail(MOE_ERR_INVALID, "%s: T, K, N (%d, %d, %d) must be > 0", op, T, K, N);
    if (a->quant < MOE_QUANT_FP8_BLOCK128 || a->quant > MOE_QUANT_W8A16)
        return fail(MOE_ERR_INVALID, "%s: quant (%d) must be one of MOE_QUANT_*", op, a->quant);
    if (a->quant != MOE_QUANT_FP8_BLOCK128 && a->quant != MOE_QUANT_MXFP8)
        return fail(MOE_ERR_UNSUPPORTED, "%s: quant (%d) must be MOE_QUANT_FP8_BLOCK128 or MOE_QUANT_MXFP8", op, a->quant);
    const bool mx = a->quant == MOE_QUANT_MXFP8;
    if (K % 128) return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) must be a multiple of 128", op, K);
    if (K > 32768) return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) must not exceed 32768", op, K);
    if (N % 16) return fail(MOE_ERR_UNSUPPORTED, "%s: N (%d) must be a multiple of 16", op, N);
    if ((int64_t)T * K >= ((int64_t)1 << 31) || (int64_t)K * N >= ((int64_t)1 << 31))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * K (%lld) and K * N (%lld) must be below 2^31 (32-bit offsets)", op,
                    (long long)T * K, (long long)K * N);
    if ((int64_t)T * N >= ((int64_t)1 << 40))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * N (%lld) must be below 2^40", op, (long long)T * N);
    if (!a->xq || !a->xs || !a->w || !a->w_scale || !a->y)
        return fail(MOE_ERR_INVALID, "%s: xq, xs, w, w_scale and y must not be NULL", op);
    if (a->activation < MOE_ACT_NONE || a->activation > MOE_ACT_GELU_TANH)
        return fail(MOE_ERR_INVALID, "%s: activation (%d) must be one of MOE_ACT_*", op, a->activation);
    if (a->out_dtype != MOE_DTYPE_F32 && a->out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID, "%s: out_dtype (%d) must be MOE_DTYPE_F32 or MOE_DTYPE_BF16", op, a->out_dtype);
    if (a->ld_y < N || (a->residual && a->ld_residual < N))
        return fail(MOE_ERR_INVALID, "%s: ld_y (%lld) and ld_residual (%lld) must be >= N (%d)", op, (long long)a->ld_y,
                    (long long)a->ld_residual, N);
    if (a->ld_y % 8 || (a->residual && a->ld_residual % 8) || !aligned(a->y, 16) || !aligned(a->residual, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: y and residual must be 16-byte aligned, rows a multiple of 8 elements "
                    "apart", op);
    if (!aligned(a->xq, 16) || !aligned(a->w, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: xq and w must be 16-byte aligned", op);
    if (mx && (!aligned(a->xs, 4) || !aligned(a->w_scale, 4)))
        return fail(MOE_ERR_UNSUPPORTED, "%s: xs and w_scale must be 4-byte aligned for MOE_QUANT_MXFP8", op);
    if (!aligned(a->bias, 4)) return fail(MOE_ERR_INVALID, "%s: bias must be 4-byte aligned", op);
    const int size = a->out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    const Span y{"y", a->y, span2(T, N, a->ld_y, size)};
    const Span in[6] = {{"xq", a->xq, (uint64_t)T * K},
                        {"xs", a->xs, (uint64_t)T * (K / (mx ? 32 : 128))},
                        {"w", a->w, (uint64_t)K * N},
                        {"w_scale", a->w_scale, mx ? (uint64_t)K * N / 32 : (uint64_t)(K / 128) * cdiv(N, 128)},
                        {"bias", a->bias, (uint64_t)N * 4},
                        {"residual", a->residual, a->residual ? span2(T, N, a->ld_residual, size) : 0}};
    for (int i = 0; i < 5; ++i)
        if (int rc = check_io(op, y, in[i])) return rc;
    // y and residual may be columns side by side in the rows of one matrix: their spans meet, they do not
    if (a->residual && a->ld_residual == a->ld_y) {
        const uint64_t row = (uint64_t)a->ld_y * size, used = (uint64_t)N * size;
        const uint64_t d = ((uintptr_t)a->y > (uintptr_t)a->residual ? (uintptr_t)a->y - (uintptr_t)a->residual
                                                                     : (uintptr_t)a->residual - (uintptr_t)a->y) % row;
        if (a->y != a->residual && d >= used && row - d >= used) return MOE_OK;
    }
    if (int rc = check_io(op, y, in[5], a->ld_residual == a->ld_y)) return rc;
    return MOE_OK;
}

int check_balance_loss(const moe_balance_loss_args* a) {
    const char* op = "moe_balance_loss";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    int rc = check_router(op, a->route, a->T, a->num_seqs, a->seq_offsets, a->router_logits, a->balance_coef, a->z_coef);
    if (rc) return rc;
    if (!a->topk_ids || !a->losses || !a->counts)
        return fail(MOE_ERR_INVALID, "%s: topk_ids, losses and counts must not be NULL", op);
    const int T = a->T, E = a->route->num_experts, k = a->route->top_k, S = a->num_seqs;
    if ((int64_t)S * E >= ((int64_t)1 << 30))
        return fail(MOE_ERR_UNSUPPORTED, "%s: num_seqs * num_experts (%lld) must be below 2^30", op, (long long)S * E);
    const size_t need = balance_plan(T, E, S).end;
    if ((rc = check_ws(op, a->workspace, a->workspace_bytes, need))) return rc;
    const Span out[4] = {{"losses", a->losses, 12},
                         {"counts", a->counts, (uint64_t)S * E * 4},
                         {"mean_probs", a->mean_probs, (uint64_t)S * E * 4},
                         {"workspace", a->workspace, need}};
    const Span in[3] = {{"router_logits", a->router_logits, (uint64_t)T * E * 4},
                        {"topk_ids", a->topk_ids, (uint64_t)T * k * 4},
                        {"seq_offsets", a->seq_offsets, (uint64_t)(S + 1) * 4}};
    if ((rc = check_words(op, out, 3)) || (rc = check_words(op, in, 3))) return rc;
    if ((rc = check_outputs(op, out, 4))) return rc;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 3; ++j)
            if ((rc = check_io(op, out[i], in[j]))) return rc;
    return MOE_OK;
}

int check_route_backward(const moe_route_backward_args* a) {
    const char* op = "moe_route_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    int rc = check_router(op, a->route, a->T, a->num_seqs, a->seq_offsets, a->router_logits, a->balance_coef, a->z_coef);
    if (rc) return rc;
    if (!a->dlogits) return fail(MOE_ERR_INVALID, "%s: dlogits must not be NULL", op);
    if (a->dtopk_weights && !a->topk_ids) return fail(MOE_ERR_INVALID, "%s: dtopk_weights needs topk_ids", op);
    if (!std::isfinite(a->route->routed_scaling_factor))
        return fail(MOE_ERR_INVALID, "%s: routed_scaling_factor must be finite", op);
    const int T = a->T, E = a->route->num_experts, k = a->route->top_k, S = a->num_seqs;
    const Span out{"dlogits", a->dlogits, (uint64_t)T * E * 4};
    const Span in[5] = {{"router_logits", a->router_logits, (uint64_t)T * E * 4},
                        {"topk_ids", a->topk_ids, (uint64_t)T * k * 4},
                        {"dtopk_weights", a->dtopk_weights, (uint64_t)T * k * 4},
                        {"counts", a->counts, (uint64_t)S * E * 4},
                        {"seq_offsets", a->seq_offsets, (uint64_t)(S + 1) * 4}};
    if ((rc = check_words(op, &out, 1)) || (rc = check_words(op, in, 5))) return rc;
    for (int j = 0; j < 5; ++j)
        if ((rc = check_io(op, out, in[j], j == 0))) return rc;
    return MOE_OK;
}

int check_combine_backward(const moe_combine_backward_args* a) {
    const char* op = "moe_combine_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    const int T = a->T, k = a->k, H = a->H;
    if (T < 1 || k < 1 || H < 1) return fail(MOE_ERR_INVALID, "%s: T, k, H (%d, %d, %d) must be > 0", op, T, k, H);
    if (a->dtype != MOE_DTYPE_F32 && a->dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID, "%s: dtype (%d) must be MOE_DTYPE_F32 or MOE_DTYPE_BF16", op, a->dtype);
    if (H % 8) return fail(MOE_ERR_UNSUPPORTED, "%s: H (%d) must be a multiple of 8", op, H);
    if ((int64_t)T * k >= ((int64_t)1 << 29))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * k (%lld) must be below 2^29", op, (long long)T * k);
    if (!a->dy || !a->assign_pos) return fail(MOE_ERR_INVALID, "%s: dy and assign_pos must not be NULL", op);
    if (!a->dtopk_weights && !a->dexpert_out)
        return fail(MOE_ERR_INVALID, "%s: one of dtopk_weights and dexpert_out must be given", op);
    if (a->dtopk_weights && !a->expert_out) return fail(MOE_ERR_INVALID, "%s: dtopk_weights needs expert_out", op);
    if (a->dexpert_out && !a->topk_weights) return fail(MOE_ERR_INVALID, "%s: dexpert_out needs topk_weights", op);
    if (a->clear_rows != 0 && a->clear_rows != 1)
        return fail(MOE_ERR_INVALID, "%s: clear_rows (%d) must be 0 or 1", op, a->clear_rows);
    if (!aligned(a->dy, 16) || !aligned(a->expert_out, 16) || !aligned(a->dexpert_out, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: dy, expert_out and dexpert_out must be 16-byte aligned", op);
    const uint64_t ne = (uint64_t)T * k * H * (a->dtype == MOE_DTYPE_BF16 ? 2 : 4), nk = (uint64_t)T * k * 4;
    const Span out[2] = {{"dtopk_weights", a->dtopk_weights, nk}, {"dexpert_out", a->dexpert_out, ne}};
    const Span in[4] = {{"dy", a->dy, (uint64_t)T * H * 2}, {"expert_out", a->expert_out, ne},
                        {"assign_pos", a->assign_pos, nk}, {"topk_weights", a->topk_weights, nk}};
    if (int rc = check_words(op, out, 1)) return rc;
    if (int rc = check_words(op, in + 2, 2)) return rc;
    if (int rc = check_outputs(op, out, 2)) return rc;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 4; ++j)
            if (int rc = check_io(op, out[i], in[j], i == 1 && j == 1 && !a->clear_rows)) return rc;
    return MOE_OK;
}

}  // namespace host
}  // namespace moe
