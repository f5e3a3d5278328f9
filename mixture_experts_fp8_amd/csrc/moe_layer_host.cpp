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
// The layer norm forms more sums per row, which more workgroups hide where a thread has two vectors (16384 x 4096:
// 110 us with 512 workgroups, and when those took 107, 143 with 256 of 512 threads; 16384 x 2048: 68 with 1024, 74 with
// 512 and one vector per thread), once each has several rows (1000 x 4096: 17.1 us with 256, 19.8 with 512).
int layernorm_bwd_parts(int T, int H) {
    if (H <= 1024 || H > 4096) return norm_bwd_parts(T, H);
    return std::min(T, T < 4096 ? 256 : H <= 2048 ? 1024 : 512);
}
size_t norm_bwd_ws_bytes(int T, int H) { return (size_t)norm_bwd_parts(T, H) * H * 4; }
size_t layernorm_bwd_ws_bytes(int T, int H) { return 2 * (size_t)layernorm_bwd_parts(T, H) * H * 4; }

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

// Tile and parts of the gated block's two products by the time that they are estimated to take.  A workgroup
// takes `busy` us per K block of 64 where all `slots` of the chip have one, `alone` us at least, and `fixed` us per
// tile; the launch takes the longer of the work shared by the slots and of the longest chain, and a quarter of the
// other.  The table is fitted to 16 shapes from 16 x 4096 x 1536 to 16384 x 2048 x 1024 with every tile: 7 to
// 9% off in the mean, and never more than 9% from the fastest of the five (4096 x 7168 x 2048: 408 us with the last
// row's tiles, 518, 632, 761 and 867 with the others'; 300 x 768 x 1152: 21 us with the first's, 43 with the last's).
// Parts: a long sum over few tiles is split over workgroups, whose float32 parts a third launch joins (3 us
// and their bytes at 4 TB/s), where the estimate gains by it: 16384 x 768 x 256 has 256 blocks per tile of dw.
ProductPlan product_plan(int T, int K, int I, bool dx, bool dw) {
    static const struct {
        int rows, cols, slots;
        double busy, alone, fixed;
    } tiles[5] = {{64, 64, 256, 0.147, 0.199, 2.0},    // two sets of waves over the K blocks
                  {64, 128, 256, 0.286, 0.286, 2.0},   // four stages, one workgroup per CU
                  {64, 128, 512, 0.434, 0.367, 3.6},   // three, two
                  {128, 256, 256, 0.70, 0.61, 4.8},    // eight waves
                  {128, 256, 512, 1.16, 0.73, 4.8}};   // weights straight to registers
    const int rows[2] = {T, K}, cols[2] = {K, 2 * I}, blocks[2] = {I / 32, (int)cdiv(T, 64)};
    const bool on[2] = {dx, dw};
    ProductPlan best{0, {dx, dw}, blocks[0] > blocks[1]};
    double least = 1e30;
    for (int t = 0; t < 5; ++t) {
        struct {
            double work, chain, join;
        } of[2][5] = {};   // of a product in 2^p parts
        int most[2] = {0, 0};
        for (int i = 0; i < 2; ++i) {
            if (!on[i]) continue;
            const double n = (double)(cdiv(rows[i], tiles[t].rows) * cdiv(cols[i], tiles[t].cols));
            for (int p = 0; p < 5; ++p) {
                const int parts = 1 << p;
                const int64_t per = cdiv(blocks[i], parts);
                if (p && per < 4) break;
                most[i] = p;
                of[i][p] = {n * parts * (per * tiles[t].busy + tiles[t].fixed) / tiles[t].slots,
                            p && per * (parts - 1) >= blocks[i] ? 1e30 : per * tiles[t].alone + tiles[t].fixed,   // (an empty part)
                            p ? (double)rows[i] * cols[i] * parts * 8 / 4e6 : 0};
            }
        }
        for (int a = 0; a <= most[0]; ++a)
            for (int b = 0; b <= most[1]; ++b) {
                const auto &x = of[0][a], &w = of[1][b];
                const double work = x.work + w.work, chain = std::max(x.chain, w.chain);
                const double us = std::max(work, chain) + 0.25 * std::min(work, chain) + x.join + w.join + (a || b ? 3 : 0);
                if (us < least) {
                    least = us;
                    best.tile = t;
                    best.parts[0] = dx ? 1 << a : 0;
                    best.parts[1] = dw ? 1 << b : 0;
                }
            }
    }
    return best;
}

GatedBwdPlan gated_bwd_plan(int T, int K, int I, bool dx, bool dw, bool dbias) {
    GatedBwdPlan p;
    p.row_blocks = (int)cdiv(T, 64);
    p.parts = std::min(p.row_blocks, 256);
    p.product = product_plan(T, K, I, dx, dw);
    const size_t N = 2 * (size_t)I, rows = 64 * (size_t)p.row_blocks;
    size_t o = 0;
    auto take = [&](bool on, size_t n) {
        const size_t r = o;
        if (on) o += align256(n);
        return r;
    };
    p.part = take(dbias, p.parts * N * 4);
    p.weights = take(dx, K * N * 2);
    p.rows = take(dw, K * rows * 2);
    p.dgu_packed = take(dw, N * rows * 2);
    p.join[0] = take(p.product.parts[0] > 1, (size_t)p.product.parts[0] * T * K * 4);
    p.join[1] = take(p.product.parts[1] > 1, (size_t)p.product.parts[1] * K * N * 4);
    p.end = o;
    return p;
}

// Windows of 32 rows read an adapter's matrices half as often as those of 16, from half as many workgroups, and are half
// empty where sequences are short.  Both measured on 4096 x 4096 with 1 to 4000 sequences; the time with 32 over the
// time with 16, its range (and mean):
//   rows, 24 and more per sequence   500, 1000        1400, 1800       2047 to 3400     5000, 8000       16384, 32768
//   ranks 16 to 64                   1.04-1.30 (1.13) 0.94-1.12 (1.04) 0.87-1.15 (1.00) 0.89-1.11 (1.00) 0.80-1.04 (0.92)
//   rank 128                         0.97-1.30 (1.06) 0.82-1.04 (0.94) 0.76-1.07 (0.91) 0.86-0.95 (0.91) 0.74-0.78 (0.76)
//   rows per sequence, 2047 to 16000 rows   4         8                12, 16           20, 24           32
//   ranks 16 to 128                         1.14-1.28 1.05-1.22        0.96-1.14        0.91-1.14        0.87-1.08
// So 32 from 2000 rows and 24 rows per sequence on.  Single sizes near those borders lie up to 15% on either side, with
// how the slots fall on the CUs; rank 128 would gain from 1400 rows on, and rank 16 gains nothing before 32768.
LoraPlan lora_plan(int T, int R, int S, bool bf16) {
    LoraPlan p;
    p.window = S && T >= 2000 && T / S >= 24 ? 32 : 16;
    p.slots = S ? cdiv(T, p.window) + S : T;
    p.steps = (int)cdiv(R, 32);
    p.split = bf16 ? 2 : 3;
    p.end = (size_t)p.slots * (p.window / 16) * p.steps * p.split * 1024;
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

// y [.., N] may be the residual itself, or other columns of one matrix's rows: side by side their spans meet,
// they do not.
int check_residual(const char* op, const Span& y, const Span& res, int64_t ld_y, int64_t ld_res, int N, int size) {
    if (res.p && ld_res == ld_y) {
        const uint64_t row = (uint64_t)ld_y * size, used = (uint64_t)N * size;
        const uintptr_t p = (uintptr_t)y.p, q = (uintptr_t)res.p;
        const uint64_t d = (p > q ? p - q : q - p) % row;
        if (p != q && d >= used && row - d >= used) return MOE_OK;
    }
    return check_io(op, y, res, ld_res == ld_y);
}

// Scheme, depth and activation of a gated block's products of T rows, N = 2I wide.
int check_gated(const char* op, int T, int K, int64_t N, int quant, int activation) {
    if (quant < MOE_QUANT_FP8_BLOCK128 || quant > MOE_QUANT_W8A16)
        return fail(MOE_ERR_INVALID, "%s: quant (%d) must be one of MOE_QUANT_*", op, quant);
    if (quant != MOE_QUANT_FP8_BLOCK128 && quant != MOE_QUANT_MXFP8)
        return fail(MOE_ERR_UNSUPPORTED, "%s: quant (%d) must be MOE_QUANT_FP8_BLOCK128 or MOE_QUANT_MXFP8", op, quant);
    if (K % 128) return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) must be a multiple of 128", op, K);
    if (K > 32768) return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) must not exceed 32768", op, K);
    if ((int64_t)T * K >= ((int64_t)1 << 31) || K * N >= ((int64_t)1 << 31))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * K (%lld) and K * 2I (%lld) must be below 2^31 (32-bit offsets)", op,
                    (long long)T * K, (long long)(K * N));
    if (activation < MOE_ACT_NONE || activation > MOE_ACT_GELU_TANH)
        return fail(MOE_ERR_INVALID, "%s: activation (%d) must be one of MOE_ACT_*", op, activation);
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

template <typename Args>
int check_norm(const char* op, const Args* a, const float* bias) {
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
        !aligned(a->weight, 16) || !aligned(bias, 16) || !aligned(a->h, 16) || !aligned(a->y, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: x, residual, weight%s, h and y must be 16-byte aligned, rows a multiple of "
                    "8 elements apart", op, bias ? ", bias" : "");
    const Span x{"x", a->x, span2(T, H, a->ld_x, 2)};
    const Span res{"residual", a->residual, a->residual ? span2(T, H, a->ld_residual, 2) : 0};
    const Span w{"weight", a->weight, (uint64_t)H * 4}, b{"bias", bias, (uint64_t)H * 4};
    const uint64_t n = (uint64_t)T * H;
    const Span out[4] = {{"h", a->h, n * 2}, {"y", a->y, n * 2}, {"yq", a->yq, n}, {"ys", a->ys, group ? n / group : 0}};
    if ((rc = check_outputs(op, out, 4))) return rc;
    for (int i = 0; i < 4; ++i) {
        if ((rc = check_io(op, out[i], x, i < 2 && a->ld_x == H))) return rc;
        if ((rc = check_io(op, out[i], res, i == 0 && a->ld_residual == H))) return rc;
        if ((rc = check_io(op, out[i], w)) || (rc = check_io(op, out[i], b))) return rc;
    }
    return MOE_OK;
}

template <typename Args>
int check_norm_backward(const char* op, const Args* a, float* dbias, size_t need) {
    int rc = check_norm_shape(op, a->T, a->H, a->eps);
    if (rc) return rc;
    if (!a->dy || !a->h || !a->weight || !a->dx)
        return fail(MOE_ERR_INVALID, "%s: dy, h, weight and dx must not be NULL", op);
    if (!aligned(a->dy, 16) || !aligned(a->h, 16) || !aligned(a->weight, 16) || !aligned(a->dh, 16) || !aligned(a->dx, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: dy, h, weight, dh and dx must be 16-byte aligned", op);
    if (!aligned(a->dweight, 4)) return fail(MOE_ERR_INVALID, "%s: dweight must be 4-byte aligned", op);
    if (!aligned(dbias, 4)) return fail(MOE_ERR_INVALID, "%s: dbias must be 4-byte aligned", op);
    if (!a->dweight && !dbias) need = 0;
    const uint64_t n = (uint64_t)a->T * a->H * 2, nw = (uint64_t)a->H * 4;
    const Span out[4] = {{"dx", a->dx, n}, {"dweight", a->dweight, nw}, {"dbias", dbias, nw},
                         {"workspace", need ? a->workspace : nullptr, need}};
    const Span in[4] = {{"dy", a->dy, n}, {"h", a->h, n}, {"dh", a->dh, n}, {"weight", a->weight, nw}};
    if ((rc = check_ws(op, a->workspace, a->workspace_bytes, need))) return rc;
    if ((rc = check_outputs(op, out, 4))) return rc;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
            if ((rc = check_io(op, out[i], in[j], i == 0 && (j == 0 || j == 2)))) return rc;
    return MOE_OK;
}

}  // namespace

int check_add_rmsnorm(const moe_add_rmsnorm_args* a) {
    const char* op = "moe_add_rmsnorm";
    return a ? check_norm(op, a, nullptr) : fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
}
int check_add_layernorm(const moe_add_layernorm_args* a) {
    const char* op = "moe_add_layernorm";
    return a ? check_norm(op, a, a->bias) : fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
}
int check_add_rmsnorm_backward(const moe_add_rmsnorm_backward_args* a) {
    const char* op = "moe_add_rmsnorm_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    return check_norm_backward(op, a, nullptr, a->T < 1 || a->H < 1 ? 0 : norm_bwd_ws_bytes(a->T, a->H));
}
int check_add_layernorm_backward(const moe_add_layernorm_backward_args* a) {
    const char* op = "moe_add_layernorm_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    return check_norm_backward(op, a, a->dbias, a->T < 1 || a->H < 1 ? 0 : layernorm_bwd_ws_bytes(a->T, a->H));
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
    return check_residual(op, y, in[5], a->ld_y, a->ld_residual, N, size);
}

int check_gated_linear(const moe_gated_linear_args* a) {
    const char* op = "moe_gated_linear";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    const int T = a->T, K = a->K, I = a->I;
    if (T < 1 || K < 1 || I < 1) return fail(MOE_ERR_INVALID, "%s: T, K, I (%d, %d, %d) must be > 0", op, T, K, I);
    if (I % 32) return fail(MOE_ERR_UNSUPPORTED, "%s: I (%d) must be a multiple of 32", op, I);
    const int64_t N = 2 * (int64_t)I;
    int rc = check_gated(op, T, K, N, a->quant, a->activation);
    if (rc) return rc;
    if (T * N >= ((int64_t)1 << 40))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * 2I (%lld) must be below 2^40", op, (long long)(T * N));
    if (!a->xq || !a->xs || !a->w || !a->w_scale || !a->h)
        return fail(MOE_ERR_INVALID, "%s: xq, xs, w, w_scale and h must not be NULL", op);
    if (!aligned(a->xq, 16) || !aligned(a->w, 16) || !aligned(a->h, 16) || !aligned(a->gu, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: xq, w, h and gu must be 16-byte aligned", op);
    const bool mx = a->quant == MOE_QUANT_MXFP8;
    if (mx && (!aligned(a->xs, 4) || !aligned(a->w_scale, 4)))
        return fail(MOE_ERR_UNSUPPORTED, "%s: xs and w_scale must be 4-byte aligned for MOE_QUANT_MXFP8", op);
    if (!aligned(a->bias, 4)) return fail(MOE_ERR_INVALID, "%s: bias must be 4-byte aligned", op);
    const Span out[2] = {{"h", a->h, (uint64_t)T * I * 2}, {"gu", a->gu, (uint64_t)T * N * 2}};
    const Span in[5] = {{"xq", a->xq, (uint64_t)T * K},
                        {"xs", a->xs, (uint64_t)T * (K / (mx ? 32 : 128))},
                        {"w", a->w, (uint64_t)K * N},
                        {"w_scale", a->w_scale, mx ? (uint64_t)K * N / 32 : (uint64_t)(K / 128) * cdiv(N, 128)},
                        {"bias", a->bias, (uint64_t)N * 4}};
    if ((rc = check_outputs(op, out, 2))) return rc;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 5; ++j)
            if ((rc = check_io(op, out[i], in[j]))) return rc;
    return MOE_OK;
}

int check_gated_linear_backward(const moe_gated_linear_backward_args* a) {
    const char* op = "moe_gated_linear_backward";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    const int T = a->T, K = a->K, I = a->I;
    if (T < 1 || K < 1 || I < 1) return fail(MOE_ERR_INVALID, "%s: T, K, I (%d, %d, %d) must be > 0", op, T, K, I);
    if (I % 32) return fail(MOE_ERR_UNSUPPORTED, "%s: I (%d) must be a multiple of 32", op, I);
    const int64_t N = 2 * (int64_t)I, rows = cdiv(T, 64) * 64;
    int rc = check_gated(op, T, K, N, a->quant, a->activation);
    if (rc) return rc;
    if (rows * N >= ((int64_t)1 << 30) || rows * K >= ((int64_t)1 << 30) || K * N >= ((int64_t)1 << 30))
        return fail(MOE_ERR_UNSUPPORTED, "%s: T * 2I, T * K (T up to a multiple of 64) and K * 2I must be below 2^30", op);
    if (!a->dh || !a->gu || !a->dgu) return fail(MOE_ERR_INVALID, "%s: dh, gu and dgu must not be NULL", op);
    if (a->dx && (!a->w || !a->w_scale)) return fail(MOE_ERR_INVALID, "%s: dx needs w and w_scale", op);
    if (a->dw && (!a->xq || !a->xs)) return fail(MOE_ERR_INVALID, "%s: dw needs xq and xs", op);
    if (a->dw && a->dw_dtype != MOE_DTYPE_F32 && a->dw_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID, "%s: dw_dtype (%d) must be MOE_DTYPE_F32 or MOE_DTYPE_BF16", op, a->dw_dtype);
    if (!aligned(a->dh, 16) || !aligned(a->gu, 16) || !aligned(a->dgu, 16) || !aligned(a->dx, 16) || !aligned(a->dw, 16) ||
        !aligned(a->xq, 16) || !aligned(a->w, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: dh, gu, dgu, dx, dw, xq and w must be 16-byte aligned", op);
    const bool mx = a->quant == MOE_QUANT_MXFP8;
    if (mx && (!aligned(a->xs, 4) || !aligned(a->w_scale, 4)))
        return fail(MOE_ERR_UNSUPPORTED, "%s: xs and w_scale must be 4-byte aligned for MOE_QUANT_MXFP8", op);
    if (!aligned(a->dbias, 4)) return fail(MOE_ERR_INVALID, "%s: dbias must be 4-byte aligned", op);
    const size_t need = gated_bwd_plan(T, K, I, a->dx, a->dw, a->dbias).end;
    if ((rc = check_ws(op, a->workspace, a->workspace_bytes, need))) return rc;
    const Span out[5] = {{"dgu", a->dgu, (uint64_t)T * N * 2},
                         {"dx", a->dx, (uint64_t)T * K * 2},
                         {"dw", a->dw, (uint64_t)K * N * (a->dw_dtype == MOE_DTYPE_BF16 ? 2 : 4)},
                         {"dbias", a->dbias, (uint64_t)N * 4},
                         {"workspace", need ? a->workspace : nullptr, need}};
    const Span in[6] = {{"gu", a->gu, (uint64_t)T * N * 2},
                        {"dh", a->dh, (uint64_t)T * I * 2},
                        {"xq", a->dw ? a->xq : nullptr, (uint64_t)T * K},
                        {"xs", a->dw ? a->xs : nullptr, (uint64_t)T * (K / (mx ? 32 : 128))},
                        {"w", a->dx ? a->w : nullptr, (uint64_t)K * N},
                        {"w_scale", a->dx ? a->w_scale : nullptr, mx ? (uint64_t)K * N / 32 : (uint64_t)(K / 128) * cdiv(N, 128)}};
    if ((rc = check_outputs(op, out, 5))) return rc;
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 6; ++j)
            if ((rc = check_io(op, out[i], in[j], i == 0 && j == 0))) return rc;
    return MOE_OK;
}

int check_lora(const moe_lora_args* a) {
    const char* op = "moe_lora";
    if (!a) return fail(MOE_ERR_INVALID, "%s: args must not be NULL", op);
    const int T = a->T, K = a->K, N = a->N, R = a->R, S = a->num_seqs;
    if (T < 1 || K < 1 || N < 1 || R < 1)
        return fail(MOE_ERR_INVALID, "%s: T, K, N, R (%d, %d, %d, %d) must be > 0", op, T, K, N, R);
    if (a->num_adapters < 1) return fail(MOE_ERR_INVALID, "%s: num_adapters (%d) must be > 0", op, a->num_adapters);
    if (K % 8 || R % 8 || N % 16)
        return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) and R (%d) must be multiples of 8, N (%d) of 16", op, K, R, N);
    if (R > 256) return fail(MOE_ERR_UNSUPPORTED, "%s: R (%d) must not exceed 256", op, R);
    if (K > 65536 || N > (1 << 20))
        return fail(MOE_ERR_UNSUPPORTED, "%s: K (%d) must not exceed 65536, N (%d) %d", op, K, N, 1 << 20);
    if (S < 1) return fail(MOE_ERR_INVALID, "%s: num_seqs (%d) must be > 0", op, S);
    if (!a->seq_offsets && S != T)
        return fail(MOE_ERR_INVALID, "%s: num_seqs (%d) must be T (%d) without seq_offsets", op, S, T);
    if (S > (1 << 20) || T > (1 << 23))
        return fail(MOE_ERR_UNSUPPORTED, "%s: num_seqs (%d) must not exceed %d, T (%d) %d", op, S, 1 << 20, T, 1 << 23);
    if (!a->x || !a->a || !a->b || !a->adapter_ids || !a->y)
        return fail(MOE_ERR_INVALID, "%s: x, a, b, adapter_ids and y must not be NULL", op);
    if (a->out_dtype != MOE_DTYPE_F32 && a->out_dtype != MOE_DTYPE_BF16)
        return fail(MOE_ERR_INVALID, "%s: out_dtype (%d) must be MOE_DTYPE_F32 or MOE_DTYPE_BF16", op, a->out_dtype);
    if (a->ld_x < K) return fail(MOE_ERR_INVALID, "%s: ld_x (%lld) must be >= K (%d)", op, (long long)a->ld_x, K);
    if (a->ld_x > (1 << 24))   // 32 rows of a window within 2^30 bytes, a quarter of what the kernel's offsets hold
        return fail(MOE_ERR_UNSUPPORTED, "%s: ld_x (%lld) must not exceed %d", op, (long long)a->ld_x, 1 << 24);
    if (a->ld_y < N || (a->residual && a->ld_residual < N))
        return fail(MOE_ERR_INVALID, "%s: ld_y (%lld) and ld_residual (%lld) must be >= N (%d)", op, (long long)a->ld_y,
                    (long long)a->ld_residual, N);
    if (a->ld_x % 8 || a->ld_y % 8 || (a->residual && a->ld_residual % 8) || !aligned(a->x, 16) || !aligned(a->y, 16) ||
        !aligned(a->residual, 16) || !aligned(a->a, 16) || !aligned(a->b, 16))
        return fail(MOE_ERR_UNSUPPORTED, "%s: x, a, b, residual and y must be 16-byte aligned, rows a multiple of 8 "
                    "elements apart", op);
    const size_t need = lora_plan(T, R, a->seq_offsets ? S : 0, a->out_dtype == MOE_DTYPE_BF16).end;
    int rc = check_ws(op, a->workspace, a->workspace_bytes, need);
    if (rc) return rc;
    const int size = a->out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    const uint64_t n = a->num_adapters;
    const Span out[2] = {{"y", a->y, span2(T, N, a->ld_y, size)}, {"workspace", a->workspace, need}};
    const Span in[6] = {{"scale", a->scale, n * 4},
                        {"adapter_ids", a->adapter_ids, (uint64_t)S * 4},
                        {"seq_offsets", a->seq_offsets, (uint64_t)(S + 1) * 4},
                        {"x", a->x, span2(T, K, a->ld_x, 2)},
                        {"a", a->a, n * R * K * 2},
                        {"b", a->b, n * N * R * 2}};
    const Span res{"residual", a->residual, a->residual ? span2(T, N, a->ld_residual, size) : 0};
    if ((rc = check_words(op, in, 3)) || (rc = check_outputs(op, out, 2)) || (rc = check_io(op, out[1], res))) return rc;
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 6; ++j)
            if ((rc = check_io(op, out[i], in[j]))) return rc;
    return check_residual(op, out[0], res, a->ld_y, a->ld_residual, N, size);
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
