// CPU driver for the host side of the operators of dense layers (moe_layer_host.cpp), built without HIP under the
// address and undefined-behaviour sanitizers by tests/test_dense_sanitized.py.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "../mixture_experts_fp8_amd/csrc/moe_layer_plan.h"

using namespace moe;

#define CHECK(cond)                                                                                   \
    do {                                                                                              \
        if (!(cond)) {                                                                                \
            std::fprintf(stderr, "%s:%d: CHECK(%s) failed; last error: %s\n", __FILE__, __LINE__, #cond, \
                         host::last_error());                                                         \
            std::exit(1);                                                                             \
        }                                                                                             \
    } while (0)

// buffers 8 GiB apart, never dereferenced
template <typename T>
static T* at(int i) { return reinterpret_cast<T*>((uintptr_t)0x10000000u + ((uintptr_t)i << 33)); }

// Parts of a sum: none is empty, together they are all of it; the workspace holds them, in places of their own.
static void products() {
    std::srand(11);
    std::set<int> tiles;
    int split[2] = {};
    for (int rep = 0; rep < 4000; ++rep) {
        const int T = 1 + std::rand() % (rep % 3 ? 3000 : 40000), K = 128 * (1 + std::rand() % 60), I = 32 * (1 + std::rand() % 120);
        const bool dx = rep % 4 != 1, dw = rep % 4 != 2, db = rep % 5 != 0;
        const GatedBwdPlan p = gated_bwd_plan(T, K, I, dx, dw, db);
        CHECK(p.product.tile >= 0 && p.product.tile < 5);
        tiles.insert(p.product.tile);
        const int blocks[2] = {I / 32, (T + 63) / 64};
        for (int i = 0; i < 2; ++i) {
            const int n = p.product.parts[i];
            CHECK((n > 0) == (i ? dw : dx) && n <= 16);
            if (n < 2) continue;
            ++split[i];
            const int per = (blocks[i] + n - 1) / n;
            CHECK(per * (n - 1) < blocks[i] && per * n >= blocks[i]);
        }
        const uint64_t N = 2 * (uint64_t)I, rows = 64 * (uint64_t)p.row_blocks;
        const uint64_t bytes[6] = {db ? p.parts * N * 4 : 0, dx ? K * N * 2 : 0, dw ? K * rows * 2 : 0, dw ? N * rows * 2 : 0,
                                   p.product.parts[0] > 1 ? (uint64_t)p.product.parts[0] * T * K * 4 : 0,
                                   p.product.parts[1] > 1 ? p.product.parts[1] * K * N * 4 : 0};
        const size_t o[7] = {p.part, p.weights, p.rows, p.dgu_packed, p.join[0], p.join[1], p.end};
        for (int i = 0; i < 6; ++i) CHECK(o[i] % 256 == 0 && o[i + 1] >= o[i] + bytes[i]);
        CHECK(rows >= (uint64_t)T && p.parts <= p.row_blocks);
    }
    CHECK(tiles.size() == 5 && split[0] && split[1]);
}

// Slots: every pair of a window and a sequence that has rows gets one of its own, in the workspace.
static void slots() {
    std::srand(12);
    for (int rep = 0; rep < 500; ++rep) {
        const int T = 1 + std::rand() % (rep % 2 ? 9000 : 300), S = 1 + std::rand() % 120, R = 8 * (1 + std::rand() % 32);
        std::vector<int> off(S + 1);
        for (int i = 0; i <= S; ++i) off[i] = std::rand() % (T + 1);
        for (int i = 1; i <= S; ++i)
            for (int j = i; j && off[j] < off[j - 1]; --j) std::swap(off[j], off[j - 1]);
        for (bool bf16 : {false, true}) {
            const LoraPlan p = lora_plan(T, R, S, bf16);
            CHECK((p.window == 16 || p.window == 32) && p.steps * 32 >= R && p.split == (bf16 ? 2 : 3));
            CHECK(p.end == (size_t)p.slots * (p.window / 16) * p.steps * p.split * 1024);
            std::set<int> seen;
            for (int s = 0; s < S; ++s)
                for (int b = off[s] / p.window; b * p.window < off[s + 1]; ++b)
                    if (off[s] < off[s + 1]) CHECK(b + s < p.slots && seen.insert(b + s).second);
        }
        CHECK(lora_plan(T, R, 0, true).slots == T);
    }
}

int main() {
    products();
    slots();
    for (int T : {1, 511, 4095, 4096, 1 << 20})
        for (int H : {8, 1024, 2048, 4096, 32768}) {
            const int n = layernorm_bwd_parts(T, H);
            CHECK(n >= 1 && n <= T && n <= 1024 && layernorm_bwd_ws_bytes(T, H) == 2 * (size_t)n * H * 4);
        }

    // accepted calls: in-place uses, columns of one matrix side by side, what is not asked for left out
    moe_add_layernorm_args n{};
    n.T = 4, n.H = 256, n.x = at<uint16_t>(0), n.ld_x = 256, n.residual = at<uint16_t>(1), n.ld_residual = 256;
    n.weight = at<float>(2), n.eps = 1e-5f, n.h = at<uint16_t>(1), n.y = at<uint16_t>(3);
    CHECK(host::check_add_layernorm(&n) == MOE_OK);
    n.bias = at<float>(4);
    CHECK(host::check_add_layernorm(&n) == MOE_OK);
    n.h = at<uint16_t>(0);
    CHECK(host::check_add_layernorm(&n) == MOE_OK);
    CHECK(host::check_add_layernorm(nullptr) == MOE_ERR_INVALID);

    moe_add_layernorm_backward_args b{};
    b.T = 4, b.H = 256, b.dy = at<uint16_t>(0), b.h = at<uint16_t>(1), b.weight = at<float>(2), b.eps = 1e-5f, b.dx = at<uint16_t>(0);
    CHECK(host::check_add_layernorm_backward(&b) == MOE_OK);
    b.dbias = at<float>(4);
    CHECK(host::check_add_layernorm_backward(&b) == MOE_ERR_WORKSPACE);
    b.workspace = at<void>(5), b.workspace_bytes = layernorm_bwd_ws_bytes(4, 256);
    CHECK(host::check_add_layernorm_backward(&b) == MOE_OK);

    moe_gated_linear_backward_args g{};
    g.T = 100, g.K = 256, g.I = 96, g.dh = at<uint16_t>(0), g.gu = at<uint16_t>(1), g.dgu = at<uint16_t>(1);
    CHECK(host::check_gated_linear_backward(&g) == MOE_OK);   // in place, no workspace
    g.dx = at<uint16_t>(2);
    CHECK(host::check_gated_linear_backward(&g) == MOE_ERR_INVALID);
    g.w = at<uint8_t>(3), g.w_scale = at<uint8_t>(4);
    CHECK(host::check_gated_linear_backward(&g) == MOE_ERR_WORKSPACE);
    g.workspace = at<void>(5), g.workspace_bytes = gated_bwd_plan(100, 256, 96, true, false, false).end;
    CHECK(host::check_gated_linear_backward(&g) == MOE_OK);
    g.T = 2147483647;
    CHECK(host::check_gated_linear_backward(&g) == MOE_ERR_UNSUPPORTED);
    g.T = 100, g.I = 2147483616;
    CHECK(host::check_gated_linear_backward(&g) == MOE_ERR_UNSUPPORTED);

    moe_gated_linear_args f{};
    f.T = 1, f.K = 128, f.I = 2147483616, f.xq = at<uint8_t>(0), f.xs = at<uint8_t>(1), f.w = at<uint8_t>(2), f.w_scale = at<uint8_t>(3), f.h = at<uint16_t>(4);
    CHECK(host::check_gated_linear(&f) == MOE_ERR_UNSUPPORTED);
    f.I = 32;
    CHECK(host::check_gated_linear(&f) == MOE_OK);

    moe_lora_args l{};
    l.T = 6, l.K = 72, l.N = 48, l.R = 24, l.num_adapters = 2147483647, l.num_seqs = 6, l.x = at<uint16_t>(0), l.ld_x = 80;
    l.a = at<uint16_t>(1), l.b = at<uint16_t>(40), l.adapter_ids = at<int32_t>(80), l.y = at<float>(81), l.ld_y = 96;
    l.workspace = at<void>(82), l.workspace_bytes = lora_plan(6, 24, 0, false).end;
    CHECK(host::check_lora(&l) == MOE_OK || host::check_lora(&l) == MOE_ERR_INVALID);   // (adapters past their buffers' distance)
    l.num_adapters = 3, l.b = at<uint16_t>(2);
    CHECK(host::check_lora(&l) == MOE_OK);
    l.residual = static_cast<float*>(l.y) + 48, l.ld_residual = 96;   // the other half of the same rows
    CHECK(host::check_lora(&l) == MOE_OK);
    l.residual = static_cast<float*>(l.y) + 40;
    CHECK(host::check_lora(&l) == MOE_ERR_INVALID);
    l.residual = l.y;
    CHECK(host::check_lora(&l) == MOE_OK);
    std::puts("dense host checks ok");
    return 0;
}
