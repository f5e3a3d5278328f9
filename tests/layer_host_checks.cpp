// CPU driver for the host side of the operators around the expert step (moe_layer_host.cpp), built
// without HIP under the address and undefined-behaviour sanitizers by tests/test_layer_sanitized.py.
#include <cstdio>
#include <cstdlib>
#include <cstring>
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

// The parts of the balance loss: every (workgroup, sequence) pair that has rows gets a slot of its
// own inside the workspace, for any boundaries.
static void balance_slots() {
    std::srand(7);
    for (int rep = 0; rep < 400; ++rep) {
        const int T = 1 + std::rand() % (rep % 2 ? 3000 : 200), S = 1 + std::rand() % 90, E = 1 + std::rand() % 1024;
        std::vector<int> off(S + 1);
        for (int i = 0; i <= S; ++i) off[i] = std::rand() % (T + 1);
        for (int i = 1; i <= S; ++i)
            for (int j = i; j && off[j] < off[j - 1]; --j) std::swap(off[j], off[j - 1]);
        const BalancePlan p = balance_plan(T, E, S);
        CHECK((int64_t)p.nblocks * p.chunk >= T && (int64_t)(p.nblocks - 1) * p.chunk < T);
        const size_t o[] = {p.probs, p.hits, p.z, p.seq, p.done, p.end};
        for (int i = 0; i + 1 < 6; ++i) CHECK(o[i] <= o[i + 1] && o[i] % 256 == 0);
        CHECK(p.stride >= E && p.stride % 4 == 0 && p.done - p.seq >= (size_t)S * 8 && p.end - p.done >= 4);
        CHECK(!p.one || p.nblocks == 1);
        if (p.one) continue;   // no parts
        CHECK(p.hits - p.probs >= (size_t)p.nslots * p.stride * 4 && p.z - p.hits >= (size_t)p.nslots * p.stride * 4);
        CHECK(p.seq - p.z >= (size_t)p.nslots * 4);
        std::set<int> seen;
        for (int b = 0; b < p.nblocks; ++b)
            for (int s = 0; s < S; ++s)
                if (std::max(off[s], b * p.chunk) < std::min(off[s + 1], std::min(T, (b + 1) * p.chunk))) {
                    CHECK(b + s < p.nslots);
                    CHECK(seen.insert(b + s).second);
                }
    }
}

int main() {
    balance_slots();
    for (int T : {1, 511, 512, 513, 1 << 20})
        for (int H : {8, 4096, 32768}) {
            const int n = norm_bwd_parts(T, H);
            CHECK(n >= 1 && n <= T && n <= 512 && norm_bwd_ws_bytes(T, H) == (size_t)n * H * 4);
        }
    {
        moe_add_rmsnorm_args a;
        std::memset(&a, 0, sizeof a);
        CHECK(host::check_add_rmsnorm(&a) == MOE_ERR_INVALID);
        a.T = 0x7fffffff, a.H = 32768, a.ld_x = 32768;   // the largest call: sizes past 32 bits
        a.x = at<uint16_t>(0x10), a.weight = at<float>(0), a.y = at<uint16_t>(0x8000);
        CHECK(host::check_add_rmsnorm(&a) == MOE_OK);
        a.y = at<uint16_t>(0x200);
        CHECK(host::check_add_rmsnorm(&a) == MOE_ERR_INVALID);
    }
    {
        moe_linear_args a;
        std::memset(&a, 0, sizeof a);
        CHECK(host::check_linear(&a) == MOE_ERR_INVALID);
        a.T = 65535, a.K = 32768, a.N = 65520;
        a.xq = at<uint8_t>(0), a.xs = at<uint8_t>(1), a.w = at<uint8_t>(2), a.w_scale = at<uint8_t>(3), a.y = at<void>(4);
        a.ld_y = 65520;
        a.out_dtype = MOE_DTYPE_F32;
        a.workspace = at<void>(64), a.workspace_bytes = (size_t)1 << 40;
        CHECK(host::check_linear(&a) == MOE_OK);
        // columns of one matrix: side by side, then one element group too close on either side
        a.T = 100, a.K = 128, a.N = 64, a.ld_y = a.ld_residual = 160, a.out_dtype = MOE_DTYPE_BF16;
        char* m = static_cast<char*>(a.y);
        a.residual = m + 64 * 2;
        CHECK(host::check_linear(&a) == MOE_OK);
        a.residual = m + 96 * 2;
        CHECK(host::check_linear(&a) == MOE_OK);
        a.residual = m - 64 * 2;
        CHECK(host::check_linear(&a) == MOE_OK);
        for (int c : {56, 104, -56, 8, 160}) {
            a.residual = m + c * 2;
            CHECK(host::check_linear(&a) == MOE_ERR_INVALID);
        }
        a.residual = m;
        CHECK(host::check_linear(&a) == MOE_OK);
        a.residual = nullptr, a.K = 32768, a.N = 65520, a.ld_y = 65520, a.out_dtype = MOE_DTYPE_F32;
        a.T = 65536;
        CHECK(host::check_linear(&a) == MOE_ERR_UNSUPPORTED);
        a.T = a.N = a.ld_y = 1 << 20, a.K = 128;
        CHECK(host::check_linear(&a) == MOE_ERR_UNSUPPORTED);
    }
    {
        moe_route_params p{};
        p.num_experts = 1024, p.top_k = 8, p.routed_scaling_factor = 1.f;
        moe_route_backward_args a;
        std::memset(&a, 0, sizeof a);
        CHECK(host::check_route_backward(&a) == MOE_ERR_INVALID);
        a.route = &p, a.T = 1 << 25, a.num_seqs = 1;
        a.router_logits = at<float>(0), a.dlogits = at<float>(0);
        CHECK(host::check_route_backward(&a) == MOE_OK);
        moe_balance_loss_args b;
        std::memset(&b, 0, sizeof b);
        b.route = &p, b.T = 1 << 25, b.num_seqs = 1 << 20;
        b.router_logits = at<float>(0), b.topk_ids = at<int32_t>(64), b.seq_offsets = at<int32_t>(65);
        b.losses = at<float>(66), b.counts = at<int32_t>(67), b.workspace = at<void>(70), b.workspace_bytes = (size_t)1 << 40;
        CHECK(host::check_balance_loss(&b) == MOE_ERR_UNSUPPORTED);
        b.num_seqs = 1 << 19;
        CHECK(host::check_balance_loss(&b) == MOE_OK);
    }
    {
        moe_combine_backward_args a;
        std::memset(&a, 0, sizeof a);
        CHECK(host::check_combine_backward(&a) == MOE_ERR_INVALID);
        moe_add_rmsnorm_backward_args b;
        std::memset(&b, 0, sizeof b);
        CHECK(host::check_add_rmsnorm_backward(&b) == MOE_ERR_INVALID);
    }
    std::printf("layer host checks ok\n");
    return 0;
}
