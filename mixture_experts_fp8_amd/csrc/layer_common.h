// Device helpers and launchers of the operators around the expert step (k_norm.hip, k_linear.hip,
// k_gated.hip, k_gated_bwd.hip, k_lora.hip, k_router_grad.hip).
#pragma once
#include "moe_common.h"
#include "moe_layer_plan.h"

#include <atomic>

namespace moe {

typedef float v2f_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two float32 values as packed bf16, a in the low half: round to nearest even, NaN stays NaN,
// past the largest finite value infinity (one conversion instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f_t{a, b}, bf16x2_t));
}

// Eight bf16 values <-> eight floats.
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Sums over aligned groups of 16 lanes, in every lane of the group.
__device__ __forceinline__ float sum16(float v) {
    v += dpp_f32<0xB1>(v);
    v += dpp_f32<0x4E>(v);
    v += dpp_f32<0x124>(v);
    v += dpp_f32<0x128>(v);
    return v;
}

// HIP takes fewer than 2^32 threads in a launch: operators with a fixed number of threads per row launch
// this many rows at a time.
constexpr int64_t launch_rows(int threads_per_row) { return ((int64_t)1 << 31) / threads_per_row; }

// More than 64 KB of LDS has to be asked for, once per kernel and device.  MOST: the largest request, less than
// all of it by what the kernel holds in static arrays.
constexpr int kLdsBytes = 160 * 1024;
template <auto Kern, size_t MOST = kLdsBytes>
static hipError_t ask_for_lds(size_t lds) {
    if (lds <= 64 * 1024) return hipSuccess;
    static std::atomic<uint64_t> asked{0};   // a bit per device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev > 63 || !(asked.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)MOST);
        if (e != hipSuccess) return e;
        asked.fetch_or(bit, std::memory_order_relaxed);
    }
    return hipSuccess;
}

struct NormArgs {
    int T, H;
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* res;
    int64_t ldr;
    const float* w;
    float eps;
    uint16_t* h;
    uint16_t* y;
    uint8_t* yq;
    uint8_t* ys;
    int group;       // columns per scale: 0 (no codes), 32 or 128
    double inv_h;    // 1 / H
    const float* b = nullptr;   // layer norm: bias or NULL
};
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t st);
hipError_t launch_add_layernorm(const NormArgs& a, hipStream_t st);

struct NormBwdArgs {
    int T, H;
    const uint16_t* dy;
    const uint16_t* h;
    const float* w;
    float eps;
    const uint16_t* dh;   // or NULL
    uint16_t* dx;
    float* dw;            // or NULL
    float* part;          // workspace: [norm_bwd_parts(T, H)][H], used with dw
    double inv_h;         // 1 / H
    float* db = nullptr;      // layer norm: the bias's gradient or NULL, and its parts as those of dw
    float* part_b = nullptr;
};
hipError_t launch_add_rmsnorm_backward(const NormBwdArgs& a, hipStream_t st);
hipError_t launch_add_layernorm_backward(const NormBwdArgs& a, hipStream_t st);

struct LinArgs {
    int T, K, N;
    const uint8_t* xq;
    const uint8_t* xs;
    const uint8_t* w;
    const uint8_t* ws;
    const float* bias;    // or NULL
    const void* res;      // or NULL; of y's type
    int64_t ldr;
    void* y;
    int64_t ldy;
    int act, out_bf16, mx;
    int nt = 0;           // outputs past the caches (set by the launchers)
    uint16_t* gu = nullptr;   // gated block: both sums, [T, N] bf16, or NULL
};
hipError_t launch_linear(const LinArgs& a, hipStream_t st);
// y = act(gate) * up, bf16 [T, N / 2] without strides; no residual
hipError_t launch_gated_linear(const LinArgs& a, hipStream_t st);

struct GatedBwdArgs {
    int T, K, I, act, mx, dw_bf16;
    const uint16_t* dh;
    const uint16_t* gu;
    const uint8_t* xq;    // with dw
    const uint8_t* xs;
    const uint8_t* w;     // with dx
    const uint8_t* wsc;
    uint16_t* dgu;        // may be gu
    uint16_t* dx;         // or NULL
    void* dw;             // or NULL
    float* dbias;         // or NULL
    uint8_t* ws;          // laid out by gated_bwd_plan
};
hipError_t launch_gated_backward(const GatedBwdArgs& a, hipStream_t st);

// out[c] = sum of the np rows of part [np][n], in a fixed order
hipError_t launch_column_sums(const float* part, int np, int n, float* out, hipStream_t st);

struct LoraArgs {
    int T, K, R, n, S;    // n adapters, S sequences
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* a;    // [n][R][K]
    const uint16_t* b;    // [n][N][R]
    const float* scale;   // [n] or NULL: 1
    const int32_t* ids;   // [S]
    const int32_t* off;   // [S + 1] or NULL: a sequence per row
    void* v;              // workspace: x A^T as operands (v_operand)
    LinArgs out;          // N, residual, y
    int steps = 0, split = 0, col_blocks = 0, slot0 = 0;   // set by launch_lora
};
hipError_t launch_lora(const LoraArgs& a, hipStream_t st);

struct BalanceArgs {
    int T, E, k, S, scoring;
    const float* logits;
    const int32_t* ids;
    const int32_t* off;   // [S + 1] or NULL: one sequence of all T rows
    float ca, cz;
    float* losses;
    int32_t* counts;
    float* mean_probs;    // or NULL
    uint8_t* ws;
};
hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t st);

struct RouteBwdArgs {
    int T, E, k, S, scoring, renorm;
    float rsf;
    const float* logits;
    const int32_t* ids;
    const float* dw;      // or NULL
    const int32_t* counts;  // or NULL
    const int32_t* off;
    float ca, cz;
    float* dlogits;
    float load;           // E / k
};
hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t st);

struct CombineBwdArgs {
    int T, k, H, bf16;
    int rows;             // T * k of the whole call (below 2^29)
    const uint16_t* dy;
    const void* eo;       // or NULL with dwt NULL
    const int32_t* pos;
    const float* wt;      // or NULL with deo NULL
    float* dwt;
    void* deo;
    int clear;            // rows of deo that pos does not name become 0
};
hipError_t launch_combine_backward(const CombineBwdArgs& a, hipStream_t st);

}  // namespace moe
