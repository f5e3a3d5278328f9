// FP8 matrix product with bias, activation and residual in its epilogue (gfx950):
//   y = act(dequant(x) @ dequant(w) + bias) + residual.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 covers one 128-deep K block; the UE8M0 scales of the row and of
// the weights are its own scale operands, so the float32 accumulator sums scaled products and the
// epilogue starts from the finished sum.  Lane l of an operand holds row (A) or column (B) l % 16;
// of K it holds 32 (l / 16) .. +31 where one scale covers the block, and chunks of 16 at
// 16 (l / 16) and 64 + 16 (l / 16) where the lane's scale covers the 32 elements of group l / 16.
#include "layer_common.h"

#include <algorithm>

namespace moe {

typedef int v4i_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float act_fn(float v, int act) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.f ? 0.f : v;
        case MOE_ACT_SILU: return v / (1.0f + expf(-v));
        case MOE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
        case MOE_ACT_GELU_TANH: {   // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
            const float u = 0.79788456080286536f * fmaf(0.044715f * v * v, v, v);
            return v / (1.0f + expf(-2.0f * u));
        }
        default: return v;
    }
}

// One output element: act(acc + bias) + residual, stored in y's type.
__device__ __forceinline__ void put(const LinArgs& a, int row, int col, float v, float bias) {
    v = act_fn(v + bias, a.act);
    if (a.out_bf16) {
        if (a.res) v += bf16_to_f32(reinterpret_cast<const uint16_t*>(a.res)[(int64_t)row * a.ldr + col]);
        reinterpret_cast<uint16_t*>(a.y)[(int64_t)row * a.ldy + col] = (uint16_t)pack_bf16(v, v);
    } else {
        if (a.res) v += reinterpret_cast<const float*>(a.res)[(int64_t)row * a.ldr + col];
        reinterpret_cast<float*>(a.y)[(int64_t)row * a.ldy + col] = v;
    }
}

// Operands straight from memory into registers, no LDS in the K loop: workgroup (column tile of
// 16 NF, row tile of 16 MF), whose WK waves take the K blocks in turn and add their sums through
// LDS in wave order.  PF K blocks are in flight per wave; blocks past the end read as zeros
// (outside the descriptors' range).
template <bool MX, int MF, int NF, int WK, int PF>
__global__ __launch_bounds__(64 * WK) void k_linear_stream(LinArgs a) {
    __shared__ __align__(16) v4f s_acc[WK][MF * NF][64];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, G = lane >> 4, KB = a.K / kGroup;
    const int n0 = blockIdx.x * NF, m0 = blockIdx.y * MF * 16, n16s = a.N / 16;
    const rsrc_t ra = make_rsrc(a.xq, (uint32_t)a.T * (uint32_t)a.K);
    const rsrc_t rw = make_rsrc(a.w, (uint32_t)a.K * (uint32_t)a.N);
    const int gpb = MX ? 4 : 1, nbs = (a.N + kGroup - 1) / kGroup;   // A scales per K block
    const rsrc_t rxs = make_rsrc(a.xs, (uint32_t)a.T * (uint32_t)(KB * gpb));
    const rsrc_t rws = make_rsrc(a.ws, MX ? (uint32_t)KB * (uint32_t)n16s * 64u : (uint32_t)KB * (uint32_t)nbs);
    constexpr uint32_t kOut = 0x80000000u;   // past every descriptor's end
    uint32_t aoff[MF], xoff[MF], boff[NF], soff[NF];
#pragma unroll
    for (int i = 0; i < MF; ++i) {
        const uint32_t row = (uint32_t)min(m0 + i * 16 + r16, a.T - 1);
        aoff[i] = row * (uint32_t)a.K + (MX ? 16 * G : 32 * G);
        xoff[i] = row * (uint32_t)(KB * gpb) + (MX ? G : 0);
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const uint32_t n16 = (uint32_t)min(n0 + j, n16s - 1);
        boff[j] = n16 * (uint32_t)KB * kFragBytes + 16 * lane;
        soff[j] = MX ? n16 * (uint32_t)KB * 64 + lane : n16 / 8;
    }
    v8i A[PF][MF], B[PF][NF];
    int sa[PF][MF], sb[PF][NF];
    auto load = [&](int p, int kb) __attribute__((always_inline)) {
        const bool in = kb < KB;
        const uint32_t k = (uint32_t)kb;
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const uint32_t o = in ? boff[j] + k * kFragBytes : kOut;
            const v4i_t lo = __builtin_amdgcn_raw_buffer_load_b128(rw, o, 0, MOE_WLOAD_AUX);
            const v4i_t hi = __builtin_amdgcn_raw_buffer_load_b128(rw, o + 1024, 0, MOE_WLOAD_AUX);
            B[p][j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            sb[p][j] = __builtin_amdgcn_raw_buffer_load_b8(rws, in ? soff[j] + (MX ? k * 64 : k * nbs) : kOut, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const uint32_t o = in ? aoff[i] + k * kGroup : kOut;
            const v4i_t lo = __builtin_amdgcn_raw_buffer_load_b128(ra, o, 0, 0);
            const v4i_t hi = __builtin_amdgcn_raw_buffer_load_b128(ra, o + (MX ? 64 : 16), 0, 0);
            A[p][i] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            sa[p][i] = __builtin_amdgcn_raw_buffer_load_b8(rxs, in ? xoff[i] + k * gpb : kOut, 0, 0);
        }
    };
    v4f acc[MF][NF];
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < PF; ++p) load(p, wv + p * WK);
    for (int kb = wv; kb < KB; kb += WK * PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j) acc[i][j] = mfma_fp8(A[p][i], B[p][j], acc[i][j], sa[p][i], sb[p][j]);
            load(p, kb + (p + PF) * WK);
        }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) s_acc[wv][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    for (int q = wv; q < MF * NF; q += WK) {
        v4f v = s_acc[0][q][lane];
#pragma unroll
        for (int w = 1; w < WK; ++w) v += s_acc[w][q][lane];
        const int i = q / NF, j = q - i * NF, col = (n0 + j) * 16 + r16, row = m0 + i * 16 + 4 * G;
        if (n0 + j < n16s) {
            const float b = a.bias ? a.bias[col] : 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (row + r < a.T) put(a, row + r, col, v[r], b);
        }
    }
}

template <int MF, int NF, int WK, int PF>
static void run_stream(const LinArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(a.N, 16 * NF), (unsigned)ceil_div(a.T, 16 * MF));
    if (a.mx) hipLaunchKernelGGL((k_linear_stream<true, MF, NF, WK, PF>), grid, dim3(64 * WK), 0, st, a);
    else hipLaunchKernelGGL((k_linear_stream<false, MF, NF, WK, PF>), grid, dim3(64 * WK), 0, st, a);
}

hipError_t launch_linear(const LinArgs& a, hipStream_t st) {
    if (a.T <= 16) run_stream<1, 1, 8, 8>(a, st);
    else if (a.T <= 32) run_stream<2, 1, 8, 4>(a, st);
    else run_stream<4, 4, 4, 2>(a, st);
    return hipGetLastError();
}

}  // namespace moe
