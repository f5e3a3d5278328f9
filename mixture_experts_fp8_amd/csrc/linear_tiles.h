// Matrix products on packed column fragments, shared by the linear layer (k_linear.hip), the gated
// block (k_gated.hip) and its backward pass (k_gated_bwd.hip): y = epilogue(x @ w).
//
// Operand formats.  Two of them are FP8: v_mfma_scale_f32_16x16x128_f8f6f4 covers one 128-deep K block; the
// UE8M0 scales of the row and of the weights are its own scale operands, so the float32 accumulator sums
// scaled products and the epilogue starts from the finished sum.  Lane l of an operand holds row (A) or
// column (B) l % 16; of K it holds 32 (l / 16) .. +31 where one scale covers the block (kBlock), and chunks of
// 16 at 16 (l / 16) and 64 + 16 (l / 16) where the lane's scale covers the 32 elements of group l / 16 (kMicro).
//   kBf16: no scales; a block of 128 bytes is 64 deep and takes two v_mfma_f32_16x16x32_bf16.  Its bytes are
// laid out as kMicro's: the lane's two 16-byte chunks, l / 16 and l / 16 + 4, are the operands of the two.
// LinArgs.K then counts bytes of a row, two per element, and a column fragment is 16 columns x 64 K, 2 KB as
// with FP8: bytes 16 l .. +15 of its halves are lane l's two chunks.
//   GATED: the columns of w are those of two products, gate columns [0, N / 2) and up columns behind them; a
// wave's column fragments are half gate, half up of the same columns, and y = act(gate) * up is N / 2 wide.
#pragma once
#include "layer_common.h"

#include <algorithm>

namespace moe {

enum Format { kBlock, kMicro, kBf16 };

typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef unsigned v4u_t __attribute__((ext_vector_type(4)));

// exp(x) by the base-2 instruction: the product's rounding moves the result by |x| 2^-24 of it, which
// the activations below multiply by at most x exp(-|x|).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// The normal distribution function, which GELU multiplies v by.
__device__ __forceinline__ float normal_cdf(float v) {
    // exp(z^2) erfc(z) / 2 with z = |v| / sqrt 2 as a polynomial in t = 1 / (1 + 0.42 z): the minimax fit
    // in relative error over z <= 9.4, 1.4e-7.  (A fit in absolute error loses the negative tail: 1e-2 of
    // the value at v = -8.)  One term fewer: 1.0e-6.
    const float t = __builtin_amdgcn_rcpf(fmaf(0.296984851f, fabsf(v), 1.0f));
    float p = fmaf(0.0352053866f, t, -0.160467133f);
    p = fmaf(p, t, 0.220853359f);
    p = fmaf(p, t, -0.0656716153f);
    p = fmaf(p, t, 0.134549260f);
    p = fmaf(p, t, 0.0973208472f);
    p = fmaf(p, t, 0.119797952f);
    p = fmaf(p, t, 0.118411876f);
    const float c = p * t * __builtin_amdgcn_exp2f(v * v * -0.72134752f);     // erfc(z) / 2
    return v < 0.f ? c : 1.0f - c;
}

// The activations take one or two transcendental instructions: with library exp, erfc and division
// the epilogue of a 768-deep product cost as much as its K loop.
__device__ __forceinline__ float act_fn(float v, int act) {
    switch (act) {
        case MOE_ACT_RELU: return v < 0.f ? 0.f : v;
        case MOE_ACT_SILU: return v * __builtin_amdgcn_rcpf(1.0f + exp_fast(-v));
        case MOE_ACT_GELU: return v * normal_cdf(v);
        case MOE_ACT_GELU_TANH: {   // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
            const float u = 0.79788456f * fmaf(0.044715f * v * v, v, v);
            return v * __builtin_amdgcn_rcpf(1.0f + exp_fast(-2.0f * u));
        }
        default: return v;
    }
}

// Bias and residual of four consecutive columns of a row, and the finished columns from their sum:
// act(v + bias) + residual, stored in y's type.
struct Extra {
    v4f bias;
    v4u_t res;   // bf16: two words
};
__device__ __forceinline__ Extra load_extra(const LinArgs& a, int64_t row, int col) {
    Extra e;
    e.bias = v4f{0.f, 0.f, 0.f, 0.f};
    e.res = v4u_t{0, 0, 0, 0};
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e.bias[i] = a.bias[col + i];   // (4-byte aligned)
    }
    if (a.res) {
        if (a.out_bf16) {
            const uint2 r = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.res) + row * a.ldr + col);
            e.res[0] = r.x;
            e.res[1] = r.y;
        } else {
            e.res = *reinterpret_cast<const v4u_t*>(reinterpret_cast<const float*>(a.res) + row * a.ldr + col);
        }
    }
    return e;
}
__device__ __forceinline__ void put4(const LinArgs& a, int64_t row, int col, v4f v, const Extra& e) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = act_fn(v[i] + e.bias[i], a.act);
    if (a.out_bf16) {
        if (a.res) {
            v[0] += __uint_as_float(e.res[0] << 16);
            v[1] += __uint_as_float(e.res[0] & 0xFFFF0000u);
            v[2] += __uint_as_float(e.res[1] << 16);
            v[3] += __uint_as_float(e.res[1] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + col) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
        if (a.res) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(e.res[i]);
        }
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(a.y) + row * a.ldy + col) = v;
    }
}

// Four consecutive columns of a row of the gated block from the two sums.
__device__ __forceinline__ void put_gated4(const LinArgs& a, int64_t row, int col, v4f g, v4f u) {
    const int I = a.N / 2;
    if (a.gu) {
        uint16_t* d = a.gu + row * a.N + col;
        *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]));
        *reinterpret_cast<uint2*>(d + I) = make_uint2(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = act_fn(g[i], a.act) * u[i];
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + row * I + col) =
        make_uint2(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]));
}

// Operands straight from memory into registers, no LDS in the K loop: workgroup (column tile of
// 16 NF, row tile of 16), whose WK waves take the K blocks in turn and add their sums through
// LDS in wave order.  PF K blocks are in flight per wave.  Bound by the weight stream: 1 x 7168 x 7168 takes
// 10.0 us, 5.1 TB/s; a small product (32 x 2816 x 2816 with gelu, 6.0 us) by one wave's chain of loads.
template <Format F, bool GATED, int NF, int WK, int PF>
__global__ __launch_bounds__(64 * WK) void k_linear_stream(LinArgs a) {
    static_assert(F != kBf16, "FP8 only");
    constexpr bool MX = F == kMicro;
    constexpr int NY = GATED ? NF / 2 : NF;   // column fragments of y
    __shared__ __align__(16) v4f s_acc[WK][NF][64];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, G = lane >> 4, KB = a.K / kGroup;
    const int n0 = blockIdx.x * NY, m0 = blockIdx.y * 16, n16s = a.N / 16, n16y = GATED ? n16s / 2 : n16s;
    constexpr int gpb = MX ? 4 : 1;   // row scales per K block
    const int nbs = (a.N + kGroup - 1) / kGroup;
    const rsrc_t rx = make_rsrc(a.xq, (uint32_t)a.T * (uint32_t)a.K);
    const rsrc_t rw = make_rsrc(a.w, (uint32_t)a.K * (uint32_t)a.N);
    const rsrc_t rxs = make_rsrc(a.xs, (uint32_t)a.T * (uint32_t)(KB * gpb));
    const rsrc_t rws = make_rsrc(a.ws, MX ? (uint32_t)KB * (uint32_t)n16s * 64u : (uint32_t)KB * (uint32_t)nbs);
    const uint32_t xrow = (uint32_t)min(m0 + r16, a.T - 1);   // (rows past the end: not stored)
    const uint32_t xoff = xrow * (uint32_t)a.K + (MX ? 16 * G : 32 * G);
    const uint32_t xsoff = xrow * (uint32_t)(KB * gpb) + (MX ? G : 0);
    uint32_t wfrag[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j)
        wfrag[j] = __builtin_amdgcn_readfirstlane((uint32_t)(min(n0 + j % NY, n16y - 1) + j / NY * n16y));
    const uint32_t l16 = 16 * lane;
    v8i X[PF], W[PF][NF];
    uint8_t sx[PF], sw[PF][NF];   // widened at their use: done at the load, that waits for it
    auto load = [&](int p, int blk) __attribute__((always_inline)) {
        const uint32_t kb = (uint32_t)min(blk, KB - 1);   // (past the end the last block again, unused)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            const uint32_t f = (wfrag[j] * (uint32_t)KB + kb);
            const v4i_t lo = __builtin_amdgcn_raw_buffer_load_b128(rw, l16, f * kFragBytes, MOE_WLOAD_AUX);
            const v4i_t hi = __builtin_amdgcn_raw_buffer_load_b128(rw, l16 + 1024, f * kFragBytes, MOE_WLOAD_AUX);
            W[p][j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            sw[p][j] = MX ? __builtin_amdgcn_raw_buffer_load_b8(rws, lane, f * 64, 0)
                          : __builtin_amdgcn_raw_buffer_load_b8(rws, 0, kb * nbs + wfrag[j] / 8, 0);
        }
        const v4i_t lo = __builtin_amdgcn_raw_buffer_load_b128(rx, xoff, kb * kGroup, 0);
        const v4i_t hi = __builtin_amdgcn_raw_buffer_load_b128(rx, xoff + (MX ? 64 : 16), kb * kGroup, 0);
        X[p] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        sx[p] = __builtin_amdgcn_raw_buffer_load_b8(rxs, xsoff, kb * gpb, 0);
    };
    v4f acc[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto products = [&](int p) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[j] = mfma_fp8(W[p][j], X[p], acc[j], sw[p][j], sx[p]);
    };
    const int nk = KB > wv ? (KB - wv + WK - 1) / WK : 0;   // blocks wv, wv + WK, ... of this wave
#pragma unroll
    for (int p = 0; p < PF; ++p) load(p, wv + p * WK);
    // wave j finishes fragment j; its bias and residual are fetched over the K loop
    static_assert(NY <= WK, "a wave per fragment");
    const int row = m0 + r16, col = (n0 + wv) * 16 + 4 * G;
    const bool live = wv < NY && n0 + wv < n16y && row < a.T;
    Extra ex, eu;
    if (live) ex = load_extra(a, row, col);
    if (GATED && live) eu = load_extra(a, row, a.N / 2 + col);   // (its bias; there is no residual)
    int i0 = 0;
    for (; i0 + PF <= nk; i0 += PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            products(p);
            // (kept in this order: hoisted over the products, the loads take registers of their own, and
            // the copies back wait for all of them)
            __builtin_amdgcn_sched_barrier(0);
            load(p, wv + (i0 + p + PF) * WK);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int p = 0; p < PF; ++p)
        if (i0 + p < nk) products(p);
#pragma unroll
    for (int j = 0; j < NF; ++j) s_acc[wv][j][lane] = acc[j];
    __syncthreads();
    if (!live) return;
    v4f v = s_acc[0][wv][lane];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += s_acc[w][wv][lane];
    if constexpr (GATED) {
        v4f u = s_acc[0][wv + NY][lane];
#pragma unroll
        for (int w = 1; w < WK; ++w) u += s_acc[w][wv + NY][lane];
        put_gated4(a, row, col, v + ex.bias, u + eu.bias);
    } else {
        put4(a, row, col, v, ex);
    }
}

// ----------------------------------------------------------------------------------------
// Tiled kernel for many rows.  Workgroup of WM x WN waves, each 16 MI rows x 16 NJ columns.  The
// instruction's first operand is the weights and its second the activations, so a lane of the
// accumulator holds row l % 16 of a fragment and four consecutive columns, 4 (l / 16) ...: the
// epilogue then works on whole vectors of a row, without LDS.
//   * Activations: every row fragment is read by WN waves, so they go through LDS, three stages of
//     one K block, filled by LDS-DMA: block kb + 2's copies are issued in block kb and waited for at its
//     end, with everything else (two workgroups share a CU, and one computes while the other waits).  A
//     row's 16-byte chunks stand at slot ^ (row % 8), where chunk c has slot c (32-element scales) or
//     c / 2 + 4 (c % 2): a lane needs slots l / 16 and l / 16 + 4 in both cases, without bank conflicts.
//   * Weights: a fragment is read by WM waves only, and its packed order is the operand's, so it goes
//     straight to registers one block ahead: staging it too would make the LDS the bound (two waves
//     per SIMD read 24 KB of operands per 32 instructions otherwise).
//   * The first row fragments of block kb + 1 are read during block kb, so that matrix instructions
//     follow the barrier at once.
// 16384 x 4096 x 4096 in bf16: 223-237 us with the operands (the clock moves), 2.3-2.5 PFLOP/s, as the
// library's FP8 product of this size; the matrix cores bound it.  With a residual 262-267 us: its 134 MB come when the K loop is over (128 x 256 tiles
// leave no registers for it before), and two workgroups per CU hide that only in part.
__device__ __forceinline__ v4i_t make_srd(const void* base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    v4i_t r;
    r[0] = (int)__builtin_amdgcn_readfirstlane((uint32_t)b);
    r[1] = (int)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xFFFFu);   // stride 0
    r[2] = (int)__builtin_amdgcn_readfirstlane(bytes);
    r[3] = 0x00020000;
    return r;
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p);
}
// Bytes from the buffer at voff + soff into LDS at base + (16 or 4) * lane.  The compiler does not
// see these loads: their end is awaited by wait_all and a barrier before the LDS is read.
__device__ __forceinline__ void dma16(const v4i_t& srd, uint32_t base, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(base), "v"(voff), "s"(srd), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void dma4(const v4i_t& srd, uint32_t base, uint32_t voff, uint32_t soff) {
    asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :
                 : "s"(base), "v"(voff), "s"(srd), "s"(soff)
                 : "memory", "m0");
}
__device__ __forceinline__ void wait_all() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

// The product with the weights' scale in byte 0 of sw and the rows' in byte bx of sx (bx is a constant
// after unrolling).
__device__ __forceinline__ v4f mfma_wx(v8i w, v8i x, v4f acc, int sw, int sx, int bx) {
    switch (bx) {
        case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw, 0, sx);
        case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw, 1, sx);
        case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw, 2, sx);
        default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw, 3, sx);
    }
}

// One K block's products of two operands; kBlock: the rows' scale in byte bx of sx.
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
template <Format F>
__device__ __forceinline__ v4f products_of(v8i w, v8i x, v4f acc, int sw, int sx, int bx) {
    if constexpr (F == kBf16) {
        const v4i_t w0 = {w[0], w[1], w[2], w[3]}, w1 = {w[4], w[5], w[6], w[7]};
        const v4i_t x0 = {x[0], x[1], x[2], x[3]}, x1 = {x[4], x[5], x[6], x[7]};
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w0), __builtin_bit_cast(bf16x8_t, x0), acc, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w1), __builtin_bit_cast(bf16x8_t, x1), acc, 0, 0, 0);
    } else {
        return mfma_wx(w, x, acc, sw, sx, bx);
    }
}

// Column fragment of w that stands in place q of the cols / 16 of column tile tn (behind the last one: the
// last again, for columns that are not stored).  GATED: of a wave's four, two are gate and two up.
template <bool GATED>
__device__ __forceinline__ int column_fragment(const LinArgs& a, int tn, int cols, int q) {
    const int n16s = a.N / 16;
    if constexpr (GATED) {
        const int n16y = n16s / 2;
        return min(tn * (cols / 32) + (q >> 2) * 2 + (q & 1), n16y - 1) + ((q >> 1) & 1) * n16y;
    } else {
        return min(tn * (cols / 16) + q, n16s - 1);
    }
}
// 128-column scales of w that a tile's waves use in a K block: one per 128 columns, or a gate and an up
// one per wave (N / 2 is a multiple of 32, so 32 columns lie in one block).
template <bool GATED>
constexpr int tile_scales(int cols) { return GATED ? cols / 32 : (cols + 127) / 128; }

__device__ __forceinline__ void store16(v4u_t* d, v4u_t v, int nt) {
    if (nt) __builtin_nontemporal_store(v, d);
    else *d = v;
}

// Exchange between neighbouring groups of 16 lanes, its own inverse: of two column fragments' values, a and b,
// lane group G then holds those of fragment G % 2, a the ones of group G & 2 and b the ones of the next.
__device__ __forceinline__ void swap_groups(uint32_t& a, uint32_t& b) {
    auto v = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = v[0];
    b = v[1];
}

// Epilogue of a wave's 64 columns col0 .. (of which those below N exist; N is a multiple of 16).
// acc[mi][j]: columns col0 + 16 j + 4 G .. +3 of row row0 + 16 mi.
//   bf16: after an exchange between neighbouring lane groups, lane group G holds the 8 columns from
//   16 (G % 2) + 8 (G / 2) of 32: residual and output move as 16-byte vectors, and one instruction covers
//   64 bytes of a row.
//   float32: a lane's four columns are 16 bytes already.
// The residual of all rows is requested before the first one is used.
template <int MI>
__device__ __forceinline__ void tile_residual(const LinArgs& a, uint4 (&q)[MI][2], int row0, int col0) {
    const int G = (threadIdx.x & 63) >> 4, col = col0 + 16 * (G & 1) + 8 * (G >> 1);
    if (a.out_bf16 && a.res) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
            const uint16_t* s = reinterpret_cast<const uint16_t*>(a.res) + (row0 + 16 * mi) * a.ldr + col;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                q[mi][h] = make_uint4(0, 0, 0, 0);
                if (col + 32 * h < a.N && row0 + 16 * mi < a.T) q[mi][h] = *reinterpret_cast<const uint4*>(s + 32 * h);
            }
        }
    }
}
template <int MI, int ACT>
__device__ __forceinline__ void tile_epilogue(const LinArgs& a, v4f (&acc)[MI][4], const v4f (&b)[4], uint4 (&q)[MI][2],
                                              int row0, int col0) {
    const int G = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
        const int64_t row = row0 + 16 * mi;
        const bool live = row < a.T;
        v4f (&v)[4] = acc[mi];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j][i] = act_fn(v[j][i] + b[j][i], ACT);
        if (a.out_bf16) {
            uint32_t lo[4], hi[4];
            if (a.res) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    lo[2 * h] = q[mi][h].x, hi[2 * h] = q[mi][h].y, lo[2 * h + 1] = q[mi][h].z, hi[2 * h + 1] = q[mi][h].w;
                    swap_groups(lo[2 * h], lo[2 * h + 1]);
                    swap_groups(hi[2 * h], hi[2 * h + 1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j][0] += __uint_as_float(lo[j] << 16);
                    v[j][1] += __uint_as_float(lo[j] & 0xFFFF0000u);
                    v[j][2] += __uint_as_float(hi[j] << 16);
                    v[j][3] += __uint_as_float(hi[j] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lo[j] = pack_bf16(v[j][0], v[j][1]);
                hi[j] = pack_bf16(v[j][2], v[j][3]);
            }
            const int col = col0 + 16 * (G & 1) + 8 * (G >> 1);
            uint16_t* d = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + col;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                swap_groups(lo[2 * h], lo[2 * h + 1]);
                swap_groups(hi[2 * h], hi[2 * h + 1]);
                if (live && col + 32 * h < a.N)
                    store16(reinterpret_cast<v4u_t*>(d + 32 * h), v4u_t{lo[2 * h], hi[2 * h], lo[2 * h + 1], hi[2 * h + 1]}, a.nt);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = col0 + 16 * j + 4 * G;
                if (live && col < a.N) {
                    if (a.res) v[j] += *reinterpret_cast<const v4f*>(reinterpret_cast<const float*>(a.res) + row * a.ldr + col);
                    store16(reinterpret_cast<v4u_t*>(reinterpret_cast<float*>(a.y) + row * a.ldy + col),
                            __builtin_bit_cast(v4u_t, v[j]), a.nt);
                }
            }
        }
    }
}

template <int MI>
__device__ __forceinline__ void tile_finish(const LinArgs& a, v4f (&acc)[MI][4], const v4f (&b)[4], uint4 (&q)[MI][2],
                                            int row0, int col0) {
    switch (a.act) {
        case MOE_ACT_RELU: return tile_epilogue<MI, MOE_ACT_RELU>(a, acc, b, q, row0, col0);
        case MOE_ACT_SILU: return tile_epilogue<MI, MOE_ACT_SILU>(a, acc, b, q, row0, col0);
        case MOE_ACT_GELU: return tile_epilogue<MI, MOE_ACT_GELU>(a, acc, b, q, row0, col0);
        case MOE_ACT_GELU_TANH: return tile_epilogue<MI, MOE_ACT_GELU_TANH>(a, acc, b, q, row0, col0);
        default: return tile_epilogue<MI, MOE_ACT_NONE>(a, acc, b, q, row0, col0);
    }
}

// Epilogue of the gated block: acc[mi][0..1] gate and acc[mi][2..3] up, columns col0 + 16 j + 4 G .. +3 of row
// row0 + 16 mi; the wave's 32 columns exist together (N / 2 is a multiple of 32).  Kept sums and h
// move as the linear layer's output does.
template <int MI, int ACT>
__device__ __forceinline__ void gated_epilogue(const LinArgs& a, v4f (&acc)[MI][4], const v4f (&b)[4], int row0, int col0) {
    const int G = (threadIdx.x & 63) >> 4, I = a.N / 2;
    const bool on = col0 < I;
#pragma unroll
    for (int mi = 0; mi < MI; ++mi) {
        const int64_t row = row0 + 16 * mi;
        const bool live = on && row < a.T;
        v4f (&v)[4] = acc[mi];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += b[j];
        const int col = col0 + 16 * (G & 1) + 8 * (G >> 1);
        if (a.gu) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t lo[2], hi[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lo[j] = pack_bf16(v[2 * h + j][0], v[2 * h + j][1]);
                    hi[j] = pack_bf16(v[2 * h + j][2], v[2 * h + j][3]);
                }
                swap_groups(lo[0], lo[1]);
                swap_groups(hi[0], hi[1]);
                if (live) store16(reinterpret_cast<v4u_t*>(a.gu + row * a.N + h * I + col), v4u_t{lo[0], hi[0], lo[1], hi[1]}, a.nt);
            }
        }
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = act_fn(v[j][i], ACT) * v[j + 2][i];
            lo[j] = pack_bf16(h[0], h[1]);
            hi[j] = pack_bf16(h[2], h[3]);
        }
        swap_groups(lo[0], lo[1]);
        swap_groups(hi[0], hi[1]);
        if (live)
            store16(reinterpret_cast<v4u_t*>(reinterpret_cast<uint16_t*>(a.y) + row * I + col), v4u_t{lo[0], hi[0], lo[1], hi[1]}, a.nt);
    }
}
template <int MI>
__device__ __forceinline__ void gated_finish(const LinArgs& a, v4f (&acc)[MI][4], const v4f (&b)[4], int row0, int col0) {
    switch (a.act) {
        case MOE_ACT_RELU: return gated_epilogue<MI, MOE_ACT_RELU>(a, acc, b, row0, col0);
        case MOE_ACT_SILU: return gated_epilogue<MI, MOE_ACT_SILU>(a, acc, b, row0, col0);
        case MOE_ACT_GELU: return gated_epilogue<MI, MOE_ACT_GELU>(a, acc, b, row0, col0);
        case MOE_ACT_GELU_TANH: return gated_epilogue<MI, MOE_ACT_GELU_TANH>(a, acc, b, row0, col0);
        default: return gated_epilogue<MI, MOE_ACT_NONE>(a, acc, b, row0, col0);
    }
}

// Work order: workgroup L runs on XCD L % 8; XCD x takes a contiguous share of the list, which walks the
// row tiles in groups of 8 with the column tile outside, so that one XCD's workgroups share both
// operands through its L2.  False for the holes behind the last tile.
__device__ __forceinline__ bool tile_of(int L, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int w = (L & 7) * per + (L >> 3);
    if ((L >> 3) >= per || w >= total) return false;
    const int sb = w / (8 * tiles_n), r = w - sb * 8 * tiles_n, g = min(8, tiles_m - sb * 8);
    tn = r / g;
    tm = sb * 8 + r - tn * g;
    return true;
}

// 128-element scales of all K blocks: the rows' as [kb][wave row][row % 16][fragment], the weights' as
// [kb][column block of the tile, or wave's gate and up block].  8 threads per row of xs.
template <bool GATED, int MI, int ROWS, int COLS, int NTH>
__device__ __forceinline__ void load_scale_tables(const LinArgs& a, uint8_t* s_x, uint8_t* s_w, int KB, int nbs, int m0,
                                                  int tn) {
    constexpr int NBW = tile_scales<GATED>(COLS);
    const int tid = threadIdx.x;
    const int c = tid & 7;
    auto pos = [&](int q) { return (q / (16 * MI)) * 16 * MI + (q % 16) * MI + (q / 16) % MI; };
    if (KB % 4 == 0 && (reinterpret_cast<uintptr_t>(a.xs) & 3) == 0) {
        for (int k4 = c; k4 < KB / 4; k4 += 8) {
            uint32_t v[ROWS * 8 / NTH];
#pragma unroll
            for (int i = 0; i < ROWS * 8 / NTH; ++i)
                v[i] = reinterpret_cast<const uint32_t*>(a.xs)[(int64_t)min(m0 + (tid >> 3) + i * (NTH / 8), a.T - 1) * (KB / 4) + k4];
#pragma unroll
            for (int i = 0; i < ROWS * 8 / NTH; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s_x[(4 * k4 + k) * ROWS + pos((tid >> 3) + i * (NTH / 8))] = (uint8_t)(v[i] >> (8 * k));
        }
    } else {
        for (int q = tid >> 3; q < ROWS; q += NTH / 8)
            for (int kb = c; kb < KB; kb += 8)
                s_x[kb * ROWS + pos(q)] = a.xs[(int64_t)min(m0 + q, a.T - 1) * KB + kb];
    }
    for (int kb = tid; kb < KB; kb += NTH)
#pragma unroll
        for (int i = 0; i < NBW; ++i)
            s_w[kb * NBW + i] = a.ws[(int64_t)kb * nbs + (GATED ? column_fragment<GATED>(a, tn, COLS, 2 * i) / 8
                                                                : min(tn * COLS / kGroup + i, nbs - 1))];
}

// Bias of the tile's columns.
template <bool GATED, int COLS, int NTH>
__device__ __forceinline__ void load_bias(const LinArgs& a, float* s_bias, int tn) {
    for (int i = threadIdx.x; i < COLS; i += NTH) {
        if constexpr (GATED) s_bias[i] = a.bias ? a.bias[column_fragment<GATED>(a, tn, COLS, i / 16) * 16 + i % 16] : 0.f;
        else s_bias[i] = a.bias && tn * COLS + i < a.N ? a.bias[tn * COLS + i] : 0.f;
    }
}

// The K blocks that a workgroup sums (kBf16; with FP8 always all of them).
struct Blocks {
    int first, n;
};

template <Format F, bool GATED, int MI, int NJ, int WM, int WN>
__device__ __forceinline__ void linear_tile(const LinArgs& a, int L, int tiles_m, int tiles_n, Blocks part = {}) {
    static_assert(NJ == 4, "the epilogue takes 64 columns");
    constexpr bool MX = F == kMicro;
    constexpr int NW = WM * WN, ROWS = 16 * MI * WM, NTH = 64 * NW, DMA = ROWS * 8 / NTH;
    constexpr int STAGE = ROWS * kGroup, SCST = MX ? ROWS * 4 : 0;
    static_assert(ROWS * 8 % NTH == 0 && (!MX || ROWS % 64 == 0), "whole copies");
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* s_a = smem;                       // [3][ROWS][128]
    uint8_t* s_x = smem + 3 * STAGE;           // MX: [3][WM][16][MI] dwords; else [KB][WM][16][MI] bytes
    const int KB = a.K / kGroup, K0 = F == kBf16 ? part.first : 0, KN = F == kBf16 ? part.n : KB, nbs = (a.N + kGroup - 1) / kGroup;
    constexpr int COLS = 16 * NJ * WN, NBW = tile_scales<GATED>(COLS);
    uint8_t* s_w = s_x + KB * ROWS;            // (128-element scales) [KB][scales of the tile]
    float* s_bias = reinterpret_cast<float*>(F != kBlock ? s_x + 3 * SCST : s_w + (KB * NBW + 15) / 16 * 16);   // [COLS]

    int tm, tn;
    if (!tile_of(L, tiles_m, tiles_n, tm, tn)) return;
    // Two workgroups share a CU.  The one that was dealt second runs ahead at equal work, so that their
    // epilogues (memory) and K loops (matrix cores) fall apart: 4 us of 267 at 16384 x 4096 x 4096.
    if (MI > 4 && ((blockIdx.x >> 8) & 1)) __builtin_amdgcn_s_setprio(1);
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv / WN, wn = wv % WN, r16 = lane & 15, G = lane >> 4, x8 = r16 & 7;
    const int m0 = tm * ROWS, n16s = a.N / 16;
    constexpr int gpb = MX ? 4 : 1;

    const v4i_t ra = make_srd(a.xq, (uint32_t)a.T * (uint32_t)a.K);
    const v4i_t rs = make_srd(a.xs, (uint32_t)a.T * (uint32_t)(KB * gpb));
    const rsrc_t rw = make_rsrc(a.w, (uint32_t)a.K * (uint32_t)a.N);
    const rsrc_t rws = make_rsrc(a.ws, MX ? (uint32_t)KB * (uint32_t)n16s * 64u : (uint32_t)KB * (uint32_t)nbs);

    // copy i of wave wv: rows 8 (wv + NW i) .. +7; lane l brings one chunk of row + l / 8 to slot l % 8
    uint32_t aoff[DMA];
#pragma unroll
    for (int i = 0; i < DMA; ++i) {
        const int row = min(m0 + 8 * (wv + NW * i) + (lane >> 3), a.T - 1), slot = (lane & 7) ^ (lane >> 3);
        const int chunk = F != kBlock ? slot : (slot < 4 ? 2 * slot : 2 * slot - 7);
        aoff[i] = (uint32_t)row * (uint32_t)a.K + 16 * chunk + K0 * kGroup;
    }
    const uint32_t lds_w = lds_addr(s_a) + wv * 1024;
    uint32_t xoff = 0, lds_x = 0;   // MX: the row scales' dwords (waves past ROWS / 64 copy the last 64 again)
    if constexpr (MX) {
        const int pos = min(wv, ROWS / 64 - 1) * 64 + lane;   // [wm][row % 16][fragment]
        const int row = min(m0 + pos / (16 * MI) * (16 * MI) + (pos % MI) * 16 + (pos / MI) % 16, a.T - 1);
        xoff = (uint32_t)row * (uint32_t)(KB * 4);
        lds_x = lds_addr(s_x) + min(wv, ROWS / 64 - 1) * 256;
    }
    auto issue = [&](int kb, int st) __attribute__((always_inline)) {
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds_w + st * STAGE);
#pragma unroll
        for (int i = 0; i < DMA; ++i) dma16(ra, base + i * NW * 1024, aoff[i], kb * kGroup);
        if constexpr (MX) {
            dma4(rs, __builtin_amdgcn_readfirstlane(lds_x + st * SCST), xoff, kb * 4);
        }
    };
    // weights: fragment j of the wave, the operand's packed order (fragments past the last column: the
    // last one again, for columns that are not stored)
    uint32_t wfrag[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        wfrag[j] = __builtin_amdgcn_readfirstlane((uint32_t)column_fragment<GATED>(a, tn, COLS, wn * NJ + j) * (uint32_t)KB + K0);
    const uint32_t l16 = 16 * lane;
    struct Wt {
        v8i w[NJ];
        uint8_t s[NJ];
    };
    auto load_w = [&](int kb, Wt& W) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t f = wfrag[j] + (uint32_t)kb;
            const v4i_t lo = __builtin_amdgcn_raw_buffer_load_b128(rw, l16, f * kFragBytes, 0);
            const v4i_t hi = __builtin_amdgcn_raw_buffer_load_b128(rw, l16 + 1024, f * kFragBytes, 0);
            W.w[j] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            if constexpr (MX) W.s[j] = __builtin_amdgcn_raw_buffer_load_b8(rws, lane, f * 64, 0);
        }
    };
    // Everything loaded so far has arrived; stating it as a use keeps the compiler from waiting again
    // behind newer loads.
    auto arrived = [&](Wt& W) __attribute__((always_inline)) {
        wait_all();
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            asm volatile("" : "+v"(W.w[j]));
        }
    };
    Wt W0, W1;
    issue(0, 0);
    issue(min(1, KN - 1), 1);
    load_w(0, W0);
    load_bias<GATED, COLS, NTH>(a, s_bias, tn);
    if constexpr (F == kBlock) load_scale_tables<GATED, MI, ROWS, COLS, NTH>(a, s_x, s_w, KB, nbs, m0, tn);

    v4f acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto frag = [&](int st, int mi) __attribute__((always_inline)) {
        const uint8_t* rowp = s_a + st * STAGE + ((wm * MI + mi) * 16 + r16) * kGroup;
        const uint4 lo = *reinterpret_cast<const uint4*>(rowp + ((G ^ x8) << 4));
        const uint4 hi = *reinterpret_cast<const uint4*>(rowp + (((G + 4) ^ x8) << 4));
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    // The residual: with registers to spare it is requested before the K loop, else behind it.
    const int col0 = (tn * COLS + wn * NJ * 16) / (GATED ? 2 : 1), row0 = m0 + wm * MI * 16 + r16;
    uint4 res[MI][2];
    if constexpr (MI <= 4 && !GATED) tile_residual<MI>(a, res, row0, col0);
    arrived(W0);
    __syncthreads();
    // Row fragments are taken P at a time, the next P being read meanwhile: 2, or 1 with 32-element
    // scales, whose eight weight-scale registers leave no room for more (2 spilled 26 registers).
    constexpr int P = MX ? 1 : 2;
    v8i xa[P];
#pragma unroll
    for (int i = 0; i < P; ++i) xa[i] = frag(0, i);
    int st = 0;
    // One K block: on entry block kb is in its stage and W, its first row fragments in xa, and block
    // kb + 1's copies have been issued before the last wait.
    auto step = [&](int kb, Wt& W, Wt& N) __attribute__((always_inline)) {
        const int s1 = st == 2 ? 0 : st + 1, s2 = s1 == 2 ? 0 : s1 + 1;
        // (past the end the last block again, unused: the loop has no branches)
        load_w(min(kb + 1, KN - 1), N);
        issue(min(kb + 2, KN - 1), s2);
        int sx[(MI + 3) / 4] = {}, sw[2] = {};   // 128-element scales: byte mi % 4 of sx[mi / 4]; gate's and up's
        if constexpr (F == kBlock) {
            const int* p = reinterpret_cast<const int*>(s_x + kb * ROWS + (wm * 16 + r16) * MI);
#pragma unroll
            for (int i = 0; i < MI / 4; ++i) sx[i] = p[i];
            sw[0] = sw[1] = s_w[kb * NBW + (GATED ? 2 * wn : (wn * NJ * 16) / 128)];
            if constexpr (GATED) sw[1] = s_w[kb * NBW + 2 * wn + 1];
        }
        const uint32_t* mxs = reinterpret_cast<const uint32_t*>(s_x + st * SCST) + (wm * 16 + r16) * MI;
#pragma unroll
        for (int p = 0; p < MI; p += P) {
            v8i xn[P];
            int s[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                s[i] = MX ? (int)(mxs[p + i] >> (8 * G)) : sx[p / 4];   // MX: byte G of the row's four
                xn[i] = p + P < MI ? frag(st, p + P + i) : frag(s1, i);
            }
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[p + i][j] = products_of<F>(W.w[j], xa[i], acc[p + i][j], MX ? W.s[j] : sw[j / 2], s[i], MX ? 0 : (p + i) & 3);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < P; ++i) xa[i] = xn[i];
        }
        arrived(N);
        __syncthreads();
        st = s1;
    };
    int kb = 0;
    for (; kb + 2 <= KN; kb += 2) {
        step(kb, W0, W1);
        step(kb + 1, W1, W0);
    }
    if (kb < KN) step(kb, W0, W1);

    if constexpr (MI > 4 && !GATED) tile_residual<MI>(a, res, row0, col0);
    v4f bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = *reinterpret_cast<const v4f*>(s_bias + wn * NJ * 16 + 16 * j + 4 * G);
    if constexpr (GATED) gated_finish<MI>(a, acc, bias, row0, col0);
    else tile_finish<MI>(a, acc, bias, res, row0, col0);
}

template <Format F, bool GATED, int MI, int NJ, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_linear_tile(LinArgs a, int tiles_m, int tiles_n) {
    linear_tile<F, GATED, MI, NJ, WM, WN>(a, blockIdx.x, tiles_m, tiles_n);
}

// Launches a tiled kernel.
template <auto Kern>
static hipError_t launch_tiles(const LinArgs& a, int tm, int tn, int threads, size_t lds, hipStream_t st) {
    if (const hipError_t e = ask_for_lds<Kern>(lds); e != hipSuccess) return e;
    hipLaunchKernelGGL(Kern, dim3((unsigned)(ceil_div((int64_t)tm * tn, 8) * 8)), dim3(threads), lds, st, a, tm, tn);
    return hipGetLastError();
}

// LDS of the stages' neighbours: bias, and the 128-element scales of all K blocks or the micro scales of
// `stages` blocks of `lines` rows (and columns).
template <Format F, bool GATED>
static constexpr size_t scales_lds(int rows, int cols, int lines, int KB) {
    return cols * 4 + (F == kMicro ? (size_t)lines * 4
                       : F == kBlock ? (size_t)KB * rows + (KB * tile_scales<GATED>(cols) + 15) / 16 * 16 : 0);
}
template <Format F, bool GATED, int MI, int NJ, int WM, int WN>
static hipError_t run_tile_t(const LinArgs& a, hipStream_t st) {
    constexpr int ROWS = 16 * MI * WM, COLS = 16 * NJ * WN;
    const int tm = (int)ceil_div(a.T, ROWS), tn = (int)ceil_div(a.N, COLS);
    const size_t lds = 3 * ROWS * kGroup + scales_lds<F, GATED>(ROWS, COLS, 3 * ROWS, a.K / kGroup);
    return launch_tiles<k_linear_tile<F, GATED, MI, NJ, WM, WN>>(a, tm, tn, 64 * WM * WN, lds, st);
}

// ----------------------------------------------------------------------------------------
// The same product where there are too few tiles to hide a K block's latency behind another workgroup:
// both operands go through LDS, so that the copies are this kernel's only outstanding loads and their
// number can be waited for.  S stages hold S - 2 K blocks on their way while block kb's products run
// and block kb + 1's operands are read.  KS = 2: a second set of waves, with stages of its own, takes
// every other K block and hands its sums over through LDS at the end.  Bound by the chain wait, LDS read,
// product of a set's K blocks, about 0.27 us each (64 x 7168 x 7168: 14.1 us for 28, 3.9 TB/s of weights;
// 512 x 4096 x 4096: 15.6 us), and by LDS reads on larger tiles (2048 x 4096 x 4096: 36.6 us, 1.9 PFLOP/s).
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

template <Format F, bool GATED, int MI, int NJ, int WM, int WN, int S, int KS>
__device__ __forceinline__ void linear_deep(const LinArgs& a, int L, int tiles_m, int tiles_n, Blocks part = {}) {
    constexpr bool MX = F == kMicro;
    constexpr int NW = WM * WN, ROWS = 16 * MI * WM, COLS = 16 * NJ * WN, NTH = 64 * NW * KS;
    constexpr int DX = ROWS / 8 / NW, DW = COLS / 8 / NW;            // 1 KB copies of a wave and block
    constexpr int XB = ROWS * kGroup, WB = COLS * kGroup;
    constexpr int XS = MX ? ROWS * 4 : 0, WS = MX ? COLS * 4 : 0;    // MX: scales of a block
    constexpr int DS = MX ? (ROWS + COLS) / 64 / NW + ((ROWS + COLS) / 64 % NW != 0) : 0;   // 256-byte copies
    constexpr int STAGE = XB + WB + XS + WS, OPS = DX + DW + DS;
    static_assert(ROWS / 8 % NW == 0 && COLS / 8 % NW == 0 && ROWS % 64 == 0 && COLS % 64 == 0 && S >= 3, "whole copies");
    extern __shared__ __align__(16) uint8_t smem[];
    const int KB = a.K / kGroup, K0 = F == kBf16 ? part.first : 0, KN = F == kBf16 ? part.n : KB, nbs = (a.N + kGroup - 1) / kGroup;
    constexpr int NBW = tile_scales<GATED>(COLS), gpb = MX ? 4 : 1;
    uint8_t* s_x = smem + KS * S * STAGE;            // (128-element scales) [KB][WM][16][MI] bytes
    uint8_t* s_w = s_x + KB * ROWS;             // (128-element scales) [KB][scales of the tile]
    float* s_bias = reinterpret_cast<float*>(F != kBlock ? s_x : s_w + (KB * NBW + 15) / 16 * 16);   // [COLS]
    int tm, tn;
    if (!tile_of(L, tiles_m, tiles_n, tm, tn)) return;
    const int tid = threadIdx.x, lane = tid & 63, w0 = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = w0 / NW, wv = w0 % NW;       // set of waves, wave of the set
    const int wm = wv / WN, wn = wv % WN, r16 = lane & 15, G = lane >> 4, x8 = r16 & 7;
    const int m0 = tm * ROWS, n16s = a.N / 16;
    uint8_t* ring = smem + ks * S * STAGE;
    const v4i_t rx = make_srd(a.xq, (uint32_t)a.T * (uint32_t)a.K);
    const v4i_t rw = make_srd(a.w, (uint32_t)a.K * (uint32_t)a.N);
    const v4i_t rxs = make_srd(a.xs, (uint32_t)a.T * (uint32_t)(KB * gpb));
    const v4i_t rws = make_srd(a.ws, MX ? (uint32_t)KB * (uint32_t)n16s * 64u : (uint32_t)KB * (uint32_t)nbs);

    uint4 res[MI][2];
    const int col0 = (tn * COLS + wn * NJ * 16) / (GATED ? 2 : 1), row0 = m0 + wm * MI * 16 + r16;
    if (!GATED && ks == 0) tile_residual<MI>(a, res, row0, col0);

    uint32_t xoff[DX], wsrc[DW];   // rows as in k_linear_tile; weights: copy i of the wave, half a fragment
#pragma unroll
    for (int i = 0; i < DX; ++i) {
        const int row = min(m0 + 8 * (wv + NW * i) + (lane >> 3), a.T - 1), slot = (lane & 7) ^ (lane >> 3);
        const int chunk = F != kBlock ? slot : (slot < 4 ? 2 * slot : 2 * slot - 7);
        xoff[i] = (uint32_t)row * (uint32_t)a.K + 16 * chunk + K0 * kGroup;
    }
#pragma unroll
    for (int i = 0; i < DW; ++i) {
        const int g = wv + NW * i;
        wsrc[i] = __builtin_amdgcn_readfirstlane((uint32_t)column_fragment<GATED>(a, tn, COLS, g >> 1) * (uint32_t)KB * kFragBytes + (g & 1) * 1024 + K0 * kFragBytes);
    }
    const uint32_t l16 = 16 * lane, lds0 = lds_addr(ring);
    uint32_t soff[DS ? DS : 1], sdst[DS ? DS : 1];
    bool srow[DS ? DS : 1];
    if constexpr (MX) {   // the rows' dwords [wm][row % 16][fragment], then the column fragments' 64 bytes each
#pragma unroll
        for (int i = 0; i < DS; ++i) {
            const int c = min(wv + NW * i, (ROWS + COLS) / 64 - 1);   // (past the last: the last again)
            srow[i] = c < ROWS / 64;
            if (srow[i]) {
                const int pos = c * 64 + lane;
                const int row = min(m0 + pos / (16 * MI) * (16 * MI) + (pos % MI) * 16 + (pos / MI) % 16, a.T - 1);
                soff[i] = (uint32_t)row * (uint32_t)(KB * 4);
            } else {
                const int q = (c - ROWS / 64) * 64 + lane;            // dword q of the tile's fragments
                soff[i] = (uint32_t)column_fragment<GATED>(a, tn, COLS, q / 16) * (uint32_t)KB * 64 + (q % 16) * 4;
            }
            sdst[i] = XB + WB + c * 256;
        }
    }
    auto issue = [&](int blk, int st) __attribute__((always_inline)) {   // the set's block: K block blk KS + ks
        const int kb = min(blk * KS + ks, KN - 1);   // (past the end the last block again: the count per step stays)
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + st * STAGE + wv * 1024);
#pragma unroll
        for (int i = 0; i < DX; ++i) dma16(rx, base + i * NW * 1024, xoff[i], kb * kGroup);
#pragma unroll
        for (int i = 0; i < DW; ++i) dma16(rw, base + XB + i * NW * 1024, l16, wsrc[i] + kb * kFragBytes);
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < DS; ++i) {
                const uint32_t d = __builtin_amdgcn_readfirstlane(lds0 + st * STAGE + sdst[i]);
                if (srow[i]) dma4(rxs, d, soff[i], kb * 4);
                else dma4(rws, d, soff[i], kb * 64);
            }
        }
    };
    if constexpr (F == kBlock) load_scale_tables<GATED, MI, ROWS, COLS, NTH>(a, s_x, s_w, KB, nbs, m0, tn);
    load_bias<GATED, COLS, NTH>(a, s_bias, tn);
#pragma unroll
    for (int s = 0; s < S - 1; ++s) issue(s, s);

    struct Ops {
        v8i x[MI], w[NJ];
        int sx[MI], sw[NJ];
    };
    auto read = [&](int blk, int st, Ops& o) __attribute__((always_inline)) {
        const uint8_t* cur = ring + st * STAGE;
        const int kb = min(blk * KS + ks, KN - 1);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const uint8_t* rowp = cur + ((wm * MI + i) * 16 + r16) * kGroup;
            const uint4 lo = *reinterpret_cast<const uint4*>(rowp + ((G ^ x8) << 4));
            const uint4 hi = *reinterpret_cast<const uint4*>(rowp + (((G + 4) ^ x8) << 4));
            o.x[i] = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            if constexpr (MX) o.sx[i] = (int)(reinterpret_cast<const uint32_t*>(cur + XB + WB)[(wm * 16 + r16) * MI + i] >> (8 * G));
            else if constexpr (F == kBlock) o.sx[i] = s_x[kb * ROWS + (wm * 16 + r16) * MI + i];
            else o.sx[i] = 0;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint8_t* f = cur + XB + (wn * NJ + j) * kFragBytes + l16;
            const uint4 lo = *reinterpret_cast<const uint4*>(f), hi = *reinterpret_cast<const uint4*>(f + 1024);
            o.w[j] = v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
            if constexpr (MX) o.sw[j] = cur[XB + WB + XS + (wn * NJ + j) * 64 + lane];
            else if constexpr (F == kBlock) o.sw[j] = s_w[kb * NBW + (GATED ? 2 * wn + j / 2 : (wn * NJ * 16) / 128)];
            else o.sw[j] = 0;
        }
    };
    v4f acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    wait_vm<(S - 2) * OPS>();
    __syncthreads();
    Ops A, B;
    read(0, 0, A);
    int st = 0;   // stage of block i
    auto step = [&](int i, Ops& C, Ops& N) __attribute__((always_inline)) {
        wait_vm<(S - 3) * OPS>();   // block i + 1 has landed (this wave's copies) ...
        __syncthreads();            // ... and everyone's; block i - 1's stage has been read by all
        issue(i + S - 1, st == 0 ? S - 1 : st - 1);
        st = st == S - 1 ? 0 : st + 1;
        read(i + 1, st, N);
    };
    auto products = [&](Ops& C) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = products_of<F>(C.w[j], C.x[i], acc[i][j], C.sw[j], C.sx[i], 0);
    };
    const int n = (KN + KS - 1) / KS;   // blocks of a set; the last may lie past the end
    int i = 0;
    for (; i + 2 < n; i += 2) {
        step(i, A, B);
        products(A);
        step(i + 1, B, A);
        products(B);
    }
    if (i + 1 < n) {
        step(i, A, B);
        products(A);
        ++i;
        if (KS == 1 || i * KS + ks < KN) products(B);
    } else if (KS == 1 || i * KS + ks < KN) {
        products(A);
    }
    wait_all();
    if constexpr (KS > 1) {   // the second set's sums, through the stages: every copy has ended, every read too
        static_assert(KS == 2 && NW * MI * NJ * 1024 <= KS * S * STAGE, "one set hands over to one");
        v4f* hand = reinterpret_cast<v4f*>(smem);
        __syncthreads();
        if (ks) {
#pragma unroll
            for (int q = 0; q < MI * NJ; ++q) hand[(wv * MI * NJ + q) * 64 + lane] = acc[q / NJ][q % NJ];
        }
        __syncthreads();
        if (ks) return;
#pragma unroll
        for (int q = 0; q < MI * NJ; ++q) acc[q / NJ][q % NJ] += hand[(wv * MI * NJ + q) * 64 + lane];
    }

    v4f bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = *reinterpret_cast<const v4f*>(s_bias + wn * NJ * 16 + 16 * j + 4 * G);
    if constexpr (GATED) gated_finish<MI>(a, acc, bias, row0, col0);
    else tile_finish<MI>(a, acc, bias, res, row0, col0);
}

// LDS of a deep tile: stages, bias, scales.
template <Format F, bool GATED>
static constexpr size_t deep_lds(int rows, int cols, int stages, int KB) {
    return (size_t)stages * (rows + cols) * kGroup + scales_lds<F, GATED>(rows, cols, stages * (rows + cols), KB);
}
template <Format F, bool GATED, int MI, int NJ, int WM, int WN, int S, int KS>
__global__ __launch_bounds__(64 * WM * WN * KS, 1) void k_linear_deep(LinArgs a, int tiles_m, int tiles_n) {
    linear_deep<F, GATED, MI, NJ, WM, WN, S, KS>(a, blockIdx.x, tiles_m, tiles_n);
}
template <Format F, bool GATED, int MI, int NJ, int WM, int WN, int S, int KS>
static hipError_t run_deep_t(const LinArgs& a, hipStream_t st) {
    constexpr int ROWS = 16 * MI * WM, COLS = 16 * NJ * WN;
    const int tm = (int)ceil_div(a.T, ROWS), tn = (int)ceil_div(a.N, COLS);
    const size_t lds = deep_lds<F, GATED>(ROWS, COLS, KS * S, a.K / kGroup);
    return launch_tiles<k_linear_deep<F, GATED, MI, NJ, WM, WN, S, KS>>(a, tm, tn, 64 * WM * WN * KS, lds, st);
}
template <bool GATED, int MI, int NJ, int WM, int WN, int S, int KS>
static hipError_t run_deep(const LinArgs& a, hipStream_t st) {
    return a.mx ? run_deep_t<kMicro, GATED, MI, NJ, WM, WN, S, KS>(a, st) : run_deep_t<kBlock, GATED, MI, NJ, WM, WN, S, KS>(a, st);
}

template <bool GATED, int NF, int WK, int PF>
static hipError_t run_stream(const LinArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)ceil_div(a.N, 16 * NF), (unsigned)ceil_div(a.T, 16));
    if (a.mx) hipLaunchKernelGGL((k_linear_stream<kMicro, GATED, NF, WK, PF>), grid, dim3(64 * WK), 0, st, a);
    else hipLaunchKernelGGL((k_linear_stream<kBlock, GATED, NF, WK, PF>), grid, dim3(64 * WK), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
