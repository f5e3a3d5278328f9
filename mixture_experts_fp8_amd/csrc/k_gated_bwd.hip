// Backward pass of the gated block (gfx950): from dh and the kept sums g, u,
//   dgu = bf16([dh u act'(g) | dh act(g)]),  dx = dgu @ W^T,  dW = x^T @ dgu,  dbias = column sums.
// The two products run in bf16 on the kernels of linear_tiles.h, whose operands are brought into its layouts
// first: rows with the summed index contiguous, and fragments of 16 columns.  E4M3 values times a power of
// two are bf16 values, so those operands lose nothing (but beyond bf16's range, which scales of 2^-124 and
// below or 2^120 and above can reach).
#include "linear_tiles.h"

namespace moe {

namespace {

// act(v) and its slope; the same functions as act_fn, and without cancellation where one of the two
// factors of a logistic is small.
struct Act {
    float a, s;
};
template <int ACT>
__device__ __forceinline__ Act act_slope(float v) {
    if constexpr (ACT == MOE_ACT_RELU) return {v < 0.f ? 0.f : v, v > 0.f ? 1.f : 0.f};
    if constexpr (ACT == MOE_ACT_SILU) {
        const float e = exp_fast(-v), p = __builtin_amdgcn_rcpf(1.0f + e);
        const float q = v < 0.f ? 1.0f - p : e * p;      // 1 - p
        const float a = v * p;
        return {a, fmaf(a, q, p)};
    }
    if constexpr (ACT == MOE_ACT_GELU) {
        const float c = normal_cdf(v), d = __builtin_amdgcn_exp2f(v * v * -0.72134752f);   // exp(-v^2 / 2)
        return {v * c, fmaf(v * 0.398942280f, d, c)};
    }
    if constexpr (ACT == MOE_ACT_GELU_TANH) {
        const float w = v * v, u = 1.59576912f * fmaf(0.044715f * w, v, v);   // twice tanh's argument
        const float e = exp_fast(-u), p = __builtin_amdgcn_rcpf(1.0f + e);
        const float q = (u < 0.f ? 1.0f - p : e * p) * p;      // p (1 - p)
        // (from |v| of 1e12 on the last factors would leave float32; q is 0 long before)
        return {v * p, q == 0.f ? p : fmaf(v * q, 1.59576912f * fmaf(0.134145f, w, 1.0f), p)};
    }
    return {v, 1.0f};
}

// 2^(s - 127) of a UE8M0 byte; 255 is NaN.
__device__ __forceinline__ float ue8m0(uint32_t s) { return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23); }

// The values of four E4M3 codes.
__device__ __forceinline__ void decode4(uint32_t q, float (&f)[4]) {
    const v2f_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q, true);
    f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
}

// Low and high halves of two words, a's first.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// 8 x 8 transpose of bf16 values: rows r[i] (8 columns each) -> the 8 rows' values of column c.
__device__ __forceinline__ v4u_t column_of(const uint4 (&r)[8], int c) {
    auto word = [&](int i) __attribute__((always_inline)) { return c < 2 ? r[i].x : c < 4 ? r[i].y : c < 6 ? r[i].z : r[i].w; };
    v4u_t v;
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = c % 2 ? high_halves(word(2 * p), word(2 * p + 1)) : low_halves(word(2 * p), word(2 * p + 1));
    return v;
}

struct DguArgs {
    int T, I, NT;           // NT: blocks of 64 rows
    const uint16_t* dh;
    const uint16_t* gu;
    uint16_t* dgu;
    uint8_t* packed;        // or NULL: dgu as column fragments whose K is the row, rows past T 0
    float* part;            // or NULL: [gridDim.x][2I] column sums
};

// A wave takes 64 columns of g and u and blocks of 64 rows, a grid apart; lane (t = l / 8, c = l % 8) the rows
// 8 t .. +7 and columns 8 c .. +7 of a block, all loads of which are in flight together.  Column sums stay in
// registers.  The fragments of the transposed result go through LDS, so that they leave in whole kilobytes;
// slots are swizzled by t, which spreads the lanes' 16-byte writes over the banks.
template <int ACT, bool PACK>
__global__ __launch_bounds__(256) void k_gated_dgu(DguArgs a) {
    __shared__ __align__(16) uint8_t s_frag[4][PACK ? 8192 : 16];
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t8 = lane >> 3, c8 = lane & 7, col = (blockIdx.y * 4 + wv) * 64 + 8 * c8;
    const bool on = col < a.I;
    if ((blockIdx.y * 4 + wv) * 64 >= a.I) return;   // (uniform; no barrier follows)
    const int64_t N = 2 * (int64_t)a.I;
    float sg[8] = {}, su[8] = {};
    for (int b = blockIdx.x; b < a.NT; b += gridDim.x) {
        uint4 g[8], u[8], d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = (int64_t)b * 64 + 8 * t8 + i;
            g[i] = u[i] = d[i] = make_uint4(0, 0, 0, 0);
            if (on && t < a.T) {
                g[i] = *reinterpret_cast<const uint4*>(a.gu + t * N + col);
                u[i] = *reinterpret_cast<const uint4*>(a.gu + t * N + a.I + col);
                d[i] = *reinterpret_cast<const uint4*>(a.dh + t * a.I + col);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = (int64_t)b * 64 + 8 * t8 + i;
            float x[8], y[8], z[8];
            unpack8(g[i], x);
            unpack8(u[i], y);
            unpack8(d[i], z);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const Act f = act_slope<ACT>(x[j]);
                x[j] = z[j] * y[j] * f.s;
                y[j] = z[j] * f.a;
                if (t >= a.T) x[j] = y[j] = 0.f;
                sg[j] += x[j];
                su[j] += y[j];
            }
            g[i] = pack8(x);
            u[i] = pack8(y);
            if (on && t < a.T) {
                *reinterpret_cast<uint4*>(a.dgu + t * N + col) = g[i];
                *reinterpret_cast<uint4*>(a.dgu + t * N + a.I + col) = u[i];
            }
        }
        if constexpr (PACK) {
            v4u_t* s = reinterpret_cast<v4u_t*>(s_frag[wv]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    s[(c8 >> 1) * 128 + t8 * 16 + ((8 * (c8 & 1) + c) ^ t8)] = column_of(half ? u : g, c);
                asm volatile("" ::: "memory");   // (a wave's LDS accesses stay in order)
                __builtin_amdgcn_wave_barrier();
                const int n0 = (half ? a.I : 0) / 16 + (blockIdx.y * 4 + wv) * 4;
#pragma unroll
                for (int q = 0; q < 8; ++q) {    // fragment q / 2, its lower and upper kilobyte
                    const int p = (q & 1) * 64 + lane, r = p >> 4;
                    const v4u_t v = s[(q >> 1) * 128 + r * 16 + ((p & 15) ^ r)];
                    if ((blockIdx.y * 4 + wv) * 64 + 16 * (q >> 1) < a.I)
                        *reinterpret_cast<v4u_t*>(a.packed + ((int64_t)(n0 + (q >> 1)) * a.NT + b) * kFragBytes + p * 16) = v;
                }
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
    if (a.part) {   // over the lanes of a column, then one row of the parts
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int m = 8; m < 64; m *= 2) {
                sg[j] += __shfl_xor(sg[j], m);
                su[j] += __shfl_xor(su[j], m);
            }
        }
        if (t8 == 0 && on) {
            float* p = a.part + (int64_t)blockIdx.x * N + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = sg[j], p[a.I + j] = su[j];
        }
    }
}

// x^T as bf16 [K][64 NT], 0 behind row T.  A wave takes 64 rows and 64 columns, a lane 8 x 8 of them; its
// 16-byte vectors of 8 rows make 128 bytes of a row of the result.
template <bool MX>
__global__ __launch_bounds__(256) void k_rows_transposed(const uint8_t* xq, const uint8_t* xs, int T, int K, int NT, uint16_t* xt) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t0 = blockIdx.x * 64 + 8 * (lane & 7), k0 = (blockIdx.y * 4 + wv) * 64 + 8 * (lane >> 3);
    if (k0 >= K) return;
    constexpr int gs = MX ? 32 : 128;
    uint2 q[8];
    uint8_t s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t t = min(t0 + i, T - 1);
        q[i] = *reinterpret_cast<const uint2*>(xq + t * K + k0);
        s[i] = xs[t * (K / gs) + k0 / gs];
    }
    uint4 r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = ue8m0(s[i]);
        float f[4], v[8];
        decode4(q[i].x, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = f[j] * m;
        decode4(q[i].y, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 + j] = f[j] * m;
        r[i] = t0 + i < T ? pack8(v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<v4u_t*>(xt + (int64_t)(k0 + c) * (NT * 64) + t0) = column_of(r, c);
}

// The packed FP8 weights [K][N] as bf16 fragments of 16 rows of w whose K is the column: a workgroup turns 4
// fragments of 16 columns x 128 rows into 8 of 16 rows x 64 columns.
template <bool MX>
__global__ __launch_bounds__(256) void k_weights_transposed(const uint8_t* w, const uint8_t* ws, int K, int N, uint8_t* out) {
    __shared__ __align__(16) uint8_t s_w[4 * kFragBytes];
    __shared__ uint8_t s_s[4 * 64];
    const int tid = threadIdx.x, jb = blockIdx.x, kb = blockIdx.y, KB = K / kGroup, NJ = N / 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int p = i * 256 + tid, f = p >> 7;
        *reinterpret_cast<uint4*>(s_w + p * 16) =
            *reinterpret_cast<const uint4*>(w + ((int64_t)(jb * 4 + f) * KB + kb) * kFragBytes + (p & 127) * 16);
    }
    if constexpr (MX) s_s[tid] = ws[((int64_t)(jb * 4 + (tid >> 6)) * KB + kb) * 64 + (tid & 63)];
    const float m = MX ? 0.f : ue8m0(ws[(int64_t)kb * ((N + kGroup - 1) / kGroup) + jb / 2]);
    __syncthreads();
    const int quad = tid >> 3, n8 = tid & 7, k = 4 * quad;   // 4 rows of w, 8 columns
    const int G = MX ? (k >> 4) & 3 : k >> 5, h = MX ? k >> 6 : (k >> 4) & 1;   // where the packing has them
    float v[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * (n8 & 1) + i;
        decode4(*reinterpret_cast<const uint32_t*>(s_w + (n8 >> 1) * kFragBytes + h * 1024 + (G * 16 + r) * 16 + (k & 15)), v[i]);
        const float mi = MX ? ue8m0(s_s[(n8 >> 1) * 64 + (k >> 5) * 16 + r]) : m;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] *= mi;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const v4u_t o = {pack_bf16(v[0][j], v[1][j]), pack_bf16(v[2][j], v[3][j]), pack_bf16(v[4][j], v[5][j]), pack_bf16(v[6][j], v[7][j])};
        const int kr = k + j;
        *reinterpret_cast<v4u_t*>(out + ((int64_t)(kb * 8 + (kr >> 4)) * NJ + jb) * kFragBytes + (n8 >> 2) * 1024 +
                                  ((n8 & 3) * 16 + (kr & 15)) * 16) = o;
    }
}

template <bool PACK>
void run_dgu(const DguArgs& a, int act, dim3 grid, hipStream_t st) {
    switch (act) {
        case MOE_ACT_RELU: hipLaunchKernelGGL((k_gated_dgu<MOE_ACT_RELU, PACK>), grid, dim3(256), 0, st, a); break;
        case MOE_ACT_SILU: hipLaunchKernelGGL((k_gated_dgu<MOE_ACT_SILU, PACK>), grid, dim3(256), 0, st, a); break;
        case MOE_ACT_GELU: hipLaunchKernelGGL((k_gated_dgu<MOE_ACT_GELU, PACK>), grid, dim3(256), 0, st, a); break;
        case MOE_ACT_GELU_TANH: hipLaunchKernelGGL((k_gated_dgu<MOE_ACT_GELU_TANH, PACK>), grid, dim3(256), 0, st, a); break;
        default: hipLaunchKernelGGL((k_gated_dgu<MOE_ACT_NONE, PACK>), grid, dim3(256), 0, st, a);
    }
}

// Tile by the number of workgroups, as launch_linear's.
hipError_t launch_product(const LinArgs& args, hipStream_t st) {
    LinArgs a = args;
    a.nt = (int64_t)a.T * a.N * (a.out_bf16 ? 2 : 4) >= (32 << 20);
    auto fits = [&](int rows, int cols, int64_t most) { return ceil_div(a.T, rows) * ceil_div(a.N, cols) <= most; };
    if (fits(64, 64, 256)) return run_deep_t<kBf16, false, 1, 4, 4, 1, 4, 2>(a, st);
    if (fits(64, 128, 256)) return run_deep_t<kBf16, false, 2, 4, 2, 2, 4, 1>(a, st);
    if (fits(64, 128, 512)) return run_deep_t<kBf16, false, 2, 4, 2, 2, 3, 1>(a, st);
    if (fits(128, 256, 256)) return run_deep_t<kBf16, false, 4, 4, 2, 4, 3, 1>(a, st);
    return run_tile_t<kBf16, false, 8, 4, 1, 4>(a, st);
}

}  // namespace

hipError_t launch_gated_backward(const GatedBwdArgs& a, hipStream_t st) {
    const GatedBwdPlan p = gated_bwd_plan(a.T, a.K, a.I, a.dx != nullptr, a.dw != nullptr, a.dbias != nullptr);
    const int N = 2 * a.I, NT = p.row_blocks;
    uint8_t* ws = a.ws;
    float* part = a.dbias ? reinterpret_cast<float*>(ws + p.part) : nullptr;
    const DguArgs d{a.T, a.I, NT, a.dh, a.gu, a.dgu, a.dw ? ws + p.dgu_packed : nullptr, part};
    const dim3 grid((unsigned)(a.dbias ? p.parts : NT), (unsigned)ceil_div(a.I, 256));
    if (a.dw) run_dgu<true>(d, a.act, grid, st);
    else run_dgu<false>(d, a.act, grid, st);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && a.dbias) e = launch_column_sums(part, p.parts, N, a.dbias, st);
    if (e != hipSuccess) return e;
    if (a.dx) {
        const dim3 g((unsigned)(N / 64), (unsigned)(a.K / kGroup));
        if (a.mx) hipLaunchKernelGGL(k_weights_transposed<true>, g, dim3(256), 0, st, a.w, a.wsc, a.K, N, ws + p.weights);
        else hipLaunchKernelGGL(k_weights_transposed<false>, g, dim3(256), 0, st, a.w, a.wsc, a.K, N, ws + p.weights);
        LinArgs l{};
        l.T = a.T, l.K = 2 * N, l.N = a.K;
        l.xq = reinterpret_cast<const uint8_t*>(a.dgu), l.w = ws + p.weights;
        l.y = a.dx, l.ldy = a.K, l.out_bf16 = 1;
        if ((e = hipGetLastError()) != hipSuccess || (e = launch_product(l, st)) != hipSuccess) return e;
    }
    if (a.dw) {
        const dim3 g((unsigned)NT, (unsigned)ceil_div(a.K, 256));
        uint16_t* xt = reinterpret_cast<uint16_t*>(ws + p.rows);
        if (a.mx) hipLaunchKernelGGL(k_rows_transposed<true>, g, dim3(256), 0, st, a.xq, a.xs, a.T, a.K, NT, xt);
        else hipLaunchKernelGGL(k_rows_transposed<false>, g, dim3(256), 0, st, a.xq, a.xs, a.T, a.K, NT, xt);
        LinArgs l{};
        l.T = a.K, l.K = 128 * NT, l.N = N;
        l.xq = ws + p.rows, l.w = ws + p.dgu_packed;
        l.y = a.dw, l.ldy = N, l.out_bf16 = a.dw_bf16;
        if ((e = hipGetLastError()) != hipSuccess || (e = launch_product(l, st)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace moe
