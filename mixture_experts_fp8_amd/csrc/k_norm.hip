// Residual addition + RMS norm with E4M3 codes, and its backward pass (gfx950).
//
// One pass: a row's vectors of 8 columns stay in registers between the sum of squares and the
// output, so every input byte is read once and every output byte written once; the kernels are
// bound by HBM.
#include "layer_common.h"

#include <algorithm>

namespace moe {

// 16- and 8-byte accesses; ST (streamed): past the caches, for matrices larger than they are.
typedef unsigned v4u_t __attribute__((ext_vector_type(4)));
typedef unsigned v2u_t __attribute__((ext_vector_type(2)));
template <bool ST>
__device__ __forceinline__ uint4 ld16(const void* p) {
    const v4u_t* q = reinterpret_cast<const v4u_t*>(p);
    const v4u_t v = ST ? __builtin_nontemporal_load(q) : *q;
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool ST>
__device__ __forceinline__ void st16(void* p, uint4 v) {
    const v4u_t x = {v.x, v.y, v.z, v.w};
    if constexpr (ST) __builtin_nontemporal_store(x, reinterpret_cast<v4u_t*>(p));
    else *reinterpret_cast<v4u_t*>(p) = x;
}
template <bool ST>
__device__ __forceinline__ void st8(void* p, uint2 v) {
    const v2u_t x = {v.x, v.y};
    if constexpr (ST) __builtin_nontemporal_store(x, reinterpret_cast<v2u_t*>(p));
    else *reinterpret_cast<v2u_t*>(p) = x;
}
// One of the matrices alone is larger than the L2s together, so none of them is found there by the next
// operator (4096 x 7168 with residual and codes 55.2 -> 51.4 us, backward at 16384 x 4096 97 -> 90; at
// 2048 x 2816, which fits, streaming costs 5%).
static bool streamed(int T, int H) { return (int64_t)T * H * 2 >= (32 << 20); }

// Lane exchange of both halves of a double by the DPP control word of dpp_f32.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp_u32<CTRL>((uint32_t)(u >> 32)) << 32 | dpp_u32<CTRL>((uint32_t)u));
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x124>(v);
    v += dpp_f64<0x128>(v);
    return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// Sum over the G threads of a row: a wave's sum, then (G > 64) the waves' sums through LDS in wave
// order.  s: G / 64 doubles, used once.
template <int G>
__device__ __forceinline__ double row_sum(double v, double* s) {
    v = wave_sum(v);
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int i = 0; i < G / 64; ++i) v += s[i];
    }
    return v;
}

// 1 / sqrt(x) to double precision: the instruction's estimate (about 2^-26 off) and one Newton step,
// which would make NaN of the infinity and the zero that the ends of the range give.
__device__ __forceinline__ double rsqrt_f64(double x) {
    const double r = __builtin_amdgcn_rsq(x);
    const double n = r * fma(-0.5 * x * r, r, 1.5);
    return x > 0.0 && x < __builtin_inf() ? n : r;
}

// A double as a float that rounds to the same bf16: rounded to odd (towards zero, the last bit set where
// anything was cut off).  Rounded to nearest it could land on the middle of two bf16 values and be
// rounded the other way then, which happens to one value in 2^17.  Infinities (of an infinite weight) and NaN
// have no remainder that compares with 0 and stay as they are.
__device__ __forceinline__ float round_odd(double d) {
    const float f = (float)d;
    const double r = d - (double)f;
    uint32_t u = __float_as_uint(f);
    if (r < 0.0 || r > 0.0) u = (u - ((r > 0.0) != (d > 0.0) ? 1u : 0u)) | 1u;
    return __uint_as_float(u);
}

// E4M3 codes of 8 values in each of LANES consecutive lanes sharing one scale (LANES * 8 columns):
// the rule of moe_quant_act on values that are bf16 already.
template <int LANES>
__device__ __forceinline__ uint2 group_codes(const float (&f)[8], int& e) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    m = fmaxf(m, dpp_f32<0xB1>(m));
    m = fmaxf(m, dpp_f32<0x4E>(m));
    if constexpr (LANES == 16) {
        m = fmaxf(m, dpp_f32<0x124>(m));
        m = fmaxf(m, dpp_f32<0x128>(m));
    }
    e = scale_exponent(m);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ldexpf(f[i], -e);
    return make_uint2(cvt4_e4m3(q[0], q[1], q[2], q[3]), cvt4_e4m3(q[4], q[5], q[6], q[7]));
}

// G threads per row, VPT vectors of 8 columns per thread (G * VPT >= H / 8); a workgroup holds
// max(1, 256 / G) rows.  The row's sum, its root and the two products are formed in double, which the
// memory hides: y is then the definition's value rounded once, and the codes, which a value beside a
// border would otherwise tip, are the definition's codes.  4096 x 7168 with residual and 32-column codes:
// 50 us, 5.3 TB/s of what it must move; 32 x 2816: 3.7 us, a launch.
template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_add_rmsnorm(NormArgs a) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    __shared__ double s_sum[G / 64];
    const int sub = threadIdx.x % G, nv = a.H >> 3;
    const int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / G;
    if (RPB > 1 && t >= a.T) return;   // (RPB > 1 only with G = 64: no barrier follows)
    const uint16_t* xr = a.x + t * a.ldx;
    const uint16_t* rr = a.res ? a.res + t * a.ldr : nullptr;
    uint4 vx[VPT], vr[VPT];
    float4 w0[VPT], w1[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = sub + i * G;
        if (v < nv) vx[i] = ld16<ST>(xr + v * 8);
        else vx[i] = make_uint4(0, 0, 0, 0);
    }
    if (rr) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            if (v < nv) vr[i] = ld16<ST>(rr + v * 8);
            else vr[i] = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = sub + i * G;
        if (v < nv) {
            w0[i] = *reinterpret_cast<const float4*>(a.w + v * 8);
            w1[i] = *reinterpret_cast<const float4*>(a.w + v * 8 + 4);
        }
    }
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float f[8];
        unpack8(vx[i], f);
        if (rr) {
            float g[8];
            unpack8(vr[i], g);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += g[j];
            vx[i] = pack8(f);      // h, rounded once; kept as bf16
            unpack8(vx[i], f);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fma((double)f[j], (double)f[j], ss);
    }
    if (a.h) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            if (v < nv) st16<ST>(a.h + t * a.H + v * 8, vx[i]);
        }
    }
    if (!a.y && !a.yq) return;   // (uniform)
    const double r = rsqrt_f64(fma(row_sum<G>(ss, s_sum), a.inv_h, (double)a.eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = sub + i * G;
        float f[8];
        unpack8(vx[i], f);
        const float w[8] = {w0[i].x, w0[i].y, w0[i].z, w0[i].w, w1[i].x, w1[i].y, w1[i].z, w1[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = round_odd((double)f[j] * r * (double)w[j]);
        const uint4 o = pack8(f);
        if (v < nv) {   // a scale's lanes are all in or all out: H is a multiple of its columns
            if (a.y) st16<ST>(a.y + t * a.H + v * 8, o);
            if (a.yq) {
                unpack8(o, f);
                int e;
                if (a.group == 128) {
                    st8<ST>(a.yq + t * a.H + v * 8, group_codes<16>(f, e));
                    if ((v & 15) == 0) a.ys[t * (a.H >> 7) + (v >> 4)] = (uint8_t)(e + 127);
                } else {
                    st8<ST>(a.yq + t * a.H + v * 8, group_codes<4>(f, e));
                    if ((v & 3) == 0) a.ys[t * (a.H >> 5) + (v >> 2)] = (uint8_t)(e + 127);
                }
            }
        }
    }
}

template <int G, int VPT>
static void run_norm(const NormArgs& args, hipStream_t st) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    const dim3 block(G < 256 ? 256 : G);
    NormArgs a = args;
    for (int64_t t = 0; t < args.T; t += launch_rows(G)) {
        a.T = (int)std::min<int64_t>(args.T - t, launch_rows(G));
        a.x = args.x + t * args.ldx;
        if (args.res) a.res = args.res + t * args.ldr;
        if (args.h) a.h = args.h + t * args.H;
        if (args.y) a.y = args.y + t * args.H;
        if (args.yq) {
            a.yq = args.yq + t * args.H;
            a.ys = args.ys + t * (args.H / args.group);
        }
        const dim3 grid((unsigned)ceil_div(a.T, RPB));
        if (streamed(args.T, args.H)) hipLaunchKernelGGL((k_add_rmsnorm<G, VPT, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_add_rmsnorm<G, VPT, false>), grid, block, 0, st, a);
    }
}

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t st) {
    const int nv = a.H / 8;
    if (nv <= 64) run_norm<64, 1>(a, st);
    else if (nv <= 256) run_norm<256, 1>(a, st);
    else if (nv <= 512) run_norm<512, 1>(a, st);
    else if (nv <= 1024) run_norm<512, 2>(a, st);   // (with one vector each, 1024 threads are 2% slower at 4096 x 7168)
    else if (nv <= 2048) run_norm<1024, 2>(a, st);
    else run_norm<1024, 4>(a, st);
    return hipGetLastError();
}

// ----------------------------------------------------------------------------------------
// Backward.  With xhat = h r and g = dy w:  dx = r (g - xhat mean(g xhat)) + dh, and the weight
// gradient sum_t dy xhat.  A workgroup of G threads (short rows: four waves with a row each) walks rows
// a grid apart, keeps its share of the weight gradient in registers; the workgroups' sums go to `part`
// and are added in workgroup order by k_norm_dw.  The two sums and xhat are formed in double, as the
// forward's: their squares would leave float32 at |h| of 1e19 and 1e-19.  Bound by HBM: 16384 x 4096 with
// dh 90 us, 6.0 TB/s of what it must move.  The next row is in flight over this one's sums, so long rows take
// more vectors per thread, not more threads: 512 threads have the registers for it (2048 x 16384: 61 us,
// 1024 threads 69, with spills).
template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_add_rmsnorm_bwd(NormBwdArgs a) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    constexpr bool AHEAD = VPT <= 4;   // else the registers hold no second row and no weights
    __shared__ double s_sum[2][2][G / 64];
    __shared__ __align__(16) float s_dw[RPB][RPB > 1 ? VPT * G * 8 : 4];
    const int sub = RPB > 1 ? threadIdx.x % G : threadIdx.x, rw = RPB > 1 ? threadIdx.x / G : 0, nv = a.H >> 3;
    const int64_t step = (int64_t)gridDim.x * RPB;
    float dw[VPT][8], wk[AHEAD ? VPT : 1][8];
    auto weights = [&](int i, float (&w)[8]) __attribute__((always_inline)) {
        const int v = sub + i * G;
        const float* p = a.w;
        if constexpr (!AHEAD) asm volatile("" : "+s"(p));   // read again each time, not kept
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = v < nv ? p[v * 8 + j] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
        if constexpr (AHEAD) weights(i, wk[i]);
    }
    struct Row {
        uint4 h[VPT], d[VPT], r[VPT];
    };
    auto load = [&](int64_t t, Row& x) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = sub + i * G;
            const int64_t o = t * a.H;
            x.h[i] = x.d[i] = x.r[i] = make_uint4(0, 0, 0, 0);
            if (v < (uint32_t)nv) {   // (a row's base, the same for all of its threads, and 32-bit offsets)
                x.h[i] = ld16<ST>(a.h + o + v * 8);
                x.d[i] = ld16<ST>(a.dy + o + v * 8);
                if (a.dh) x.r[i] = ld16<ST>(a.dh + o + v * 8);
            }
        }
    };
    int par = 0;
    Row nx;
    const int64_t first = (int64_t)blockIdx.x * RPB + rw;
    if (AHEAD && first < a.T) load(first, nx);
    for (int64_t t = first; t < a.T; t += step, par ^= 1) {
        if (!AHEAD) load(t, nx);
        uint4 vh[VPT], vd[VPT], vr[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) vh[i] = nx.h[i], vd[i] = nx.d[i], vr[i] = nx.r[i];
        if (AHEAD && t + step < a.T) load(t + step, nx);   // in flight over this row's sums
        // sum h^2 and sum g h in one exchange: mean(g xhat) = r sum(g h) / H
        double ss = 0.0, gh = 0.0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float h[8], d[8], wt[8];
            unpack8(vh[i], h);
            unpack8(vd[i], d);
            if constexpr (!AHEAD) weights(i, wt);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fma((double)h[j], (double)h[j], ss);
                gh = fma((double)(d[j] * (AHEAD ? wk[AHEAD ? i : 0][j] : wt[j])), (double)h[j], gh);
            }
            if constexpr (VPT > 2) __builtin_amdgcn_sched_barrier(0);   // one vector's values at a time
        }
        ss = wave_sum(ss);
        gh = wave_sum(gh);
        if constexpr (G > 64) {
            if ((sub & 63) == 0) {
                s_sum[par][0][sub >> 6] = ss;
                s_sum[par][1][sub >> 6] = gh;
            }
            __syncthreads();
            ss = gh = 0.0;
#pragma unroll
            for (int i = 0; i < G / 64; ++i) {
                ss += s_sum[par][0][i];
                gh += s_sum[par][1][i];
            }
        }
        const double rd = rsqrt_f64(fma(ss, a.inv_h, (double)a.eps));
        const float r = (float)rd, m = (float)(gh * a.inv_h * rd);   // m = mean(g xhat)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            float h[8], d[8], e[8], wt[8];
            if constexpr (VPT > 2) {   // unpacked again: kept, the values of the first pass would fill the registers
                asm volatile("" : "+v"(vh[i].x), "+v"(vh[i].y), "+v"(vh[i].z), "+v"(vh[i].w));
                asm volatile("" : "+v"(vd[i].x), "+v"(vd[i].y), "+v"(vd[i].z), "+v"(vd[i].w));
            }
            unpack8(vh[i], h);
            unpack8(vd[i], d);
            unpack8(vr[i], e);
            if constexpr (!AHEAD) weights(i, wt);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = (float)((double)h[j] * rd);
                dw[i][j] = fmaf(d[j], x, dw[i][j]);
                const float g = r * (d[j] * (AHEAD ? wk[AHEAD ? i : 0][j] : wt[j]) - x * m);
                e[j] = a.dh ? g + e[j] : g;
            }
            if (v < nv) st16<ST>(a.dx + t * a.H + v * 8, pack8(e));
            if constexpr (VPT > 2) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (a.dw) {
        if constexpr (RPB > 1) {   // the waves' sums, in order
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s_dw[rw][(sub + i * G) * 8 + j] = dw[i][j];
            __syncthreads();
            if (rw) return;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int w = 1; w < RPB; ++w) dw[i][j] += s_dw[w][(sub + i * G) * 8 + j];
                }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            if (v < nv) {
                float* p = a.part + (int64_t)blockIdx.x * a.H + v * 8;
                *reinterpret_cast<float4*>(p) = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
            }
        }
    }
}

// dweight[c] = sum of the partial rows: 32 columns per workgroup as 8 vectors of 4, 32 row groups, whose
// sums are then added in order through LDS.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ part, int np, int H, float* __restrict__ dw) {
    __shared__ __align__(16) float s[32][32];
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3, col = blockIdx.x * 32 + 4 * c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < H) {   // (H is a multiple of 8)
#pragma unroll 16
        for (int p = g; p < np; p += 32) {
            const float4 x = *reinterpret_cast<const float4*>(part + (int64_t)p * H + col);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
        }
    }
    *reinterpret_cast<float4*>(&s[g][4 * c]) = v;
    __syncthreads();
    const int o = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x < 32 && o < H) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
        dw[o] = t;
    }
}

template <int G, int VPT>
static void run_norm_bwd(const NormBwdArgs& a, int grid, hipStream_t st) {
    if (streamed(a.T, a.H)) hipLaunchKernelGGL((k_add_rmsnorm_bwd<G, VPT, true>), dim3(grid), dim3(G < 256 ? 256 : G), 0, st, a);
    else hipLaunchKernelGGL((k_add_rmsnorm_bwd<G, VPT, false>), dim3(grid), dim3(G < 256 ? 256 : G), 0, st, a);
}

hipError_t launch_add_rmsnorm_backward(const NormBwdArgs& args, hipStream_t st) {
    NormBwdArgs a = args;
    const int nv = a.H / 8, grid = norm_bwd_parts(a.T, a.H);
    const bool one = grid == 1 && !(reinterpret_cast<uintptr_t>(a.dw) & 15);   // the only part is the sum
    if (one) a.part = a.dw;
    if (nv <= 64) run_norm_bwd<64, 1>(a, grid, st);
    else if (nv <= 128) run_norm_bwd<64, 2>(a, grid, st);
    else if (nv <= 256) run_norm_bwd<256, 1>(a, grid, st);
    else if (nv <= 512) run_norm_bwd<512, 1>(a, grid, st);
    else if (nv <= 1024) run_norm_bwd<512, 2>(a, grid, st);
    else if (nv <= 2048) run_norm_bwd<512, 4>(a, grid, st);
    else run_norm_bwd<512, 8>(a, grid, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dw || one) return e;
    hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)ceil_div(a.H, 32)), dim3(256), 0, st, a.part, grid, a.H, a.dw);
    return hipGetLastError();
}

}  // namespace moe
