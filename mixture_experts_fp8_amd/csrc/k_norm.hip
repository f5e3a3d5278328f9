// Residual addition + RMS norm or layer norm with E4M3 codes, and their backward passes (gfx950).
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

// The same for two sums in one exchange.
template <int G>
__device__ __forceinline__ void row_sums(double& v, double& u, double* s, double* t) {
    v = wave_sum(v);
    u = wave_sum(u);
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) {
            s[threadIdx.x >> 6] = v;
            t[threadIdx.x >> 6] = u;
        }
        __syncthreads();
        v = u = 0.0;
#pragma unroll
        for (int i = 0; i < G / 64; ++i) {
            v += s[i];
            u += t[i];
        }
    }
}

// 1 / sqrt(x) to double precision: the instruction's estimate (about 2^-26 off) and one Newton step,
// which would make NaN of the infinity and the zero that the ends of the range give.
__device__ __forceinline__ double rsqrt_f64(double x) {
    const double r = __builtin_amdgcn_rsq(x);
    const double n = r * fma(-0.5 * x * r, r, 1.5);
    return x > 0.0 && x < __builtin_inf() ? n : r;
}

// Doubles as floats that round to the same bf16.  A float beside the double does, unless it lands on the middle
// of two bf16 values (one in 2^16 does) and the double does not: then the next float towards the double.
// Infinities (of an infinite weight) and NaN are no such middle.
__device__ __forceinline__ void round_towards(const double (&d)[8], float (&f)[8]) {
    bool middle = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        f[j] = (float)d[j];
        middle |= (__float_as_uint(f[j]) & 0xFFFFu) == 0x8000u;
    }
    if (middle) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = __float_as_uint(f[j]);
            const double r = d[j] - (double)f[j];
            if ((u & 0xFFFFu) == 0x8000u && (r < 0.0 || r > 0.0)) f[j] = __uint_as_float((r > 0.0) == (d[j] > 0.0) ? u + 1 : u - 1);
        }
    }
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
//
// LN: layer norm, y = (h - m) r w + b with r = 1 / sqrt(mean((h - m)^2) + eps).  Both sums in one exchange:
// of d = h - h[0] and of d^2, in double, from which m - h[0] = mean(d) and the variance mean(d^2) - mean(d)^2
// follow.  The shift by a value of the row itself keeps them from cancelling: the two terms differ by a factor
// of at most H, and a constant row's variance is 0.
template <int G, int VPT, bool ST, bool LN>
__device__ __forceinline__ void add_norm(const NormArgs& a) {
    constexpr int RPB = G == 64 ? 4 : 1;
    __shared__ double s_sum[LN ? 2 : 1][G / 64];
    const int sub = threadIdx.x % G, nv = a.H >> 3;
    const int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / G;
    if (RPB > 1 && t >= a.T) return;   // (RPB > 1 only with G = 64: no barrier follows)
    const uint16_t* xr = a.x + t * a.ldx;
    const uint16_t* rr = a.res ? a.res + t * a.ldr : nullptr;
    uint4 vx[VPT], vr[VPT];
    auto load_bias = [&](int v, float4& lo, float4& hi) __attribute__((always_inline)) {
        lo = hi = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.b && v < nv) {
            lo = *reinterpret_cast<const float4*>(a.b + v * 8);
            hi = *reinterpret_cast<const float4*>(a.b + v * 8 + 4);
        }
    };
    // Weight and bias before the sums, where the registers hold them (4096 x 7168: 62 us, the bias behind them 68).
    constexpr bool EARLY = LN && G < 1024, EARLY_W = !LN || G * VPT < 4096;
    float4 w0[VPT], w1[VPT], b0[EARLY ? VPT : 1], b1[EARLY ? VPT : 1];
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
    auto load_weight = [&](int i) __attribute__((always_inline)) {
        const int v = sub + i * G;
        if (v < nv) {
            w0[i] = *reinterpret_cast<const float4*>(a.w + v * 8);
            w1[i] = *reinterpret_cast<const float4*>(a.w + v * 8 + 4);
        }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (EARLY_W) load_weight(i);
        if constexpr (EARLY) load_bias(sub + i * G, b0[i], b1[i]);
    }
    double ss = 0.0, sd = 0.0, h0 = 0.0;
    if constexpr (LN) {   // h[0]
        float f = bf16_to_f32(xr[0]);
        if (rr) f = bf16_to_f32(pack_bf16(f + bf16_to_f32(rr[0]), 0.f) & 0xFFFFu);
        h0 = (double)f;
    }
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
        if constexpr (LN) {
            if (sub + i * G < nv) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const double d = (double)f[j] - h0;
                    sd += d;
                    ss = fma(d, d, ss);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fma((double)f[j], (double)f[j], ss);
        }
    }
    const auto put_h = [&]() __attribute__((always_inline)) {
        if (!a.h) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            if (v < nv) st16<ST>(a.h + t * a.H + v * 8, vx[i]);
        }
    };
    if (!LN || (!a.y && !a.yq)) put_h();
    if (!a.y && !a.yq) return;   // (uniform)
    double r, mean = 0.0;
    if constexpr (LN) {
        row_sums<G>(ss, sd, s_sum[0], s_sum[1]);
        put_h();   // behind the exchange: h may be x or residual, and every wave has read its first column by now
        const double m = sd * a.inv_h;
        r = rsqrt_f64(fma(-m, m, ss * a.inv_h) + (double)a.eps);
        mean = h0 + m;
    } else {
        r = rsqrt_f64(fma(row_sum<G>(ss, s_sum[0]), a.inv_h, (double)a.eps));
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = sub + i * G;
        float f[8];
        unpack8(vx[i], f);
        if constexpr (!EARLY_W) load_weight(i);
        const float w[8] = {w0[i].x, w0[i].y, w0[i].z, w0[i].w, w1[i].x, w1[i].y, w1[i].z, w1[i].w};
        float b[8] = {};
        double d[8];
        if constexpr (LN) {
            float4 lo, hi;
            if constexpr (EARLY) lo = b0[i], hi = b1[i];
            else load_bias(v, lo, hi);
            b[0] = lo.x, b[1] = lo.y, b[2] = lo.z, b[3] = lo.w, b[4] = hi.x, b[5] = hi.y, b[6] = hi.z, b[7] = hi.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (LN) d[j] = fma(((double)f[j] - mean) * r, (double)w[j], (double)b[j]);
            else d[j] = (double)f[j] * r * (double)w[j];
        }
        round_towards(d, f);
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

template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G == 64 ? 256 : G) void k_add_rmsnorm(NormArgs a) {
    add_norm<G, VPT, ST, false>(a);
}
template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G == 64 ? 256 : G) void k_add_layernorm(NormArgs a) {
    add_norm<G, VPT, ST, true>(a);
}

template <int G, int VPT, bool LN>
static void run_norm(const NormArgs& args, hipStream_t st) {
    constexpr int RPB = G == 64 ? 4 : 1;
    const dim3 block(G == 64 ? 256 : G);
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
        const bool far = streamed(args.T, args.H);
        if constexpr (LN) {
            if (far) hipLaunchKernelGGL((k_add_layernorm<G, VPT, true>), grid, block, 0, st, a);
            else hipLaunchKernelGGL((k_add_layernorm<G, VPT, false>), grid, block, 0, st, a);
        } else {
            if (far) hipLaunchKernelGGL((k_add_rmsnorm<G, VPT, true>), grid, block, 0, st, a);
            else hipLaunchKernelGGL((k_add_rmsnorm<G, VPT, false>), grid, block, 0, st, a);
        }
    }
}

template <bool LN>
static hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
    const int nv = a.H / 8;
    if (nv <= 64) run_norm<64, 1, LN>(a, st);
    else if (nv <= 256) run_norm<256, 1, LN>(a, st);
    else if (nv <= 512) run_norm<512, 1, LN>(a, st);
    else if (nv <= 1024) run_norm<512, 2, LN>(a, st);   // (with one vector each, 1024 threads are 2% slower at 4096 x 7168)
    else if (nv <= 2048) run_norm<1024, 2, LN>(a, st);
    else run_norm<1024, 4, LN>(a, st);
    return hipGetLastError();
}
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t st) { return launch_norm<false>(a, st); }
hipError_t launch_add_layernorm(const NormArgs& a, hipStream_t st) { return launch_norm<true>(a, st); }

// ----------------------------------------------------------------------------------------
// Backward.  With xhat = h r and g = dy w:  dx = r (g - xhat mean(g xhat)) + dh, and the weight
// gradient sum_t dy xhat.  A workgroup of G threads (short rows: four waves with a row each) walks rows
// a grid apart, keeps its share of the weight gradient in registers; the workgroups' sums go to `part`
// and are added in workgroup order by k_norm_dw.  The two sums and xhat are formed in double, as the
// forward's: their squares would leave float32 at |h| of 1e19 and 1e-19.  Bound by HBM: 16384 x 4096 with
// dh 90 us, 6.0 TB/s of what it must move.  The next row is in flight over this one's sums, so long rows take
// more vectors per thread, not more threads: 512 threads have the registers for it (2048 x 16384: 61 us,
// 1024 threads 69, with spills).
//
// LN: xhat = (h - m) r and dx = r (g - mean(g) - xhat mean(g xhat)) + dh; the bias's gradient sum_t dy takes
// its place beside the weight's, in registers and in a second set of parts.  With d = h - h[0], in double as in the
// forward pass (float32 would keep 2^-24 of h[0], not of d, and has no difference of two values of 3e38), the four
// sums of d, d^2, g and g d need one exchange: sum g (h - m) = sum g d - mean(d) sum g.
template <int G, int VPT, bool ST, bool LN>
__device__ __forceinline__ void add_norm_bwd(const NormBwdArgs& a) {
    constexpr int RPB = G == 64 ? 4 : 1;
    constexpr bool AHEAD = VPT <= 4;   // else the registers hold no second row and no weights
    constexpr int NS = LN ? 4 : 2;
    __shared__ double s_sum[2][NS][G / 64];
    __shared__ __align__(16) float s_dw[RPB][RPB > 1 ? VPT * G * 8 : 4];
    // The bias's sums: in registers, or, where those do not hold them beside the rest, in LDS, each thread its own.
    constexpr bool DB_LDS = LN && VPT > 4;
    extern __shared__ __align__(16) float s_db[];   // [VPT][2][G] vectors of four
    float db[LN ? VPT : 1][8];
    if constexpr (LN) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) db[i][j] = 0.f;
    }
    auto db_slot = [&](int i, int h) __attribute__((always_inline)) { return reinterpret_cast<v4f*>(s_db) + (2 * i + h) * G + (threadIdx.x % G); };
    if constexpr (DB_LDS) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) *db_slot(i, 0) = *db_slot(i, 1) = v4f{0.f, 0.f, 0.f, 0.f};
    }
    const int sub = RPB > 1 ? threadIdx.x % G : threadIdx.x, rw = RPB > 1 ? threadIdx.x / G : 0, nv = a.H >> 3;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const bool tiny = a.eps < 0x1p-120f;
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
        double ss = 0.0, gh = 0.0, sd = 0.0, sg = 0.0;
        double h0 = 0.0;
        if constexpr (LN) h0 = (double)bf16_to_f32(a.h[t * a.H]);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float h[8], d[8], wt[8];
            unpack8(vh[i], h);
            unpack8(vd[i], d);
            if constexpr (!AHEAD) weights(i, wt);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (LN) {
                    // (no weight, and no gradient, behind the row's end: only d has to be left out there)
                    const double x = sub + i * G < nv ? (double)h[j] - h0 : 0.0;
                    const double g = (double)(d[j] * (AHEAD ? wk[AHEAD ? i : 0][j] : wt[j]));
                    sd += x;
                    sg += g;
                    ss = fma(x, x, ss);
                    gh = fma(g, x, gh);
                } else {
                    ss = fma((double)h[j], (double)h[j], ss);
                    gh = fma((double)(d[j] * (AHEAD ? wk[AHEAD ? i : 0][j] : wt[j])), (double)h[j], gh);
                }
            }
            if constexpr (VPT > 2) __builtin_amdgcn_sched_barrier(0);   // one vector's values at a time
        }
        ss = wave_sum(ss);
        gh = wave_sum(gh);
        if constexpr (LN) {
            sd = wave_sum(sd);
            sg = wave_sum(sg);
        }
        if constexpr (G > 64) {
            if ((sub & 63) == 0) {
                s_sum[par][0][sub >> 6] = ss;
                s_sum[par][1][sub >> 6] = gh;
                if constexpr (LN) {
                    s_sum[par][2][sub >> 6] = sd;
                    s_sum[par][3][sub >> 6] = sg;
                }
            }
            __syncthreads();
            ss = gh = sd = sg = 0.0;
#pragma unroll
            for (int i = 0; i < G / 64; ++i) {
                ss += s_sum[par][0][i];
                gh += s_sum[par][1][i];
                if constexpr (LN) {
                    sd += s_sum[par][2][i];
                    sg += s_sum[par][3][i];
                }
            }
        }
        double rd, mean = 0.0;   // LN: mean(h)
        float mg = 0.f;          // LN: mean(g)
        if constexpr (LN) {
            const double md = sd * a.inv_h;   // mean(d)
            mean = h0 + md;
            rd = rsqrt_f64(fma(-md, md, ss * a.inv_h) + (double)a.eps);
            mg = (float)(sg * a.inv_h);
            gh -= md * sg;
        } else {
            rd = rsqrt_f64(fma(ss, a.inv_h, (double)a.eps));
        }
        // r of a row of bf16's smallest steps passes float32 where eps is 0 or next to it: two factors then.  (One
        // multiplication more for every eps costs 3% at 4096 x 7168.)
        float far = 1.f;
        if (tiny) far = rd > 0x1p64 ? 0x1p64f : 1.f;
        const float r = (float)(tiny && rd > 0x1p64 ? rd * 0x1p-64 : rd), m = (float)(gh * a.inv_h * rd);   // m = mean(g xhat)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            float h[8], d[8], e[8], g[8], wt[8];
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
                const float x = LN ? (float)(((double)h[j] - mean) * rd) : (float)((double)h[j] * rd);
                dw[i][j] = fmaf(d[j], x, dw[i][j]);
                if constexpr (LN && !DB_LDS) db[i][j] += d[j];
                const float gw = d[j] * (AHEAD ? wk[AHEAD ? i : 0][j] : wt[j]);
                g[j] = r * ((LN ? gw - mg : gw) - x * m);
            }
            if (tiny) {
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] *= far;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = a.dh ? g[j] + e[j] : g[j];
            if constexpr (DB_LDS) {
                *db_slot(i, 0) += v4f{d[0], d[1], d[2], d[3]};
                *db_slot(i, 1) += v4f{d[4], d[5], d[6], d[7]};
            }
            if (v < nv) st16<ST>(a.dx + t * a.H + v * 8, pack8(e));
            if constexpr (VPT > 2) __builtin_amdgcn_sched_barrier(0);
        }
    }
    auto part = [&](float (&dw)[VPT][8], float* out) __attribute__((always_inline)) {
        if constexpr (RPB > 1) {   // the waves' sums, in order
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s_dw[rw][(sub + i * G) * 8 + j] = dw[i][j];
            __syncthreads();
            if (rw == 0) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
#pragma unroll
                        for (int w = 1; w < RPB; ++w) dw[i][j] += s_dw[w][(sub + i * G) * 8 + j];
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = sub + i * G;
            if (rw == 0 && v < nv) {
                float* p = out + (int64_t)blockIdx.x * a.H + v * 8;
                *reinterpret_cast<float4*>(p) = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
                *reinterpret_cast<float4*>(p + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
            }
        }
    };
    if (a.dw) part(dw, a.part);
    if constexpr (LN) {
        if constexpr (DB_LDS) {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) db[i][j] = (*db_slot(i, j / 4))[j % 4];
        }
        if (a.db) {
            if (RPB > 1 && a.dw) __syncthreads();   // s_dw has been read
            part(db, a.part_b);
        }
    }
}

template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G == 64 ? 256 : G) void k_add_rmsnorm_bwd(NormBwdArgs a) {
    add_norm_bwd<G, VPT, ST, false>(a);
}
template <int G, int VPT, bool ST>
__global__ __launch_bounds__(G == 64 ? 256 : G) void k_add_layernorm_bwd(NormBwdArgs a) {
    add_norm_bwd<G, VPT, ST, true>(a);
}

// dweight[c] = sum of the partial rows: 32 columns per workgroup as 8 vectors of 4, 32 row groups, whose
// sums are then added in order through LDS.  Workgroups (.., 1) sum a second set, the bias's.
__global__ __launch_bounds__(256) void k_norm_dw(const float* part, int np, int H, float* dw, const float* part1, float* dw1) {
    if (blockIdx.y) part = part1, dw = dw1;
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

template <auto Kern, size_t LDS>
static hipError_t run_layernorm_bwd(const NormBwdArgs& a, int grid, dim3 block, hipStream_t st) {
    if (const hipError_t e = ask_for_lds<Kern, LDS>(LDS); e != hipSuccess) return e;
    hipLaunchKernelGGL(Kern, dim3(grid), block, LDS, st, a);
    return hipGetLastError();
}
template <int G, int VPT, bool LN>
static hipError_t run_norm_bwd(const NormBwdArgs& a, int grid, hipStream_t st) {
    const dim3 block(G == 64 ? 256 : G);
    const bool far = streamed(a.T, a.H);
    if constexpr (LN) {
        constexpr size_t lds = VPT > 4 ? (size_t)VPT * G * 32 : 0;
        return far ? run_layernorm_bwd<k_add_layernorm_bwd<G, VPT, true>, lds>(a, grid, block, st)
                   : run_layernorm_bwd<k_add_layernorm_bwd<G, VPT, false>, lds>(a, grid, block, st);
    } else {
        if (far) hipLaunchKernelGGL((k_add_rmsnorm_bwd<G, VPT, true>), dim3(grid), block, 0, st, a);
        else hipLaunchKernelGGL((k_add_rmsnorm_bwd<G, VPT, false>), dim3(grid), block, 0, st, a);
        return hipGetLastError();
    }
}

template <bool LN>
static hipError_t launch_norm_backward(const NormBwdArgs& args, hipStream_t st) {
    NormBwdArgs a = args;
    const int nv = a.H / 8, grid = LN ? layernorm_bwd_parts(a.T, a.H) : norm_bwd_parts(a.T, a.H);
    const auto odd = [](const float* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
    const bool one = grid == 1 && !odd(a.dw) && !odd(a.db);   // the only part is the sum
    if (one) a.part = a.dw, a.part_b = a.db;
    hipError_t e;
    if (nv <= 64) e = run_norm_bwd<64, 1, LN>(a, grid, st);
    else if (nv <= 128) e = run_norm_bwd<64, 2, LN>(a, grid, st);
    else if (nv <= 256) e = run_norm_bwd<LN ? 128 : 256, LN ? 2 : 1, LN>(a, grid, st);
    else if (nv <= 512) e = run_norm_bwd<LN ? 256 : 512, LN ? 2 : 1, LN>(a, grid, st);
    else if (nv <= 1024) e = run_norm_bwd<512, 2, LN>(a, grid, st);
    else if (nv <= 2048) e = run_norm_bwd<512, 4, LN>(a, grid, st);
    else e = run_norm_bwd<512, 8, LN>(a, grid, st);
    if (e != hipSuccess || (!a.dw && !a.db) || one) return e;
    const float* first = a.dw ? a.part : a.part_b;
    hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)ceil_div(a.H, 32), a.dw && a.db ? 2 : 1), dim3(256), 0, st, first, grid, a.H,
                       a.dw ? a.dw : a.db, a.part_b, a.db);
    return hipGetLastError();
}
hipError_t launch_column_sums(const float* part, int np, int n, float* out, hipStream_t st) {
    hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)ceil_div(n, 32)), dim3(256), 0, st, part, np, n, out, nullptr, nullptr);
    return hipGetLastError();
}
hipError_t launch_add_rmsnorm_backward(const NormBwdArgs& a, hipStream_t st) { return launch_norm_backward<false>(a, st); }
hipError_t launch_add_layernorm_backward(const NormBwdArgs& a, hipStream_t st) { return launch_norm_backward<true>(a, st); }

}  // namespace moe
