// Backward pass of the gated block (gfx950): from dh and the kept sums g, u,
//   dgu = bf16([dh u act'(g) | dh act(g)]),  dx = dgu @ W^T,  dW = x^T @ dgu,  dbias = column sums.
// The two products run in bf16 on the kernels of linear_tiles.h, whose operands are brought into its layouts
// first: rows with the summed index contiguous, and fragments of 16 columns.  E4M3 values times a power of
// two are bf16 values, so those operands lose nothing (but beyond bf16's range, which scales of 2^-124 and
// below or 2^120 and above can reach).
#include "linear_tiles.h"

namespace moe {

namespace {

// 1 / (1 + exp(-v)) and its complement q = 1 - p.  With u = 2^-24 and the base-2 instruction's own error of up to 2 u
// (1.4 u was the most seen): p is within 5 u of its value (its exponential's 3 u, where they count in full, 1 + e and
// the last step of the reciprocal 1 u each) and q within 6 u (the product 1 u more), where those are 2^-126 or more.
// Over all bf16 arguments the most seen was 2.1 and 2.7 u, over 4 million floats 3.3 and 4.0 u.  Below 2^-126,
// where 1 + e is 1e38 or more, p has no Newton step and ends as 0.  act_fn's argument of the instruction is |v| u off
// and its reciprocal 2 u; a gradient that is rounded to bf16 and then summed shows that in the values beside the middle
// of two, so both are mended here: by the rest of the argument's product, and by one Newton step.
struct Logistic {
    float p, q;
};
__device__ __forceinline__ Logistic logistic(float v) {
    const float c = fminf(fmaxf(v, -100.f), 100.f);       // exp(100) is infinite, exp(-100) counts as 0
    const float t = c * -1.44269502f;
    float lo = fmaf(c, -1.44269502f, -t);
    lo = fmaf(c, -1.92596303e-8f, lo);                    // log2(e) = 1.44269502 + 1.92596303e-8
    float e = __builtin_amdgcn_exp2f(t);
    e = e < 3e38f ? fmaf(e * lo, 0.693147182f, e) : e;
    const float d = 1.0f + e;
    float p = __builtin_amdgcn_rcpf(d);
    if (d < 1e38f) p = fmaf(fmaf(-d, p, 1.0f), p, p);
    return {v != v ? v : p, v < 0.f ? 1.0f - p : e * p};
}

// act(v) and its slope; the same functions as act_fn, and without cancellation where one of the two
// factors of a logistic is small.
struct Act {
    float a, s;
};
template <int ACT>
__device__ __forceinline__ Act act_slope(float v) {
    if constexpr (ACT == MOE_ACT_RELU) return {v < 0.f ? 0.f : v, v > 0.f ? 1.f : 0.f};
    if constexpr (ACT == MOE_ACT_SILU) {
        const Logistic l = logistic(v);
        const float a = v * l.p;
        return {a, fmaf(a, l.q, l.p)};
    }
    if constexpr (ACT == MOE_ACT_GELU) {
        const float c = normal_cdf(v), d = __builtin_amdgcn_exp2f(v * v * -0.72134752f);   // exp(-v^2 / 2)
        return {v * c, fmaf(v * 0.398942280f, d, c)};
    }
    if constexpr (ACT == MOE_ACT_GELU_TANH) {
        const float w = v * v, u = 1.59576912f * fmaf(0.044715f * w, v, v);   // twice tanh's argument
        const Logistic l = logistic(u);
        const float q = l.q * l.p;
        // (from |v| of 1e12 on the last factors would leave float32; q is 0 long before)
        return {v * l.p, q == 0.f ? l.p : fmaf(v * q, 1.59576912f * fmaf(0.134145f, w, 1.0f), l.p)};
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

// The 8 rows' bf16 values of column c.
template <int W>
__device__ __forceinline__ v4u_t column_of(const uint32_t (&r)[8][W], int c) {
    v4u_t v;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        v[p] = c % 2 ? high_halves(r[2 * p][c / 2], r[2 * p + 1][c / 2]) : low_halves(r[2 * p][c / 2], r[2 * p + 1][c / 2]);
    return v;
}
// 2 W bf16 values (W 2 or 4) from and to memory, and as floats.
template <int W>
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t (&r)[W]) {
    typedef uint32_t vec __attribute__((ext_vector_type(W)));
    const vec v = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = v[i];
}
template <int W>
__device__ __forceinline__ void store_words(uint16_t* p, const uint32_t (&r)[W]) {
    typedef uint32_t vec __attribute__((ext_vector_type(W)));
    vec v;
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = r[i];
    *reinterpret_cast<vec*>(p) = v;
}
template <int W>
__device__ __forceinline__ void unpack_words(const uint32_t (&r)[W], float (&f)[2 * W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        f[2 * i] = __uint_as_float(r[i] << 16);
        f[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
}

struct DguArgs {
    int T, I, NT, parts;    // blocks of 64 rows; block b is of part b % parts
    const uint16_t* dh;
    const uint16_t* gu;
    uint16_t* dgu;
    uint8_t* packed;        // or NULL: dgu as column fragments whose K is the row, rows past T 0
    float* part;            // or NULL: [parts][2I] column sums
};

// A wave takes 8 CW columns of g and u and blocks of 64 rows, `parts` apart; lane (t = l / 8, c = l % 8) the rows
// 8 t .. +7 and CW columns from CW c of a block, all loads of which are in flight together.  Column sums stay in
// registers.  The fragments of the transposed result go through LDS, so that they leave in whole kilobytes;
// slots are swizzled by t, which spreads the lanes' 16-byte writes over the banks.  CW 8, or 4 where that leaves SIMDs
// without a wave: a lane's 64 activations are one chain (the whole call at 512 x 2048 x 1024: 29.0 us, 32.5 with 8;
// 4096 x 7168 x 2048: 419 with 4, 411 with 8).
template <int ACT, bool PACK, int CW>
__device__ __forceinline__ void gated_dgu(const DguArgs& a, int unit, uint8_t* smem) {
    constexpr int W = CW / 2, WAVE = 8 * CW, FR = WAVE / 16;   // words of a lane's row; columns, fragments of a wave
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = (unit / a.parts * 4 + wv) * WAVE, first = unit % a.parts;
    const int t8 = lane >> 3, c8 = lane & 7, col = cols + CW * c8;
    const bool on = col < a.I;
    if (cols >= a.I) return;   // (uniform; no barrier follows)
    const int64_t N = 2 * (int64_t)a.I;
    float sg[CW] = {}, su[CW] = {};
    for (int b = first; b < a.NT; b += a.parts) {
        uint32_t g[8][W] = {}, u[8][W] = {}, d[8][W] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = (int64_t)b * 64 + 8 * t8 + i;
            if (on && t < a.T) {
                load_words<W>(a.gu + t * N + col, g[i]);
                load_words<W>(a.gu + t * N + a.I + col, u[i]);
                load_words<W>(a.dh + t * a.I + col, d[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t t = (int64_t)b * 64 + 8 * t8 + i;
            float x[CW], y[CW], z[CW];
            unpack_words<W>(g[i], x);
            unpack_words<W>(u[i], y);
            unpack_words<W>(d[i], z);
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                const Act f = act_slope<ACT>(x[j]);
                // (dh u beyond float32 comes back where the slope is small; dh is then above 1, and dh act' does not vanish)
                const float zy = z[j] * y[j];
                x[j] = fabsf(zy) < __builtin_inff() ? zy * f.s : z[j] * f.s * y[j];
                y[j] = z[j] * f.a;
                if (t >= a.T) x[j] = y[j] = 0.f;
                sg[j] += x[j];
                su[j] += y[j];
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                g[i][j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                u[i][j] = pack_bf16(y[2 * j], y[2 * j + 1]);
            }
            if (on && t < a.T) {
                store_words<W>(a.dgu + t * N + col, g[i]);
                store_words<W>(a.dgu + t * N + a.I + col, u[i]);
            }
        }
        if constexpr (PACK) {
            v4u_t* s = reinterpret_cast<v4u_t*>(smem + wv * FR * kFragBytes);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    const int q = CW * c8 + c;   // column of the wave
                    s[(q >> 4) * 128 + t8 * 16 + ((q & 15) ^ t8)] = column_of<W>(half ? u : g, c);
                }
                asm volatile("" ::: "memory");   // (a wave's LDS accesses stay in order)
                __builtin_amdgcn_wave_barrier();
                const int n0 = ((half ? a.I : 0) + cols) / 16;
#pragma unroll
                for (int q = 0; q < 2 * FR; ++q) {    // fragment q / 2, its lower and upper kilobyte
                    const int p = (q & 1) * 64 + lane, r = p >> 4;
                    const v4u_t v = s[(q >> 1) * 128 + r * 16 + ((p & 15) ^ r)];
                    if (cols + 16 * (q >> 1) < a.I)
                        *reinterpret_cast<v4u_t*>(a.packed + ((int64_t)(n0 + (q >> 1)) * a.NT + b) * kFragBytes + p * 16) = v;
                }
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
    if (a.part) {   // over the lanes of a column, then one row of the parts
#pragma unroll
        for (int j = 0; j < CW; ++j) {
#pragma unroll
            for (int m = 8; m < 64; m *= 2) {
                sg[j] += __shfl_xor(sg[j], m);
                su[j] += __shfl_xor(su[j], m);
            }
        }
        if (t8 == 0 && on) {
            float* p = a.part + (int64_t)first * N + col;
#pragma unroll
            for (int j = 0; j < CW; ++j) p[j] = sg[j], p[a.I + j] = su[j];
        }
    }
}

// x^T as bf16 [K][64 NT], 0 behind row T.  A wave takes 64 rows and 64 columns, a lane 8 x 8 of them; its
// 16-byte vectors of 8 rows make 128 bytes of a row of the result.
template <bool MX>
__device__ __forceinline__ void rows_transposed(const uint8_t* xq, const uint8_t* xs, int T, int K, int NT, uint16_t* xt, int unit) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t0 = unit % NT * 64 + 8 * (lane & 7), k0 = (unit / NT * 4 + wv) * 64 + 8 * (lane >> 3);
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
    uint32_t r[8][4];
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
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = t0 + i < T ? pack_bf16(v[2 * j], v[2 * j + 1]) : 0;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<v4u_t*>(xt + (int64_t)(k0 + c) * (NT * 64) + t0) = column_of<4>(r, c);
}

// The packed FP8 weights [K][N] as bf16 fragments of 16 rows of w whose K is the column: a workgroup turns 4
// fragments of 16 columns x 128 rows into 8 of 16 rows x 64 columns.
template <bool MX>
__device__ __forceinline__ void weights_transposed(const uint8_t* w, const uint8_t* ws, int K, int N, uint8_t* out, int unit,
                                                   uint8_t* s_w) {
    uint8_t* s_s = s_w + 4 * kFragBytes;
    const int tid = threadIdx.x, KB = K / kGroup, NJ = N / 64, jb = unit % NJ, kb = unit / NJ;
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

// The operands of both products in one launch: workgroups of dgu, of x^T and of the weights.  (One after the other
// the three took 13.3, 4.6 and 4.2 us at 2047 x 768 x 1152, where neither fills the chip.)
struct PrepareArgs {
    DguArgs d;
    int K, dgu_units, row_units;          // workgroups of each, the rest the weights'
    const uint8_t *xq, *xs, *w, *ws;
    uint16_t* xt;
    uint8_t* wt;
};
template <int ACT, bool MX, bool PACK, int CW>
__global__ __launch_bounds__(256) void k_gated_prepare(PrepareArgs a) {
    __shared__ __align__(16) uint8_t smem[PACK ? 2 * CW * kFragBytes : 4 * kFragBytes + 256];   // (CW 4: 16 KB, enough for both)
    int unit = blockIdx.x;
    if (unit < a.dgu_units) return gated_dgu<ACT, PACK, CW>(a.d, unit, smem);
    unit -= a.dgu_units;
    if (unit < a.row_units) return rows_transposed<MX>(a.xq, a.xs, a.d.T, a.K, a.d.NT, a.xt, unit);
    weights_transposed<MX>(a.w, a.ws, a.K, 2 * a.d.I, a.wt, unit - a.row_units, smem);
}

template <int ACT, int CW>
void run_prepare_cw(PrepareArgs& a, bool mx, unsigned rest, hipStream_t st) {
    a.dgu_units = a.d.parts * (int)ceil_div(a.d.I, 32 * CW);
    const dim3 grid(a.dgu_units + rest);
    if (a.xt) {
        if (mx) hipLaunchKernelGGL((k_gated_prepare<ACT, true, true, CW>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_gated_prepare<ACT, false, true, CW>), grid, dim3(256), 0, st, a);
    } else {
        if (mx) hipLaunchKernelGGL((k_gated_prepare<ACT, true, false, CW>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((k_gated_prepare<ACT, false, false, CW>), grid, dim3(256), 0, st, a);
    }
}
template <int ACT>
void run_prepare(PrepareArgs& a, bool mx, unsigned rest, hipStream_t st) {
    if (a.d.parts * ceil_div(a.d.I, 64) < 1024) run_prepare_cw<ACT, 4>(a, mx, rest, st);
    else run_prepare_cw<ACT, 8>(a, mx, rest, st);
}

// Both products in one launch: workgroups [0, first_units) compute the tiles of p[0], the next ones those of p[1], the
// last ones the bias's gradient from its parts.  One launch fills the chip where either product alone leaves it half
// empty, and has one last round.
struct ProductsArgs {
    LinArgs p[2];
    int tm[2], tn[2];
    int units[2], parts[2], per[2];   // workgroups of a part, parts of the sum (0: not asked for), K blocks of one
    float* join[2];              // more than one part: [parts][rows][columns]
    const float* sums;           // the bias's parts, [sum_parts][n]
    int sum_parts, n;
    float* dbias;
};
// 32 columns of the parts' sum, as k_norm_dw adds them.
__device__ __forceinline__ void column_sums(const float* part, int np, int n, float* out, int unit, float* s) {
    const int c = threadIdx.x & 7, g = threadIdx.x >> 3, col = unit * 32 + 4 * c;   // (256 threads, or the first 256)
    if (g < 32) {
        v4f v = {0.f, 0.f, 0.f, 0.f};
        if (col < n) {
#pragma unroll 8
            for (int p = g; p < np; p += 32) v += *reinterpret_cast<const v4f*>(part + (int64_t)p * n + col);
        }
        *reinterpret_cast<v4f*>(s + g * 32 + 4 * c) = v;
    }
    __syncthreads();
    const int o = unit * 32 + threadIdx.x;
    if (threadIdx.x < 32 && o < n) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i * 32 + threadIdx.x];
        out[o] = t;
    }
}
template <int MI, int WM, int WN, int S, int KS, bool TILE>
__global__ __launch_bounds__(64 * WM * WN * KS, TILE ? 2 : 1) void k_gated_products(ProductsArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    int unit = blockIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (unit < a.units[i] * a.parts[i]) {
            LinArgs l = a.p[i];
            const int KB = l.K / kGroup;
            Blocks b{0, KB};
            if (a.parts[i] > 1) {
                int z = 0;   // (few parts: no division)
                while (unit >= a.units[i]) unit -= a.units[i], ++z;
                b = {z * a.per[i], min(a.per[i], KB - z * a.per[i])};   // (no part is empty: product_plan)
                l.y = a.join[i] + (int64_t)z * l.T * l.N;
                l.ldy = l.N, l.out_bf16 = 0;
            }
            if constexpr (TILE) return linear_tile<kBf16, false, MI, 4, WM, WN>(l, unit, a.tm[i], a.tn[i], b);
            else return linear_deep<kBf16, false, MI, 4, WM, WN, S, KS>(l, unit, a.tm[i], a.tn[i], b);
        }
        unit -= a.units[i] * a.parts[i];
    }
    column_sums(a.sums, a.sum_parts, a.n, a.dbias, unit, reinterpret_cast<float*>(smem));
}

// The sum of a product's parts, eight values per thread.
struct JoinArgs {
    const float* join[2];
    void* y[2];
    int parts[2], bf16[2];
    int64_t n[2];            // values; 0: not in parts
};
__global__ __launch_bounds__(256) void k_gated_join(JoinArgs a) {
    int64_t v = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    int i = 0;
    if (v >= a.n[0]) v -= a.n[0], i = 1;
    if (v >= a.n[i]) return;
    v4f s[2] = {};
#pragma unroll 4
    for (int z = 0; z < a.parts[i]; ++z) {
        const v4f* p = reinterpret_cast<const v4f*>(a.join[i] + z * a.n[i] + v);
        s[0] += p[0];
        s[1] += p[1];
    }
    if (a.bf16[i]) {
        const float f[8] = {s[0][0], s[0][1], s[0][2], s[0][3], s[1][0], s[1][1], s[1][2], s[1][3]};
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y[i]) + v) = pack8(f);
    } else {
        v4f* d = reinterpret_cast<v4f*>(static_cast<float*>(a.y[i]) + v);
        d[0] = s[0];
        d[1] = s[1];
    }
}

template <int MI, int WM, int WN, int S, int KS, bool TILE>
hipError_t run_products(ProductsArgs a, int bias_units, hipStream_t st) {
    constexpr int ROWS = 16 * MI * WM, COLS = 64 * WN;
    unsigned grid = bias_units;
    for (int i = 0; i < 2; ++i) {
        if (!a.parts[i]) continue;
        a.tm[i] = (int)ceil_div(a.p[i].T, ROWS);
        a.tn[i] = (int)ceil_div(a.p[i].N, COLS);
        a.units[i] = (int)(ceil_div((int64_t)a.tm[i] * a.tn[i], 8) * 8);
        a.per[i] = (int)ceil_div(a.p[i].K / kGroup, a.parts[i]);
        grid += a.units[i] * a.parts[i];
    }
    constexpr size_t lds = TILE ? 3 * ROWS * kGroup + scales_lds<kBf16, false>(ROWS, COLS, 0, 0) : deep_lds<kBf16, false>(ROWS, COLS, KS * S, 1);
    if (const hipError_t e = ask_for_lds<k_gated_products<MI, WM, WN, S, KS, TILE>>(lds); e != hipSuccess) return e;
    hipLaunchKernelGGL((k_gated_products<MI, WM, WN, S, KS, TILE>), dim3(grid), dim3(64 * WM * WN * KS), lds, st, a);
    return hipGetLastError();
}

hipError_t launch_products(const ProductsArgs& a, int tile, int bias_units, hipStream_t st) {
    switch (tile) {   // (product_plan's table)
        case 0: return run_products<1, 4, 1, 4, 2, false>(a, bias_units, st);
        case 1: return run_products<2, 2, 2, 4, 1, false>(a, bias_units, st);
        case 2: return run_products<2, 2, 2, 3, 1, false>(a, bias_units, st);
        case 3: return run_products<4, 2, 4, 3, 1, false>(a, bias_units, st);
        default: return run_products<8, 1, 4, 1, 1, true>(a, bias_units, st);
    }
}

}  // namespace

hipError_t launch_gated_backward(const GatedBwdArgs& a, hipStream_t st) {
    const GatedBwdPlan p = gated_bwd_plan(a.T, a.K, a.I, a.dx != nullptr, a.dw != nullptr, a.dbias != nullptr);
    const int N = 2 * a.I, NT = p.row_blocks;
    uint8_t* ws = a.ws;
    float* part = a.dbias ? reinterpret_cast<float*>(ws + p.part) : nullptr;
    PrepareArgs r{{a.T, a.I, NT, a.dbias ? p.parts : NT, a.dh, a.gu, a.dgu, a.dw ? ws + p.dgu_packed : nullptr, part},
                  a.K, 0, 0, a.xq, a.xs, a.w, a.wsc, a.dw ? reinterpret_cast<uint16_t*>(ws + p.rows) : nullptr,
                  a.dx ? ws + p.weights : nullptr};
    r.row_units = a.dw ? NT * (int)ceil_div(a.K, 256) : 0;
    const unsigned rest = r.row_units + (a.dx ? N / 64 * (a.K / kGroup) : 0);
    switch (a.act) {
        case MOE_ACT_RELU: run_prepare<MOE_ACT_RELU>(r, a.mx, rest, st); break;
        case MOE_ACT_SILU: run_prepare<MOE_ACT_SILU>(r, a.mx, rest, st); break;
        case MOE_ACT_GELU: run_prepare<MOE_ACT_GELU>(r, a.mx, rest, st); break;
        case MOE_ACT_GELU_TANH: run_prepare<MOE_ACT_GELU_TANH>(r, a.mx, rest, st); break;
        default: run_prepare<MOE_ACT_NONE>(r, a.mx, rest, st);
    }
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (!a.dx && !a.dw) return a.dbias ? launch_column_sums(part, p.parts, N, a.dbias, st) : hipSuccess;
    ProductsArgs q{};
    const int kw = p.product.first;   // the product with the longer sums first
    LinArgs &dw = q.p[kw], &dx = q.p[!kw];
    dx.T = a.T, dx.K = 2 * N, dx.N = a.K;
    dx.xq = reinterpret_cast<const uint8_t*>(a.dgu), dx.w = ws + p.weights;
    dx.y = a.dx, dx.ldy = a.K, dx.out_bf16 = 1, dx.nt = (int64_t)a.T * a.K * 2 >= (32 << 20);
    dw.T = a.K, dw.K = 128 * NT, dw.N = N;
    dw.xq = ws + p.rows, dw.w = ws + p.dgu_packed;
    dw.y = a.dw, dw.ldy = N, dw.out_bf16 = a.dw_bf16, dw.nt = (int64_t)a.K * N * (a.dw_bf16 ? 2 : 4) >= (32 << 20);
    JoinArgs j{};
    int64_t joined = 0;
    for (int i = 0; i < 2; ++i) {
        const int which = i == kw ? 1 : 0;   // the plan's order: dx, dw
        q.parts[i] = p.product.parts[which];
        if (q.parts[i] < 2) continue;
        q.join[i] = reinterpret_cast<float*>(ws + p.join[which]);
        q.p[i].nt = 0;                       // read again at once
        j.join[i] = q.join[i], j.y[i] = q.p[i].y, j.parts[i] = q.parts[i], j.bf16[i] = q.p[i].out_bf16;
        j.n[i] = (int64_t)q.p[i].T * q.p[i].N;
        joined += j.n[i];
    }
    q.n = N, q.sums = part, q.sum_parts = p.parts, q.dbias = a.dbias;
    if (const hipError_t e = launch_products(q, p.product.tile, a.dbias ? (int)ceil_div(N, 32) : 0, st); e != hipSuccess || !joined) return e;
    hipLaunchKernelGGL(k_gated_join, dim3((unsigned)ceil_div(joined, 2048)), dim3(256), 0, st, j);
    return hipGetLastError();
}

}  // namespace moe
