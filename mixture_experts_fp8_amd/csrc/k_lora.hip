// Low-rank adapters of many requests beside a shared projection (gfx950):
//   y[t] = residual[t] + scale[a] (x[t] A_a^T) B_a^T,  a the adapter of the row's sequence.
//
// Two launches.  k_lora_down forms v = x A^T, float32 [parts][T][R up to 16], k_lora_up adds v B^T to the
// residual.  Both work on slots: the rows of one sequence inside one window of W rows.  Window b and sequence
// s have slot b + s, which no other pair with rows has, so a launch of T / W + sequences workgroups covers
// every batch without the host knowing a length.
#include "linear_tiles.h"

namespace moe {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Slot {
    int seq, first, end;   // rows first .. end - 1 of sequence seq; first >= end: nothing
};
// The pair of a slot.  The first slot of sequence s is off[s] / W + s, which grows with s, so the sequence is the
// last one whose first slot is not behind `slot`: 64 candidates at a time, one per lane.
template <int W>
__device__ __forceinline__ Slot find_slot(const int32_t* off, int S, int T, int slot) {
    const int lane = threadIdx.x & 63;
    if (!off) return {slot, slot, slot + 1};
    auto clamped = [&](int s) { return min(max(off[s], 0), T); };
    int lo = 0, n = S;   // the sequence is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 63) / 64, s = lo + lane * step;
        const bool before = lane * step < n && clamped(s) / W + s <= slot;
        // (lane 0 holds for lo = 0 unless slot 0 starts behind the first sequence's first window)
        const int k = max((int)__popcll(__ballot(before)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    const int a = clamped(lo), e = clamped(lo + 1), b = slot - lo;
    if (b < a / W) return {lo, 0, 0};
    return {lo, max(a, b * W), (int)min((int64_t)e, (int64_t)(b + 1) * W)};
}

// v of a slot's rows.  The four waves, and gridDim.z workgroups, take the blocks of 64 K in turn; a lane holds row
// l % 16 of a fragment and 32 bytes of the block at 32 (l / 16), the operands of two matrix instructions (x and
// A alike, so the order of K inside a block does not matter).  PF blocks of loads are in flight per wave, straight
// to registers: every byte of x is used once per 16 NR columns of v.
template <int MT, int NR, int PF>
__global__ __launch_bounds__(256) void k_lora_down(LoraArgs p) {
    __shared__ __align__(16) v4f s_acc[3][MT][NR][64];
    const Slot sl = find_slot<16 * MT>(p.off, p.S, p.T, blockIdx.x);
    if (sl.first >= sl.end) return;
    const int ad = p.ids[sl.seq];
    if (ad < 0 || ad >= p.n) return;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, G = lane >> 4, r0 = blockIdx.y * 16 * NR;
    const uint16_t* xp[MT];
    const uint16_t* ap[NR];
#pragma unroll
    for (int i = 0; i < MT; ++i) xp[i] = p.x + (int64_t)min(sl.first + 16 * i + r16, sl.end - 1) * p.ldx + 16 * G;
#pragma unroll
    for (int j = 0; j < NR; ++j) ap[j] = p.a + ((int64_t)ad * p.R + min(r0 + 16 * j + r16, p.R - 1)) * p.K + 16 * G;
    v4u_t X[PF][MT][2], A[PF][NR][2];
    const int whole = p.K / 64, step = 4 * gridDim.z, b0 = blockIdx.z * 4 + wv;
    auto load = [&](int q, int b) __attribute__((always_inline)) {
        const int o = min(b, whole - 1) * 64;   // (past the end the last block again, unused)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < MT; ++i) X[q][i][h] = *reinterpret_cast<const v4u_t*>(xp[i] + o + 8 * h);
#pragma unroll
            for (int j = 0; j < NR; ++j) A[q][j][h] = *reinterpret_cast<const v4u_t*>(ap[j] + o + 8 * h);
        }
    };
    v4f acc[MT][NR];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto products = [&](int q) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, A[q][j][h]),
                                                                        __builtin_bit_cast(bf16x8, X[q][i][h]), acc[i][j], 0, 0, 0);
    };
    const int nb = whole > b0 ? (whole - b0 + step - 1) / step : 0;
    if (nb) {
#pragma unroll
        for (int q = 0; q < PF; ++q) load(q, b0 + q * step);
        int i0 = 0;
        for (; i0 + PF <= nb; i0 += PF) {
#pragma unroll
            for (int q = 0; q < PF; ++q) {
                products(q);
                __builtin_amdgcn_sched_barrier(0);
                load(q, b0 + (i0 + q + PF) * step);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int q = 0; q < PF; ++q)
            if (i0 + q < nb) products(q);
    }
    if (p.K % 64 && blockIdx.z == 0 && wv == 0) {   // the last K, fewer than 64: chunks of 8 behind them are 0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = whole * 64 + 16 * G + 8 * h;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                X[0][i][h] = v4u_t{0, 0, 0, 0};
                if (k < p.K) X[0][i][h] = *reinterpret_cast<const v4u_t*>(xp[i] + whole * 64 + 8 * h);
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                A[0][j][h] = v4u_t{0, 0, 0, 0};
                if (k < p.K) A[0][j][h] = *reinterpret_cast<const v4u_t*>(ap[j] + whole * 64 + 8 * h);
            }
        }
        products(0);
    }
    if (wv) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j) s_acc[wv - 1][i][j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wv) return;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int t = sl.first + 16 * i + r16;
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            v4f v = acc[i][j];
#pragma unroll
            for (int w = 0; w < 3; ++w) v += s_acc[w][i][j][lane];
            const int r = r0 + 16 * j + 4 * G;
            if (t < sl.end && r < p.ldv)
                *reinterpret_cast<v4f*>(p.v + ((int64_t)blockIdx.z * p.T + t) * p.ldv + r) = v;
        }
    }
}

// y of a slot's rows and 64 columns per wave at a time.  scale v goes to the matrix cores as a sum of PARTS bf16
// values, each the rounding of what the ones before leave: 2 leave 2^-17 of v, under the rounding of a bf16 y, 3
// nothing of float32.  They are formed once per workgroup, as operands in LDS.
template <int MT, int PARTS>
__global__ __launch_bounds__(256) void k_lora_up(LoraArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    v4u_t* s_v = reinterpret_cast<v4u_t*>(smem);   // [PARTS][steps][MT][64]
    const Slot sl = find_slot<16 * MT>(p.off, p.S, p.T, blockIdx.x);
    if (sl.first >= sl.end) return;
    const int ad = p.ids[sl.seq];
    const bool has = ad >= 0 && ad < p.n;
    LinArgs l = p.out;
    l.T = sl.end;
    if (!has && l.res == l.y) return;   // (the same rows: they stay)
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, G = lane >> 4, steps = (p.R + 31) / 32;
    if (has) {
        const float scale = p.scale ? p.scale[ad] : 1.f;
        for (int q = tid; q < steps * MT * 64; q += 256) {
            const int t = sl.first + 16 * ((q >> 6) % MT) + (q & 15), r = (q >> 6) / MT * 32 + 8 * ((q >> 4) & 3);
            float f[8] = {};
            if (t < sl.end && r < p.R) {
                for (int z = 0; z < p.parts; ++z) {
                    const v4f* s = reinterpret_cast<const v4f*>(p.v + ((int64_t)z * p.T + t) * p.ldv + r);
                    const v4f a = s[0], b = s[1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] += a[i], f[4 + i] += b[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                const uint4 h = pack8(f);
                s_v[part * steps * MT * 64 + q] = v4u_t{h.x, h.y, h.z, h.w};
                float g[8];
                unpack8(h, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = fabsf(g[i]) < __builtin_inff() ? f[i] - g[i] : 0.f;
            }
        }
        __syncthreads();
    }
    const v4f zero[4] = {};
    for (int c = 0; c < p.chunks; ++c) {
        const int col0 = ((blockIdx.y * p.chunks + c) * 4 + wv) * 64;
        if (col0 >= l.N) return;   // (no barrier follows)
        uint4 res[MT][2];
        tile_residual<MT>(l, res, sl.first + r16, col0);
        v4f acc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
        if (has) {
            const uint16_t* bp[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) bp[j] = p.b + ((int64_t)ad * l.N + min(col0 + 16 * j + r16, l.N - 1)) * p.R + 8 * G;
            for (int s = 0; s < steps; ++s) {
                v4u_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[j] = v4u_t{0, 0, 0, 0};
                    if (32 * s + 8 * G < p.R) b[j] = *reinterpret_cast<const v4u_t*>(bp[j] + 32 * s);
                }
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const v4u_t v = s_v[((part * steps + s) * MT + i) * 64 + lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[j]),
                                                                                __builtin_bit_cast(bf16x8, v), acc[i][j], 0, 0, 0);
                    }
            }
        }
        tile_epilogue<MT, MOE_ACT_NONE>(l, acc, zero, res, sl.first + r16, col0);
    }
}

template <int MT, int NR, int PF>
void run_down(const LoraArgs& a, const LoraPlan& p, hipStream_t st) {
    hipLaunchKernelGGL((k_lora_down<MT, NR, PF>), dim3((unsigned)p.slots, (unsigned)ceil_div(a.ldv, 16 * NR), (unsigned)p.parts),
                       dim3(256), 0, st, a);
}
template <int MT, int PARTS>
hipError_t run_up(const LoraArgs& a, const LoraPlan& p, hipStream_t st) {
    const size_t lds = (size_t)PARTS * ((a.R + 31) / 32) * MT * 1024;
    if (const hipError_t e = ask_for_lds<k_lora_up<MT, PARTS>>(lds); e != hipSuccess) return e;
    const dim3 grid((unsigned)p.slots, (unsigned)ceil_div(a.out.N, 256 * a.chunks));
    hipLaunchKernelGGL((k_lora_up<MT, PARTS>), grid, dim3(256), lds, st, a);
    return hipGetLastError();
}
template <int MT>
hipError_t run_lora(const LoraArgs& a, const LoraPlan& p, hipStream_t st) {
    constexpr int PF = MT > 1 ? 2 : 4;
    if (a.R <= 16) run_down<MT, 1, PF>(a, p, st);
    else if (a.R <= 32) run_down<MT, 2, PF>(a, p, st);
    else run_down<MT, 4, PF>(a, p, st);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    return a.out.out_bf16 ? run_up<MT, 2>(a, p, st) : run_up<MT, 3>(a, p, st);
}

}  // namespace

hipError_t launch_lora(const LoraArgs& args, hipStream_t st) {
    LoraArgs a = args;
    const LoraPlan p = lora_plan(a.T, a.K, a.R, a.off ? a.S : 0);
    a.ldv = p.ldv;
    a.parts = p.parts;
    a.chunks = 1;
    a.out.nt = (int64_t)a.T * a.out.N * (a.out.out_bf16 ? 2 : 4) >= (32 << 20);
    return p.window == 64 ? run_lora<4>(a, p, st) : run_lora<1>(a, p, st);
}

}  // namespace moe
