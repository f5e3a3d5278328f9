// Low-rank adapters of many requests beside a shared projection (gfx950):
//   y[t] = residual[t] + scale[a] (x[t] A_a^T) B_a^T,  a the adapter of the row's sequence.
//
// Two launches.  k_lora_down forms scale x A^T and stores it as the matrix cores' operands, k_lora_up multiplies
// them by B^T and adds the residual.  Both work on slots: the rows of one sequence inside one window of W rows.
// Window b and sequence s have slot b + s, which no other pair with rows has, so a launch of T / W + sequences
// workgroups covers every batch without the host knowing a length.
#include "linear_tiles.h"

namespace moe {

namespace {

struct Slot {
    int first, end, adapter;   // rows first .. end - 1; first >= end: nothing
};
// The pair of a slot.  The first slot of sequence s is off[s] / W + s, which grows with s, so the sequence is the
// last one whose first slot is not behind `slot`: up to 63 candidates at a time, one per lane.  The boundaries
// and the adapter of the one found are in the lanes already then: up to 63 sequences cost one round of loads.
template <int W>
__device__ __forceinline__ Slot find_slot(const LoraArgs& p, int slot) {
    const int lane = threadIdx.x & 63;
    if (!p.off) return {slot, slot + 1, p.ids[slot]};
    auto clamped = [&](int s) { return min(max(p.off[s], 0), p.T); };
    auto last = [](bool before) { return max((int)__popcll(__ballot(before)) - 1, 0); };   // (slots in front of all: 0)
    int lo = 0, n = p.S;   // the sequence is in [lo, lo + n)
    while (n > 63) {
        const int step = (n + 62) / 63, i = lane * step;
        const int k = last(i < n && clamped(lo + i) / W + lo + i <= slot);
        lo += k * step;
        n = min(step, n - k * step);
    }
    const int off = lane <= n ? clamped(lo + lane) : 0, id = lane < n ? p.ids[lo + lane] : 0;
    const int k = last(lane < n && off / W + lo + lane <= slot), b = slot - lo - k;
    const int a = __builtin_amdgcn_readlane(off, k), e = __builtin_amdgcn_readlane(off, k + 1);
    if (b < a / W) return {0, 0, 0};
    return {max(a, b * W), min(e, (b + 1) * W), __builtin_amdgcn_readlane(id, k)};
}

// The parts of v's 16-row, 32-column operand (mi, s) of a slot, one kilobyte each: lane l holds row l % 16 and
// the columns from 32 s + 16 (l / 16 % 2) + 8 (l / 32), eight of them.
__device__ __forceinline__ v4u_t* v_operand(const LoraArgs& p, int64_t slot, int mt, int mi, int s) {
    return reinterpret_cast<v4u_t*>(p.v) + (((slot * mt + mi) * p.steps + s) * p.split) * 64;
}

// scale x A^T of a slot's rows and 16 NR columns.  Each of the NW waves takes every NW-th block of 64 K and
// brings its operands through LDS stages of its own, S of them in flight, by LDS-DMA: eight neighbouring lanes
// read 128 bytes of one row then.  (Straight to registers the operands' layout puts neighbouring lanes in
// different rows, 64 requests of 16 bytes per instruction: 16384 x 4096, rank 32, took 45 us for 134 MB; this way 35 to
// 39, traced.)  A row's 16-byte chunk c stands at place c ^ (row % 8).  The waves' sums meet in LDS, in wave order, and leave as operands: a
// sum of `split` bf16 values, each the rounding of what the ones before leave.  Two leave 2^-17 of it, under the
// rounding of a bf16 y, three nothing of float32.  Columns from R on are 0.
//   Bound by HBM for many rows of few sequences, and by the chain of a wave's blocks where slots are few: in a decode
// step, and also at 2047 rows in 40 sequences x 4096, rank 64 (12 us), where 104 workgroups leave 152 CUs idle and
// bring 107 MB of rows and adapters, 86 bytes per ns and busy CU.  Waves and
// stages leave room for two workgroups per CU (16000 x 512 in 2000 sequences, rank 16: 37 us with its other half, with
// one workgroup of twice the waves 53; 1 x 7168 10.7 and 10.5).
template <int MT, int NR, int NW, int S>
__global__ __launch_bounds__(64 * NW) void k_lora_down(LoraArgs p) {
    constexpr int STAGE = (MT + NR) * 2048, OPS = 2 * (MT + NR);
    static_assert(MT * NR * 1024 <= S * STAGE, "the sums fit where the stages were");
    extern __shared__ __align__(16) uint8_t smem[];
    v4f* s_acc = reinterpret_cast<v4f*>(smem);   // [NW][MT][NR][64]
    const Slot sl = find_slot<16 * MT>(p, p.slot0 + blockIdx.x);
    const int ad = sl.adapter;
    if (sl.first >= sl.end || ad < 0 || ad >= p.n) return;
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, G = lane >> 4, x8 = r16 & 7, r0 = blockIdx.y * 16 * NR;
    const int whole = p.K / 64, rows = sl.end - sl.first;
    const uint16_t* xb = p.x + sl.first * p.ldx;
    const uint16_t* ab = p.a + (int64_t)ad * p.R * p.K;
    const v4i_t rx = make_srd(xb, (uint32_t)(((rows - 1) * p.ldx + p.K) * 2)), ra = make_srd(ab, (uint32_t)(p.R * p.K * 2));
    // copy i: rows 8 i .. +7 of the fragments, lane l the chunk of row l / 8 that stands at place l % 8
    uint32_t xoff[2 * MT], aoff[2 * NR];
    const int l8 = lane >> 3, chunk = 16 * ((lane & 7) ^ l8);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) xoff[i] = (uint32_t)(min(8 * i + l8, rows - 1) * p.ldx * 2) + chunk;
#pragma unroll
    for (int j = 0; j < 2 * NR; ++j) aoff[j] = (uint32_t)(min(r0 + 8 * j + l8, p.R - 1) * p.K * 2) + chunk;
    uint8_t* ring = smem + wv * S * STAGE;
    const uint32_t lds0 = lds_addr(ring);
    auto issue = [&](int st, int i) __attribute__((always_inline)) {
        const uint32_t o = (uint32_t)min(wv + i * NW, whole - 1) * 128;   // (past the end the last block again, unused)
        const uint32_t base = __builtin_amdgcn_readfirstlane(lds0 + st * STAGE);
#pragma unroll
        for (int j = 0; j < 2 * MT; ++j) dma16(rx, base + j * 1024, xoff[j], o);
#pragma unroll
        for (int j = 0; j < 2 * NR; ++j) dma16(ra, base + (2 * MT + j) * 1024, aoff[j], o);
    };
    v4f acc[MT][NR];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    auto products = [&](const v4u_t (&X)[MT], const v4u_t (&A)[NR]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NR; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, A[j]), __builtin_bit_cast(bf16x8_t, X[i]),
                                                                    acc[i][j], 0, 0, 0);
    };
    const int nb = whole > wv ? (whole - wv + NW - 1) / NW : 0;
    if (nb) {
#pragma unroll
        for (int s = 0; s < S; ++s) issue(s, s);
        int st = 0;
        for (int i = 0; i < nb; ++i) {
            wait_vm<(S - 1) * OPS>();
            const uint8_t* f = ring + st * STAGE + r16 * 128;
            v4u_t X[2][MT], A[2][NR];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int j = 0; j < MT; ++j) X[h][j] = *reinterpret_cast<const v4u_t*>(f + j * 2048 + (((G + 4 * h) ^ x8) << 4));
#pragma unroll
                for (int j = 0; j < NR; ++j) A[h][j] = *reinterpret_cast<const v4u_t*>(f + (MT + j) * 2048 + (((G + 4 * h) ^ x8) << 4));
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read: the stage may be filled again
            __builtin_amdgcn_sched_barrier(0);
            issue(st, i + S);
            st = st == S - 1 ? 0 : st + 1;
            products(X[0], A[0]);
            products(X[1], A[1]);
        }
        wait_all();
    }
    if (p.K % 64 && wv == NW - 1) {   // the last K, fewer than 64: chunks of 8 behind them are 0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = whole * 64 + 8 * G + 32 * h;
            v4u_t X[MT], A[NR];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                X[i] = v4u_t{0, 0, 0, 0};
                if (k < p.K) X[i] = *reinterpret_cast<const v4u_t*>(xb + min(16 * i + r16, rows - 1) * p.ldx + k);
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                A[j] = v4u_t{0, 0, 0, 0};
                if (k < p.K) A[j] = *reinterpret_cast<const v4u_t*>(ab + min(r0 + 16 * j + r16, p.R - 1) * p.K + k);
            }
            products(X, A);
        }
    }
    const float scale = p.scale ? p.scale[ad] : 1.f;
    __syncthreads();   // every wave's copies have ended: the stages become the sums' place
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j) s_acc[((wv * MT + i) * NR + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    constexpr int NS = (NR + 1) / 2;   // operands of a row fragment
    for (int q = wv; q < MT * NS; q += NW) {
        const int i = q / NS, s = q % NS;
        if (r0 / 32 + s >= p.steps) continue;   // (the last workgroup's columns may end before its second operand)
        v4f v[2] = {};
#pragma unroll
        for (int j = 0; j < (NR > 1 ? 2 : 1); ++j)
#pragma unroll
            for (int w = 0; w < NW; ++w) v[j] += s_acc[((w * MT + i) * NR + 2 * s + j) * 64 + lane];
        // eight consecutive columns in a lane
        uint32_t u[2][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u[0][c] = __float_as_uint(v[0][c]);
            u[1][c] = __float_as_uint(v[1][c]);
            swap_groups(u[0][c], u[1][c]);
        }
        const bool in = r0 + 32 * s + 16 * (G & 1) + 8 * (G >> 1) < p.R;
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = in ? __uint_as_float(u[c >> 2][c & 3]) * scale : 0.f;
        v4u_t* o = v_operand(p, p.slot0 + blockIdx.x, MT, i, r0 / 32 + s);
        for (int part = 0; part < p.split; ++part) {
            const uint4 h = pack8(f);
            o[part * 64 + lane] = v4u_t{h.x, h.y, h.z, h.w};
            float g[8];
            unpack8(h, g);
#pragma unroll
            for (int c = 0; c < 8; ++c) f[c] = fabsf(g[c]) < __builtin_inff() ? f[c] - g[c] : 0.f;
        }
    }
}

// y of a slot's rows, 16 MI of them and 128 columns per wave.  v is the first operand and B the second, so that a
// lane of the accumulators holds rows 4 (l / 16) .. +3 and one column of each of eight fragments; which column of B
// stands where in a fragment is free, and is chosen such that those eight are consecutive (float32: four and four):
// 16 neighbouring lanes then move 256 bytes of a row.  The residual, B and v are requested at once.  Bound by HBM for many
// rows (16384 x 4096, rank 32: 58 us, 4.6 TB/s of residual and y), by the chain of a workgroup's loads and products where
// slots are few: 2048 rows in 40 sequences take 18.7 us at rank 64, 12.8 at rank 8.  Three workgroups per CU make
// 768 places, and a second round for the 832 workgroups there costs too: 31 sequences, 760 workgroups, take 15.7 us,
// 64 sequences, 1024 workgroups, 22.2.
template <int MT, int MI, bool BF16>
__global__ __launch_bounds__(256, 3) void k_lora_up(LoraArgs p) {
    constexpr int SPLIT = BF16 ? 2 : 3, WR = MT / MI, WC = 4 / WR;   // waves along rows and columns
    const int64_t slot = p.slot0 + blockIdx.x / p.col_blocks;
    const Slot sl = find_slot<16 * MT>(p, (int)slot);
    if (sl.first >= sl.end) return;
    const bool has = sl.adapter >= 0 && sl.adapter < p.n;
    const LinArgs& l = p.out;
    if (!has && l.res == l.y) return;   // (the same rows: they stay)
    const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, G = lane >> 4, m0 = wv % WR * MI;
    const int col0 = ((int)(blockIdx.x % p.col_blocks) * WC + wv / WR) * 128, row0 = sl.first + 16 * m0 + 4 * G;
    if (col0 >= l.N || sl.first + 16 * m0 >= sl.end) return;
    // a lane's columns: eight from col, or four from there and four 64 further
    const int col = col0 + (BF16 ? 8 : 4) * r16;
    auto there = [&](int i, int e, int h) __attribute__((always_inline)) { return row0 + 16 * i + e < sl.end && col + 64 * h < l.N; };
    auto at = [&](int i, int e) __attribute__((always_inline)) { return (int64_t)(row0 + 16 * i + e); };
    v4u_t res[MI][4][BF16 ? 1 : 2];
    if (l.res) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int h = 0; h < (BF16 ? 1 : 2); ++h) {
                    res[i][e][h] = v4u_t{0, 0, 0, 0};
                    if (there(i, e, h)) {
                        const int64_t o = at(i, e) * l.ldr + col + 64 * h;
                        res[i][e][h] = BF16 ? *reinterpret_cast<const v4u_t*>(reinterpret_cast<const uint16_t*>(l.res) + o)
                                            : *reinterpret_cast<const v4u_t*>(reinterpret_cast<const float*>(l.res) + o);
                    }
                }
    }
    v4f acc[MI][8];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    if (has) {
        const int c = 16 * (G & 1) + 8 * (G >> 1);   // v's order of columns
        const uint16_t* bb = p.b + (int64_t)sl.adapter * l.N * p.R + c;
        uint32_t boff[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) boff[j] = (uint32_t)min(BF16 ? col + j : col + (j & 3) + 64 * (j >> 2), l.N - 1) * (uint32_t)p.R;
        const v4u_t* vp = v_operand(p, slot, MT, m0, 0) + lane;
        for (int s = 0; s < p.steps; ++s) {
            v4u_t b[8], v[MI][SPLIT];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                b[j] = v4u_t{0, 0, 0, 0};
                if (32 * s + c < p.R) b[j] = *reinterpret_cast<const v4u_t*>(bb + boff[j] + 32 * s);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int part = 0; part < SPLIT; ++part) v[i][part] = vp[((i * p.steps + s) * SPLIT + part) * 64];
#pragma unroll
            for (int part = 0; part < SPLIT; ++part)
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, v[i][part]),
                                                                            __builtin_bit_cast(bf16x8_t, b[j]), acc[i][j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = acc[i][j][e];
            if constexpr (BF16) {
                if (l.res) {
                    float g[8];
                    unpack8(__builtin_bit_cast(uint4, res[i][e][0]), g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] += g[j];
                }
                if (there(i, e, 0))
                    store16(reinterpret_cast<v4u_t*>(reinterpret_cast<uint16_t*>(l.y) + at(i, e) * l.ldy + col),
                            __builtin_bit_cast(v4u_t, pack8(f)), l.nt);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v4f o = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
                    if (l.res) o += __builtin_bit_cast(v4f, res[i][e][h]);
                    if (there(i, e, h))
                        store16(reinterpret_cast<v4u_t*>(reinterpret_cast<float*>(l.y) + at(i, e) * l.ldy + col + 64 * h),
                                __builtin_bit_cast(v4u_t, o), l.nt);
                }
            }
        }
}

// HIP takes fewer than 2^32 threads in a launch: slots go in parts where that would not do.
template <int MT, int NR, int NW, int S>
hipError_t run_down(LoraArgs a, int64_t slots, hipStream_t st) {
    constexpr size_t lds = (size_t)NW * S * (MT + NR) * 2048;
    if (const hipError_t e = ask_for_lds<k_lora_down<MT, NR, NW, S>>(lds); e != hipSuccess) return e;
    const unsigned groups = (unsigned)ceil_div(a.R, 16 * NR);
    const int64_t most = launch_rows(64 * NW * groups);
    for (int64_t s = 0; s < slots; s += most) {
        a.slot0 = (int)s;
        hipLaunchKernelGGL((k_lora_down<MT, NR, NW, S>), dim3((unsigned)std::min(most, slots - s), groups), dim3(64 * NW), lds, st, a);
    }
    return hipGetLastError();
}
template <int MT, int MI, bool BF16>
hipError_t run_up(LoraArgs a, int64_t slots, hipStream_t st) {
    a.col_blocks = (int)ceil_div(a.out.N, 512 * MI / MT);
    const int64_t most = launch_rows(256) / a.col_blocks;
    for (int64_t s = 0; s < slots; s += most) {
        a.slot0 = (int)s;
        hipLaunchKernelGGL((k_lora_up<MT, MI, BF16>), dim3((unsigned)(std::min(most, slots - s) * a.col_blocks)), dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs& args, hipStream_t st) {
    LoraArgs a = args;
    const bool bf16 = a.out.out_bf16;
    const LoraPlan p = lora_plan(a.T, a.R, a.off ? a.S : 0, bf16);
    a.steps = p.steps;
    a.split = p.split;
    a.out.nt = (int64_t)a.T * a.out.N * (bf16 ? 2 : 4) >= (32 << 20);
    hipError_t e;
    if (p.window == 32) {
        if (a.R <= 16) e = run_down<2, 1, 4, 3>(a, p.slots, st);
        else if (a.R <= 32) e = run_down<2, 2, 4, 2>(a, p.slots, st);
        else e = run_down<2, 4, 3, 2>(a, p.slots, st);
        if (e != hipSuccess) return e;
        return bf16 ? run_up<2, 2, true>(a, p.slots, st) : run_up<2, 1, false>(a, p.slots, st);
    }
    if (a.R <= 16) e = run_down<1, 1, 4, 4>(a, p.slots, st);
    else if (a.R <= 32) e = run_down<1, 2, 4, 3>(a, p.slots, st);
    else e = run_down<1, 4, 4, 2>(a, p.slots, st);
    if (e != hipSuccess) return e;
    return bf16 ? run_up<1, 1, true>(a, p.slots, st) : run_up<1, 1, false>(a, p.slots, st);
}

}  // namespace moe
