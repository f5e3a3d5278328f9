// Router training (gfx950): load-balance and z losses with per-expert counts, the gradient of the
// router logits, and the gradients of the weighted combine.
//
// A row of logits is held by L lanes (16 up to 256 experts, a whole wave above), 4 * Q values each;
// lane `sub` has experts 4 * (sub + L * i) + c.  Softmax sums stay inside the L lanes.
#include "layer_common.h"

#include <algorithm>

namespace moe {

template <int L>
__device__ __forceinline__ float rsum(float v) {
    if constexpr (L == 16) return sum16(v);
    else return wave_sum(v);
}
template <int L>
__device__ __forceinline__ float rmax(float v) {
    if constexpr (L == 16) return max16(v);
    else return wave_max(v);
}

// Elements of row p (E of them) that the lane holds; `pad` behind the end.
template <int L, int Q, bool VEC, typename V>
__device__ __forceinline__ void load_row(const V* __restrict__ p, int E, int sub, V pad, V (&v)[4 * Q]) {
    typedef V v4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const int e = 4 * (sub + L * i);
        if constexpr (VEC) {
            v4 x = {pad, pad, pad, pad};
            if (e < E) x = *reinterpret_cast<const v4*>(p + e);
#pragma unroll
            for (int c = 0; c < 4; ++c) v[4 * i + c] = x[c];
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) v[4 * i + c] = e + c < E ? p[e + c] : pad;
        }
    }
}

// Sequence s of the packed rows: [begin, end), clamped into [0, T].
struct Seqs {
    const int32_t* off;   // NULL: one sequence of all rows
    int S, T;
    __device__ __forceinline__ int at(int i) const { return min(max(off[i], 0), T); }
    __device__ __forceinline__ int begin(int s) const { return off ? at(s) : 0; }
    __device__ __forceinline__ int end(int s) const { return off ? max(at(s + 1), at(s)) : T; }
    // the sequence that row t lies in if it lies in one: the last one that begins at or before t
    __device__ __forceinline__ int find(int t) const {
        if (!off) return 0;
        int lo = 0, hi = S;   // begin(lo) <= t (or lo == 0), begin(hi) > t (or hi == S)
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (at(m) <= t) lo = m;
            else hi = m;
        }
        return lo;
    }
};

// exp(x) by the base-2 instruction: off by |x| 2^-24 and a unit in the last place, of which a softmax
// sees its row's spread of logits.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Natural logarithm and reciprocal by their instructions (one unit in the last place): with IEEE
// divisions and library logarithms the gradient of 16384 x 128 logits takes 7.6 us instead of 6.9.
__device__ __forceinline__ float log_fast(float x) { return __builtin_amdgcn_logf(x) * 0.69314718f; }
__device__ __forceinline__ float rcp_or_0(float x) { return x != 0.f ? __builtin_amdgcn_rcpf(x) : 0.f; }

// Softmax numerators of a row: v -> exp(v - max); returns their sum (0 only where every logit is
// -infinity) and the shift.  NaN logits make the sum NaN.
template <int L, int Q>
__device__ __forceinline__ float softmax_row(float (&v)[4 * Q], float& shift) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < 4 * Q; ++i) m = fmaxf(m, v[i]);
    m = rmax<L>(m);
    shift = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) {
        v[i] = exp_fast(v[i] - shift);
        s += v[i];
    }
    return rsum<L>(s);
}

// Sums over a workgroup's threads, in wave order; s: one float per wave.
template <int NW>
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = wave_sum(v);
    __syncthreads();   // (an earlier sum has been read)
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += s[i];
    return v;
}

// losses from the sums over the sequences (bal: sum_s sum_e c P / T_s; z: sum of squared log-sums)
__device__ __forceinline__ void put_losses(const BalanceArgs& a, float bal, float z, int live, int valid) {
    bal = live ? a.ca * bal * ((float)a.E / (float)a.k) / (float)live : 0.f;
    z = valid && a.cz != 0.f ? a.cz * z / (float)valid : 0.f;   // (a log-sum past 2^64 has no finite square)
    a.losses[0] = bal + z;
    a.losses[1] = bal;
    a.losses[2] = z;
}

// ----------------------------------------------------------------------------------------
// Sums of probabilities, counts and squared log-sums of each (workgroup, sequence) part, into the
// part's slot.  ONE: a single workgroup holds all rows and writes the results itself, which saves the
// second launch and its latency (64 x 8: 10 -> 4 us).  16384 x 128 takes 4.8 us (8.4 MB, 1.8 TB/s), 4096 x 256 in
// 9 sequences 7.9: latency, the boundaries' search and then one or two rounds of rows per workgroup.
constexpr int kRowsThreads = 512;
constexpr int kSeqLds = 1024;   // sequence boundaries held in LDS (a search in memory waits for every step)
template <int L, int Q, bool VEC, bool ONE>
__global__ __launch_bounds__(kRowsThreads) void k_balance_rows(BalanceArgs a, BalancePlan p) {
    constexpr int NT = kRowsThreads, NG = NT / L, N = 4 * Q;
    __shared__ __align__(16) float s_p[NG][L * N];
    __shared__ int s_hit[L * N];
    __shared__ float s_z[NG], s_w[NT / 64];
    __shared__ int s_off[kSeqLds + 1];
    const int tid = threadIdx.x, g = tid / L, sub = tid % L, b = blockIdx.x;
    if (!ONE && b == 0 && tid == 0) *reinterpret_cast<int*>(a.ws + p.done) = 0;   // the second kernel's ticket
    const bool staged = a.off && a.S <= kSeqLds;
    if (staged) {
        for (int i = tid; i <= a.S; i += NT) s_off[i] = a.off[i];
        __syncthreads();
    }
    const Seqs sq{staged ? s_off : a.off, a.S, a.T};
    const int lo = b * p.chunk, hi = lo + min(p.chunk, a.T - lo);
    if constexpr (ONE) {   // what no sequence with rows overwrites below
        for (int64_t i = tid; i < (int64_t)a.S * a.E; i += NT) {
            a.counts[i] = 0;
            if (a.mean_probs) a.mean_probs[i] = 0.f;
        }
        __syncthreads();
    }
    float bal = 0.f, ztot = 0.f;
    int live = 0, valid = 0, s, r1;
    // from row to row over the sequences that have rows here (empty ones are stepped over by the search)
    for (int r0 = max(lo, sq.begin(0)); r0 < hi; r0 = r1) {
        s = sq.find(r0);
        r1 = min(sq.end(s), hi);
        if (r1 <= r0) break;   // behind the last sequence
        float acc[N], z = 0.f, v[N];
        if (r0 + g < r1) load_row<L, Q, VEC>(a.logits + (int64_t)(r0 + g) * a.E, a.E, sub, -INFINITY, v);
        for (int e = tid; e < a.E; e += NT) s_hit[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)r0 * a.k + tid; i < (int64_t)r1 * a.k; i += NT) {
            const int id = a.ids[i];
            if (id >= 0 && id < a.E) atomicAdd(&s_hit[id], 1);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        for (int r = r0 + g; r < r1; r += NG) {
            float num[N], shift, nx[N];
            if (r + NG < r1) load_row<L, Q, VEC>(a.logits + (int64_t)(r + NG) * a.E, a.E, sub, -INFINITY, nx);
            float tot = 0.f;
            if (a.scoring == MOE_SCORING_SIGMOID) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    num[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-v[i]));
                    tot += num[i];
                }
                tot = rsum<L>(tot);
            }
            if (a.scoring != MOE_SCORING_SIGMOID || a.cz != 0.f) {
                const float sum = softmax_row<L, Q>(v, shift);
                if (sum != 0.f) {
                    const float lse = shift + log_fast(sum);
                    z = fmaf(lse, lse, z);
                }
                if (a.scoring != MOE_SCORING_SIGMOID) {
                    tot = sum;
#pragma unroll
                    for (int i = 0; i < N; ++i) num[i] = v[i];
                }
            }
            const float inv = rcp_or_0(tot);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                acc[i] = fmaf(num[i], inv, acc[i]);
                v[i] = nx[i];
            }
        }
#pragma unroll
        for (int i = 0; i < Q; ++i)
            *reinterpret_cast<float4*>(&s_p[g][4 * (sub + L * i)]) =
                make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        if (sub == 0) s_z[g] = z;
        __syncthreads();
        const int len = r1 - r0;
        float dot = 0.f;
        for (int e = tid; e < a.E; e += NT) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < NG; ++i) t += s_p[i][e];
            if constexpr (ONE) {
                const float mean = t / (float)len;
                a.counts[(int64_t)s * a.E + e] = s_hit[e];
                if (a.mean_probs) a.mean_probs[(int64_t)s * a.E + e] = mean;
                dot = fmaf(mean, (float)s_hit[e] / (float)len, dot);
            } else {
                const int64_t slot = (int64_t)(b + s) * p.stride;
                reinterpret_cast<float*>(a.ws + p.probs)[slot + e] = t;
                reinterpret_cast<int*>(a.ws + p.hits)[slot + e] = s_hit[e];
            }
        }
        float t = 0.f;
        if (tid == 0) {
#pragma unroll
            for (int i = 0; i < NG; ++i) t += s_z[i];
            if constexpr (!ONE) reinterpret_cast<float*>(a.ws + p.z)[b + s] = t;
        }
        if constexpr (ONE) {
            bal += block_sum<NT / 64>(dot, s_w);
            ztot += t;
            live += 1;
            valid += len;
        }
        __syncthreads();
    }
    if (ONE && tid == 0) put_losses(a, bal, ztot, live, valid);
}

// One workgroup per sequence: its parts' sums in row order -> counts, mean probabilities and the
// sequence's share of the losses.  A thread takes four experts of every NG-th part; with several sequences
// the last workgroup to finish adds the shares in sequence order.  6.3 us for 16384 x 128, 7.4 for 4096 x 256
// in 9 sequences: latency, of boundaries, parts, the sums through LDS and the ticket, each waiting for the
// one before.
__global__ __launch_bounds__(1024) void k_balance_reduce(BalanceArgs a, BalancePlan p, int c4) {
    __shared__ __align__(16) float4 s_p[1024];
    __shared__ __align__(16) int4 s_h[1024];
    __shared__ float s_w[16];
    __shared__ int s_n[2][16], s_last;
    const int tid = threadIdx.x, NG = 1024 / c4, c = tid & (c4 - 1), g = tid / c4;   // c4: a power of two >= E / 4
    const int s = blockIdx.x, e0 = 4 * c;
    const Seqs sq{a.off, a.S, a.T};
    const int t0 = sq.begin(s), t1 = sq.end(s);
    const float* probs = reinterpret_cast<const float*>(a.ws + p.probs);
    const int* hits = reinterpret_cast<const int*>(a.ws + p.hits);
    const float* zs = reinterpret_cast<const float*>(a.ws + p.z);
    float* seq = reinterpret_cast<float*>(a.ws + p.seq);
    const int b0 = t0 / p.chunk, b1 = t1 > t0 ? (t1 - 1) / p.chunk + 1 : b0;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 n = make_int4(0, 0, 0, 0);
    if (e0 < a.E) {
#pragma unroll 8
        for (int b = b0 + g; b < b1; b += NG) {
            const int64_t o = (int64_t)(b + s) * p.stride + e0;   // (rows of `stride` = E rounded up to 4)
            const float4 x = *reinterpret_cast<const float4*>(probs + o);
            const int4 h = *reinterpret_cast<const int4*>(hits + o);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            n.x += h.x, n.y += h.y, n.z += h.z, n.w += h.w;
        }
    }
    float z = 0.f;
    for (int b = b0 + tid; b < b1; b += 1024) z += zs[b + s];
    s_p[tid] = v;
    s_h[tid] = n;
    __syncthreads();
    const float len = (float)(t1 - t0);
    float dot = 0.f;
    for (int e = tid; e < a.E; e += 1024) {
        float t = 0.f;
        int m = 0;
#pragma unroll 8
        for (int i = 0; i < NG; ++i) {
            t += reinterpret_cast<const float*>(s_p)[4 * i * c4 + e];
            m += reinterpret_cast<const int*>(s_h)[4 * i * c4 + e];
        }
        const float mean = t1 > t0 ? t / len : 0.f;
        a.counts[(int64_t)s * a.E + e] = m;
        if (a.mean_probs) a.mean_probs[(int64_t)s * a.E + e] = mean;
        if (t1 > t0) dot = fmaf(mean, (float)m / len, dot);
    }
    dot = block_sum<16>(dot, s_w);
    z = block_sum<16>(z, s_w);
    if (a.S == 1) {
        if (tid == 0) put_losses(a, dot, z, t1 > t0, max(t1 - t0, 0));
        return;
    }
    if (tid == 0) {
        __hip_atomic_store(&seq[2 * s], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&seq[2 * s + 1], z, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(reinterpret_cast<int*>(a.ws + p.done), 1, __ATOMIC_ACQ_REL,
                                        __HIP_MEMORY_SCOPE_AGENT) == a.S - 1;
    }
    __syncthreads();
    if (!s_last) return;
    float bal = 0.f;
    z = 0.f;
    int live = 0, valid = 0;
    for (int i = tid; i < a.S; i += 1024) {
        bal += __hip_atomic_load(&seq[2 * i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        z += __hip_atomic_load(&seq[2 * i + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int l = sq.end(i) - sq.begin(i);
        live += l > 0;
        valid += l;
    }
    bal = block_sum<16>(bal, s_w);
    z = block_sum<16>(z, s_w);
#pragma unroll
    for (int o = 32; o; o >>= 1) {
        live += __shfl_xor(live, o);
        valid += __shfl_xor(valid, o);
    }
    if ((tid & 63) == 0) {
        s_n[0][tid >> 6] = live;
        s_n[1][tid >> 6] = valid;
    }
    __syncthreads();
    if (tid == 0) {
        live = valid = 0;
        for (int i = 0; i < 16; ++i) {
            live += s_n[0][i];
            valid += s_n[1][i];
        }
        put_losses(a, bal, z, live, valid);
    }
}

// Experts per row -> lanes per row, vectors per lane.
#define MOE_ROW_DISPATCH(E, VEC, CALL)                    \
    do {                                                  \
        if ((E) <= 64) { if (VEC) CALL(16, 1, true); else CALL(16, 1, false); }        \
        else if ((E) <= 128) { if (VEC) CALL(16, 2, true); else CALL(16, 2, false); }  \
        else if ((E) <= 256) { if (VEC) CALL(16, 4, true); else CALL(16, 4, false); }  \
        else if ((E) <= 512) { if (VEC) CALL(64, 2, true); else CALL(64, 2, false); }  \
        else { if (VEC) CALL(64, 4, true); else CALL(64, 4, false); }                  \
    } while (0)

static bool vec4(const void* p, int E) { return E % 4 == 0 && (uintptr_t)p % 16 == 0; }

hipError_t launch_balance_loss(const BalanceArgs& a, hipStream_t st) {
    const BalancePlan p = balance_plan(a.T, a.E, a.S);
    const bool v = vec4(a.logits, a.E);
    if (p.one) {
#define MOE_CALL(L, Q, V) hipLaunchKernelGGL((k_balance_rows<L, Q, V, true>), dim3(1), dim3(kRowsThreads), 0, st, a, p)
        MOE_ROW_DISPATCH(a.E, v, MOE_CALL);
#undef MOE_CALL
        return hipGetLastError();
    }
#define MOE_CALL(L, Q, V) \
    hipLaunchKernelGGL((k_balance_rows<L, Q, V, false>), dim3(p.nblocks), dim3(kRowsThreads), 0, st, a, p)
    MOE_ROW_DISPATCH(a.E, v, MOE_CALL);
#undef MOE_CALL
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int c4 = 32;   // (fewer columns would leave more than 32 row groups to add up one by one)
    while (4 * c4 < a.E) c4 *= 2;
    hipLaunchKernelGGL(k_balance_reduce, dim3(a.S), dim3(1024), 0, st, a, p, c4);
    return hipGetLastError();
}

// ----------------------------------------------------------------------------------------
// Gradient of the router logits.  With p the probabilities, u_e = dL/dp_e of the balance loss
// (the sequence's counts times a constant), s the scores and D_e = sum of dw_j over the slots that
// chose e, m_e their number:
//   balance, softmax   p (u - sum p u)
//            sigmoid   p (1 - s) (u - sum p u)
//   z                  2 cz lse / T_v softmax
//   weights, softmax   rsf p (D - sum p D)
//            over the chosen (softmax renormalised; sigmoid with a factor 1 - s):
//                      rsf q (D - m sum q D),  q = score / sum m score
// One row per L lanes, read once and written once: 16384 x 128 with every part 7.0 us (18 MB, 2.6 TB/s),
// 4096 x 256 with sigmoid 7.4; the exponentials and the chain search, row, counts, slots bound it.
// Orders the LDS accesses of a wave's own lanes (a row's lanes are in one wave).
__device__ __forceinline__ void wave_lds_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// WALK: more rows than the grid holds, a workgroup takes several (in a loop the kernel needs a third more
// registers).
template <int L, int Q, bool VEC, bool WALK>
__global__ __launch_bounds__(256) void k_route_bwd(RouteBwdArgs a) {
    constexpr int NG = 256 / L, N = 4 * Q;
    __shared__ int s_off[kSeqLds + 1];
    __shared__ int s_n[2][4];
    __shared__ __align__(16) float s_d[NG][L * N], s_m[NG][L * N];
    const int tid = threadIdx.x, g = tid / L, sub = tid % L;
    const Seqs sq{a.off, a.S, a.T};
    const bool staged = a.off && a.S <= kSeqLds;
    int live = 1, valid = a.T;
    if (a.off && !staged && !a.counts) {   // (live is the balance loss's alone)
        valid = max(sq.at(a.S) - sq.begin(0), 0);
    } else if (a.off) {
        live = valid = 0;
        for (int i = tid; i < a.S; i += 256) {
            const int b = sq.begin(i), len = sq.end(i) - b;
            live += len > 0;
            valid += len;
            if (staged) s_off[i] = b;
        }
        if (staged && tid == 0) s_off[a.S] = sq.at(a.S);
#pragma unroll
        for (int o = 32; o; o >>= 1) {
            live += __shfl_xor(live, o);
            valid += __shfl_xor(valid, o);
        }
        if ((tid & 63) == 0) {
            s_n[0][tid >> 6] = live;
            s_n[1][tid >> 6] = valid;
        }
        __syncthreads();
        live = s_n[0][0] + s_n[0][1] + s_n[0][2] + s_n[0][3];
        valid = s_n[1][0] + s_n[1][1] + s_n[1][2] + s_n[1][3];
    }
    const Seqs sl{staged ? s_off : a.off, a.S, a.T};
    for (int64_t t = (int64_t)blockIdx.x * NG + g; t < a.T; t += (int64_t)gridDim.x * NG) {
        const int s = sl.find((int)t), t0 = sl.begin(s), t1 = sl.end(s);
        float d[N];
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = 0.f;
        if (t >= t0 && t < t1) {
            const bool sig = a.scoring == MOE_SCORING_SIGMOID;
            float l[N], v[N], sc[N], om[N], shift;   // om: 1 - s for the sigmoid, 1 for softmax
            load_row<L, Q, VEC>(a.logits + t * a.E, a.E, sub, -INFINITY, l);
            int id0 = -1, c[N];     // everything else the row needs is requested now as well
            float dw0 = 0.f;
            if (a.dw && sub < a.k) {
                id0 = a.ids[t * a.k + sub];
                dw0 = a.dw[t * a.k + sub];
            }
            if (a.counts) load_row<L, Q, VEC>(a.counts + (int64_t)s * a.E, a.E, sub, 0, c);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = l[i];
            float sum = 0.f;
            if (!sig || a.cz != 0.f) sum = softmax_row<L, Q>(v, shift);
            const float inv = rcp_or_0(sum);
            float pinv = inv;
            if (sig) {
                float z = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float ex = exp_fast(-l[i]);
                    sc[i] = __builtin_amdgcn_rcpf(1.0f + ex);
                    om[i] = ex < INFINITY ? ex * sc[i] : 1.0f - sc[i];
                    z += sc[i];
                }
                z = rsum<L>(z);
                pinv = rcp_or_0(z);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    sc[i] = v[i];
                    om[i] = 1.0f;
                }
            }
            if (a.counts) {
                const float rl = __builtin_amdgcn_rcpf((float)(t1 - t0));
                const float cu = a.ca * __builtin_amdgcn_rcpf((float)live) * a.load * rl * rl;
                float pu = 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) pu = fmaf(sc[i], (float)c[i], pu);
                pu = rsum<L>(pu) * pinv;      // sum p c
                const float f = cu * pinv;
                if (sig) {
#pragma unroll
                    for (int i = 0; i < N; ++i) d[i] = f * sc[i] * om[i] * ((float)c[i] - pu);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) d[i] = f * sc[i] * ((float)c[i] - pu);
                }
            }
            if (a.cz != 0.f && sum != 0.f) {
                const float cz = 2.0f * a.cz * __builtin_amdgcn_rcpf((float)valid) * (shift + log_fast(sum)) * inv;
#pragma unroll
                for (int i = 0; i < N; ++i) d[i] = fmaf(cz, v[i], d[i]);
            }
            if (a.dw) {
                // D and m through the row's LDS lines: lane j adds up the slots that chose the same expert as
                // slot j, in slot order, and all of them store that sum (comparing every expert with every
                // slot instead took 640 instructions of a row's 1100 at 256 experts and 8 slots)
                float D[N], m[N];
                float* dl = s_d[g];
                float* ml = s_m[g];
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    *reinterpret_cast<float4*>(dl + 4 * (sub + L * i)) = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4*>(ml + 4 * (sub + L * i)) = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                wave_lds_fence();
                for (int j0 = 0; j0 < a.k; j0 += L) {
                    const int id = j0 == 0 ? id0 : j0 + sub < a.k ? a.ids[t * a.k + j0 + sub] : -1;
                    const float w = j0 == 0 ? dw0 : j0 + sub < a.k ? a.dw[t * a.k + j0 + sub] : 0.f;
                    const bool in = id >= 0 && id < a.E;
                    float sum = in ? dl[id] : 0.f, cnt = in ? ml[id] : 0.f;   // (slots of earlier rounds)
                    wave_lds_fence();
                    const int n = min(L, a.k - j0);
                    for (int j = 0; j < n; ++j) {
                        const bool same = __shfl(id, j, L) == id;
                        const float wj = __shfl(w, j, L);
                        sum += same ? wj : 0.f;
                        cnt += same ? 1.f : 0.f;
                    }
                    if (in) {
                        dl[id] = sum;
                        ml[id] = cnt;
                    }
                    wave_lds_fence();
                }
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    const float4 x = *reinterpret_cast<const float4*>(dl + 4 * (sub + L * i));
                    const float4 y = *reinterpret_cast<const float4*>(ml + 4 * (sub + L * i));
                    D[4 * i] = x.x, D[4 * i + 1] = x.y, D[4 * i + 2] = x.z, D[4 * i + 3] = x.w;
                    m[4 * i] = y.x, m[4 * i + 1] = y.y, m[4 * i + 2] = y.z, m[4 * i + 3] = y.w;
                }
                if (!sig && !a.renorm) {
                    float pd = 0.f;
#pragma unroll
                    for (int i = 0; i < N; ++i) pd = fmaf(v[i], D[i], pd);
                    pd = rsum<L>(pd) * inv;
                    const float f = a.rsf * inv;
#pragma unroll
                    for (int i = 0; i < N; ++i) d[i] = fmaf(f * v[i], D[i] - pd, d[i]);
                } else {
                    // Scores relative to the largest chosen one, as the forward weights are (softmax: by its
                    // logit), and exactly 1 there: a row with a single choice then has the gradient 0, not
                    // the rounding of D - D (which a small balance loss would be lost in).
                    float q[N], mx = -INFINITY, z = 0.f, qd = 0.f;
#pragma unroll
                    for (int i = 0; i < N; ++i) mx = m[i] > 0.f ? fmaxf(mx, sig ? sc[i] : l[i]) : mx;
                    mx = rmax<L>(mx);
                    if (mx == -INFINITY) mx = 0.f;
                    const float rmx = rcp_or_0(mx);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float s = sig ? (sc[i] == mx && mx > 0.f ? 1.f : sc[i] * rmx) : exp_fast(l[i] - mx);
                        q[i] = m[i] > 0.f ? s : 0.f;
                        z = fmaf(m[i], q[i], z);
                        qd = fmaf(q[i], D[i], qd);
                    }
                    z = rsum<L>(z);
                    qd = rsum<L>(qd);
                    const float zi = rcp_or_0(z);
                    qd *= zi;
                    const float f = a.rsf * zi;
#pragma unroll
                    for (int i = 0; i < N; ++i) d[i] = fmaf(f * q[i] * om[i], D[i] - m[i] * qd, d[i]);
                }
            }
        }
        float* o = a.dlogits + t * a.E;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int e = 4 * (sub + L * i);
            if constexpr (VEC) {
                if (e < a.E) *reinterpret_cast<float4*>(o + e) = make_float4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (e + c < a.E) o[e + c] = d[4 * i + c];
            }
        }
        if constexpr (!WALK) break;
    }
}

hipError_t launch_route_backward(const RouteBwdArgs& a, hipStream_t st) {
    const bool v = vec4(a.logits, a.E) && vec4(a.dlogits, a.E) && (!a.counts || vec4(a.counts, a.E));
    // With counts every workgroup reads all boundaries for the number of sequences that have rows; beyond those
    // that LDS holds, no more workgroups than stay resident, each with more rows (2^20 rows of 8 logits, a sequence
    // each: 2.5 ms, one workgroup for every 16 rows 33.9; 131072 x 64 in 30000: 87 us and 134).
    const int64_t most = a.off && a.counts && a.S > kSeqLds ? 2048 : launch_rows(256);
#define MOE_CALL(L, Q, V)                                                                                       \
    do {                                                                                                        \
        const int64_t n = ceil_div(a.T, 256 / L);                                                               \
        if (n > most) hipLaunchKernelGGL((k_route_bwd<L, Q, V, true>), dim3((unsigned)most), dim3(256), 0, st, a); \
        else hipLaunchKernelGGL((k_route_bwd<L, Q, V, false>), dim3((unsigned)n), dim3(256), 0, st, a);         \
    } while (0)
    MOE_ROW_DISPATCH(a.E, v, MOE_CALL);
#undef MOE_CALL
    return hipGetLastError();
}

// ----------------------------------------------------------------------------------------
// Gradients of the combine: G threads per token walk its columns, 16 bytes of every expert row at a
// time (8 bf16 or 4 float32 columns); up to 8 expert rows are in flight per vector, so dy is read once
// for every 8 slots.  Bound by HBM: the expert rows are read once and (dexpert_out) written once, both
// past the caches.
typedef unsigned v4u_t __attribute__((ext_vector_type(4)));

// Rows that no assignment names: each of the first nclear workgroups takes `per` rows, marks in LDS
// those that an entry of pos names (all entries pass by, from the caches) and writes zeros to the others:
// no launch, workspace or atomic in memory of its own.
constexpr int kClearMost = 128, kClearRows = 1 << 17;   // workgroups, rows of one
template <bool BF16, int NT>
__device__ __forceinline__ void clear_rows(const CombineBwdArgs& a, int per, uint32_t* s_bits) {
    const int tid = threadIdx.x, A = a.rows;
    const int lo = blockIdx.x * per, n = min(per, A - lo);
    for (int i = tid; i < (per + 31) / 32; i += NT) s_bits[i] = 0;
    __syncthreads();
    auto mark = [&](int p) __attribute__((always_inline)) {
        const uint32_t r = (uint32_t)p - (uint32_t)lo;
        if (r < (uint32_t)n) atomicOr(&s_bits[r >> 5], 1u << (r & 31));
    };
    const int head = min(A, (int)(-(reinterpret_cast<uintptr_t>(a.pos) >> 2) & 3)), nq = (A - head) / 4;
    const int4* q = reinterpret_cast<const int4*>(a.pos + head);
    for (int i0 = 0; i0 < nq; i0 += 8 * NT) {   // eight vectors of 4 in flight
        int4 p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * NT + tid;
            p[u] = i < nq ? q[i] : make_int4(-1, -1, -1, -1);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mark(p[u].x), mark(p[u].y), mark(p[u].z), mark(p[u].w);
    }
    if (tid < head) mark(a.pos[tid]);
    if (tid < A - head - 4 * nq) mark(a.pos[head + 4 * nq + tid]);
    __syncthreads();
    const int nv = a.H / (BF16 ? 8 : 4);
    for (int r = tid >> 6; r < n; r += NT / 64)
        if (!(s_bits[r >> 5] >> (r & 31) & 1))
            for (int v = tid & 63; v < nv; v += 64)
                __builtin_nontemporal_store(v4u_t{0, 0, 0, 0}, reinterpret_cast<v4u_t*>(a.deo) + (int64_t)(lo + r) * nv + v);
}

template <bool BF16, int G, bool DOUT>
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_combine_bwd(CombineBwdArgs a, int nclear, int per) {
    constexpr int RPB = G < 256 ? 256 / G : 1, CW = BF16 ? 8 : 4, NW = G / 64;
    __shared__ float s_dot[RPB][NW][8];
    if constexpr (DOUT) {
        __shared__ uint32_t s_bits[kClearRows / 32];
        if (blockIdx.x < nclear) return clear_rows<BF16, G * RPB>(a, per, s_bits);   // (uniform)
    }
    const int sub = threadIdx.x % G, r = threadIdx.x / G;
    const int64_t tt = (int64_t)(blockIdx.x - (DOUT ? nclear : 0)) * RPB + r;
    const bool on = tt < a.T;           // (the barriers below are for every thread)
    const int64_t t = on ? tt : a.T - 1;
    const int nv = on ? a.H / CW : 0;
    const int A = a.rows;
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        int64_t p[8];
        float wj[8], dot[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int64_t f = t * a.k + j0 + u;
            p[u] = j0 + u < a.k ? a.pos[f] : -1;
            if (p[u] >= A) p[u] = -1;
            wj[u] = DOUT && p[u] >= 0 ? a.wt[f] : 0.f;
            dot[u] = 0.f;
        }
        for (int v = sub; v < nv; v += G) {
            v4u_t e[8];
            if (a.dwt) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    e[u] = v4u_t{0, 0, 0, 0};
                    if (p[u] >= 0)
                        e[u] = __builtin_nontemporal_load(reinterpret_cast<const v4u_t*>(a.eo) + p[u] * (a.H / CW) + v);
                }
            }
            float d[8];
            if constexpr (BF16) {
                unpack8(*reinterpret_cast<const uint4*>(a.dy + t * a.H + v * 8), d);
            } else {
                const uint2 x = *reinterpret_cast<const uint2*>(a.dy + t * a.H + v * 4);
                d[0] = __uint_as_float(x.x << 16), d[1] = __uint_as_float(x.x & 0xFFFF0000u);
                d[2] = __uint_as_float(x.y << 16), d[3] = __uint_as_float(x.y & 0xFFFF0000u);
            }
            if (a.dwt) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int i = 0; i < CW; ++i) {
                        float x;
                        if constexpr (BF16)
                            x = i & 1 ? __uint_as_float(e[u][i / 2] & 0xFFFF0000u) : __uint_as_float(e[u][i / 2] << 16);
                        else
                            x = __uint_as_float(e[u][i]);
                        dot[u] = fmaf(d[i], x, dot[u]);
                    }
            }
            if constexpr (DOUT) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (p[u] >= 0) {
                        v4u_t o;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (BF16) o[i] = pack_bf16(wj[u] * d[2 * i], wj[u] * d[2 * i + 1]);
                            else o[i] = __float_as_uint(wj[u] * d[i]);
                        }
                        __builtin_nontemporal_store(o, reinterpret_cast<v4u_t*>(a.deo) + p[u] * (a.H / CW) + v);
                    }
                }
            }
        }
        if (a.dwt) {
#pragma unroll
            for (int u = 0; u < 8; ++u) dot[u] = wave_sum(dot[u]);
            if constexpr (NW > 1) {
                if (j0) __syncthreads();   // the previous slots' sums have been read
                if ((sub & 63) == 0) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) s_dot[r][sub >> 6][u] = dot[u];
                }
                __syncthreads();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    dot[u] = s_dot[r][0][u];
#pragma unroll
                    for (int w = 1; w < NW; ++w) dot[u] += s_dot[r][w][u];
                }
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (on && sub == u && j0 + u < a.k) a.dwt[t * a.k + j0 + u] = p[u] >= 0 ? dot[u] : 0.f;
        }
    }
}

// Zeros for all of dexpert_out, before the rows that are named.
__global__ __launch_bounds__(256) void k_zero(v4u_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        __builtin_nontemporal_store(v4u_t{0, 0, 0, 0}, p + i);
}

template <bool BF16, int G>
static void run_combine_bwd(const CombineBwdArgs& args, hipStream_t st) {
    constexpr int RPB = G < 256 ? 256 / G : 1;
    CombineBwdArgs a = args;
    const int64_t A = a.rows;
    int nclear = 0, per = 0;
    // In the kernel itself (16384 x 8 x 4096 bf16 over three sets of inputs: 457 us, without clearing 455, a fill
    // before it 598 to 432 on one set; 32 x 8 x 2816: 5.6, 5.7 and 7.5; with 256 workgroups 461, with 64 456 but 326
    // instead of 313 where seven of eight are dropped).  Zeros first where reading all entries 128 times takes
    // longer than writing the rows (16384 x 8 x 128 bf16: 42 us, in the kernel 46; 65536 x 8 x 256: 191 and 187) or
    // LDS holds too few marks.
    if (a.clear && A <= (int64_t)kClearMost * kClearRows && (A <= (1 << 16) || a.H * (BF16 ? 2 : 4) >= 512)) {
        per = (int)std::max<int64_t>(64, ceil_div(A, kClearMost));
        nclear = (int)ceil_div(A, per);
    } else if (a.clear) {
        hipLaunchKernelGGL(k_zero, dim3(2048), dim3(256), 0, st, static_cast<v4u_t*>(a.deo), A * a.H / (BF16 ? 8 : 4));
    }
    for (int64_t t = 0; t < args.T; t += launch_rows(G)) {
        a.T = (int)std::min<int64_t>(args.T - t, launch_rows(G));
        a.dy = args.dy + t * a.H;
        a.pos = args.pos + t * a.k;
        if (args.wt) a.wt = args.wt + t * a.k;
        if (args.dwt) a.dwt = args.dwt + t * a.k;
        const dim3 grid((unsigned)ceil_div(a.T, RPB) + nclear), block(G * RPB);
        if (a.deo) hipLaunchKernelGGL((k_combine_bwd<BF16, G, true>), grid, block, 0, st, a, nclear, per);
        else hipLaunchKernelGGL((k_combine_bwd<BF16, G, false>), grid, block, 0, st, a, 0, 0);
        nclear = 0;   // (the first launch reads all entries)
    }
}

// Threads per token, by its nv vectors.  Few tokens: as many as there are vectors, one round of loads
// (64 x 4096 bf16: 5.4 us with 512 threads, 6.1 with 256, 15 with 64; 1024 have no registers for eight
// rows in flight), but no more than 256 where there are more tokens than CUs (512 x 7168: 27 us, 512
// threads 30).  Otherwise fewer where rows are short, for more rounds in flight from fewer workgroups: 128
// (2047 x 768 float32: 11.3 us, 256 threads 14.8; 1100 x 4000 bf16: 17.8, 64 threads 23.6), and a wave where
// every CU has 16 tokens (16384 x 768 bf16: 45.9 us, 128 threads 52.6; 4096 x 1024: 9.9 and 11.9); 256 from
// 512 vectors on (4096 x 4096 bf16 with dexpert_out: 108 us, 64 threads 138).  The choice does not look at
// dexpert_out: the weights' gradient has the same bits with and without it.
template <bool BF16>
static void pick_combine_bwd(const CombineBwdArgs& a, hipStream_t st) {
    const int nv = a.H / (BF16 ? 8 : 4);
    if (nv <= 64 || (a.T >= 4096 && nv < 512)) run_combine_bwd<BF16, 64>(a, st);
    else if (nv <= 128 || (a.T >= 1024 && nv < 512)) run_combine_bwd<BF16, 128>(a, st);
    else if (a.T <= 256 && nv > 256) run_combine_bwd<BF16, 512>(a, st);
    else run_combine_bwd<BF16, 256>(a, st);
}

hipError_t launch_combine_backward(const CombineBwdArgs& a, hipStream_t st) {
    if (a.bf16) pick_combine_bwd<true>(a, st);
    else pick_combine_bwd<false>(a, st);
    return hipGetLastError();
}

}  // namespace moe
