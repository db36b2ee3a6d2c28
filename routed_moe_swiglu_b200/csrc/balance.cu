// balance.cu -- training operators of the router: the balance loss and the z
// loss with per-expert route counts (moe_balance_loss), and the gradient of
// the logits (moe_route_backward).
//
// Mathematics.  A token t counts when it is live, lies in a sequence, is not
// masked and has a logit above -infinity.  With p_t = softmax(l_t), lse_t the
// log of its denominator, T_s the counted tokens of sequence s, T their sum
// and S' the sequences with T_s > 0:
//   counts[s,e]    = routes of counted tokens of s to expert e
//   prob_sums[s,e] = sum of p_t[e] over the counted tokens of s
//   a_s            = balance_coef * E / (S' * k * T_s^2)
//   losses[0]      = sum_s a_s * sum_e counts[s,e] * prob_sums[s,e]
//                    (the mean over sequences of E * <share of routes, mean p>)
//   losses[1]      = z_coef / T * sum_t lse_t^2
//   dlogits[t,e]   = p_t[e] * (g0 a_s (c_e - <c, p_t>) + g1 2 z_coef / T lse_t)
//                    + (e chosen as route j) w_j (d_j - <w, d>)
// with c = counts[s,:], w the chosen experts' renormalised probabilities and d
// their gradients: the two parts of a softmax's gradient, over all E and over
// the chosen k.
//
// Work split.  A group of L lanes holds one token's E logits, V per lane, in
// registers: the softmax is one pass over the logits.  A block takes a
// contiguous run of tokens and walks the sequences it meets; each (block b,
// sequence s) pair it meets writes its sums to slot b + s.  Blocks and
// sequences both advance along the tokens, so no two pairs share a slot, and
// the second kernel adds a sequence's slots in block order: no float atomics,
// the same bits every run.
#include <cmath>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kBalSumRows = kBalWarps / 2;  // rows of sums in shared memory: half of the warps add the other half's
constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kFinThreads = 1024;
constexpr int kFinWarps = kFinThreads / 32;
constexpr int kFinCols = 32;  // columns of an item of the finish: a warp per slot row, a lane per column
constexpr float kLog2e = 1.4426950408889634f;

struct BalanceArgs {
    const float* logits;
    const int* ids;
    const uint8_t* mask;
    const int* seq_off;  // null: one sequence, all live tokens
    const int* live;
    int max_live, E, k, num_seqs, blocks;
    float balance_coef, z_coef;
    int* counts;
    float* prob_sums;
    float* lse;
    float* losses;
    float* grad_scales;
    // workspace: one row per slot, then per sequence
    float* slot_p;      // [slots][E]
    int* slot_c;        // [slots][E]
    float* slot_z;      // [slots]
    int* slot_n;        // [slots]
    float* seq_dot;     // [num_seqs][col blocks]
    float* seq_z;       // [num_seqs]
    int* seq_n;         // [num_seqs]
    unsigned* ticket;
};

__device__ __forceinline__ int seq_begin(const int* off, int s, int n) {
    if (off == nullptr) return s == 0 ? 0 : n;
    const int o = __ldg(off + s);
    return o < 0 ? 0 : (o > n ? n : o);
}
// The sequence that holds token t: the first s with off[s + 1] > t (num_seqs when none has).
__device__ __forceinline__ int find_seq(const int* off, int num_seqs, int t) {
    if (off == nullptr) return 0;
    int lo = 0, hi = num_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid + 1) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Column of value v of group lane gl: 16-byte runs (kVec) or single values.
template <int L, bool kVec>
__device__ __forceinline__ int col_of(int v, int gl) {
    return kVec ? (v >> 2) * (4 * L) + gl * 4 + (v & 3) : v * L + gl;
}
// V values of a row per lane; columns from E on, and all of an absent row, read as `fill`.
template <int L, int V, bool kVec>
__device__ __forceinline__ void load_row(const float* row, int E, int gl, bool have, float fill, float (&x)[V]) {
    if (kVec) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const int c = q * (4 * L) + gl * 4;  // E % 4 == 0: a run is in or out
            float4 f = make_float4(fill, fill, fill, fill);
            if (have && c < E) f = __ldg(reinterpret_cast<const float4*>(row + c));
            x[4 * q] = f.x;
            x[4 * q + 1] = f.y;
            x[4 * q + 2] = f.z;
            x[4 * q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * L + gl;
            x[v] = have && c < E ? __ldg(row + c) : fill;
        }
    }
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 0 for -infinity
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct StatsShared {
    float z[kBalWarps];
    int n[kBalWarps];
};
struct FinishShared {
    float p[kFinWarps][kFinCols + 1];
    int c[kFinWarps][kFinCols + 1];
    double a[kFinWarps], b[kFinWarps];
    int i[kFinWarps], j[kFinWarps];
};

// Sums of this block's tokens, one slot for each sequence it meets.  The next token's row is on
// its way while this one's softmax is computed.
template <int L, int V, bool kVec>
__device__ __forceinline__ void balance_stats(const BalanceArgs& a, int n, float* s_sum, int* s_cnt,
                                              StatsShared& sh) {
    const int E = a.E, k = a.k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (L - 1);
    constexpr int kGroups = 32 / L;  // tokens a warp holds at once
    const int chunk = (n + a.blocks - 1) / a.blocks;
    const int c0 = min(n, (int)blockIdx.x * chunk), c1 = min(n, c0 + chunk);
    if (c0 >= c1) return;
    // tokens before the first and behind the last sequence count for nothing
    const int first = seq_begin(a.seq_off, 0, n), last = seq_begin(a.seq_off, a.num_seqs, n);
    for (int t = c0 + threadIdx.x; t < c1; t += kBalThreads)
        if (t < first || t >= last) a.lse[t] = -INFINITY;

    for (int s = find_seq(a.seq_off, a.num_seqs, c0); s < a.num_seqs; ++s) {
        const int sb = seq_begin(a.seq_off, s, n);
        if (sb >= c1) break;
        const int t_lo = max(sb, c0), t_hi = min(seq_begin(a.seq_off, s + 1, n), c1);
        if (t_lo >= t_hi) continue;
        for (int e = threadIdx.x; e < E; e += kBalThreads) s_cnt[e] = 0;
        __syncthreads();
        float acc[V], next[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.0f;
        float z = 0.0f;
        int cnt = 0;
        constexpr int kStep = kBalWarps * kGroups;
        int t = t_lo + warp * kGroups + lane / L;
        auto kept = [&](int tt) { return tt < t_hi && (a.mask == nullptr || __ldg(a.mask + tt) != 0); };
        bool have_next = kept(t);
        load_row<L, V, kVec>(a.logits + (size_t)t * E, E, gl, have_next, -INFINITY, next);
        for (int tw = t_lo + warp * kGroups; tw < t_hi; tw += kStep, t += kStep) {
            const bool have = have_next;
            float x[V];
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = next[v];
            have_next = kept(t + kStep);
            load_row<L, V, kVec>(a.logits + (size_t)(t + kStep) * E, E, gl, have_next, -INFINITY, next);
            float mx = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) mx = fmaxf(mx, x[v]);
            mx = group_max<L>(mx);
            if (mx == -INFINITY) mx = 0.0f;  // all -infinity: the sum below is 0 (NaN with a NaN logit)
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v] = exp2_approx((x[v] - mx) * kLog2e);  // the difference first: rows near the type's bounds
                sum += x[v];
            }
            sum = group_sum<L>(sum);
            const bool counted = have && sum != 0.0f;  // true for NaN: it shows in the losses
            const float inv = counted ? __frcp_rn(sum) : 0.0f;
            const float lse = counted ? mx + logf(sum) : -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] = fmaf(x[v], inv, acc[v]);  // 0 * 0 where it does not count
            if (t < t_hi && gl == 0) {
                a.lse[t] = lse;
                if (counted) {
                    z += lse * lse;
                    ++cnt;
                }
            }
            if (counted)
                for (int j = gl; j < k; j += L) {
                    const int id = __ldg(a.ids + (size_t)t * k + j);
                    if (id >= 0 && id < E) atomicAdd(&s_cnt[id], 1);  // integers: any order
                }
        }
        // groups of the warp, then warps in order: the upper half's rows first go through shared
        // memory to the lower half, which adds them and leaves its rows there
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int o = L; o < 32; o <<= 1) acc[v] += __shfl_xor_sync(0xffffffffu, acc[v], o);
        z = group_sum<32>(z);
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) {
            sh.z[warp] = z;
            sh.n[warp] = cnt;
        }
        float* mine = s_sum + (warp & (kBalSumRows - 1)) * E;
        if (warp >= kBalSumRows && lane < L)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = col_of<L, kVec>(v, gl);
                if (c < E) mine[c] = acc[v];
            }
        __syncthreads();
        if (warp < kBalSumRows && lane < L)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = col_of<L, kVec>(v, gl);
                if (c < E) mine[c] += acc[v];
            }
        __syncthreads();
        const size_t slot = (size_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            float p = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalSumRows; ++w) p += s_sum[w * E + e];
            a.slot_p[slot * E + e] = p;
            a.slot_c[slot * E + e] = s_cnt[e];
        }
        if (threadIdx.x == 0) {
            float zs = 0.0f;
            int ns = 0;
            for (int w = 0; w < kBalWarps; ++w) {
                zs += sh.z[w];
                ns += sh.n[w];
            }
            a.slot_z[slot] = zs;
            a.slot_n[slot] = ns;
        }
        __syncthreads();
    }
}

// Adds the slots of a sequence for 32 experts; `item` is one (sequence, 32 experts) of the
// num_seqs * ceil(E / 32) that `size` blocks share.
__device__ __forceinline__ void finish_items(const BalanceArgs& a, int n, int rank, int size, FinishShared& sh) {
    const int E = a.E, S = a.num_seqs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int col_blocks = (E + kFinCols - 1) / kFinCols;
    const int chunk = (n + a.blocks - 1) / a.blocks;
    for (int it = rank; it < S * col_blocks; it += size) {
        const int s = it / col_blocks, cb = it - s * col_blocks;
        const int e = cb * kFinCols + lane;
        const int sb = seq_begin(a.seq_off, s, n), se = seq_begin(a.seq_off, s + 1, n);
        // blocks that met the sequence
        const int b0 = se > sb ? sb / chunk : 0, b1 = se > sb ? (se - 1) / chunk + 1 : 0;
        float p = 0.0f;
        int c = 0;
        if (e < E)
#pragma unroll 8
            for (int b = b0 + warp; b < b1; b += warps) {
                const size_t at = (size_t)(b + s) * E + e;
                p += __ldcg(a.slot_p + at);
                c += __ldcg(a.slot_c + at);
            }
        sh.p[warp][lane] = p;
        sh.c[warp][lane] = c;
        __syncthreads();
        if (warp == 0) {
            p = 0.0f;
            c = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) {
                p += sh.p[w][lane];
                c += sh.c[w][lane];
            }
            if (e < E) {
                a.prob_sums[(size_t)s * E + e] = p;
                a.counts[(size_t)s * E + e] = c;
            }
            const float dot = group_sum<32>(e < E ? (float)c * p : 0.0f);
            if (lane == 0) a.seq_dot[it] = dot;
        }
        if (warp == 1 && cb == 0) {
            float z = 0.0f;
            int m = 0;
            for (int b = b0 + lane; b < b1; b += 32) {
                z += __ldcg(a.slot_z + b + s);
                m += __ldcg(a.slot_n + b + s);
            }
            z = group_sum<32>(z);
            m = __reduce_add_sync(0xffffffffu, m);
            if (lane == 0) {
                a.seq_z[s] = z;
                a.seq_n[s] = m;
            }
        }
        __syncthreads();
    }
}

// One block: S', T and the z sum, then the sequences' factors and the losses.  Each thread takes
// every blockDim-th sequence, and the threads' sums are added in a fixed order.
__device__ __forceinline__ void finish_total(const BalanceArgs& a, FinishShared& sh) {
    const int S = a.num_seqs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int col_blocks = (a.E + kFinCols - 1) / kFinCols;
    int filled = 0, total = 0;
    double z = 0.0;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int m = __ldcg(a.seq_n + s);
        filled += m > 0;
        total += m;
        z += (double)__ldcg(a.seq_z + s);
    }
    filled = __reduce_add_sync(0xffffffffu, filled);
    total = __reduce_add_sync(0xffffffffu, total);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lane == 0) {
        sh.i[warp] = filled;
        sh.j[warp] = total;
        sh.b[warp] = z;
    }
    __syncthreads();
    filled = total = 0;
    z = 0.0;
    const int used = min(warps, (S + 31) / 32);  // the other warps' sums are 0
    for (int w = 0; w < used; ++w) {
        filled += sh.i[w];
        total += sh.j[w];
        z += sh.b[w];
    }
    double loss = 0.0;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const double m = (double)__ldcg(a.seq_n + s);
        const double as = m > 0.0 ? (double)a.balance_coef * a.E / ((double)filled * a.k * m * m) : 0.0;
        double dot = 0.0;
        for (int cb = 0; cb < col_blocks; ++cb) dot += (double)__ldcg(a.seq_dot + (size_t)s * col_blocks + cb);
        if (m > 0.0) loss += as * dot;
        a.grad_scales[s] = (float)as;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    if (lane == 0) sh.a[warp] = loss;
    __syncthreads();
    if (threadIdx.x == 0) {
        loss = 0.0;
        for (int w = 0; w < used; ++w) loss += sh.a[w];
        const double zt = total > 0 ? (double)a.z_coef / total : 0.0;
        a.losses[0] = (float)loss;
        a.losses[1] = (float)(total > 0 ? zt * z : 0.0);
        a.grad_scales[S] = (float)(2.0 * zt);
    }
}

// kOne: the grid is one cluster, which meets in its own barrier between the sums, the finish and
// the totals; else balance_finish_kernel does the rest.
template <int L, int V, bool kVec, bool kOne>
__global__ void __launch_bounds__(kBalThreads, 1) balance_stats_kernel(const BalanceArgs a) {
    extern __shared__ float s_bal[];  // [kBalSumRows][E] sums, then [E] counts
    __shared__ StatsShared sh;
    pdl_trigger();
    pdl_wait();
    const int n = clamp_live(a.live, a.max_live);
    if (!kOne && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    balance_stats<L, V, kVec>(a, n, s_bal, reinterpret_cast<int*>(s_bal + kBalSumRows * a.E), sh);
    if constexpr (kOne) {
        __shared__ FinishShared fin;
        cluster_sync();  // the slots of every block are written
        finish_items(a, n, blockIdx.x, gridDim.x, fin);
        cluster_sync();
        if (blockIdx.x == 0) finish_total(a, fin);
    }
}

__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalanceArgs a) {
    __shared__ FinishShared fin;
    __shared__ int s_last;
    pdl_trigger();
    pdl_wait();
    finish_items(a, clamp_live(a.live, a.max_live), blockIdx.x, gridDim.x, fin);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1 ? 1 : 0;
    __syncthreads();
    if (!s_last) return;  // the last block to finish has every sequence's sums
    __threadfence();
    finish_total(a, fin);
}

struct RouteGradArgs {
    const float* logits;
    const int* ids;
    const int* live;
    int max_live, E, k, num_seqs, blocks;
    const float* lse;
    const int* counts;
    const float* grad_scales;
    const float* grad_losses;  // null: 1, 1
    const float* probs;        // null with dprobs
    const float* dprobs;       // null: no chosen part
    const int* seq_off;
    float* dlogits;
};

// A group of lanes per token, as the forward: the losses' part in registers; the chosen part
// is added to the row in shared memory, in route order (an expert named twice gets both adds in
// that order), from where the whole row leaves in wide stores.  Route j of a token belongs to
// lane j % L of its group.
template <int L, int V, bool kVec>
__global__ void __launch_bounds__(kGradThreads) route_backward_kernel(const RouteGradArgs a) {
    extern __shared__ __align__(16) float s_row_all[];
    constexpr int kGroups = 32 / L;
    constexpr int kSlots = (kMaxTopK + L - 1) / L;  // routes of a lane
    pdl_trigger();
    pdl_wait();
    const int E = a.E, k = a.k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (L - 1), g = warp * kGroups + lane / L;
    const int pitch = (E + 3) & ~3;
    float* s_row = s_row_all + (size_t)g * pitch;
    const int n = clamp_live(a.live, a.max_live);
    const bool has_loss = a.counts != nullptr;
    const float g0 = a.grad_losses != nullptr ? __ldg(a.grad_losses) : 1.0f;
    const float g1 = a.grad_losses != nullptr ? __ldg(a.grad_losses + 1) : 1.0f;
    const float zs = has_loss ? g1 * __ldg(a.grad_scales + a.num_seqs) : 0.0f;
    int s_lo = 0, s_hi = 0;  // tokens of the sequence whose counts are in cnt
    float cnt[V], as = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) cnt[v] = 0.0f;

    const int chunk = (n + a.blocks - 1) / a.blocks;
    const int c0 = min(n, (int)blockIdx.x * chunk), c1 = min(n, c0 + chunk);
    constexpr int kStep = kGradWarps * kGroups;
    int t = c0 + warp * kGroups + lane / L;
    auto lse_of = [&](int tt) {
        return tt < c1 ? (a.lse != nullptr ? __ldg(a.lse + tt) : 0.0f) : -INFINITY;
    };
    float lse_next = lse_of(t);
    float next[V];
    if (has_loss) load_row<L, V, kVec>(a.logits + (size_t)t * E, E, gl, t < c1, -INFINITY, next);
    for (int tw = c0 + warp * kGroups; tw < c1; tw += kStep, t += kStep) {
        const bool in = t < c1;
        const float lse = lse_next;
        const bool counted = lse != -INFINITY;  // true for NaN
        float x[V];
        if (has_loss) {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = next[v];
        }
        // the next token's row and this one's routes are on their way meanwhile
        lse_next = lse_of(t + kStep);
        if (has_loss)
            load_row<L, V, kVec>(a.logits + (size_t)(t + kStep) * E, E, gl, t + kStep < c1, -INFINITY, next);
        int id[kSlots];
        float w[kSlots], d[kSlots];
        if (a.dprobs != nullptr) {
#pragma unroll
            for (int r = 0; r < kSlots; ++r) {
                const int j = r * L + gl;
                const bool on = counted && j < k;
                id[r] = on ? __ldg(a.ids + (size_t)t * k + j) : -1;
                w[r] = on ? __ldg(a.probs + (size_t)t * k + j) : 0.0f;
                d[r] = on ? __ldg(a.dprobs + (size_t)t * k + j) : 0.0f;
                if (id[r] < 0 || id[r] >= E) {
                    id[r] = -1;
                    w[r] = d[r] = 0.0f;
                }
            }
        }
        if (has_loss) {
            if (counted && (t < s_lo || t >= s_hi)) {
                int s = find_seq(a.seq_off, a.num_seqs, t);
                s = s < a.num_seqs ? s : a.num_seqs - 1;
                s_lo = seq_begin(a.seq_off, s, n);
                s_hi = seq_begin(a.seq_off, s + 1, n);
                as = g0 * __ldg(a.grad_scales + s);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = col_of<L, kVec>(v, gl);
                    cnt[v] = c < E ? (float)__ldg(a.counts + (size_t)s * E + c) : 0.0f;
                }
            }
            // p from the row's own maximum and sum: lse has lost the sum where it is large
            float mx = -INFINITY;
#pragma unroll
            for (int v = 0; v < V; ++v) mx = fmaxf(mx, x[v]);
            mx = group_max<L>(mx);
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v] = exp2_approx((x[v] - mx) * kLog2e);
                sum += x[v];
                dot = fmaf(cnt[v], x[v], dot);
            }
            sum = group_sum<L>(sum);
            dot = group_sum<L>(dot);
            const float inv = __frcp_rn(sum);
            const float base = fmaf(zs, lse, -as * (dot * inv));  // as * (c - <c, p>) + zs * lse
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = counted ? x[v] * inv * fmaf(as, cnt[v], base) : 0.0f;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = 0.0f;
        }
        if (a.dprobs != nullptr) {
            float wd = 0.0f;
#pragma unroll
            for (int r = 0; r < kSlots; ++r) wd = fmaf(w[r], d[r], wd);
            wd = group_sum<L>(wd);
            if (kVec) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const int c = q * (4 * L) + gl * 4;
                    if (c < E)
                        *reinterpret_cast<float4*>(s_row + c) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2],
                                                                            x[4 * q + 3]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v * L + gl < E) s_row[v * L + gl] = x[v];
            }
            __syncwarp();
            // routes of different experts add in any order; an expert named twice, or more routes
            // than lanes: one route after another
            bool apart = k <= L;
            if (apart) {
                const unsigned key = id[0] >= 0 ? (unsigned)(id[0] * kGroups + lane / L) : 0x80000000u + lane;
                apart = __all_sync(0xffffffffu, __popc(__match_any_sync(0xffffffffu, key)) == 1);
            }
            if (apart) {
                if (id[0] >= 0) s_row[id[0]] += w[0] * (d[0] - wd);
                __syncwarp();
            } else {
#pragma unroll
                for (int r = 0; r < kSlots; ++r)
                    for (int j = r * L; j < min(k, r * L + L); ++j) {
                        if (gl == j - r * L && id[r] >= 0) s_row[id[r]] += w[r] * (d[r] - wd);
                        __syncwarp();
                    }
            }
            if (kVec) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const int c = q * (4 * L) + gl * 4;
                    if (c < E) {
                        const float4 f = *reinterpret_cast<const float4*>(s_row + c);
                        x[4 * q] = f.x;
                        x[4 * q + 1] = f.y;
                        x[4 * q + 2] = f.z;
                        x[4 * q + 3] = f.w;
                    }
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v * L + gl < E) x[v] = s_row[v * L + gl];
            }
            __syncwarp();
        }
        if (in) {
            float* out = a.dlogits + (size_t)t * E;
            if (kVec) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const int c = q * (4 * L) + gl * 4;
                    if (c < E)
                        *reinterpret_cast<float4*>(out + c) = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2],
                                                                          x[4 * q + 3]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v * L + gl < E) out[v * L + gl] = x[v];
            }
        }
    }
}

// Tokens that a warp holds at once (32 / L, as by_width picks L).
int tokens_per_warp(int E) { return E <= 16 ? 8 : E <= 128 ? 4 : E <= 256 ? 2 : 1; }

int blocks_for(long long max_live, int tokens, long long cap) {
    const long long want = (max_live + tokens - 1) / tokens;
    return (int)(want < 1 ? 1 : (want > cap ? cap : want));
}

// Up to this many blocks are one cluster (of a power of two) and one launch.
constexpr int kClusterBlocks = 8;
// The workspace has rows for the largest grid any device may ask for.
constexpr int kMaxBalBlocks = 256;

// Blocks of the sums: one pass of each block's warps at least, `cap` at most.
int balance_blocks(long long max_live, int E, long long cap) {
    const int b = blocks_for(max_live, kBalWarps * tokens_per_warp(E), cap);
    if (b > kClusterBlocks) return b;
    return b > 4 ? 8 : b > 2 ? 4 : b;
}

struct BalanceLayout {
    size_t p, c, z, n, dot, sz, sn, ticket, total;
};
BalanceLayout balance_layout(const moe_plan* plan, int num_seqs) {
    const size_t E = (size_t)plan->d.num_experts, S = (size_t)num_seqs;
    const int b = balance_blocks(plan->max_live, plan->d.num_experts, kMaxBalBlocks);
    const size_t slots = (size_t)b + S;
    BalanceLayout l;
    size_t off = 0;
    auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~size_t(255);
        return at;
    };
    l.p = take(slots * E * 4);
    l.c = take(slots * E * 4);
    l.z = take(slots * 4);
    l.n = take(slots * 4);
    l.dot = take(S * ((E + kFinCols - 1) / kFinCols) * 4);
    l.sz = take(S * 4);
    l.sn = take(S * 4);
    l.ticket = take(4);
    l.total = off;
    return l;
}

bool ptr_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The lanes and values per lane of a token: the smallest pair that holds E.
template <template <int, int, bool> class Launch, class Args>
cudaError_t by_width(int E, bool vec, const Args& a, cudaStream_t s) {
#define MOE_BY_WIDTH(L, V) return vec ? Launch<L, V, true>::go(a, s) : Launch<L, V, false>::go(a, s)
    if (E <= 16) MOE_BY_WIDTH(4, 4);
    if (E <= 32) MOE_BY_WIDTH(8, 4);
    if (E <= 64) MOE_BY_WIDTH(8, 8);
    if (E <= 128) MOE_BY_WIDTH(8, 16);
    if (E <= 256) MOE_BY_WIDTH(16, 16);
    if (E <= 512) MOE_BY_WIDTH(32, 16);
    MOE_BY_WIDTH(32, 32);
#undef MOE_BY_WIDTH
}

template <int L, int V, bool kVec>
struct LaunchStats {
    static cudaError_t go(const BalanceArgs& a, cudaStream_t s) {
        const size_t smem = (size_t)(kBalSumRows + 1) * a.E * 4;  // at most 36 KB
        if (a.blocks > kClusterBlocks)
            return launch_dependent(balance_stats_kernel<L, V, kVec, false>, dim3(a.blocks), dim3(kBalThreads), smem, s,
                                    a);
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)a.blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(a.blocks);
        cfg.blockDim = dim3(kBalThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        const cudaError_t err = cudaLaunchKernelEx(&cfg, balance_stats_kernel<L, V, kVec, true>, a);
        return err != cudaSuccess ? err : cudaGetLastError();
    }
};
template <int L, int V, bool kVec>
struct LaunchBackward {
    static cudaError_t go(const RouteGradArgs& a, cudaStream_t s) {
        const size_t smem = a.dprobs != nullptr ? (size_t)kGradWarps * (32 / L) * ((a.E + 3) & ~3) * 4 : 0;  // <= 32 KB
        return launch_dependent(route_backward_kernel<L, V, kVec>, dim3(a.blocks), dim3(kGradThreads), smem, s, a);
    }
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_bytes(const moe_plan* plan, int num_seqs) {
    if (plan == nullptr || num_seqs < 1 || num_seqs > MOE_MAX_SEQS) return 0;
    return balance_layout(plan, num_seqs).total;
}

moe_status moe_balance_loss(const moe_plan* plan, const float* logits, const int* ids, const uint8_t* token_mask,
                            const int* seq_offsets, int num_seqs, float balance_coef, float z_coef,
                            const int* live_count_dev, int* counts, float* prob_sums, float* lse, float* losses,
                            float* grad_scales, void* workspace, size_t ws_bytes, void* stream) {
    if (plan == nullptr || logits == nullptr || ids == nullptr || live_count_dev == nullptr || counts == nullptr ||
        prob_sums == nullptr || lse == nullptr || losses == nullptr || grad_scales == nullptr || workspace == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (num_seqs < 1 || (seq_offsets == nullptr && num_seqs != 1)) return MOE_ERR_INVALID_ARG;
    if (num_seqs > MOE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
    if (!std::isfinite(balance_coef) || !std::isfinite(z_coef)) return MOE_ERR_INVALID_ARG;
    const BalanceLayout l = balance_layout(plan, num_seqs);
    if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!ptr_aligned(workspace, 256)) return MOE_ERR_ALIGNMENT;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    BalanceArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.mask = token_mask;
    a.seq_off = seq_offsets;
    a.live = live_count_dev;
    a.max_live = (int)plan->max_live;
    a.E = plan->d.num_experts;
    a.k = plan->d.top_k;
    a.num_seqs = num_seqs;
    a.blocks = balance_blocks(plan->max_live, a.E, num_sms() < kMaxBalBlocks ? num_sms() : kMaxBalBlocks);
    a.balance_coef = balance_coef;
    a.z_coef = z_coef;
    a.counts = counts;
    a.prob_sums = prob_sums;
    a.lse = lse;
    a.losses = losses;
    a.grad_scales = grad_scales;
    a.slot_p = reinterpret_cast<float*>(ws + l.p);
    a.slot_c = reinterpret_cast<int*>(ws + l.c);
    a.slot_z = reinterpret_cast<float*>(ws + l.z);
    a.slot_n = reinterpret_cast<int*>(ws + l.n);
    a.seq_dot = reinterpret_cast<float*>(ws + l.dot);
    a.seq_z = reinterpret_cast<float*>(ws + l.sz);
    a.seq_n = reinterpret_cast<int*>(ws + l.sn);
    a.ticket = reinterpret_cast<unsigned*>(ws + l.ticket);
    const bool vec = a.E % 4 == 0 && ptr_aligned(logits, 16);
    cudaError_t e = by_width<LaunchStats>(a.E, vec, a, s);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    if (a.blocks <= kClusterBlocks) return MOE_OK;
    const long long items = (long long)num_seqs * ((a.E + kFinCols - 1) / kFinCols);
    const long long cap = (long long)num_sms() * 2;
    e = launch_dependent(balance_finish_kernel, dim3((unsigned)(items < cap ? items : cap)), dim3(kFinThreads), 0, s,
                         a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_route_backward(const moe_plan* plan, const float* logits, const int* ids, const float* lse,
                              const int* counts, const float* grad_scales, const float* grad_losses,
                              const float* probs, const float* dprobs, const int* seq_offsets, int num_seqs,
                              const int* live_count_dev, float* dlogits, void* stream) {
    if (plan == nullptr || live_count_dev == nullptr || dlogits == nullptr) return MOE_ERR_INVALID_ARG;
    const bool has_loss = counts != nullptr;
    // the losses' part needs all of its inputs, the chosen part all of its own, and one is there
    if (has_loss != (grad_scales != nullptr)) return MOE_ERR_INVALID_ARG;
    if (has_loss && (logits == nullptr || lse == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!has_loss && grad_losses != nullptr) return MOE_ERR_INVALID_ARG;
    if ((probs != nullptr) != (dprobs != nullptr) || (dprobs != nullptr && ids == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!has_loss && dprobs == nullptr) return MOE_ERR_INVALID_ARG;
    if (num_seqs < 1 || (seq_offsets == nullptr && num_seqs != 1)) return MOE_ERR_INVALID_ARG;
    if (num_seqs > MOE_MAX_SEQS) return MOE_ERR_UNSUPPORTED;
    RouteGradArgs a{};
    a.logits = logits;
    a.ids = ids;
    a.live = live_count_dev;
    a.max_live = (int)plan->max_live;
    a.E = plan->d.num_experts;
    a.k = plan->d.top_k;
    a.num_seqs = num_seqs;
    a.blocks = blocks_for(plan->max_live, kGradWarps * tokens_per_warp(a.E), (long long)num_sms() * 4);
    a.lse = lse;
    a.counts = counts;
    a.grad_scales = grad_scales;
    a.grad_losses = grad_losses;
    a.probs = probs;
    a.dprobs = dprobs;
    a.seq_off = seq_offsets;
    a.dlogits = dlogits;
    const bool vec = a.E % 4 == 0 && (logits == nullptr || ptr_aligned(logits, 16)) && ptr_aligned(dlogits, 16);
    const cudaError_t e = by_width<LaunchBackward>(a.E, vec, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
