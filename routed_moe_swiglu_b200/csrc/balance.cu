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
// sequences both advance along the tokens, so no two pairs share a slot, and a
// finishing step adds a sequence's slots in block order: no float atomics, the
// same bits every run.  The warps of a block share the runs it meets, all at once:
// long ones in segments, short ones whole.  The rows come through a ring in shared
// memory that each lane fills for itself (cp.async), two rows ahead (one for more than
// 512 experts).
//
// What bounds it (B200).  Both launches read the logits and the gradient writes as
// much; with 65,536 tokens x 128 experts, k 8, 16 sequences (74 MB from and to memory
// when the gradient's read of the 34 MB of logits comes from L2, 11 us at the copy
// rate) the losses take 18.3 us, 5.5 of them the finishing kernel, and the gradient
// 18.6, where a plain copy of the same 34 MB takes 11.8.  Neither memory (26% and 24%
// of DRAM's rate in the profile) nor the issue slots (47% and 40%) are full: 16 warps
// an SM in the sums, 24 in the gradient (103 registers at this width) leave the chain
// of a row (its arrival, maximum, exponentials, sum) in the open.  Short batches are
// bound by the chain of launches and meetings, and by the sums' way through memory
// between them, a lone block's too: 64 tokens x 8 experts, one cluster and one launch,
// 6.7 us and the gradient 3.2; 4,099 x 128 in seven sequences 10.6 and 4.5; 3,001 x
// 1,000 15 and 10.
#include <climits>
#include <cmath>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;
constexpr int kCutRuns = kBalWarps / 2;     // runs of a block that can be shared by warps
template <int V>
constexpr int kRingOf = V <= 16 ? 3 : 2;    // rows of a lane group in flight or in use
constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
template <int V>
constexpr int kGradBlocks = V <= 8 ? 4 : V <= 16 ? 3 : 2;  // of an SM: the grid is one wave of them
constexpr int kFinThreads = 1024;
constexpr int kFinWarps = kFinThreads / 32;
constexpr int kFinBlocks = 8;               // of the finishing kernel where it is one cluster
constexpr int kFinGroup = 8;                // its warps that add an item's slots together
constexpr int kFinCols = 32;                // columns of an item of the finish
constexpr int kBatch = 8;                   // loads of the finish in flight
constexpr int kBadOffsets = 1 << 17;        // added to a count of sequences by each thread that found a decrease
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
    int* seq_n;         // [num_seqs]; -1 where the offsets decrease
    unsigned* ticket;   // zeroed by the sums' kernel, counted by the finishing one
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

// The same for a whole warp that asks for one token.
__device__ __forceinline__ int find_seq_warp(const int* off, int num_seqs, int t) {
    if (off == nullptr) return 0;
    int lo = 0, hi = num_seqs;
    while (hi - lo > 32) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid + 1) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int s = lo + (int)(threadIdx.x & 31);
    const unsigned past = __ballot_sync(0xffffffffu, s >= hi || __ldg(off + s + 1) > t);
    return past != 0u ? lo + __ffs(past) - 1 : hi;
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
// One row per lane group on its way into the lanes' own places of a ring slot: 16-byte runs, or
// single floats where rows do not start on 16 bytes.
template <int L, int V, bool kVec>
__device__ __forceinline__ void ring_request(float* slot, const float* row, int E, int gl, bool have) {
    const int lane = threadIdx.x & 31;
    if (have) {
        if (kVec) {
#pragma unroll
            for (int q = 0; q < V / 4; ++q) {
                const int c = q * (4 * L) + gl * 4;  // E % 4 == 0: a run is in or out
                if (c < E)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot + (q * 32 + lane) * 4)),
                                 "l"(row + c)
                                 : "memory");
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = v * L + gl;
                if (c < E)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot + v * 32 + lane)),
                                 "l"(row + c)
                                 : "memory");
            }
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kRing>
__device__ __forceinline__ void ring_wait() {  // the oldest of kRing - 1 requests is there
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
}
__device__ __forceinline__ void ring_drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// The lane's V values of a row, as the slot has them.
template <int V, bool kVec>
__device__ __forceinline__ void ring_read(const float* slot, float (&x)[V]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kVec) {
            if (v % 4 == 0) {
                const float4 f = *reinterpret_cast<const float4*>(slot + (v / 4 * 32 + lane) * 4);
                x[v] = f.x;
                x[v + 1] = f.y;
                x[v + 2] = f.z;
                x[v + 3] = f.w;
            }
        } else {
            x[v] = slot[v * 32 + lane];
        }
    }
}
// The same with -infinity in columns from E on, and in all of a row that was not requested.
template <int L, int V, bool kVec>
__device__ __forceinline__ void ring_read(const float* slot, int E, int gl, bool have, float (&x)[V]) {
    ring_read<V, kVec>(slot, x);
    if (E == L * V && __all_sync(0xffffffffu, have)) return;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (!(have && col_of<L, kVec>(v, gl) < E)) x[v] = -INFINITY;
}
// Writes the lane's values back to its places.
template <int V, bool kVec>
__device__ __forceinline__ void ring_write(float* slot, const float (&x)[V]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (kVec) {
            if (v % 4 == 0)
                *reinterpret_cast<float4*>(slot + (v / 4 * 32 + lane) * 4) = make_float4(x[v], x[v + 1], x[v + 2],
                                                                                       x[v + 3]);
        } else {
            slot[v * 32 + lane] = x[v];
        }
    }
}
// Where column c of the row of group `group` lies in a slot.
template <int L, bool kVec>
__device__ __forceinline__ int ring_place(int c, int group) {
    return kVec ? ((c / (4 * L)) * 32 + group * L + (c / 4) % L) * 4 + c % 4 : c / L * 32 + group * L + c % L;
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 0 for -infinity
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x = exp(x - mx).  The difference first: near the type's bounds a product with log2(e) overflows.
template <int V>
__device__ __forceinline__ void exp_terms(float (&x)[V], float mx) {
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = exp2_approx((x[v] - mx) * kLog2e);
}

struct StatsShared {
    float z[kBalWarps];
    int n[kBalWarps];
};
struct FinishShared {
    float p[kFinWarps][kFinCols];
    int c[kFinWarps][kFinCols];
    float z[kFinWarps];
    int n[kFinWarps];
    int i[kFinWarps], j[kFinWarps];
};

// Sums over the tokens t, t + step, ... < t_hi of one sequence, t the first of this lane's group
// and tw the first of the warp's groups: acc += p, z += lse^2, cnt += 1 for each that counts;
// `count(id)` for each of its routes.
template <int L, int V, bool kVec, class Count>
__device__ __forceinline__ void sum_tokens(const BalanceArgs& a, float* ring, int tw, int t_hi, int step,
                                           float (&acc)[V], float& z, int& cnt, Count count) {
    const int E = a.E, k = a.k;
    const int lane = threadIdx.x & 31, gl = lane & (L - 1);
    constexpr int kSlot = 32 * V, kRing = kRingOf<V>;
    int t = tw + lane / L;
    auto kept = [&](int tt) { return tt < t_hi && (a.mask == nullptr || __ldg(a.mask + tt) != 0); };
    bool have[kRing];  // of the rows in the ring's slots, the oldest first
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) {
        have[i] = kept(t + i * step);
        ring_request<L, V, kVec>(ring + i * kSlot, a.logits + (size_t)(t + i * step) * E, E, gl, have[i]);
    }
    int slot = 0;
    for (; tw < t_hi; tw += step, t += step) {
        have[kRing - 1] = kept(t + (kRing - 1) * step);
        // the routes are on their way before the softmax needs its row
        int id0 = -1;
        if (have[0] && gl < k) id0 = __ldg(a.ids + (size_t)t * k + gl);
        ring_wait<kRing>();
        float x[V];
        ring_read<L, V, kVec>(ring + slot * kSlot, E, gl, have[0], x);
        const int refill = slot + kRing - 1 < kRing ? slot + kRing - 1 : slot - 1;
        ring_request<L, V, kVec>(ring + refill * kSlot, a.logits + (size_t)(t + (kRing - 1) * step) * E, E, gl,
                                 have[kRing - 1]);
        float mx = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) mx = fmaxf(mx, x[v]);
        mx = group_max<L>(mx);
        if (mx == -INFINITY) mx = 0.0f;  // all -infinity: the sum below is 0 (NaN with a NaN logit)
        exp_terms<V>(x, mx);
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += x[v];
        sum = group_sum<L>(sum);
        const bool counted = have[0] && sum != 0.0f;  // true for NaN: it shows in the losses
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
        if (counted) {
            if (id0 >= 0 && id0 < E) count(id0);
            for (int j = gl + L; j < k; j += L) {
                const int id = __ldg(a.ids + (size_t)t * k + j);
                if (id >= 0 && id < E) count(id);
            }
        }
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) have[i] = have[i + 1];
        slot = slot + 1 == kRing ? 0 : slot + 1;
    }
    ring_drain();
    // the groups of the warp: every lane then holds the warp's sum of its columns
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[v] += __shfl_xor_sync(0xffffffffu, acc[v], o);
    z = group_sum<32>(z);
    cnt = __reduce_add_sync(0xffffffffu, cnt);
}

// Sums of this block's tokens, one slot for each sequence it meets.
template <int L, int V, bool kVec>
__device__ __forceinline__ void balance_stats(const BalanceArgs& a, int n, float* ring, float* s_sum, int* s_cnt,
                                              StatsShared& sh) {
    const int E = a.E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane & (L - 1);
    constexpr int kGroups = 32 / L;  // tokens a warp holds at once
    const int chunk = (n + a.blocks - 1) / a.blocks;
    const int c0 = min(n, (int)blockIdx.x * chunk), c1 = min(n, c0 + chunk);
    if (c0 >= c1) return;
    // tokens before the first and behind the last sequence count for nothing
    const int first = seq_begin(a.seq_off, 0, n), last = seq_begin(a.seq_off, a.num_seqs, n);
    for (int t = c0 + threadIdx.x; t < c1; t += kBalThreads)
        if (t < first || t >= last) a.lse[t] = -INFINITY;

    // The runs of this block: of each sequence it meets, its tokens [lo, hi) here.  Runs of more than
    // `most` tokens are cut into segments of so many, one a warp (`most` is the least that leaves a
    // warp one segment or run, but at most twice what the tokens alone ask for); a shorter run is a
    // warp's own.  So all runs are read at once: 512 tokens of 1,000 experts in 16 sequences take
    // 14.6 us, 19.6 run after run, each with its own start.
    const int s0 = find_seq_warp(a.seq_off, a.num_seqs, c0);
    if (s0 >= a.num_seqs) return;
    struct Run {
        int lo, hi;
        __device__ int len() const { return hi > lo ? hi - lo : 0; }
    };
    auto run_of = [&](int s) {  // in the sweeps lane l's, of sequence s
        if (s >= a.num_seqs) return Run{c1, c1};
        return Run{max(seq_begin(a.seq_off, s, n), c0), min(seq_begin(a.seq_off, s + 1, n), c1)};
    };
    auto ends = [&](int base) { return base + 32 >= a.num_seqs || seq_begin(a.seq_off, base + 32, n) >= c1; };
    int passes = (c1 - c0 + kBalWarps * kGroups - 1) / (kBalWarps * kGroups);
    const Run whole = run_of(s0);
    const bool alone = whole.hi >= c1 || s0 + 1 == a.num_seqs;  // no other run
    if (!alone) {
        if (ends(s0)) {
            const int len = run_of(s0 + lane).len();
            for (const int least = passes; passes < 2 * least; ++passes) {
                const int most = passes * kGroups;
                if (__reduce_add_sync(0xffffffffu, (len + most - 1) / most) <= kBalWarps) break;
            }
        } else {
            passes *= 2;  // always enough
        }
    }
    const int most = passes * kGroups;
    auto segments = [&](const Run& r) { return r.len() > most ? (r.len() + most - 1) / most : 0; };
    // f(base, the lane's run, its segments, the first of them, cut runs before base) for every 32
    // sequences; returns the segments
    auto sweep = [&](auto f) {
        int total = 0, runs = 0;
        for (int base = s0;; base += 32) {
            const Run r = run_of(base + lane);
            const int m = segments(r);
            int sum = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int below = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += below;
            }
            f(base, r, m, total + sum - m, runs);
            runs += __popc(__ballot_sync(0xffffffffu, m > 0));
            total += __shfl_sync(0xffffffffu, sum, 31);
            if (ends(base)) return total;
        }
    };
    // this warp's segment, and the row of its run's counts (at least two segments each, but for a run
    // alone: below kCutRuns, whatever the offsets)
    int seg_lo = 0, seg_hi = 0, row = 0, cut;
    int step = kGroups;
    if (alone) {  // every warp in turn
        cut = min(kBalWarps, (whole.len() + kGroups - 1) / kGroups);
        step = kBalWarps * kGroups;
        seg_lo = whole.lo + warp * kGroups;
        seg_hi = whole.hi;
    } else {
        cut = sweep([&](int, const Run& r, int m, int first, int runs) {
            const unsigned cuts = __ballot_sync(0xffffffffu, m > 0);
            const unsigned mine = __ballot_sync(0xffffffffu, first <= warp && warp < first + m);
            if (mine != 0u) {
                const int from = __ffs(mine) - 1;
                seg_lo = __shfl_sync(0xffffffffu, r.lo, from) + (warp - __shfl_sync(0xffffffffu, first, from)) * most;
                seg_hi = min(seg_lo + most, __shfl_sync(0xffffffffu, r.hi, from));
                row = runs + __popc(cuts & ((1u << from) - 1u));
            }
        });
    }
    if (cut > 0) {
        for (int e = threadIdx.x; e < (alone ? 1 : kCutRuns) * E; e += kBalThreads) s_cnt[e] = 0;
        __syncthreads();
    }
    float acc[V], z = 0.0f;
    int cnt = 0;
    auto clear = [&] {
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.0f;
        z = 0.0f;
        cnt = 0;
    };
    auto leave = [&](float* to) {  // the warp's sums
        if (lane < L)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = col_of<L, kVec>(v, gl);
                if (c < E) to[c] = acc[v];
            }
    };
    if (seg_lo < seg_hi) {
        int* counts = s_cnt + row * E;
        clear();
        sum_tokens<L, V, kVec>(a, ring, seg_lo, seg_hi, step, acc, z, cnt,
                               [&](int id) { atomicAdd(counts + id, 1); });  // integers: any order
        leave(s_sum + warp * E);
        if (lane == 0) {
            sh.z[warp] = z;
            sh.n[warp] = cnt;
        }
    }
    // the i-th short run is warp (cut + i) % kBalWarps's
    for (int base = s0, shorts = 0; !alone; base += 32) {
        const Run r = run_of(base + lane);
        const bool is = r.len() > 0 && segments(r) == 0;
        const unsigned all = __ballot_sync(0xffffffffu, is);
        const int at = cut + shorts + __popc(all & ((1u << lane) - 1u));
        shorts += __popc(all);
        for (unsigned left = __ballot_sync(0xffffffffu, is && at % kBalWarps == warp); left != 0u; left &= left - 1) {
            const int from = __ffs(left) - 1;
            const size_t slot = (size_t)blockIdx.x + base + from;
            int* counts = a.slot_c + slot * E;
            for (int e = lane; e < E; e += 32) counts[e] = 0;
            __syncwarp();
            clear();
            sum_tokens<L, V, kVec>(a, ring, __shfl_sync(0xffffffffu, r.lo, from), __shfl_sync(0xffffffffu, r.hi, from),
                                   kGroups, acc, z, cnt, [&](int id) { atomicAdd(counts + id, 1); });
            leave(a.slot_p + slot * E);
            if (lane == 0) {
                a.slot_z[slot] = z;
                a.slot_n[slot] = cnt;
            }
        }
        if (ends(base)) break;
    }
    if (cut == 0) return;
    // the segments of each cut run, in order
    __syncthreads();
    auto join = [&](int s, int w0, int w1, const int* counts) {
        const size_t slot = (size_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            float p = 0.0f;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) p += w >= w0 && w < w1 ? s_sum[w * E + e] : 0.0f;
            a.slot_p[slot * E + e] = p;
            a.slot_c[slot * E + e] = counts[e];
        }
        if (threadIdx.x == 0) {
            float zs = 0.0f;
            int ns = 0;
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) {
                zs += w >= w0 && w < w1 ? sh.z[w] : 0.0f;
                ns += w >= w0 && w < w1 ? sh.n[w] : 0;
            }
            a.slot_z[slot] = zs;
            a.slot_n[slot] = ns;
        }
    };
    if (alone)
        join(s0, 0, cut, s_cnt);
    else
        sweep([&](int base, const Run&, int m, int first, int runs) {
            // (more than kCutRuns only where the offsets decrease, which finish_total finds)
            for (unsigned cuts = __ballot_sync(0xffffffffu, m > 0); cuts != 0u && runs < kCutRuns;
                 cuts &= cuts - 1, ++runs) {
                const int from = __ffs(cuts) - 1, w0 = __shfl_sync(0xffffffffu, first, from);
                join(base + from, w0, w0 + __shfl_sync(0xffffffffu, m, from), s_cnt + runs * E);
            }
        });
}

// Adds the slots of sequence s for 32 experts: an item is one (sequence, 32 experts) of the
// num_seqs * ceil(E / 32), which the cluster's warps share in groups of kGroup.  kGroup == 1 needs
// no meeting of warps.
template <int kGroup>
__device__ __forceinline__ void finish_items(const BalanceArgs& a, int n, int rank, int size, FinishShared& sh) {
    const int E = a.E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_block = (int)(blockDim.x >> 5) / kGroup;  // items a block has at once
    const int member = warp % kGroup;
    const int col_blocks = (E + kFinCols - 1) / kFinCols, items = a.num_seqs * col_blocks;
    const int chunk = (n + a.blocks - 1) / a.blocks;
    for (int i0 = rank * per_block; i0 < items; i0 += size * per_block) {  // uniform over the block
        const int it = i0 + warp / kGroup;
        const bool on = it < items;
        const int s = on ? it / col_blocks : 0, cb = it - s * col_blocks;
        const int e = cb * kFinCols + lane;
        const int sb = seq_begin(a.seq_off, s, n), se = seq_begin(a.seq_off, s + 1, n);
        // blocks that met the sequence
        const int b0 = se > sb ? sb / chunk : 0, b1 = on && se > sb ? (se - 1) / chunk + 1 : 0;
        float p = 0.0f, z = 0.0f;
        int c = 0, m = 0;
        if (cb == 0)
            for (int b = b0 + member * 32 + lane; b < b1; b += 32 * kGroup) {
                z += __ldcg(a.slot_z + b + s);
                m += __ldcg(a.slot_n + b + s);
            }
        for (int b = b0 + member; b < b1; b += kBatch * kGroup) {  // kBatch slots on their way at once
            float pv[kBatch];
            int cv[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const size_t at = (size_t)(b + i * kGroup + s) * E + e;
                const bool in = e < E && b + i * kGroup < b1;
                pv[i] = in ? __ldcg(a.slot_p + at) : 0.0f;
                cv[i] = in ? __ldcg(a.slot_c + at) : 0;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                p += pv[i];
                c += cv[i];
            }
        }
        z = group_sum<32>(z);
        m = __reduce_add_sync(0xffffffffu, m);
        if (kGroup > 1) {
            sh.p[warp][lane] = p;
            sh.c[warp][lane] = c;
            if (lane == 0) {
                sh.z[warp] = z;
                sh.n[warp] = m;
            }
            __syncthreads();
            if (member == 0) {
#pragma unroll
                for (int w = 1; w < kGroup; ++w) {
                    p += sh.p[warp + w][lane];
                    c += sh.c[warp + w][lane];
                    z += sh.z[warp + w];
                    m += sh.n[warp + w];
                }
            }
        }
        if (on && member == 0) {
            if (e < E) {
                a.prob_sums[(size_t)s * E + e] = p;
                a.counts[(size_t)s * E + e] = c;
            }
            const float dot = group_sum<32>(e < E ? (float)c * p : 0.0f);
            if (lane == 0) {
                a.seq_dot[it] = dot;
                if (cb == 0) {
                    a.seq_z[s] = z;
                    a.seq_n[s] = se < sb ? -1 : m;
                }
            }
        }
        if (kGroup > 1) __syncthreads();
    }
}

// One block: S', T and the z sum, then the sequences' factors and the losses.  Each thread takes
// every blockDim-th sequence, and the threads' sums are added in a fixed order.  Offsets that
// decrease have no sums: every factor and loss is then NaN.
__device__ __forceinline__ void finish_total(const BalanceArgs& a, FinishShared& sh) {
    static_assert(MOE_MAX_SEQS < kBadOffsets && kFinThreads <= INT_MAX / kBadOffsets - 1, "counted in `filled`");
    const int S = a.num_seqs, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int used = min(warps, (S + 31) / 32);  // warps that have a sequence
    const int col_blocks = (a.E + kFinCols - 1) / kFinCols;
    if (used == 1 && warp > 0) return;  // one warp does it, and meets nobody
    auto dot_of = [&](int s) {
        float dot = 0.0f;
        for (int cb = 0; cb < col_blocks; cb += kBatch) {
            float v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                v[i] = cb + i < col_blocks ? __ldcg(a.seq_dot + (size_t)s * col_blocks + cb + i) : 0.0f;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) dot += v[i];
        }
        return dot;
    };
    // this thread's first sequence in registers
    const bool mine = (int)threadIdx.x < S;
    const int m0 = mine ? __ldcg(a.seq_n + threadIdx.x) : 0;
    float z = mine ? __ldcg(a.seq_z + threadIdx.x) : 0.0f;
    const float dot0 = mine ? dot_of(threadIdx.x) : 0.0f;
    bool bad = m0 < 0;
    int filled = m0 > 0, total = m0;
    for (int s = threadIdx.x + blockDim.x; s < S; s += blockDim.x) {
        const int m = __ldcg(a.seq_n + s);
        bad |= m < 0;
        filled += m > 0;
        total += m;
        z += __ldcg(a.seq_z + s);
    }
    if (bad) filled += kBadOffsets;
    filled = __reduce_add_sync(0xffffffffu, filled);
    total = __reduce_add_sync(0xffffffffu, total);
    z = group_sum<32>(z);
    if (used > 1) {
        if (lane == 0) {
            sh.i[warp] = filled;
            sh.j[warp] = total;
            sh.z[warp] = z;
        }
        __syncthreads();
        filled = total = 0;
        z = 0.0f;
        for (int w = 0; w < used; ++w) {
            filled += sh.i[w];
            total += sh.j[w];
            z += sh.z[w];
        }
        __syncthreads();
    }
    bad = filled >= kBadOffsets;
    const float nan = __uint_as_float(0x7fc00000u);
    const float scale = a.balance_coef * (float)a.E / ((float)max(filled, 1) * (float)a.k);
    float loss = 0.0f;
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const bool first = s == (int)threadIdx.x;
        const int m = first ? m0 : __ldcg(a.seq_n + s);
        const float as = m > 0 ? scale / (float)m / (float)m : 0.0f;
        if (m > 0) loss = fmaf(as, first ? dot0 : dot_of(s), loss);
        a.grad_scales[s] = bad ? nan : as;
    }
    loss = group_sum<32>(loss);
    if (used > 1) {
        if (lane == 0) sh.z[warp] = loss;
        __syncthreads();
        loss = 0.0f;
        for (int w = 0; w < used; ++w) loss += sh.z[w];
    }
    if (threadIdx.x == 0) {
        const float zt = total > 0 ? a.z_coef / (float)total : 0.0f;
        a.losses[0] = bad ? nan : loss;
        a.losses[1] = bad ? nan : zt != 0.0f ? zt * z : 0.0f;  // without a z loss, 0 even where lse^2 overflows
        a.grad_scales[S] = bad ? nan : 2.0f * zt;
    }
}

// kOne: the grid is one cluster, which meets in its own barrier between the sums, the finish and
// the totals; else balance_finish_kernel does the rest.
template <int L, int V, bool kVec, bool kOne>
__global__ void __launch_bounds__(kBalThreads, 1) balance_stats_kernel(const BalanceArgs a) {
    extern __shared__ __align__(16) float s_bal[];  // the warps' rings, [kBalWarps][E] sums, [kCutRuns][E] counts
    __shared__ StatsShared sh;
    pdl_wait();
    pdl_trigger();  // after the wait: the finishing kernel reads sizes and offsets before its own
    const int n = clamp_live(a.live, a.max_live);
    if (!kOne && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;
    constexpr int kRingFloats = kRingOf<V> * 32 * V;  // of a warp
    float* s_sum = s_bal + kBalWarps * kRingFloats;
    balance_stats<L, V, kVec>(a, n, s_bal + (threadIdx.x >> 5) * kRingFloats, s_sum,
                              reinterpret_cast<int*>(s_sum + kBalWarps * a.E), sh);
    if constexpr (kOne) {
        static_assert(sizeof(FinishShared) <= kBalWarps * kRingFloats * 4, "the finish takes the rings' place");
        FinishShared& fin = *reinterpret_cast<FinishShared*>(s_bal);
        cluster_sync();  // the slots of every block are written
        finish_items<1>(a, n, blockIdx.x, gridDim.x, fin);
        cluster_sync();
        if (blockIdx.x == 0) finish_total(a, fin);
    }
}

// kCluster: one cluster, which meets in its own barrier; else (many sequences or experts) any number
// of blocks, the last of which to come to the ticket does the totals.
template <bool kCluster>
__global__ void __launch_bounds__(kFinThreads) balance_finish_kernel(const BalanceArgs a) {
    __shared__ FinishShared fin;
    __shared__ int s_last;
    pdl_trigger();
    // the kernel before this one waited before it released this one: sizes and offsets are there
    const int n = clamp_live(a.live, a.max_live);
    pdl_wait();
    finish_items<kFinGroup>(a, n, blockIdx.x, gridDim.x, fin);
    if (kCluster) {
        cluster_sync();
        if (blockIdx.x == 0) finish_total(a, fin);
        return;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1 ? 1 : 0;
    __syncthreads();
    if (!s_last) return;
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

// A group of lanes per token, as the forward: the losses' part in registers; the chosen part is
// added to the row in its ring slot, from where the whole row leaves in wide stores.  Route j of a
// token belongs to lane j % L of its group; routes of different experts add in any order, an
// expert named twice (and any, where there are more routes than lanes) in route order.
template <int L, int V, bool kVec>
__global__ void __launch_bounds__(kGradThreads, kGradBlocks<V>) route_backward_kernel(const RouteGradArgs a) {
    extern __shared__ __align__(16) float s_rings[];
    constexpr int kGroups = 32 / L;
    constexpr int kSlots = (kMaxTopK + L - 1) / L;  // routes of a lane
    constexpr int kSlot = 32 * V, kRing = kRingOf<V>;
    pdl_trigger();
    pdl_wait();
    const int E = a.E, k = a.k;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gl = lane & (L - 1), group = lane / L;
    float* ring = s_rings + warp * kRing * kSlot;
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
    int t = c0 + warp * kGroups + group;
    auto lse_of = [&](int tt) {
        return tt < c1 ? (a.lse != nullptr ? __ldg(a.lse + tt) : 0.0f) : -INFINITY;
    };
    float lse_next = lse_of(t);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i)
        ring_request<L, V, kVec>(ring + i * kSlot, a.logits + (size_t)(t + i * kStep) * E, E, gl,
                                 has_loss && t + i * kStep < c1);
    int slot = 0;
    for (int tw = c0 + warp * kGroups; tw < c1; tw += kStep, t += kStep) {
        const bool in = t < c1;
        const float lse = lse_next;
        const bool counted = lse != -INFINITY;  // true for NaN
        lse_next = lse_of(t + kStep);
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
        float* row = ring + slot * kSlot;
        const int refill = slot + kRing - 1 < kRing ? slot + kRing - 1 : slot - 1;
        float x[V];
        ring_wait<kRing>();
        if (has_loss) {
            ring_read<L, V, kVec>(row, E, gl, counted, x);
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
            if (mx == -INFINITY) mx = 0.0f;
            exp_terms<V>(x, mx);
            float sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                sum += x[v];
                dot = fmaf(cnt[v], x[v], dot);
            }
            sum = group_sum<L>(sum);
            dot = group_sum<L>(dot);
            // p (as (c - <c, p>) + zs lse), with p = x / sum; 0 where the token does not count
            // (both factors: `as` and zs hold the caller's scale, which may have overflowed)
            const float inv = counted ? __frcp_rn(sum) : 0.0f;
            const float slope = counted ? as * inv : 0.0f;
            const float base = counted ? fmaf(zs, lse, -as * (dot * inv)) * inv : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] *= fmaf(slope, cnt[v], base);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[v] = 0.0f;
        }
        if (a.dprobs != nullptr) {
            float wd = 0.0f;
#pragma unroll
            for (int r = 0; r < kSlots; ++r) wd = fmaf(w[r], d[r], wd);
            wd = group_sum<L>(wd);
            ring_write<V, kVec>(row, x);
            bool apart = k <= L;
            if (apart) {
                const unsigned key = id[0] >= 0 ? (unsigned)(id[0] * kGroups + group) : 0x80000000u + lane;
                apart = __all_sync(0xffffffffu, __popc(__match_any_sync(0xffffffffu, key)) == 1);
            }
            __syncwarp();
            if (apart) {
                if (id[0] >= 0) row[ring_place<L, kVec>(id[0], group)] += w[0] * (d[0] - wd);
                __syncwarp();
            } else {
#pragma unroll
                for (int r = 0; r < kSlots; ++r)
                    for (int j = r * L; j < min(k, r * L + L); ++j) {
                        if (gl == j - r * L && id[r] >= 0)
                            row[ring_place<L, kVec>(id[r], group)] += w[r] * (d[r] - wd);
                        __syncwarp();
                    }
            }
            ring_read<V, kVec>(row, x);  // columns from E on are not stored
        }
        ring_request<L, V, kVec>(ring + refill * kSlot, a.logits + (size_t)(t + (kRing - 1) * kStep) * E, E, gl,
                                 has_loss && t + (kRing - 1) * kStep < c1);
        slot = slot + 1 == kRing ? 0 : slot + 1;
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
    ring_drain();
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

// Blocks of the sums: one pass of each block's warps at least, `cap` at most; in one cluster as many
// as give each item of the finish a warp (117 tokens of 16 experts in 64 sequences: 9.2 us, 16.8 with
// the one block that the tokens need).
int balance_blocks(long long max_live, int E, int num_seqs, long long cap) {
    const int b = blocks_for(max_live, kBalWarps * tokens_per_warp(E), cap);
    if (b > kClusterBlocks) return b;
    const long long items = (long long)num_seqs * ((E + kFinCols - 1) / kFinCols);
    const int f = blocks_for(items, kBalWarps, kClusterBlocks), w = b > f ? b : f;
    return w > 4 ? 8 : w > 2 ? 4 : w;
}

struct BalanceLayout {
    size_t p, c, z, n, dot, sz, sn, ticket, total;
};
BalanceLayout balance_layout(const moe_plan* plan, int num_seqs) {
    const size_t E = (size_t)plan->d.num_experts, S = (size_t)num_seqs;
    const int b = balance_blocks(plan->max_live, plan->d.num_experts, num_seqs, kMaxBalBlocks);
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

// Dynamic shared memory over 48 KB is asked for once per kernel and device.
template <class Kernel>
cudaError_t allow_smem(Kernel kern, size_t bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev]) return cudaSuccess;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (err == cudaSuccess) done[dev] = true;
    return err;
}

// A launch of one cluster of `blocks` blocks.
template <class... KArgs, class... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), int blocks, int threads, size_t smem, cudaStream_t s,
                           Args&&... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
    return err != cudaSuccess ? err : cudaGetLastError();
}

template <int L, int V, bool kVec>
struct LaunchStats {
    static constexpr size_t smem(int E, bool one_seq) {  // of a sequence alone no block meets two
        return (size_t)(kBalWarps * kRingOf<V> * 32 * V + (kBalWarps + (one_seq ? 1 : kCutRuns)) * E) * 4;
    }
    static cudaError_t go(const BalanceArgs& a, cudaStream_t s) {
        static_assert(smem(L * V, false) + sizeof(StatsShared) + 1024 <= 232448, "shared memory budget");
        static bool done[2][64];
        const bool one = a.blocks <= kClusterBlocks;
        const size_t most = smem(L * V, false), need = smem(a.E, a.num_seqs == 1);
        cudaError_t err = one ? allow_smem(balance_stats_kernel<L, V, kVec, true>, most, done[1])
                              : allow_smem(balance_stats_kernel<L, V, kVec, false>, most, done[0]);
        if (err != cudaSuccess) return err;
        if (one)
            return launch_cluster(balance_stats_kernel<L, V, kVec, true>, a.blocks, kBalThreads, need, s, a);
        return launch_dependent(balance_stats_kernel<L, V, kVec, false>, dim3(a.blocks), dim3(kBalThreads), need, s, a);
    }
};
template <int L, int V, bool kVec>
struct LaunchBackward {
    static cudaError_t go(RouteGradArgs a, cudaStream_t s) {
        a.blocks = blocks_for(a.max_live, kGradWarps * (32 / L), (long long)num_sms() * kGradBlocks<V>);
        constexpr size_t smem = (size_t)kGradWarps * kRingOf<V> * 32 * V * 4;  // at most 64 KB
        static bool done[64];
        const cudaError_t err = allow_smem(route_backward_kernel<L, V, kVec>, smem, done);
        if (err != cudaSuccess) return err;
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
    a.blocks = balance_blocks(plan->max_live, a.E, num_seqs, num_sms() < kMaxBalBlocks ? num_sms() : kMaxBalBlocks);
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
    constexpr int kPerBlock = kFinWarps / kFinGroup;
    if (items <= 2 * kFinBlocks * kPerBlock) {
        e = launch_cluster(balance_finish_kernel<true>, kFinBlocks, kFinThreads, 0, s, a);
    } else {
        const long long want = (items + kPerBlock - 1) / kPerBlock, cap = num_sms();
        e = launch_dependent(balance_finish_kernel<false>, dim3((unsigned)(want < cap ? want : cap)),
                             dim3(kFinThreads), 0, s, a);
    }
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
