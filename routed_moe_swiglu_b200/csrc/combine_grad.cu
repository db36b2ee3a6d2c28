// combine_grad.cu -- the gradient of the combine (moe_combine_backward).
//
// The combine is out_t = sum_j p[t,j] y[r(t,j)], so with d_t the gradient of
// out_t:  dprobs[t,j] = <d_t, y[r(t,j)]>  and  dy[r(t,j)] = p[t,j] d_t.
// Both are one pass over the y rows with d_t in registers, so that d_t is read
// once for all of a token's rows: rows of up to 2,048 elements a token a group of
// lanes, longer ones a token a block (with few tokens the routes are spread, each
// item reading d_t again from L2).  A dot product is a sum of lanes' or threads'
// partial sums in fp32, added in an order fixed by H alone.
//
// Bound by memory: y is read and dy written once.  8,192 tokens x 8 routes x
// 2,048: 181 us for 1.14 GB, 6.3 TB/s, 0.96 of the measured copy rate; 333 x 6 x
// 2,688 with bf16 gradients: 10.7 us for 45 MB, where start and end count.
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kCgThreads = 128;
constexpr int kCgWarps = kCgThreads / 32;
constexpr int kRowChunks = 512;  // 16-byte chunks of a row that a warp takes

struct CombineGradArgs {
    const void* dout;
    const float4* y;
    const int* rows;
    const float* probs;
    const int* live;
    int max_live, H, k;
    int fill;       // items that fill the SMs
    float* dprobs;  // null: not wanted
    float4* dy;     // null: not wanted
};

template <bool kBf16>
__device__ __forceinline__ float4 load_grad(const void* p, size_t i) {
    if (kBf16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p) + i);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xffff0000u));
    }
    return __ldg(reinterpret_cast<const float4*>(p) + i);
}

// kRoutes rows of y (from jb on, of the item's m) at kChunks of this thread's chunks, c and every
// kCgThreads-th after it: all loads before the first sum.  A route's products are added in chunk
// order whatever kRoutes and kChunks are.
template <bool kBf16, int kRoutes, int kChunks>
__device__ __forceinline__ void walk(const CombineGradArgs& a, int t, int c, int chunks, int jb, int m,
                                     const int* s_row, const float* s_p, float* dot) {
    float4 d[kChunks], v[kChunks][kRoutes];
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
        const int cu = c + u * kCgThreads;
        d[u] = cu < chunks ? load_grad<kBf16>(a.dout, (size_t)t * chunks + cu) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.dprobs != nullptr)
#pragma unroll
            for (int j = 0; j < kRoutes; ++j) {
                const int r = jb + j < m ? s_row[jb + j] : -1;
                v[u][j] = r >= 0 && cu < chunks ? __ldg(a.y + (size_t)r * chunks + cu) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
    }
    if (a.dprobs != nullptr)
#pragma unroll
        for (int u = 0; u < kChunks; ++u)
#pragma unroll
            for (int j = 0; j < kRoutes; ++j) {
                float x = dot[j];
                x = fmaf(d[u].x, v[u][j].x, x);
                x = fmaf(d[u].y, v[u][j].y, x);
                x = fmaf(d[u].z, v[u][j].z, x);
                dot[j] = fmaf(d[u].w, v[u][j].w, x);
            }
    if (a.dy != nullptr)
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int cu = c + u * kCgThreads;
            if (cu >= chunks) break;
#pragma unroll
            for (int j = 0; j < kRoutes; ++j) {
                const int r = jb + j < m ? s_row[jb + j] : -1;
                const float p = jb + j < m ? s_p[jb + j] : 0.0f;
                // written once and not read here: past the lines of y that are still to come
                if (r >= 0)
                    __stcs(a.dy + (size_t)r * chunks + cu, make_float4(p * d[u].x, p * d[u].y, p * d[u].z, p * d[u].w));
            }
        }
}

// Items are (token, group of its routes).  With fewer live tokens than `fill` the k routes are spread
// over several blocks, each reading d_t again (from L2) for its own rows.  With more, a block for
// each token leaves the SMs no uneven last round (8,192 tokens x 8 x 2,048: 186 us, against 200 with
// eight blocks an SM that walk the tokens; the lane groups below take rows of that length now).
// kMost: the most routes a token may have, 8 or 16.
template <bool kBf16, int kMost>
__global__ void __launch_bounds__(kCgThreads, kMost > 8 ? 5 : 7) combine_backward_kernel(const CombineGradArgs a) {
    __shared__ int s_row[kMaxTopK];
    __shared__ float s_p[kMaxTopK];
    __shared__ float s_dot[kCgWarps][kMaxTopK];
    pdl_trigger();
    pdl_wait();
    const int n = clamp_live(a.live, a.max_live), k = a.k;
    const int chunks = a.H / 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int parts = n > 0 ? a.fill / n : 1;
    parts = parts < 1 ? 1 : (parts > k ? k : parts);
    const int span = (k + parts - 1) / parts;  // routes per item
    const long long items = (long long)n * parts;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int t = (int)(it / parts);
        const int j0 = (int)(it % parts) * span, m = min(k - j0, span);  // this item's routes
        if (m <= 0) continue;
        __syncthreads();
        if (threadIdx.x < m) {
            s_row[threadIdx.x] = __ldg(a.rows + (size_t)t * k + j0 + threadIdx.x);
            s_p[threadIdx.x] = __ldg(a.probs + (size_t)t * k + j0 + threadIdx.x);
        }
        __syncthreads();
        float dot[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j) dot[j] = 0.0f;
        if (m <= 2) {
            for (int c = threadIdx.x; c < chunks; c += 2 * kCgThreads)
                walk<kBf16, 2, 2>(a, t, c, chunks, 0, m, s_row, s_p, dot);
        } else {
            for (int c = threadIdx.x; c < chunks; c += kCgThreads) {
                walk<kBf16, 8, 1>(a, t, c, chunks, 0, m, s_row, s_p, dot);
                if (kMost > 8 && m > 8) walk<kBf16, 8, 1>(a, t, c, chunks, 8, m, s_row, s_p, dot + (kMost - 8));
            }
        }
        if (a.dprobs != nullptr) {
#pragma unroll
            for (int j = 0; j < kMost; ++j) {
                if (j < m) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
                    if (lane == 0) s_dot[warp][j] = dot[j];
                }
            }
            __syncthreads();
            if (threadIdx.x < m) {
                float x = 0.0f;
#pragma unroll
                for (int w = 0; w < kCgWarps; ++w) x += s_dot[w][threadIdx.x];
                // a route without a row has no gradient (its d_t may hold anything)
                a.dprobs[(size_t)t * k + j0 + threadIdx.x] = s_row[threadIdx.x] >= 0 ? x : 0.0f;
            }
        }
    }
}

// Rows that L lanes can hold: d_t in registers, C 16-byte chunks a lane, and the token's rows J at a time;
// 32 / L tokens a warp.  A block a token has a chain of launch, loads and meetings for each, and leaves
// threads without a chunk (46,692 tokens x 1 x 80: 10.2 us, 87 with a block a token; 36,057 x 2 x 520:
// 72 and 117; 8,192 x 8 x 2,048: 181 and 186; past 2,048 the registers of d_t leave too few warps).
template <bool kBf16, int L, int C, int J, int kBlocks>
__global__ void __launch_bounds__(kCgThreads, kBlocks) combine_backward_rows_kernel(const CombineGradArgs a) {
    pdl_trigger();
    pdl_wait();
    const int n = clamp_live(a.live, a.max_live), k = a.k, chunks = a.H / 4;
    const int gl = threadIdx.x & (L - 1);
    const long long step = (long long)gridDim.x * (kCgThreads / L);
    // items: a token, or with few of them J of its routes
    const int batches = (k + J - 1) / J;
    const int split = (long long)n * batches <= step ? batches : 1;
    // every lane of a warp goes round as often as its first group
    for (long long i0 = (long long)blockIdx.x * (kCgThreads / L) + (threadIdx.x & ~31) / L; i0 < (long long)n * split;
         i0 += step) {
        const long long item = i0 + (threadIdx.x & 31) / L, t = item / split;
        const bool on = t < n;
        const int j_lo = (int)(item - t * split) * J;
        float4 d[C];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int c = gl + u * L;
            d[u] = on && c < chunks ? load_grad<kBf16>(a.dout, (size_t)t * chunks + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // the token's rows and probabilities, a route a lane (k <= 16: two with L = 8)
        int row[2] = {-1, -1};
        float pr[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (on && gl + i * L < k && (i == 0 || L < kMaxTopK)) {
                row[i] = __ldg(a.rows + t * k + gl + i * L);
                pr[i] = __ldg(a.probs + t * k + gl + i * L);
            }
        for (int j0 = j_lo, i = 0; i < (split > 1 ? 1 : batches); ++i, j0 += J) {
            int r[J];
            float p[J];
            float4 v[J][C];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int at = j0 + j;
                const bool second = at >= L;
                r[j] = __shfl_sync(0xffffffffu, second ? row[1] : row[0], at & (L - 1), L);
                p[j] = __shfl_sync(0xffffffffu, second ? pr[1] : pr[0], at & (L - 1), L);
                if (at >= k) r[j] = -1;
            }
            if (a.dprobs != nullptr) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int u = 0; u < C; ++u) {
                        const int c = gl + u * L;
                        v[j][u] = r[j] >= 0 && c < chunks ? __ldg(a.y + (size_t)r[j] * chunks + c)
                                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                float mine = 0.0f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float x = 0.0f;
#pragma unroll
                    for (int u = 0; u < C; ++u)
                        x = fmaf(d[u].w, v[j][u].w, fmaf(d[u].z, v[j][u].z, fmaf(d[u].y, v[j][u].y, fmaf(d[u].x, v[j][u].x, x))));
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    if (gl == j) mine = r[j] >= 0 ? x : 0.0f;  // a route without a row has no gradient
                }
                if (on && gl < J && j0 + gl < k) a.dprobs[t * k + j0 + gl] = mine;
            }
            if (a.dy != nullptr) {
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (r[j] >= 0)
#pragma unroll
                        for (int u = 0; u < C; ++u) {
                            const int c = gl + u * L;
                            if (c < chunks)
                                __stcs(a.dy + (size_t)r[j] * chunks + c,
                                       make_float4(p[j] * d[u].x, p[j] * d[u].y, p[j] * d[u].z, p[j] * d[u].w));
                        }
            }
        }
    }
}

template <int L, int C, int J, int kBlocks>
cudaError_t launch_rows(const CombineGradArgs& a, bool bf16, cudaStream_t s) {
    const long long items = (long long)a.max_live * ((a.k + J - 1) / J);
    const long long want = (items + kCgThreads / L - 1) / (kCgThreads / L), cap = (long long)num_sms() * kBlocks * 2;
    return launch_dependent(bf16 ? combine_backward_rows_kernel<true, L, C, J, kBlocks>
                                 : combine_backward_rows_kernel<false, L, C, J, kBlocks>,
                            dim3((unsigned)(want < cap ? want : cap)), dim3(kCgThreads), 0, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_combine_backward(const moe_plan* plan, const void* dout, const float* y_rows,
                                           const int* route_rows, const float* route_probs,
                                           const int* live_count_dev, float* dprobs, float* dy_rows, void* stream) {
    if (plan == nullptr || dout == nullptr || route_rows == nullptr || route_probs == nullptr ||
        live_count_dev == nullptr)
        return MOE_ERR_INVALID_ARG;
    if (dprobs == nullptr && dy_rows == nullptr) return MOE_ERR_INVALID_ARG;
    if (dprobs != nullptr && y_rows == nullptr) return MOE_ERR_INVALID_ARG;
    auto off16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; };
    if (off16(dout) || off16(y_rows) || off16(dy_rows)) return MOE_ERR_ALIGNMENT;
    CombineGradArgs a{};
    a.dout = dout;
    a.y = reinterpret_cast<const float4*>(y_rows);
    a.rows = route_rows;
    a.probs = route_probs;
    a.live = live_count_dev;
    a.max_live = (int)plan->max_live;
    a.H = plan->d.hidden;
    a.k = plan->d.top_k;
    a.dprobs = dprobs;
    a.dy = reinterpret_cast<float4*>(dy_rows);
    a.fill = num_sms() * 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = (plan->d.flags & MOE_FLAG_OUT_BF16) != 0;
    const int chunks = a.H / 4;
    if (chunks <= kRowChunks) {
        const cudaError_t e = chunks <= 32    ? launch_rows<8, 4, 4, 5>(a, bf16, s)
                              : chunks <= 64  ? launch_rows<16, 4, 4, 5>(a, bf16, s)
                              : chunks <= 128 ? launch_rows<32, 4, 4, 5>(a, bf16, s)
                              : chunks <= 256 ? launch_rows<32, 8, 2, 4>(a, bf16, s)
                                              : launch_rows<32, 16, 1, 3>(a, bf16, s);
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    const long long most = plan->max_live > a.fill ? plan->max_live : a.fill;
    const long long grid = plan->max_live * a.k < most ? plan->max_live * a.k : most;
    void (*kern)(CombineGradArgs) = a.k > 8 ? (bf16 ? combine_backward_kernel<true, 16> : combine_backward_kernel<false, 16>)
                                            : (bf16 ? combine_backward_kernel<true, 8> : combine_backward_kernel<false, 8>);
    const cudaError_t e = launch_dependent(kern, dim3((unsigned)grid), dim3(kCgThreads), 0, s, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
