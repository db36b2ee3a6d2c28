// combine_grad.cu -- the gradient of the combine (moe_combine_backward).
//
// The combine is out_t = sum_j p[t,j] y[r(t,j)], so with d_t the gradient of
// out_t:  dprobs[t,j] = <d_t, y[r(t,j)]>  and  dy[r(t,j)] = p[t,j] d_t.
// Both are one pass over the y rows: a block holds a slice of d_t in registers
// and walks the token's rows, so that d_t is read once for all of them.  The
// dot products are sums of 128 threads' partial sums in fp32, added in a fixed
// order whatever the number of routes a block takes.
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kCgThreads = 128;
constexpr int kCgWarps = kCgThreads / 32;

struct CombineGradArgs {
    const void* dout;
    const float4* y;
    const int* rows;
    const float* probs;
    const int* live;
    int max_live, H, k;
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

// Items are (token, group of its routes): with fewer live tokens than blocks the k routes are
// spread over several blocks, each reading d_t again (from L2) for its own rows.
template <bool kBf16>
__global__ void __launch_bounds__(kCgThreads) combine_backward_kernel(const CombineGradArgs a) {
    __shared__ int s_row[kMaxTopK];
    __shared__ float s_p[kMaxTopK];
    __shared__ float s_dot[kCgWarps][kMaxTopK];
    pdl_trigger();
    pdl_wait();
    const int n = clamp_live(a.live, a.max_live), k = a.k;
    const int chunks = a.H / 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int parts = n > 0 ? (int)(gridDim.x / (unsigned)n) : 1;
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
        float dot[kMaxTopK];
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.0f;
        for (int c = threadIdx.x; c < chunks; c += kCgThreads) {
            const float4 d = load_grad<kBf16>(a.dout, (size_t)t * chunks + c);
#pragma unroll
            for (int jb = 0; jb < kMaxTopK; jb += 8) {
                if (jb >= m) break;
                float4 v[8];
                if (a.dprobs != nullptr) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = jb + j < m ? s_row[jb + j] : -1;
                        v[j] = r >= 0 ? __ldg(a.y + (size_t)r * chunks + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x = dot[jb + j];
                        x = fmaf(d.x, v[j].x, x);
                        x = fmaf(d.y, v[j].y, x);
                        x = fmaf(d.z, v[j].z, x);
                        dot[jb + j] = fmaf(d.w, v[j].w, x);
                    }
                }
                if (a.dy != nullptr) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = jb + j < m ? s_row[jb + j] : -1;
                        const float p = jb + j < m ? s_p[jb + j] : 0.0f;
                        if (r >= 0)
                            a.dy[(size_t)r * chunks + c] = make_float4(p * d.x, p * d.y, p * d.z, p * d.w);
                    }
                }
            }
        }
        if (a.dprobs != nullptr) {
#pragma unroll
            for (int j = 0; j < kMaxTopK; ++j) {
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
    long long grid = plan->max_live * a.k;
    const long long cap = (long long)num_sms() * 8;
    if (grid > cap) grid = cap;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = (plan->d.flags & MOE_FLAG_OUT_BF16) != 0
                              ? launch_dependent(combine_backward_kernel<true>, dim3((unsigned)grid), dim3(kCgThreads),
                                                 0, s, a)
                              : launch_dependent(combine_backward_kernel<false>, dim3((unsigned)grid),
                                                 dim3(kCgThreads), 0, s, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
