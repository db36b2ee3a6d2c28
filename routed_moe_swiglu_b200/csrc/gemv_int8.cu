// gemv_int8.cu -- the expert products of very few tokens in 8-bit integers, on
// the integer dot-product instruction (dp4a).
//
// With a token or two the time is that of reading the routed experts' weights,
// and the wide kernels spend it on their fixed steps: 256-row tiles that leave
// SMs idle or give some two, and passes of their own that quantise x and h.
// Here a warp takes eight weight rows of one expert, reads them straight from
// memory in 512-byte runs (the prepared layout holds a row's 128 codes of an
// atom together, and four rows one after another), and multiplies them with the
// expert's at most four tokens, whose codes each block computes for itself into
// shared memory.  Many small independent blocks keep memory busy without any
// block waiting for another.
//   gate/up  four gate rows and the four up rows of the same f -> SwiGLU ->
//            bf16 h rows (squared ReLU: eight rows of the one projection)
//   down     eight output columns of bf16 h rows -> fp32 y rows
// The sums are exact and what follows is the wide kernels' arithmetic: the same
// bits.
//
// One token, six experts of H 2,688, F 1,856 (90 MB of weights, 13.7 us at the
// copy rate): the whole forward takes 29.2 us, 42.8 on the wide kernels; 13 us of
// it are five launches' (32.2 with a warp a row where a block's codes are computed),
// two of which only put the token's routes in order.  Eight tokens an expert would cost
// 96-115 us against 77: hence the limit of four.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kGvThreads = 128;
constexpr int kGvWarps = kGvThreads / 32;
constexpr int kGvTokens = 4;        // tokens of an expert at most
constexpr int kUnitRows = 8;        // weight rows of a warp
constexpr int kAhead = 4;           // atoms whose weights are on their way at once
constexpr size_t kGvSmemMax = kGvTokens * 16384;  // rows of the widest plan

struct GemvArgs {
    Int8Gemm g;
    const uint4* x;        // gate/up: bf16 token rows; down: bf16 h rows
    long long ld_x;        // 16-byte chunks
    const uint8_t* w;      // prepared weights
    int cols_in, top_k, units;
};

__device__ __forceinline__ int dot16(int4 a, int4 b, int c) {
    c = __dp4a(a.x, b.x, c);
    c = __dp4a(a.y, b.y, c);
    c = __dp4a(a.z, b.z, c);
    return __dp4a(a.w, b.w, c);
}

// kTokens: the most tokens an expert of this plan can have, 1, 2 or 4.
template <bool kGateUp, int kTokens>
__global__ void __launch_bounds__(kGvThreads) moe_gemv_int8_kernel(const GemvArgs a) {
    extern __shared__ __align__(16) uint8_t s_codes[];  // [tokens][atoms * 128]
    __shared__ float s_xs[kGvTokens];
    __shared__ uint32_t s_red[kGvWarps];
    const Int8Gemm& p = a.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = p.atoms * 128;
    // The gate/up kernel lets the down kernel start after its own wait: the latter reads the tiles
    // and asks L2 for its weights before it waits for the h rows.
    if (kGateUp) {
        pdl_wait();
        pdl_trigger();
    } else {
        pdl_trigger();
    }
    const bool any = !forward_poisoned(p.status_words) && blockIdx.y < p.status_words[kStNumMTiles];
    const int4 ti = any ? __ldg(p.tiles + blockIdx.y) : make_int4(0, 0, 0, 0);
    const int nt = min(ti.z, kTokens);
    // this warp's weight rows: two runs of four, of which lane l reads 16 bytes of row l / 8
    const int unit = blockIdx.x * kGvWarps + warp;
    const bool swiglu = kGateUp && p.relu2 == 0;
    const int f0 = swiglu ? unit * 4 : unit * kUnitRows;  // first f (SwiGLU: of four), or first row of eight
    const int row0 = swiglu ? (f0 >> 6) * 128 + ((f0 >> 4) & 3) * 32 + (f0 & 15) : f0;
    const int apart = swiglu ? 16 : 4;  // rows between the two runs
    const long long grow = (long long)ti.x * p.a_rows + row0;
    const uint8_t* w = a.w + ((size_t)(grow >> 7) * p.atoms * 128 + (grow & 127) + (lane >> 3)) * 128 + (lane & 7) * 16;
    const bool work = any && unit < a.units;
    // The weights of kAhead atoms at a time, the next ones on their way while these are multiplied; the
    // first before the codes are computed.
    int4 wa[2][kAhead], wb[2][kAhead];
    auto request = [&](int k0, int4 (&ra)[kAhead], int4 (&rb)[kAhead]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const bool in = work && k0 + i < p.atoms;
            const uint8_t* q = w + (size_t)(k0 + i) * (128 * 128);
            ra[i] = in ? __ldcs(reinterpret_cast<const int4*>(q)) : make_int4(0, 0, 0, 0);
            rb[i] = in ? __ldcs(reinterpret_cast<const int4*>(q + apart * 128)) : make_int4(0, 0, 0, 0);
        }
    };
    request(0, wa[0], wb[0]);
    if (!kGateUp) {
        if (work)  // the rest of the weights into L2, a line a row and atom
            for (int i = lane + kAhead * kUnitRows; i < p.atoms * kUnitRows; i += 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w + ((size_t)(grow >> 7) * p.atoms * 128 +
                                                                    (size_t)(i / kUnitRows) * 128 + (grow & 127) +
                                                                    i % kUnitRows) *
                                                                       128));
        pdl_wait();
    }
    if (nt <= 0) return;

    // codes of the tokens' rows, the block's warps spread over them (past a row the weights' codes are
    // 0, and what stands in shared memory is of no account)
    constexpr int kRowWarps = kGvWarps / kTokens;
    const int r = warp / kRowWarps;
    const long long at = r >= nt ? 0 : kGateUp ? __ldg(p.perm + ti.w + r) / a.top_k : ti.y + r;
    const float scale = int8_quantize_row<kRowWarps, 4>(
        a.x + (size_t)at * a.ld_x, a.cols_in / 8, r < nt, s_red, [] {},
        [&](int c, uint2 codes) { reinterpret_cast<uint2*>(s_codes + (size_t)r * pitch)[c] = codes; });
    if (r < nt && (threadIdx.x & (kRowWarps * 32 - 1)) == 0) s_xs[r] = scale;
    __syncthreads();
    if (!work) return;

    int acc[kTokens][2];
#pragma unroll
    for (int t = 0; t < kTokens; ++t) acc[t][0] = acc[t][1] = 0;
    const uint8_t* codes = s_codes + (lane & 7) * 16;
    auto multiply = [&](int k0, const int4 (&ra)[kAhead], const int4 (&rb)[kAhead]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k0 + i >= p.atoms) break;
#pragma unroll
            for (int t = 0; t < kTokens; ++t)
                if (t < nt) {
                    const int4 x = *reinterpret_cast<const int4*>(codes + (size_t)t * pitch + (k0 + i) * 128);
                    acc[t][0] = dot16(ra[i], x, acc[t][0]);
                    acc[t][1] = dot16(rb[i], x, acc[t][1]);
                }
        }
    };
    for (int k0 = 0; k0 < p.atoms; k0 += 2 * kAhead) {
        request(k0 + kAhead, wa[1], wb[1]);
        multiply(k0, wa[0], wb[0]);
        request(k0 + 2 * kAhead, wa[0], wb[0]);
        multiply(k0 + kAhead, wa[1], wb[1]);
    }
    // the eight lanes of a row
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            acc[t][0] += __shfl_xor_sync(0xffffffffu, acc[t][0], o);
            acc[t][1] += __shfl_xor_sync(0xffffffffu, acc[t][1], o);
        }
    // lane j of a row's eight finishes token j
    const int q = lane >> 3;
    const float* ws = p.w_scale + (size_t)ti.x * p.a_rows + row0 + q;
    const float wsa = __ldg(ws), wsb = __ldg(ws + apart);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
        if (t >= nt || (lane & 7) != t) continue;
        const float xs = s_xs[t];
        const float va = __int2float_rn(acc[t][0]) * xs * wsa, vb = __int2float_rn(acc[t][1]) * xs * wsb;
        const size_t out_row = (size_t)(ti.y + t) * (size_t)p.out_ld;
        if (!kGateUp) {
            float* y = reinterpret_cast<float*>(p.out) + out_row + f0 + q;
            y[0] = va;
            y[4] = vb;
            continue;
        }
        __nv_bfloat16* h = reinterpret_cast<__nv_bfloat16*>(p.out) + out_row + f0 + q;
        const float g = p.clamp > 0.0f ? clamp_nan(va, p.clamp) : va;
        const float u = p.clamp > 0.0f ? clamp_nan(vb, p.clamp) : vb;
        const float pr = p.route_probs != nullptr ? __ldg(p.route_probs + __ldg(p.perm + ti.w + t)) : 1.0f;
        if (swiglu) {
            float hv = g * sigmoid_approx(g) * u;
            if (p.route_probs != nullptr) hv *= pr;
            h[0] = __float2bfloat16_rn(hv);
        } else {
            const float ra = g > 0.0f || g != g ? g : 0.0f, rb = u > 0.0f || u != u ? u : 0.0f;  // a NaN stays NaN
            float ha = ra * ra, hb = rb * rb;
            if (p.route_probs != nullptr) {
                ha *= pr;
                hb *= pr;
            }
            h[0] = __float2bfloat16_rn(ha);
            h[4] = __float2bfloat16_rn(hb);
        }
    }
}

template <bool kGateUp, int kTokens>
cudaError_t launch_gemv(const GemvArgs& a, int tokens, int max_tiles, cudaStream_t s) {
    constexpr int kDevices = 64;
    static bool done[kDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!done[dev]) {
        err = cudaFuncSetAttribute(moe_gemv_int8_kernel<kGateUp, kTokens>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)kGvSmemMax);
        if (err != cudaSuccess) return err;
        done[dev] = true;
    }
    const dim3 grid((unsigned)((a.units + kGvWarps - 1) / kGvWarps), (unsigned)max_tiles);
    return launch_dependent(moe_gemv_int8_kernel<kGateUp, kTokens>, grid, dim3(kGvThreads),
                            (size_t)tokens * a.g.atoms * 128, s, a);
}

template <bool kGateUp>
cudaError_t launch_by_tokens(const GemvArgs& a, int tokens, int max_tiles, cudaStream_t s) {
    if (tokens == 1) return launch_gemv<kGateUp, 1>(a, tokens, max_tiles, s);
    if (tokens == 2) return launch_gemv<kGateUp, 2>(a, tokens, max_tiles, s);
    return launch_gemv<kGateUp, kGvTokens>(a, tokens, max_tiles, s);
}

}  // namespace

bool int8_gemv_experts(long long max_live) { return max_live <= kGvTokens; }

cudaError_t launch_gemv1_int8(const uint8_t* w, const __nv_bfloat16* x, const Int8Gemm& g, int hidden, int top_k,
                              int tokens, int max_tiles, cudaStream_t s) {
    GemvArgs a{};
    a.g = g;
    a.x = reinterpret_cast<const uint4*>(x);
    a.ld_x = hidden / 8;
    a.w = w;
    a.cols_in = hidden;
    a.top_k = top_k;
    a.units = g.out_cols / (g.relu2 ? kUnitRows : kUnitRows / 2);
    return launch_by_tokens<true>(a, tokens, max_tiles, s);
}

cudaError_t launch_gemv2_int8(const uint8_t* w, const __nv_bfloat16* h, const Int8Gemm& g, int ffn, long long ld_h,
                              int tokens, int max_tiles, cudaStream_t s) {
    GemvArgs a{};
    a.g = g;
    a.x = reinterpret_cast<const uint4*>(h);
    a.ld_x = ld_h / 8;
    a.w = w;
    a.cols_in = ffn;
    a.units = g.out_cols / kUnitRows;
    return launch_by_tokens<false>(a, tokens, max_tiles, s);
}

}  // namespace moe
