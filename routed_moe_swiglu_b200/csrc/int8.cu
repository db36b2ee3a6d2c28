// int8.cu -- the 8-bit integer precision's quantisers: rows of bf16 through the
// public entry point, token rows of x into their padded route rows, the bf16 h
// rows of the gate/up GEMM, and the expert weights into the GEMMs' layout (the
// arithmetic is in int8.cuh); and the dense product's entry points.
//
// Layout of the expert weights: blocks of 16 KB, one per (expert, 128 weight
// rows, 128 elements of K), [128 rows][128 codes], the blocks of one row block
// after one another along K, so that a pipeline stage of two blocks is one
// 32 KB run of memory.  W1's rows interleave gate and up in groups of 16 as the
// bf16 weights do; padding (K past H or F, rows past F or H) holds code 0 and
// scale 0.  Each weight row's scale stands at the row's own place in [E][rows].
#include <cmath>
#include <type_traits>

#include "int8.cuh"
#include "mxfp8.cuh"

namespace moe {
namespace {

constexpr int kI8Threads = 128;

// A row is taken by kWarps warps, which hold up to kHeld 16-byte chunks a lane: one read of the
// row serves its largest magnitude and its codes.  Rows longer than the most held read the rest
// twice.
constexpr int kMostHeld = 8;

// Rows of bf16, kWarps warps a row.
template <int kWarps, int kHeld>
__global__ void __launch_bounds__(kI8Threads, kHeld > 4 ? 6 : 10) int8_quantize_rows_kernel(const uint4* __restrict__ in, long long rows,
                                                                        int chunks, long long ld_chunks,
                                                                        const int* __restrict__ live,
                                                                        uint2* __restrict__ q,
                                                                        float* __restrict__ scales) {
    constexpr int kRows = kI8Threads / 32 / kWarps;  // rows a block holds
    __shared__ uint32_t s_red[kI8Threads / 32];
    pdl_wait();
    pdl_trigger();  // after the wait: a kernel released here may read what came before this one
    long long n = rows;
    if (live != nullptr) {
        const long long l = (long long)__ldg(live);
        n = l < 0 ? 0 : (l < rows ? l : rows);
    }
    for (long long r0 = (long long)blockIdx.x * kRows; r0 < n; r0 += (long long)gridDim.x * kRows) {
        const long long r = r0 + threadIdx.x / (kWarps * 32);
        const bool on = r < n;
        const float s = int8_quantize_row<kWarps, kHeld>(in + r * ld_chunks, chunks, on, s_red, [] {},
                                                    [&](int c, uint2 codes) { q[r * chunks + c] = codes; });
        if (on && (threadIdx.x & (kWarps * 32 - 1)) == 0) scales[r] = s;
    }
}

// x rows: a block per token writes the token's codes and scale to each of its k padded route
// rows (zero codes from H to the pitch hp).
template <int kHeld>
__global__ void __launch_bounds__(kI8Threads) gather_rows_int8_kernel(const uint4* __restrict__ x,
                                                                      const int* __restrict__ live, int max_live,
                                                                      int H, int hp, int k,
                                                                      const int* __restrict__ inv,
                                                                      uint2* __restrict__ xq, float* __restrict__ xs,
                                                                      const unsigned* status) {
    __shared__ int s_prow[kMaxTopK];
    __shared__ uint32_t s_red[kI8Threads / 32];
    // The permute before this kernel releases it after its own wait, so x and the live count are
    // there: the first row's codes are computed before this kernel waits for the permutation.  The
    // gate/up GEMM is released after that wait (its `early`).
    const int n = clamp_live(live, max_live);
    const int chunks = H / 8, chunks_out = hp / 8;
    bool waited = false, go = true;
    auto wait = [&] {
        if (!waited) {
            pdl_wait();
            pdl_trigger();
            go = !forward_poisoned(status);
            waited = true;
        }
    };
    for (int t = blockIdx.x; t < n && go; t += gridDim.x) {
        auto ready = [&] {
            wait();
            __syncthreads();  // the last token's readers of s_prow are done
            if (threadIdx.x < k) s_prow[threadIdx.x] = go ? __ldg(inv + (size_t)t * k + threadIdx.x) : -1;
            __syncthreads();
        };
        auto put = [&](int c, uint2 codes) {
            for (int j = 0; j < k; ++j) {
                const int pr = s_prow[j];
                if (pr >= 0) xq[(size_t)pr * chunks_out + c] = codes;
            }
        };
        const float s = int8_quantize_row<kI8Threads / 32, kHeld>(x + (size_t)t * chunks, chunks, true, s_red, ready, put);
        if (threadIdx.x < k && s_prow[threadIdx.x] >= 0) xs[s_prow[threadIdx.x]] = s;
        for (int c = chunks + threadIdx.x; c < chunks_out; c += kI8Threads) put(c, make_uint2(0u, 0u));
    }
    wait();  // every block, so that the kernel never ends before the permute
}

// h rows: kWarps warps per live route quantise its bf16 row of the gate/up GEMM (pitch fp, zeros
// past F) with the row's own scale.
template <int kWarps, int kHeld>
__global__ void __launch_bounds__(kI8Threads, kHeld > 4 ? 6 : 10) quantize_h_int8_kernel(const uint4* __restrict__ h,
                                                                     const int* __restrict__ live, int max_live,
                                                                     int k, int fp, const int* __restrict__ inv,
                                                                     uint2* __restrict__ hq, float* __restrict__ hs,
                                                                     const unsigned* status) {
    constexpr int kRows = kI8Threads / 32 / kWarps;
    __shared__ uint32_t s_red[kI8Threads / 32];
    pdl_wait();
    pdl_trigger();  // after the wait: the down GEMM's `early`
    const long long n = (long long)live_rows(live, max_live, status) * k;
    const int chunks = fp / 8;
    for (long long i0 = (long long)blockIdx.x * kRows; i0 < n; i0 += (long long)gridDim.x * kRows) {
        const long long i = i0 + threadIdx.x / (kWarps * 32);
        const int pr = i < n ? __ldg(inv + i) : -1;
        const float s = int8_quantize_row<kWarps, kHeld>(h + (size_t)(pr < 0 ? 0 : pr) * chunks, chunks, pr >= 0, s_red,
                                                    [] {}, [&](int c, uint2 codes) { hq[(size_t)pr * chunks + c] = codes; });
        if (pr >= 0 && (threadIdx.x & (kWarps * 32 - 1)) == 0) hs[pr] = s;
    }
}

// Weights: a block per weight row, codes in 16 KB blocks (see the header), scale beside.
__global__ void __launch_bounds__(kI8Threads) prepare_int8_kernel(
    const uint4* __restrict__ wg, const uint4* __restrict__ wu, const uint4* __restrict__ wd, uint2* __restrict__ w1q,
    float* __restrict__ w1s, uint2* __restrict__ w2q, float* __restrict__ w2s, int E, int F, int H, int w1r, int hr,
    int at1, int at2, int relu2) {
    __shared__ uint32_t s_red[kI8Threads / 32];
    const long long rows1 = (long long)E * (relu2 ? 1 : 2) * F;
    const long long rows2 = (long long)E * H;
    for (long long row = blockIdx.x; row < rows1 + rows2; row += gridDim.x) {
        const bool first = row < rows1;
        const uint4* src;
        long long e;
        int wrow;  // row within the expert's prepared matrix
        if (first) {
            const int per_e = relu2 ? F : 2 * F;
            e = row / per_e;
            const int rem = (int)(row - e * per_e);
            const int gu = rem / F, f = rem - gu * F;
            src = (gu ? wu : wg) + ((size_t)e * F + f) * (H / 8);
            wrow = relu2 ? f : (f >> 6) * 128 + ((f >> 4) & 3) * 32 + gu * 16 + (f & 15);
        } else {
            const long long r2 = row - rows1;
            e = r2 / H;
            wrow = (int)(r2 - e * H);
            src = wd + (size_t)r2 * (F / 8);
        }
        const int chunks = (first ? H : F) / 8, atoms = first ? at1 : at2, per = first ? w1r : hr;
        const long long grow = e * per + wrow;
        uint2* dst = (first ? w1q : w2q) + ((size_t)(grow >> 7) * atoms * 128 + (grow & 127)) * 16;
        const float s = int8_quantize_row<kI8Threads / 32, kMostHeld>(src, chunks, true, s_red, [] {}, [&](int c, uint2 codes) {
            dst[(size_t)(c >> 4) * (128 * 16) + (c & 15)] = codes;
        });
        if (threadIdx.x == 0) (first ? w1s : w2s)[grow] = s;
    }
}

int capped_grid(long long items, int per_sm) {
    const long long cap = (long long)num_sms() * per_sm;
    return (int)(items < 1 ? 1 : (items > cap ? cap : items));
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

constexpr long long kMaxRowsI8 = 1ll << 24;
constexpr int kMaxColsI8 = 1 << 20;

// Checks that int8_matmul and int8_linear share (the activations apart).
moe_status check_product(long long rows, int cols_in, const void* w, const float* w_scales, int cols_out,
                         const void* out, long long ld_out) {
    if (w == nullptr || w_scales == nullptr || (rows != 0 && out == nullptr)) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || cols_in <= 0 || cols_out <= 0 || ld_out < cols_out) return MOE_ERR_INVALID_ARG;
    // 131,071 products of -128 * -128 fill an int32 sum
    if (cols_in % 16 != 0 || cols_in > MOE_INT8_MAX_K || cols_out > kMaxColsI8 || rows > kMaxRowsI8)
        return MOE_ERR_UNSUPPORTED;
    if (!is_aligned(w, 16) || !is_aligned(w_scales, 4)) return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

// Activation rows of a tile of the wide product: fewer than 256 where the last round of tiles would
// leave most CTA pairs idle and more, smaller tiles fill it.  A tile takes what its SMs take in, 128
// weight rows and half of its own each (1236 x 2224 -> 7678: 150 tiles of 256 on 74 pairs, 31.0 us, or
// 210 of 192, 28.6).
int dense_tile_rows(long long rows, int n_tiles) {
    int best = kRouteTile;
    double least = 0.0;
    for (int h = kRouteTile; h >= 128 && rows > kRouteTile; h -= 32) {
        const long long tiles = (rows + h - 1) / h * n_tiles, pairs = num_sms() / 2;
        const double cost = (double)((tiles + pairs - 1) / pairs) * (128 + h / 2);
        if (h == kRouteTile || cost < 0.97 * least) {
            best = h;
            least = cost;
        }
    }
    return best;
}

Int8Gemm dense_params(long long rows, int cols_in, const float* x_scales, const float* w_scales, int cols_out,
                      void* out, long long ld_out, int out_bf16, const int* live, unsigned* status) {
    Int8Gemm g{};
    g.status_flags = status;
    g.out = out;
    g.out_ld = ld_out;
    g.out_cols = cols_out;
    g.n_tiles = (cols_out + 255) / 256;
    g.atoms = (cols_in + kAtomK8 - 1) / kAtomK8;
    g.wait_limit_ns = kWaitLimitNs;
    g.row_scale = x_scales;
    g.w_scale = w_scales;
    g.live = live;
    g.rows = (int)rows;
    g.out_bf16 = out_bf16;
    g.tile_rows = dense_tile_rows(rows, g.n_tiles);
    // Weights that take much of L2: blocks of eight row tiles, so that the pairs of a wave read few
    // rows of both operands (8192^3: 17 of each operand's 32 tiles a wave instead of 34, 423 -> 398 us
    // sustained); smaller ones stay in L2 in any order, and row by row writes out in longer runs
    // (16384 x 2048 -> 8192: 209 us, 218 in blocks).
    g.raster = (long long)cols_in * cols_out > (32ll << 20) ? 8 : 1;
    return g;
}

// Rows of K bytes; columns past K and rows past the last read as zero.
bool row_map(CUtensorMap* map, const void* base, long long rows, int cols, long long ld, unsigned box_rows) {
    const unsigned long long dims[2] = {(unsigned long long)cols, (unsigned long long)rows};
    const unsigned long long pitch[1] = {(unsigned long long)ld};
    const unsigned box[2] = {128, box_rows};
    return make_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, pitch, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Whether 128 x 128 tiles with K split over clusters (gemm_int8_few.cu) beat 256 x 256 tiles of CTA
// pairs.  Both are bound by what an SM takes in, and the split one pays for draining and adding
// partial sums.  Estimates in us, fitted to 105 sizes (K 1024..8192, N 512..16384, 16..1024
// tokens); at K 8192, N 4096: 64 tokens 11.6 split against 18.0, 256 tokens 17.4 against 24.5,
// 1024 tokens 38.8 against 26.1.
bool few_is_faster(const Int8Gemm& g, int cols_in) {
    const double sms = num_sms(), K = cols_in;
    const long long rows = g.rows;
    if (rows > 128ll * 65535) return false;  // row tiles are a grid's second dimension
    const double wide_n = rows < g.tile_rows ? (double)((rows + 31) / 32 * 32) : (double)g.tile_rows;
    const long long wide = (rows + g.tile_rows - 1) / g.tile_rows * g.n_tiles;
    const double waves = (double)((wide + (long long)(sms / 2) - 1) / (long long)(sms / 2));
    const double t_wide = 3.0 + (rows > 128 ? 2.2 : 0.0) + waves * K * (128.0 + wide_n / 2) / 88e3;
    const double few_n = rows < 128 ? (double)((rows + 15) / 16 * 16) : 128.0;
    const long long tiles = (rows + 127) / 128 * ((g.out_cols + 127) / 128);
    const int split = int8_split_for(tiles, g.atoms);
    const double per_sm = (double)((tiles * split + (long long)sms - 1) / (long long)sms);  // CTAs
    const double t_few = 3.3 + 3.6 * few_n / 128 + per_sm * K / split * (128.0 + few_n) / 70e3;
    return t_few < t_wide;
}

moe_status run_dense(const Int8Gemm& g, const int8_t* x, int cols_in, long long ld_x, const int8_t* w,
                     cudaStream_t s) {
    CUtensorMap tA;
    BoxMaps8 tB;
    if (!row_map(&tA, w, g.out_cols, cols_in, cols_in, 128)) return MOE_ERR_CUDA;
    const long long tiles = ((long long)g.rows + g.tile_rows - 1) / g.tile_rows * g.n_tiles;
    const bool few = few_is_faster(g, cols_in);
    // the heights that tiles of these rows can have: any with a live count, else a full and a last one
    for (int i = 0; i < 8; ++i) {
        const int h = few ? 16 * (i + 1) : 32 * (i + 1);
        const int top = few ? 128 : g.tile_rows, last = (int)(g.rows % top), step = few ? 16 : 32;
        const bool used = g.live != nullptr || (g.rows >= top && h == top) ||
                          (last != 0 && h == (last + step - 1) / step * step);
        if (used && !row_map(&tB.m[i], x, g.rows, cols_in, ld_x, 16u * (unsigned)(i + 1))) return MOE_ERR_CUDA;
    }
    const cudaError_t e = few ? launch_int8_few(tA, tB, g, cols_in, s) : launch_gemm_dense_int8(tA, tB, g, tiles, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t linear_scales_offset(long long rows, int cols_in) {
    return ((size_t)rows * (size_t)cols_in + 255) & ~size_t(255);
}

}  // namespace

// Whether `rows` rows of `chunks` 16-byte chunks are taken by a warp each: rows a warp can hold,
// and enough of them to fill the SMs; else a block of four warps takes one.
static bool warp_per_row(long long rows, int chunks) {
    return chunks <= kMostHeld * 32 && rows >= (long long)num_sms() * 16;
}

// Calls f with the warps a row gets and the chunks a lane holds (2, 4 or 8) as constants.
template <class F>
static cudaError_t by_row(bool warp, int chunks, F f) {
    const int need = (chunks + (warp ? 31 : 127)) / (warp ? 32 : 128);
    auto held = [&](auto warps) {
        if (need <= 2) return f(warps, std::integral_constant<int, 2>());
        if (need <= 4) return f(warps, std::integral_constant<int, 4>());
        return f(warps, std::integral_constant<int, kMostHeld>());
    };
    return warp ? held(std::integral_constant<int, 1>()) : held(std::integral_constant<int, 4>());
}

cudaError_t launch_int8_quantize_rows(const __nv_bfloat16* in, long long rows, int cols, long long ld_in, int8_t* q,
                                      float* scales, const int* live, cudaStream_t s) {
    return by_row(warp_per_row(rows, cols / 8), cols / 8, [&](auto warps, auto held) {
        constexpr int kRows = 4 / warps.value;
        return launch_dependent(int8_quantize_rows_kernel<warps.value, held.value>,
                                dim3(capped_grid((rows + kRows - 1) / kRows, 64)), dim3(kI8Threads), 0, s,
                                reinterpret_cast<const uint4*>(in), rows, cols / 8, ld_in / 8, live,
                                reinterpret_cast<uint2*>(q), scales);
    });
}

cudaError_t launch_gather_int8(const __nv_bfloat16* x, const int* live, int max_live, int H, int hp, int k,
                               const int* inv, uint8_t* xq, float* xs, const unsigned* status, cudaStream_t s) {
    return by_row(false, H / 8, [&](auto, auto held) {
        return launch_dependent(gather_rows_int8_kernel<held.value>, dim3(capped_grid(max_live, 16)),
                                dim3(kI8Threads), 0, s, reinterpret_cast<const uint4*>(x), live, max_live, H, hp, k,
                                inv, reinterpret_cast<uint2*>(xq), xs, status);
    });
}

cudaError_t launch_quantize_h_int8(const __nv_bfloat16* h, const int* live, int max_live, int k, int fp,
                                   const int* inv, uint8_t* hq, float* hs, const unsigned* status, cudaStream_t s) {
    const long long rows = (long long)max_live * k;
    return by_row(warp_per_row(rows, fp / 8), fp / 8, [&](auto warps, auto held) {
        constexpr int kRows = 4 / warps.value;
        return launch_dependent(quantize_h_int8_kernel<warps.value, held.value>,
                                dim3(capped_grid((rows + kRows - 1) / kRows, 64)), dim3(kI8Threads), 0, s,
                                reinterpret_cast<const uint4*>(h), live, max_live, k, fp, inv,
                                reinterpret_cast<uint2*>(hq), hs, status);
    });
}

cudaError_t launch_prepare_int8(const moe_plan* p, const __nv_bfloat16* wg, const __nv_bfloat16* wu,
                                const __nv_bfloat16* wd, void* buf, cudaStream_t s) {
    uint8_t* base = static_cast<uint8_t*>(buf);
    const int E = p->d.num_experts, F = p->d.ffn, H = p->d.hidden;
    const bool relu2 = (p->d.flags & MOE_FLAG_SQUARED_RELU) != 0;
    // padding codes and scales are zero
    const cudaError_t err = cudaMemsetAsync(base, 0, p->wb.total, s);
    if (err != cudaSuccess) return err;
    prepare_int8_kernel<<<num_sms() * 16, kI8Threads, 0, s>>>(
        reinterpret_cast<const uint4*>(wg), reinterpret_cast<const uint4*>(wu), reinterpret_cast<const uint4*>(wd),
        reinterpret_cast<uint2*>(base + p->wb.w1), reinterpret_cast<float*>(base + p->wb.w1s),
        reinterpret_cast<uint2*>(base + p->wb.w2), reinterpret_cast<float*>(base + p->wb.w2s), E, F, H, (int)p->w1r,
        (int)p->hr, p->ks1, p->ks2, relu2 ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status int8_quantize_rows(const void* in, long long rows, int cols, long long ld_in, int8_t* q, float* scales,
                              const int* live_rows_dev, void* stream) {
    if (rows != 0 && (in == nullptr || q == nullptr || scales == nullptr)) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || cols <= 0 || ld_in < cols) return MOE_ERR_INVALID_ARG;
    if (cols % 8 != 0) return MOE_ERR_UNSUPPORTED;
    if (ld_in % 8 != 0 || !is_aligned(in, 16) || !is_aligned(q, 8) || !is_aligned(scales, 4)) return MOE_ERR_ALIGNMENT;
    if (rows == 0) return MOE_OK;
    const cudaError_t e = launch_int8_quantize_rows(static_cast<const __nv_bfloat16*>(in), rows, cols, ld_in, q, scales,
                                                    live_rows_dev, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status int8_matmul(const int8_t* x, const float* x_scales, long long rows, int cols_in, long long ld_x,
                       const int8_t* w, const float* w_scales, int cols_out, void* out, long long ld_out,
                       int out_bf16, const int* live_rows_dev, unsigned* status_dev, void* stream) {
    if ((rows != 0 && (x == nullptr || x_scales == nullptr)) || ld_x < cols_in) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_product(rows, cols_in, w, w_scales, cols_out, out, ld_out);
    if (st != MOE_OK) return st;
    if (ld_x % 16 != 0 || !is_aligned(x, 16) || !is_aligned(x_scales, 4) || !is_aligned(out, out_bf16 ? 2 : 4))
        return MOE_ERR_ALIGNMENT;
    if (rows == 0) return MOE_OK;
    const Int8Gemm g = dense_params(rows, cols_in, x_scales, w_scales, cols_out, out, ld_out, out_bf16, live_rows_dev,
                                    status_dev);
    return run_dense(g, x, cols_in, ld_x, w, static_cast<cudaStream_t>(stream));
}

size_t int8_linear_workspace_bytes(long long rows, int cols_in) {
    if (rows < 0 || cols_in <= 0) return 0;
    return linear_scales_offset(rows, cols_in) + (((size_t)rows * 4 + 255) & ~size_t(255)) + 256;
}

moe_status int8_linear(const void* x, long long rows, int cols_in, long long ld_x, const int8_t* w,
                       const float* w_scales, int cols_out, void* out, long long ld_out, int out_bf16,
                       const int* live_rows_dev, void* workspace, size_t ws_bytes, unsigned* status_dev,
                       void* stream) {
    if ((rows != 0 && x == nullptr) || workspace == nullptr || ld_x < cols_in) return MOE_ERR_INVALID_ARG;
    const moe_status st = check_product(rows, cols_in, w, w_scales, cols_out, out, ld_out);
    if (st != MOE_OK) return st;
    if (ws_bytes < int8_linear_workspace_bytes(rows, cols_in)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (ld_x % 8 != 0 || !is_aligned(x, 16) || !is_aligned(workspace, 256) || !is_aligned(out, out_bf16 ? 2 : 4))
        return MOE_ERR_ALIGNMENT;
    if (rows == 0) return MOE_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int8_t* q = static_cast<int8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + linear_scales_offset(rows, cols_in));
    Int8Gemm g = dense_params(rows, cols_in, scales, w_scales, cols_out, out, ld_out, out_bf16, live_rows_dev,
                              status_dev);
    const __nv_bfloat16* rows_in = static_cast<const __nv_bfloat16*>(x);
    if (int8_few_fused_fits(rows, cols_in, cols_out)) {
        CUtensorMap tA;
        if (!row_map(&tA, w, cols_out, cols_in, cols_in, 128)) return MOE_ERR_CUDA;
        return launch_int8_few_fused(tA, rows_in, ld_x, g, cols_in, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    if (launch_int8_quantize_rows(rows_in, rows, cols_in, ld_x, q, scales, live_rows_dev, s) != cudaSuccess)
        return MOE_ERR_CUDA;
    g.early = 1;  // the quantiser releases the product after its own wait
    return run_dense(g, q, cols_in, cols_in, w, s);
}

}  // extern "C"
