// int8.cuh -- the 8-bit integer precision: the quantiser's arithmetic, the
// integer tensor-core instruction and the launchers of int8.cu and gemm_int8.cu.
//
// A row (a token's activations, a weight channel) is held as whole numbers of
// [-127, 127] and one fp32 scale:
//   amax  = the largest magnitude of the row
//   scale = amax / 127 in fp32 (1 for a row of zeros)
//   code  = value / scale in fp32 (correctly rounded), to the nearest whole
//           number, halves to even, clamped to [-127, 127] (a subnormal scale's
//           own rounding can leave a quotient past 127)
// A row with a NaN or an infinity gets scale NaN and codes 0: every product with
// it is NaN, and it never passes for a number.
#pragma once

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kAtomK8 = 128;  // int8 elements of a 128-byte swizzle atom

__device__ __forceinline__ float int8_scale(float amax) {
    if (!(amax < INFINITY)) return __uint_as_float(0x7fc00000u);
    return amax > 0.0f ? __fdiv_rn(amax, 127.0f) : 1.0f;
}
__device__ __forceinline__ int int8_code(float v, float scale) {
    const float q = __fdiv_rn(v, scale);
    return __float2int_rn(fminf(fmaxf(q, -127.0f), 127.0f));
}
__device__ __forceinline__ uint32_t int8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A row's scale with what its codes are computed by.
//
// Codes without a division.  With amax = A 2^a and |value| = X 2^b (A, X whole numbers below
// 256: bf16), value / scale is 127 X 2^e / A but for the roundings of the scale and of the
// quotient, e = b - a <= 0.  Either that ratio is a half (m + 1/2) or it lies at least
// 2^e / (2 A) > 2^e / 512 from every half, while the roundings move it by less than
// 254 * 2^e * 2^-23 < 2^e / 2^15: away from halves, value * inv with any inv within 2^-20 of
// 1 / scale gives the code.  A half needs 254 X 2^e = (2m + 1) A.  As 127 is a prime and
// 2m + 1 <= 254, either 127 divides A (A = 254: the scale is a power of two, 1 / scale and every
// product are exact, and halves go to even as they do in the division) or 2m + 1 = 127: the
// value is half of the largest.  Its quotient is one number for the whole row; inv is moved by
// 2^-21 of itself so that value * inv falls to the side of 63.5 that this quotient is rounded to.
struct Int8Row {
    float scale;
    float inv;
    bool divide;  // a subnormal scale (its rounding is coarser), or a row of NaN: see int8_codes8
};
__device__ __forceinline__ Int8Row int8_row(float amax) {
    Int8Row r;
    r.scale = int8_scale(amax);
    r.divide = !(r.scale >= 1.1754943508222875e-38f);
    r.inv = __frcp_rn(r.scale);
    if ((__float_as_uint(amax) & 0x007f0000u) != 0x007e0000u) {  // A != 254
        const float half = __fdiv_rn(0.5f * amax, r.scale);
        r.inv *= __float2int_rn(half) == 64 ? 1.0f + 0x1p-21f : 1.0f - 0x1p-21f;
    }
    return r;
}

// Codes of eight bf16 (16 bytes) of a row.
__device__ __forceinline__ uint2 int8_codes8(uint4 v, const Int8Row& row) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t q[8];
    if (!row.divide) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
            // adding 1.5 * 2^23 leaves the nearest whole number (halves to even) in the low bits
            q[i] = __float_as_uint(fmaf(f, row.inv, 12582912.0f));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
            q[i] = row.scale == row.scale ? (uint32_t)int8_code(f, row.scale) : 0u;
        }
    }
    return make_uint2(int8_pack4(q[0], q[1], q[2], q[3]), int8_pack4(q[4], q[5], q[6], q[7]));
}

// The largest magnitudes of bf16 pairs, as their 15 bits: these order as the values, with
// infinity and then NaN above every number.
__device__ __forceinline__ uint32_t int8_amax_pairs(uint4 v, uint32_t a) {
    a = __vmaxu2(a, v.x & 0x7fff7fffu);
    a = __vmaxu2(a, v.y & 0x7fff7fffu);
    a = __vmaxu2(a, v.z & 0x7fff7fffu);
    return __vmaxu2(a, v.w & 0x7fff7fffu);
}
// The larger of a pair, as the bits of an fp32.
__device__ __forceinline__ uint32_t int8_amax_bits(uint32_t a) { return max(a << 16, a & 0xffff0000u); }

// The largest of a row's kWarps warps (s_red: a word a warp of the block).
template <int kWarps>
__device__ __forceinline__ uint32_t int8_row_max(uint32_t a, uint32_t* s_red) {
    a = __reduce_max_sync(0xffffffffu, a);
    if (kWarps > 1) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s_red[warp] = a;
        __syncthreads();
        const int w0 = warp / kWarps * kWarps;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) a = max(a, s_red[w0 + w]);
    }
    return a;
}

// Quantises the row of `chunks` 16-byte chunks at src (none when !on): store(c, codes) for each
// chunk, after ready(); returns the scale.  Every thread of the row's warps calls it (with kWarps
// > 1, of the block).
template <int kWarps, int kHeld, class Ready, class Store>
__device__ __forceinline__ float int8_quantize_row(const uint4* src, int chunks, bool on, uint32_t* s_red, Ready ready,
                                                   Store store) {
    constexpr int kLanes = kWarps * 32;
    const int lane = threadIdx.x & (kLanes - 1);
    uint4 v[kHeld];
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int c = i * kLanes + lane;
        v[i] = on && c < chunks ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) a = int8_amax_pairs(v[i], a);
    if (on)
        for (int c = kHeld * kLanes + lane; c < chunks; c += kLanes) a = int8_amax_pairs(__ldg(src + c), a);
    const Int8Row row = int8_row(__uint_as_float(int8_row_max<kWarps>(int8_amax_bits(a), s_red)));
    ready();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int c = i * kLanes + lane;
        if (on && c < chunks) store(c, int8_codes8(v[i], row));
    }
    if (on)
        for (int c = kHeld * kLanes + lane; c < chunks; c += kLanes) store(c, int8_codes8(__ldg(src + c), row));
    return row.scale;
}

// Each thread of the warp reads 16 consecutive 32-bit columns of its TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// x clamped to [-c, c]; a NaN (a row that holds one) stays NaN.
__device__ __forceinline__ float clamp_nan(float x, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n\tmin.NaN.f32 %0, %0, %3;" : "=f"(r) : "f"(x), "f"(-c), "f"(c));
    return r;
}
// 1 / (1 + exp(-g)) from the approximate exponential and reciprocal (2^-22 and 1 ulp; the
// exponent's rounding adds |g| 2^-24): far below the bf16 step that h is rounded to.  0 below -87.3,
// where it is a subnormal; the other precisions' quotient is 0 there too.
__device__ __forceinline__ float sigmoid_approx(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// The MMA issuer's part of giving up at fill i of its n stages: no copy may land in shared memory that
// is no longer the kernel's.  Fills i to i + n - 1 are all that can be on their way, as a stage is
// refilled only once the issuer has used it.  Each gets 0.1 s: one that was asked for lands, one that
// was not ends the wait (nor does a pair's, if only the other CTA asked: its copies land meanwhile).
// (Called, not inlined: with the rare path out of the way one token's product takes 0.1 us less.)
static __device__ __noinline__ void int8_fills_land(uint64_t* full, int n, int i) {
    volatile int never = 0;
    for (int j = i; j < i + n; ++j) (void)mbar_wait_bounded(&full[j % n], (uint32_t)(j / n) & 1u, &never, 100000000ull);
}

struct Int8Gemm {
    const int4* tiles;              // grouped: {expert, first padded row, valid rows, first permuted row}
    const unsigned* status_words;   // grouped: the workspace's status words
    unsigned* status_flags;         // MOE_DEV_* bits (dense: may be null)
    void* out;                      // gate/up: bf16 h; down: fp32 y; dense: bf16 or fp32 rows
    long long out_ld;               // row pitch of out, elements
    int out_cols;                   // valid output columns
    int n_tiles;                    // tiles of 256 weight rows
    int atoms;                      // 128-byte atoms of K
    long long a_rows;               // grouped: weight rows of one expert (a multiple of 128)
    unsigned long long wait_limit_ns;
    const float* row_scale;         // per activation row (grouped: padded route row)
    const float* w_scale;           // per weight row (grouped: [E][a_rows])
    // gate/up variants, as GemmParams
    const int* perm;
    const float* route_probs;
    float clamp;
    int relu2;
    // dense
    const int* live;                // null: all rows
    int rows;
    int out_bf16;
    int tile_rows;                  // activation rows of a tile, a multiple of 32 up to 256
    int raster;                     // row tiles of a block of tiles
    int early;                      // launched by a kernel that waited before it released this one
};

cudaError_t launch_gemm1_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s);
cudaError_t launch_gemm2_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s);
cudaError_t launch_gemm_dense_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                                   cudaStream_t s);
// Few tokens (gemm_int8_few.cu): bf16 rows quantised in the same launch, where they fit, or codes.
int int8_split_for(long long tiles, int atoms);  // CTAs that share a tile's K
// The expert products of very few tokens (gemv_int8.cu), which quantise x and h themselves: whether a
// plan takes them, and the two products (w: the prepared weights; tokens:
// the plan's most live rows; max_tiles: experts with a route at most).
bool int8_gemv_experts(long long max_live);
cudaError_t launch_gemv1_int8(const uint8_t* w, const __nv_bfloat16* x, const Int8Gemm& g, int hidden, int top_k,
                              int tokens, int max_tiles, cudaStream_t s);
cudaError_t launch_gemv2_int8(const uint8_t* w, const __nv_bfloat16* h, const Int8Gemm& g, int ffn, long long ld_h,
                              int tokens, int max_tiles, cudaStream_t s);
bool int8_few_fused_fits(long long rows, int cols_in, int cols_out);
cudaError_t launch_int8_few_fused(const CUtensorMap& a, const __nv_bfloat16* x, long long ld_x, const Int8Gemm& g,
                                  int cols_in, cudaStream_t s);
cudaError_t launch_int8_few(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, int cols_in, cudaStream_t s);
cudaError_t launch_int8_quantize_rows(const __nv_bfloat16* in, long long rows, int cols, long long ld_in, int8_t* q,
                                      float* scales, const int* live, cudaStream_t s);
cudaError_t launch_gather_int8(const __nv_bfloat16* x, const int* live, int max_live, int H, int hp, int k,
                               const int* inv, uint8_t* xq, float* xs, const unsigned* status, cudaStream_t s);
cudaError_t launch_quantize_h_int8(const __nv_bfloat16* h, const int* live, int max_live, int k, int fp,
                                   const int* inv, uint8_t* hq, float* hs, const unsigned* status, cudaStream_t s);
cudaError_t launch_prepare_int8(const moe_plan* p, const __nv_bfloat16* wg, const __nv_bfloat16* wu,
                                const __nv_bfloat16* wd, void* buf, cudaStream_t s);

}  // namespace moe
