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

namespace moe {

constexpr int kAtomK8 = 128;  // int8 elements of a 128-byte swizzle atom

__device__ __forceinline__ float int8_scale(float amax) {
    if (!(amax < INFINITY)) return __uint_as_float(0x7fc00000u);
    return amax > 0.0f ? __fdiv_rn(amax, 127.0f) : 1.0f;
}
__device__ __forceinline__ int int8_code(float v, float scale) {
    const float q = __fdiv_rn(v, scale);  // NaN when the scale is: cvt gives 0
    return __float2int_rn(fminf(fmaxf(q, -127.0f), 127.0f));
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
};

cudaError_t launch_gemm1_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s);
cudaError_t launch_gemm2_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s);
cudaError_t launch_gemm_dense_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                                   cudaStream_t s);
cudaError_t launch_int8_quantize_rows(const __nv_bfloat16* in, long long rows, int cols, long long ld_in, int8_t* q,
                                      float* scales, const int* live, cudaStream_t s);
cudaError_t launch_gather_int8(const __nv_bfloat16* x, const int* live, int max_live, int H, int hp, int k,
                               const int* inv, uint8_t* xq, float* xs, const unsigned* status, cudaStream_t s);
cudaError_t launch_quantize_h_int8(const __nv_bfloat16* h, const int* live, int max_live, int k, int fp,
                                   const int* inv, uint8_t* hq, float* hs, const unsigned* status, cudaStream_t s);
cudaError_t launch_prepare_int8(const moe_plan* p, const __nv_bfloat16* wg, const __nv_bfloat16* wu,
                                const __nv_bfloat16* wd, void* buf, cudaStream_t s);

}  // namespace moe
