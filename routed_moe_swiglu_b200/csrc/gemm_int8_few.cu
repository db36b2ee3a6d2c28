// gemm_int8_few.cu -- the dense 8-bit product of few tokens: K is split over the
// CTAs of a cluster.
//
// With few tokens the time is that of reading the weights, and a wide tile of
// weight rows leaves most SMs without one.  Here a CTA takes 128 weight rows and
// a slice of K, the up to eight CTAs of a cluster share a tile's K, and their
// int32 partial sums (exact, so their order is of no account) are added through
// distributed shared memory; each CTA finishes every S-th token.
//
//   kFused   up to 16 tokens of bf16: each CTA quantises its own slice of the
//            rows into the swizzled operand layout in shared memory; the rows'
//            largest magnitudes meet in one cluster barrier.  One launch does all.
//   !kFused  up to 128 tokens a tile, whose codes TMA loads beside the weights.
//
// Roles (6 warps): warp 0 issues TMA loads, warp 1 owns TMEM and issues the MMAs
// (tcgen05 kind::i8, M = 128), warps 2-5 quantise (kFused) and drain.  Every
// mbarrier wait is bounded; a wait that gave up is followed by the same cluster
// barriers as any other, so no CTA is left alone in one.
//
// One token, 2048 -> 4096: 5.95 us, where reading the weights takes 1.3: launch,
// cluster start, quantising, one chain of loads, the exchange of partial sums and
// the end, about a microsecond each.  As two launches of the wide kernels 8.8 us.
// Sixteen tokens: 7.3 us, their rows' loads side by side (9.0 row after row).
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kFewThreads = 192;
constexpr int kWorkers = 128;              // warps 2..5
constexpr int kFewTokens = 128;            // tokens of a tile at most
constexpr int kFusedTokens = 16;
constexpr int kFusedAtoms = 16;            // 128-element atoms of a K slice that kFused holds
constexpr uint32_t kAAtom = 128 * 128;     // 128 weight rows of 128 bytes
constexpr int kMaxCluster = 8;

template <bool kFused>
struct FewCfg {
    static constexpr int kTokens = kFused ? kFusedTokens : kFewTokens;
    static constexpr int kStages = kFused ? 4 : 3;
    static constexpr uint32_t kBSlot = kTokens * 128;  // an atom of the tokens
    static constexpr uint32_t kBBytes = kBSlot * (kFused ? kFusedAtoms : kStages);
    static constexpr uint32_t kPartBytes = kTokens * 128 * 4;  // takes the weight stages' place after the MMAs
    static constexpr uint32_t kOperands = kStages * kAAtom + kBBytes;
    static constexpr uint32_t kTmemCols = kFused ? 32 : 128;
    static constexpr size_t kSmem = 1024 + kOperands;
    static_assert(kPartBytes <= kOperands, "the partial sums take the operands' place");
};

struct __align__(8) FewShared {
    uint64_t full[4], empty[4], acc_full, b_ready;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t amax[kMaxCluster][kFusedTokens];  // kFused: each CTA of the cluster writes its row
};

struct FewArgs {
    const uint4* x;          // kFused: bf16 rows
    long long ld_x;          // their pitch, 16-byte chunks
    const float* x_scales;   // !kFused
    const float* w_scales;
    void* out;
    long long ld_out;
    int cols_in, cols_out, rows;
    const int* live;
    int out_bf16, split, early;
    unsigned* status;
    unsigned long long wait_limit_ns;
};

__host__ __device__ constexpr uint32_t idesc_i8_cta(int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_i8_cta(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The two halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <bool kFused>
__global__ void __launch_bounds__(kFewThreads) gemm_int8_few_kernel(const __grid_constant__ CUtensorMap tmA,
                                                                    const __grid_constant__ BoxMaps8 tmB,
                                                                    const FewArgs a) {
    using C = FewCfg<kFused>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewShared sh;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + kStages * kAAtom;
    int* s_part = reinterpret_cast<int*>(smem);  // [token][128 channels], once every operand has been read
    volatile int* abort_flag = &sh.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = a.split, rank = (int)cluster_ctarank();
    const int n0 = (int)(blockIdx.x / S) * 128;                 // first weight row (output column)
    const int m0 = (int)blockIdx.y * kFewTokens;                // first token
    const int atoms = (a.cols_in + kAtomK8 - 1) / kAtomK8;
    const int k0 = (int)((long long)atoms * rank / S), k1 = (int)((long long)atoms * (rank + 1) / S);
    const int steps = k1 - k0;                                  // at least 1: S <= atoms
    pdl_trigger();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.acc_full, 1);
        mbar_init(&sh.b_ready, kWorkers);
        sh.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = sh.tmem_base;
    if (kFused) cluster_arrive();  // every CTA runs before another writes into its shared memory
    // `early` (see gemm_int8.cu): weights and sizes need no wait
    if (!a.early) pdl_wait();
    const int rows = a.live != nullptr ? clamp_live(a.live, a.rows) : a.rows;
    const int nt = min(rows - m0, kFewTokens);  // tokens of this tile
    if (kFused) cluster_wait();
    if (nt <= 0) {                              // the whole cluster: same tile
        if (a.early) pdl_wait();
        __syncthreads();
        if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
        return;
    }
    const int N = (nt + 15) & ~15;
    const uint32_t b_atom = kFused ? C::kBSlot : (uint32_t)N * 128u;
    auto timed_out = [&]() {
        *abort_flag = 1;
        if (a.status != nullptr) atomicOr(a.status, MOE_DEV_TIMEOUT);
    };

    float ws[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int issued = 0;
    bool ok = true;
    // step i of the slice into its stage: weights, and the tokens' codes (!kFused)
    auto request = [&](int i, bool w, bool b) {
        const int s = i % kStages;
        if (w) {
            mbar_arrive_expect_tx(&sh.full[s], kAAtom + (kFused ? 0u : b_atom));
            tma_load_2d(sA + s * kAAtom, &tmA, &sh.full[s], (k0 + i) * 128, n0);
        }
        if (b && !kFused)
            tma_load_2d(sB + s * C::kBSlot, &tmB.m[(N >> 4) - 1], &sh.full[s], (k0 + i) * 128, m0);
    };
    if (warp == 0 && lane == 0) {
        const int first = min(steps, kStages);
        for (int i = 0; i < first; ++i) request(i, true, false);
        if (a.early) pdl_wait();
        for (int i = 0; i < first; ++i) request(i, false, true);
        issued = first;
    } else if (a.early) {
        pdl_wait();
    }
    __syncwarp();

    // ---------------- kFused: worker warp w quantises rows w, w + 4, ... of the tile
    const int wt = (int)threadIdx.x - 64;  // worker thread
    if (kFused) {
        constexpr int kRows = kFusedTokens / 4;
        const int units = min(steps * 8, (a.cols_in - k0 * 128 + 15) / 16);  // 16 elements each, of a row's slice
        const uint4* src[kRows];
        if (wt >= 0) {
            uint32_t p[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = warp - 2 + 4 * i;
                src[i] = a.x + (size_t)(m0 + min(r, nt - 1)) * a.ld_x + (size_t)k0 * 16;
                p[i] = 0u;
            }
            for (int u = lane; u < units; u += 32)
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (warp - 2 + 4 * i < nt)
                        p[i] = int8_amax_pairs(__ldg(src[i] + 2 * u), int8_amax_pairs(__ldg(src[i] + 2 * u + 1), p[i]));
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int r = warp - 2 + 4 * i;
                const uint32_t m = __reduce_max_sync(0xffffffffu, int8_amax_bits(p[i]));
                // this slice's magnitude into every CTA's table
                if (r < nt && lane < S) st_cluster_u32(map_to_cta(smem_u32(&sh.amax[rank][r]), (uint32_t)lane), m);
            }
        }
        cluster_sync();
        if (wt >= 0) {
            // lane l works out row l % kRows of the warp's; all rows are then read side by side
            const int mine = warp - 2 + 4 * (lane % kRows);
            uint32_t m = 0u;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) m = c < S && mine < nt ? max(m, sh.amax[c][mine]) : m;
            const Int8Row own = int8_row(__uint_as_float(m));
            Int8Row row[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                row[i].scale = __shfl_sync(0xffffffffu, own.scale, i);
                row[i].inv = __shfl_sync(0xffffffffu, own.inv, i);
                row[i].divide = __shfl_sync(0xffffffffu, (int)own.divide, i) != 0;
            }
            for (int u = lane; u < units; u += 32) {
                uint4 v[kRows][2];
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (warp - 2 + 4 * i < nt) {
                        v[i][0] = __ldg(src[i] + 2 * u);
                        v[i][1] = __ldg(src[i] + 2 * u + 1);
                    }
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int r = warp - 2 + 4 * i;
                    if (r >= nt) break;
                    const uint2 lo = int8_codes8(v[i][0], row[i]), hi = int8_codes8(v[i][1], row[i]);
                    // the 128-byte swizzle: 16-byte chunk c of row r lies at c ^ (r % 8)
                    *reinterpret_cast<uint4*>(sB + r * 128 + (u >> 3) * C::kBSlot + (((u & 7) ^ (r & 7)) << 4)) =
                        make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&sh.b_ready);
        }
    }

    if (warp == 0) {
        if (lane == 0) {
            for (int i = issued; i < steps && ok; ++i) {
                ok = mbar_wait_bounded(&sh.empty[i % kStages], ((i / kStages) & 1) ^ 1, abort_flag, a.wait_limit_ns);
                if (ok) request(i, true, true);
            }
            if (!ok) timed_out();  // the MMA issuer then gives up too, and sees the copies land
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(sA)), b0 = sdesc_kmajor_sw128(smem_u32(sB));
            const uint32_t idesc = idesc_i8_cta(N);
            if (kFused) ok = mbar_wait_bounded(&sh.b_ready, 0, abort_flag, a.wait_limit_ns);
            int i = 0;
            for (; i < steps && ok; ++i) {
                const int s = i % kStages;
                ok = mbar_wait_bounded(&sh.full[s], (i / kStages) & 1, abort_flag, a.wait_limit_ns);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t da = a0 + (uint64_t)(s * (kAAtom >> 4));
                const uint64_t db = b0 + (uint64_t)((kFused ? i : s) * (C::kBSlot >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 32 elements of K each
                    mma_i8_cta(tmem_base, da + kk * 2, db + kk * 2, idesc, (i | kk) != 0 ? 1u : 0u);
                mma_commit(&sh.empty[s]);
            }
            if (!ok) {
                timed_out();
                int8_fills_land(sh.full, kStages, i);
            }
            mma_commit(&sh.acc_full);
        }
        __syncwarp();
    } else {
        // ---------------- drain: lanes are channels, TMEM columns tokens
        const int quad = warp & 3, ch = quad * 32 + lane;
        // the scales of this lane's four columns in the last step, meanwhile
        const int left = a.cols_out - n0 - lane * 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) ws[q] = q < left ? __ldg(a.w_scales + n0 + lane * 4 + q) : 0.0f;
        const bool got = __all_sync(0xffffffffu,
                                    mbar_wait_bounded(&sh.acc_full, 0, abort_flag, a.wait_limit_ns));
        if (!got && lane == 0) {
            timed_out();
            int8_fills_land(&sh.acc_full, 1, 0);  // told to stop by another role: MMAs in flight end before TMEM goes
        }
        __syncwarp();
        if (got) {
            tc_fence_after_sync();
            for (int c = 0; c < N; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(quad * 32) << 16) + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < nt) s_part[(c + j) * 128 + ch] = (int)v[j];
            }
            tc_fence_before_sync();
        }
    }
    cluster_sync();  // every CTA's partial sums are in its shared memory
    if (wt >= 0) {
        // a warp takes a token, a lane four channels: rows rank + S * (w, w + 4, ...)
        const int col = n0 + lane * 4, left = a.cols_out - col;  // columns of this lane inside out (may be <= 0)
        // whole stores of the lane's four columns: all inside, rows and base aligned for them
        const bool wide = left >= 4 && a.ld_out % 4 == 0 &&
                          (reinterpret_cast<uintptr_t>(a.out) & (a.out_bf16 != 0 ? 7 : 15)) == 0;
        const uint32_t part = smem_u32(s_part) + (uint32_t)lane * 16u;
#pragma unroll 1
        for (int r = rank + S * (warp - 2); r < nt; r += 4 * S) {
            int4 v[kMaxCluster];  // all on their way before the first is added
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                v[c] = c < S ? ld_cluster_v4(map_to_cta(part + (uint32_t)r * 512u, (uint32_t)c)) : make_int4(0, 0, 0, 0);
            int4 sum = v[0];
#pragma unroll
            for (int c = 1; c < kMaxCluster; ++c) {
                sum.x += v[c].x;
                sum.y += v[c].y;
                sum.z += v[c].z;
                sum.w += v[c].w;
            }
            float xs;
            if (kFused) {
                uint32_t m = 0u;
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c) m = c < S ? max(m, sh.amax[c][r]) : m;
                xs = int8_scale(__uint_as_float(m));
            } else {
                xs = __ldg(a.x_scales + m0 + r);
            }
            const float y[4] = {__int2float_rn(sum.x) * xs * ws[0], __int2float_rn(sum.y) * xs * ws[1],
                                __int2float_rn(sum.z) * xs * ws[2], __int2float_rn(sum.w) * xs * ws[3]};
            const size_t at = (size_t)(m0 + r) * (size_t)a.ld_out + col;
            if (a.out_bf16 != 0) {
                __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + at;
                if (wide) {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
                    *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                                *reinterpret_cast<const uint32_t*>(&hi));
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < left) dst[q] = __float2bfloat16_rn(y[q]);
                }
            } else {
                float* dst = reinterpret_cast<float*>(a.out) + at;
                if (wide) {
                    *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (q < left) dst[q] = y[q];
                }
            }
        }
    }
    cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, C::kTmemCols);
    }
}

template <bool kFused>
cudaError_t launch_few(const CUtensorMap& ta, const BoxMaps8& tb, FewArgs a, int row_tiles, cudaStream_t s) {
    constexpr int kDevices = 64;
    static bool configured[kDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        err = cudaFuncSetAttribute(gemm_int8_few_kernel<kFused>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)FewCfg<kFused>::kSmem);
        if (err != cudaSuccess) return err;
        configured[dev] = true;
    }
    const int col_tiles = (a.cols_out + 127) / 128;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(col_tiles * a.split), (unsigned)row_tiles);
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = FewCfg<kFused>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, gemm_int8_few_kernel<kFused>, ta, tb, a);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

// CTAs of a cluster: as many as fill the SMs once, or twice where each keeps four atoms of K (one
// token, 2048 -> 4096: 5.9 us with four CTAs of four atoms, 6.6 us with eight of two; 16 tokens,
// 8192 -> 4096: 9.5 us with eight of eight, 11.4 us with four of sixteen).
int int8_split_for(long long tiles, int atoms) {
    int s = 1;
    while (s < kMaxCluster && atoms >= 2 * s &&
           (tiles * s * 2 <= num_sms() || (tiles * s <= num_sms() && atoms >= 8 * s)))
        s *= 2;
    return s;
}

bool int8_few_fused_fits(long long rows, int cols_in, int cols_out) {
    if (rows > kFusedTokens) return false;
    const int atoms = (cols_in + kAtomK8 - 1) / kAtomK8;
    const int s = int8_split_for((cols_out + 127) / 128, atoms);
    return (atoms + s - 1) / s <= kFusedAtoms;
}

cudaError_t launch_int8_few_fused(const CUtensorMap& ta, const __nv_bfloat16* x, long long ld_x, const Int8Gemm& g,
                                  int cols_in, cudaStream_t s) {
    FewArgs a{};
    a.x = reinterpret_cast<const uint4*>(x);
    a.ld_x = ld_x / 8;
    a.w_scales = g.w_scale;
    a.out = g.out;
    a.ld_out = g.out_ld;
    a.cols_in = cols_in;
    a.cols_out = g.out_cols;
    a.rows = g.rows;
    a.live = g.live;
    a.out_bf16 = g.out_bf16;
    a.split = int8_split_for((g.out_cols + 127) / 128, (cols_in + kAtomK8 - 1) / kAtomK8);
    a.status = g.status_flags;
    a.wait_limit_ns = g.wait_limit_ns;
    return launch_few<true>(ta, BoxMaps8{}, a, 1, s);
}

cudaError_t launch_int8_few(const CUtensorMap& ta, const BoxMaps8& tb, const Int8Gemm& g, int cols_in, cudaStream_t s) {
    FewArgs a{};
    a.x_scales = g.row_scale;
    a.w_scales = g.w_scale;
    a.out = g.out;
    a.ld_out = g.out_ld;
    a.cols_in = cols_in;
    a.cols_out = g.out_cols;
    a.rows = g.rows;
    a.live = g.live;
    a.out_bf16 = g.out_bf16;
    a.early = g.early;
    a.status = g.status_flags;
    a.wait_limit_ns = g.wait_limit_ns;
    const int row_tiles = (g.rows + kFewTokens - 1) / kFewTokens;
    a.split = int8_split_for((long long)((g.out_cols + 127) / 128) * row_tiles, (cols_in + kAtomK8 - 1) / kAtomK8);
    return launch_few<false>(ta, tb, a, row_tiles, s);
}

}  // namespace moe
