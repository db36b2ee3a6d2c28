// gemm_int8.cu -- matrix products in 8-bit integers with an fp32 scale for each
// activation row and each weight row: the two grouped expert products and the
// dense product, each tile computed by a pair of CTAs on two SMs with one
// tcgen05 MMA (cta_group::2, kind::i8: int8 operands, exact int32 sums).
//
//   out[t, c] = (float(sum_k x[t, k] * w[c, k]) * x_scale[t]) * w_scale[c]
//
// The sum is exact, so it does not depend on the tile, on the K order or on how
// K is split; the conversion and the two products round once each.
//
// Weights are the MMA's M operand (256 rows, 128 per CTA) and activation rows
// its N operand (a multiple of 32 up to 256), so that an expert's last tile and
// a short batch cost their own row count, as in the bf16 kernels:
//   gate/up  256 rows of W1 (gate and up interleaved in groups of 16, so that
//            a thread reads both of an f from its TMEM quarter) -> SwiGLU ->
//            bf16 h rows, quantised by a pass of their own (a row's scale needs
//            all of F)
//   down     256 rows of W2 -> fp32 y rows
//   dense    256 weight rows -> bf16 or fp32 rows of out
// A K stage is two 128-byte swizzle atoms, 256 elements, 8 MMAs.  Where K has an
// odd number of atoms the last stage's second one holds zeros on the activation
// side; what stands there on the weight side is then of no account (integers
// have no NaN).
//
// Roles (18 warps per CTA): warp 0 issues TMA loads; warp 1 owns TMEM and, in
// CTA 0, issues the MMAs; warps 2-17 drain two accumulators of 256 columns.
// Every mbarrier wait is bounded; the pair meets in cluster barriers only at
// start-up and before TMEM is released.
//
// What bounds it (B200).  Dense, 8192^3: 350 us cold and 370-420 sustained, 2.6 to
// 3.1 POP/s, where twice the measured bf16 rate is 3.3: the power limit lowers the
// clock.  65,536 routes of 128 experts, H 2,048, F 1,024: gate/up 245 us (2.2
// POP/s), down 178 us.  Without epilogues they take 210 and 78: gate/up is bound by
// what an SM takes in from L2 (88 bytes a nanosecond), as its 320 row tiles hold 205
// rows on average and each loads all of its weights; down by all that it moves, 537 MB
// of fp32 y rows out (91 us alone), 268 MB of weights and 67 MB of codes in, 133 us at
// the copy rate.
// 256 tokens of the same experts (16 rows each): 92 us and 51 us for 537 and 268 MB
// of weights, 5.8 and 5.2 TB/s of the measured 6.5; a launch's first loads and last
// tile, ten us together, are what is missing.
#include "int8.cuh"

namespace moe {
namespace {

constexpr int kStagesMax = 6;
constexpr int kEpiWarps = 8;    // of a group: each drains a quarter of the lanes and half of the columns
constexpr int kEpiGroups = 2;   // groups of epilogue warps, which take tiles in turn
constexpr int kThreads = (2 + kEpiGroups * kEpiWarps) * 32;
constexpr int kChunk = 16;      // accumulator columns a warp takes at once
constexpr int kPairM = 256;
constexpr int kAtoms = 2;                            // 128-byte swizzle atoms per stage
constexpr uint32_t kAtomBytes = 128 * 128;           // 128 rows of 128 bytes
constexpr uint32_t kABytes = kAtoms * kAtomBytes;    // 32 KB: this CTA's 128 weight rows
constexpr uint32_t kBBytesMax = kAtoms * kAtomBytes; // up to 128 activation rows per CTA
constexpr uint32_t kAccCols = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kStageRegion = 6 * (kABytes + 4096);  // also 5 * (32 + 8), 4 * (32 + 16) and 3 * (32 + 32) KB
constexpr int kWarpCols = 128;                            // activation rows of a tile that an epilogue warp drains
constexpr uint32_t kEpiBytes = kWarpCols * 4;             // their scales
constexpr size_t kSmemBytes = 1024 + kStageRegion + kEpiGroups * kEpiWarps * kEpiBytes + 256;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kStageRegion >= 3 * (kABytes + kBBytesMax) && kStageRegion >= 4 * (kABytes + 16384) &&
                  kStageRegion >= 5 * (kABytes + 8192), "stages");

struct __align__(8) Barriers {
    uint64_t full[kStagesMax];   // CTA 0's counts both CTAs' loads of a stage
    uint64_t empty[kStagesMax];  // each CTA's: its stage may be refilled
    uint64_t acc_full[2];        // each CTA's: its accumulator rows are ready
    uint64_t acc_empty[2];       // CTA 0's: both CTAs drained the accumulator
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

// Instruction descriptor of kind::i8: int32 sums of signed 8-bit A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t mbar_cluster, int c0,
                                                 int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar_cluster), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ int tile_n(int nvalid) { return (nvalid + 31) & ~31; }

struct StageCfg {
    int n;       // stages
    uint32_t b;  // activation slot bytes
};
__device__ __forceinline__ StageCfg stage_cfg(int widest_tile) {
    const int hb = tile_n(widest_tile) >> 1;  // activation rows per CTA
    if (hb <= 16) return {6, 4096u};
    if (hb <= 32) return {5, 8192u};
    if (hb <= 64) return {4, 16384u};
    return {3, kBBytesMax};
}

enum { kGateUp = 0, kDown = 1, kDense = 2 };

// The row tile (x) and weight tile (y) of tile t.  Blocks of p.raster row tiles are walked weight tile
// by weight tile; with 1 (grouped: always) a row tile's weight tiles follow one another.
template <int kMode>
__device__ __forceinline__ int2 place_of(const Int8Gemm& p, int num_m, int t) {
    const int raster = kMode == kDense ? p.raster : 1;
    const int block = t / (raster * p.n_tiles), m0 = block * raster;
    const int high = min(raster, num_m - m0), in = t - m0 * p.n_tiles;
    const int nt = in / high;
    return make_int2(m0 + in - nt * high, nt);
}

// Row tile mt of the launch: {expert, first activation row, valid rows, first permuted row}.
template <int kMode>
__device__ __forceinline__ int4 tile_of(const Int8Gemm& p, int mt, int rows) {
    if (kMode != kDense) return __ldg(p.tiles + mt);
    const int m0 = mt * p.tile_rows;
    return make_int4(0, m0, min(p.tile_rows, rows - m0), m0);
}

// Threads 0-15 read 8 columns of 16 TMEM lanes from taddr, threads 16-31 the next 8 of the same lanes.
__device__ __forceinline__ void tmem_ld_16x32bx2_x8(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
// Two fp32 products or sums in one instruction, each rounded as alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
// sigmoid_approx of two.
__device__ __forceinline__ float2 sigmoid_approx2(float2 g) {
    float2 e = mul2(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    e = add2(e, make_float2(1.0f, 1.0f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    return e;
}
// float(a) * xs * ws of two sums.
__device__ __forceinline__ float2 scaled2(uint32_t a0, uint32_t a1, float2 xs, float2 ws) {
    return mul2(mul2(make_float2(__int2float_rn((int)a0), __int2float_rn((int)a1)), xs), ws);
}
__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// The lane's values of n rows, ld apart; of the first `left` of them only.
template <int n, class T>
__device__ __forceinline__ void store_rows(T* dst, long long ld, const float (&v)[n], int left) {
    if (left >= n) {
#pragma unroll
        for (int j = 0; j < n; ++j) store_as(dst + (size_t)j * (size_t)ld, v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (j < left) store_as(dst + (size_t)j * (size_t)ld, v[j]);
    }
}
// Arrive on an mbarrier of the cluster without ordering this thread's stores before it: what the
// arrival says is that the accumulator's loads are done, which tcgen05.wait::ld has waited for.  The
// next MMA into it is ordered behind them by the tcgen05 fences on both sides of the barrier, for
// which the PTX manual's patterns ask an execution order and no more (a relaxed arrival).  Releasing
// the warp's stores of h or y as well: 65,536 routes 727 us for 710, 777 x 2,688 -> 3,712 17.0 for 16.3.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

template <int kMode>
__device__ __forceinline__ void int8_gemm_body(const CUtensorMap& tmA, const BoxMaps8* tmB, const Int8Gemm& p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sEpi = smem + kStageRegion;
    Barriers* bars = reinterpret_cast<Barriers*>(sEpi + kEpiGroups * kEpiWarps * kEpiBytes);
    volatile int* abort_flag = &bars->abort_flag;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = (int)cluster_id_x();
    const int npairs = (int)cluster_count_x();
    pdl_trigger();

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStagesMax; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], 2 * kEpiWarps);  // (of a tile that both groups share nobody waits for it)
        }
        mbar_init(&bars->done, 1);
        bars->abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&bars->tmem_base, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM exist before any cross-CTA traffic
    tc_fence_after_sync();
    const uint32_t tmem_base = bars->tmem_base;
    // `early`: the kernel before this one let it start only once all that came before that kernel
    // was done.  Sizes, tiles and weights then need no wait, and the first stages' weights are on
    // their way while that kernel still writes this one's activation rows.
    if (!p.early) pdl_wait();

    int num_m, rows = 0, widest;
    if (kMode == kDense) {
        rows = p.live != nullptr ? clamp_live(p.live, p.rows) : p.rows;
        num_m = (rows + p.tile_rows - 1) / p.tile_rows;
        widest = min(rows, p.tile_rows);
    } else {
        num_m = forward_poisoned(p.status_words) ? 0 : (int)p.status_words[kStNumMTiles];
        widest = (int)p.status_words[kStMaxTileRows];
    }
    const int total_tiles = num_m * p.n_tiles;
    const int kb_count = (p.atoms + kAtoms - 1) / kAtoms;
    const StageCfg sc = stage_cfg(widest);
    const int kStages = sc.n;
    const uint32_t kBBytes = sc.b;
    uint8_t* sB = smem + kStages * kABytes;
    if (p.early && warp != 0) pdl_wait();
    auto timed_out = [&]() {
        *abort_flag = 1;
        if (p.status_flags != nullptr) atomicOr(p.status_flags, MOE_DEV_TIMEOUT);
    };

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (one thread of each CTA)
            tma_prefetch_desc(&tmA);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            // Experts with one route tile each (decode): every weight tile is read once; its lines go
            // first out of L2, which keeps the rows that the next kernels read there.
            const bool weights_once = kMode != kDense && widest < kRouteTile;
            const uint64_t pol_once = l2_policy_evict_first();
            auto weights = [&](int s, int e, int w_row, int kb) {  // K stage kb of 128 weight rows into stage s
                const uint32_t full0 = map_to_cta(smem_u32(&bars->full[s]), 0);
                uint8_t* dst = sA + s * kABytes;
                if (kMode == kDense) {
                    // atoms of plain rows; columns from K on are filled with zeros
#pragma unroll
                    for (int at = 0; at < kAtoms; ++at)
                        tma_load_2d_pair(dst + at * kAtomBytes, &tmA, full0, (kb * kAtoms + at) * 128, w_row);
                } else {
                    const int atom = (int)(((long long)e * p.a_rows + w_row) / 128 * p.atoms) + kb * kAtoms;
                    if (weights_once)
                        tma_load_3d_pair_hint(dst, &tmA, full0, 0, 0, atom, pol_once);
                    else
                        tma_load_3d_pair(dst, &tmA, full0, 0, 0, atom);
                }
            };
            auto stage_bytes = [&](int z) {  // both CTAs' loads of a stage of a tile of z rows
                return 2u * (kABytes + (uint32_t)(tile_n(z) >> 1) * (kAtoms * 128u));
            };
            int pre = 0;  // stages whose weights are requested before the wait
            if (p.early) {
                int kb = 0;
                for (int t = pair; t < total_tiles && pre < kStages;) {
                    const int2 at = place_of<kMode>(p, num_m, t);
                    const int4 ti = tile_of<kMode>(p, at.x, rows);
                    if (leader) mbar_arrive_expect_tx(&bars->full[pre], stage_bytes(ti.z));
                    weights(pre, ti.x, at.y * kPairM + 128 * (int)rank, kb);
                    ++pre;
                    if (++kb == kb_count) {
                        kb = 0;
                        t += npairs;
                    }
                }
                pdl_wait();
            }
            auto tile_at = [&](int t) {
                return t < total_tiles ? tile_of<kMode>(p, place_of<kMode>(p, num_m, t).x, rows) : make_int4(0, 0, 0, 0);
            };
            int4 ti_n = tile_at(pair);
            for (int t = pair; t < total_tiles && ok; t += npairs) {
                const int nt = place_of<kMode>(p, num_m, t).y;
                const int4 ti = ti_n;
                ti_n = tile_at(t + npairs);
                const int hb = tile_n(ti.z) >> 1;
                const uint32_t tx = stage_bytes(ti.z);
                const CUtensorMap* mb = &tmB->m[(hb >> 4) - 1];
                const int w_row = nt * kPairM + 128 * (int)rank;
                const int b_row = ti.y + hb * (int)rank;
                for (int kb = 0; kb < kb_count; ++kb) {
                    if (pre > 0) {
                        --pre;
                    } else {
                        if (!mbar_wait_bounded(&bars->empty[stage], phase ^ 1u, abort_flag, p.wait_limit_ns)) {
                            ok = false;
                            break;
                        }
                        if (leader) mbar_arrive_expect_tx(&bars->full[stage], tx);
                        weights(stage, ti.x, w_row, kb);
                    }
                    const uint32_t full0 = map_to_cta(smem_u32(&bars->full[stage]), 0);
                    uint8_t* b_dst = sB + stage * kBBytes;
                    if (kMode == kDense) {
#pragma unroll
                        for (int at = 0; at < kAtoms; ++at)
                            tma_load_2d_pair(b_dst + (uint32_t)at * (uint32_t)hb * 128u, mb, full0,
                                             (kb * kAtoms + at) * 128, b_row);
                    } else {
                        tma_load_3d_pair(b_dst, mb, full0, 0, b_row, kb * kAtoms);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) timed_out();  // the MMA issuer then gives up too, and sees the copies land
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ---------------- pair MMA issuer (CTA 0)
            const uint64_t a_desc0 = sdesc_kmajor_sw128(smem_u32(sA)), b_desc0 = sdesc_kmajor_sw128(smem_u32(sB));
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            int it = 0;
            // rows of the next tile, fetched ahead
            auto rows_at = [&](int t) {
                return t < total_tiles ? tile_of<kMode>(p, place_of<kMode>(p, num_m, t).x, rows).z : 0;
            };
            int zn = rows_at(pair);
            for (int t = pair; t < total_tiles && ok; t += npairs, ++it) {
                const int buf = it & 1;
                const uint32_t acc_phase = (uint32_t)(it >> 1) & 1u;
                const int n = tile_n(zn);
                zn = rows_at(t + npairs);
                const uint32_t idesc = idesc_i8(kPairM, n);
                const uint32_t b_atom16 = (uint32_t)(n >> 1) * 8u;  // one atom of this CTA's rows, in 16 bytes
                if (!mbar_wait_bounded(&bars->acc_empty[buf], acc_phase ^ 1u, abort_flag, p.wait_limit_ns)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + (uint32_t)buf * kAccCols;
                for (int kb = 0; kb < kb_count; ++kb) {
                    if (!mbar_wait_bounded(&bars->full[stage], phase, abort_flag, p.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    // operand addresses are descriptor fields in units of 16 bytes: a stage's, an
                    // atom's and a step's offsets are added to the first stage's descriptors
                    const uint64_t da = a_desc0 + (uint64_t)((uint32_t)stage * (kABytes >> 4));
                    const uint64_t db = b_desc0 + (uint64_t)((uint32_t)stage * (kBBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kAtoms * 4; ++kk)  // 32 elements of K each
                        mma_i8_pair(d_tmem, da + (uint64_t)((kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2),
                                    db + (uint64_t)((kk >> 2) * b_atom16 + (uint32_t)(kk & 3) * 2), idesc,
                                    (kb | kk) != 0 ? 1u : 0u);
                    mma_commit_pair_multicast(&bars->empty[stage], 0x3);  // both CTAs may refill the stage
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair_multicast(&bars->acc_full[buf], 0x3);
            }
            if (!ok) {
                timed_out();
                int8_fills_land(bars->full, kStages, (int)phase * kStages + stage);  // (parities repeat every 2 n fills)
            }
            mma_commit_pair(&bars->done);
            volatile int never = 0;
            (void)mbar_wait_bounded(&bars->done, 0, &never, 100000000ull);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: warps 2..17, in two groups of eight, which take the pair's tiles in
        // turn, one accumulator each: a group's loads and stores wait while the other's run (65,536
        // routes: gate/up with the pass over h 294 us, 298 where both share each tile; down 178 and
        // 181).  A pair with one tile at most shares it.  TMEM lanes are weight rows (output columns),
        // TMEM columns activation rows: a lane's weight scale is a register, a row's scale comes from
        // shared memory, and the 32 lanes' stores of one row are neighbours.  The next tile's scales
        // are fetched while this one is drained.
        const int ew = (warp - 2) & (kEpiWarps - 1), group = (warp - 2) / kEpiWarps;
        const int quad = warp & 3;  // TMEM lane quarter this warp may read
        const bool share = total_tiles <= npairs;
        // this warp takes the chunks c = c0, c0 + cs, ... of kChunk columns
        const int c0 = (ew >> 2) + (share ? 2 * group : 0), cs = share ? 4 : 2;
        const int step = share ? npairs : kEpiGroups * npairs;
        const uint32_t acc_empty0[2] = {map_to_cta(smem_u32(&bars->acc_empty[0]), 0),
                                        map_to_cta(smem_u32(&bars->acc_empty[1]), 0)};
        float* s_xs = reinterpret_cast<float*>(sEpi + (size_t)(warp - 2) * kEpiBytes);
        auto first_row = [&](int t) {  // this warp's first weight row in tile t
            return place_of<kMode>(p, num_m, t).y * kPairM + 128 * (int)rank + 32 * quad;
        };
        auto tile_at = [&](int t) {
            return t < total_tiles ? tile_of<kMode>(p, place_of<kMode>(p, num_m, t).x, rows) : make_int4(0, 0, 0, 0);
        };
        float xs_next[4], ws_next = 0.0f;
        auto fetch = [&](int t, int4 ti) {  // scales of tile t: lane l holds its rows l, l + 32, ... of this warp
            if (t >= total_tiles) return;
            const int w = first_row(t) + lane;
            if (kMode == kGateUp || w < p.out_cols)
                ws_next = __ldg(p.w_scale + (kMode == kDense ? 0 : (size_t)ti.x * p.a_rows) + w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = (c0 + (2 * i + (lane >> 4)) * cs) * kChunk + (lane & 15);
                xs_next[i] = r < ti.z ? __ldg(p.row_scale + ti.y + r) : 0.0f;
            }
        };
        const int t_first = pair + (share ? 0 : group * npairs);
        int4 ti_next = tile_at(t_first), ti_after = tile_at(t_first + step);
        fetch(t_first, ti_next);
        int it = share ? 0 : group;
        for (int t = t_first; t < total_tiles; t += step, it += share ? 1 : kEpiGroups) {
            const int buf = it & 1;
            const uint32_t acc_phase = (uint32_t)(it >> 1) & 1u;
            const int4 ti = ti_next;
            const float ws = ws_next;
            const int nch = tile_n(ti.z) / kChunk;
            const int w0 = first_row(t);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) s_xs[i * 32 + lane] = xs_next[i];
            __syncwarp();
            ti_next = ti_after;
            fetch(t + step, ti_next);
            ti_after = tile_at(t + 2 * step);
            const bool got = __all_sync(0xffffffffu,
                                        mbar_wait_bounded(&bars->acc_full[buf], acc_phase, abort_flag, p.wait_limit_ns));
            if (!got) {
                if (lane == 0) timed_out();
                break;
            }
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)buf * kAccCols;
            const int f0 = p.relu2 ? w0 : w0 >> 1;  // gate/up: first of this warp's 32 (16) f
            const bool cols = (kMode == kGateUp ? f0 : w0) < p.out_cols;
            const bool glu = kMode == kGateUp && !p.relu2;
            const float ws_gate = glu ? __shfl_sync(0xffffffffu, ws, lane & 15) : 0.0f;
            const float ws_up = glu ? __shfl_sync(0xffffffffu, ws, 16 + (lane & 15)) : 0.0f;
#pragma unroll 1
            for (int c = c0, i = 0; c < nch; c += cs, ++i) {
                // SwiGLU: lanes < 16 take the chunk's first eight rows, the others its last, of gate (the
                // quarter's first 16 TMEM lanes) and of up (its last 16) alike
                constexpr int kHalf = kChunk / 2;
                uint32_t v[kChunk];
                if (glu) {
                    tmem_ld_16x32bx2_x8(taddr + c * kChunk, v);
                    tmem_ld_16x32bx2_x8(taddr + (16u << 16) + c * kChunk, v + kHalf);
                } else {
                    tmem_ld_32x32b_x16(taddr + c * kChunk, v);
                }
                float pv = 1.0f;  // gate/up with probabilities: lane l holds row l's
                if (kMode == kGateUp && p.route_probs != nullptr && c * kChunk + (lane & 15) < ti.z)
                    pv = __ldg(p.route_probs + __ldg(p.perm + ti.w + c * kChunk + (lane & 15)));
                tmem_ld_wait();
                if (c + cs >= nch) {  // the last of this warp's columns is in registers
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0[buf]);
                }
                if (!cols) continue;
                // rows of this chunk that exist; a whole chunk is stored without asking row by row
                // (branches around each store cost a quarter of the epilogue's time)
                const int left = ti.z - c * kChunk;
                __nv_bfloat16* h = kMode == kGateUp ? reinterpret_cast<__nv_bfloat16*>(p.out) +
                                                          (size_t)(ti.y + c * kChunk) * (size_t)p.out_ld + f0
                                                    : nullptr;
                if (glu) {
                    // silu(g) * u, silu first: g * u alone may pass fp32's range
                    const int r0 = lane < 16 ? 0 : kHalf;
                    const float4* xs4 = reinterpret_cast<const float4*>(s_xs + i * kChunk + r0);
                    float hv[kHalf];
#pragma unroll
                    for (int q = 0; q < kHalf / 2; ++q) {
                        const float4 x4 = xs4[q >> 1];
                        const float2 xs = q & 1 ? make_float2(x4.z, x4.w) : make_float2(x4.x, x4.y);
                        float2 gt = scaled2(v[2 * q], v[2 * q + 1], xs, make_float2(ws_gate, ws_gate));
                        float2 up = scaled2(v[kHalf + 2 * q], v[kHalf + 2 * q + 1], xs, make_float2(ws_up, ws_up));
                        if (p.clamp > 0.0f) {
                            gt = make_float2(clamp_nan(gt.x, p.clamp), clamp_nan(gt.y, p.clamp));
                            up = make_float2(clamp_nan(up.x, p.clamp), clamp_nan(up.y, p.clamp));
                        }
                        float2 o = mul2(mul2(gt, sigmoid_approx2(gt)), up);
                        if (p.route_probs != nullptr)
                            o = mul2(o, make_float2(__shfl_sync(0xffffffffu, pv, r0 + 2 * q),
                                                    __shfl_sync(0xffffffffu, pv, r0 + 2 * q + 1)));
                        hv[2 * q] = o.x;
                        hv[2 * q + 1] = o.y;
                    }
                    store_rows<kHalf>(h + (size_t)r0 * (size_t)p.out_ld + (lane & 15), p.out_ld, hv,
                                      left >= kChunk ? kHalf : left - r0);
                    continue;
                }
                const float4* xs4 = reinterpret_cast<const float4*>(s_xs + i * kChunk);
                float g[kChunk];
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q) {
                    const float4 xs = xs4[q];
                    const float2 a = scaled2(v[4 * q], v[4 * q + 1], make_float2(xs.x, xs.y), make_float2(ws, ws));
                    const float2 b = scaled2(v[4 * q + 2], v[4 * q + 3], make_float2(xs.z, xs.w), make_float2(ws, ws));
                    g[4 * q] = a.x;
                    g[4 * q + 1] = a.y;
                    g[4 * q + 2] = b.x;
                    g[4 * q + 3] = b.y;
                }
                if (kMode == kGateUp) {
                    if (p.clamp > 0.0f) {
#pragma unroll
                        for (int j = 0; j < kChunk; ++j) g[j] = clamp_nan(g[j], p.clamp);
                    }
#pragma unroll
                    for (int j = 0; j < kChunk; ++j) {
                        const float r = g[j] > 0.0f || g[j] != g[j] ? g[j] : 0.0f;  // a NaN row stays NaN
                        g[j] = r * r;
                        if (p.route_probs != nullptr) g[j] *= __shfl_sync(0xffffffffu, pv, j);
                    }
                    store_rows<kChunk>(h + lane, p.out_ld, g, left);
                } else if (w0 + lane < p.out_cols) {
                    const size_t at = (size_t)(ti.y + c * kChunk) * (size_t)p.out_ld + w0 + lane;
                    if (kMode == kDense && p.out_bf16 != 0)
                        store_rows<kChunk>(reinterpret_cast<__nv_bfloat16*>(p.out) + at, p.out_ld, g, left);
                    else
                        store_rows<kChunk>(reinterpret_cast<float*>(p.out) + at, p.out_ld, g, left);
                }
            }
            if (nch <= c0 && lane == 0) mbar_arrive_cluster_relaxed(acc_empty0[buf]);  // no column of this warp
        }
    }

    // ---------------- teardown: no pair MMA is in flight once CTA 0 has seen "done", and no copy once
    // its issuer has used every fill or seen it land
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_gate_up_swiglu_int8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BoxMaps8 tmB,
                                 const Int8Gemm p) {
    int8_gemm_body<kGateUp>(tmA, &tmB, p);
}
__global__ void __launch_bounds__(kThreads, 1)
    moe_gemm_down_int8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BoxMaps8 tmB,
                       const Int8Gemm p) {
    int8_gemm_body<kDown>(tmA, &tmB, p);
}
__global__ void __launch_bounds__(kThreads, 1)
    gemm_dense_int8(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BoxMaps8 tmB, const Int8Gemm p) {
    int8_gemm_body<kDense>(tmA, &tmB, p);
}

typedef void (*GemmKernel)(CUtensorMap, BoxMaps8, Int8Gemm);

cudaError_t launch_pair(GemmKernel kern, int which, const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g,
                        long long max_tiles, cudaStream_t s) {
    constexpr int kDevices = 64;
    static int resident[3][kDevices];  // pairs that can be resident, per kernel and device (0: not asked yet)
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait()
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (resident[which][dev] == 0) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (err != cudaSuccess) return err;
        int clusters = 0;
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        err = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
        if (err != cudaSuccess) return err;
        if (clusters < 1) return cudaErrorInvalidConfiguration;
        resident[which][dev] = clusters < num_sms() / 2 ? clusters : num_sms() / 2;
    }
    long long pairs = resident[which][dev];
    if (pairs > max_tiles) pairs = max_tiles;
    if (pairs < 1) pairs = 1;
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kern, a, b, g);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm1_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s) {
    return launch_pair(moe_gemm_gate_up_swiglu_int8, kGateUp, a, b, g, max_tiles, s);
}
cudaError_t launch_gemm2_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                              cudaStream_t s) {
    return launch_pair(moe_gemm_down_int8, kDown, a, b, g, max_tiles, s);
}
cudaError_t launch_gemm_dense_int8(const CUtensorMap& a, const BoxMaps8& b, const Int8Gemm& g, long long max_tiles,
                                   cudaStream_t s) {
    return launch_pair(gemm_dense_int8, kDense, a, b, g, max_tiles, s);
}

}  // namespace moe
