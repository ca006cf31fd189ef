// The product of two microscaled tensors for many tokens: a persistent grid of CTA
// pairs on tcgen05's block-scaled instructions (cta_group::2, sm_103a).
//
// A pair computes tiles of 256 tokens x up to 192 output features, D = x_tile W_tile^T in fp32:
// each CTA holds the rows of 128 tokens (lane = token, column = feature) in its tensor memory,
// twice, so that one tile is written while the next is computed, and half of W's tile in its
// shared memory.  The pairs share the product out in units of 256 tokens x 64 features, as
// evenly as those allow: equal tiles of 256 features leave 8 % to 16 % of the pairs' time
// unused (2.5 or 10.1 of them a pair for 2048 or 8192 tokens x 6144 features).
//
// One warp streams operands and scales through a ring of 5 stages (128 bytes of every row) with
// TMA.  Four warps carry each stage's scales from shared to tensor memory, one quarter of its
// lanes each: copied by the issuing thread (tcgen05.cp) they held the products up by some
// 200 cycles a stage, whatever their number (4096 x 8192 x 8192 in 4 bits: 120 us).
// One thread of the even CTA issues a stage's four products.  Two groups of four warps write
// y, one accumulator each, in bf16 through shared memory with TMA.
#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 480;                 // 4 warps of scales, 2 x 4 of the epilogue, products, operands' and scales' loads
constexpr int kSpan = 128;                    // bytes of a row a stage
constexpr int kTileM = 256, kTileN = 192;     // tokens, output features at most
constexpr int kUnit = 64;                     // features that the pairs share out
constexpr int kStages = 5;
constexpr int kBox = 64 * 2 * 128;            // 64 features x 128 tokens of y

template <int kType>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kA = 128 * kSpan, kB = kTileN / 2 * kSpan, kStageBytes = kA + kB;  // tokens, features
    static constexpr int kOut = kStages * kStageBytes;              // two boxes of y for each group of the epilogue
    static constexpr int kSf = kOut + 4 * kBox, kSfBlock = kSfTiles * kMxTileBytes;  // x's block, W's two
    static constexpr int kBars = kSf + kStages * 3 * kSfBlock;      // landed, ready, empty [S], acc, free [2]
    static constexpr int kTmemSlot = kBars + 8 * (3 * kStages + 4);
    static constexpr int kAlloc = kTmemSlot + 16 + 1024;
    // tensor memory: two accumulators, then a stage's scales for each of the ring's: x's tiles, and two
    // blocks of 128 features for each of W's
    static constexpr int kSfCol = 2 * kTileN, kSfCols = 12 * kSfTiles, kCols = 512;
    static_assert(kSfCol + kStages * kSfCols <= kCols, "columns");
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap x, w, sfx, sfw, y[3];
};

struct Params {
    uint32_t* err;
    int seg_end[3];
    int tokens, in, out, units;  // units: of 64 features in a row of tiles
};

// A pair's share of the units (tokens' tiles one behind the other), as a walk over its tiles.
struct Walk {
    int64_t at, end;
    int units, m, f, n;  // the tile: tokens from 256 m, n units from feature 64 f
    __device__ Walk(const Params& p) : units(p.units)
    {
        const int64_t all = (int64_t)((p.tokens + kTileM - 1) / kTileM) * p.units;
        const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
        at = all * pair / pairs;
        end = all * (pair + 1) / pairs;
    }
    __device__ __forceinline__ bool next()
    {
        if (at >= end) return false;
        m = (int)(at / units);
        f = (int)(at % units);
        const int left = (int)min(end - at, (int64_t)(units - f));
        const int tiles = (left + kTileN / kUnit - 1) / (kTileN / kUnit);
        n = (left + tiles - 1) / tiles;
        at += n;
        return true;
    }
};

// Stages of the ring in turn, with the parity of the barriers' present phase.
struct Ring {
    int st = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++st == kStages) st = 0, parity ^= 1;
    }
};

template <int kType>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_pair_kernel(const __grid_constant__ Maps maps, Params p)
{
    using S = Shape<kType>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;  // (the same offset in both CTAs)
    uint8_t* sbase = smem_raw + (base - raw_base);
    const uint32_t bar_landed = base + S::kBars, bar_ready = bar_landed + 8 * kStages, bar_empty = bar_ready + 8 * kStages,
                   bar_acc = bar_empty + 8 * kStages, bar_free = bar_acc + 16;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    Walk walk(p);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar_landed + 8 * i, 1);
            mbar_init(bar_ready + 8 * i, 9);  // the pair's operands, and its warps of scales
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_acc + 8 * i, 1);
            mbar_init(bar_free + 8 * i, 8);  // the pair's four warps each
        }
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.sfx);
        tma_prefetch_desc(&maps.sfw);
    }
    if (warp == 13) tmem_alloc_pair(base + S::kTmemSlot, S::kCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sbase + S::kTmemSlot), 0);
    pdl_wait();
    pdl_launch_dependents();

    if (warp < 4) {
        // ---- scales: row 32 j + lane of a block to column j, the same in each warp's quarter of the lanes
        const uint32_t to = tmem + ((uint32_t)(32 * warp) << 16) + S::kSfCol, bar0 = cluster_map(bar_ready, 0);
        Ring ring;
        bool ok = true;
        while (walk.next())
            for (int k = 0; k < nk; ++k, ring.next()) {
                ok &= mbar_wait_spin(bar_landed + 8 * ring.st, ring.parity, ok ? kWaitLimitNs : 0);
                tc_fence_after();  // (the stage's columns: its last products were done before it was loaded again)
                const uint4* from = reinterpret_cast<const uint4*>(sbase + S::kSf + ring.st * 3 * S::kSfBlock) + lane;
                const uint32_t at = to + ring.st * S::kSfCols;
#pragma unroll
                for (int s = 0; s < S::kSfTiles; ++s) {
                    tmem_st4(at + 4 * s, from[32 * s]);
                    tmem_st4(at + 4 * S::kSfTiles + 8 * s, from[32 * (S::kSfTiles + s)]);
                    tmem_st4(at + 4 * S::kSfTiles + 8 * s + 4, from[32 * (2 * S::kSfTiles + s)]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(bar0 + 8 * ring.st);
            }
        if (!ok && lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 12) {
        // ---- operands: they complete on the even CTA's barrier
        const uint64_t keep = l2_policy_evict_last();  // both are read again by other pairs
        Ring ring;
        bool ok = true, again = false;
        while (ok && walk.next()) {
            const int m0 = walk.m * kTileM + (int)rank * 128;
            const int n0 = walk.f * kUnit + (int)rank * (walk.n * kUnit / 2);  // (rows beyond half of the tile are not used)
            for (int k = 0; k < nk; ++k, ring.next()) {
                if (again) ok &= mbar_wait_spin(bar_empty + 8 * ring.st, ring.parity ^ 1, ok ? kWaitLimitNs : 0);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t a = base + ring.st * S::kStageBytes, bar = bar_ready + 8 * ring.st;
                if (rank == 0) mbar_arrive_expect_tx_warp(bar, 2 * S::kStageBytes);
                tma_load_2d_pair_warp(a, &maps.x, k * kSpan, m0, bar, keep);
                tma_load_2d_pair_warp(a + S::kA, &maps.w, k * kSpan, n0, bar, keep);
                again |= ring.st == kStages - 1;
            }
        }
        // the last stages' products are done with this CTA's ring and barriers before it leaves
        for (int i = 0; i < kStages; ++i, ring.next())
            if (again || ring.parity) ok &= mbar_wait_spin(bar_empty + 8 * ring.st, ring.parity ^ 1, ok ? kWaitLimitNs : 0);
        if (!ok && lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 14) {
        // ---- scales: x's block of 128 tokens and W's two of features, on this CTA's barrier
        const uint64_t keep = l2_policy_evict_last();
        Ring ring;
        bool ok = true, again = false;
        while (ok && walk.next()) {
            const int mb = walk.m * 2 + (int)rank, nb = walk.f / 2;
            for (int k = 0; k < nk; ++k, ring.next()) {
                if (again) ok &= mbar_wait_spin(bar_empty + 8 * ring.st, ring.parity ^ 1, ok ? kWaitLimitNs : 0);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t to = base + S::kSf + ring.st * 3 * S::kSfBlock, bar = bar_landed + 8 * ring.st;
                mbar_arrive_expect_tx_warp(bar, 3 * S::kSfBlock);
                tma_load_2d_warp(to, &maps.sfx, k * S::kSfTiles * 128, mb, bar, keep);
                tma_load_2d_warp(to + S::kSfBlock, &maps.sfw, k * S::kSfTiles * 128, nb, bar, keep);
                again |= ring.st == kStages - 1;
            }
        }
        if (!ok && lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 13) {
        if (rank == 0) {
            // ---- products of the pair (a wait that ran out does not end the loop, which would make its
            // counters differ between lanes: the later waits are single looks, the results are void)
            Ring ring;
            bool ok = true, there = false;
            for (int done = 0; walk.next(); ++done) {
                const uint32_t half = done & 1, acc = tmem + half * kTileN;
                if (done >= 2) ok &= mbar_wait_spin(bar_free + 8 * half, (done / 2 - 1) & 1, ok ? kWaitLimitNs : 0);
                const uint32_t shape = umma_idesc_mx(kType == PKV_MX4, kTileM, 0, 0) | ((uint32_t)(walk.n * kUnit / 8) << 17);
                const uint32_t odd = walk.f & 1 ? 2 : 0;  // columns: the tile starts in the middle of a block of 128
                for (int k = 0; k < nk; ++k) {
                    // (the next stage is looked for before this one's products are issued)
                    if (!there) ok &= mbar_wait_spin(bar_ready + 8 * ring.st, ring.parity, ok ? kWaitLimitNs : 0);
                    __syncwarp();
                    const int st = ring.st;
                    ring.next();
                    there = mbar_test_wait(bar_ready + 8 * ring.st, ring.parity);
                    tc_fence_after();
                    const uint32_t a = base + st * S::kStageBytes, sfc = tmem + S::kSfCol + st * S::kSfCols;
                    const int have = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
                    const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(a + S::kA, 16, 1024);
                    constexpr int kPer = 4 / S::kSfTiles;  // products a tile of scales
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int s = kk / kPer;
                        if (s < have)
                            umma_mx_pair_warp<kType == PKV_MX4>(acc, da + 2 * kk, db + 2 * kk,
                                                                shape | umma_idesc_sf(kk % kPer * (4 / kPer)), sfc + 4 * s,
                                                                sfc + 4 * S::kSfTiles + 8 * s + odd, k > 0 || kk > 0);
                    }
                    umma_commit_pair_warp(bar_empty + 8 * st);
                }
                umma_commit_pair_warp(bar_acc + 8 * half);
            }
            if (!ok && lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
        }
    } else {
        // ---- epilogue: group h writes every other tile; its warp q holds tokens 32 q .. + 31 of this CTA
        const int q = warp & 3, h = (warp - 4) >> 2, row = 32 * q + lane;
        const bool issuer = q == 0 && lane == 0;
        const uint32_t box0 = base + S::kOut + 2 * kBox * h, acc = tmem + ((uint32_t)(32 * q) << 16) + h * kTileN;
        const uint32_t free0 = cluster_map(bar_free + 8 * h, 0);
        int done = 0, boxes = 0;
        for (; walk.next(); ++done) {
            if ((done & 1) != h) continue;
            const int m0 = walk.m * kTileM + (int)rank * 128;
            const bool ok = named_all(1 + h, 128, mbar_wait_spin(bar_acc + 8 * h, (done / 2) & 1));  // (they leave together)
            if (!ok) {
                if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int r = 0; r < walk.n; ++r, ++boxes) {  // 64 features a round
                uint32_t v[2][32], packed[32];
                tmem_ld32(acc + 64 * r, v[0]);
                tmem_ld32(acc + 64 * r + 32, v[1]);
                tmem_wait_ld_regs(v[0]);
                tmem_wait_ld_regs(v[1]);
                if (r == walk.n - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(free0);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(packed[j])
                        : "f"(__uint_as_float(v[j / 16][2 * (j % 16) + 1])), "f"(__uint_as_float(v[j / 16][2 * (j % 16)])));
                const uint32_t box = box0 + (boxes & 1) * kBox, mine = box + row * 128;
                if (issuer) bulk_wait_read_1();  // the box's last store, two rounds ago, has been read
                named_sync(1 + h, 128);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((c ^ (row & 7)) << 4)),
                                 "r"(packed[4 * c]), "r"(packed[4 * c + 1]), "r"(packed[4 * c + 2]), "r"(packed[4 * c + 3])
                                 : "memory");
                fence_async_shared();
                named_sync(1 + h, 128);
                if (issuer) {
                    const int n0 = (walk.f + r) * kUnit, seg = n0 < p.seg_end[0] ? 0 : (n0 < p.seg_end[1] ? 1 : 2);
                    if (m0 < p.tokens) tma_store_2d(&maps.y[seg], n0 - (seg ? p.seg_end[seg - 1] : 0), m0, box);
                    bulk_commit();
                }
            }
        }
        if (issuer) bulk_wait();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // no CTA leaves while the other's products or arrivals may reach it
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, S::kCols);
    }
}

template <int kType>
cudaError_t launch(const pkv_pool* pool, const MxLinear& a, cudaStream_t s)
{
    using S = Shape<kType>;
    Maps m;
    Params p = {};
    int end = 0;
    for (int i = 0; i < 3; ++i) {
        end += i < a.segments ? a.widths[i] : 0;
        p.seg_end[i] = end;
        if (i >= a.segments)
            m.y[i] = m.y[0];
        else if (!make_tmap_2d(&m.y[i], a.y[i], a.widths[i], a.tokens, (uint64_t)a.widths[i] * 2, 64, 128))
            return cudaErrorInvalidValue;
    }
    const int row = mx_row_bytes(kType, a.in), sf_tiles = a.in / kMxTileCols;
    if (!make_tmap_bytes(&m.x, a.x_codes, row, a.tokens, 128) || !make_tmap_bytes(&m.w, a.w_codes, row, end, kTileN / 2) ||
        !make_tmap_scales(&m.sfx, a.x_scales, sf_tiles, (a.tokens + 127) / 128, S::kSfTiles, 1) ||
        !make_tmap_scales(&m.sfw, a.w_scales, sf_tiles, end / 128, S::kSfTiles, 2))
        return cudaErrorInvalidValue;
    p.err = pool->err;
    p.tokens = a.tokens;
    p.in = a.in;
    p.out = end;
    p.units = end / kUnit;
    const int64_t units = (int64_t)(a.tokens + kTileM - 1) / kTileM * p.units;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (units < pool->mx_pairs ? units : pool->mx_pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kAlloc;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx_pair_kernel<kType>, m, p);
}

template <int kType>
cudaError_t configure(int* pairs)
{
    cudaError_t e = cudaFuncSetAttribute(mx_pair_kernel<kType>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Shape<kType>::kAlloc);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<kType>::kAlloc;
    return cudaOccupancyMaxActiveClusters(pairs, mx_pair_kernel<kType>, &cfg);
}

}  // namespace

cudaError_t configure_mx_pair(pkv_pool* pool)
{
    int eight = 0, four = 0;
    cudaError_t e = configure<PKV_MX8>(&eight);
    if (e == cudaSuccess) e = configure<PKV_MX4>(&four);
    pool->mx_pairs = eight < four ? eight : four;
    return e != cudaSuccess ? e : pool->mx_pairs > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

cudaError_t launch_mx_pair(const pkv_pool* pool, const MxLinear& a, cudaStream_t s)
{
    return a.type == PKV_MX8 ? launch<PKV_MX8>(pool, a, s) : launch<PKV_MX4>(pool, a, s);
}

}  // namespace pkv
