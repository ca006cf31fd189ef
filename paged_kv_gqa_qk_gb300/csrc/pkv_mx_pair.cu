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
// One warp streams operands through a ring of 6 stages (128 bytes of every row) with TMA: a stage
// is there again some 2300 cycles after its products were issued, which take 384 (8192 x 4096 x
// 6144 in 8 bits with 3 / 4 / 5 / 6 / 7 stages: 173 / 143 / 128 / 123 / 124 us).  Another streams
// their scales, which four warps carry from shared to tensor memory, one quarter of its lanes
// each: copied by the issuing warp (tcgen05.cp) they held the products up by some 200 cycles a
// stage, whatever their number (8192 x 4096 x 6144 in 4 bits: 102 us, without them 79).  One warp
// of the even CTA issues a stage's four products.  Two groups of four warps write y in bf16
// through shared memory with TMA, an accumulator each.
//
// Measured (of four and two times the measured bf16 rate, which instructions of K = 64 and 32 give; those of
// K = 96 that 4 bits have besides are not used here): 8192 x 4096 x 6144 in 4 bits 62 us, 6.6 PFLOP/s (0.88), in 8
// bits 123 us, 3.4 (0.89); 2048 tokens 20.9 and 34.3 us; 4096 x 8192 x 8192 79 and 169.  For a second on end, under the
// power cap, in 8 bits 130 to 138 and 183 to 195.  A call's start and end take some 7 us in all of them.
#include <atomic>

#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 480;                 // 4 warps of scales, 2 x 4 of the epilogue, products, operands' and scales' loads
constexpr int kSpan = 128;                    // bytes of a row a stage
constexpr int kTileM = 256, kTileN = 192;     // tokens, output features at most
constexpr int kUnit = 64;                     // features that the pairs share out
constexpr int kStages = 6;                    // of operands in shared memory
constexpr int kSfStages = 4, kSfSlots = 5;    // of scales in shared and in tensor memory
constexpr int kOutCols = 64, kBox = kOutCols * 2 * 128;  // features of 128 tokens of y that are written at a time

template <int kType>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kA = 128 * kSpan, kB = kTileN / 2 * kSpan, kStageBytes = kA + kB;  // tokens, features
    static constexpr int kOut = kStages * kStageBytes;              // a box of y for each group of the epilogue
    static constexpr int kSf = kOut + 2 * kBox, kSfBlock = kSfTiles * kMxTileBytes;  // x's block, W's two
    static constexpr int kBars = kSf + kSfStages * 3 * kSfBlock;    // full, empty, landed, taken, scales, acc, free
    static constexpr int kTmemSlot = kBars + 8 * (2 * kStages + 2 * kSfStages + kSfSlots + 4);
    static constexpr int kAlloc = kTmemSlot + 16 + 1024;
    // tensor memory: two accumulators, then slots for a stage's scales: x's tiles, and two blocks of 128 features
    // for each of W's
    static constexpr int kSfCol = 2 * kTileN, kSfCols = 12 * kSfTiles, kCols = 512;
    static_assert(kSfCol + kSfSlots * kSfCols <= kCols, "columns");
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap x, w, sfx, sfw, y[3];
};

struct Params {
    uint32_t* err;
    uint64_t wait_ns;  // limit of a wait
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

// Stages of a ring in turn, with the parity of the barriers' present phase.
template <int kCount>
struct RingOf {
    int st = 0;
    uint32_t parity = 0;
    bool again = false;  // beyond the first turn
    __device__ __forceinline__ void next()
    {
        if (++st == kCount) st = 0, parity ^= 1, again = true;
    }
};
using Ring = RingOf<kStages>;
using SfRing = RingOf<kSfStages>;
using SlotRing = RingOf<kSfSlots>;

template <int kType>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_pair_kernel(const __grid_constant__ Maps maps, Params p)
{
    using S = Shape<kType>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;  // (the same offset in both CTAs)
    uint8_t* sbase = smem_raw + (base - raw_base);
    const uint32_t bar_full = base + S::kBars, bar_empty = bar_full + 8 * kStages, bar_landed = bar_empty + 8 * kStages,
                   bar_taken = bar_landed + 8 * kSfStages, bar_sf = bar_taken + 8 * kSfStages, bar_acc = bar_sf + 8 * kSfSlots,
                   bar_free = bar_acc + 16;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    Walk walk(p);

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < kSfStages; ++i) {
            mbar_init(bar_landed + 8 * i, 1);
            mbar_init(bar_taken + 8 * i, 4);  // this CTA's warps of scales
        }
        for (int i = 0; i < kSfSlots; ++i) mbar_init(bar_sf + 8 * i, 8);  // the pair's warps of scales
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
    if (warp == 12) {
        // the first stages of W on their way to L2 before the wait for the kernel before this one, which may still be
        // writing it: what is read comes after (8192 x 4096 x 6144 in 4 bits 65 -> 62 us)
        Walk first = walk;
        if (first.next())
            for (int k = 0; k < min(nk, kStages); ++k)
                tma_prefetch_2d_warp(&maps.w, k * kSpan, first.f * kUnit + (int)rank * (first.n * kUnit / 2));
    }
    pdl_wait();
    pdl_launch_dependents();

    if (warp < 4) {
        // ---- scales: row 32 j + lane of a block to column j, the same in each warp's quarter of the lanes
        const uint32_t to = tmem + ((uint32_t)(32 * warp) << 16) + S::kSfCol, bar0 = cluster_map(bar_sf, 0);
        Ring before;  // the stage whose products used the slot last
        SfRing sf;
        SlotRing slot;
        Waits wait(p.wait_ns);
        while (walk.next())
            for (int k = 0; k < nk; ++k, slot.next(), sf.next()) {
                wait.on(bar_landed + 8 * sf.st, sf.parity);
                const uint4* from = reinterpret_cast<const uint4*>(sbase + S::kSf + sf.st * 3 * S::kSfBlock) + lane;
                uint4 v[3 * S::kSfTiles];
#pragma unroll
                for (int i = 0; i < 3 * S::kSfTiles; ++i) v[i] = from[32 * i];
                if (slot.again) {
                    wait.on(bar_empty + 8 * before.st, before.parity);
                    before.next();
                }
                tc_fence_after();
                const uint32_t at = to + slot.st * S::kSfCols;
#pragma unroll
                for (int s = 0; s < S::kSfTiles; ++s) {
                    tmem_st4(at + 4 * s, v[s]);
                    tmem_st4(at + 4 * S::kSfTiles + 8 * s, v[S::kSfTiles + s]);
                    tmem_st4(at + 4 * S::kSfTiles + 8 * s + 4, v[2 * S::kSfTiles + s]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_taken + 8 * sf.st);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(bar0 + 8 * slot.st);
            }
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 12) {
        // ---- operands: they complete on the even CTA's barrier
        const uint64_t keep = l2_policy_evict_last();  // both are read again by other pairs
        Ring ring;
        Waits wait(p.wait_ns);
        bool ok = true;
        while (ok && walk.next()) {
            const int m0 = walk.m * kTileM + (int)rank * 128;
            const int n0 = walk.f * kUnit + (int)rank * (walk.n * kUnit / 2);  // (rows beyond half of the tile are not used)
            for (int k = 0; k < nk; ++k, ring.next()) {
                if (ring.again) ok = wait.on(bar_empty + 8 * ring.st, ring.parity ^ 1);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t a = base + ring.st * S::kStageBytes, bar = bar_full + 8 * ring.st;
                if (rank == 0) mbar_arrive_expect_tx_warp(bar, 2 * S::kStageBytes);
                tma_load_2d_pair_warp(a, &maps.x, k * kSpan, m0, bar, keep);
                tma_load_2d_pair_warp(a + S::kA, &maps.w, k * kSpan, n0, bar, keep);
            }
        }
        // the last stages' products are done with this CTA's ring and barriers before it leaves
        for (int i = 0; i < kStages; ++i, ring.next())
            if (ring.again) wait.on(bar_empty + 8 * ring.st, ring.parity ^ 1);
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 14) {
        // ---- scales: x's block of 128 tokens and W's two of features, on this CTA's barrier; ahead of the operands
        const uint64_t keep = l2_policy_evict_last();
        SfRing sf;
        Waits wait(p.wait_ns);
        bool ok = true;
        while (ok && walk.next()) {
            const int mb = walk.m * 2 + (int)rank, nb = walk.f / 2;
            for (int k = 0; k < nk; ++k, sf.next()) {
                if (sf.again) ok = wait.on(bar_taken + 8 * sf.st, sf.parity ^ 1);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t to = base + S::kSf + sf.st * 3 * S::kSfBlock, bar = bar_landed + 8 * sf.st;
                mbar_arrive_expect_tx_warp(bar, 3 * S::kSfBlock);
                tma_load_2d_warp(to, &maps.sfx, k * S::kSfTiles * 128, mb, bar, keep);
                tma_load_2d_warp(to + S::kSfBlock, &maps.sfw, k * S::kSfTiles * 128, nb, bar, keep);
            }
        }
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 13) {
        if (rank == 0) {
            // ---- products of the pair (a wait that ran out does not end the loop, which would make its
            // counters differ between lanes)
            Ring ring;
            SlotRing slot;
            Waits wait(p.wait_ns);
            bool there = false, scaled = false;
            for (int done = 0; walk.next(); ++done) {
                const uint32_t half = done & 1, acc = tmem + half * kTileN;
                if (done >= 2) wait.on(bar_free + 8 * half, (done / 2 - 1) & 1);
                const uint32_t shape = umma_idesc_mx(kType == PKV_MX4, kTileM, 0, 0) | ((uint32_t)(walk.n * kUnit / 8) << 17);
                const uint32_t odd = walk.f & 1 ? 2 : 0;  // columns: the tile starts in the middle of a block of 128
                for (int k = 0; k < nk; ++k) {
                    // (the next stage is looked for before this one's products are issued)
                    if (!there) wait.on(bar_full + 8 * ring.st, ring.parity);
                    if (!scaled) wait.on(bar_sf + 8 * slot.st, slot.parity);
                    __syncwarp();
                    const int st = ring.st;
                    const uint32_t a = base + st * S::kStageBytes, sfc = tmem + S::kSfCol + slot.st * S::kSfCols;
                    ring.next();
                    slot.next();
                    there = mbar_test_wait(bar_full + 8 * ring.st, ring.parity);
                    scaled = mbar_test_wait(bar_sf + 8 * slot.st, slot.parity);
                    tc_fence_after();
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
            if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
        }
    } else {
        // ---- epilogue: group h writes every other tile; its warp q holds tokens 32 q .. + 31 of this CTA
        const int q = warp & 3, h = (warp - 4) >> 2, row = 32 * q + lane;
        const bool issuer = q == 0 && lane == 0;
        const uint32_t box = base + S::kOut + kBox * h, mine = box + row * (2 * kOutCols);
        const int swizzle = row & 7;
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + h * kTileN, free0 = cluster_map(bar_free + 8 * h, 0);
        Waits wait(p.wait_ns);
        for (int done = 0; walk.next(); ++done) {
            if ((done & 1) != h) continue;
            const int m0 = walk.m * kTileM + (int)rank * 128, rounds = walk.n * (kUnit / kOutCols);
            if (!named_all(1 + h, 128, wait.on(bar_acc + 8 * h, (done / 2) & 1))) break;  // (they leave together)
            tc_fence_after();
#pragma unroll 1
            for (int r = 0; r < rounds; ++r) {
                uint32_t v[kOutCols / 32][32], packed[kOutCols / 2];
#pragma unroll
                for (int g = 0; g < kOutCols / 32; ++g) tmem_ld32(acc + kOutCols * r + 32 * g, v[g]);
#pragma unroll
                for (int g = 0; g < kOutCols / 32; ++g) tmem_wait_ld_regs(v[g]);
                if (r == rounds - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(free0);
                }
#pragma unroll
                for (int j = 0; j < kOutCols / 2; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(packed[j])
                        : "f"(__uint_as_float(v[j / 16][2 * (j % 16) + 1])), "f"(__uint_as_float(v[j / 16][2 * (j % 16)])));
                if (issuer) bulk_wait_read();  // the box's last store has been read
                named_sync(1 + h, 128);
#pragma unroll
                for (int c = 0; c < kOutCols / 8; ++c)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((c ^ swizzle) << 4)),
                                 "r"(packed[4 * c]), "r"(packed[4 * c + 1]), "r"(packed[4 * c + 2]), "r"(packed[4 * c + 3])
                                 : "memory");
                fence_async_shared();
                named_sync(1 + h, 128);
                if (issuer && m0 < p.tokens) {
                    const int n0 = walk.f * kUnit + kOutCols * r, seg = n0 < p.seg_end[0] ? 0 : (n0 < p.seg_end[1] ? 1 : 2);
                    tma_store_2d(&maps.y[seg], n0 - (seg ? p.seg_end[seg - 1] : 0), m0, box);
                    bulk_commit();
                }
            }
        }
        if (issuer) bulk_wait();
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // no CTA leaves while the other's products or arrivals may reach it
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, S::kCols);
    }
}

// CTA pairs that a device holds at a time (found at its first call), or 0 on an error.
template <int kType>
int resident_pairs(int device)
{
    static std::atomic<int> known[64];
    const bool keep = device >= 0 && device < 64;
    int pairs = keep ? known[device].load(std::memory_order_relaxed) : 0;
    if (cudaFuncSetAttribute(mx_pair_kernel<kType>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<kType>::kAlloc) !=
        cudaSuccess)
        return 0;
    if (pairs) return pairs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<kType>::kAlloc;
    if (cudaOccupancyMaxActiveClusters(&pairs, mx_pair_kernel<kType>, &cfg) != cudaSuccess) return 0;
    if (keep) known[device].store(pairs, std::memory_order_relaxed);
    return pairs;
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
        else if (!make_tmap_2d(&m.y[i], a.y[i], a.widths[i], a.tokens, (uint64_t)a.widths[i] * 2, kOutCols, 128))
            return cudaErrorInvalidValue;
    }
    const int row = mx_row_bytes(kType, a.in), sf_tiles = a.in / kMxTileCols;
    if (!make_tmap_bytes(&m.x, a.x_codes, row, a.tokens, 128) || !make_tmap_bytes(&m.w, a.w_codes, row, end, kTileN / 2) ||
        !make_tmap_scales(&m.sfx, a.x_scales, sf_tiles, (a.tokens + 127) / 128, S::kSfTiles, 1) ||
        !make_tmap_scales(&m.sfw, a.w_scales, sf_tiles, end / 128, S::kSfTiles, 2))
        return cudaErrorInvalidValue;
    p.err = pool->err;
    p.wait_ns = pool->wait_ns;
    p.tokens = a.tokens;
    p.in = a.in;
    p.out = end;
    p.units = end / kUnit;
    const int64_t units = (int64_t)(a.tokens + kTileM - 1) / kTileM * p.units, pairs = resident_pairs<kType>(pool->device);
    if (pairs <= 0) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (units < pairs ? units : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kAlloc;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mx_pair_kernel<kType>, m, p);
}

}  // namespace

cudaError_t launch_mx_pair(const pkv_pool* pool, const MxLinear& a, cudaStream_t s)
{
    return a.type == PKV_MX8 ? launch<PKV_MX8>(pool, a, s) : launch<PKV_MX4>(pool, a, s);
}

}  // namespace pkv
