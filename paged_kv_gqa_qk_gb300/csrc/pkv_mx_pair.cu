// The product of two microscaled tensors for many tokens: a persistent grid of CTA
// pairs on tcgen05's block-scaled instructions (cta_group::2, sm_103a).
//
// A pair computes tiles of 256 tokens x 256 output features, D = x_tile W_tile^T in fp32: each
// CTA holds the rows of 128 tokens (lane = token, column = feature) in 256 columns of its
// tensor memory, and half of W's tile in its shared memory, so that an SM reads 32 KiB of
// operands for 128 x 256 x 128-byte products instead of 48.
//
// One warp streams operands and scales through a ring of 5 stages (128 bytes of every row) with
// TMA.  Four warps carry each stage's scales from shared to tensor memory, one quarter of its
// lanes each: copied by the issuing thread (tcgen05.cp) they held the products up by some
// 200 cycles a stage, whatever their number (4096 x 8192 x 8192 in 4 bits: 120 us).
// One thread of the even CTA issues a stage's four products.  Eight warps take the accumulator
// out in bf16 (64 registers), hand tensor memory back at once, and write y through 32 KiB of
// shared memory with TMA while the next tile's products run.
#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 448;                 // 4 warps of scales, 8 of the epilogue, the producer's, the products'
constexpr int kSpan = 128;                    // bytes of a row a stage
constexpr int kTileM = 256, kTileN = 256;     // tokens, output features
constexpr int kStages = 5;

template <int kType>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kA = 128 * kSpan, kStageBytes = 2 * kA;    // tokens, features
    static constexpr int kOut = kStages * kStageBytes;              // two boxes of 64 features x 128 tokens
    static constexpr int kSf = kOut + 2 * 16384, kSfBlock = kSfTiles * kMxTileBytes;  // x's block, W's two
    static constexpr int kBars = kSf + kStages * 3 * kSfBlock;      // full, landed, scales, empty [S], acc, free
    static constexpr int kTmemSlot = kBars + 8 * (4 * kStages + 2);
    static constexpr int kAlloc = kTmemSlot + 16 + 1024;
    // tensor memory: the accumulator, then a stage's scales for each of the ring's: x's tiles, and two
    // blocks of features for each of W's
    static constexpr int kSfCols = 12 * kSfTiles, kCols = 512;
    static_assert(kTileN + kStages * kSfCols <= kCols, "columns");
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap x, w, y[3];
};

struct Params {
    uint32_t* err;
    const uint8_t *x_scales, *w_scales;
    int seg_end[3];
    int tokens, in, out, m_tiles, n_tiles;
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
    const uint32_t bar_full = base + S::kBars, bar_landed = bar_full + 8 * kStages, bar_sf = bar_landed + 8 * kStages,
                   bar_empty = bar_sf + 8 * kStages, bar_acc = bar_empty + 8 * kStages, bar_free = bar_acc + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    const int tiles = p.m_tiles * p.n_tiles, pairs = gridDim.x / 2, first = blockIdx.x / 2;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(bar_full + 8 * i, 1);
            mbar_init(bar_landed + 8 * i, 1);
            mbar_init(bar_sf + 8 * i, 8);  // the pair's warps of scales
            mbar_init(bar_empty + 8 * i, 1);
        }
        mbar_init(bar_acc, 1);
        mbar_init(bar_free, 16);  // the pair's epilogue warps
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 13) tmem_alloc_pair(base + S::kTmemSlot, S::kCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + S::kTmemSlot);
    pdl_wait();
    pdl_launch_dependents();

    if (warp < 4) {
        // ---- scales: row 32 j + lane of a block to column j, the same in each warp's quarter of the lanes
        const int total = (tiles - first + pairs - 1) / pairs * nk;
        const uint32_t to = tmem + ((uint32_t)(32 * warp) << 16) + kTileN, bar0 = cluster_map(bar_sf, 0);
        for (int it = 0; it < total; ++it) {
            const int st = it % kStages;
            const bool ok = __all_sync(0xffffffffu, mbar_wait_spin(bar_landed + 8 * st, (it / kStages) & 1));
            if (!ok) {
                if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            tc_fence_after();  // (the stage's columns: its last products were done before it was loaded again)
            const uint4* from = reinterpret_cast<const uint4*>(sbase + S::kSf + st * 3 * S::kSfBlock) + lane;
            const uint32_t at = to + st * S::kSfCols;
#pragma unroll
            for (int s = 0; s < S::kSfTiles; ++s) {
                tmem_st4(at + 4 * s, from[32 * s]);
                tmem_st4(at + 4 * S::kSfTiles + 8 * s, from[32 * (S::kSfTiles + s)]);
                tmem_st4(at + 4 * S::kSfTiles + 8 * s + 4, from[32 * (2 * S::kSfTiles + s)]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(bar0 + 8 * st);
        }
    } else if (warp == 12) {
        if (lane == 0) {
            // ---- producer: this CTA's operands; bytes complete on the even CTA's barrier
            const uint64_t keep = l2_policy_evict_last();  // both operands are read again by other pairs
            int it = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += pairs) {
                const int mt = t % p.m_tiles, nt = t / p.m_tiles;
                const int m0 = mt * kTileM + (int)rank * 128, n0 = nt * kTileN + (int)rank * 128;
                const uint8_t* sx = p.x_scales + (int64_t)(m0 / 128) * sf_tiles * kMxTileBytes;
                const uint8_t* sw = p.w_scales + (int64_t)nt * 2 * sf_tiles * kMxTileBytes;
                const bool has_x = m0 < p.tokens, has_w = nt * kTileN + 128 < p.out;  // (else unused: nothing to load)
                for (int k = 0; k < nk; ++k, ++it) {
                    const int st = it % kStages;
                    if (it >= kStages && !(ok = mbar_wait_spin(bar_empty + 8 * st, ((it / kStages) - 1) & 1))) {
                        atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                        break;
                    }
                    const uint32_t a = base + st * S::kStageBytes, fb = bar_full + 8 * st;
                    if (rank == 0) mbar_arrive_expect_tx(fb, 2 * S::kStageBytes);
                    tma_load_2d_pair(a, &maps.x, k * kSpan, m0, fb, keep);
                    tma_load_2d_pair(a + S::kA, &maps.w, k * kSpan, n0, fb, keep);
                    const uint32_t sf = base + S::kSf + st * 3 * S::kSfBlock, lb = bar_landed + 8 * st;
                    const uint32_t bytes = min(S::kSfTiles, sf_tiles - k * S::kSfTiles) * kMxTileBytes;
                    const int64_t at = (int64_t)k * S::kSfBlock;
                    mbar_arrive_expect_tx(lb, (1 + has_x + has_w) * bytes);
                    if (has_x) bulk_copy_g2s(sf, sx + at, bytes, lb);
                    bulk_copy_g2s(sf + S::kSfBlock, sw + at, bytes, lb);
                    if (has_w) bulk_copy_g2s(sf + 2 * S::kSfBlock, sw + (int64_t)sf_tiles * kMxTileBytes + at, bytes, lb);
                }
            }
            // the last stages' products are done with this CTA's ring and barriers before it leaves
            for (int i = it > kStages ? it - kStages : 0; i < it && ok; ++i)
                ok = mbar_wait(bar_empty + 8 * (i % kStages), (i / kStages) & 1);
        }
    } else if (warp == 13) {
        if (lane == 0 && rank == 0) {
            // ---- products of the pair
            int it = 0, done = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += pairs, ++done) {
                if (done && !(ok = mbar_wait_spin(bar_free, (done - 1) & 1))) {
                    atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                    break;
                }
                for (int k = 0; k < nk; ++k, ++it) {
                    const int st = it % kStages;
                    ok = mbar_wait_spin(bar_full + 8 * st, (it / kStages) & 1) &&
                         mbar_wait_spin(bar_sf + 8 * st, (it / kStages) & 1);
                    if (!ok) {
                        atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = base + st * S::kStageBytes, sfc = tmem + kTileN + st * S::kSfCols;
                    const int have = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
                    const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(a + S::kA, 16, 1024);
                    constexpr int kPer = 4 / S::kSfTiles;  // products a tile of scales
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int s = kk / kPer;
                        if (s < have)
                            umma_mx_pair<kType == PKV_MX4>(
                                tmem, da + 2 * kk, db + 2 * kk,
                                umma_idesc_mx(kType == PKV_MX4, kTileM, kTileN, kk % kPer * (4 / kPer)), sfc + 4 * s,
                                sfc + 4 * S::kSfTiles + 8 * s, k > 0 || kk > 0);
                    }
                    umma_commit_pair(bar_empty + 8 * st);
                }
                umma_commit_pair(bar_acc);
            }
        }
    } else {
        // ---- epilogue: warp w holds tokens 32 (w % 4) .. + 31 of this CTA, features 128 h .. + 127 of the tile
        const int q = warp & 3, h = (warp - 4) >> 2, row = 32 * q + lane;
        const bool issuer = q == 0 && lane == 0;
        const uint32_t box = base + S::kOut + 16384 * h, mine = box + row * 128, free0 = cluster_map(bar_free, 0);
        int done = 0;
        for (int t = first; t < tiles; t += pairs, ++done) {
            const int mt = t % p.m_tiles, nt = t / p.m_tiles;
            const int m0 = mt * kTileM + (int)rank * 128, n0 = nt * kTileN + 128 * h;
            const bool ok = named_all(1 + h, 128, mbar_wait_spin(bar_acc, done & 1));  // (its warps leave together)
            if (!ok) {
                if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            uint32_t packed[64];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t v[2][32];
                const uint32_t from = tmem + ((uint32_t)(32 * q) << 16) + 128 * h + 64 * g;
                tmem_ld32(from, v[0]);
                tmem_ld32(from + 32, v[1]);
                tmem_wait_ld_regs(v[0]);
                tmem_wait_ld_regs(v[1]);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(packed[32 * g + j])
                        : "f"(__uint_as_float(v[j / 16][2 * (j % 16) + 1])), "f"(__uint_as_float(v[j / 16][2 * (j % 16)])));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(free0);
            const int seg = n0 < p.seg_end[0] ? 0 : (n0 < p.seg_end[1] ? 1 : 2);
            const int col = n0 - (seg ? p.seg_end[seg - 1] : 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // 64 features a round
                if (issuer) bulk_wait_read();
                named_sync(1 + h, 128);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((c ^ (row & 7)) << 4)),
                                 "r"(packed[32 * r + 4 * c]), "r"(packed[32 * r + 4 * c + 1]),
                                 "r"(packed[32 * r + 4 * c + 2]), "r"(packed[32 * r + 4 * c + 3])
                                 : "memory");
                fence_async_shared();
                named_sync(1 + h, 128);
                if (issuer && n0 < p.out && m0 < p.tokens) {
                    tma_store_2d(&maps.y[seg], col + 64 * r, m0, box);
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
    const int row = mx_row_bytes(kType, a.in);
    if (!make_tmap_bytes(&m.x, a.x_codes, row, a.tokens, 128) || !make_tmap_bytes(&m.w, a.w_codes, row, end, 128))
        return cudaErrorInvalidValue;
    p.x_scales = static_cast<const uint8_t*>(a.x_scales);
    p.w_scales = static_cast<const uint8_t*>(a.w_scales);
    p.err = pool->err;
    p.tokens = a.tokens;
    p.in = a.in;
    p.out = end;
    p.m_tiles = (a.tokens + kTileM - 1) / kTileM;
    p.n_tiles = (end + kTileN - 1) / kTileN;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pool->mx_pairs ? tiles : pool->mx_pairs)));
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
