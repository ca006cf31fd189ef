// The product of two microscaled tensors for many tokens: a persistent grid of CTA
// pairs on tcgen05's block-scaled instructions (cta_group::2, sm_103a).
//
// A pair computes tiles of 256 tokens x 256 output features, D = x_tile W_tile^T in fp32: each
// CTA holds the rows of 128 tokens (lane = token, column = feature) in 256 columns of its
// tensor memory, and half of W's tile in its shared memory, so that an SM reads 32 KiB of
// operands for 128 x 256 x 128-byte products instead of 48.
//
// Warp 0 streams operands and scales through a ring of 5 stages (128 bytes of every row) with
// TMA; one thread of the even CTA copies each stage's scales to both tensor memories and
// issues its four products; eight warps take the accumulator out in bf16 (64 registers), hand
// tensor memory back at once, and write y through 32 KiB of shared memory with TMA while the
// next tile's products run.
#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 384;
constexpr int kSpan = 128;                    // bytes of a row a stage
constexpr int kTileM = 256, kTileN = 256;     // tokens, output features
constexpr int kStages = 5;

template <int kType>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kA = 128 * kSpan, kB = 128 * kSpan, kSfA = kSfTiles * kMxTileBytes, kSfB = 2 * kSfA;
    static constexpr int kTx = kA + kB + kSfA + kSfB;               // bytes a CTA loads a stage
    static constexpr int kStageBytes = (kTx + 1023) / 1024 * 1024;
    static constexpr int kOut = kStages * kStageBytes;              // two boxes of 64 features x 128 tokens
    static constexpr int kBars = kOut + 2 * 16384;                  // full[S], empty[S], acc_full, acc_empty
    static constexpr int kTmemSlot = kBars + 8 * (2 * kStages + 2);
    static constexpr int kAlloc = kTmemSlot + 16 + 1024;
    static constexpr int kSfaCol = kTileN, kSfbCol = kTileN + 4 * kSfTiles, kCols = 512;
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap x, w, sfx, sfw, y[3];
};

struct Params {
    uint32_t* err;
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
    const uint32_t bar_full = base + S::kBars, bar_empty = bar_full + 8 * kStages, bar_acc = bar_empty + 8 * kStages,
                   bar_free = bar_acc + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    const int tiles = p.m_tiles * p.n_tiles, pairs = gridDim.x / 2, first = blockIdx.x / 2;

    if (tid == 0) {
        for (int i = 0; i < 2 * kStages + 1; ++i) mbar_init(bar_full + 8 * i, 1);
        mbar_init(bar_free, 16);  // the pair's epilogue warps
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.sfx);
        tma_prefetch_desc(&maps.sfw);
    }
    if (warp == 2) tmem_alloc_pair(base + S::kTmemSlot, S::kCols);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + S::kTmemSlot);
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            // ---- producer: this CTA's operands; bytes complete on the even CTA's barrier
            const uint64_t keep = l2_policy_evict_last();  // both operands are read again by other pairs
            int it = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += pairs) {
                const int mt = t % p.m_tiles, nt = t / p.m_tiles;
                const int m0 = mt * kTileM + (int)rank * 128, n0 = nt * kTileN + (int)rank * 128;
                for (int k = 0; k < nk; ++k, ++it) {
                    const int st = it % kStages;
                    if (it >= kStages && !(ok = mbar_wait(bar_empty + 8 * st, ((it / kStages) - 1) & 1))) {
                        atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                        break;
                    }
                    const uint32_t a = base + st * S::kStageBytes, b = a + S::kA, sa = b + S::kB, sb = sa + S::kSfA;
                    const uint32_t fb = bar_full + 8 * st;
                    if (rank == 0) mbar_arrive_expect_tx(fb, 2 * S::kTx);
                    tma_load_2d_pair(a, &maps.x, k * kSpan, m0, fb, keep);
                    tma_load_2d_pair(b, &maps.w, k * kSpan, n0, fb, keep);
                    tma_load_2d_pair(sa, &maps.sfx, k * S::kSfTiles * 128, m0 / 128, fb, keep);
                    tma_load_2d_pair(sb, &maps.sfw, k * S::kSfTiles * 128, nt * (kTileN / 128), fb, keep);
                }
            }
            // the last stages' products are done with this CTA's ring and barriers before it leaves
            for (int i = it > kStages ? it - kStages : 0; i < it && ok; ++i)
                ok = mbar_wait(bar_empty + 8 * (i % kStages), (i / kStages) & 1);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---- products of the pair
            int it = 0, done = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += pairs, ++done) {
                if (done && !(ok = mbar_wait_spin(bar_free, (done - 1) & 1))) {
                    atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                    break;
                }
                tc_fence_after();
                for (int k = 0; k < nk; ++k, ++it) {
                    const int st = it % kStages;
                    if (!(ok = mbar_wait_spin(bar_full + 8 * st, (it / kStages) & 1))) {
                        atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = base + st * S::kStageBytes, b = a + S::kA, sa = b + S::kB, sb = sa + S::kSfA;
                    const int have = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
                    const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
                    constexpr int kPer = 4 / S::kSfTiles;  // products a tile of scales
#pragma unroll
                    for (int s = 0; s < S::kSfTiles; ++s) {
                        umma_copy_scales_pair(tmem + S::kSfaCol + 4 * s, sa + s * kMxTileBytes);
                        umma_copy_scales_pair(tmem + S::kSfbCol + 8 * s, sb + s * kMxTileBytes);
                        umma_copy_scales_pair(tmem + S::kSfbCol + 8 * s + 4, sb + S::kSfA + s * kMxTileBytes);
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const int s = kk / kPer;
                        if (s < have)
                            umma_mx_pair<kType == PKV_MX4>(
                                tmem, da + 2 * kk, db + 2 * kk,
                                umma_idesc_mx(kType == PKV_MX4, kTileM, kTileN, kk % kPer * (4 / kPer)),
                                tmem + S::kSfaCol + 4 * s, tmem + S::kSfbCol + 8 * s, k > 0 || kk > 0);
                    }
                    umma_commit_pair(bar_empty + 8 * st);
                }
                umma_commit_pair(bar_acc);
            }
        }
    } else if (warp >= 4) {
        // ---- epilogue: warp w holds tokens 32 (w % 4) .. + 31 of this CTA, features 128 h .. + 127 of the tile
        const int q = warp & 3, h = (warp - 4) >> 2, row = 32 * q + lane;
        const bool issuer = q == 0 && lane == 0;
        const uint32_t box = base + S::kOut + 16384 * h, mine = box + row * 128, free0 = cluster_map(bar_free, 0);
        int done = 0;
        for (int t = first; t < tiles; t += pairs, ++done) {
            const int mt = t % p.m_tiles, nt = t / p.m_tiles;
            const int m0 = mt * kTileM + (int)rank * 128, n0 = nt * kTileN + 128 * h;
            const bool ok = named_all(1 + h, 128, mbar_wait(bar_acc, done & 1));  // (its warps leave together)
            if (!ok) {
                if (lane == 0) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            uint32_t packed[64];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + 128 * h + 32 * g, v);
                tmem_wait_ld_regs(v);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                        : "=r"(packed[16 * g + j])
                        : "f"(__uint_as_float(v[2 * j + 1])), "f"(__uint_as_float(v[2 * j])));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free0);
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
    if (warp == 2) {
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
    if (!make_tmap_bytes(&m.x, a.x_codes, row, a.tokens, 128) || !make_tmap_bytes(&m.w, a.w_codes, row, end, 128) ||
        !make_tmap_scales(&m.sfx, a.x_scales, sf_tiles, (a.tokens + 127) / 128, S::kSfTiles, 1) ||
        !make_tmap_scales(&m.sfw, a.w_scales, sf_tiles, end / 128, S::kSfTiles, 2))
        return cudaErrorInvalidValue;
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
