// The product of two microscaled tensors, y = x W^T, on tcgen05's block-scaled
// instructions (sm_103a): pkv_mx_linear and pkv_mx_qkv_proj.
//
// qwen3-8b Nest files, src/attention.linnet, GroupedQueryAttention.decode_paged (q_proj, k_proj,
// v_proj, o_proj), with both operands held as codes of 8 or 4 bits and a power of two on every
// 32 of them: y[t][o] = sum_g 2^(ex + ew) sum_{k in g} x[t][k] w[o][k].
//
// A CTA computes 128 output features x BN tokens, D = W_tile x_tile^T, in tensor memory
// (lane = feature, column = token).  A stage of its ring holds 128 bytes of every row (128
// or 256 values) and their scales' tiles; one thread copies the scales to tensor memory
// and issues the four products of a stage.  Where the tiles alone would leave SMs idle,
// the input features are split over the CTAs of a cluster, which sum their tiles over
// distributed shared memory in a fixed order.
#include <type_traits>

#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kBM = 128;        // output features a tile
constexpr int kSpan = 128;      // bytes of a row a stage
constexpr int kMaxSplits = 8;   // a portable cluster

template <int kType, int BN>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kRowBlocks = (BN + 127) / 128;
    static constexpr int kABytes = kBM * kSpan, kBBytes = BN * kSpan;
    static constexpr int kSfA = kSfTiles * kMxTileBytes, kSfB = kRowBlocks * kSfA;
    static constexpr int kStageBytes = (kABytes + kBBytes + kSfA + kSfB + 1023) / 1024 * 1024;
    static constexpr int kStages = BN == 64 ? 4 : (200 * 1024) / kStageBytes;
    static_assert(kStages * kStageBytes >= kBM * BN * 4, "the ring holds the fp32 partial tile");
    static constexpr int kBars = kStages * kStageBytes;  // full[S], empty[S], done
    static constexpr int kTmemSlot = kBars + 8 * (2 * kStages + 1);
    static constexpr int kAlloc = kTmemSlot + 16 + 1024;
    // tensor memory: the accumulator, then the scales of W and of x, 4 columns a tile
    static constexpr int kSfaCol = BN, kSfbCol = BN + 4 * kSfTiles;
    static constexpr int kCols = BN == 64 ? 128 : BN == 128 ? 256 : 512;
    static_assert(kSfbCol + 4 * kSfTiles * kRowBlocks <= kCols, "columns");
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Params {
    const uint8_t *x_scales, *w_scales;
    __nv_bfloat16* y[3];
    int seg_end[3];     // cumulative widths; seg_end[2] == out
    uint32_t* err;
    int tokens, in, out, splits, row_blocks;  // row_blocks: of 128 tokens, in x's scales
};

// The segment holding output features from m0: its tensor, its width and the tile's column in it.
__device__ __forceinline__ __nv_bfloat16* segment(const Params& p, int m0, int& width, int& col)
{
    const int s = m0 < p.seg_end[0] ? 0 : (m0 < p.seg_end[1] ? 1 : 2);
    const int start = s ? p.seg_end[s - 1] : 0;
    width = p.seg_end[s] - start;
    col = m0 - start;
    return p.y[s];
}

template <int kType, int BN>
__global__ void __launch_bounds__(kThreads, BN == 64 ? 2 : 1)
    mx_linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, Params p)
{
    using S = Shape<kType, BN>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    uint8_t* sbase = smem_raw + (base - raw_base);
    const uint32_t bar_full = base + S::kBars, bar_empty = bar_full + 8 * S::kStages, bar_done = bar_empty + 8 * S::kStages;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m_tiles = p.out / kBM, split = blockIdx.z;
    const int m0 = (blockIdx.x % m_tiles) * kBM, n0 = (blockIdx.x / m_tiles) * BN;
    // this CTA's share of the input features, in stages; the last one of a 4-bit row may be half
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    const int k0 = (int)((int64_t)nk * split / p.splits), k1 = (int)((int64_t)nk * (split + 1) / p.splits);

    if (tid == 0) {
        for (int i = 0; i < 2 * S::kStages + 1; ++i) mbar_init(bar_full + 8 * i, 1);
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(base + S::kTmemSlot, S::kCols);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + S::kTmemSlot);

    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0 && lane == 0) {
        // ---- producer
        const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
        const uint8_t* sfw = p.w_scales + (int64_t)(m0 / 128) * sf_tiles * kMxTileBytes;
        const uint8_t* sfx = p.x_scales + (int64_t)(n0 / 128) * sf_tiles * kMxTileBytes;
        const int blocks = min(S::kRowBlocks, p.row_blocks - n0 / 128);
        for (int k = k0; k < k1; ++k) {
            const int i = k - k0, st = i % S::kStages;
            if (i >= S::kStages && !mbar_wait(bar_empty + 8 * st, ((i / S::kStages) - 1) & 1)) {
                atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            const uint32_t a = base + st * S::kStageBytes, b = a + S::kABytes, sa = b + S::kBBytes, sb = sa + S::kSfA;
            const uint32_t fb = bar_full + 8 * st;
            const int tiles = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
            const uint32_t sf_bytes = tiles * kMxTileBytes;
            mbar_arrive_expect_tx(fb, S::kABytes + S::kBBytes + (1 + blocks) * sf_bytes);
            tma_load_2d(a, &tmW, k * kSpan, m0, fb, pol_w);
            tma_load_2d(b, &tmX, k * kSpan, n0, fb, pol_x);
            const int64_t at = (int64_t)k * S::kSfTiles * kMxTileBytes;
            bulk_copy_g2s(sa, sfw + at, sf_bytes, fb);
            for (int r = 0; r < blocks; ++r)
                bulk_copy_g2s(sb + r * S::kSfA, sfx + (int64_t)r * sf_tiles * kMxTileBytes + at, sf_bytes, fb);
        }
    } else if (warp == 1 && lane == 0) {
        // ---- MMA issuer
        for (int k = k0; k < k1; ++k) {
            const int i = k - k0, st = i % S::kStages;
            if (!mbar_wait_spin(bar_full + 8 * st, (i / S::kStages) & 1)) {
                atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            const uint32_t a = base + st * S::kStageBytes, b = a + S::kABytes, sa = b + S::kBBytes, sb = sa + S::kSfA;
            const int tiles = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
            for (int t = 0; t < tiles; ++t) {  // columns: [tile][row block], 4 each
                umma_copy_scales(tmem + S::kSfaCol + 4 * t, sa + t * kMxTileBytes);
                for (int r = 0; r < S::kRowBlocks; ++r)
                    umma_copy_scales(tmem + S::kSfbCol + 4 * (t * S::kRowBlocks + r), sb + r * S::kSfA + t * kMxTileBytes);
            }
            const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
            constexpr int kPer = 4 / S::kSfTiles;  // products a tile of scales
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int t = kk / kPer;
                if (t < tiles)
                    umma_mx<kType == PKV_MX4>(tmem, da + 2 * kk, db + 2 * kk,
                                              umma_idesc_mx(kType == PKV_MX4, kBM, BN, kk % kPer * (4 / kPer)),
                                              tmem + S::kSfaCol + 4 * t, tmem + S::kSfbCol + 4 * t * S::kRowBlocks,
                                              i > 0 || kk > 0);
            }
            umma_commit(bar_empty + 8 * st);
        }
        umma_commit(bar_done);  // also on a timeout: the epilogue and the release wait for it
    }
    __syncwarp();

    // ---- epilogue: thread (warp w, lane l) holds output feature m0 + 32 w + l for BN tokens
    const bool ok = mbar_wait(bar_done, 0);
    tc_fence_after();
    int yw, yc;
    __nv_bfloat16* const y = segment(p, m0, yw, yc);
    if (p.splits == 1) {
        const int o = yc + 32 * warp + lane;
        if (ok) {
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(32 * warp) << 16) + c0, v);
                tmem_wait_ld_regs(v);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int t = n0 + c0 + j;
                    if (t < p.tokens) y[(int64_t)t * yw + o] = __float2bfloat16_rn(__uint_as_float(v[j]));
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(tmem, S::kCols);
        }
        return;
    }
    // ---- split over the cluster: the partial tile, [token][feature] fp32, in this CTA's idle ring
    float* part = reinterpret_cast<float*>(sbase);
#pragma unroll 1
    for (int c0 = 0; c0 < BN; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(32 * warp) << 16) + c0, v);
        tmem_wait_ld_regs(v);
#pragma unroll
        for (int j = 0; j < 32; ++j) part[(c0 + j) * kBM + 32 * warp + lane] = ok ? __uint_as_float(v[j]) : 0.f;
    }
    tc_fence_before();
    cluster_sync();  // every partial tile of the cluster is in place
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
    // CTA r sums features [r 128 / splits, (r + 1) 128 / splits), four a thread, in rank order
    const int r = (int)cluster_rank(), per = kBM / 4 / p.splits;
    const uint32_t local = smem_u32(part);
    for (int i = tid; i < BN * per; i += kThreads) {
        const int t = i / per, f = 4 * (r * per + i % per);
        if (n0 + t >= p.tokens) break;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < p.splits; ++q) {
            const float4 v = ld_cluster_f32x4(cluster_map(local, q) + (uint32_t)(t * kBM + f) * 4);
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
        uint2 o2;
        o2.x = pack_bf16(__float2bfloat16_rn(acc.x), __float2bfloat16_rn(acc.y));
        o2.y = pack_bf16(__float2bfloat16_rn(acc.z), __float2bfloat16_rn(acc.w));
        *reinterpret_cast<uint2*>(y + (int64_t)(n0 + t) * yw + yc + f) = o2;
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <int kType, int BN>
cudaError_t launch(const pkv_pool* pool, const MxLinear& a, Params& p, cudaStream_t s)
{
    using S = Shape<kType, BN>;
    CUtensorMap tmW, tmX;
    const int row = mx_row_bytes(kType, a.in);
    if (!make_tmap_bytes(&tmW, a.w_codes, row, p.out, kBM) || !make_tmap_bytes(&tmX, a.x_codes, row, a.tokens, BN))
        return cudaErrorInvalidValue;
    const int tiles = (p.out / kBM) * ((a.tokens + BN - 1) / BN), steps = row / kSpan;
    const int slots = pool->num_sms * (BN == 64 ? 2 : 1);
    p.splits = 1;
    while (p.splits < kMaxSplits && tiles * p.splits * 2 <= slots && steps / (p.splits * 2) >= 2) p.splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, 1, p.splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kAlloc;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = p.splits;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx_linear_kernel<kType, BN>, tmW, tmX, p);
}

template <int kType>
cudaError_t launch_type(const pkv_pool* pool, const MxLinear& a, Params& p, cudaStream_t s)
{
    if (a.tokens <= 64) return launch<kType, 64>(pool, a, p, s);
    if (a.tokens <= 128) return launch<kType, 128>(pool, a, p, s);
    return launch<kType, 256>(pool, a, p, s);
}

template <int kType, int BN>
bool configure()
{
    return cudaFuncSetAttribute(mx_linear_kernel<kType, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Shape<kType, BN>::kAlloc) == cudaSuccess;
}

}  // namespace

cudaError_t configure_mx_linear()
{
    const bool ok = configure<PKV_MX8, 64>() && configure<PKV_MX8, 128>() && configure<PKV_MX8, 256>() &&
                    configure<PKV_MX4, 64>() && configure<PKV_MX4, 128>() && configure<PKV_MX4, 256>();
    return ok ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_mx_linear(const pkv_pool* pool, const MxLinear& a, cudaStream_t s)
{
    Params p = {};
    for (int i = 0, end = 0; i < 3; ++i) {
        end += i < a.segments ? a.widths[i] : 0;
        p.y[i] = static_cast<__nv_bfloat16*>(i < a.segments ? a.y[i] : nullptr);
        p.seg_end[i] = end;
    }
    p.x_scales = static_cast<const uint8_t*>(a.x_scales);
    p.w_scales = static_cast<const uint8_t*>(a.w_scales);
    p.err = pool->err;
    p.tokens = a.tokens;
    p.in = a.in;
    p.out = p.seg_end[2];
    p.row_blocks = (a.tokens + 127) / 128;
    if (a.tokens > 256) return launch_mx_pair(pool, a, s);
    return a.type == PKV_MX8 ? launch_type<PKV_MX8>(pool, a, p, s) : launch_type<PKV_MX4>(pool, a, p, s);
}

}  // namespace pkv
