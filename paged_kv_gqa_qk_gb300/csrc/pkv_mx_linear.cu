// The product of two microscaled tensors, y = x W^T, on tcgen05's block-scaled
// instructions (sm_103a): pkv_mx_linear and pkv_mx_qkv_proj.
//
// qwen3-8b Nest files, src/attention.linnet, GroupedQueryAttention.decode_paged (q_proj, k_proj,
// v_proj, o_proj), with both operands held as codes of 8 or 4 bits and a power of two on every
// 32 of them: y[t][o] = sum_g 2^(ex + ew) sum_{k in g} x[t][k] w[o][k].
//
// The kernel here is for few tokens, where reading W bounds the product; pkv_mx_pair.cu has the
// one for many.  A CTA computes 128 output features x BN tokens, D = W_tile x_tile^T, in tensor
// memory (lane = feature, column = token).  A stage of its ring holds 128 bytes of every row
// (128 or 256 values) and their scales' tiles; one warp copies the scales to tensor memory and
// issues the four products of a stage.  The input features are split over the CTAs of a cluster,
// so that every SM has a part of W to read; each CTA sends its sums of a part of the tokens to
// each other, which adds those of its tokens in the CTAs' order.
//
// Bound by latencies up to some MB of W: one token, 4096 x 6144 in 4 bits, 13.4 MB, 4.3 us, of which 1 from the
// launch to the first copy, 0.9 until it is there, 1 for four stages, 1.1 for the exchange of the sums; by the way from
// L2 with 64 tokens (4096 x 4096 in 8 bits: 26 MB into 128 SMs, W's and x's part for every tile of W, 1.8 of 6.9 us);
// by memory beyond (16 tokens, 4096 x 65536 in 8 bits, 277 MB, 40 us, 6.9 TB/s).  Scales by four warps and sums by
// st.async in place of the cluster's barrier took as long here.
#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;
constexpr int kBM = 128;        // output features a tile
constexpr int kSpan = 128;      // bytes of a row a stage

template <int kType, int BN, int NS>
struct Shape {
    static constexpr int kSfTiles = kType == PKV_MX4 ? 2 : 1;       // tiles of scales a stage and 128 rows
    static constexpr int kABytes = kBM * kSpan, kBBytes = BN * kSpan, kSf = kSfTiles * kMxTileBytes;
    static constexpr int kStageBytes = kABytes + kBBytes + 2 * kSf;
    static_assert(kStageBytes % 1024 == 0, "operands on 1024-byte borders");
    static constexpr int kSums = NS > 1 ? kBM * BN * 4 : 0;         // the cluster's sums of this CTA's tokens
    static constexpr int kMost = (BN <= 32 ? 112 : 220) * 1024;     // shared memory: two CTAs an SM, or one
    static constexpr int kMaxStages = (kMost - kSums - 2048) / kStageBytes;
    // tensor memory: the accumulator, then the scales of W and of x, 4 columns a tile.  As many CTAs with a cluster as an
    // SM's shared memory holds (7, 5 and 3 of them) never have to wait for columns, which a CTA keeps until its cluster
    // is done.  (More CTAs without one may have to, for others that wait for none.)
    static constexpr int kSfaCol = BN, kSfbCol = BN + 4 * kSfTiles, kUsed = kSfbCol + 4 * kSfTiles;
    static constexpr int kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : 128;
    static constexpr int alloc(int stages) { return stages * kStageBytes + kSums + 8 * (2 * stages + 1) + 16 + 1024; }
};

struct Params {
    const uint8_t *x_scales, *w_scales;
    __nv_bfloat16* y[3];
    int seg_end[3];     // cumulative widths; seg_end[2] == out
    uint32_t* err;
    uint64_t wait_ns;   // limit of a wait
    int tokens, in, out, stages;
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

template <int kType, int BN, int NS>
__global__ void __launch_bounds__(kThreads)
    mx_linear_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, Params p)
{
    using S = Shape<kType, BN, NS>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;  // (the same offset in the cluster's CTAs)
    uint8_t* sbase = smem_raw + (base - raw_base);
    const uint32_t sums = base + p.stages * S::kStageBytes, bar_full = sums + S::kSums, bar_empty = bar_full + 8 * p.stages,
                   bar_done = bar_empty + 8 * p.stages, slot = bar_done + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int m_tiles = p.out / kBM, rank = blockIdx.x % NS, tile = blockIdx.x / NS;
    const int m0 = (tile % m_tiles) * kBM, n0 = (tile / m_tiles) * BN;
    // this CTA's share of the input features, in stages; the last one of a 4-bit row may be half
    const int sf_tiles = p.in / kMxTileCols, nk = (sf_tiles + S::kSfTiles - 1) / S::kSfTiles;
    const int k0 = nk * rank / NS, k1 = nk * (rank + 1) / NS;

    // ---- operands and scales of one stage (warp 0)
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    const uint8_t* sfw = p.w_scales + (int64_t)(m0 / 128) * sf_tiles * kMxTileBytes;
    const uint8_t* sfx = p.x_scales + (int64_t)(n0 / 128) * sf_tiles * kMxTileBytes;
    auto load = [&](int k, int st) {
        const uint32_t a = base + st * S::kStageBytes, b = a + S::kABytes, sf = b + S::kBBytes, bar = bar_full + 8 * st;
        const uint32_t sf_bytes = min(S::kSfTiles, sf_tiles - k * S::kSfTiles) * kMxTileBytes;
        mbar_arrive_expect_tx_warp(bar, S::kABytes + S::kBBytes + 2 * sf_bytes);
        tma_load_2d_warp(a, &tmW, k * kSpan, m0, bar, pol_w);
        tma_load_2d_warp(b, &tmX, k * kSpan, n0, bar, pol_x);
        bulk_copy_g2s_warp(sf, sfw + k * S::kSf, sf_bytes, bar);
        bulk_copy_g2s_warp(sf + S::kSf, sfx + k * S::kSf, sf_bytes, bar);
    };

    if (NS > 1) cluster_arrive();  // (waited for before the first store to another CTA: it has started then)
    const int early = min(k1 - k0, p.stages);
    if (warp == 0) {
        if (elect_one()) {
            for (int i = 0; i < 2 * p.stages + 1; ++i) mbar_init(bar_full + 8 * i, 1);
            fence_mbar_init();
        }
        __syncwarp();
        // W on its way to L2 before the wait for the kernel before this one (which may have written it:
        // what is read comes after the wait)
        for (int k = k0; k < k0 + early; ++k) tma_prefetch_2d_warp(&tmW, k * kSpan, m0);
        pdl_wait();
        for (int k = 0; k < early; ++k) load(k0 + k, k);
    } else if (warp == 1) {
        tmem_alloc(slot, S::kCols);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sbase + (slot - base)), 0);
    pdl_launch_dependents();

    if (warp == 0) {
        Waits wait(p.wait_ns);
        int st = 0;
        uint32_t parity = 0;
        for (int k = k0 + early; k < k1; ++k) {
            if (!__all_sync(0xffffffffu, wait.on(bar_empty + 8 * st, parity))) break;
            load(k, st);
            if (++st == p.stages) st = 0, parity ^= 1;
        }
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    } else if (warp == 1) {
        // ---- products (a wait that ran out does not end the loop, which would make its counters differ between
        // lanes).  A stage is looked for before the products of the one before it are issued, which takes as long as
        // the look.
        Waits wait(p.wait_ns);
        bool there = mbar_try_wait(bar_full, 0);
        int st = 0;
        uint32_t parity = 0;
        for (int k = k0; k < k1; ++k) {
            if (!there) wait.on(bar_full + 8 * st, parity);
            __syncwarp();
            const int cur = st;
            if (++st == p.stages) st = 0, parity ^= 1;
            there = k + 1 < k1 && mbar_test_wait(bar_full + 8 * st, parity);
            tc_fence_after();
            const uint32_t a = base + cur * S::kStageBytes, b = a + S::kABytes, sf = b + S::kBBytes;
            const int have = min(S::kSfTiles, sf_tiles - k * S::kSfTiles);
            const uint32_t sfb = tmem + S::kSfbCol + (BN == 64 ? n0 % 128 / 32 : 0);  // (the second half of a block)
            const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
            constexpr int kPer = 4 / S::kSfTiles;  // products a tile of scales
#pragma unroll
            for (int s = 0; s < S::kSfTiles; ++s) {
                umma_copy_scales_warp(tmem + S::kSfaCol + 4 * s, sf + s * kMxTileBytes);
                umma_copy_scales_warp(tmem + S::kSfbCol + 4 * s, sf + S::kSf + s * kMxTileBytes);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const int s = kk / kPer;
                if (s < have)
                    umma_mx_warp<kType == PKV_MX4>(tmem, da + 2 * kk, db + 2 * kk,
                                                   umma_idesc_mx(kType == PKV_MX4, kBM, BN, kk % kPer * (4 / kPer)),
                                                   tmem + S::kSfaCol + 4 * s, sfb + 4 * s, k > k0 || kk > 0);
            }
            if (k1 - k0 > p.stages) umma_commit_warp(bar_empty + 8 * cur);  // (else no stage is loaded again)
        }
        umma_commit_warp(bar_done);
        if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    }
    __syncwarp();

    // ---- each thread has a feature of every token
    constexpr int kOwn = BN / NS, kVec = kOwn < 4 ? kOwn : 4, kRounds = kOwn / kVec;
    static_assert(kVec >= 2, "two tokens a CTA at least");
    Waits wait(p.wait_ns);
    const bool ok = wait.on(bar_done, 0);
    if (!wait.ok()) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    tc_fence_after();
    if (NS > 1) cluster_wait();
    const int tokens = min(BN, p.tokens - n0), feature = 32 * warp + lane;
    constexpr int kCols = BN < 32 ? BN : 32;  // of a load
    uint32_t v[BN / kCols][kCols];
#pragma unroll
    for (int c = 0; c < BN / kCols; ++c) {
        const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16) + kCols * c;
        if constexpr (kCols == 16)
            tmem_ld16(at, v[c]);
        else
            tmem_ld32(at, v[c]);
    }
#pragma unroll
    for (int c = 0; c < BN / kCols; ++c) tmem_wait_ld_regs(v[c]);
    if constexpr (NS == 1) {
        // no cluster: two lanes share their tokens out, so that each writes two features of a token at a time (128 tokens,
        // 4096 x 6144 in 4 bits 6.5 us; 0.9 more through shared memory as below)
        int yw, yc;
        __nv_bfloat16* const y = segment(p, m0, yw, yc) + (int64_t)n0 * yw + yc + (feature & ~1);
        const bool odd = lane & 1;
#pragma unroll
        for (int t = 0; t < BN; t += 2) {
            const float lo = __uint_as_float(v[t / kCols][t % kCols]), hi = __uint_as_float(v[t / kCols][t % kCols + 1]);
            const float other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            const float a = odd ? other : lo, b = odd ? hi : other;
            if (t + odd < tokens)
                *reinterpret_cast<uint32_t*>(y + (int64_t)(t + odd) * yw) =
                    ok ? pack_bf16(__float2bfloat16_rn(a), __float2bfloat16_rn(b)) : 0u;
        }
        tc_fence_before();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(tmem, S::kCols);
        }
        return;
    }
    // ---- to the token's CTA: [CTA it comes from][its tokens / 4][features][4]
#pragma unroll
    for (int t = 0; t < BN; t += kVec) {
        if (t >= tokens) break;
        float f[4];
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = ok ? __uint_as_float(v[t / kCols][t % kCols + i]) : 0.f;
        const uint32_t at = sums + (uint32_t)((rank * kRounds + t % kOwn / kVec) * kBM + feature) * (4 * kVec);
        const uint32_t to = cluster_map(at, t / kOwn);
        if constexpr (kVec == 4)
            st_cluster_f32x4(to, f[0], f[1], f[2], f[3]);
        else
            st_cluster_f32x2(to, f[0], f[1]);
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kCols);
    }
    // ---- this CTA's tokens: a thread adds up its feature of kVec of them; two lanes then share theirs out
    int yw, yc;
    __nv_bfloat16* const y = segment(p, m0, yw, yc) + (int64_t)n0 * yw;
    const bool odd = lane & 1;
    for (int i = 0; i < kRounds; ++i) {
        const int t0 = rank * kOwn + i * kVec;
        if (t0 >= tokens) break;
        float acc[kVec];
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            const float* from = reinterpret_cast<const float*>(sbase + (sums - base)) + (size_t)((q * kRounds + i) * kBM + feature) * kVec;
            float part[kVec];
            if constexpr (kVec == 4) {
                const float4 u = *reinterpret_cast<const float4*>(from);
                part[0] = u.x, part[1] = u.y, part[2] = u.z, part[3] = u.w;
            } else {
                const float2 u = *reinterpret_cast<const float2*>(from);
                part[0] = u.x, part[1] = u.y;
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) acc[j] = q ? acc[j] + part[j] : part[j];
        }
        // the even lane takes the first half of the tokens for both features, the odd lane the second
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {
            const float lo = acc[j], hi = acc[j + kVec / 2];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
            const int t = t0 + j + (odd ? kVec / 2 : 0);
            const float a = odd ? other : lo, b = odd ? hi : other;
            if (t < tokens)
                *reinterpret_cast<uint32_t*>(y + (int64_t)t * yw + yc + (feature & ~1)) =
                    pack_bf16(__float2bfloat16_rn(a), __float2bfloat16_rn(b));
        }
    }
}

template <int kType, int BN, int NS>
cudaError_t launch(const MxLinear& a, Params& p, const CUtensorMap& tmW, const CUtensorMap& tmX, cudaStream_t s)
{
    using S = Shape<kType, BN, NS>;
    const cudaError_t e = cudaFuncSetAttribute(mx_linear_kernel<kType, BN, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               S::alloc(S::kMaxStages));
    if (e != cudaSuccess) return e;
    const int nk = (mx_row_bytes(kType, a.in) + kSpan - 1) / kSpan, share = (nk + NS - 1) / NS;
    p.stages = share < S::kMaxStages ? share : S::kMaxStages;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = NS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.out / kBM) * ((a.tokens + BN - 1) / BN) * NS));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::alloc(p.stages);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mx_linear_kernel<kType, BN, NS>, tmW, tmX, p);
}

template <int kType, int BN>
cudaError_t launch_bn(const MxLinear& a, Params& p, int splits, cudaStream_t s)
{
    CUtensorMap tmW, tmX;
    const int row = mx_row_bytes(kType, a.in);
    if (!make_tmap_bytes(&tmW, a.w_codes, row, p.out, kBM) || !make_tmap_bytes(&tmX, a.x_codes, row, a.tokens, BN))
        return cudaErrorInvalidValue;
    switch (splits) {
        case 1: return launch<kType, BN, 1>(a, p, tmW, tmX, s);
        case 2: return launch<kType, BN, 2>(a, p, tmW, tmX, s);
        case 4: return launch<kType, BN, 4>(a, p, tmW, tmX, s);
        default: return launch<kType, BN, 8>(a, p, tmW, tmX, s);
    }
}

template <int kType>
cudaError_t launch_type(const MxLinear& a, Params& p, const MxRoute& r, cudaStream_t s)
{
    switch (r.tile) {
        case 16: return launch_bn<kType, 16>(a, p, r.splits, s);
        case 32: return launch_bn<kType, 32>(a, p, r.splits, s);
        default: return launch_bn<kType, 64>(a, p, r.splits, s);
    }
}

}  // namespace

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
    p.wait_ns = pool->wait_ns;
    p.tokens = a.tokens;
    p.in = a.in;
    p.out = p.seg_end[2];
    const MxRoute r = mx_route(a.type == PKV_MX8 ? a.in : a.in / 2, p.tokens, p.out, pool->num_sms);
    if (r.pairs) return launch_mx_pair(pool, a, s);
    return a.type == PKV_MX8 ? launch_type<PKV_MX8>(a, p, r, s) : launch_type<PKV_MX4>(a, p, r, s);
}

}  // namespace pkv
