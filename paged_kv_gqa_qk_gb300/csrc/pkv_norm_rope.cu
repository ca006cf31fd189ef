// QK-norm of every query and key head and the rotation of its position in one
// pass over a batch of tokens (sm_103a): pkv_norm_rope.
//
//   y = rope(x / sqrt(mean(x^2) + eps) * w)
//
// qwen3-8b Nest files, src/norm.linnet (RmsNorm) and src/rope.linnet (tables);
// pairs (i, i + R/2) of the first R dims (half layout) or (2i, 2i + 1)
// (interleaved), the rest of the head as it is.  cos and sin are the pool's
// fp32 tables; the arithmetic is fp32, rounded once to the output's type.
#include <algorithm>

#include "pkv_internal.h"
#include "pkv_rope.cuh"

namespace pkv {

struct NormRopeParams {
    const __nv_bfloat16* x[2];  // q and k
    const __nv_bfloat16* w[2];  // norm weights, or null: no norm
    void* y[2];
    int64_t x_stride[2], y_stride[2];  // elements between tokens
    const int32_t* positions;
    const float2* rope;         // (cos, sin) [max_seq][64]
    uint32_t* err;
    int heads[2];               // 0: not given
    int tokens, max_seq, rot;
    float eps;
};

constexpr int kNormRopeBatch = 5;  // heads a warp loads before the first use

// One CTA per token; of W warps, warp w takes heads w, w + W, ... of q's and k's heads in
// one list.  Bound by memory for many tokens, where 4 warps measured best (8192 tokens of
// 40 heads, fp32 out, 252 MB: 44 us; 8 warps 49, 10 warps 54), and by one token's latency
// for few, where each warp gets at most 4 heads (one token: 3.0 us a call, 4.2 with 4 warps).
template <bool kInterleaved, bool kF32, int kMaxWarps>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_rope_kernel(NormRopeParams p)
{
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nq = p.heads[0], all = nq + p.heads[1];
    pdl_wait();  // (launched while the kernel before it drains)
    pdl_launch_dependents();
    const int pos = p.positions[t];
    const bool ok = pos >= 0 && pos < p.max_seq;
    if (!ok && pos != -1 && threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_POSITION);

    const KRope kr = krope(lane, p.rot);
    float2 cs[4];
    if (ok) {
        const float2* row = p.rope + (int64_t)pos * kRopeHalf;
        if constexpr (kInterleaved) {
            const float4 a = *reinterpret_cast<const float4*>(row + 2 * lane);  // pairs 2 lane, 2 lane + 1
            cs[0] = cs[1] = make_float2(a.x, a.y);
            cs[2] = cs[3] = make_float2(a.z, a.w);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(row + kr.f0), b = *reinterpret_cast<const float4*>(row + kr.f0 + 2);
            cs[0] = make_float2(a.x, a.y), cs[1] = make_float2(a.z, a.w);
            cs[2] = make_float2(b.x, b.y), cs[3] = make_float2(b.z, b.w);
        }
    }
    float w[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i][0] = w[i][1] = w[i][2] = w[i][3] = 1.f;
        if (p.w[i]) unpack4(*reinterpret_cast<const uint2*>(p.w[i] + 4 * lane), w[i]);
    }
    for (int h0 = warp; h0 < all; h0 += warps * kNormRopeBatch) {
        uint2 raw[kNormRopeBatch];
#pragma unroll
        for (int b = 0; b < kNormRopeBatch; ++b) {
            const int h = h0 + b * warps, is_k = h >= nq;
            if (h < all)
                raw[b] = *reinterpret_cast<const uint2*>((is_k ? p.x[1] + t * p.x_stride[1] - nq * kHeadDim : p.x[0] + t * p.x_stride[0]) +
                                                         h * kHeadDim + 4 * lane);
        }
#pragma unroll
        for (int b = 0; b < kNormRopeBatch; ++b) {
            const int h = h0 + b * warps, is_k = h >= nq;
            if (h >= all) break;
            float x[4], y[4] = {0.f, 0.f, 0.f, 0.f};
            unpack4(raw[b], x);
            const float inv = (is_k ? p.w[1] : p.w[0]) ? inv_rms(x, p.eps) : 1.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] *= is_k ? w[1][k] : w[0][k];
            if constexpr (kInterleaved) {
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const bool rot = 4 * lane < p.rot;
                    const float a = x[k], c = x[k + 1];
                    y[k] = inv * (rot ? a * cs[k].x - c * cs[k].y : a);
                    y[k + 1] = inv * (rot ? c * cs[k].x + a * cs[k].y : c);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float up = kr.sgn * __shfl_sync(kFull, x[k], kr.src);
                    y[k] = inv * (kr.rot ? x[k] * cs[k].x + up * cs[k].y : x[k]);
                }
            }
            if (!ok) y[0] = y[1] = y[2] = y[3] = 0.f;  // no position, no vector
            const int64_t at = (is_k ? t * p.y_stride[1] - nq * kHeadDim : t * p.y_stride[0]) + h * kHeadDim + 4 * lane;
            void* dst = is_k ? p.y[1] : p.y[0];
            if constexpr (kF32)
                *reinterpret_cast<float4*>(static_cast<float*>(dst) + at) = make_float4(y[0], y[1], y[2], y[3]);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + at) = pack4(y);
        }
    }
}

cudaError_t launch_norm_rope(const pkv_pool* pool, const NormRope& a, cudaStream_t s)
{
    NormRopeParams p;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const __nv_bfloat16*>(a.x[i]);
        p.w[i] = static_cast<const __nv_bfloat16*>(a.w[i]);
        p.y[i] = a.y[i];
        p.x_stride[i] = a.x_stride[i];
        p.y_stride[i] = a.y_stride[i];
        p.heads[i] = a.x[i] ? (i ? pool->cfg.kv_heads : pool->cfg.heads) : 0;
    }
    p.positions = a.positions;
    p.rope = pool->rope_hi;
    p.err = pool->err;
    p.tokens = a.tokens;
    p.max_seq = pool->cfg.max_seq;
    p.rot = pool->cfg.rotary_dim > 0 ? pool->cfg.rotary_dim : kHeadDim;
    p.eps = (float)pool->cfg.eps;
    const int all = p.heads[0] + p.heads[1];
    const bool few = a.tokens <= 2 * pool->num_sms;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.tokens);
    cfg.blockDim = dim3(32 * (few ? std::min((all + 3) / 4, 16) : 4));
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto launch = [&](auto kernel_few, auto kernel) { return cudaLaunchKernelEx(&cfg, few ? kernel_few : kernel, p); };
    if (a.interleaved)
        return a.f32 ? launch(norm_rope_kernel<true, true, 16>, norm_rope_kernel<true, true, 4>)
                     : launch(norm_rope_kernel<true, false, 16>, norm_rope_kernel<true, false, 4>);
    return a.f32 ? launch(norm_rope_kernel<false, true, 16>, norm_rope_kernel<false, true, 4>)
                 : launch(norm_rope_kernel<false, false, 16>, norm_rope_kernel<false, false, 4>);
}

}  // namespace pkv
