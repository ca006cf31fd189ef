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

// Eight lanes a head: lane j holds dims 4j + 32m .. + 3 for m = 0..3, so that loads and
// stores of 8 lanes are whole lines, the sum of squares takes three shuffles for four
// heads, and the partner of a dim lies in the lane itself (interleaved pairs, and
// halves of 128 or 64 rotated dims) or in lane j ^ 4 (32 and 96).
//
// One CTA per token; warp w of W takes the groups w, w + W, ... of 4 heads (q's, then k's),
// the next group's loads out before one is computed.
template <bool kInterleaved, bool kF32, bool kFullRot>
__global__ void __launch_bounds__(512) norm_rope_kernel(NormRopeParams p)
{
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int j = lane & 7, sub = lane >> 3;
    const int qg = (p.heads[0] + 3) / 4, groups = qg + (p.heads[1] + 3) / 4;
    pdl_wait();  // (launched while the kernel before it drains)
    pdl_launch_dependents();
    uint2 raw[4] = {};
    auto load = [&](int grp) {
        const bool is_k = grp >= qg;
        const int h = 4 * (grp - (is_k ? qg : 0)) + sub;
        if (grp >= groups || h >= (is_k ? p.heads[1] : p.heads[0])) return;
        const __nv_bfloat16* x = (is_k ? p.x[1] + t * p.x_stride[1] : p.x[0] + t * p.x_stride[0]) + h * kHeadDim + 4 * j;
#pragma unroll
        for (int m = 0; m < 4; ++m) raw[m] = *reinterpret_cast<const uint2*>(x + 32 * m);
    };
    load(warp);
    const int pos = p.positions[t];
    const bool ok = pos >= 0 && pos < p.max_seq;
    if (!ok && pos != -1 && threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_POSITION);

    // (cos, sin) of the lane's dims; part[m]: where their partners are (half layout)
    float2 cs[4][4];
    int part[4];
    float sgn[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int d = 4 * j + 32 * m, half = p.rot / 2;
        const bool rotated = d < p.rot, first = d < half;
        const int pd = kInterleaved ? d : (first ? d + half : d - half);
        part[m] = pd >> 5;
        sgn[m] = first ? -1.f : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) cs[m][k] = make_float2(1.f, 0.f);
        if (!ok || !rotated || (kFullRot && !kInterleaved && m >= 2)) continue;
        const float2* row = p.rope + (int64_t)pos * kRopeHalf + (kInterleaved ? d / 2 : (first ? d : pd));
        const float4 a = *reinterpret_cast<const float4*>(row);
        if constexpr (kInterleaved) {
            cs[m][0] = cs[m][1] = make_float2(a.x, a.y);
            cs[m][2] = cs[m][3] = make_float2(a.z, a.w);
        } else {
            const float4 b = *reinterpret_cast<const float4*>(row + 2);
            cs[m][0] = make_float2(a.x, a.y), cs[m][1] = make_float2(a.z, a.w);
            cs[m][2] = make_float2(b.x, b.y), cs[m][3] = make_float2(b.z, b.w);
        }
    }
    const bool near = kInterleaved || p.rot % 64 == 0;  // partners in the lane itself
    float w[4][4];
    const __nv_bfloat16* have = nullptr;
    for (int grp = warp; grp < groups; grp += warps) {
        const bool is_k = grp >= qg;
        const int h = 4 * (grp - (is_k ? qg : 0)) + sub;
        float x[4][4], y[4][4];
#pragma unroll
        for (int m = 0; m < 4; ++m) unpack4(raw[m], x[m]);
        load(grp + warps);
        const __nv_bfloat16* wp = is_k ? p.w[1] : p.w[0];
        float inv = 1.f;
        if (wp) {
            if (wp != have) {
#pragma unroll
                for (int m = 0; m < 4; ++m) unpack4(*reinterpret_cast<const uint2*>(wp + 4 * j + 32 * m), w[m]);
                have = wp;
            }
            float ss = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) ss = __fmaf_rn(x[m][k], x[m][k], ss);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
            inv = rsqrtf(__fmaf_rn(ss, 1.0f / kHeadDim, p.eps));
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) x[m][k] *= w[m][k];
        }
        if constexpr (kInterleaved) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {  // (not rotated: cos 1, sin 0)
                    y[m][k] = inv * (x[m][k] * cs[m][k].x - x[m][k + 1] * cs[m][k].y);
                    y[m][k + 1] = inv * (x[m][k + 1] * cs[m][k].x + x[m][k] * cs[m][k].y);
                }
        } else if constexpr (kFullRot) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    y[m][k] = inv * (x[m][k] * cs[m][k].x - x[m + 2][k] * cs[m][k].y);
                    y[m + 2][k] = inv * (x[m + 2][k] * cs[m][k].x + x[m][k] * cs[m][k].y);
                }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float other[4];  // dims + 32m of the lane with the partners (m = 3 is never rotated)
#pragma unroll
                for (int m = 0; m < 3; ++m) other[m] = near ? x[m][k] : __shfl_xor_sync(kFull, x[m][k], 4);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float up = sgn[m] * (part[m] == 0 ? other[0] : part[m] == 1 ? other[1] : other[2]);
                    y[m][k] = inv * (x[m][k] * cs[m][k].x + up * cs[m][k].y);
                }
            }
        }
        if (h >= (is_k ? p.heads[1] : p.heads[0])) continue;
        const int64_t at = (is_k ? t * p.y_stride[1] : t * p.y_stride[0]) + h * kHeadDim + 4 * j;
        void* dst = is_k ? p.y[1] : p.y[0];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (!ok) y[m][0] = y[m][1] = y[m][2] = y[m][3] = 0.f;  // no position, no vector
            if constexpr (kF32)
                *reinterpret_cast<float4*>(static_cast<float*>(dst) + at + 32 * m) = make_float4(y[m][0], y[m][1], y[m][2], y[m][3]);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(dst) + at + 32 * m) = pack4(y[m]);
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
    const int groups = (p.heads[0] + 3) / 4 + (p.heads[1] + 3) / 4;
    // few tokens: a warp a group of heads, for the latency; many: as few warps a token as leave 32 an SM,
    // which share the loads of its tables and weights (8192 tokens of 40 heads, interleaved, fp32 out, 252 MB:
    // 42.3 us with one warp a token, 43.0 with two, 46.5 with four; one token 2.1 us a call with ten)
    const int warps = std::min(std::min(groups, 16), std::max(1, 32 * pool->num_sms / a.tokens));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.tokens);
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool full = p.rot == kHeadDim;
    auto launch = [&](auto kernel_full, auto kernel) { return cudaLaunchKernelEx(&cfg, full ? kernel_full : kernel, p); };
    if (a.interleaved)
        return a.f32 ? launch(norm_rope_kernel<true, true, true>, norm_rope_kernel<true, true, true>)
                     : launch(norm_rope_kernel<true, false, true>, norm_rope_kernel<true, false, true>);
    return a.f32 ? launch(norm_rope_kernel<false, true, true>, norm_rope_kernel<false, true, false>)
                 : launch(norm_rope_kernel<false, false, true>, norm_rope_kernel<false, false, false>);
}

}  // namespace pkv
