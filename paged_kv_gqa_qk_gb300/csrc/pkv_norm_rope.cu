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
// Bound by memory: 8192 tokens of 40 heads to fp32, 252 MB, in 40.1 us, 6.3 TB/s; to bf16, 168 MB,
// in 31.5, 5.3 TB/s.
//
// One CTA per token; warp w of W takes the groups w, w + W, ... of 4 heads (q's, then k's),
// the next group's loads out before one is computed.
//
// kRot: the rotated dims in the half layout, whose pairs lie differently for each of the four
// that a pool can have (one form for all of them took 47 us for 8192 tokens to fp32, and 4.1
// instead of 2.7 for 300, with its selects).  Interleaved pairs are alike for every p.rot.
template <bool kInterleaved, bool kF32, int kRot>
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

    // (cos, sin) of the lane's dims 32 m + 4 j .. + 3, or of those that share their pairs: half layout, the sets are m = 0
    // (32 and 64 rotated dims), 0 and 1 (128), 0, 1 and 2 (96)
    constexpr int kSets = kInterleaved ? 4 : kRot == 128 ? 2 : kRot == 96 ? 3 : 1;
    float2 cs[kSets][4];
    const bool low = j < 4;
#pragma unroll
    for (int m = 0; m < kSets; ++m) {
        const int d = 4 * j + 32 * m;
#pragma unroll
        for (int k = 0; k < 4; ++k) cs[m][k] = make_float2(1.f, 0.f);
        if (!ok || (kInterleaved && d >= p.rot)) continue;
        const bool second = !kInterleaved && kRot % 64 != 0 && d >= kRot / 2;  // of its pair: its partner's term is added
        const float2* row = p.rope + (int64_t)pos * kRopeHalf + (kInterleaved ? d / 2 : second ? d - kRot / 2 : d);
        const float4 a = *reinterpret_cast<const float4*>(row);
        if constexpr (kInterleaved) {
            cs[m][0] = cs[m][1] = make_float2(a.x, a.y);
            cs[m][2] = cs[m][3] = make_float2(a.z, a.w);
        } else {
            const float4 b = *reinterpret_cast<const float4*>(row + 2);
            cs[m][0] = make_float2(a.x, a.y), cs[m][1] = make_float2(a.z, a.w);
            cs[m][2] = make_float2(b.x, b.y), cs[m][3] = make_float2(b.z, b.w);
            if (kRot % 64 != 0 && !second)
#pragma unroll
                for (int k = 0; k < 4; ++k) cs[m][k].y = -cs[m][k].y;
        }
    }
    // weights as they are where the pairs take two sets of cos and sin or more: 64 registers instead of 86, and with
    // them more warps (8192 tokens to fp32 40.8 us, 41.9 as floats); else as floats (to bf16 28.9 us, 31.0)
    constexpr bool kPacked = kInterleaved || kRot == 128;
    uint2 packed[kPacked ? 4 : 1];
    float w[kPacked ? 1 : 4][4];
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
                for (int m = 0; m < 4; ++m) {
                    const uint2 a = *reinterpret_cast<const uint2*>(wp + 4 * j + 32 * m);
                    if constexpr (kPacked)
                        packed[m] = a;
                    else
                        unpack4(a, w[m]);
                }
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
            for (int m = 0; m < 4; ++m) {
                float unpacked[4];
                if constexpr (kPacked) unpack4(packed[m], unpacked);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (kPacked)
                        x[m][k] *= unpacked[k];
                    else
                        x[m][k] *= w[m][k];
                }
            }
        }
        if constexpr (kInterleaved) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {  // (not rotated: cos 1, sin 0)
                    y[m][k] = inv * (x[m][k] * cs[m][k].x - x[m][k + 1] * cs[m][k].y);
                    y[m][k + 1] = inv * (x[m][k + 1] * cs[m][k].x + x[m][k] * cs[m][k].y);
                }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kRot % 64 == 0) {  // partners in the lane itself
#pragma unroll
                    for (int m = 0; m < kSets; ++m) {
                        constexpr int kTo = kRot / 64;
                        y[m][k] = inv * (x[m][k] * cs[m][k].x - x[m + kTo][k] * cs[m][k].y);
                        y[m + kTo][k] = inv * (x[m + kTo][k] * cs[m][k].x + x[m][k] * cs[m][k].y);
                    }
                } else {  // in lane j ^ 4: of 96 dims, dims + 48 or - 48
                    float other[kSets];
#pragma unroll
                    for (int m = 0; m < kSets; ++m) other[m] = __shfl_xor_sync(kFull, x[m][k], 4);
#pragma unroll
                    for (int m = 0; m < kSets; ++m) {
                        const float up = kSets == 1 ? other[0] : low ? other[(m + 1) % kSets] : other[(m + 2) % kSets];
                        y[m][k] = inv * (x[m][k] * cs[m][k].x + up * cs[m][k].y);
                    }
                }
#pragma unroll
                for (int m = kRot / 32; m < 4; ++m) y[m][k] = inv * x[m][k];
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
    // up to a token an SM: a warp a group of heads, for the latency; more: half of that, and with more tokens as few as
    // leave 32 warps an SM, which share the loads of a token's tables and weights, but two (40 heads, 10 groups, to
    // fp32; us with 1 / 2 / 4 / 5 / 10 warps: 300 tokens 5.2 / 3.6 / 2.9 / 2.7 / 3.2, 1000 9.4 / 6.5 / 6.0 / 6.8 / 7.7,
    // 4000 22.4 / 20.9 / 21.4 / 22.0, 8192 40.8 / 40.1; one token 2.1 with five, 2.0 with ten)
    const int most = std::min(groups, 16), fair = std::min((groups + 1) / 2, 32 * pool->num_sms / a.tokens);
    const int warps = a.tokens <= pool->num_sms ? most : std::min(most, std::max(2, fair));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.tokens);
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto launch = [&](auto to_f32, auto to_bf16) { return cudaLaunchKernelEx(&cfg, a.f32 ? to_f32 : to_bf16, p); };
    if (a.interleaved) return launch(norm_rope_kernel<true, true, 128>, norm_rope_kernel<true, false, 128>);
    switch (p.rot) {
        case 32: return launch(norm_rope_kernel<false, true, 32>, norm_rope_kernel<false, false, 32>);
        case 64: return launch(norm_rope_kernel<false, true, 64>, norm_rope_kernel<false, false, 64>);
        case 96: return launch(norm_rope_kernel<false, true, 96>, norm_rope_kernel<false, false, 96>);
        default: return launch(norm_rope_kernel<false, true, 128>, norm_rope_kernel<false, false, 128>);
    }
}

}  // namespace pkv
