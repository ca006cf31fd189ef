// The 4-bit page format and its device helpers: where codes and scales lie in a
// page, quantising a head held by a warp, and k at the accuracy the quantiser
// needs.
//
// A value is code * scale * s: the code in 4 bits (sign, two exponent bits, one
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), the scale of its group of 16 dims in
// 8 bits (e4m3), s a power of two of the whole pool.  One head vector of 128 dims
// takes 72 bytes instead of 256.
//
// A page of one kv head is 4 blocks of 16 positions, 2304 contiguous bytes each
// (so the positions a row has used are a prefix of the page, to 16 positions):
//   K codes [16][64], V codes [16][64], K scales [128], V scales [128].
// Positions and scales are placed for the loads of the attention's tensor-core
// fragments (q4_attn_kernel), which then are conflict-free 16-, 8- and 4-byte
// reads of shared memory:
//   codes of position i: byte j (dims 2j low half, 2j + 1 high half) at 64 i + (j ^ 32 bit1(i));
//   with b = bit2(i), c = (i & 3) ^ b:
//   K scale of group g at 16 (2c + b) + 4 (g >> 1) + (g & 1) + 2 (i >> 3)
//   V scale of group g at 16 g + 4 c + b + 2 (i >> 3).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pkv_rope.cuh"

namespace pkv {

constexpr int kQ4Block = 16;                                     // positions of a block
constexpr int kQ4BlockBytes = 2 * kQ4Block * (kHeadDim / 2 + kHeadDim / 16);  // 2304
constexpr int kQ4VCodes = kQ4Block * kHeadDim / 2;               // 1024
constexpr int kQ4KScales = 2 * kQ4VCodes;                        // 2048
constexpr int kQ4VScales = kQ4KScales + kQ4Block * kHeadDim / 16;  // 2176

__device__ __forceinline__ int q4_code_row(int i, int byte) { return 64 * i + (byte ^ (((i >> 1) & 1) << 5)); }
__device__ __forceinline__ int q4_k_scale(int i, int g)
{
    const int b = (i >> 2) & 1, c = (i & 3) ^ b;
    return kQ4KScales + 16 * (2 * c + b) + 4 * (g >> 1) + (g & 1) + 2 * (i >> 3);
}
__device__ __forceinline__ int q4_v_scale(int i, int g)
{
    const int b = (i >> 2) & 1, c = (i & 3) ^ b;
    return kQ4VScales + 16 * g + 4 * c + b + 2 * (i >> 3);
}

// Block holding position s of pool page `page` for kv head g.
__device__ __forceinline__ int64_t q4_block(int64_t page, int kv_heads, int g, int s)
{
    return (page * kv_heads + g) * kQ4PageBytes + (s / kQ4Block) * kQ4BlockBytes;
}

// Two codes (one byte: low half first) as fp16, and two e4m3 scales as fp16.  Both are exact, and
// so is their product: 2 + 4 significant bits, at most 6 * 448, at least 2^-10 where not 0.
__device__ __forceinline__ void q4_unpack(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t two)
{
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// ---- a head vector over 8 lanes ---------------------------------------------------------
// Lane j of 8 holds dims 8j .. 8j + 7 (elements 0-7) and 64 + 8j .. 64 + 8j + 7 (8-15): two
// 16-byte loads of bf16, the rotate-half partners of a full rotation in the lane
// itself, and halves of groups j >> 1 and 4 + (j >> 1), whose other halves lane j ^ 1
// holds.  (With 4 dims a lane over a whole warp, sums over the head and the scales of
// a group cost four times the instructions.)
__device__ __forceinline__ void unpack16(uint4 lo, uint4 hi, float (&x)[16])
{
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

// The largest |x| of 8 bf16 (4 words of two) as its bits, sign cleared; Inf and NaN order above the rest.
__device__ __forceinline__ uint32_t max8_bits(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t e = d & kAbs, m = __vimax3_u16x2(__vimax3_u16x2(a & kAbs, b & kAbs, c & kAbs), e, e);
    return max(m >> 16, m & 0xffffu);
}

// Quantises the head vector (x: bf16 values in fp32, w: the same as they are) to
// position i of `block`.  s is a power of two.
//   scale = e4m3(max |x| / (6 s)), codes = e2m1(x / (scale s)), both to nearest, ties to even.
// x has 8 significant bits, and a tie of a scale (5 bits) times 6 or of a code (3 bits)
// times a scale (4 bits) at most 7, so a quotient that is not a tie is off it by more
// than 2^-10 of its value: only the ties themselves need care.  Those of a scale come
// out exact from the product with 1 / 6 to nearest (checked for all 32), those of a
// code from the product with the inverse as a pair of floats.  A group that holds an
// Inf or a NaN gets the scale NaN: the positions that read it are NaN, as with a bf16 pool.
//   inv6s = 1 / (6 s) to nearest, inv_s = 1 / s
__device__ __forceinline__ void q4_store(uint8_t* block, bool is_v, int i, const float (&x)[16], const uint32_t (&w)[8],
                                         float inv6s, float inv_s, int j, bool live)
{
    uint32_t word[2], scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t top = max8_bits(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        uint16_t sc;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(sc) : "f"(__uint_as_float(top << 16) * inv6s));
        scale[h] = top >= 0x7f80u ? 0x7fu : sc & 0xffu;
        const float step = __half2float(__ushort_as_half((unsigned short)(e4m3x2_half2(scale[h]) & 0xffffu)));
        float r = 0.f, rl = 0.f;
        if (step > 0.f) {  // (NaN: 0, any code will do)
            r = __frcp_rn(step);
            rl = __fmaf_rn(-step, r, 1.f) * r * inv_s;
            r *= inv_s;
        }
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)  // (rounded towards 0, the correction cannot overflow: far beyond the scale x r decides)
            y[k] = __fmaf_rn(x[8 * h + k], r, __fmul_rz(x[8 * h + k], rl));
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(word[h])
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    }
    if (!live) return;
    uint8_t* codes = block + (is_v ? kQ4VCodes : 0);
    *reinterpret_cast<uint32_t*>(codes + q4_code_row(i, 4 * j)) = word[0];
    *reinterpret_cast<uint32_t*>(codes + q4_code_row(i, 32 + 4 * j)) = word[1];
    const int g = (j >> 1) + 4 * (j & 1);  // one of the pair's two groups each
    block[is_v ? q4_v_scale(i, g) : q4_k_scale(i, g)] = (uint8_t)(j & 1 ? scale[1] : scale[0]);
}

// The sum of two floats and its rounding error, exactly.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e)
{
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// The RoPE partner of every element of the head, for a rotation of rot < 128 dims
// (rot a multiple of 32): dims d and d + rot/2 lie in blocks of 8 dims rot/16 apart.
// Also the block's table entries, and the sign of the partner's term; sgn 0: not rotated.
struct RopeBlock {
    int src, hi;   // the partner's lane of 8, and whether it is there among elements 8-15
    int f0;        // first table entry
    float sgn;
};
__device__ __forceinline__ RopeBlock rope_block(int block, int rot)
{
    const int half = rot / 16;
    RopeBlock r;
    const bool first = block < half;
    const int partner = block < 2 * half ? (first ? block + half : block - half) : block;
    r.src = partner & 7;
    r.hi = partner >> 3;
    r.f0 = block < 2 * half ? 8 * (first ? block : block - half) : 0;
    r.sgn = block < 2 * half ? (first ? -1.f : 1.f) : 0.f;
    return r;
}
__device__ __forceinline__ void rope_partners(const float (&u)[16], const RopeBlock (&rb)[2], int lane, float (&up)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int src = (lane & 24) | rb[h].src;
            const float lo = __shfl_sync(kFull, u[k], src), hi = __shfl_sync(kFull, u[8 + k], src);
            up[8 * h + k] = rb[h].sgn * (rb[h].hi ? hi : lo);
        }
}

// Eight (cos, sin) entries of a table row.
__device__ __forceinline__ void load_rope8(const float2* row, float2 (&t)[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 a = reinterpret_cast<const float4*>(row)[k];
        t[2 * k] = make_float2(a.x, a.y);
        t[2 * k + 1] = make_float2(a.z, a.w);
    }
}

// u cos + up sin as a pair of floats, exact to about 2^-47 of `grid` (up: the partner with
// its sign).  Added to `grid`, a power of two 8 times any such sum or more, both
// products are rounded to its ulp; the additions are exact to take apart again, and
// what the rounding left of each product is one fma.  cos and sin with their low parts.
__device__ __forceinline__ void rotate_paired(float u, float up, float2 hi, float2 lo, float grid, float& a, float& al)
{
    const float s1 = __fmaf_rn(u, hi.x, grid), s2 = __fmaf_rn(up, hi.y, s1);
    const float e1 = __fmaf_rn(u, hi.x, -__fsub_rn(s1, grid)), e2 = __fmaf_rn(up, hi.y, -__fsub_rn(s2, s1));
    a = __fsub_rn(s2, grid);
    al = __fadd_rn(__fmaf_rn(u, lo.x, e1), __fmaf_rn(up, lo.y, e2));
}

// 2^e as a float, e kept within [lo, hi].
__device__ __forceinline__ float pow2_clamped(int e, int lo, int hi)
{
    return __uint_as_float((uint32_t)(127 + min(max(e, lo), hi)) << 23);
}

// The bf16 values of the lanes' k head (kraw) after QK-norm + RoPE, as words of two
// (out) and in fp32 (x): the fp32 nearest to the exact value, but for errors of about
// 2^-36, rounded to bf16.  A bf16 that rounds the other way can move a code by a whole
// step, a third of its value, so k is carried here in pairs of floats (hi + lo) to that
// rounding.
//   k = a inv,  a = u cos -/+ u' sin,  u = x w (exact),  inv = 1 / sqrt(mean(x^2) + eps)
// The sum of squares: x^2 is exact in 32 bits; added to a power of two above the
// lane's sum, each addition's rounding error is exact by one fma.  One Newton step
// takes rsqrtf's inv to 2^-43; cos and sin come as hi + lo of the double values, |cos|
// and |sin| at most 2^rope_exp.
template <bool kFullRot>
__device__ __forceinline__ void norm_rope_k_paired(const uint4 (&kraw)[2], const uint4 (&w)[2], const float2* rhi,
                                                   const float2* rlo, float2 eps, int rope_exp, int lane, int rot,
                                                   float (&x)[16], uint32_t (&out)[8])
{
    const int j = lane & 7;
    unpack16(kraw[0], kraw[1], x);
    // 2^ex <= the lane's largest |x| < 2^(ex + 1), and the same of the weights
    int ex = (int)(max(max8_bits(kraw[0].x, kraw[0].y, kraw[0].z, kraw[0].w),
                       max8_bits(kraw[1].x, kraw[1].y, kraw[1].z, kraw[1].w)) >> 7) - 127;
    int ew = (int)(max(max8_bits(w[0].x, w[0].y, w[0].z, w[0].w), max8_bits(w[1].x, w[1].y, w[1].z, w[1].w)) >> 7) - 127;
    const float base = pow2_clamped(2 * ex + 6, -100, 126);  // above 16 (2^(ex + 1))^2
    float ss = base, sc = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float s = __fmaf_rn(x[k], x[k], ss);
        sc = __fadd_rn(sc, __fmaf_rn(x[k], x[k], -__fsub_rn(s, ss)));
        ss = s;
    }
    ss = __fsub_rn(ss, base);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float so = __shfl_xor_sync(kFull, ss, o), co = __shfl_xor_sync(kFull, sc, o);
        float e;
        two_sum(ss, so, ss, e);
        sc = __fadd_rn(__fadd_rn(sc, co), e);
    }
    float h, l, e;
    two_sum(__fmul_rn(ss, 1.f / kHeadDim), eps.x, h, e);
    l = __fadd_rn(__fmul_rn(sc, 1.f / kHeadDim), __fadd_rn(e, eps.y));
    two_sum(h, l, h, l);
    const float y = rsqrtf(h);
    const float p = __fmul_rn(y, y), pe = __fmaf_rn(y, y, -p);
    // r = 1 - (h + l) y^2, then inv = y (1 + r/2 + 3 r^2 / 8)
    const float r = __fmaf_rn(-l, p, __fmaf_rn(-h, pe, __fmaf_rn(-h, p, 1.f)));
    const float yl = __fmul_rn(y, __fmaf_rn(__fmul_rn(0.375f, r), r, __fmul_rn(0.5f, r)));
    // (a + al) (y + yl), rounded once
    auto finish = [&](float a, float al) { return __fmaf_rn(a, y, __fmaf_rn(a, yl, __fmul_rn(al, y))); };
    float u[16];
    {
        float wk[16];
        unpack16(w[0], w[1], wk);
#pragma unroll
        for (int k = 0; k < 16; ++k) u[k] = __fmul_rn(x[k], wk[k]);
    }
    if constexpr (kFullRot) {
        // |u| < 2^(ex + ew + 2), a sum of two terms < 2^(ex + ew + 3 + rope_exp)
        const float grid = pow2_clamped(ex + ew + 6 + rope_exp, -100, 126);
        float2 ch[8], cl[8];
        load_rope8(rhi + 8 * j, ch);
        load_rope8(rlo + 8 * j, cl);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, al;
            rotate_paired(u[k], -u[8 + k], ch[k], cl[k], grid, a, al);
            x[k] = finish(a, al);
            rotate_paired(u[8 + k], u[k], ch[k], cl[k], grid, a, al);
            x[8 + k] = finish(a, al);
        }
    } else {
        // the partners lie in other lanes: the head's largest
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            ex = max(ex, __shfl_xor_sync(kFull, ex, o));
            ew = max(ew, __shfl_xor_sync(kFull, ew, o));
        }
        const float grid = pow2_clamped(ex + ew + 6 + rope_exp, -100, 126);
        const RopeBlock rb[2] = {rope_block(j, rot), rope_block(8 + j, rot)};
        float up[16];
        rope_partners(u, rb, lane, up);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float2 ch[8], cl[8];
            load_rope8(rhi + rb[b].f0, ch);
            load_rope8(rlo + rb[b].f0, cl);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float a = u[8 * b + k], al = 0.f;
                if (rb[b].sgn != 0.f) rotate_paired(u[8 * b + k], up[8 * b + k], ch[k], cl[k], grid, a, al);
                x[8 * b + k] = finish(a, al);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        out[k] = *reinterpret_cast<const uint32_t*>(&b2);
        x[2 * k] = __uint_as_float(out[k] << 16);
        x[2 * k + 1] = __uint_as_float(out[k] & 0xffff0000u);
    }
}

// The lanes' q head after QK-norm + RoPE, in fp32 (cos and sin the nearest fp32).
template <bool kFullRot>
__device__ __forceinline__ void norm_rope_q16(const float (&x)[16], const uint4 (&w)[2], const float2* rhi, float eps,
                                              int lane, int rot, float (&out)[16])
{
    const int j = lane & 7;
    float wq[16], u[16], ss = 0.f;
    unpack16(w[0], w[1], wq);
#pragma unroll
    for (int k = 0; k < 16; ++k) ss = __fmaf_rn(x[k], x[k], ss);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float inv = rsqrtf(__fmaf_rn(ss, 1.0f / kHeadDim, eps));
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = x[k] * wq[k];
    if constexpr (kFullRot) {
        float2 ch[8];
        load_rope8(rhi + 8 * j, ch);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            out[k] = inv * (u[k] * ch[k].x - u[8 + k] * ch[k].y);
            out[8 + k] = inv * (u[8 + k] * ch[k].x + u[k] * ch[k].y);
        }
    } else {
        const RopeBlock rb[2] = {rope_block(j, rot), rope_block(8 + j, rot)};
        float up[16];
        rope_partners(u, rb, lane, up);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float2 ch[8];
            load_rope8(rhi + rb[b].f0, ch);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float v = u[8 * b + k];
                out[8 * b + k] = inv * (rb[b].sgn != 0.f ? v * ch[k].x + up[8 * b + k] * ch[k].y : v);
            }
        }
    }
}

}  // namespace pkv
