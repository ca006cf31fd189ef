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
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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

// x rounded to 20 significant bits.
__device__ __forceinline__ float snap20(float x) { return __uint_as_float((__float_as_uint(x) + 8u) & ~15u); }

// Quantises the head vector (x: bf16 values in fp32) to position i of `block`.
// s is a power of two.
//   scale = e4m3(max |x| / (6 s)), codes = e2m1(x / (scale s)), both to nearest, ties to even.
// Every quotient here has few enough bits for its ties to be told exactly: x has 8
// significant bits, and a tie of a scale (5 bits) times 6 or of a code (3 bits) times
// a scale (4 bits) at most 7, so a quotient that is not a tie is off it by more than
// 2^-10 of its value.  The products with rounded inverses, off by 2^-23 at most, are
// rounded to 20 bits, which puts the ties back in place.  A group that holds an Inf or
// a NaN gets the scale NaN: the positions that read it are NaN, as with a bf16 pool.
//   inv6s = 1 / (6 s) to nearest, inv_s = 1 / s
__device__ __forceinline__ void q4_store(uint8_t* block, bool is_v, int i, const float (&x)[16], float inv6s,
                                         float inv_s, int j, bool live)
{
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 16; ++k) top[k >> 3] = max(top[k >> 3], __float_as_uint(x[k]) & 0x7fffffffu);  // Inf, NaN on top
    uint32_t word[2], scale[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        top[h] = max(top[h], __shfl_xor_sync(kFull, top[h], 1));
        uint16_t sc;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(sc) : "f"(snap20(__uint_as_float(top[h]) * inv6s)));
        scale[h] = top[h] >= 0x7f800000u ? 0x7fu : sc & 0xffu;
        const float step = __half2float(__ushort_as_half((unsigned short)(e4m3x2_half2(scale[h]) & 0xffffu)));
        const float r = step > 0.f ? __frcp_rn(step) * inv_s : 0.f;  // (NaN: 0, any code will do)
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = snap20(x[8 * h + k] * r);
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

// u cos + up sin as a pair of floats (up: the partner with its sign): the products'
// errors by fma, the sum's by two_sum, cos and sin with their low parts.
__device__ __forceinline__ void rotate_paired(float u, float up, float2 hi, float2 lo, float& a, float& al)
{
    const float p1 = __fmul_rn(u, hi.x), e1 = __fmaf_rn(u, hi.x, -p1);
    const float p2 = __fmul_rn(up, hi.y), e2 = __fmaf_rn(up, hi.y, -p2);
    float e3;
    two_sum(p1, p2, a, e3);
    al = __fmaf_rn(u, lo.x, __fmaf_rn(up, lo.y, __fadd_rn(__fadd_rn(e1, e2), e3)));
}

// The bf16 values (in fp32) of the lanes' k head after QK-norm + RoPE: the fp32
// nearest to the exact value, but for errors of about 2^-37, rounded to bf16.  A
// bf16 that rounds the other way can move a code by a whole step, a third of its
// value, so k is carried here in pairs of floats (hi + lo) to that rounding.
//   k = a inv,  a = u cos -/+ u' sin,  u = x w (exact),  inv = 1 / sqrt(mean(x^2) + eps)
// The sum of squares: x^2 is exact in 32 bits; added to a power of two above the
// lane's sum, each addition's rounding error is exact by one fma.  One Newton step
// takes rsqrtf's inv to 2^-43; cos and sin come as hi + lo of the double values.
//   row: lane's table entries (full rotation: 8j .. 8j + 7 of both tables);
//   rot < 128: tables rhi, rlo of the position.
template <bool kFullRot>
__device__ __forceinline__ void norm_rope_k_paired(const float (&x)[16], const uint4 (&w)[2], const float2* rhi,
                                                   const float2* rlo, float2 eps, int lane, int rot, float (&out)[16])
{
    const int j = lane & 7;
    float wk[16];
    unpack16(w[0], w[1], wk);
    float big = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) big = fmaxf(big, fabsf(x[k]));
    // 2^(2e + 6) > 16 big^2 for big < 2^(e + 1)
    const int ex = min(max((int)(__float_as_uint(big) >> 23) - 127, -60), 60);
    const float base = __uint_as_float((uint32_t)(127 + 2 * ex + 6) << 23);
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
    auto finish = [&](float a, float al) {  // (a + al) (y + yl)
        const float q = __fmul_rn(a, y), qe = __fmaf_rn(a, y, -q);
        return __bfloat162float(__float2bfloat16_rn(__fadd_rn(q, __fmaf_rn(a, yl, __fmaf_rn(al, y, qe)))));
    };
    float u[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = __fmul_rn(x[k], wk[k]);
    if constexpr (kFullRot) {
        float2 ch[8], cl[8];
        load_rope8(rhi + 8 * j, ch);
        load_rope8(rlo + 8 * j, cl);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, al;
            rotate_paired(u[k], -u[8 + k], ch[k], cl[k], a, al);
            out[k] = finish(a, al);
            rotate_paired(u[8 + k], u[k], ch[k], cl[k], a, al);
            out[8 + k] = finish(a, al);
        }
    } else {
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
                if (rb[b].sgn != 0.f) rotate_paired(u[8 * b + k], up[8 * b + k], ch[k], cl[k], a, al);
                out[8 * b + k] = finish(a, al);
            }
        }
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
