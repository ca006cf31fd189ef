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

// Quantises a warp's head vector, 4 dims a lane (x: bf16 values in fp32), and
// stores it at position i of `block`.  s is a power of two.
//   scale = e4m3(max |x| / (6 s)), codes = e2m1(x / (scale s)), both to nearest, ties to even.
// Every quotient here has few enough bits for its ties to be told exactly: x has 8
// significant bits and a tie of the scale (5 bits) or of a code (3 bits times a
// scale of 4) times 6 at most 7, so a quotient that is not a tie is off it by more
// than 2^-10 of its value.  x * (1 / (scale s)), off by 2^-23 at most, is rounded to
// 20 bits, which puts the ties back in place.  A group that holds an Inf or a NaN
// gets the scale NaN: the positions that read it are NaN, as with a bf16 pool.
__device__ __forceinline__ void q4_store(uint8_t* block, bool is_v, int i, const float (&x)[4], float s, int lane)
{
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);  // orders Inf and NaN above
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    uint32_t scale;
    float r;
    if (top >= 0x7f800000u) {
        scale = 0x7fu;
        r = 0.f;
    } else {
        uint16_t sc;
        const float want = __fdiv_rn(__uint_as_float(top), 6.f * s);
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(sc) : "f"(want));
        scale = sc & 0xffu;
        const uint32_t h2 = e4m3x2_half2(scale);
        const float step = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu))) * s;
        r = step > 0.f ? __frcp_rn(step) : 0.f;
    }
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __uint_as_float((__float_as_uint(x[k] * r) + 8u) & ~15u);
    uint32_t codes;
    asm("{\n\t.reg .b8 b0, b1;\n\t.reg .b16 h;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "mov.b16 h, {b0, b1};\n\tcvt.u32.u16 %0, h;\n\t}"
        : "=r"(codes)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
    *reinterpret_cast<uint16_t*>(block + (is_v ? kQ4VCodes : 0) + q4_code_row(i, 2 * lane)) = (uint16_t)codes;
    if ((lane & 3) == 0) {
        const int g = lane >> 2;
        block[is_v ? q4_v_scale(i, g) : q4_k_scale(i, g)] = (uint8_t)scale;
    }
}

// The sum of two floats and its rounding error, exactly.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e)
{
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// The bf16 values of the warp's k after QK-norm + RoPE (4 dims a lane), correctly
// rounded but for errors of about 2^-43: a bf16 that rounds the other way can
// move a code by a whole step, a third of its value, so k is carried here in
// pairs of floats (hi + lo) to the rounding.
//   k = a inv,  a = u cos -/+ u' sin,  u = x w (exact),  inv = 1 / sqrt(mean(x^2) + eps)
// The squares are exact (bf16 inputs), their sum keeps its errors, one Newton
// step from rsqrtf gives inv to 2^-43; cos and sin come as hi + lo of the double values.
__device__ __forceinline__ void norm_rope_k_paired(uint2 kraw, const float (&wk)[4], const float2 (&rh)[4],
                                                   const float2 (&rl)[4], float2 eps, int lane, int rot, float (&out)[4])
{
    float x[4];
    unpack4(kraw, x);
    float ss = 0.f, sc = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float e;
        two_sum(ss, __fmul_rn(x[k], x[k]), ss, e);
        sc = __fadd_rn(sc, e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
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
    // 1 - (h + l) y^2, then inv = y (1 + r/2 + 3 r^2 / 8)
    const float r = __fmaf_rn(-l, p, __fmaf_rn(-h, pe, __fmaf_rn(-h, p, 1.f)));
    const float yl = __fmul_rn(y, __fmaf_rn(__fmul_rn(0.375f, r), r, __fmul_rn(0.5f, r)));
    const KRope kr = krope(lane, rot);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float u = __fmul_rn(x[k], wk[k]);
        const float up = kr.sgn * __shfl_sync(kFull, u, kr.src);
        float a = u, al = 0.f;
        if (kr.rot) {
            const float p1 = __fmul_rn(u, rh[k].x), e1 = __fmaf_rn(u, rh[k].x, -p1);
            const float p2 = __fmul_rn(up, rh[k].y), e2 = __fmaf_rn(up, rh[k].y, -p2);
            float e3;
            two_sum(p1, p2, a, e3);
            al = __fmaf_rn(u, rl[k].x, __fmaf_rn(up, rl[k].y, __fadd_rn(__fadd_rn(e1, e2), e3)));
        }
        const float q = __fmul_rn(a, y), qe = __fmaf_rn(a, y, -q);
        const float lo = __fmaf_rn(a, yl, __fmaf_rn(al, y, qe));
        const float hi = __fadd_rn(q, lo), rest = __fsub_rn(lo, __fsub_rn(hi, q));
        // round hi + rest to odd in fp32, so that the one rounding to bf16 below sees which side of a tie it is on
        uint32_t bits = __float_as_uint(hi);
        if (rest != 0.f && !(bits & 1u)) bits += ((rest > 0.f) == (hi > 0.f)) ? 1u : ~0u;
        out[k] = __bfloat162float(__float2bfloat16_rn(__uint_as_float(bits)));
    }
}

}  // namespace pkv
