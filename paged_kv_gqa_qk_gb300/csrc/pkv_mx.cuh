// Microscaled tensors: groups of 32 consecutive values of a row held as code * 2^e
// (OCP Microscaling Formats (MX) Specification v1.0: elements e4m3 or e2m1, scales e8m0).
//
//   e = the least whole number >= -127 with max |x| <= top * 2^e   (top 448 or 6)
//   code = x / 2^e rounded to nearest, ties to even
// so that no finite value saturates.  A group holding an Inf or a NaN has scale byte 255
// (NaN) and codes 0.
//
// Scale bytes (e + 127) lie in tiles of 128 rows by 4 groups, the order in which the tensor
// cores take them from shared memory: 512 bytes, byte 16 (r % 32) + 4 (r / 32) + g.
#pragma once

#include <stdint.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kMxGroup = 32;
constexpr int kMxTileRows = 128, kMxTileCols = 128, kMxTileBytes = 512;

__host__ __device__ constexpr int mx_row_bytes(int type, int cols) { return type == PKV_MX8 ? cols : cols / 2; }

// The scale byte of a group whose largest magnitude has the fp32 bits `top` (integers
// order as magnitudes do, an Inf or a NaN above all numbers).  The addend carries into the
// exponent where the mantissa is beyond 1.75 (448 = 1.75 * 2^8) or 1.5 (6 = 1.5 * 2^2).
template <int kType>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top)
{
    constexpr uint32_t beyond = kType == PKV_MX8 ? 0x7fffffu - 0x600000u : 0x7fffffu - 0x400000u;
    constexpr int emax = kType == PKV_MX8 ? 8 : 2;
    const int e = (int)((top + beyond) >> 23) - emax;
    return top >= 0x7f800000u ? 255u : (uint32_t)(e > 0 ? e : 0);
}

// 2^-e of a scale byte (255: any number, its codes are 0).
__device__ __forceinline__ float mx_inverse(uint32_t byte)
{
    return __uint_as_float((byte == 255u ? 127u : 254u - byte) << 23);
}

// Codes of 8 scaled values: 8 bytes, or 4 (in .x).
template <int kType>
__device__ __forceinline__ uint2 mx_codes8(const float (&y)[8])
{
    uint2 r = make_uint2(0, 0);
    if constexpr (kType == PKV_MX8) {
        asm("{\n\t.reg .b16 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\tcvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
            "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}"
            : "=r"(r.x), "=r"(r.y)
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(r.x)
            : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    }
    return r;
}

// The values of 8 codes (exact in fp16, hence in fp32).
template <int kType>
__device__ __forceinline__ void mx_decode8(uint2 c, float (&y)[8])
{
    uint32_t h[4];
    if constexpr (kType == PKV_MX8) {
        asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(c.x), "r"(c.y));
    } else {
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(c.x));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(y[2 * i]), "=f"(y[2 * i + 1])
            : "r"(h[i]));
}

// Where the scale of (row, group) lies; `tiles` = cols / 128.
__device__ __forceinline__ int64_t mx_scale_at(int64_t row, int group, int tiles)
{
    const int r = (int)(row % kMxTileRows);
    return ((row / kMxTileRows) * tiles + group / 4) * kMxTileBytes + 16 * (r % 32) + 4 * (r / 32) + group % 4;
}

__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8])
{
    const uint32_t a[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(a[i] << 16);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(a[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(a[0], a[1], a[2], a[3]);
}

}  // namespace pkv
