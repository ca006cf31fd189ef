// Microscaled tensors written and read (pkv_mx_quantize, pkv_mx_read), and the residual's
// addition with the layer's RMS norm, to bf16 or to a microscaled tensor (pkv_add_norm).
//
//   h = bf16(x + residual),   y = h / sqrt(mean(h^2) + eps) * w
//
// qwen3-8b Nest files, src/norm.linnet (RmsNorm) and DecoderLayer.decode_paged, which runs
// attention_norm before the attention and the residual's addition with mlp_norm after it.
#include <algorithm>
#include <type_traits>

#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---- bf16 -> microscaled ----
// 8 lanes take 128 columns of a row, 16 each; a group of 32 is 2 lanes.
template <int kType, int kPasses>
__global__ void __launch_bounds__(256)
    mx_quantize_kernel(const __nv_bfloat16* x, int64_t x_stride, int rows, int cols, uint8_t* codes,
                       uint8_t* scales)
{
    const int tiles = cols / kMxTileCols, tile = blockIdx.x % tiles, step = blockDim.x >> 3;
    const int64_t row0 = (int64_t)(blockIdx.x / tiles) * (step * kPasses);
    const int sub = threadIdx.x >> 3, j = threadIdx.x & 7;
    const int col = tile * kMxTileCols + 16 * j;
    pdl_wait();
    uint4 raw[kPasses][2];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + step * i + sub;
        const uint4* const from = reinterpret_cast<const uint4*>(x + r * x_stride + col);
#pragma unroll
        for (int k = 0; k < 2; ++k) raw[i][k] = r < rows ? from[k] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + step * i + sub;
        // the largest magnitude of the group, as 16-bit integers (a NaN above an Inf above all numbers)
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            two = __vmaxu2(two, __vmaxu2(__vmaxu2(raw[i][k].x & 0x7fff7fffu, raw[i][k].y & 0x7fff7fffu),
                                         __vmaxu2(raw[i][k].z & 0x7fff7fffu, raw[i][k].w & 0x7fff7fffu)));
        two = __vmaxu2(two, __shfl_xor_sync(kAll, two, 1));
        const uint32_t top = max(two << 16, two & 0xffff0000u);
        const uint32_t byte = mx_scale_byte<kType>(top);
        const float inv = mx_inverse(byte);
        uint2 c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float v[8];
            unpack8(raw[i][k], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= inv;
            c[k] = mx_codes8<kType>(v);
            if (byte == 255u) c[k] = make_uint2(0, 0);
        }
        if (r >= rows) continue;
        uint8_t* dst = codes + r * mx_row_bytes(kType, cols) + mx_row_bytes(kType, col);
        if constexpr (kType == PKV_MX8)
            *reinterpret_cast<uint4*>(dst) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
        else
            *reinterpret_cast<uint2*>(dst) = make_uint2(c[0].x, c[1].x);
        if ((j & 1) == 0) scales[mx_scale_at(r, 4 * tile + (j >> 1), tiles)] = (uint8_t)byte;
    }
}

// ---- microscaled -> bf16 ----
template <int kType, int kPasses>
__global__ void __launch_bounds__(256)
    mx_read_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int cols,
                   __nv_bfloat16* y, int64_t y_stride)
{
    const int tiles = cols / kMxTileCols, tile = blockIdx.x % tiles;
    const int64_t row0 = (int64_t)(blockIdx.x / tiles) * (16 * kPasses);
    const int sub = threadIdx.x >> 4, j = threadIdx.x & 15;
    const int col = tile * kMxTileCols + 8 * j;
    pdl_wait();
    uint2 raw[kPasses];
    uint32_t byte[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + 16 * i + sub;
        raw[i] = make_uint2(0, 0);
        byte[i] = 0;
        if (r >= rows) continue;
        const uint8_t* src = codes + r * mx_row_bytes(kType, cols) + mx_row_bytes(kType, col);
        if constexpr (kType == PKV_MX8)
            raw[i] = *reinterpret_cast<const uint2*>(src);
        else
            raw[i].x = *reinterpret_cast<const uint32_t*>(src);
        byte[i] = scales[mx_scale_at(r, 4 * tile + (j >> 2), tiles)];
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + 16 * i + sub;
        if (r >= rows) continue;
        float v[8];
        mx_decode8<kType>(raw[i], v);
        // 2^(byte - 127): 2^-127 is subnormal, byte 255 a NaN
        const float s = __uint_as_float(byte[i] == 0 ? 0x00400000u : byte[i] == 255u ? 0x7fc00000u : byte[i] << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= s;
        *reinterpret_cast<uint4*>(y + r * y_stride + col) = pack8(v);
    }
}

// ---- pairs of floats ----
struct Pair {
    float h, l;
};

// a + b as a rounded sum and its exact error (Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const Pair s = two_sum(a.h, b.h);
    return {s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l))};
}

// The sum over a warp of pairs >= 0, in every lane, through integers: each lane's value in units of 2^-24 of what makes
// the warp's largest one 2^24 to 2^25, as two integers that add up without loss.  Beyond fp32's range or NaN: NaN.
// (A butterfly of pairs takes twice the instructions and five dependent exchanges.)
__device__ __forceinline__ Pair warp_sum(Pair a)
{
    const float h = __fadd_rn(a.h, a.l), l = __fadd_rn(a.l, __fsub_rn(a.h, h));
    const uint32_t top = __reduce_max_sync(kAll, __float_as_uint(h));
    if (top >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.f};
    const uint32_t e = max(top >> 23, 26u);                               // (units below fp32's least number do no harm)
    const float up = __uint_as_float((278u - e) << 23), down = __uint_as_float((e - 24u) << 23);  // 2^(24 - E), 2^(E - 24)
    const float x = __fmul_rn(h, up);
    const int whole = __float2int_rz(x);
    const int part = __float2int_rn(__fmul_rn(__fsub_rn(x, __int2float_rn(whole)), 0x1p24f)) +
                     __float2int_rn(__fmul_rn(__fmul_rn(l, up), 0x1p24f));
    const int w = __reduce_add_sync(kAll, whole), p = __reduce_add_sync(kAll, part);
    const float wf = __int2float_rn(w);
    const float rest = __fmaf_rn(__int2float_rn(p), 0x1p-24f, __int2float_rn(w - __float2int_rn(wf)));
    return {__fmul_rn(wf, down), __fmul_rn(rest, down)};
}

// ss * inv_n + eps.
__device__ __forceinline__ Pair mean_pair(Pair ss, Pair inv_n, Pair eps)
{
    const float t = __fmul_rn(ss.h, inv_n.h);
    const float te = __fmaf_rn(ss.h, inv_n.l, __fmaf_rn(ss.l, inv_n.h, __fmaf_rn(ss.h, inv_n.h, -t)));
    Pair v = two_sum(t, eps.h);
    v.l = __fadd_rn(v.l, __fadd_rn(te, eps.l));
    return v;
}

// 1 / sqrt(v) to about 2^-44: a fp32 root and one step of Newton's iteration, whose residual
// 1 - v r^2 is formed without loss.
__device__ __forceinline__ Pair inv_root_pair(Pair v)
{
    const float r = rsqrtf(v.h);
    const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
    const float q = __fmul_rn(v.h, p);
    const float qe = __fmaf_rn(v.l, p, __fmaf_rn(v.h, pe, __fmaf_rn(v.h, p, -q)));
    const float e = __fsub_rn(__fsub_rn(1.0f, q), qe);
    return {r, __fmul_rn(__fmul_rn(r, 0.5f), e)};
}

// 1 / sqrt(ss * inv_n + eps).
__device__ __forceinline__ Pair inv_rms_pair(Pair ss, Pair inv_n, Pair eps)
{
    // With v from 2^-80 to 2^100 every term is a normal number (r^2's error is some 2^-48 of 1 / v, which would be subnormal
    // from 2^102 on, r^2 itself infinite below 2^-128).  Otherwise the sum and eps take an even power of two, whose root goes
    // back into r.  (The look costs 1001 x 5120 to 4 bits 7.08 -> 7.18 us; a power of two that suits all rows, which eps
    // would have to bound, 7.16.)
    constexpr uint32_t kLeast = (127 - 80) << 23, kMost = (127 + 100) << 23;
    const Pair v = mean_pair(ss, inv_n, eps);
    if (__float_as_uint(v.h) - kLeast <= kMost - kLeast) return inv_root_pair(v);
    const float h = __fadd_rn(ss.h, ss.l);  // (a sum of subnormal squares may come with all of it in l)
    const int a = min(max(-(((int)(__float_as_uint(fmaxf(h, eps.h)) >> 23) - 127) & ~1), -126), 126);
    const float up = __uint_as_float((uint32_t)(a + 127) << 23), back = __uint_as_float((uint32_t)(a / 2 + 127) << 23);
    const Pair r = inv_root_pair(mean_pair({__fmul_rn(h, up), __fmul_rn(__fadd_rn(ss.l, __fsub_rn(ss.h, h)), up)}, inv_n,
                                           {__fmul_rn(eps.h, up), __fmul_rn(eps.l, up)}));
    return {__fmul_rn(r.h, back), __fmul_rn(r.l, back)};
}

struct AddNormParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* residual;
    __nv_bfloat16* residual_out;
    const __nv_bfloat16* w;
    void* out;
    uint8_t* scales;
    int64_t x_stride;
    int tokens, hidden;
    Pair inv_n, eps;
};

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma_rz(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// a * b + c for two bf16 each of a and b (as fast as two of fp32, without their conversions)
__device__ __forceinline__ uint64_t f2_fma_bf16(uint32_t a, uint32_t b, uint64_t c)
{
    float c0, c1, d0, d1;
    f2_unpack(c, c0, c1);
    asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\tmov.b32 {a0, a1}, %2;\n\tmov.b32 {b0, b1}, %3;\n\t"
        "fma.rn.f32.bf16 %0, a0, b0, %4;\n\tfma.rn.f32.bf16 %1, a1, b1, %5;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "r"(a), "r"(b), "f"(c0), "f"(c1));
    return f2_pack(d0, d1);
}
// two sums of bf16, each rounded once
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the larger magnitude, a NaN if either is one
__device__ __forceinline__ float max_abs(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// hw * r for two elements, truncated, the last bit set where something was cut off: what a rounding
// of it to fewer bits gives is then the rounding of the exact value (but for 2^-44 of it).  Nothing
// is cut off only where r is a float (kExact: its rest beyond 2^-70 of it, looked at for a row) and the product
// fits one; with the rest of r at least the products are never floats.
template <bool kExact>
__device__ __forceinline__ void scaled_odd(uint64_t hw, uint64_t rh, uint64_t rl, float& a, float& b)
{
    const uint64_t p = f2_fma_rz(hw, rh, f2_mul(hw, rl));
    f2_unpack(p, a, b);
    uint32_t cut_a = 1u, cut_b = 1u;
    if constexpr (kExact) {
        float ea, eb;
        const uint64_t minus = f2_pack(-a, -b);
        f2_unpack(f2_fma(hw, rh, minus), ea, eb);
        cut_a = ea != 0.f, cut_b = eb != 0.f;
    }
    a = __uint_as_float(__float_as_uint(a) | cut_a);
    b = __uint_as_float(__float_as_uint(b) | cut_b);
}

// A CTA takes tokens blockIdx.x, + gridDim.x, ...; its thread i holds chunks i, i + T, ... of 8 columns of each.
// Every warp forms the sum of the warps' sums and the root by itself, with one barrier a token.
//
// Bound by memory where a residual is added: 8192 x 4096 to 8 bits, 236 MB, in 37.1 us, 6.4 TB/s, to 4, 219 MB, in 35.2, to
// bf16, 268 MB, in 41.7; without one by instructions, some 23 an element with a token's share of the sums (to 4 bits, 85 MB,
// in 28.7 us, to 8, 102 MB, in 29.0, to bf16, 134 MB, in 25.2; 1001 x 5120 to 4 bits in 7.2, in three turns of the CTAs that
// fit).  Four chunks and a residual do not fit 64 registers a thread: 56 bytes of each are spilled above 16384 columns (2048 x
// 20480 to 8 bits, 295 MB, 58.8 us, 5.0 TB/s).
template <int kType, bool kAdd, int kChunks>
__global__ void __launch_bounds__(1024) add_norm_kernel(AddNormParams p)
{
    __shared__ Pair part[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
    const int chunks = p.hidden / 8;
    // Pairs of chunks beside each other where none of bf16 is written: a group of 32 is two lanes then, not four (8192 x
    // 4096 to 4 bits 30 -> 28 us).  Stores of 16 bytes 32 apart would cost more than that.
    constexpr bool kNear = !kAdd && kType != PKV_BF16 && kChunks > 1;
    auto chunk = [&](int c) { return kNear ? 2 * (tid + c / 2 * T) + c % 2 : tid + c * T; };
    constexpr int kCodes = kType == PKV_BF16 ? 16 : mx_row_bytes(kType, 8);  // bytes of a chunk in out
    pdl_wait();
    pdl_launch_dependents();
    uint4 x[kChunks], more[kChunks], w[kChunks];
    auto load = [&](int t) {
        const uint4* const from = reinterpret_cast<const uint4*>(p.x + t * p.x_stride) + chunk(0);
        const uint4* const add = reinterpret_cast<const uint4*>(p.residual + (int64_t)t * p.hidden) + chunk(0);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (chunk(c) >= chunks) continue;
            x[c] = from[chunk(c) - chunk(0)];
            if (kAdd) more[c] = add[c * T];
        }
    };
#pragma unroll
    for (int c = 0; c < kChunks; ++c) x[c] = more[c] = w[c] = make_uint4(0, 0, 0, 0);
    load((int)blockIdx.x);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
        if (chunk(c) < chunks) w[c] = *reinterpret_cast<const uint4*>(p.w + 8 * chunk(c));
    int turn = 0;
    for (int t = blockIdx.x; t < p.tokens; t += gridDim.x, turn ^= 1) {
        uint32_t h[kChunks][4];
        uint4* const h_out = reinterpret_cast<uint4*>(p.residual_out + (int64_t)t * p.hidden) + tid;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            h[c][0] = x[c].x, h[c][1] = x[c].y, h[c][2] = x[c].z, h[c][3] = x[c].w;
            if constexpr (kAdd) {
                h[c][0] = add_bf16x2(h[c][0], more[c].x), h[c][1] = add_bf16x2(h[c][1], more[c].y);
                h[c][2] = add_bf16x2(h[c][2], more[c].z), h[c][3] = add_bf16x2(h[c][3], more[c].w);
                if (tid + c * T < chunks) h_out[c * T] = make_uint4(h[c][0], h[c][1], h[c][2], h[c][3]);
            }
        }
        if (t + (int)gridDim.x < p.tokens) load(t + (int)gridDim.x);
        // squares (exact) added up with what each addition loses
        const uint64_t minus_one = f2_pack(-1.f, -1.f);
        uint64_t s2 = 0, l2 = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint64_t sum = f2_fma_bf16(h[c][k], h[c][k], s2);
                const uint64_t back = f2_fma(sum, minus_one, s2);             // minus the part of h^2 that went in
                const uint64_t lost = f2_add(f2_fma(f2_add(sum, back), minus_one, s2), f2_fma_bf16(h[c][k], h[c][k], back));
                l2 = f2_add(l2, lost);
                s2 = sum;
            }
        Pair ss, other;
        f2_unpack(s2, ss.h, other.h);
        f2_unpack(l2, ss.l, other.l);
        ss = add(ss, other);
        ss = warp_sum(ss);
        if (warps > 1) {
            if (lane == 0) part[turn][warp] = ss;
            __syncthreads();
            ss = warp_sum(lane < warps ? part[turn][lane] : Pair{0.f, 0.f});
        }
        const Pair r = inv_rms_pair(ss, p.inv_n, p.eps);
        const uint64_t rh = f2_pack(r.h, r.h), rl = f2_pack(r.l, r.l);
        const bool exact = fabsf(r.l) <= r.h * 0x1p-70f;
        uint8_t* const dst = static_cast<uint8_t*>(p.out) + t * (int64_t)(chunks * kCodes) + chunk(0) * kCodes;
        uint8_t* const scale = p.scales + mx_scale_at(t, chunk(0) / 4, p.hidden / kMxTileCols);
        auto scaled = [&](int c, float (&v)[8]) {
            const uint32_t wc[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            uint64_t hw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) hw[k] = f2_fma_bf16(h[c][k], wc[k], f2_pack(-0.f, -0.f));  // (exact)
            if (exact) {
#pragma unroll
                for (int k = 0; k < 4; ++k) scaled_odd<true>(hw[k], rh, rl, v[2 * k], v[2 * k + 1]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) scaled_odd<false>(hw[k], rh, rl, v[2 * k], v[2 * k + 1]);
            }
        };
        // (chunk c lies c T chunks, or T / 16 tiles of scales, further along)
        if constexpr (kType == PKV_BF16) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                float v[8];
                scaled(c, v);
                if (chunk(c) < chunks) *reinterpret_cast<uint4*>(dst + c * T * kCodes) = pack8(v);
            }
        } else {
            constexpr int kSet = kNear ? 2 : 1;  // chunks of a set, 16 or 8 columns that lie together
#pragma unroll
            for (int c = 0; c < kChunks; c += kSet) {
                float v[kSet][8];
                uint32_t top = 0;
#pragma unroll
                for (int s = 0; s < kSet; ++s) {
                    scaled(c + s, v[s]);
                    top = max(top, __float_as_uint(max_abs(max_abs(max_abs(v[s][0], v[s][1]), max_abs(v[s][2], v[s][3])),
                                                           max_abs(max_abs(v[s][4], v[s][5]), max_abs(v[s][6], v[s][7])))) &
                                       0x7fffffffu);
                }
                top = max(top, __shfl_xor_sync(kAll, top, 1));
                if (kSet == 1) top = max(top, __shfl_xor_sync(kAll, top, 2));
                const uint32_t byte = mx_scale_byte<kType>(top);
                const float inv = mx_inverse(byte);
                const uint64_t inv2 = f2_pack(inv, inv);
                uint2 code[kSet];
#pragma unroll
                for (int s = 0; s < kSet; ++s) {
#pragma unroll
                    for (int k = 0; k < 8; k += 2) f2_unpack(f2_mul(f2_pack(v[s][k], v[s][k + 1]), inv2), v[s][k], v[s][k + 1]);
                    code[s] = mx_codes8<kType>(v[s]);
                    if (byte == 255u) code[s] = make_uint2(0, 0);
                }
                if (chunk(c) >= chunks) continue;
                uint8_t* const to = dst + (chunk(c) - chunk(0)) * kCodes;
                if constexpr (kNear && kType == PKV_MX8)
                    *reinterpret_cast<uint4*>(to) = make_uint4(code[0].x, code[0].y, code[kSet - 1].x, code[kSet - 1].y);
                else if constexpr (kNear)
                    *reinterpret_cast<uint2*>(to) = make_uint2(code[0].x, code[kSet - 1].x);
                else if constexpr (kType == PKV_MX8)
                    *reinterpret_cast<uint2*>(to) = code[0];
                else
                    *reinterpret_cast<uint32_t*>(to) = code[0].x;
                if ((lane & (4 / kSet - 1)) == 0) scale[(chunk(c) - chunk(0)) / 16 * kMxTileBytes] = (uint8_t)byte;
            }
        }
    }
}

cudaLaunchConfig_t config(unsigned grid, unsigned block, cudaLaunchAttribute* attr, cudaStream_t s)
{
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

Pair pair_of(double x)
{
    const float h = (float)x;
    return {h, (float)(x - (double)h)};
}

}  // namespace

cudaError_t launch_mx_quantize(const pkv_pool* pool, const void* x, int64_t x_stride, int rows, int cols, int type,
                               void* codes, void* scales, cudaStream_t s)
{
    const int tiles = cols / kMxTileCols;
    const bool many = (int64_t)(rows + 127) / 128 * tiles >= 2 * pool->num_sms;
    const int step = many ? 64 : 16, threads = many ? 256 : 128;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((rows + step - 1) / step * tiles), threads, attr, s);
    auto launch = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const __nv_bfloat16*>(x), x_stride, rows, cols,
                                  static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    };
    if (type == PKV_MX8) return many ? launch(mx_quantize_kernel<PKV_MX8, 2>) : launch(mx_quantize_kernel<PKV_MX8, 1>);
    return many ? launch(mx_quantize_kernel<PKV_MX4, 2>) : launch(mx_quantize_kernel<PKV_MX4, 1>);
}

cudaError_t launch_mx_read(const pkv_pool* pool, int type, const void* codes, const void* scales, int rows, int cols,
                           void* y, int64_t y_stride, cudaStream_t s)
{
    const int tiles = cols / kMxTileCols;
    const bool many = (int64_t)(rows + 127) / 128 * tiles >= 2 * pool->num_sms;
    const int step = many ? 64 : 16;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((rows + step - 1) / step * tiles), 256, attr, s);
    auto launch = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                  rows, cols, static_cast<__nv_bfloat16*>(y), y_stride);
    };
    if (type == PKV_MX8) return many ? launch(mx_read_kernel<PKV_MX8, 4>) : launch(mx_read_kernel<PKV_MX8, 1>);
    return many ? launch(mx_read_kernel<PKV_MX4, 4>) : launch(mx_read_kernel<PKV_MX4, 1>);
}

cudaError_t launch_add_norm(const pkv_pool* pool, const AddNorm& a, cudaStream_t s)
{
    AddNormParams p;
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.residual = static_cast<const __nv_bfloat16*>(a.residual);
    p.residual_out = static_cast<__nv_bfloat16*>(a.residual_out);
    p.w = static_cast<const __nv_bfloat16*>(a.w);
    p.out = a.out;
    p.scales = static_cast<uint8_t*>(a.scales);
    p.x_stride = a.x_stride;
    p.tokens = a.tokens;
    p.hidden = a.hidden;
    p.inv_n = pair_of(1.0 / a.hidden);
    p.eps = pair_of(pool->cfg.eps);
    const int chunks = a.hidden / 8;
    // chunks a thread: two (8192 x 4096 with a residual to 8 bits us with 1 / 2 / 4: 48 / 37.0 / 43), four where 1024 threads
    // need it, one for a few short rows (64 x 1024 to bf16 1.60 / 1.67, 150 x 2048 without a residual 1.67 / 1.77, 300 x 2048
    // the same)
    const int per = chunks > 2048 ? 4 : chunks <= 256 && a.tokens <= 2 * pool->num_sms ? 1 : 2;
    const unsigned threads = (unsigned)((chunks + 32 * per - 1) / (32 * per) * 32);
    // CTAs for twice the threads that registers let be resident, each loading its next token while it works on one (a CTA a token 42 us)
    const unsigned grid = std::min((unsigned)a.tokens, (unsigned)pool->num_sms * std::max(1u, std::min(32u, 2048 / threads)));
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config(grid, threads, attr, s);
    auto with = [&](auto type, auto add) {
        constexpr int kType = decltype(type)::value;
        constexpr bool kAdd = decltype(add)::value;
        switch (per) {
            case 1: return cudaLaunchKernelEx(&cfg, add_norm_kernel<kType, kAdd, 1>, p);
            case 2: return cudaLaunchKernelEx(&cfg, add_norm_kernel<kType, kAdd, 2>, p);
            default: return cudaLaunchKernelEx(&cfg, add_norm_kernel<kType, kAdd, 4>, p);
        }
    };
    auto of = [&](auto type) { return a.residual ? with(type, std::true_type{}) : with(type, std::false_type{}); };
    switch (a.type) {
        case PKV_MX8: return of(std::integral_constant<int, PKV_MX8>{});
        case PKV_MX4: return of(std::integral_constant<int, PKV_MX4>{});
        default: return of(std::integral_constant<int, PKV_BF16>{});
    }
}

}  // namespace pkv
