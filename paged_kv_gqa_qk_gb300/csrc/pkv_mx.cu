// Microscaled tensors written and read (pkv_mx_quantize, pkv_mx_read), and the residual's
// addition with the layer's RMS norm, to bf16 or to a microscaled tensor (pkv_add_norm).
//
//   h = bf16(x + residual),   y = h / sqrt(mean(h^2) + eps) * w
//
// qwen3-8b Nest files, src/norm.linnet (RmsNorm) and DecoderLayer.decode_paged, which runs
// attention_norm before the attention and the residual's addition with mlp_norm after it.
#include <algorithm>

#include "pkv_mx.cuh"

namespace pkv {

namespace {

constexpr uint32_t kAll = 0xffffffffu;

// ---- bf16 -> microscaled ----
// 16 lanes take 128 columns of a row, 8 each; a group of 32 is 4 lanes.
template <int kType, int kPasses>
__global__ void __launch_bounds__(256)
    mx_quantize_kernel(const __nv_bfloat16* x, int64_t x_stride, int rows, int cols, uint8_t* codes,
                       uint8_t* scales)
{
    const int tiles = cols / kMxTileCols, tile = blockIdx.x % tiles;
    const int64_t row0 = (int64_t)(blockIdx.x / tiles) * (16 * kPasses);
    const int sub = threadIdx.x >> 4, j = threadIdx.x & 15;
    const int col = tile * kMxTileCols + 8 * j;
    pdl_wait();
    uint4 raw[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + 16 * i + sub;
        raw[i] = r < rows ? *reinterpret_cast<const uint4*>(x + r * x_stride + col) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = row0 + 16 * i + sub;
        float v[8];
        unpack8(raw[i], v);
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(kAll, top, 1));
        top = max(top, __shfl_xor_sync(kAll, top, 2));
        const uint32_t byte = mx_scale_byte<kType>(top);
        const float inv = mx_inverse(byte);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= inv;
        uint2 c = mx_codes8<kType>(v);
        if (byte == 255u) c = make_uint2(0, 0);
        uint32_t word = byte << (8 * (j >> 2));   // the row's four bytes of the tile
        word |= __shfl_xor_sync(kAll, word, 4);
        word |= __shfl_xor_sync(kAll, word, 8);
        if (r >= rows) continue;
        uint8_t* dst = codes + r * mx_row_bytes(kType, cols) + mx_row_bytes(kType, col);
        if constexpr (kType == PKV_MX8)
            *reinterpret_cast<uint2*>(dst) = c;
        else
            *reinterpret_cast<uint32_t*>(dst) = c.x;
        if (j == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_at(r, 4 * tile, tiles)) = word;
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

// 1 / sqrt(ss * inv_n + eps) to about 2^-44: a fp32 root and one step of Newton's
// iteration, whose residual 1 - v r^2 is formed without loss.
__device__ __forceinline__ Pair inv_rms_pair(Pair ss, Pair inv_n, Pair eps)
{
    const float t = __fmul_rn(ss.h, inv_n.h);
    const float te = __fmaf_rn(ss.h, inv_n.l, __fmaf_rn(ss.l, inv_n.h, __fmaf_rn(ss.h, inv_n.h, -t)));
    Pair v = two_sum(t, eps.h);
    v.l = __fadd_rn(v.l, __fadd_rn(te, eps.l));
    const float r = rsqrtf(v.h);
    const float p = __fmul_rn(r, r), pe = __fmaf_rn(r, r, -p);
    const float q = __fmul_rn(v.h, p);
    const float qe = __fmaf_rn(v.l, p, __fmaf_rn(v.h, pe, __fmaf_rn(v.h, p, -q)));
    const float e = __fsub_rn(__fsub_rn(1.0f, q), qe);
    return {r, __fmul_rn(__fmul_rn(r, 0.5f), e)};
}

struct AddNormParams {
    const __nv_bfloat16* x;
    const __nv_bfloat16* residual;  // null: nothing to add
    __nv_bfloat16* residual_out;
    const __nv_bfloat16* w;
    void* out;
    uint8_t* scales;
    int64_t x_stride;
    int tokens, hidden;
    Pair inv_n, eps;
};

// h * w * r as a float and the rest of it, rounded to odd: what a rounding of it to
// fewer bits gives is then the rounding of the exact value (but for 2^-44 of it).
__device__ __forceinline__ float scaled_odd(float hw, Pair r)
{
    const float q = __fmul_rn(hw, r.l), p = __fmaf_rn(hw, r.h, q);
    const float e = __fadd_rn(__fmaf_rn(hw, r.h, -p), q);
    const uint32_t b = __float_as_uint(p);
    const uint32_t odd = (b - ((b ^ __float_as_uint(e)) >> 31)) | 1u;
    return e != 0.f && (b << 1) != 0 && (b << 1) < 0xff000000u ? __uint_as_float(odd) : p;
}

// One CTA per token; thread i holds chunks i, i + T, ... of 8 columns.
template <int kType, int kChunks>
__global__ void __launch_bounds__(1024) add_norm_kernel(AddNormParams p)
{
    __shared__ Pair part[32];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x;
    const int chunks = p.hidden / 8;
    pdl_wait();
    uint4 raw[kChunks];
    Pair ss = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = tid + c * T;
        raw[c] = make_uint4(0, 0, 0, 0);
        if (at >= chunks) continue;
        raw[c] = *reinterpret_cast<const uint4*>(p.x + t * p.x_stride + 8 * at);
        if (p.residual) {
            const uint4 more = *reinterpret_cast<const uint4*>(p.residual + t * p.hidden + 8 * at);
            float a[8], b[8];
            unpack8(raw[c], a);
            unpack8(more, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] += b[k];
            raw[c] = pack8(a);
            *reinterpret_cast<uint4*>(p.residual_out + t * p.hidden + 8 * at) = raw[c];
        }
        float h[8];
        unpack8(raw[c], h);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const Pair s = two_sum(ss.h, __fmul_rn(h[k], h[k]));
            ss.h = s.h;
            ss.l = __fadd_rn(ss.l, s.l);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss = add(ss, {__shfl_xor_sync(kAll, ss.h, o), __shfl_xor_sync(kAll, ss.l, o)});
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    ss = part[0];
    for (int i = 1; i < T / 32; ++i) ss = add(ss, part[i]);
    const Pair r = inv_rms_pair(ss, p.inv_n, p.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = tid + c * T;
        float v[8], w[8];
        unpack8(raw[c], v);
        if (at < chunks) {
            unpack8(*reinterpret_cast<const uint4*>(p.w + 8 * at), w);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = 0.f;
        }
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = scaled_odd(__fmul_rn(v[k], w[k]), r);
            top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
        }
        if constexpr (kType == PKV_BF16) {
            if (at < chunks) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + t * p.hidden + 8 * at) = pack8(v);
        } else {
            top = max(top, __shfl_xor_sync(kAll, top, 1));
            top = max(top, __shfl_xor_sync(kAll, top, 2));
            const uint32_t byte = mx_scale_byte<kType>(top);
            const float inv = mx_inverse(byte);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= inv;
            uint2 code = mx_codes8<kType>(v);
            if (byte == 255u) code = make_uint2(0, 0);
            uint32_t word = byte << (8 * ((at & 15) >> 2));
            word |= __shfl_xor_sync(kAll, word, 4);
            word |= __shfl_xor_sync(kAll, word, 8);
            if (at >= chunks) continue;
            uint8_t* dst = static_cast<uint8_t*>(p.out) + t * mx_row_bytes(kType, p.hidden) + mx_row_bytes(kType, 8 * at);
            if constexpr (kType == PKV_MX8)
                *reinterpret_cast<uint2*>(dst) = code;
            else
                *reinterpret_cast<uint32_t*>(dst) = code.x;
            if ((at & 15) == 0)
                *reinterpret_cast<uint32_t*>(p.scales + mx_scale_at(t, at / 4, p.hidden / kMxTileCols)) = word;
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
    const int step = many ? 128 : 16;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((rows + step - 1) / step * tiles), 256, attr, s);
    auto launch = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const __nv_bfloat16*>(x), x_stride, rows, cols,
                                  static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales));
    };
    if (type == PKV_MX8) return many ? launch(mx_quantize_kernel<PKV_MX8, 8>) : launch(mx_quantize_kernel<PKV_MX8, 1>);
    return many ? launch(mx_quantize_kernel<PKV_MX4, 8>) : launch(mx_quantize_kernel<PKV_MX4, 1>);
}

cudaError_t launch_mx_read(const pkv_pool* pool, int type, const void* codes, const void* scales, int rows, int cols,
                           void* y, int64_t y_stride, cudaStream_t s)
{
    const int tiles = cols / kMxTileCols;
    const bool many = (int64_t)(rows + 127) / 128 * tiles >= 2 * pool->num_sms;
    const int step = many ? 128 : 16;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)((rows + step - 1) / step * tiles), 256, attr, s);
    auto launch = [&](auto kernel) {
        return cudaLaunchKernelEx(&cfg, kernel, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales),
                                  rows, cols, static_cast<__nv_bfloat16*>(y), y_stride);
    };
    if (type == PKV_MX8) return many ? launch(mx_read_kernel<PKV_MX8, 8>) : launch(mx_read_kernel<PKV_MX8, 1>);
    return many ? launch(mx_read_kernel<PKV_MX4, 8>) : launch(mx_read_kernel<PKV_MX4, 1>);
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
    const int per = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
    const unsigned threads = (unsigned)((chunks + 32 * per - 1) / (32 * per) * 32);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = config((unsigned)a.tokens, threads, attr, s);
    auto launch = [&](auto one, auto two, auto four) {
        return cudaLaunchKernelEx(&cfg, per == 1 ? one : per == 2 ? two : four, p);
    };
    switch (a.type) {
        case PKV_MX8: return launch(add_norm_kernel<PKV_MX8, 1>, add_norm_kernel<PKV_MX8, 2>, add_norm_kernel<PKV_MX8, 4>);
        case PKV_MX4: return launch(add_norm_kernel<PKV_MX4, 1>, add_norm_kernel<PKV_MX4, 2>, add_norm_kernel<PKV_MX4, 4>);
        default: return launch(add_norm_kernel<PKV_BF16, 1>, add_norm_kernel<PKV_BF16, 2>, add_norm_kernel<PKV_BF16, 4>);
    }
}

}  // namespace pkv
