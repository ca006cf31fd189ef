// A page pool in 4 bits: appending to it, reading it back, and the decode
// attention over it (sm_103a).  The format is in pkv_q4.cuh.
//
//   q4_append_kernel  QK-norm + RoPE of k, quantise k and v, write them to their slots
//   q4_prep_kernel    the same in front of the attention, with each row's check, its
//                     attended length and its prepared query heads
//   q4_attn_kernel    split attention: every warp streams its own share of the
//                     call's pages through its own ring of bulk
//                     copies and keeps its own softmax state
//   q4_combine_kernel merge of the pieces of a (token, kv head) that several
//                     warps shared
//   q4_unit_kernel    the whole decode call of few short rows in one launch
//   q4_read_kernel    cached k and v of a list of tokens as bf16
//
// Source of the computation (as the bf16 pool's): qwen3-8b Nest files,
// src/attention.linnet, GroupedQueryAttention.decode_paged.
#include <math_constants.h>

#include <algorithm>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "pkv_q4.cuh"

namespace pkv {

// A launch that may start while the kernel before it on the stream drains: every kernel
// here waits for that one (pdl_wait) before it reads or writes memory (the split attention
// reads and writes what the preparation does not touch before).  The short ones let
// the next one's CTAs come early (pdl_launch_dependents); the append and the split
// attention, which fill the SMs by themselves, do not: CTAs that wait beside theirs cost
// more than their early start saves (append and read of 2048 tokens 13.0 -> 9.1 us, steps
// of 64 rows 43.5 -> 40.9, of 256 rows 210.1 -> 207.8 us without; a trigger at the
// attention's end 41.4 and 210.7).
template <class P>
static cudaError_t launch_dependent(void (*kernel)(P), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                                    const P& p, bool early = true)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// =====================================================================================
// q4_append_kernel, q4_prep_kernel
// =====================================================================================
struct Q4AppendParams {
    const __nv_bfloat16* q;     // decode: [tokens][heads][128]
    const __nv_bfloat16* k;     // [tokens][kv_heads][128]
    const __nv_bfloat16* v;
    const __nv_bfloat16* qw;
    const __nv_bfloat16* kw;
    const int32_t* positions;   // [tokens]; -1: nothing to do
    const int32_t* prow;        // [tokens], or null: token t is table row t
    const int32_t* table;       // [rows][pages], or null: contiguous rows
    const float2* rope_hi;
    const float2* rope_lo;
    uint8_t* data;
    __half* q_hat;              // decode: [tokens][kv_heads][4][2][128]: each head times a power of two, and its remainder
    float* q_mul;               // decode: [tokens][heads], what a score of it is multiplied with
    __nv_bfloat16* out;         // decode: [tokens][heads][128], zeroed for skipped tokens
    int32_t* tok_len;           // decode: [tokens], 0: skip
    uint32_t* err;
    int tokens, rows, pages, num_pages, max_seq, heads, kv_heads, rot;
    float eps, k_scale;
    float2 eps2;                // eps as a pair of floats
    float k_inv6, k_inv, v_inv6, v_inv;  // 1 / (6 s) and 1 / s of the pool's scales
    const int* rope_exp;        // |cos|, |sin| <= 2^rope_exp (on the device: a captured call follows pkv_pool_set_rope)
};

// The two 16-byte pieces of a head vector that lane j of 8 holds.
__device__ __forceinline__ void load16(const __nv_bfloat16* head, int j, uint4 (&r)[2])
{
    r[0] = *reinterpret_cast<const uint4*>(head + 8 * j);
    r[1] = *reinterpret_cast<const uint4*>(head + 64 + 8 * j);
}
// The same of norm weights, which may lie on an 8-byte border.
__device__ __forceinline__ void load16_weights(const __nv_bfloat16* w, int j, uint4 (&r)[2])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint2 a = *reinterpret_cast<const uint2*>(w + 64 * h + 8 * j);
        const uint2 b = *reinterpret_cast<const uint2*>(w + 64 * h + 8 * j + 4);
        r[h] = make_uint4(a.x, a.y, b.x, b.y);
    }
}

// What is wrong with a token's position and row, as an error bit; 0: nothing, or no step (-1).
__device__ __forceinline__ uint32_t q4_fault(const Q4AppendParams& p, int pos, int row)
{
    if (pos == -1) return 0;
    if (row < 0 || row >= p.rows) return PKV_DEVERR_ROW;
    if (pos < 0 || pos >= p.max_seq || pos / kPageSize >= p.pages) return PKV_DEVERR_POSITION;
    return 0;
}

// The position's rows of the RoPE tables into L1 (512 bytes each), a line a thread.
__device__ __forceinline__ void prefetch_rope(const Q4AppendParams& p, int pos, int thread)
{
    constexpr int kLines = kRopeHalf * (int)sizeof(float2) / 128;
    if (thread < 2 * kLines)
        asm volatile("prefetch.global.L1 [%0];" ::"l"((thread < kLines ? p.rope_hi : p.rope_lo) + (int64_t)pos * kRopeHalf +
                                                      thread % kLines * (128 / (int)sizeof(float2))));
}

// k and v of up to 4 kv heads of one token, 8 lanes each (kraw, vraw: this lane's
// pieces; g: its head; live: there is such a head).  All lanes take part.
template <bool kFullRot>
__device__ __forceinline__ void q4_append_heads(const Q4AppendParams& p, const uint4 (&kraw)[2], const uint4 (&vraw)[2],
                                                const uint4 (&wk)[2], int rope_exp, int g, bool live, int page, int pos,
                                                int lane)
{
    const int64_t at = (int64_t)pos * kRopeHalf;
    float x[16];
    uint32_t bits[8];
    norm_rope_k_paired<kFullRot>(kraw, wk, p.rope_hi + at, p.rope_lo + at, p.eps2, rope_exp, lane, p.rot, x, bits);
    // (heads beyond the last quantise zeros and store nothing: the shuffles want every lane)
    uint8_t* block = p.data + q4_block(page, p.kv_heads, live ? g : 0, pos % kPageSize);
    q4_store(block, false, pos % kQ4Block, x, bits, p.k_inv6, p.k_inv, lane & 7, live);
    unpack16(vraw[0], vraw[1], x);
    const uint32_t vbits[8] = {vraw[0].x, vraw[0].y, vraw[0].z, vraw[0].w, vraw[1].x, vraw[1].y, vraw[1].z, vraw[1].w};
    q4_store(block, true, pos % kQ4Block, x, vbits, p.v_inv6, p.v_inv, lane & 7, live);
}

constexpr int kQ4AppendWarps = 4;

// pkv_q4_append: a warp takes kQuads times 4 kv heads of one token.  Bound by its
// instructions: about 860 a quad, half of them k's norm and rotation in pairs of floats
// (16384 tokens of 8 heads, 86 MB: 33.9 us, 2.5 TB/s, 0.71 of the issue slots).  Resident
// CTAs by measurement: 6 an SM of the two-quad form (5: 35.8, 8: 36.9 us), 7 of the other.
template <bool kFullRot, int kQuads>
__global__ void __launch_bounds__(32 * kQ4AppendWarps, !kFullRot ? 4 : kQuads == 1 ? 7 : 6) q4_append_kernel(Q4AppendParams p)
{
    const int lane = threadIdx.x & 31, j = lane & 7, groups = (p.kv_heads + 4 * kQuads - 1) / (4 * kQuads);
    const int item = blockIdx.x * kQ4AppendWarps + (threadIdx.x >> 5), t = item / groups;
    pdl_wait();
    if (t >= p.tokens) return;
    const int g0 = 4 * kQuads * (item - t * groups) + (lane >> 3);  // this lane's heads: g0, g0 + 4, ...
    uint4 kraw[kQuads][2] = {}, vraw[kQuads][2] = {}, wk[2];
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
        if (g0 + 4 * q < p.kv_heads) {
            const int64_t src = ((int64_t)t * p.kv_heads + g0 + 4 * q) * kHeadDim;
            load16(p.k + src, j, kraw[q]);
            load16(p.v + src, j, vraw[q]);
        }
    load16_weights(p.kw, j, wk);
    const int pos = p.positions[t], row = p.prow ? p.prow[t] : t, rope_exp = *p.rope_exp;
    const bool active = pos != -1;
    uint32_t e = q4_fault(p, pos, row);
    int page = 0;
    if (active && !e) {
        page = page_of(p.table, p.pages, row, pos / kPageSize);
        if (page < 0 || page >= p.num_pages) e = PKV_DEVERR_PAGE;
    }
    if (e && lane == 0) atomicOr(p.err, e);
    if (!active || e) return;
#pragma unroll
    for (int q = 0; q < kQuads; ++q)
        q4_append_heads<kFullRot>(p, kraw[q], vraw[q], wk, rope_exp, g0 + 4 * q, g0 + 4 * q < p.kv_heads, page, pos, lane);
}

// Two floats as fp16, and the fp16 of what that leaves of them (lo).
__device__ __forceinline__ __half2 split_half2(float x, float y, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(__fsub_rn(x, f.x), __fsub_rn(y, f.y));
    lo = *reinterpret_cast<const uint32_t*>(&l);
    return h;
}

// A query head over 8 lanes as an fp16 head (r) and the fp16 of its remainder (rl), times the
// power of two that brings its largest value into [1, 2): 22 bits of it, or 2^-25 of the
// largest value, whatever its size.  Returns what a score of it is multiplied with: never
// 0, which would make a masked score NaN (below 1e-30 the scores are 0 either way).
__device__ __forceinline__ float q4_query(const float (&y)[16], float k_scale, uint32_t (&r)[8], uint32_t (&rl)[8])
{
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(y[k]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const int ex = min(max((int)(__float_as_uint(top) >> 23), 1), 253);  // 2^(ex - 127) <= top < twice that
    const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const __half2 h = split_half2(y[2 * k] * down, y[2 * k + 1] * down, rl[k]);
        r[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return fmaxf(__uint_as_float((uint32_t)ex << 23) * kQScale * k_scale, 1e-30f);
}

// The 8 columns of a (token, kv head) in the score product: column 2h its query head h, column 2h + 1 the remainder.
// `to`: of this lane's head; lane j of 8.
constexpr int kQ4Columns = 2 * kGroup;
__device__ __forceinline__ void store_query(__half* to, int j, const uint32_t (&r)[8], const uint32_t (&rl)[8])
{
    __half* rest = to + kHeadDim;
    *reinterpret_cast<uint4*>(to + 8 * j) = make_uint4(r[0], r[1], r[2], r[3]);
    *reinterpret_cast<uint4*>(to + 64 + 8 * j) = make_uint4(r[4], r[5], r[6], r[7]);
    *reinterpret_cast<uint4*>(rest + 8 * j) = make_uint4(rl[0], rl[1], rl[2], rl[3]);
    *reinterpret_cast<uint4*>(rest + 64 + 8 * j) = make_uint4(rl[4], rl[5], rl[6], rl[7]);
}

// In front of the attention: one CTA per row checks every page that the row will read,
// writes its attended length (and the zeros of a skipped row's output), appends its k and v
// (items 0 .. quads - 1 of 4 kv heads) and prepares its queries (items from there on, the 4
// query heads of a kv head each).  A chain of latencies (position, page ids, k and the
// tables, sums over a head): 7 us alone for 8 to 64 rows, 11 for 256, all under 4 MB; most
// of it runs beside the attention's own start (without that overlap 64 rows take 1.9 us more).
template <bool kFullRot>
__global__ void __launch_bounds__(512) q4_prep_kernel(Q4AppendParams p)
{
    const int t = blockIdx.x, lane = threadIdx.x & 31, j = lane & 7, sub = lane >> 3, warps = blockDim.x >> 5;
    const int quads = (p.kv_heads + 3) / 4, items = quads + p.kv_heads;
    pdl_wait();               // (launched while the kernel before this call drains)
    pdl_launch_dependents();  // after the wait: the attention reads this call's inputs before it waits for this grid
    // a warp's first item's inputs go out before anything that they do not depend on
    int item = threadIdx.x >> 5;
    uint4 a[2] = {}, b[2] = {}, w[2];
    auto load = [&]() {
        if (item < quads) {
            const int g = 4 * item + sub;
            if (g < p.kv_heads) {
                const int64_t src = ((int64_t)t * p.kv_heads + g) * kHeadDim;
                load16(p.k + src, j, a);
                load16(p.v + src, j, b);
            }
            load16_weights(p.kw, j, w);
        } else if (item < items) {
            load16(p.q + ((int64_t)t * p.heads + 4 * (item - quads) + sub) * kHeadDim, j, a);
            load16_weights(p.qw, j, w);
        }
    };
    load();
    const int pos = p.positions[t], row = t, rope_exp = *p.rope_exp;
    const bool active = pos != -1;
    uint32_t e = q4_fault(p, pos, row);
    int page = 0, bad = 0;
    if (active && !e) {
        prefetch_rope(p, pos, threadIdx.x);
        const int last = pos / kPageSize;
        page = page_of(p.table, p.pages, row, last);
        for (int i = threadIdx.x; i <= last; i += blockDim.x) {
            const int id = page_of(p.table, p.pages, row, i);
            bad |= id < 0 || id >= p.num_pages;
        }
    }
    if (__syncthreads_or(bad)) e = PKV_DEVERR_PAGE;
    const bool ok = active && !e;
    if (threadIdx.x == 0) {
        p.tok_len[t] = ok ? pos + 1 : 0;
        if (e) atomicOr(p.err, e);
    }
    if (!ok) {
        uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)t * p.heads * kHeadDim);
        for (int i = threadIdx.x; i < p.heads * kHeadDim / 8; i += blockDim.x) out[i] = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    for (; item < items; item += warps, load()) {
        if (item < quads) {
            const int g = 4 * item + sub;
            q4_append_heads<kFullRot>(p, a, b, w, rope_exp, g, g < p.kv_heads, page, pos, lane);
            continue;
        }
        float x[16], y[16];
        uint32_t r[8], rl[8];
        unpack16(a[0], a[1], x);
        norm_rope_q16<kFullRot>(x, w, p.rope_hi + (int64_t)pos * kRopeHalf, p.eps, lane, p.rot, y);
        const float mul = q4_query(y, p.k_scale, r, rl);
        const int64_t u = (int64_t)t * p.kv_heads + (item - quads);
        store_query(p.q_hat + (u * kQ4Columns + 2 * sub) * kHeadDim, j, r, rl);
        if (j == 0) p.q_mul[u * kGroup + sub] = mul;
    }
}

static Q4AppendParams append_params(const pkv_pool* pool)
{
    Q4AppendParams p = {};
    p.rope_hi = pool->rope_hi;
    p.rope_lo = pool->rope_lo;
    p.data = static_cast<uint8_t*>(pool->q4);
    p.err = pool->err;
    p.num_pages = pool->num_pages;
    p.max_seq = pool->cfg.max_seq;
    p.heads = pool->cfg.heads;
    p.kv_heads = pool->cfg.kv_heads;
    p.rot = pool->cfg.rotary_dim > 0 ? pool->cfg.rotary_dim : kHeadDim;
    p.eps = (float)pool->cfg.eps;
    p.eps2 = make_float2(p.eps, (float)(pool->cfg.eps - (double)p.eps));
    p.rope_exp = reinterpret_cast<const int*>(pool->err + 1);
    p.k_scale = pool->k_scale;
    p.k_inv6 = (1.f / 6.f) / pool->k_scale;  // (the scales are powers of two)
    p.k_inv = 1.f / pool->k_scale;
    p.v_inv6 = (1.f / 6.f) / pool->v_scale;
    p.v_inv = 1.f / pool->v_scale;
    return p;
}

cudaError_t launch_q4_append(const pkv_pool* pool, const void* k, const void* v, const void* k_norm_w,
                             const int32_t* positions, const int32_t* prow, const int32_t* table, int tokens, int rows,
                             int pages, cudaStream_t s)
{
    Q4AppendParams p = append_params(pool);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.kw = static_cast<const __nv_bfloat16*>(k_norm_w);
    p.positions = positions;
    p.prow = prow;
    p.table = table;
    p.tokens = tokens;
    p.rows = rows;
    p.pages = pages;
    // few tokens: 4 heads a warp, for the shorter chain; many: 8, which share the token's address arithmetic (8 heads, us
    // with 4 / 8: 77 tokens 2.5 / 3.5, 2048 5.8 / 6.2, 3000 8.1 / 7.3, 16384 38.8 / 34.2)
    const int quads = (p.kv_heads + 3) / 4, per = quads > 1 && (int64_t)tokens * quads >= 32 * (int64_t)pool->num_sms ? 2 : 1;
    const int64_t items = (int64_t)tokens * ((quads + per - 1) / per);
    const unsigned grid = (unsigned)((items + kQ4AppendWarps - 1) / kQ4AppendWarps);
    const bool full = p.rot == kHeadDim;
    return launch_dependent(per == 1 ? (full ? q4_append_kernel<true, 1> : q4_append_kernel<false, 1>)
                                     : (full ? q4_append_kernel<true, 2> : q4_append_kernel<false, 2>),
                            grid, 32 * kQ4AppendWarps, 0, s, p);
}

// =====================================================================================
// q4_attn_kernel
// =====================================================================================
//
// Work.  A (token, kv head) unit's positions are cut into chunks of a page (9216
// contiguous bytes); units in order, kv heads within tokens, make one sequence of T
// chunks, and warp w of W streams chunks [w T / W, (w + 1) T / W).  Warps of one CTA
// are far apart in that sequence (w = warp * CTAs + CTA): a small call spreads over
// all SMs.  A unit inside one warp's share is written out; the pieces of the others
// go to index u + w of the partials (unique: units and warps both increase along the
// sequence), and q4_combine_kernel merges them, in an order that depends on the sizes
// alone.  No warp waits for a warp of another CTA.  (Merging in this kernel, by the warp or
// the CTA that counts itself last at a unit, took longer than the launch: 8 rows of 36000
// 74 and 86 us a call, 61 so.)
//
// The kernel starts beside q4_prep_kernel (programmatic launch): it splits the work
// by the positions and starts its first copies at once -- all but a row's last chunk,
// which holds the position that the preparation writes -- and waits for the
// preparation before it needs the queries.
//
// Per 16 positions (a block), with lane = 4 r + c:
//   S[16 pos][8] = K[16][128] q[128][8], m16n8k16 fp16: column 2h = query head h of the
//     group in fp16, column 2h + 1 = the fp16 of its remainder (S = the two columns' sum, in one
//     lane: 22 bits of q), row i = position pi(i), row i + 8 = pi(i) + 8, pi(2c + b) = (c ^ b) + 4b.  Lane (r, c) holds dims 32c..32c+31 of rows r and r + 8:
//     one 16-byte read of codes each, two scales each.
//   O^T[128][8] += V^T[128][16 pos] P[16][8]: lane (r, c) holds dims 16r..16r+15 (one
//     group) of positions pi(2c), pi(2c + 1) and the same + 8: four 8-byte reads, four scales.
//     P's columns as q's, added at the segment's end; a weight is kept to 2^-21 of itself or 2^-32 of
//     the largest, nearly the fp32 it was computed in.
// The codes become fp16 by the conversion instruction and are multiplied by their
// scales as fp16 pairs, exactly; V's are first regrouped so that one byte holds a
// dim's codes of two positions.  P is turned between the fragments by movmatrix.
//
// What bounds it (alone, cold cache): long rows by memory, 8 rows of 32768-40960 331 MB in
// 58.6 us, 5.6 TB/s; 64 rows of 512-4096 182 MB in 37.5 us, 4.9 TB/s, 5 us of them the start and
// the last warps' ends; many rows by instructions, 256 rows of 1024-8192 1.04 GB in 206 us,
// 5.1 TB/s: about 237 warp instructions a block, 111 of them on the integer pipe (the
// conversions and the scales' products), at 2.4 an SM and cycle.  mma.sync m16n8k16 is used a third of
// its rate there; an instruction with K = 16 takes the 16 dims of a scale whole.
// The remainders of q and P cost 5 us of the 256 rows (the longer chain from score to weight) and nothing
// where memory bounds; with heads in columns 0-3 and remainders in 4-7, whose halves meet by
// shuffles, they cost 10, and the 64 rows 1.
// 12 warps of 2 stages of a page: 16 warps of half pages 50 / 69 / 237 us a call on these three
// workloads against 45 / 64 / 212 then, 8 warps of 3 stages no better, a copying warp
// beside 11 others 51 / 75 / 257 (all without remainders).
constexpr int kQ4Warps = 12;
constexpr int kQ4MostCtas = 4096;                    // of a grid that pkv_set_ctas asks for
constexpr int kQ4Stages = 2;
constexpr int kQ4Chunk = 64;                         // positions: a page
constexpr int kQ4Blocks = kQ4Chunk / kQ4Block;
constexpr int kQ4ChunkBytes = kQ4Blocks * kQ4BlockBytes;
constexpr float kQ4Lift = 8.f;                       // base-2 exponent of the largest weight when it is set (Q4State)
constexpr float kQ4Most = 15.f;                      // that a weight may reach: 2^15 is within fp16

struct Q4AttnParams {
    const __half* q_hat;
    const float* q_mul;
    const int32_t* positions;
    const int32_t* tok_len;  // 0: a row that the preparation skipped
    const int32_t* table;
    const uint8_t* data;
    __nv_bfloat16* out;
    float* part_o;      // [U + W][4][128]
    float* part_lse;    // [U + W][4]
    int32_t* prefix;    // [ntok + 1]: chunks before each token, written by CTA 0 for the combine
    uint32_t* err;
    int ntok, pages, num_pages, max_seq, heads, kv_heads;
    float v_scale;
    uint64_t wait_ns;
};

struct Q4Smem {
    static constexpr int kRing = 0;
    static constexpr int kBars = kQ4Warps * kQ4Stages * kQ4ChunkBytes;
    static constexpr int kT0 = kBars + 8 * kQ4Warps * kQ4Stages;
    static constexpr int kP0 = kT0 + 4 * 32 * kQ4Warps;
    static constexpr int kLen = kP0 + 4 * 32 * kQ4Warps;
    static constexpr int kScan = kLen + 4 * 32 * kQ4Warps;
    static constexpr int kBytes = kScan + 4 * kQ4Warps;
    static constexpr int kAlloc = kBytes + 128;  // slack to align the base
};
static_assert(Q4Smem::kAlloc <= 227 * 1024, "the ring fits");

// Attended length of token t and its chunks (rows with a bad page count: they are
// streamed, with the page ids put in range, and not written out).
__device__ __forceinline__ int q4_len(const Q4AttnParams& p, int t)
{
    const int pos = p.positions[t];
    return pos >= 0 && pos < p.max_seq && pos / kPageSize < p.pages ? pos + 1 : 0;
}
__device__ __forceinline__ int q4_chunks(int len) { return (len + kQ4Chunk - 1) / kQ4Chunk; }

// The split of T chunks over W <= T warps: warp w has chunks [floor(w T / W), floor((w + 1) T / W)),
// in unsigned 32-bit arithmetic: rem < W and w <= W, so w rem < W^2.
static_assert((uint64_t)kQ4MostCtas * kQ4Warps * kQ4MostCtas * kQ4Warps < (uint64_t(1) << 32), "w rem fits 32 bits");
struct Q4Split {
    int T, W, q, rem;
    __device__ __forceinline__ Q4Split(int T_, int W_) : T(T_), W(W_), q(W_ ? T_ / W_ : 0), rem(W_ ? T_ - q * W_ : 0) {}
    __device__ __forceinline__ int start(int w) const { return w * q + (int)((uint32_t)w * (uint32_t)rem / (uint32_t)W); }
    __device__ __forceinline__ int warp_of(int x) const  // the warp that has chunk x
    {
        int w = min(max((int)((float)x * ((float)W / (float)T)), 0), W - 1);
        while (start(w) > x) --w;
        while (w + 1 < W && start(w + 1) <= x) ++w;
        return w;
    }
};

// Warp-wide: the token holding chunk x (x < T), its length, and the chunks of one kv head before it.
__device__ __forceinline__ void q4_find(const Q4AttnParams& p, const int* sT0, const int* sP0, const int* sLen,
                                        int x, int lane, int& t_out, int& len_out, int& pre_out)
{
    const int G = p.kv_heads;
    int lo = 0, hi = 32 * kQ4Warps - 1;
    while (lo < hi) {  // last run of tokens whose prefix is at or before x
        const int mid = (lo + hi + 1) >> 1;
        if (G * sP0[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    int t = sT0[lo], pre = sP0[lo];
    if (p.ntok <= 32 * kQ4Warps) {  // runs of one token: it is this one (those after it start beyond x)
        t_out = t;
        len_out = sLen[lo];
        pre_out = pre;
        return;
    }
    for (; t < p.ntok; t += 32) {
        const int len = t + lane < p.ntok ? q4_len(p, t + lane) : 0, n = q4_chunks(len);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        const int before = pre + incl - n;
        const unsigned m = __ballot_sync(kFull, n > 0 && G * before <= x && x < G * (before + n));
        if (m) {
            const int l = __ffs(m) - 1;
            t_out = t + l;
            len_out = __shfl_sync(kFull, len, l);
            pre_out = __shfl_sync(kFull, before, l);
            return;
        }
        pre += __shfl_sync(kFull, incl, 31);
    }
    t_out = p.ntok - 1;  // not reached: x < T lies in some token
    len_out = 1;
    pre_out = pre;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of 16-bit elements (lane 4i + j: row i, columns 2j, 2j + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
__device__ __forceinline__ __half2 lows(uint32_t x) { return __low2half2(as_half2(x)); }
__device__ __forceinline__ __half2 highs(uint32_t x) { return __high2half2(as_half2(x)); }
constexpr uint32_t kOnes = 0x3c003c00u;  // two fp16 ones

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// What a lane keeps of its place in the fragments (lane = 4 r + c).
struct Q4Lane {
    int r, c;
    int pi_r;         // position of row r
    int pi_0, pi_1;   // positions of k = 2c, 2c + 1
    uint32_t koff, voff0, voff1, soff;
    __device__ __forceinline__ explicit Q4Lane(int lane)
    {
        r = lane >> 2;
        c = lane & 3;
        pi_r = ((r >> 1) ^ (r & 1)) | ((r & 1) << 2);
        pi_0 = c;
        pi_1 = (c ^ 1) | 4;
        koff = 64 * pi_r + ((16 * c) ^ (((pi_r >> 1) & 1) << 5));
        voff0 = kQ4VCodes + 64 * pi_0 + ((8 * r) ^ (((pi_0 >> 1) & 1) << 5));
        voff1 = kQ4VCodes + 64 * pi_1 + ((8 * r) ^ (((pi_1 >> 1) & 1) << 5));
        soff = kQ4KScales + 16 * r + 4 * c;
    }
};

// A warp's attention of one (token, kv head) over some of its chunks.  Lanes c hold head c: of a product's two
// columns, the one with the fp16 heads of the queries or weights and the one with their remainders.
struct Q4State {
    uint32_t bq[8][2];   // the queries' fragments
    float mul;           // what scores are multiplied with
    float o[9][4];       // o[k][0] + [1]: dim 16r + 2k, [2] + [3]: dim 16r + 2k + 1; not normalised; o[8]: the weights'
                         // sum (the product with ones), [0] + [1] as [2] + [3], in every row
    float m;             // weights are 2^(score - m)

    // q_hat: 8 columns of 128 fp16; q_mul: the 4 heads' multipliers
    __device__ __forceinline__ void open(const Q4Lane& L, const __half* q_hat, const float* q_mul)
    {
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = reinterpret_cast<const uint4*>(q_hat + L.r * kHeadDim + 32 * L.c)[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bq[2 * k][0] = x[k].x;
            bq[2 * k][1] = x[k].y;
            bq[2 * k + 1][0] = x[k].z;
            bq[2 * k + 1][1] = x[k].w;
        }
        mul = q_mul[L.c];
#pragma unroll
        for (int k = 0; k < 9; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
        m = -CUDART_INF_F;
    }

    // Heads and remainders added: dims 16r + 2k and + 1 of the lane's head, and the weights' sum.
    __device__ __forceinline__ float2 pair(int k) const { return make_float2(o[k][0] + o[k][1], o[k][2] + o[k][3]); }
    __device__ __forceinline__ float sum() const { return o[8][0] + o[8][1]; }

    // One chunk of kBlocks blocks in shared memory at sb, of which the unit has `left` positions (as many or more: all).
    template <int kBlocks>
    __device__ __forceinline__ void chunk(const Q4Lane& L, const uint8_t* sb, int left)
    {
        // ---- S = K q^T
        float s[kBlocks][4];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
            const uint8_t* kb = sb + b * kQ4BlockBytes;
            const uint4 k0 = *reinterpret_cast<const uint4*>(kb + L.koff), k1 = *reinterpret_cast<const uint4*>(kb + L.koff + 512);
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(kb + L.soff);
            const uint32_t s0 = e4m3x2_half2(sc), s1 = e4m3x2_half2(sc >> 16);
            const __half2 sd[2][2] = {{lows(s0), highs(s0)}, {lows(s1), highs(s1)}};
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t h0[4], h1[4];
                q4_unpack(w0[q], h0);
                q4_unpack(w1[q], h1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h0[e] = as_u32(__hmul2(as_half2(h0[e]), sd[0][q >> 1]));
                    h1[e] = as_u32(__hmul2(as_half2(h1[e]), sd[1][q >> 1]));
                }
                mma_f16_16816(s[b], h0[0], h1[0], h0[1], h1[1], bq[2 * q][0], bq[2 * q][1]);
                mma_f16_16816(s[b], h0[2], h1[2], h0[3], h1[3], bq[2 * q + 1][0], bq[2 * q + 1][1]);
            }
        }

        // ---- softmax, base 2, of the lane's head: s[b][0] + [1] at position L.pi_r of block b, [2] + [3] at L.pi_r + 8
        float t[kBlocks][2];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            t[b][0] = s[b][0] + s[b][1];
            t[b][1] = s[b][2] + s[b][3];
        }
        // Positions past the row's end: scores of -inf, and V scales of 0 (the codes are finite
        // whatever lies there), in a row's last chunk only.
        uint32_t vmask[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) vmask[b] = ~0u;
        if (left < kBlocks * kQ4Block) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int at = left - kQ4Block * b;
                if (L.pi_r >= at) t[b][0] = -CUDART_INF_F;
                if (L.pi_r + 8 >= at) t[b][1] = -CUDART_INF_F;
                vmask[b] = (L.pi_0 < at ? 0xffu : 0u) | (L.pi_1 < at ? 0xff00u : 0u) | (L.pi_0 + 8 < at ? 0xff0000u : 0u) |
                           (L.pi_1 + 8 < at ? 0xff000000u : 0u);
            }
        }
        float top = fmaxf(t[0][0], t[0][1]);
#pragma unroll
        for (int b = 1; b < kBlocks; ++b) top = fmaxf(top, fmaxf(t[b][0], t[b][1]));
        top *= mul;
        // m lies kQ4Lift below the largest score it was set at, and follows only when a lane's passes it by more than
        // kQ4Most: weights stay below 2^kQ4Most, inside fp16, and most chunks need no maximum over the lanes and
        // rescale nothing
        if (__any_sync(kFull, top > m + kQ4Most)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
            top = fmaxf(top - kQ4Lift, m);
            // (a maximum still at -inf -- scores that are all NaN -- leaves nothing to rescale)
            const float f = top == -CUDART_INF_F ? 1.f : ex2(m - top);
            m = top;
#pragma unroll
            for (int k = 0; k < 9; ++k) {
                o[k][0] *= f;
                o[k][1] *= f;
                o[k][2] *= f;
                o[k][3] *= f;
            }
        }
        // the weights of both rows, each as its upper 11 bits and the fp16 of what they leave, side by side
        uint32_t pb[kBlocks][2];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float w = ex2(__fmaf_rn(t[b][e], mul, -m)), head = __uint_as_float(__float_as_uint(w) & ~0x1fffu);
                pb[b][e] = movmatrix_trans(as_u32(__floats2half2_rn(head, __fsub_rn(w, head))));
            }

        // ---- O^T += V^T P
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const uint8_t* vb = sb + b * kQ4BlockBytes;
            const uint2 v0 = *reinterpret_cast<const uint2*>(vb + L.voff0), v1 = *reinterpret_cast<const uint2*>(vb + L.voff1);
            const uint2 v2 = *reinterpret_cast<const uint2*>(vb + L.voff0 + 512), v3 = *reinterpret_cast<const uint2*>(vb + L.voff1 + 512);
            const uint32_t sc = *reinterpret_cast<const uint32_t*>(vb + L.soff + 128) & vmask[b];
            const uint32_t s01 = e4m3x2_half2(sc), s23 = e4m3x2_half2(sc >> 16);
            mma_f16_16816(o[8], kOnes, kOnes, kOnes, kOnes, pb[b][0], pb[b][1]);
            const uint32_t a0[2] = {v0.x, v0.y}, a1[2] = {v1.x, v1.y}, a2[2] = {v2.x, v2.y}, a3[2] = {v3.x, v3.y};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                constexpr uint32_t kLow = 0x0f0f0f0fu;
                uint32_t e01[4], d01[4], e23[4], d23[4];  // even and odd dims of the two pairs of positions
                q4_unpack((a0[q] & kLow) | ((a1[q] << 4) & ~kLow), e01);
                q4_unpack(((a0[q] >> 4) & kLow) | (a1[q] & ~kLow), d01);
                q4_unpack((a2[q] & kLow) | ((a3[q] << 4) & ~kLow), e23);
                q4_unpack(((a2[q] >> 4) & kLow) | (a3[q] & ~kLow), d23);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mma_f16_16816(o[4 * q + e], as_u32(__hmul2(as_half2(e01[e]), as_half2(s01))),
                                  as_u32(__hmul2(as_half2(d01[e]), as_half2(s01))),
                                  as_u32(__hmul2(as_half2(e23[e]), as_half2(s23))),
                                  as_u32(__hmul2(as_half2(d23[e]), as_half2(s23))), pb[b][0], pb[b][1]);
            }
        }
    }
};

__global__ void __launch_bounds__(32 * kQ4Warps, 1) q4_attn_kernel(Q4AttnParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    uint8_t* sbase = smem_raw + (base - raw);
    int* sT0 = reinterpret_cast<int*>(sbase + Q4Smem::kT0);
    int* sP0 = reinterpret_cast<int*>(sbase + Q4Smem::kP0);
    int* sLen = reinterpret_cast<int*>(sbase + Q4Smem::kLen);  // of each token, where every token has a thread
    int* sScan = reinterpret_cast<int*>(sbase + Q4Smem::kScan);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.kv_heads, H = p.heads;
    const uint32_t ring = base + warp * (kQ4Stages * kQ4ChunkBytes);
    const uint32_t bars = base + Q4Smem::kBars + 8 * kQ4Stages * warp;
    if (lane == 0) {
        for (int i = 0; i < kQ4Stages; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    // chunks per token and their prefix over tokens (one run of tokens a thread; every CTA computes it)
    const int nt = p.ntok, per = (nt + 32 * kQ4Warps - 1) / (32 * kQ4Warps);
    const int t0 = min(nt, tid * per), t1 = min(nt, t0 + per);
    int local = 0, tlen = 0;
    for (int t = t0; t < t1; ++t) local += q4_chunks(tlen = q4_len(p, t));
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sScan[warp] = incl;
    __syncthreads();
    int total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kQ4Warps; ++w) {
        before += w < warp ? sScan[w] : 0;
        total += sScan[w];
    }
    sT0[tid] = t0;
    sP0[tid] = before + incl - local;
    sLen[tid] = tlen;
    if (blockIdx.x == 0) {
        int run = before + incl - local;
        for (int t = t0; t < t1; ++t) {
            p.prefix[t] = run;
            run += q4_chunks(q4_len(p, t));
        }
        if (tid == 0) p.prefix[nt] = total;
    }
    __syncthreads();

    const int T = G * total;  // (the host bounds rows * pages * kv_heads)
    const Q4Split sp(T, min((int)gridDim.x * kQ4Warps, T));
    const int W = sp.W;
    const int w = warp * gridDim.x + blockIdx.x;
    const int xb = w < W ? sp.start(w) : 0, count = w < W ? sp.start(w + 1) - xb : 0;

    // chunk j of n of unit (t, g): where the warp computes, and (the i... values) where it issues copies
    int t = 0, g = 0, j = 0, n = 1, len = 0;
    if (count > 0) {
        int pre;
        q4_find(p, sT0, sP0, sLen, xb, lane, t, len, pre);
        n = q4_chunks(len);
        const int off = xb - G * pre;
        g = off / n;
        j = off - g * n;
    }
    auto next_unit = [&](int& t, int& g, int& j, int& n, int& len) {  // (only where chunks remain)
        j = 0;
        if (++g < G) return;
        g = 0;
        do {
            len = q4_len(p, ++t);
        } while (len == 0);
        n = q4_chunks(len);
    };
    int it = t, ig = g, ij = j, in = n, ilen = len, issued = 0, ist = 0;
    constexpr int kPerPage = kPageSize / kQ4Chunk;
    int entries = 0;     // table entries 32 k .. 32 k + 31 of the row, one a lane
    uint32_t shared = 0;  // which of them the row before or after lists too
    bool reload = true;
    // pages are read once, but those of a prefix that rows share: these stay in L2, the rest go first
    const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
    auto issue = [&]() {
        const int pg = ij / kPerPage;
        if (reload || (ij % (32 * kPerPage)) == 0) {
            const int e = (pg & ~31) + lane;
            const bool in_row = e <= (ilen - 1) / kPageSize;
            entries = in_row ? page_of(p.table, p.pages, it, e) : 0;
            bool same = false;
            if (in_row && p.table)
                same = (it > 0 && page_of(p.table, p.pages, it - 1, e) == entries) ||
                       (it + 1 < p.ntok && page_of(p.table, p.pages, it + 1, e) == entries);
            shared = __ballot_sync(kFull, same);
            if (entries < 0 || entries >= p.num_pages) entries = 0;  // (then the row is not written out)
            reload = false;
        }
        const int page = __shfl_sync(kFull, entries, pg & 31);
        if (lane == 0) {
            const uint32_t bytes = min((ilen - ij * kQ4Chunk + kQ4Block - 1) / kQ4Block, kQ4Blocks) * kQ4BlockBytes;
            mbar_arrive_expect_tx(bars + 8 * ist, bytes);
            const uint8_t* src = p.data + ((int64_t)page * G + ig) * kQ4PageBytes + (ij % kPerPage) * kQ4ChunkBytes;
            bulk_copy_g2s_hint(ring + ist * kQ4ChunkBytes, src, bytes, bars + 8 * ist, (shared >> (pg & 31)) & 1 ? again : once);
        }
        ++issued;
        ist = ist == kQ4Stages - 1 ? 0 : ist + 1;
        if (++ij == in && issued < count) {
            next_unit(it, ig, ij, in, ilen);
            reload = true;
        }
    };
    // before the preparation is waited for: what it does not write
    while (issued < kQ4Stages - 1 && issued < count && ij != in - 1) issue();
    pdl_wait();
    while (issued < kQ4Stages - 1 && issued < count) issue();

    const Q4Lane L(lane);
    const uint8_t* wring = sbase + warp * (kQ4Stages * kQ4ChunkBytes);
    Q4State S;
    bool fresh = true;   // the next chunk opens a segment
    bool whole = false;  // the segment began with its unit's first chunk
    bool live = false;   // its row has an output (the preparation found no fault with it)
    bool ok = true;
    int st = 0;
    uint32_t phase = 0;

    for (int i = 0; i < count; ++i) {
        if (issued < count) issue();
        if (fresh) {
            const int64_t u = (int64_t)t * G + g;
            S.open(L, p.q_hat + u * kQ4Columns * kHeadDim, p.q_mul + u * kGroup);
            live = p.tok_len[t] > 0;
            whole = j == 0;
            fresh = false;
        }
        if (__any_sync(kFull, !mbar_wait(bars + 8 * st, phase, p.wait_ns))) {
            ok = false;
            break;
        }
        S.chunk<kQ4Blocks>(L, wring + st * kQ4ChunkBytes, len - j * kQ4Chunk);
        __syncwarp();  // every lane has read the stage: it may be filled again

        if (++st == kQ4Stages) {
            st = 0;
            phase ^= 1;
        }
        const bool last = j == n - 1;
        if ((last || i == count - 1) && live) {  // end of the segment
            const float sum = S.sum(), inv = p.v_scale / sum;
            const int64_t u = (int64_t)t * G + g;
            if (whole && last) {
                __nv_bfloat16* dst = p.out + ((int64_t)t * H + g * kGroup + L.c) * kHeadDim + 16 * L.r;
                uint32_t x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 y = S.pair(k);
                    x[k] = pack_bf16(__float2bfloat16_rn(y.x * inv), __float2bfloat16_rn(y.y * inv));
                }
                *reinterpret_cast<uint4*>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4*>(dst + 8) = make_uint4(x[4], x[5], x[6], x[7]);
            } else {
                float* po = p.part_o + ((u + w) * kGroup + L.c) * kHeadDim + 16 * L.r;
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const float2 y = S.pair(k), z = S.pair(k + 1);
                    *reinterpret_cast<float4*>(po + 2 * k) = make_float4(y.x * inv, y.y * inv, z.x * inv, z.y * inv);
                }
                if (L.r == 0) p.part_lse[(u + w) * kGroup + L.c] = S.m + log2f(sum);
            }
        }
        fresh |= last;
        if (++j == n && i + 1 < count) next_unit(t, g, j, n, len);
    }
    if (!ok) {  // the awaited copy is late: report, and let the copies in flight land before the CTA may exit
        if (lane == 0) {
            atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            for (int k = max(0, issued - kQ4Stages); k < issued; ++k)
                mbar_wait(bars + 8 * (k % kQ4Stages), (k / kQ4Stages) & 1, kWaitLimitNs);
        }
        __syncwarp();
    }
}

// =====================================================================================
// q4_combine_kernel: kHeads query heads of a (token, kv head) unit per CTA, kSub warps each;
// a lane holds 4 dims
// =====================================================================================
struct Q4CombineParams {
    const int32_t* prefix;
    const int32_t* tok_len;
    const float* part_o;
    const float* part_lse;
    __nv_bfloat16* out;
    int ntok, heads, kv_heads, warps;  // warps: of the attention's grid
};

// out = sum_k 2^(lse_k - M) o_k / sum_k 2^(lse_k - M).  Each warp takes every kSub-th piece,
// kBatch of them in flight, and its own maximum; the warps' sums are joined in warp order.
// Few units mean many pieces each, and few CTAs: a head's pieces get up to 16 warps, and every
// head its own CTA.
template <int kHeads, int kSub>
__global__ void __launch_bounds__(32 * kHeads * kSub) q4_combine_kernel(Q4CombineParams p)
{
    constexpr int kBatch = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.kv_heads;
    const int mine = warp % kHeads, sub = warp / kHeads, head = blockIdx.x % (kGroup / kHeads) * kHeads + mine;
    const int u = blockIdx.x / (kGroup / kHeads), t = u / G, g = u % G;
    pdl_wait();
    pdl_launch_dependents();
    const int pre = p.prefix[t], n = p.prefix[t + 1] - pre, total = p.prefix[p.ntok];
    if (p.tok_len[t] == 0) return;  // a skipped token: its zeros are there
    const int T = G * total, x0 = G * pre + g * n;
    const Q4Split sp(T, min(p.warps, T));
    const int wf = sp.warp_of(x0), wl = sp.warp_of(x0 + n - 1);
    if (wf == wl) return;  // one warp held it and wrote it out
    const int np = wl - wf + 1;
    const float* lse = p.part_lse + ((int64_t)u + wf) * kGroup + head;
    const float* po = p.part_o + (((int64_t)u + wf) * kGroup + head) * kHeadDim + 4 * lane;
    float M = -CUDART_INF_F, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = sub; k0 < np; k0 += kSub * kBatch) {
        float4 x[kBatch];
        float l[kBatch], m = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t at = min(k0 + k * kSub, np - 1);
            x[k] = *reinterpret_cast<const float4*>(po + at * kGroup * kHeadDim);
            l[k] = k0 + k * kSub < np ? lse[at * kGroup] : -CUDART_INF_F;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) m = fmaxf(m, l[k]);
        const float f0 = M == -CUDART_INF_F ? 0.f : exp2f(M - m);
        sum *= f0;
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[d] *= f0;
        M = m;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k0 + k * kSub >= np) break;
            const float f = exp2f(l[k] - M);  // (all pieces NaN: M stays -inf, and this is NaN)
            sum += f;
            acc[0] += f * x[k].x;
            acc[1] += f * x[k].y;
            acc[2] += f * x[k].z;
            acc[3] += f * x[k].w;
        }
    }
    if constexpr (kSub > 1) {
        __shared__ float part[kSub][kHeads][6][32];
        float(&my)[6][32] = part[sub][mine];
        my[0][lane] = acc[0], my[1][lane] = acc[1], my[2][lane] = acc[2], my[3][lane] = acc[3];
        my[4][lane] = sum, my[5][lane] = M;
        __syncthreads();
        if (sub != 0) return;
        float all = -CUDART_INF_F;
#pragma unroll
        for (int q = 0; q < kSub; ++q) all = fmaxf(all, part[q][mine][5][lane]);
        sum = acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
        for (int q = 0; q < kSub; ++q) {
            if (q >= np) break;  // no piece, no maximum
            const float(&o)[6][32] = part[q][mine];
            const float f = exp2f(o[5][lane] - all);
            sum += f * o[4][lane];
#pragma unroll
            for (int d = 0; d < 4; ++d) acc[d] += f * o[d][lane];
        }
    }
    const float inv = 1.f / sum;
    const float y[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.heads + g * kGroup + head) * kHeadDim + 4 * lane) = pack4(y);
}

// =====================================================================================
// q4_unit_kernel: a whole decode call in one launch, for small calls
// =====================================================================================
//
// A cluster of CTAs per (token, kv head) unit; its warps take the unit's pieces (pages or
// half pages) in turn (piece j: warp j mod the cluster's warps, spread over its CTAs first).
// Every CTA checks the row and prepares the unit's queries; the warp that has the last piece
// quantises the row's k and v while that piece is on its way, and puts them into the
// pool and into the staged piece.  A CTA joins its warps' sums, and the first CTA of the
// cluster the CTAs', through distributed shared memory.
//
// A call of few short rows is bound by its chain of latencies, not by bytes: this has
// one launch and one trip to memory after the table, where preparation, split attention
// and combine are three launches (one row of 700: 5.7 us a call instead of 8.9).  Half pages
// halve the chain of a warp's first piece, 1.3 us, where there are warps for all of them;
// whole pages carry more a round.  Both have 8 warps, two a scheduler, of which one computes
// while the other waits (4 warps of pages: 16 rows of 500-1500 10.8 us, 9.4 with 8).  The
// rule and its other figures are at q4_unit_choice.
constexpr int kUnitStages = 2;

// The forms of the kernel: a warp takes a piece of kBlocks blocks of 16 positions at a time.
template <int kBlocks_>
struct Q4Unit {
    static constexpr int kWarps = 8, kBlocks = kBlocks_;
    static constexpr int kPiece = kBlocks * kQ4Block, kPerPage = kPageSize / kPiece;
    static constexpr int kPieceBytes = kBlocks * kQ4BlockBytes;
    static constexpr int kRing = kUnitStages * kPieceBytes;          // of a warp; later its sums
    static constexpr int kBars = kWarps * kRing;
    static constexpr int kQ = kBars + 8 * kWarps * kUnitStages;      // __half [4][2][128]
    static constexpr int kMul = kQ + 2 * kQ4Columns * kHeadDim;      // float [4]
    static constexpr int kML = kMul + 4 * kGroup;                    // float2 [warps][4]: maximum and sum
    static constexpr int kBytes = kML + 8 * kWarps * kGroup;
    static constexpr int kAlloc = kBytes + 128;
    static constexpr int kCtas = kBlocks == 4 ? 1 : 2;               // an SM (bounds the registers)
    static_assert(4 * kGroup * kHeadDim <= kRing, "a warp's sums fit its ring");
    static_assert(kCtas * kAlloc <= 227 * 1024, "the rings fit");
};

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

template <class U, bool kFullRot>
__global__ void __launch_bounds__(32 * U::kWarps, U::kCtas) q4_unit_kernel(Q4AppendParams p, float v_scale, uint64_t wait_ns, int cs)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    uint8_t* sbase = smem_raw + (base - raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lj = lane & 7, sub = lane >> 3, G = p.kv_heads;
    const int u = blockIdx.x / cs, t = u / G, g = u % G, rank = (int)cluster_rank();
    const uint32_t bars = base + U::kBars + 8 * kUnitStages * warp;
    uint8_t* ring = sbase + warp * U::kRing;
    __half* sQ = reinterpret_cast<__half*>(sbase + U::kQ);
    float* sMul = reinterpret_cast<float*>(sbase + U::kMul);
    float2* sML = reinterpret_cast<float2*>(sbase + U::kML);
    if (lane == 0) {
        for (int i = 0; i < kUnitStages; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();

    // the inputs that depend on nothing: q (warp 0, 8 lanes a head), k and v (8 lanes, all four times)
    uint4 qraw[2], kraw[2], vraw[2], wq[2], wk[2];
    if (warp == 0) {
        load16(p.q + ((int64_t)t * p.heads + g * kGroup + sub) * kHeadDim, lj, qraw);
        load16_weights(p.qw, lj, wq);
    }
    const int64_t kv = ((int64_t)t * G + g) * kHeadDim;
    load16(p.k + kv, lj, kraw);
    load16(p.v + kv, lj, vraw);
    load16_weights(p.kw, lj, wk);
    const int pos = p.positions[t], row = t, rope_exp = *p.rope_exp;
    const bool active = pos != -1;
    uint32_t e = q4_fault(p, pos, row);
    const int n = active && !e ? pos / U::kPiece + 1 : 0;  // pieces
    int bad = 0;
    if (n) prefetch_rope(p, pos, threadIdx.x);
    for (int i = threadIdx.x; i * U::kPerPage < n; i += blockDim.x) {
        const int id = page_of(p.table, p.pages, row, i);
        bad |= id < 0 || id >= p.num_pages;
    }
    if (__syncthreads_or(bad)) e = PKV_DEVERR_PAGE;
    if (!active || e) {  // (the same for the whole cluster)
        if (rank == 0) {
            uint4* out = reinterpret_cast<uint4*>(p.out + ((int64_t)t * p.heads + g * kGroup) * kHeadDim);
            if (threadIdx.x < kGroup * kHeadDim / 8) out[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
            if (e && g == 0 && threadIdx.x == 0) atomicOr(p.err, e);
        }
        return;
    }

    // this warp's pieces first, first + step, ...; the copies of the first stages
    const int step = cs * U::kWarps, first = warp * cs + rank;
    int issued = first;
    auto issue = [&](int st) {  // (one lane)
        const int page = page_of(p.table, p.pages, row, issued / U::kPerPage);
        const uint32_t bytes = min((pos - issued * U::kPiece) / kQ4Block + 1, U::kBlocks) * kQ4BlockBytes;
        mbar_arrive_expect_tx(bars + 8 * st, bytes);
        bulk_copy_g2s(smem_u32(ring) + st * U::kPieceBytes, p.data + q4_block(page, G, g, issued % U::kPerPage * U::kPiece), bytes, bars + 8 * st);
    };
    for (int st = 0; st < kUnitStages && issued < n; ++st, issued += step)
        if (lane == 0) issue(st);

    const int64_t at = (int64_t)pos * kRopeHalf;
    if (warp == 0) {
        float x[16], y[16];
        uint32_t h[8], hl[8];
        unpack16(qraw[0], qraw[1], x);
        norm_rope_q16<kFullRot>(x, wq, p.rope_hi + at, p.eps, lane, p.rot, y);
        const float mul = q4_query(y, p.k_scale, h, hl);
        store_query(sQ + 2 * sub * kHeadDim, lj, h, hl);
        if (lj == 0) sMul[sub] = mul;
    }
    const bool owner = first < n && (n - 1 - first) % step == 0;  // this warp has the last piece
    float xn[16];      // lanes of sub 0 and 1: the new k, of 2 and 3: v
    uint32_t bits[8];  // the same as bf16
    if (owner) {
        norm_rope_k_paired<kFullRot>(kraw, wk, p.rope_hi + at, p.rope_lo + at, p.eps2, rope_exp, lane, p.rot, xn, bits);
        if (sub >= 2) {
            unpack16(vraw[0], vraw[1], xn);
            bits[0] = vraw[0].x, bits[1] = vraw[0].y, bits[2] = vraw[0].z, bits[3] = vraw[0].w;
            bits[4] = vraw[1].x, bits[5] = vraw[1].y, bits[6] = vraw[1].z, bits[7] = vraw[1].w;
        }
    }
    __syncthreads();

    const Q4Lane L(lane);
    Q4State S;
    S.open(L, sQ, sMul);
    bool ok = true;
    int i = 0;
    for (int j = first; j < n; j += step, ++i) {
        const int st = i % kUnitStages;
        if (__any_sync(kFull, !mbar_wait(bars + 8 * st, (i / kUnitStages) & 1, wait_ns))) {
            ok = false;
            break;
        }
        uint8_t* sb = ring + st * U::kPieceBytes;
        if (j == n - 1) {  // the new position into the staged piece (sub 0, 2) and into the pool (1, 3)
            const int s = pos % kPageSize;
            uint8_t* pool = p.data + q4_block(page_of(p.table, p.pages, row, j / U::kPerPage), G, g, s);
            q4_store((sub & 1) ? pool : sb + s % U::kPiece / kQ4Block * kQ4BlockBytes, sub >= 2, s % kQ4Block, xn, bits,
                     sub < 2 ? p.k_inv6 : p.v_inv6, sub < 2 ? p.k_inv : p.v_inv, lj, true);
            __syncwarp();
        }
        S.chunk<U::kBlocks>(L, sb, pos + 1 - j * U::kPiece);
        __syncwarp();
        if (issued < n) {
            if (lane == 0) issue(st);
            issued += step;
        }
    }
    if (!ok) {  // the awaited copy is late: report, and let the copies in flight land
        if (lane == 0) {
            atomicOr(p.err, PKV_DEVERR_TIMEOUT);
            const int all = (issued - first) / step;
            for (int k = max(0, all - kUnitStages); k < all; ++k)
                mbar_wait(bars + 8 * (k % kUnitStages), (k / kUnitStages) & 1, kWaitLimitNs);
        }
        __syncwarp();
    }

    // ---- the warps' sums into their own ring (nothing in flight there any more); one warp a head joins the CTA's,
    // and the first CTA's those of the cluster
    float* part = reinterpret_cast<float*>(ring);
    if (first < n) {
        float* pa = part + L.c * kHeadDim + 16 * L.r;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const float2 y = S.pair(k), z = S.pair(k + 1);
            *reinterpret_cast<float4*>(pa + 2 * k) = make_float4(y.x, y.y, z.x, z.y);
        }
        if (L.r == 0) sML[warp * kGroup + L.c] = make_float2(S.m, S.sum());
    }
    __syncthreads();
    const int h = warp;
    float M = -CUDART_INF_F, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    float4* joined = reinterpret_cast<float4*>(sbase + 4 * (h * kHeadDim + 4 * lane));  // warp 0's part, of this warp's head
    if (h < kGroup && rank < n) {  // (warp w has a part if piece w cs + rank is there)
        float2 ml[U::kWarps];
#pragma unroll
        for (int w = 0; w < U::kWarps; ++w) {
            ml[w] = w * cs + rank < n ? sML[w * kGroup + h] : make_float2(-CUDART_INF_F, 0.f);
            M = fmaxf(M, ml[w].x);
        }
#pragma unroll
        for (int w = 0; w < U::kWarps; ++w) {
            if (w * cs + rank >= n) break;
            const float f = exp2f(ml[w].x - M);  // (NaN sums: M is theirs or above; f * NaN or NaN)
            const float4 x = joined[w * (U::kRing / 16)];
            sum += f * ml[w].y;
            acc[0] += f * x.x;
            acc[1] += f * x.y;
            acc[2] += f * x.z;
            acc[3] += f * x.w;
        }
    }
    if (cs > 1) {
        __syncwarp();  // every lane has read the warps' maxima and sums of this head
        if (h < kGroup) {
            *joined = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (lane == 0) sML[h] = make_float2(M, sum);
        }
        cluster_sync();
        if (h < kGroup && rank == 0) {
            const int parts = min(n, cs);  // the CTAs that have one, its maximum and sum a lane
            float2 ml = make_float2(-CUDART_INF_F, 0.f);
            if (lane < parts) ml = ld_cluster_f32x2(cluster_map(base + U::kML + 8 * h, lane));
            M = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            const float f = lane < parts ? exp2f(ml.x - M) : 0.f;
            sum = f * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
            constexpr int kBatch = 4;
            for (int k0 = 0; k0 < parts; k0 += kBatch) {
                float4 x[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    x[k] = ld_cluster_f32x4(cluster_map(base + 4 * (h * kHeadDim + 4 * lane), min(k0 + k, parts - 1)));
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float fk = __shfl_sync(kFull, f, min(k0 + k, parts - 1));
                    if (k0 + k < parts) {
                        acc[0] += fk * x[k].x;
                        acc[1] += fk * x[k].y;
                        acc[2] += fk * x[k].z;
                        acc[3] += fk * x[k].w;
                    }
                }
            }
        }
    }
    if (h < kGroup && rank == 0) {
        const float inv = v_scale / sum;
        const float y[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
        *reinterpret_cast<uint2*>(p.out + ((int64_t)t * p.heads + g * kGroup + h) * kHeadDim + 4 * lane) = pack4(y);
    }
    if (cs > 1) cluster_sync();  // the others' shared memory is read until here
}

// =====================================================================================
// the decode call
// =====================================================================================
Q4Plan make_q4_plan(const pkv_pool* pool, int rows)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    Q4Plan pl;
    pl.ctas = std::min(pool->ctas_override > 0 ? pool->ctas_override : pool->num_sms, kQ4MostCtas);  // (Q4Split's 32 bits)
    const size_t units = (size_t)rows * pool->cfg.kv_heads, slots = units + (size_t)pl.ctas * kQ4Warps;
    const size_t heads = (size_t)rows * pool->cfg.heads;
    size_t off = 0;
    pl.off_len = off, off = up(off + sizeof(int32_t) * rows);
    pl.off_prefix = off, off = up(off + sizeof(int32_t) * (rows + 1));
    pl.off_qhat = off, off = up(off + sizeof(__half) * 2 * heads * kHeadDim);  // (and the remainders)
    pl.off_qmul = off, off = up(off + sizeof(float) * heads);
    pl.off_po = off, off = up(off + sizeof(float) * slots * kGroup * kHeadDim);
    pl.off_plse = off, off = up(off + sizeof(float) * slots * kGroup);
    pl.total = off;
    return pl;
}

using Q4UnitHalf = Q4Unit<2>;
using Q4UnitPage = Q4Unit<4>;

// f(kernel, threads, shared memory) of a form.
template <class F>
static cudaError_t with_unit_kernel(bool whole_pages, bool full, F f)
{
    if (whole_pages)
        return f(full ? q4_unit_kernel<Q4UnitPage, true> : q4_unit_kernel<Q4UnitPage, false>, 32 * Q4UnitPage::kWarps,
                 Q4UnitPage::kAlloc);
    return f(full ? q4_unit_kernel<Q4UnitHalf, true> : q4_unit_kernel<Q4UnitHalf, false>, 32 * Q4UnitHalf::kWarps,
             Q4UnitHalf::kAlloc);
}

static bool full_rotation(const pkv_pool* pool) { return pool->cfg.rotary_dim <= 0 || pool->cfg.rotary_dim == kHeadDim; }

cudaError_t configure_q4(pkv_pool* pool)
{
    cudaError_t rc = cudaFuncSetAttribute(q4_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Q4Smem::kAlloc);
    for (int whole = 0; whole < 2 && rc == cudaSuccess; ++whole)
        rc = with_unit_kernel(whole, full_rotation(pool), [&](auto kernel, int threads, int smem) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            for (int k = 0; k < 5; ++k) {  // clusters of 2^k CTAs that the device holds at a time
                cudaLaunchAttribute attr[1];
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = 1u << k;
                attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(1u << k);
                cfg.blockDim = dim3(threads);
                cfg.dynamicSmemBytes = smem;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                if (cudaOccupancyMaxActiveClusters(&pool->q4_clusters[whole][k], kernel, &cfg) != cudaSuccess) {
                    cudaGetLastError();  // (a size that the device does not have)
                    pool->q4_clusters[whole][k] = 0;
                }
            }
            return cudaSuccess;
        });
    return rc;
}

// How q4_unit_kernel takes a call: its form and the CTAs (2^k, a cluster) of each unit; cs 0: the call goes through the
// split attention.
struct Q4UnitChoice {
    bool whole_pages;
    int cs;
};

// The kernel's life is 4.5 to 5.5 us, 0.6 us more in a cluster, and 1.3 to 1.8 us for every further round of its warps'
// pieces; the split attention's is 8 to 11 us and the time of its bytes, and more where few units are cut into many
// pieces.  Measured (us; half pages / whole pages, CTAs a unit in brackets / split; 8 kv heads unless named):
//   rows that one CTA takes in one round: 8 of 1-128 5.0 / 5.8 / 9.1, 8 of 400 6.1 / 5.5 / 10.4, 16 of 100-300 6.1 / 5.6 / 10.7
//   in one round of a cluster, about one CTA an SM: 1 of 700 5.7 [4] / 6.4 [2] / 8.9, 24 of 1-640 (2 heads) 6.4 [4] /
//     6.8 [2], 1 of 1500 (1 head) 5.7 [8] / 6.2 [4] / 8.7; more CTAs than that: 4 of 2000 7.6 [8] / 6.8 [4] / 11.6
//   longer: 1 of 4000 7.1 [8] / 6.7 [8] / 11.2, of 16000 13.9 [8] / 11.8 [8] / 18.0, of 32000 20.2 [16] / 18.7 [8] / 20.4, 2
//     of 16000 22.8 [4] / 18.5 [4] / 18.2, 4 of 8000 14.0 [4] / 12.2 [4] / 17.5, 16 of 500-1500 10.6 / 9.4 / 14.5, of 3000
//     18.1 / 16.0 / 20.5; clusters beyond what the device holds at a time take turns: 4 of 8000 24.2 [8]
//   longest: 1 of 40000 22.7 [8] / 23.4, of 60000 32.5 [8] / 26.9, 8 of 10000 24.5 [2] / 25.7, 16 of 200-5000 22.1 / 22.0; in
//     clusters of 16 (1 head) 1 of 80000 22.4 / 38.8, of 130000 33.1 / 53.2, of 300000 70.8 / 57.7
//   more units than SMs: 32 of 500-1500 15.1 / 17.4 / 17.7, 64 of 1-640 15.6 / 21.4 / 16.9
// The rows' lengths are not known here: `pages`, the table's width, stands for the longest, so that short rows under a
// wide table go through the split attention (8 rows of 1-128 under 640 pages 9.3 us instead of 5.0, 16 of 500-1500 14.6
// instead of 9.4; one row of 700 5.9).  A grid size set by pkv_set_ctas is the split attention's.
static Q4UnitChoice q4_unit_choice(const pkv_pool* pool, int rows, int64_t pages)
{
    constexpr int kWarps = Q4UnitPage::kWarps, kRounds = 10, kRoundsOf16 = 16, kRoundsInTurn = 6;
    const int64_t units = (int64_t)rows * pool->cfg.kv_heads, sms = pool->num_sms;
    const int *half = pool->q4_clusters[0], *whole = pool->q4_clusters[1];
    if (pool->ctas_override > 0 || units > 4 * sms) return {false, 0};
    if (units <= whole[0]) {
        if (2 * pages <= kWarps) return {false, 1};
        if (pages <= kWarps) return {true, 1};
        int k = 1;
        while (k < 3 && (kWarps << k) < 2 * pages) ++k;
        if ((kWarps << k) >= 2 * pages && units <= half[k] && 3 * (units << k) <= 4 * sms) return {false, 1 << k};
        k = 0;
        while (k < 4 && units <= whole[k + 1] && (kWarps << k) < pages) ++k;
        return {true, pages <= ((k < 4 ? kRounds : kRoundsOf16) * kWarps) << k ? 1 << k : 0};
    }
    const int64_t turns = half[0] > 0 ? (units + half[0] - 1) / half[0] : kRoundsInTurn + 1;
    return {false, turns * ((2 * pages + kWarps - 1) / kWarps) <= kRoundsInTurn ? 1 : 0};
}

static cudaError_t launch_q4_units(const pkv_pool* pool, const Q4AppendParams& ap, Q4UnitChoice c, cudaStream_t s)
{
    return with_unit_kernel(c.whole_pages, full_rotation(pool), [&](auto kernel, int threads, int smem) {
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)c.cs;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(ap.tokens * ap.kv_heads * c.cs));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, kernel, ap, pool->v_scale, pool->wait_ns, c.cs);
    });
}

cudaError_t launch_q4_decode(pkv_pool* pool, const StepArgs& a, const Q4Plan& plan, cudaStream_t s)
{
    Q4AppendParams ap = append_params(pool);
    ap.q = static_cast<const __nv_bfloat16*>(a.q);
    ap.k = static_cast<const __nv_bfloat16*>(a.k);
    ap.v = static_cast<const __nv_bfloat16*>(a.v);
    ap.qw = static_cast<const __nv_bfloat16*>(a.q_norm_w);
    ap.kw = static_cast<const __nv_bfloat16*>(a.k_norm_w);
    ap.positions = a.step_positions;
    ap.table = a.table;
    ap.tokens = ap.rows = a.rows;
    ap.pages = a.pages;
    ap.q_hat = reinterpret_cast<__half*>(a.ws + plan.off_qhat);
    ap.q_mul = reinterpret_cast<float*>(a.ws + plan.off_qmul);
    ap.tok_len = reinterpret_cast<int32_t*>(a.ws + plan.off_len);
    ap.out = static_cast<__nv_bfloat16*>(a.out);
    cudaError_t rc;
    const bool timed = pool->timer_on != 0;
    const int slot = timed ? (int)(pool->timer_count.fetch_add(1) % kTimerSlots) : 0;
    if (const Q4UnitChoice c = q4_unit_choice(pool, a.rows, a.pages); c.cs) {
        if (timed && (rc = cudaEventRecord(pool->ev_start[slot], s)) != cudaSuccess) return rc;
        if ((rc = launch_q4_units(pool, ap, c, s)) != cudaSuccess) return rc;
        return timed ? cudaEventRecord(pool->ev_stop[slot], s) : cudaSuccess;
    }
    const int items = (ap.kv_heads + 3) / 4 + ap.kv_heads;
    rc = launch_dependent(ap.rot == kHeadDim ? q4_prep_kernel<true> : q4_prep_kernel<false>, (unsigned)a.rows,
                                      32 * std::min(items, 16), 0, s, ap);
    if (rc != cudaSuccess) return rc;

    Q4AttnParams p;
    p.q_hat = ap.q_hat;
    p.q_mul = ap.q_mul;
    p.positions = a.step_positions;
    p.tok_len = ap.tok_len;
    p.table = a.table;
    p.data = ap.data;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.part_o = reinterpret_cast<float*>(a.ws + plan.off_po);
    p.part_lse = reinterpret_cast<float*>(a.ws + plan.off_plse);
    p.prefix = reinterpret_cast<int32_t*>(a.ws + plan.off_prefix);
    p.err = pool->err;
    p.ntok = a.rows;
    p.pages = a.pages;
    p.num_pages = pool->num_pages;
    p.max_seq = pool->cfg.max_seq;
    p.heads = pool->cfg.heads;
    p.kv_heads = pool->cfg.kv_heads;
    p.v_scale = pool->v_scale;
    p.wait_ns = pool->wait_ns;
    if (timed && (rc = cudaEventRecord(pool->ev_start[slot], s)) != cudaSuccess) return rc;
    // (timed: the attention alone between the events)
    rc = launch_dependent(q4_attn_kernel, (unsigned)plan.ctas, 32 * kQ4Warps, Q4Smem::kAlloc, s, p, !timed);
    if (rc != cudaSuccess) return rc;
    if (timed && (rc = cudaEventRecord(pool->ev_stop[slot], s)) != cudaSuccess) return rc;

    Q4CombineParams cp;
    cp.prefix = p.prefix;
    cp.tok_len = p.tok_len;
    cp.part_o = p.part_o;
    cp.part_lse = p.part_lse;
    cp.out = p.out;
    cp.ntok = a.rows;
    cp.heads = p.heads;
    cp.kv_heads = p.kv_heads;
    cp.warps = plan.ctas * kQ4Warps;
    const unsigned units = (unsigned)(a.rows * p.kv_heads), pieces = cp.warps / units;
    // pieces of a unit, measured with 4 / 8 / 16 warps a head (us a call): 9 (24 rows of 8000) 44.3 / 44.7 / 46.9,
    // 28 (8 of 36000) 58.8 / 58.2 / 59.3, 114 (2 of 65000) 41.3 / 36.7 / 34.8, 228 (1 of 130000) 50.3 / 41.3 /
    // 36.9; and less than six (64 rows): one warp a head 41.0, 4 42.6
    if (units >= 2u * plan.ctas) return launch_dependent(q4_combine_kernel<kGroup, 1>, units, 32 * kGroup, 0, s, cp);
    return pieces < 20    ? launch_dependent(q4_combine_kernel<1, 4>, kGroup * units, 32 * 4, 0, s, cp)
           : pieces < 100 ? launch_dependent(q4_combine_kernel<1, 8>, kGroup * units, 32 * 8, 0, s, cp)
                          : launch_dependent(q4_combine_kernel<1, 16>, kGroup * units, 32 * 16, 0, s, cp);
}

// =====================================================================================
// q4_read_kernel: a warp takes kQuads times 4 kv heads of one token, 8 lanes a head, lane j
// the dims 8j .. 8j + 7 and 64 + 8j .. of k and v (as the append's lanes): 16-byte stores.
// Bound by its stores: 33800 tokens of 8 heads, 39 MB read and 138 MB written, in 31 us, 5.7
// TB/s, at 0.58 of the issue slots; 8 heads a warp share a token's address arithmetic.  (Several
// tokens a warp in turn: 33 to 35 us.)  Few tokens are one launch and four trips to memory.
// =====================================================================================
struct Q4ReadParams {
    const uint8_t* data;
    const int32_t* positions;
    const int32_t* prow;
    const int32_t* table;
    __nv_bfloat16* k;
    __nv_bfloat16* v;
    uint32_t* err;
    int64_t token_stride, head_stride;
    int tokens, rows, pages, num_pages, max_seq, kv_heads;
    float k_scale, v_scale;
};

constexpr int kQ4ReadWarps = 4;

template <int kQuads>
__global__ void __launch_bounds__(32 * kQ4ReadWarps) q4_read_kernel(Q4ReadParams p)
{
    const int lane = threadIdx.x & 31, j = lane & 7, groups = (p.kv_heads + 4 * kQuads - 1) / (4 * kQuads);
    const int item = blockIdx.x * kQ4ReadWarps + (threadIdx.x >> 5), t = item / groups;
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.tokens) return;
    const int g0 = 4 * kQuads * (item - t * groups) + (lane >> 3);  // this lane's heads: g0, g0 + 4, ...
    const int pos = p.positions[t];
    const int row = p.prow ? p.prow[t] : t;
    uint32_t e = 0;
    int page = -1;
    if (pos != -1) {
        if (row < 0 || row >= p.rows) {
            e = PKV_DEVERR_ROW;
        } else if (pos < 0 || pos >= p.max_seq || pos / kPageSize >= p.pages) {
            e = PKV_DEVERR_POSITION;
        } else {
            page = page_of(p.table, p.pages, row, pos / kPageSize);
            if (page < 0 || page >= p.num_pages) e = PKV_DEVERR_PAGE, page = -1;
        }
    }
    if (e && lane == 0) atomicOr(p.err, e);
    uint32_t word[kQuads][2][2] = {}, scale[kQuads][2][2] = {};
    if (page >= 0) {
        const int i = pos % kQ4Block;
        const uint8_t* block = p.data + q4_block(page, p.kv_heads, g0, pos % kPageSize);
        const uint8_t* codes = block + q4_code_row(i, 4 * j);
        const int other = q4_code_row(i, 32 + 4 * j) - q4_code_row(i, 4 * j);  // 32 or -32
        const uint8_t *ks = block + q4_k_scale(i, j >> 1), *vs = block + q4_v_scale(i, j >> 1);
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            if (g0 + 4 * q >= p.kv_heads) break;
            const int at = 4 * q * kQ4PageBytes;
            word[q][0][0] = *reinterpret_cast<const uint32_t*>(codes + at);
            word[q][0][1] = *reinterpret_cast<const uint32_t*>(codes + at + other);
            word[q][1][0] = *reinterpret_cast<const uint32_t*>(codes + at + kQ4VCodes);
            word[q][1][1] = *reinterpret_cast<const uint32_t*>(codes + at + kQ4VCodes + other);
            scale[q][0][0] = ks[at];  // (group g + 4: 8 bytes on for K, 64 for V)
            scale[q][0][1] = ks[at + 8];
            scale[q][1][0] = vs[at];
            scale[q][1][1] = vs[at + 64];
        }
    }
    __nv_bfloat16* dst[2] = {p.k + t * p.token_stride + g0 * p.head_stride + 8 * j,
                             p.v + t * p.token_stride + g0 * p.head_stride + 8 * j};
#pragma unroll
    for (int q = 0; q < kQuads; ++q) {
        if (g0 + 4 * q >= p.kv_heads) break;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t c[4], r[4];
                q4_unpack(word[q][which][h], c);
                const float s = (which ? p.v_scale : p.k_scale) *
                                __half2float(__ushort_as_half((unsigned short)e4m3x2_half2(scale[q][which][h])));
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // code * scale has 6 bits: exact in bf16
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[k]));
                    r[k] = pack_bf16(__float2bfloat16_rn(f.x * s), __float2bfloat16_rn(f.y * s));
                }
                __stcs(reinterpret_cast<uint4*>(dst[which] + 64 * h), make_uint4(r[0], r[1], r[2], r[3]));
            }
            dst[which] += 4 * p.head_stride;
        }
    }
}

cudaError_t launch_q4_read(const pkv_pool* pool, const int32_t* positions, const int32_t* prow, const int32_t* table,
                           int tokens, int rows, int pages, void* k, void* v, int64_t token_stride, int64_t head_stride,
                           cudaStream_t s)
{
    Q4ReadParams p;
    p.data = static_cast<const uint8_t*>(pool->q4);
    p.positions = positions;
    p.prow = prow;
    p.table = table;
    p.k = static_cast<__nv_bfloat16*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.err = pool->err;
    p.token_stride = token_stride;
    p.head_stride = head_stride;
    p.tokens = tokens;
    p.rows = rows;
    p.pages = pages;
    p.num_pages = pool->num_pages;
    p.max_seq = pool->cfg.max_seq;
    p.kv_heads = pool->cfg.kv_heads;
    p.k_scale = pool->k_scale;
    p.v_scale = pool->v_scale;
    // few tokens: 4 heads a warp, for the shorter chain; many: 8 (8 heads, us with 4 / 8: 77 tokens 1.7 / 2.0, 2048
    // 2.9 / 3.0, 4096 4.7 / 4.3, 16384 17.2 / 16.3)
    const int quads = (p.kv_heads + 3) / 4, per = quads > 1 && (int64_t)tokens * quads >= 32 * (int64_t)pool->num_sms ? 2 : 1;
    const int64_t items = (int64_t)tokens * ((quads + per - 1) / per);
    const unsigned grid = (unsigned)((items + kQ4ReadWarps - 1) / kQ4ReadWarps);
    return launch_dependent(per == 1 ? q4_read_kernel<1> : q4_read_kernel<2>, grid, 32 * kQ4ReadWarps, 0, s, p);
}

}  // namespace pkv
