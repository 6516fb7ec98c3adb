// pmqa_cache.cuh -- what the kernels over the paged 8-bit K/V cache share: the
// device view of a problem with its clamped request bounds, the walk over
// (request, kv head, row block, token tile) items, fp8 conversions and the
// warp-level matrix product.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/pmqa.h"
#include "pmqa_mla_ptx.cuh"

namespace pmqa {
namespace cache {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMaxGroup = 128;       // query heads per kv head
constexpr int kMaxBlock = 1024;      // tokens per block
constexpr int kMaxContext = 0x7FFF0000;  // slots rounded up to tiles stay in 32 bits
constexpr int kMaxCtas = 512;        // CTAs of the short-row attention (workspace parts: 2 each)
constexpr int kMaxWide = 320;        // the same with 32 rows a block (8 and 16: kMaxCtas)
constexpr int kPromptRows = 256;     // packed rows per CTA of the many-row attention
constexpr int kMaxParts = 160;       // its CTAs where contexts are cut (workspace parts: 1 each)
constexpr size_t kStatusBytes = 256;

// Device view of a pmqa_cache_problem.
struct View {
    uint8_t *k, *v;           // e4m3 [num_blocks, H, P, D]
    float *ks, *vs;           // [num_blocks, H]
    const int32_t *bt;        // [bs, W]
    const int32_t *ctx;       // [bs]
    const int32_t *row_begin; // [bs + 1] or null
    int bs, H, D, P, W, rows, max_rows;
    uint32_t p_inv;           // min(2^32 - 1, floor(2^32 / P))
    long long nb;
    uint32_t *status;

    // t / P for t >= 0: the product is below the quotient by less than 1
    __device__ __forceinline__ int page_of(int t) const
    {
        const int q = (int)__umulhi((uint32_t)t, p_inv);
        return q + ((uint32_t)(q + 1) * (uint32_t)P <= (uint32_t)t ? 1 : 0);
    }
};

// A request's rows and context, clamped to what the arrays can hold; what had
// to be clamped is recorded as PMQA_DEV_BAD_CONTEXT by the thread with `tell`.
struct Request {
    int r0, n, ctx;
};

__device__ __forceinline__ int clamp_ctx(const View &a, int i, bool tell)
{
    const int c = __ldg(a.ctx + i);
    const long long cap = (long long)a.P * a.W;
    const int hi = cap < kMaxContext ? (int)cap : kMaxContext;
    if (tell && (c < 0 || c > hi))
        atomicOr(a.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
    return min(max(c, 0), hi);
}

__device__ __forceinline__ Request load_request(const View &a, int i, bool tell)
{
    Request q;
    const int b = __ldg(a.row_begin + i), e = __ldg(a.row_begin + i + 1);
    q.r0 = min(max(b, 0), a.rows);
    q.n = min(min(max(e, q.r0), a.rows) - q.r0, a.max_rows);
    if (tell && (q.r0 != b || q.n != e - b))
        atomicOr(a.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
    q.ctx = clamp_ctx(a, i, tell);
    return q;
}

// What has to be clamped in any request, for kernels that do not look at all of them;
// called by one whole CTA. Not inlined: in the kernels' bodies the loop costs registers
// (the many-row attention spills, prompt chunks 479 us instead of 414; append of 15730
// rows 26.9 us instead of 23.1).
inline __device__ __noinline__ void report_requests(const View &a)
{
    for (int i = threadIdx.x; i < a.bs; i += blockDim.x)
        load_request(a, i, true);
}

// e4m3 pairs (bytes 0-1 and 2-3 of w) to f16 pairs: exact.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// D[16 x 8] += A[16 x 16] B[16 x 8], f16 inputs, fp32 accumulation.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held as pairs (row lane / 4,
// columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The power of two s = 2^ceil(log2(a / 448)), at least 2^-100, so that a / s
// <= 448, the largest e4m3 value; a finite and not negative. With a = m 2^e,
// m in [1, 2), and 448 = 1.75 * 2^8 the exponent is e - 8 or e - 7.
__device__ __forceinline__ float pow2_scale(float a)
{
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 127;  // a subnormal a gives -127: below the floor all the same
    const int s = e - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(s, -100) + 127) << 23);
}

// Round to nearest even e4m3 with saturation (NaN stays NaN).
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d)
{
    return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
}

// A bf16 value of at most 2^8 as the sum of an e4m3 and an e5m2 value, for products of
// kind::f8f6f4 (where the two operands may have different types). The first leaves a
// remainder of at most 8 units of the value's last bit while the value is 2^-6 or more:
// three bits, which e5m2 has, down to 2^-16. Below, where e4m3's step stays 2^-9,
// the remainder of at most 2^-10 is off by up to 2^-14. With the largest value of a row
// scaled into [2^7, 2^8): exact for values from 2^-13 of it on, off by at most 2^-21
// of it below. (A second e4m3 value of the same cost ends at 2^-9 and 2^-17.)
__device__ __forceinline__ uint32_t f32x4_to_e5m2x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ void split_terms(float a, float b, float c, float d, uint32_t &first, uint32_t &second)
{
    first = f32x4_to_e4m3x4(a, b, c, d);
    float h0, h1, h2, h3;
    e4m3x2_to_f32x2(first & 0xFFFFu, h0, h1);
    e4m3x2_to_f32x2(first >> 16, h2, h3);
    second = f32x4_to_e5m2x4(a - h0, b - h1, c - h2, d - h3);
}

// Instruction descriptor of kind::f8f6f4, bits 7-9 and 10-12: the type of A and of B.
constexpr uint32_t kIdescAE5m2 = 1u << 7, kIdescBE5m2 = 1u << 10;

// ------------------------------------------------------------- walk over items
//
// Item = (request i, kv head h, row block b, tile t of TILE tokens), in that
// order with t fastest; request i has H * B_i * T_i of them, T_i =
// max(1, ceil(ctx_i / TILE)) and B_i = ceil(n_i * group / ROWS); a request with
// fewer than `least` or more than `most` query rows (n_i * group) has none.
// With ROWS = 0 the rows are not cut (B_i = 1) and T_i = ceil(ctx_i / TILE).
// PAD more items without work follow each context's tiles: what loading its rows
// and writing its result costs, so that CTAs with many short contexts get less.
// CTA c of C takes the items [c N / C, (c + 1) N / C).
struct Walk {
    int i, h, b, t;       // current item
    int T, B;             // tiles and row blocks of request i
    Request q;

    template <int TILE, int ROWS, int PAD>
    __device__ __forceinline__ static long long items(const View &a, const Request &q, int group,
                                                      int least, int most, int &T, int &B)
    {
        const bool in = q.n * group >= least && q.n * group <= most;
        T = max(ROWS > 0 ? 1 : 0, (q.ctx + TILE - 1) / TILE);
        if constexpr (ROWS > 0)
            B = in ? (q.n * group + ROWS - 1) / ROWS : 0;
        else
            B = in ? 1 : 0;
        return (long long)a.H * B * (T > 0 ? T + PAD : 0);
    }

    // Step to the next item; false past the last request.
    template <int TILE, int ROWS, int PAD>
    __device__ __forceinline__ bool next(const View &a, int group, int least, int most)
    {
        if (++t < T)
            return true;
        t = 0;
        if (++b < B)
            return true;
        b = 0;
        if (++h < a.H)
            return true;
        h = 0;
        while (++i < a.bs) {
            q = load_request(a, i, false);
            if (items<TILE, ROWS, PAD>(a, q, group, least, most, T, B) > 0)
                return true;
        }
        return false;
    }
};

// What every CTA finds out at its start: its item range and the first item.
struct Range {
    long long x0, x1, total;
    long long C;       // CTAs that take items
    int i;             // request of item x0
    long long before;  // items before request i
};

// Called by all THREADS threads of the CTA. Two passes over the requests: the
// number of items, then the request that holds item x0. `least_items`: no CTA
// takes fewer items than this while there are any left; `join_cost`: what it costs
// to join one more part of a (request, head, row block), in items (0: nothing).
// With T items and k CTAs each such context takes T / k + k join_cost, least at
// k = sqrt(T / join_cost): so many CTAs per context at most, on average.
template <int TILE, int ROWS, int PAD, int THREADS>
__device__ __forceinline__ void find_range(const View &a, int group, int least, int most,
                                           int least_items, float join_cost, Range &out,
                                           Walk &w)
{
    __shared__ long long s_sum[THREADS / 32], s_pairs[THREADS / 32];
    __shared__ Range s_range;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long sum = 0, pairs = 0;
    int T, B;
    for (int i = tid; i < a.bs; i += THREADS) {
        const Request q = load_request(a, i, blockIdx.x == 0);
        sum += Walk::items<TILE, ROWS, PAD>(a, q, group, least, most, T, B);
        pairs += (long long)a.H * B;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(kFull, sum, o);
        pairs += __shfl_xor_sync(kFull, pairs, o);
    }
    if (lane == 0) {
        s_sum[warp] = sum;
        s_pairs[warp] = pairs;
    }
    __syncthreads();
    long long total = 0;
    pairs = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
        total += s_sum[k];
        pairs += s_pairs[k];
    }
    long long want = (total + least_items - 1) / least_items;
    if (join_cost > 0.0f)
        want = min(want, max(pairs, (long long)sqrtf((float)total * (float)pairs / join_cost)));
    const long long C = want < (long long)gridDim.x ? want : (long long)gridDim.x;
    const long long c = blockIdx.x;
    const long long x0 = c < C ? c * total / C : total, x1 = c < C ? (c + 1) * total / C : total;
    long long base = 0;
    for (int i0 = 0; x0 < x1 && i0 < a.bs; i0 += THREADS) {
        const int i = i0 + tid;
        long long n = 0;
        if (i < a.bs) {
            const Request q = load_request(a, i, false);
            n = Walk::items<TILE, ROWS, PAD>(a, q, group, least, most, T, B);
        }
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o)
                inc += y;
        }
        __syncthreads();
        if (lane == 31)
            s_sum[warp] = inc;
        __syncthreads();
        long long off = base, all = 0;
#pragma unroll
        for (int k = 0; k < THREADS / 32; ++k) {
            if (k < warp)
                off += s_sum[k];
            all += s_sum[k];
        }
        const long long lo = off + inc - n;
        if (n > 0 && lo <= x0 && x0 < lo + n) {
            s_range.i = i;
            s_range.before = lo;
        }
        base += all;
        if (base > x0)
            break;  // the same for every thread
    }
    __syncthreads();
    out.x0 = x0;
    out.x1 = x1;
    out.total = total;
    out.C = C;
    if (x0 < x1) {
        out.i = s_range.i;
        out.before = s_range.before;
        w.i = out.i;
        w.q = load_request(a, w.i, false);
        Walk::items<TILE, ROWS, PAD>(a, w.q, group, least, most, w.T, w.B);
        long long y = x0 - out.before;
        w.t = (int)(y % (w.T + PAD));  // T and above: behind the tiles
        y /= w.T + PAD;
        w.b = (int)(y % w.B);
        w.h = (int)(y / w.B);
    }
}

}  // namespace cache
}  // namespace pmqa
