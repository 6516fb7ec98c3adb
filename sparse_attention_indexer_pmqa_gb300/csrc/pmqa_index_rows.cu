// pmqa_index_rows.cu -- the indexer's cache written and read back:
// pmqa_index_append, pmqa_index_read.
//
// Append: per row one key (layer or RMS norm, rotary, one fp32 scale, 132 bytes into
// the row's slot) and `heads` queries (rotary, a scale each, which goes into the
// head's weight): 384 bytes a query head. Half a warp holds four vectors of 128 values at
// a time, eight values a lane (16-byte loads); rotated pairs meet by shuffles of the packed
// inputs, the four largest values are reduced together. A CTA takes one row, or four
// where rows are many, and forms their angles once for all heads. 15.7 k rows of 64 heads
// (400 MB): 82 us, 72 % of the copy rate; the rest is instructions (102 a vector pair, 56 %
// of the issue slots) and loads that wait between a row's passes. The next pass's loads ahead
// of the work cost more in occupancy than they hid (98 us).
//
// Read: a warp moves 32 rows (8 where there are few), whose places its lanes look up;
// rows of 132 bytes are aligned to 4 bytes only, so a lane moves one word of each row
// (through the read-only path: neighbouring rows share sectors; as loads that are not kept
// 72 us against 56 for 1.3 M rows, 89 % of the copy rate).
#include <algorithm>

#include "pmqa_paged.cuh"

namespace pmqa {
namespace paged {

constexpr int kDimI = 128;       // values of a key or of a query head
constexpr int kRowI = 132;       // bytes of a cached row
constexpr int kIndexThreads = 64;  // the cost of a CTA's start is shared by more CTAs of an SM (128: 88 us, 82)
constexpr float kLeast = 0x1p-100f;

struct IndexArgs {
    View c;
    Rotary r;
    Norm n;
    uint8_t *kv;
    const uint16_t *k, *q;
    const void *w;
    uint8_t *q_out;
    float *w_out;
    long long k_row, q_row, q_head, w_row;
    int heads, w_bf16;
    float w_scale;
};

__device__ __forceinline__ float half_sum(uint32_t mask, float x)
{
#pragma unroll
    for (int k = 8; k > 0; k >>= 1)
        x += __shfl_xor_sync(mask, x, k);
    return x;
}

__device__ __forceinline__ float half_max(uint32_t mask, float x)
{
#pragma unroll
    for (int k = 8; k > 0; k >>= 1)
        x = fmaxf(x, __shfl_xor_sync(mask, x, k));
    return x;
}

// The largest finite |y| of a lane's values (0 or NaN where there is none).
__device__ __forceinline__ float top8(const float (&y)[8])
{
    float top = fabsf(y[0]);
#pragma unroll
    for (int e = 1; e < 7; e += 2)
        top = fmaxf(top, fmaxf(fabsf(y[e]), fabsf(y[e + 1])));
    top = fmaxf(top, fabsf(y[7]));
    if (top == INFINITY) {
        top = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = fmaxf(top, fabsf(y[e]) < INFINITY ? fabsf(y[e]) : 0.0f);
    }
    return top;
}

// Of four vectors of a half warp the largest m, at least 2^-100: that of vector at / 4.
// Each step halves what a lane holds on to: 5 exchanges for four vectors instead of 16,
// and one quotient (15.7 k rows of 64 heads 93 -> 86 us).
__device__ __forceinline__ float largest4(const float (&m)[4], int at)
{
    const bool b8 = at & 8, b4 = at & 4;
    const float x = fmaxf(b8 ? m[2] : m[0], __shfl_xor_sync(kFull, b8 ? m[0] : m[2], 8));
    const float y = fmaxf(b8 ? m[3] : m[1], __shfl_xor_sync(kFull, b8 ? m[1] : m[3], 8));
    float z = fmaxf(b4 ? y : x, __shfl_xor_sync(kFull, b4 ? x : y, 4));
    z = fmaxf(z, __shfl_xor_sync(kFull, z, 2));
    return fmaxf(kLeast, fmaxf(z, __shfl_xor_sync(kFull, z, 1)));
}

// 448 / top to two units of 2^-23, for any finite top >= 2^-100: the approximate division
// takes divisors up to 2^126 (the exact one, a call on its rare path: 99 us instead of 82).
__device__ __forceinline__ float quotient(float top) { return __fdividef(112.0f, top * 0.25f); }

// The rotation of a half warp's vector, whose packed inputs are u.
template <bool PAIRS>
__device__ __forceinline__ void rotate_packed(const Rotary &r, const Turn &turn, uint32_t mask, const uint4 &u, float (&y)[8])
{
    float other[8];
    if (!PAIRS && r.dim) {
        const int from = ((threadIdx.x & 31) + turn.partner) & 31;
        const uint4 p = make_uint4(__shfl_sync(mask, u.x, from), __shfl_sync(mask, u.y, from),
                                   __shfl_sync(mask, u.z, from), __shfl_sync(mask, u.w, from));
        unpack8(p, other);
    }
    turn.apply(PAIRS, y, other);
}

template <bool PAIRS>
__device__ __forceinline__ void write_index_key(const IndexArgs &a, const Turn &turn, uint32_t mask, long long r, uint32_t dst)
{
    const int lane = threadIdx.x & 31, at = lane & 15;
    const uint4 u = load_input(a.k + r * a.k_row + 8 * at);
    float y[8], other[8];
    unpack8(u, y);
    if (a.n.kind != PMQA_NORM_NONE) {
        if (a.n.kind == PMQA_NORM_LAYER) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += y[e];
            const float mean = half_sum(mask, s) * (1.0f / kDimI);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] -= mean;
        }
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s += y[e] * y[e];
        const float f = rsqrtf(half_sum(mask, s) * (1.0f / kDimI) + a.n.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = y[e] * f * (a.n.weight ? __ldg(a.n.weight + 8 * at + e) : 1.0f) +
                   (a.n.bias ? __ldg(a.n.bias + 8 * at + e) : 0.0f);
        if (!PAIRS && a.r.dim) {
            const int from = (lane + turn.partner) & 31;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                other[e] = __shfl_sync(mask, y[e], from);
        }
        turn.apply(PAIRS, y, other);
    } else {
        rotate_packed<PAIRS>(a.r, turn, mask, u, y);
    }
    const float top = fmaxf(kLeast, half_max(mask, top8(y)));
    const uint2 code = codes8(y, quotient(top));
    if (dst == kNoRow)
        return;
    uint32_t *const p = reinterpret_cast<uint32_t *>(a.kv + (unsigned long long)dst * kRowI);
    p[2 * at] = code.x;
    p[2 * at + 1] = code.y;
    if (at == 0)
        p[kDimI / 4] = __float_as_uint(top / 448.0f);
}

template <int ROWS, bool PAIRS>
__global__ void __launch_bounds__(kIndexThreads) index_append_kernel(const __grid_constant__ IndexArgs a)
{
    __shared__ RowTable<ROWS, kDimI> t;
    constexpr int kWarps = kIndexThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, at = lane & 15, warp = tid >> 5;
    const uint32_t mask = 0xFFFFu << (lane & 16);
    const int row0 = blockIdx.x * ROWS;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        cache::report_requests(a.c);
    load_turns(t, a.r);
    load_rows(t, a.c, a.r, row0, a.k != nullptr);
    Turn turn;
#pragma unroll 1
    for (int row = 0; row < ROWS; ++row) {
        if (!t.place[row].valid)
            continue;
        const long long r = row0 + row;
        turn.load(a.r, t.cs[row], at);
        const int step = 2 * kWarps * gridDim.y;
        const uint16_t *const q = a.q + r * a.q_row + 8 * at;
        uint8_t *const out = a.q_out + r * a.heads * kDimI + 8 * at;
        // heads h0, h0 + step, ... of each half of the warp
        for (int hw = 2 * ((int)blockIdx.y * kWarps + warp); hw < a.heads; hw += 4 * step) {
            const int h0 = hw + (lane >> 4), mine = h0 + (at >> 2) * step;
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                u[k] = load_input(q + min(h0 + k * step, a.heads - 1) * a.q_head);
            const bool first = (at & 3) == 0 && mine < a.heads;
            float w = 0.0f;
            if (first) {
                const long long iw = r * a.w_row + mine;
                w = a.w_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.w)[iw] << 16)
                             : static_cast<const float *>(a.w)[iw];
            }
            float y[4][8], m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unpack8(u[k], y[k]);
                rotate_packed<PAIRS>(a.r, turn, kFull, u[k], y[k]);
                m[k] = top8(y[k]);
            }
            const float top = largest4(m, at), f = quotient(top);
            if (first)
                a.w_out[r * a.heads + mine] = w * (top * (1.0f / 448.0f)) * a.w_scale;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint2 code = codes8(y[k], __shfl_sync(kFull, f, (lane & 16) + 4 * k));
                if (h0 + k * step < a.heads)
                    *reinterpret_cast<uint2 *>(out + (h0 + k * step) * kDimI) = code;
            }
        }
    }
    // the keys: a half warp each, after the queries
    if (a.k && blockIdx.y == gridDim.y - 1)
        for (int k = tid >> 4; k < ROWS; k += kIndexThreads / 16) {
            if (!t.place[k].valid)
                continue;
            turn.load(a.r, t.cs[k], at);
            write_index_key<PAIRS>(a, turn, mask, row0 + k, t.place[k].row);
        }
}

struct ReadArgs {
    View c;
    const uint8_t *kv;
    const int32_t *start;
    uint8_t *k;
    float *s;
};

template <int ROWS>
__global__ void __launch_bounds__(128) index_read_kernel(const __grid_constant__ ReadArgs a)
{
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.c.bs; i += 128) {
            const int b = __ldg(a.c.row_begin + i), e = __ldg(a.c.row_begin + i + 1);
            if (b < 0 || e < b || e > a.c.rows)
                atomicOr(a.c.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
        }
    const long long first = ((long long)blockIdx.x * 4 + (threadIdx.x >> 5)) * ROWS;
    if (first >= a.c.rows)
        return;
    // lane k looks up row first + k
    const long long r = first + lane;
    uint32_t src = kNoRow;
    bool mine = false;
    int i = request_of(a.c, (int)first);
    if (lane < ROWS && r < a.c.rows) {
        i = request_from(a.c, i, r);  // the rows behind may belong to later requests
        const int b = __ldg(a.c.row_begin + i);
        mine = r >= b && r < __ldg(a.c.row_begin + i + 1);
        if (mine)
            src = pool_row(a.c, i, (a.start ? (long long)__ldg(a.start + i) : 0ll) + (r - b));
    }
    const uint32_t *const pool = reinterpret_cast<const uint32_t *>(a.kv);
    uint32_t *const out = reinterpret_cast<uint32_t *>(a.k);
    const uint32_t owned = __ballot_sync(kFull, mine);
    uint32_t scale = 0;
    if (src != kNoRow)
        scale = __ldg(pool + (unsigned long long)src * (kRowI / 4) + kDimI / 4);
    constexpr int AHEAD = 8;
#pragma unroll
    for (int k0 = 0; k0 < ROWS; k0 += AHEAD) {
        uint32_t w[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const uint32_t row = __shfl_sync(kFull, src, k0 + k);
            w[k] = row == kNoRow ? 0u : __ldg(pool + (unsigned long long)row * (kRowI / 4) + lane);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (owned >> (k0 + k) & 1u)
                out[(first + k0 + k) * (kDimI / 4) + lane] = w[k];
    }
    if (mine)
        a.s[r] = __uint_as_float(scale);
}

}  // namespace paged
}  // namespace pmqa

using namespace pmqa;
using namespace pmqa::paged;

extern "C" int pmqa_index_append(const pmqa_paged_rows *p, void *kv_cache, const pmqa_index_rows *x,
                                 const pmqa_norm *norm, const pmqa_rotary *rotary, void *ws, size_t ws_bytes,
                                 pmqa_stream_t stream)
{
    int rc = check_rows(p, true, ws, ws_bytes, cache::kStatusBytes);
    if (rc != PMQA_OK)
        return rc;
    IndexArgs a{};
    if (!x || (rc = check_norm(norm, &a.n)) != PMQA_OK || (rc = check_rotary(rotary, kDimI, false, &a.r)) != PMQA_OK)
        return x ? rc : PMQA_ERR_INVALID_ARG;
    if (x->q && (x->heads < 1 || !std::isfinite(x->weight_scale) || (x->weights_row < 0 && p->rows > 1)))
        return PMQA_ERR_INVALID_ARG;
    if (x->q && (x->heads > kMaxHeads || (long long)x->heads * p->rows > 0x7FFFFFFFll))
        return PMQA_ERR_UNSUPPORTED;
    if (p->bs == 0 || p->rows == 0 || (!x->k && !x->q))
        return PMQA_OK;
    if (x->k && (cache::missing(kv_cache, 4) || bad_rows(x->k, 16, p->rows, x->k_row)))
        return PMQA_ERR_INVALID_ARG;
    if (x->q) {
        const long long n = (long long)p->rows * x->heads;
        if (bad_rows(x->q, 16, p->rows, x->q_row, x->heads, x->q_head) || cache::missing(x->q_out, 8) ||
            cache::missing(x->weights, x->weights_bf16 ? 2 : 4) || cache::missing(x->weights_out, 4))
            return PMQA_ERR_INVALID_ARG;
        // weights in place, or apart
        const long long in = ((p->rows > 1 ? (p->rows - 1ll) * x->weights_row : 0ll) + x->heads) * (x->weights_bf16 ? 2 : 4);
        const bool same = x->weights == x->weights_out && !x->weights_bf16 &&
                          (x->weights_row == x->heads || p->rows == 1);
        if (!same && cache::overlap(x->weights, in, x->weights_out, 4 * n))
            return PMQA_ERR_INVALID_ARG;
    }
    a.c = view(p, ws);
    a.kv = static_cast<uint8_t *>(kv_cache);
    a.k = static_cast<const uint16_t *>(x->k);
    a.q = static_cast<const uint16_t *>(x->q);
    a.w = x->weights;
    a.q_out = static_cast<uint8_t *>(x->q_out);
    a.w_out = x->weights_out;
    a.k_row = x->k_row;
    a.q_row = x->q_row;
    a.q_head = x->q_head;
    a.w_row = x->weights_row;
    a.heads = x->q ? x->heads : 0;
    a.w_bf16 = x->weights_bf16 ? 1 : 0;
    a.w_scale = x->weight_scale;
    int sms = 0;
    if ((rc = cache::sm_count(&sms)) != PMQA_OK)
        return rc;
    const int rows = p->rows;
    const cudaStream_t st = cache::cuda(stream);
    // many rows: four to a CTA; few: a row's heads over several CTAs, up to 8 per SM
    const bool many = rows >= 16 * sms, pairs = a.r.interleaved != 0;
    const dim3 grid = many ? dim3((unsigned)((rows + 3ll) / 4)) : dim3(rows, std::max(1, std::min((a.heads + 15) / 16, 8 * sms / rows)));
    auto *const kernel = many ? (pairs ? index_append_kernel<4, true> : index_append_kernel<4, false>)
                              : (pairs ? index_append_kernel<1, true> : index_append_kernel<1, false>);
    kernel<<<grid, kIndexThreads, 0, st>>>(a);
    return cache::code_of(cudaGetLastError());
}

extern "C" int pmqa_index_read(const pmqa_paged_rows *p, const void *kv_cache, const int32_t *start, void *k,
                               float *k_scale, void *ws, size_t ws_bytes, pmqa_stream_t stream)
{
    int rc = check_rows(p, false, ws, ws_bytes, cache::kStatusBytes);
    if (rc != PMQA_OK)
        return rc;
    if (p->bs == 0 || p->rows == 0)
        return PMQA_OK;
    if (cache::missing(kv_cache, 4) || !cache::aligned(start, 4) || cache::missing(k, 16) ||
        cache::missing(k_scale, 4))
        return PMQA_ERR_INVALID_ARG;
    ReadArgs a{view(p, ws), static_cast<const uint8_t *>(kv_cache), start, static_cast<uint8_t *>(k), k_scale};
    int sms = 0;
    if ((rc = cache::sm_count(&sms)) != PMQA_OK)
        return rc;
    const long long rows = p->rows;
    const cudaStream_t st = cache::cuda(stream);
    if (rows >= 32ll * 32 * sms)
        index_read_kernel<32><<<(unsigned)((rows + 127) / 128), 128, 0, st>>>(a);
    else
        index_read_kernel<8><<<(unsigned)((rows + 31) / 32), 128, 0, st>>>(a);
    return cache::code_of(cudaGetLastError());
}
