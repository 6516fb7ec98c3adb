// pmqa_rope.cu -- rotary positions: pmqa_rope and pmqa_rope_frequencies.
//
// Of every head the values begin .. begin + dim turn in pairs (include/pmqa.h,
// pmqa_rotary). Bound by memory: each value is read once and written once. A CTA takes
// one row (four where rows are many), forms the dim / 2 angles once for all heads of both
// tensors, and takes the heads of all its rows in one sequence, whose rows and heads are
// counted up (by divisions 1.6 us more, row by row 71 us instead of 56). A thread keeps
// its 16 values' place in a head, the two 16-byte chunks that pair up. 12,000 rows of 33
// heads of 192 values, 64 of them rotated (304 MB): 51.4 us, 87 % of the copy rate.
#include <algorithm>

#include "pmqa_paged.cuh"

namespace pmqa {
namespace paged {

constexpr int kRopeThreads = 256;
constexpr long long kMaxAll = 1 << 24;  // heads of both tensors

struct RopeArgs {
    Rotary r;
    int rows;
    int D[2], heads[2];
    const uint16_t *x[2];
    uint16_t *out[2];
    long long x_row[2], x_head[2], out_row[2], out_head[2];
    int items;    // of 16 values a head that a thread takes: the larger of both tensors
    int copies;   // bit t: the values outside tensor t's rotated part are copied
};

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = __bfloat16_as_ushort(__float2bfloat16_rn(f[2 * e])) |
               (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * e + 1])) << 16;
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Many rows do not stay in the L2 cache anyway: written as what leaves it first, they leave it
// to the loads (12,000 rows of 33 heads of 192: 51.4 us, 54.7 without).
template <int ROWS>
__device__ __forceinline__ void store(uint16_t *p, const uint4 &u)
{
    if (ROWS > 1)
        __stcs(reinterpret_cast<uint4 *>(p), u);
    else
        *reinterpret_cast<uint4 *>(p) = u;
}

template <int ROWS, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int half = a.r.dim / 2, tid = threadIdx.x;
    unsigned long long *const freq = reinterpret_cast<unsigned long long *>(smem);
    float2 *const cs = reinterpret_cast<float2 *>(freq + half);
    for (int i = tid; i < half; i += kRopeThreads)
        freq[i] = turns(a.r.inv_freq[i]);
    __syncthreads();
    const long long row0 = (long long)blockIdx.x * ROWS;
    for (int k = tid; k < ROWS * half; k += kRopeThreads) {
        const int row = k / half, f = k - row * half;
        if (row0 + row < a.rows)
            cs[k] = angle(__ldg(a.r.positions + row0 + row), freq[f], a.r.scale);
    }
    __syncthreads();

    const int it = tid % a.items, hv = tid / a.items, step = kRopeThreads / a.items;
    if (hv >= step)
        return;
    const int turning = a.r.dim / 16;
    const int all = a.heads[0] + a.heads[1];
    // the two chunks of 8 values of this thread, -1 for none, in either tensor
    int ca[2], cb[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (it < turning) {
            ca[t] = a.r.begin + (a.r.interleaved ? 16 * it : 8 * it);
            cb[t] = ca[t] + (a.r.interleaved ? 8 : half);
        } else {
            const int n = 2 * (it - turning), left = (a.D[t] - a.r.dim) / 8, b8 = a.r.begin / 8;
            ca[t] = (a.copies >> t & 1) && n < left ? 8 * (n < b8 ? n : n + a.r.dim / 8) : -1;
            cb[t] = (a.copies >> t & 1) && n + 1 < left ? 8 * (n + 1 < b8 ? n + 1 : n + 1 + a.r.dim / 8) : -1;
        }
    }
    // heads of all rows of the CTA in one sequence, four loads in flight
    constexpr int AHEAD = 4;
    const int stride = step * gridDim.y, rows = (int)min((long long)ROWS, a.rows - row0);
    const int over = ROWS == 1 ? 0 : stride / all, on = stride - over * all;
    int h = hv + step * blockIdx.y, row = ROWS == 1 ? 0 : h / all;
    h -= row * all;
    while (ROWS == 1 ? h < all : row < rows) {
        uint4 ua[AHEAD], ub[AHEAD];
        int hs[AHEAD], rs[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            hs[k] = h;
            rs[k] = row;
            h += on;
            if (ROWS > 1) {
                row += over;
                if (h >= all) {
                    h -= all;
                    ++row;
                }
            }
            if (ROWS == 1 ? hs[k] >= all : rs[k] >= rows)
                continue;
            const int t = hs[k] >= a.heads[0];
            const uint16_t *const p = a.x[t] + (row0 + rs[k]) * a.x_row[t] + (long long)(hs[k] - (t ? a.heads[0] : 0)) * a.x_head[t];
            const int ka = t ? ca[1] : ca[0], kb = t ? cb[1] : cb[0];
            if (ka >= 0)
                ua[k] = __ldcs(reinterpret_cast<const uint4 *>(p + ka));
            if (kb >= 0)
                ub[k] = __ldcs(reinterpret_cast<const uint4 *>(p + kb));
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (ROWS == 1 ? hs[k] >= all : rs[k] >= rows)
                continue;
            const int t = hs[k] >= a.heads[0];
            if (it < turning) {
                float x[8], y[8];
                unpack8(ua[k], x);
                unpack8(ub[k], y);
                const float2 *const w = cs + rs[k] * half + 8 * it;
                // pairs: (x[e], y[e]), or neighbours in x and then in y
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 c = w[e];
                    float &p0 = PAIRS ? (e < 4 ? x[(2 * e) & 7] : y[(2 * e) & 7]) : x[e];
                    float &p1 = PAIRS ? (e < 4 ? x[(2 * e + 1) & 7] : y[(2 * e + 1) & 7]) : y[e];
                    const float f = p0, g = p1;
                    p0 = f * c.x - g * c.y;
                    p1 = g * c.x + f * c.y;
                }
                ua[k] = pack8(x);
                ub[k] = pack8(y);
            }
            uint16_t *const p = a.out[t] + (row0 + rs[k]) * a.out_row[t] + (long long)(hs[k] - (t ? a.heads[0] : 0)) * a.out_head[t];
            const int ka = t ? ca[1] : ca[0], kb = t ? cb[1] : cb[0];
            if (ka >= 0)
                store<ROWS>(p + ka, ua[k]);
            if (kb >= 0)
                store<ROWS>(p + kb, ub[k]);
        }
    }
}

// Sizes, strides and addresses of one tensor (the stride of a dimension of one
// entry does not count).
int check_heads(const pmqa_heads *h, int rows)
{
    if (h->heads < 0 || h->head_dim < 1)
        return PMQA_ERR_INVALID_ARG;
    if (h->head_dim % 8 != 0 || h->head_dim > kMaxRotary)
        return PMQA_ERR_UNSUPPORTED;
    if (rows == 0 || h->heads == 0)
        return PMQA_OK;
    if (bad_rows(h->x, 16, rows, h->x_row, h->heads, h->x_head) ||
        bad_rows(h->out, 16, rows, h->out_row, h->heads, h->out_head))
        return PMQA_ERR_INVALID_ARG;
    const long long n = h->heads, d = h->head_dim, reach = 1ll << 60;
    const long long xr = rows > 1 ? h->x_row : 0, xh = n > 1 ? h->x_head : 0;
    const long long yr = rows > 1 ? h->out_row : 0, yh = n > 1 ? h->out_head : 0;
    if (xr > reach / rows || yr > reach / rows || xh > reach / n || yh > reach / n)
        return PMQA_ERR_INVALID_ARG;
    // results of different rows and heads are apart
    if ((n > 1 && yh < d) || (rows > 1 && yr < d) ||
        (n > 1 && rows > 1 && yr < (n - 1) * yh + d && yh < (rows - 1ll) * yr + d))
        return PMQA_ERR_INVALID_ARG;
    const long long xs = 2 * ((rows - 1ll) * xr + (n - 1) * xh + d), os = 2 * ((rows - 1ll) * yr + (n - 1) * yh + d);
    if (h->x == h->out ? xr != yr || xh != yh : cache::overlap(h->x, xs, h->out, os))
        return PMQA_ERR_INVALID_ARG;
    return PMQA_OK;
}

}  // namespace paged
}  // namespace pmqa

using namespace pmqa;
using namespace pmqa::paged;

extern "C" int pmqa_rope(const pmqa_rotary *rotary, int32_t rows, const pmqa_heads *a, const pmqa_heads *b,
                         pmqa_stream_t stream)
{
    if (!rotary || !a || rows < 0)
        return PMQA_ERR_INVALID_ARG;
    int rc = check_heads(a, rows);
    if (rc == PMQA_OK && b)
        rc = check_heads(b, rows);
    if (rc != PMQA_OK)
        return rc;
    const long long all = (long long)a->heads + (b ? b->heads : 0);
    if (all > kMaxAll)  // counted in 32 bits, over the rows of a CTA
        return PMQA_ERR_UNSUPPORTED;
    // one tensor's result on the other's (where both begin alike; a fused projection's slices do not)
    if (b && rows > 0 && a->heads > 0 && b->heads > 0 && (a->out == b->out || a->out == b->x || b->out == a->x))
        return PMQA_ERR_INVALID_ARG;
    RopeArgs k{};
    const int width = b ? std::min(a->head_dim, b->head_dim) : a->head_dim;
    if ((rc = check_rotary(rotary, width, rows > 0, &k.r)) != PMQA_OK)
        return rc;
    const pmqa_heads *both[2] = {a, b};
    int widest = 0;  // of the tensors that are copied
    k.rows = rows;
    for (int t = 0; t < 2; ++t) {
        const pmqa_heads *h = both[t];
        if (!h || h->heads == 0)
            continue;
        k.heads[t] = h->heads;
        k.D[t] = h->head_dim;
        k.x[t] = static_cast<const uint16_t *>(h->x);
        k.out[t] = static_cast<uint16_t *>(h->out);
        k.x_row[t] = h->x_row;
        k.x_head[t] = h->x_head;
        k.out_row[t] = h->out_row;
        k.out_head[t] = h->out_head;
        if (h->x != h->out) {
            k.copies |= 1 << t;
            widest = std::max(widest, h->head_dim);
        }
    }
    k.items = k.r.dim / 16 + (k.copies ? (widest - k.r.dim + 15) / 16 : 0);
    if (rows == 0 || all == 0 || k.items == 0)
        return PMQA_OK;
    int sms = 0;
    if ((rc = cache::sm_count(&sms)) != PMQA_OK)
        return rc;
    // Rows of a CTA, and CTAs of a row: with few rows the heads are spread over the SMs; with
    // many, four rows share what a CTA does at its start.
    const int step = kRopeThreads / k.items;
    const long long passes = (all + step - 1) / step;
    const int per = rows >= 16 * sms ? 4 : 1;
    const unsigned split = (unsigned)std::max<long long>(1, std::min<long long>(passes, 2 * sms / rows));
    const dim3 grid((unsigned)((rows + (long long)per - 1) / per), split);
    const size_t smem = (size_t)k.r.dim / 2 * 8 * (1 + per);
    auto *const kernel = per == 4 ? (k.r.interleaved ? rope_kernel<4, true> : rope_kernel<4, false>)
                                  : (k.r.interleaved ? rope_kernel<1, true> : rope_kernel<1, false>);
    kernel<<<grid, kRopeThreads, smem, cache::cuda(stream)>>>(k);
    return cache::code_of(cudaGetLastError());
}

extern "C" int pmqa_rope_frequencies(int32_t dim, double base, int kind, double factor, double trained,
                                     double slow_turns, double fast_turns, double *inv_freq, float *scale)
{
    if (dim < 2 || dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base) || !inv_freq || !scale ||
        kind < PMQA_ROPE_PLAIN || kind > PMQA_ROPE_PARTS)
        return PMQA_ERR_INVALID_ARG;
    if (kind != PMQA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return PMQA_ERR_INVALID_ARG;
    if (kind == PMQA_ROPE_PARTS && (!(trained >= 1.0) || !std::isfinite(trained) || !(slow_turns > 0.0) ||
                                    !(fast_turns > slow_turns) || !std::isfinite(fast_turns)))
        return PMQA_ERR_INVALID_ARG;
    const int n = dim / 2;
    double lo = 0.0, hi = 0.0;
    if (kind == PMQA_ROPE_PARTS) {
        // pair i turns trained base^(-2 i / dim) / (2 pi) times over the trained positions
        auto pair_of = [&](double t) {
            return dim * std::log(trained / (t * 6.283185307179586477)) / (2.0 * std::log(base));
        };
        lo = std::max(0.0, std::floor(pair_of(fast_turns)));
        hi = std::min(dim - 1.0, std::ceil(pair_of(slow_turns)));
    }
    for (int i = 0; i < n; ++i) {
        const double f = std::pow(base, -2.0 * i / dim);
        double slowed = 0.0;  // the share that is divided
        if (kind == PMQA_ROPE_LINEAR)
            slowed = 1.0;
        else if (kind == PMQA_ROPE_PARTS)
            slowed = i >= hi ? 1.0 : i <= lo ? 0.0 : (i - lo) / (hi - lo);
        inv_freq[i] = kind == PMQA_ROPE_PLAIN ? f : f * (1.0 - slowed) + f / factor * slowed;
    }
    *scale = kind == PMQA_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PMQA_OK;
}
