// pmqa_paged.cuh -- what the calls on a pmqa_paged_rows share: host checks and
// the device view (the cache operators' View, without its pools), a row's request
// and slot, rotary angles, the loads and conversions of bf16 rows.
#pragma once

#include <cmath>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace paged {

using cache::kFull;
using cache::View;

// ------------------------------------------------------------------ host

inline int check_rows(const pmqa_paged_rows *p, bool lens, const void *ws, size_t ws_bytes, size_t need)
{
    if (!p || p->bs < 0 || p->block_size < 1 || p->max_blocks_per_seq < 1 || p->rows < 0 ||
        p->num_blocks < 1 || (lens && p->max_rows < 1))
        return PMQA_ERR_INVALID_ARG;
    // table entries and rows of a pool are counted in 32 bits
    if ((long long)p->bs * p->max_blocks_per_seq > 0x7FFFFFFFll || p->num_blocks > 0xFFFFFFFEll / p->block_size)
        return PMQA_ERR_UNSUPPORTED;
    if (!ws || !cache::aligned(ws, 256))
        return PMQA_ERR_INVALID_ARG;
    if (ws_bytes < need)
        return PMQA_ERR_WORKSPACE;
    if (p->bs == 0 || p->rows == 0)
        return PMQA_OK;
    if (cache::missing(p->block_tables, 4) || cache::missing(p->row_begin, 4) ||
        (lens && cache::missing(p->context_lens, 4)))
        return PMQA_ERR_INVALID_ARG;
    return PMQA_OK;
}

inline View view(const pmqa_paged_rows *p, void *ws)
{
    View c{};
    c.bt = p->block_tables;
    c.ctx = p->context_lens;
    c.row_begin = p->row_begin;
    c.bs = p->bs;
    c.H = 1;
    c.P = p->block_size;
    c.W = p->max_blocks_per_seq;
    c.rows = p->rows;
    c.max_rows = p->max_rows;
    c.p_inv = c.P == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / (uint32_t)c.P);
    c.nb = p->num_blocks;
    c.status = static_cast<uint32_t *>(ws);
    return c;
}

constexpr int kMaxRotary = 1024;  // rotated values of a head at most
constexpr int kMaxHeads = 65535;  // query heads of a row: a row's values are counted in 32 bits

struct Rotary {
    const double *inv_freq;
    const int32_t *positions;
    int dim, begin, interleaved;
    float scale;
};

// `width`: of the heads that are rotated
inline int check_rotary(const pmqa_rotary *r, int width, bool positions, Rotary *out)
{
    *out = Rotary{nullptr, nullptr, 0, 0, 0, 1.0f};
    if (!r || r->dim == 0)
        return PMQA_OK;
    if (r->dim < 0 || r->begin < 0 || (long long)r->begin + r->dim > width || !std::isfinite(r->scale) ||
        (r->interleaved != 0 && r->interleaved != 1))
        return PMQA_ERR_INVALID_ARG;
    if (r->dim % 16 != 0 || r->begin % 8 != 0)
        return PMQA_ERR_UNSUPPORTED;
    if (cache::missing(r->inv_freq, 8) || (positions && !r->positions) || !cache::aligned(r->positions, 4))
        return PMQA_ERR_INVALID_ARG;
    *out = Rotary{r->inv_freq, r->positions, r->dim, r->begin, r->interleaved, r->scale};
    return PMQA_OK;
}

struct Norm {
    int kind;
    float eps;
    const float *weight, *bias;
};

inline int check_norm(const pmqa_norm *n, Norm *out)
{
    *out = Norm{PMQA_NORM_NONE, 0.0f, nullptr, nullptr};
    if (!n || n->kind == PMQA_NORM_NONE)
        return PMQA_OK;
    if ((n->kind != PMQA_NORM_LAYER && n->kind != PMQA_NORM_RMS) || !(n->eps >= 0.0f) || !std::isfinite(n->eps) ||
        !cache::aligned(n->weight, 16) || !cache::aligned(n->bias, 16))
        return PMQA_ERR_INVALID_ARG;
    *out = Norm{n->kind, n->eps, n->weight, n->bias};
    return PMQA_OK;
}

// A tensor read or written 8 elements at a time: its address and strides (that of a
// dimension of one entry does not count).
inline bool bad_rows(const void *p, uintptr_t align, int rows, long long row, int heads = 1, long long head = 0)
{
    return cache::missing(p, align) || (rows > 1 && (row < 0 || row % 8 != 0)) ||
           (heads > 1 && (head < 0 || head % 8 != 0));
}

// ------------------------------------------------------------------ device

// The request that holds row r, by a search of 32 places a step: the last i with
// row_begin[i] <= r (any i of [0, bs) where row_begin decreases). One whole warp.
__device__ __forceinline__ int request_of(const View &c, int r)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = c.bs;
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const uint32_t le = __ballot_sync(kFull, lane * step < len && __ldg(c.row_begin + lo + lane * step) <= r);
        const int k = max(__popc(le) - 1, 0);
        lo += k * step;
        len = min(step, len - k * step);
    }
    return lo;
}

// The same for a lane's own row r, from request i on, which begins at or before r: in steps
// of 1, 2, 4 and so on, and back.
__device__ __forceinline__ int request_from(const View &c, int i, long long r)
{
    const uint32_t bs = c.bs;
    uint32_t at = i, d = 1;
    while (at + d < bs && __ldg(c.row_begin + at + d) <= r) {
        at += d;
        d *= 2;
    }
    for (d /= 2; d > 0; d /= 2)
        if (at + d < bs && __ldg(c.row_begin + at + d) <= r)
            at += d;
    return (int)at;
}

constexpr uint32_t kNoRow = 0xFFFFFFFFu;

// Whether the table has a slot; recorded where it has not.
__device__ __forceinline__ bool has_slot(const View &c, long long slot)
{
    if (slot >= 0 && slot < (long long)c.P * c.W && slot <= 0x7FFFFFFFll)
        return true;
    atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
    return false;
}

// The pool row of a slot; kNoRow (recorded) where it has none.
__device__ __forceinline__ uint32_t pool_row(const View &c, int req, long long slot)
{
    if (!has_slot(c, slot))
        return kNoRow;
    const int b = c.page_of((int)slot), page = __ldg(c.bt + (long long)req * c.W + b);
    if (page < 0 || (long long)page >= c.nb) {
        atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
        return kNoRow;
    }
    return (uint32_t)page * (uint32_t)c.P + (uint32_t)((int)slot - b * c.P);
}

// Radians per position as turns modulo 1 in units of 2^-64 (fp64: off by 2^-53 of
// the frequency).
__device__ __forceinline__ unsigned long long turns(double inv_freq)
{
    const double f = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
}

// (cos, sin) of position * frequency, times scale. The product modulo 2^64 is the
// angle modulo a turn, exactly; its upper 32 bits as a signed number of 2^-31 half
// turns are within 2^-25 of a half turn as fp32 (less for small angles).
__device__ __forceinline__ float2 angle(int position, unsigned long long turn, float scale)
{
    const unsigned long long t = (unsigned long long)(long long)position * turn;
    float s, c;
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8])
{
    const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(e[k] << 16);
        f[2 * k + 1] = __uint_as_float(e[k] & 0xFFFF0000u);
    }
}

// 16 bytes of an input that no output overlaps: loads stay in flight over the stores
// between them (through plain loads, which do not, 15.7 k rows of 64 index heads take 117 us
// instead of 93).
__device__ __forceinline__ uint4 load_input(const void *p)
{
    return __ldg(reinterpret_cast<const uint4 *>(p));
}

// 8 values times f as e4m3 codes
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float f)
{
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        fmul2(z[e], z[e + 1], y[e], y[e + 1], f, f);
    return make_uint2(cache::f32x4_to_e4m3x4(z[0], z[1], z[2], z[3]), cache::f32x4_to_e4m3x4(z[4], z[5], z[6], z[7]));
}

// A lane's share of the rotation: eight values of a head whose rotated part it may
// hold (`in`). Halves: the partner's eight are LANES / 2 of the rotated part's
// lanes away and cs holds (cos, -sin) or (cos, sin) of eight pairs; interleaved: four
// pairs of its own.
struct Turn {
    float2 cs[8];
    int partner;
    bool in;

    // lane `at` of a head, table: (cos, sin) of the row's dim / 2 pairs
    __device__ __forceinline__ void load(const Rotary &r, const float2 *table, int at)
    {
        const int k = at - r.begin / 8, n = r.dim / 8;
        in = k >= 0 && k < n;
        const bool first = k < n / 2;
        partner = in ? (first ? n / 2 : -n / 2) : 0;
        const float2 *t = table + (!in ? 0 : r.interleaved ? 4 * k : 8 * (first ? k : k - n / 2));
        if (!in)
            return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (r.interleaved && e >= 4)
                break;
            cs[e] = t[e];
            if (!r.interleaved && first)
                cs[e].y = -cs[e].y;
        }
    }

    // x: this lane's values, other: the partner's (halves only)
    __device__ __forceinline__ void apply(bool interleaved, float (&x)[8], const float (&other)[8]) const
    {
        if (!in)
            return;
        if (interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float a = x[2 * e], b = x[2 * e + 1];
                x[2 * e] = a * cs[e].x - b * cs[e].y;
                x[2 * e + 1] = b * cs[e].x + a * cs[e].y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = x[e] * cs[e].x + other[e] * cs[e].y;
        }
    }
};

// A row's place: slot, pool row, whether it is a row of a request at all, and its
// position.
struct Place {
    uint32_t row;
    int position;
    int valid;
};

// i: a request that begins at or before the row
__device__ __forceinline__ Place place_of(const View &c, const Rotary &r, int i, long long row, bool keys)
{
    Place o{kNoRow, 0, 0};
    if (row >= c.rows)
        return o;
    i = request_from(c, i, row);
    const int b = __ldg(c.row_begin + i), e = __ldg(c.row_begin + i + 1);
    const long long j = row - b;
    if (j < 0 || row >= e || j >= c.max_rows)
        return o;
    const long long slot = (long long)__ldg(c.ctx + i) - ((long long)e - b) + j;
    o.valid = 1;
    o.position = r.positions && r.dim ? __ldg(r.positions + row) : (int)slot;
    if (keys)
        o.row = pool_row(c, i, slot);
    else
        has_slot(c, slot);
    return o;
}

// The rows [row0, row0 + ROWS) of a CTA: their places, and (cos, sin) of their
// angles. `freq`: the frequencies as turns, filled once by load_turns.
template <int ROWS, int DIM>
struct RowTable {
    unsigned long long freq[DIM / 2];
    float2 cs[ROWS][DIM / 2];
    Place place[ROWS];
};

template <int ROWS, int DIM>
__device__ __forceinline__ void load_turns(RowTable<ROWS, DIM> &t, const Rotary &r)
{
    for (int i = threadIdx.x; i < r.dim / 2; i += blockDim.x)
        t.freq[i] = turns(r.inv_freq[i]);
}

// Called by the whole CTA after load_turns, and again once its work on the rows
// before is done; begins and ends with a barrier.
template <int ROWS, int DIM>
__device__ __forceinline__ void load_rows(RowTable<ROWS, DIM> &t, const View &c, const Rotary &r, int row0, bool keys)
{
    static_assert(ROWS <= 32, "a lane a row");
    __syncthreads();
    if (threadIdx.x < 32) {
        const int i = request_of(c, row0);
        if (threadIdx.x < ROWS)
            t.place[threadIdx.x] = place_of(c, r, i, (long long)row0 + threadIdx.x, keys);
    }
    __syncthreads();
    const int half = r.dim / 2;
    for (int k = threadIdx.x; k < ROWS * half; k += blockDim.x) {
        const int row = k / half, f = k - row * half;
        t.cs[row][f] = angle(t.place[row].position, t.freq[f], r.scale);
    }
    __syncthreads();
}

}  // namespace paged
}  // namespace pmqa
