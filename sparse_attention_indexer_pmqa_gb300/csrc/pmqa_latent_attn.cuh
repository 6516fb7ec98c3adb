// pmqa_latent_attn.cuh -- what the kernels of the attention to all latent tokens share:
// the sequence of (unit, tile) that is split over the CTAs, the warp that walks it
// ahead of the others and looks tokens up, and the two fp8 terms of a weight.
#pragma once

#include "pmqa_latent.cuh"
#include "pmqa_paged.cuh"

namespace pmqa {
namespace latent {

using cache::Request;
using cache::View;
using namespace mla;

constexpr uint32_t kFull = cache::kFull;
constexpr int kMaxHeads = 128;
constexpr int kMaxCtas = 160;   // workspace parts: 2 per CTA, 64 rows of 512 columns or 128 of 256
constexpr int kNoPage = (int)0x80000000;  // no token there (a table entry is negative where it is bad)
constexpr int kWhole = 512;     // tables of up to so many tokens: blocks are not cut
// p = 2^(x - m), and a weight's terms are off by up to 2^-14 however small it is. So
// a row's m is not its largest score (32 k light tokens behind a heavy one with about 80 % of the weight
// then lose 90 % of what they add), but moves with the sum of its weights, up and down:
//   * where a weight would pass 2^kTop, m moves up, so that this weight is 2^aim;
//   * behind n tiles of the piece the sum is at least kEnough for each of their tokens. Where it
//     is not, m moves down: the sum then is 2^kSlack of that, and the tile's largest weight at
//     least 2^0, as far as it stays below 2^kTop and the sum below 2^kReach (or, where that is of
//     some of the tiles, m within kReach of the highest it was: O has to stay in fp32's range).
// A token loses at most 2^-14 beside its own share, and so the tokens of tile n together at most
// 2^-14 / (kEnough n) of the row's weight, 2^-14 (1 + ln n) / kEnough over all tiles: 2^-7.6 (1 + ln n).
// (In earnest far less: the light tokens behind a heavy one are in range a tile or two later, and
// their output is within 1 % from 8 k to 128 k of them.) The price is the moves. Scores with a standard
// deviation of 2.2, by graph: batch decode of 128 heads 239 us, verify of 64 packed rows 186, prompt chunks
// 1850 (3, 5 and 3 % less with m at the largest score); with four times the sum 265, 209 and 2103; m moved
// down wherever a tile's largest weight is below 2, a third more time. Standard deviation 4.4: 297, 230, 2339.
constexpr float kTop = 8.0f, kSlack = 1.0f, kReach = 30.0f;
constexpr float kEnough = 1.5f / 128.0f;
constexpr float kUnseen = 1e30f;   // -m of a row that has seen no score: above every |x|
// m is an fp32 number: past this its step, a factor that all weights of a row have in common,
// takes them out of the range of their terms (448 = 2^8.8 against 2^kTop).
constexpr float kFarScore = 0x1p23f;
constexpr double kMaxFactor = 1e20;  // |c_log2|: times a product of two rows (1.2e8) well below kUnseen

constexpr size_t kWsMeta = cache::kStatusBytes;
constexpr size_t kWsMl = kWsMeta + kMaxCtas * 16;
constexpr size_t kWsPart = kWsMl + (size_t)2 * kMaxCtas * 64 * 2 * 4;
constexpr size_t kWorkspace = kWsPart + (size_t)2 * kMaxCtas * 64 * kVDim * 4;

struct Args {
    View c;
    const uint8_t *q;   // [rows, heads, 576]
    const uint8_t *kv;  // [num_blocks * P, 576]
    uint16_t *out;
    float *lse;
    float c_log2;       // sm_scale * q_scale * kv_scale * log2(e)
    float kv_scale;
    int heads;
    int tile;           // tokens per tile: 128, or 64 (the wide kernel)
    int N;              // packed rows of a block
    int toks;           // query tokens of a block (a power of two up to the tile's)
    int pad;            // tiles' worth of starting and ending a block
    int least;          // fewest tiles that a range has
    int ranges;         // parts that the sequence is cut into at most
    int whole;          // blocks are not cut
    int4 *meta;         // [ranges]: (first row of q and out, rows, parts, 0) of the unit cut at the range's end
    float *ml;          // [2 ranges][N][2]
    float *part;        // [2 ranges][N][512]
};

// ------------------------------------------------------------- the sequence
//
// Request i has units u < U_i = ceil(n_i / toks) of `toks` query tokens; unit u has
// the tiles up to the slot of its last token, whether or not that token exists:
//   T = floor((ctx - n + toks u + toks - 1) / tile) + 1 = floor((f + u) / w) + 1,
// f = ceil((ctx - n) / toks), w = tile / toks. `pad` places without work follow each
// unit's tiles.

struct Req {
    Request q;
    int f, U;
};

__device__ __forceinline__ Req load_req(const Args &a, int i, bool tell)
{
    Req r;
    r.q = cache::load_request(a.c, i, tell);
    if (tell && r.q.n > r.q.ctx)  // rows before slot 0
        atomicOr(a.c.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
    r.U = (r.q.n + a.toks - 1) / a.toks;
    r.f = (max(r.q.ctx - r.q.n, 0) + a.toks - 1) / a.toks;
    return r;
}

// sum of floor(y / w) over y < x
__device__ __forceinline__ long long floor_sum(long long x, int w)
{
    const long long q = x / w;
    return (long long)w * (q * (q - 1) / 2) + q * (x - q * w);
}

// places of the first u units
__device__ __forceinline__ long long places(const Args &a, const Req &r, int u)
{
    const int w = a.tile / a.toks;
    return floor_sum((long long)r.f + u, w) - floor_sum(r.f, w) + (long long)u * (1 + a.pad);
}

// Where a role is: unit u of request i, tile t of T, at place x of the sequence.
struct Cursor {
    Req r;
    int i, u, t, T;
    long long x;

    __device__ __forceinline__ void set_unit(const Args &a) { T = (r.f + u) / (a.tile / a.toks) + 1; }

    // the next unit; false where it is not before place x1 (the last one's end is not after
    // any range's, so the requests behind it are not looked at)
    __device__ __forceinline__ bool next_unit(const Args &a, long long x1)
    {
        x += T + a.pad - t;
        t = 0;
        ++u;
        if (x >= x1)
            return false;
        while (u >= r.U) {
            // past requests without rows, eight at a time: each look costs the latency of memory
            ++i;
            for (int k = 8; k == 8; i += k) {
                int b[9];
#pragma unroll
                for (int j = 0; j < 9; ++j)
                    b[j] = __ldg(a.c.row_begin + min(i + j, a.c.bs));
                k = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    k += k == j && b[j] == b[j + 1] && i + j < a.c.bs ? 1 : 0;
            }
            if (i >= a.c.bs)
                return false;
            r = load_req(a, i, false);
            u = 0;
        }
        set_unit(a);
        return true;
    }
};

struct Range {
    long long x0, x1, total;
    int C;       // ranges with work
    Cursor at;   // place x0
    int any;
};

__device__ __forceinline__ long long range_start(long long total, int C, long long b)
{
    return b * total / C;
}

__device__ __forceinline__ int range_of(long long total, int C, long long x)
{
    return (int)(((x + 1) * (long long)C - 1) / total);
}

// Called by the whole CTA; the result is in *s_range after the last barrier. s_sum:
// THREADS / 16 words.
template <int THREADS>
__device__ __forceinline__ void find_range(const Args &a, int g, long long *s_sum, Range *s_range)
{
    long long *const s_units = s_sum + THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long sum = 0, units = 0;
    for (int i = tid; i < a.c.bs; i += THREADS) {
        const Req r = load_req(a, i, blockIdx.x == 0);
        sum += places(a, r, r.U);
        units += r.U;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(kFull, sum, o);
        units += __shfl_xor_sync(kFull, units, o);
    }
    if (lane == 0) {
        s_sum[warp] = sum;
        s_units[warp] = units;
    }
    if (tid == 0)
        s_range->any = 0;
    __syncthreads();
    long long total = 0;
    units = 0;
    for (int k = 0; k < THREADS / 32; ++k) {
        total += s_sum[k];
        units += s_units[k];
    }
    // no more ranges than keep a.least tiles each
    const int C = (int)min((long long)a.ranges, max(units > 0 ? 1ll : 0ll, (total - units * a.pad) / a.least));
    const long long x0 = g < C ? range_start(total, C, g) : total;
    const long long x1 = g < C ? range_start(total, C, g + 1) : total;
    long long base = 0;
    for (int i0 = 0; x0 < x1 && i0 < a.c.bs; i0 += THREADS) {
        const int i = i0 + tid;
        long long n = 0;
        Req r{};
        if (i < a.c.bs) {
            r = load_req(a, i, false);
            n = places(a, r, r.U);
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
        long long lo = base + inc - n, all = 0;
        for (int k = 0; k < THREADS / 32; ++k) {
            if (k < warp)
                lo += s_sum[k];
            all += s_sum[k];
        }
        if (n > 0 && lo <= x0 && x0 < lo + n) {
            // the unit that holds place x0
            const long long y = x0 - lo;
            int ua = 0, ub = r.U;
            while (ub - ua > 1) {
                const int mid = ua + (ub - ua) / 2;
                if (places(a, r, mid) <= y)
                    ua = mid;
                else
                    ub = mid;
            }
            Cursor c;
            c.r = r;
            c.i = i;
            c.u = ua;
            c.t = (int)(y - places(a, r, ua));
            c.x = x0;
            c.set_unit(a);
            // behind the tiles, or (whole) inside a unit: the next one
            bool any = true;
            if (c.t >= c.T || (a.whole && c.t > 0))
                any = c.next_unit(a, x1);
            s_range->at = c;
            s_range->any = any;
        }
        base += all;
        if (base > x0)
            break;  // the same for every thread
    }
    if (tid == 0) {
        s_range->x0 = x0;
        s_range->x1 = x1;
        s_range->total = total;
        s_range->C = C;
    }
    __syncthreads();
}

// The next tile of a range; false at its end.
__device__ __forceinline__ bool next_tile(const Args &a, Cursor &c, long long x1)
{
    ++c.t;
    ++c.x;
    if (c.t < c.T)
        return a.whole || c.x < x1;
    return c.next_unit(a, x1);
}

// ------------------------------------------------------------- one block of rows

// The packed rows of a unit.
struct Block {
    long long first;  // row of q and out
    int rows;         // packed rows
    int last;         // last slot that the first row sees
    int end;          // slots that some row sees
};

__device__ __forceinline__ Block block_of(const Args &a, const Cursor &c)
{
    Block b;
    const int j0 = c.u * a.toks;
    const int n = min(a.toks, c.r.q.n - j0);
    b.rows = n * a.heads;
    b.first = ((long long)c.r.q.r0 + j0) * a.heads;
    b.last = c.r.q.ctx - c.r.q.n + j0;
    b.end = min(c.r.q.ctx, max(0, b.last + n));
    return b;
}

// mbar_wait with all but its first try out of line: the roles' loops wait in many
// places, and their code together should stay in the instruction caches.
inline __device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, const volatile int *abort_flag)
{
    return mbar_wait(bar, parity, abort_flag);
}

__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, const volatile int *abort_flag)
{
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag);
}

// A wait that ran out: recorded, and the CTA's other waits end.
__device__ __forceinline__ void fail(const Args &a, volatile int *abort_flag)
{
    atomicOr(a.c.status, (uint32_t)PMQA_DEV_TIMEOUT);
    *abort_flag = 1;
}

// What the planner tells the others of a tile, and of its piece of a unit (the tiles of
// a unit in one range).
enum { kFirst = 1, kLast = 2, kEnd = 4, kSteady = 8 };  // first or last of its piece, last of the range, two more in the piece
struct Tile {
    uint32_t have[4];  // a bit per token that is there
    int tok;           // first token
    uint32_t flags;
    uint32_t unused[2];
};
struct Piece {
    long long first;   // row of q and out
    int rows;          // packed rows
    int last;          // last slot that the first row sees
    int sole;          // the unit lies in this range whole
    int slot;          // otherwise: of its part
    int unused[2];
};
static_assert(sizeof(Tile) == 32 && sizeof(Piece) == 32, "places in shared memory");

// The planner's warp. A lane looks up tokens lane, lane + 32, ... of a tile, whose
// table entries were asked for a tile earlier. A tile is described once the producers
// took the tile kAhead before it, and with it the slot of the tile kStages before that: so
// the values of that one, whose place the description takes (or of the next one after it, where
// kTiles is larger), have been read, and its description by all that work on it. (A piece's
// place: kPieces > kTiles + 1 pieces later, when the output of the piece there is out.)
template <class K>
__device__ __forceinline__ void plan_tiles(const Args &a, uint8_t *smem, uint64_t *bar, const Range *range, int g,
                                           bool joins, volatile int *abort_flag)
{
    constexpr int W = K::kTile / 32;
    Cursor c = range->at;
    const long long x0 = range->x0, x1 = range->x1;
    const int lane = threadIdx.x & 31;
    int page[W], off[W], seg = -1, e = 0;
    Block b = block_of(a, c);
    auto look_up = [&](const Cursor &f, int end) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int tok = f.t * (32 * W) + 32 * k + lane;
            page[k] = kNoPage;
            if (tok < end) {
                const int n = a.c.page_of(tok);
                page[k] = __ldg(a.c.bt + (long long)f.i * a.c.W + n);
                off[k] = tok - n * a.c.P;
            }
        }
    };
    look_up(c, b.end);
    for (int it = 0;; ++it) {
        const bool first = it == 0 || c.t == 0;
        uint32_t row[W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            row[k] = paged::kNoRow;
            if (page[k] != kNoPage) {
                if (page[k] < 0 || (long long)page[k] >= a.c.nb)
                    atomicOr(a.c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
                else
                    row[k] = (uint32_t)page[k] * (uint32_t)a.c.P + (uint32_t)off[k];
            }
        }
        Cursor d = c;
        const bool more = next_tile(a, d, x1), last = !more || d.t == 0;
        const Block here = b;
        if (more) {
            if (last)
                b = block_of(a, d);
            look_up(d, b.end);
        }
        if (it >= K::kAhead) {
            const int j = it - K::kAhead;
            if (!__all_sync(kFull, wait_for(&bar[K::kBUsed + j % K::kTiles], (uint32_t)(j / K::kTiles) & 1u, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
        }
        Tile *const tile = reinterpret_cast<Tile *>(smem + K::kOffInfo) + e;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const uint32_t have = __ballot_sync(kFull, row[k] != paged::kNoRow);
            reinterpret_cast<uint32_t *>(smem + K::kOffRows)[it % K::kAhead * (32 * W) + 32 * k + lane] = row[k];
            if (lane == k)
                tile->have[k] = have;
        }
        if (first)
            ++seg;
        if (lane == 0) {
            tile->tok = c.t * (32 * W);
            tile->flags = (first ? kFirst : 0) | (last ? kLast : 0) | (more ? 0 : kEnd) |
                          (c.t + 2 < c.T && (a.whole || c.x + 2 < x1) ? kSteady : 0);
            if (first) {
                const long long xs = c.x - c.t;
                const bool starts = xs >= x0;
                Piece *const piece = reinterpret_cast<Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
                piece->first = here.first;
                piece->rows = here.rows;
                piece->last = here.last;
                piece->sole = a.whole || (starts && xs + c.T <= x1);
                piece->slot = 2 * g + (starts ? 1 : 0);
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bar[K::kBInfo + e]);
        if (!more)
            break;
        c = d;
        if (++e == K::kTiles)
            e = 0;
    }
    if (joins && lane == 0) {
        // the last unit goes on in later ranges and starts in this one: to be joined
        const long long xs = c.x - c.t, xe = xs + c.T;
        if (!a.whole && xs >= x0 && xe > x1)
            a.meta[g] = make_int4((int)b.first, b.rows, range_of(range->total, range->C, xe - 1) - g + 1, 0);
    }
}

__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h2)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
    return r;
}

__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t b)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)b));
    return r;
}

__device__ __forceinline__ uint32_t e5m2x2_of_f16x2(uint32_t h2)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
    return r;
}

// Two weights, an f16 pair, as their terms (bytes 0 and 1): the f16 value of p is off
// by 2^-11 at most, its difference from the first term exact: at most 2^-4 p, or 2^-10 below
// p = 2^-6. SAME: both terms go into one accumulator, so the second has the first's unit:
// e5m2, which reaches down to 2^-17 and leaves 2^-7 p or 2^-13. Otherwise it is e4m3 of 16
// times the difference, which leaves 2^-8 p or 2^-14.
template <bool SAME>
__device__ __forceinline__ void split2(uint32_t p, uint32_t &hi, uint32_t &lo)
{
    hi = e4m3x2_of_f16x2(p);
    uint32_t d = f16x2_of_e4m3x2(hi);
    asm("sub.rn.f16x2 %0, %1, %0;" : "+r"(d) : "r"(p));
    if (SAME) {
        lo = e5m2x2_of_f16x2(d);
    } else {
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(d) : "r"(0x4C004C00u));  // 16
        lo = e4m3x2_of_f16x2(d);
    }
}

// (d0, d1) = (a0, a1) * (b, b) + (c0, c1): one packed fp32x2 multiply-add.
__device__ __forceinline__ void ffma2_of(float &d0, float &d1, uint32_t a0, uint32_t a1, float b, float c0, float c1)
{
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "mov.b64 rb, {%4, %4};\n\t"
        "mov.b64 rc, {%5, %6};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "r"(a0), "r"(a1), "f"(b), "f"(c0), "f"(c1));
}

// Whether m, of a row that has seen scores (-m is not kUnseen), is past where weights stay in range.
// Decided when a row is done: an m that a later one leaves behind does no harm.
__device__ __forceinline__ bool too_far(float mneg) { return fabsf(mneg) > kFarScore && mneg != kUnseen; }

// A sum in another unit. Past kFarScore weights, and so the sum, may be infinite; a factor of 0 leaves
// nothing of it then either (NaN stays NaN).
__device__ __forceinline__ float finite(float l) { return l == INFINITY ? 3.402823466e38f : l; }

// -m of a row for a tile whose largest score is x (-inf: it sees none of them), where the weights
// before it add up to l, and with its own should to `need`; stays_short: they do not.
// most: what -m may be at most.
__device__ __forceinline__ float moved_to(float aim, float mneg, float x, float l, float need, bool &stays_short,
                                          float most = INFINITY)
{
    const float to = x + mneg > kTop ? aim - x : mneg;
    const float sum = l * ex2_approx(to - mneg) + ex2_approx(x + to);  // the factor: 0 where no score was seen before
    stays_short = false;
    if (!(sum < need && sum > 0.0f))
        return to;
    const float bits = __log2f(__fdividef(need, sum)), room = kTop - (x + to);
    const float light = x > -INFINITY ? -(x + to) : 0.0f;
    stays_short = room < bits;
    return fminf(most, to + fminf(room, fminf(fmaxf(bits + kSlack, light), kReach - __log2f(sum))));
}

// Four codes, NaN (0x7F, 0xFF) replaced by 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t x)
{
    const uint32_t is = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    return x & ~((is >> 7) * 0xFFu);
}

cudaError_t launch_wide(Args &a, int sms, cudaStream_t st);

}  // namespace latent
}  // namespace pmqa
