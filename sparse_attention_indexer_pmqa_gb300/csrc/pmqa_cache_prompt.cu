// pmqa_cache_prompt.cu -- attention over the paged 8-bit K/V cache for requests
// with many query rows (prompts, prompt chunks) on the 5th-generation tensor
// cores.
//
// Rows of one request and kv head are packed as R = j * group + g (query token
// j, head g of the group), 256 of them to a CTA in two tiles of 128. With the
// tokens in tiles of 128:
//   S = Q K^T    kind::f8f6f4 on the cached codes as they are: q, scaled by a
//                power of two per row, is the sum of an e4m3 and an e5m2 term,
//                exact for bf16 values from 2^-13 of their row's largest on and
//                off by at most 2^-21 of it below that (split_terms); both terms add
//                into one accumulator, at the cost of one bf16 product;
//   p = 2^(x - m), x = S ks_t c_row, masked by slot; running m and l per row,
//                one thread per row; P is written as f16 over the columns that
//                held S;
//   O += P V     kind::f16 with P from tensor memory and V as f16: the codes
//                times vs_t / vref, vref the largest block scale so far, so that O
//                needs no factor per token. Power-of-two scales make that exact down
//                to 2^-30 vref; others, and smaller ones, are multiplied in fp32 and
//                rounded once, by 2^-11 of the value or 2^-31 of vref.
// Roles of a CTA's 16 warps: 0-3 and 4-7 are the softmax (and the final output)
// of the two row tiles, 8-11 convert V, 12 issues the products, 13 and 14 look up
// the blocks and copy K and V rows (cp.async). While
// one tile's softmax runs the tensor cores work for the other.
//
// Bound by the tensor cores: 4 D flops per visible (row, head, token) at the
// bf16 rate, 512 cycles per 128 x 128 x 128 product and tile against about 4.2
// issue slots per score, 1100 cycles for both tiles. 6415 rows of 32 heads over 8
// behind 2 to 8 k tokens take 415 us, 950 TFLOP/s (49 % of the measured bf16 rate;
// the tensor pipe is active 43 % of the time): the rest are the gaps between a
// tile's softmax and its products, instruction fetches (the code is larger than
// the innermost cache) and the uneven lengths of the items.
//
// Where there are fewer row blocks than SMs, contexts are cut over the CTAs too and
// the parts joined by the kernel of the short rows: 16 rows of 64 heads on 32 k
// tokens take 55 us, uncut 427; 4 requests of 5 rows 140, uncut 445.
#include <algorithm>
#include <cmath>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace cache {

constexpr int kPrRows = kPromptRows;  // packed rows per CTA (two tiles of 128)
constexpr int kRankedRequests = 128;  // so many at most are put in order: each CTA goes over them about 8 times
constexpr int kLeastPart = 4;     // token tiles (about 9 us): a context is not cut finer
constexpr int kPrTok = 128;       // tokens per tile
constexpr int kPrThreads = 512;
constexpr int kKStages = 2, kRawSlots = 3, kVStages = 2, kMeta = 4;
constexpr uint32_t kTileBytes = 128 * 128;           // 128 rows of 128 bytes
constexpr float kVUp = 64.0f;                        // V is held times 64 / vref in f16

// shared memory: operands (1024-byte aligned), then per-tile values, barriers
constexpr uint32_t kPrOffQ = 0;                                   // [tile][hi, lo]
constexpr uint32_t kPrOffK = kPrOffQ + 4 * kTileBytes;
constexpr uint32_t kPrOffRaw = kPrOffK + kKStages * kTileBytes;   // V codes, 3 slots
constexpr uint32_t kPrOffV = kPrOffRaw + kRawSlots * kTileBytes;          // V f16, 2 slots of 32 KB
constexpr uint32_t kPrOffKs = kPrOffV + kVStages * 2 * kTileBytes;  // [kMeta][128] fp32
constexpr uint32_t kPrOffVs = kPrOffKs + kMeta * 512;             // [kMeta][128] fp32
constexpr uint32_t kPrOffTile = kPrOffVs + kMeta * 512;           // [kMeta]: 4 mask words, vfac, vref, 4 bytes: even scales
constexpr uint32_t kPrOffRed = kPrOffTile + kMeta * 32;           // [2][largest, smallest][4] fp32
constexpr uint32_t kPrOffBar = kPrOffRed + 64;
enum {
    kBKFull = 0,                  // [2] K rows, scales, mask landed: 32 cp.async arrivals and lane 0's own
    kBKEmpty = kBKFull + kKStages,  // [2] scores done with the stage (MMA commit), its scales read (4 warps)
    kBVFull = kBKEmpty + kKStages,       // [2] V converted, factors written: 4 warps
    kBVEmpty = kBVFull + 2,       // [2] output update done with the slot: MMA commit
    kBSFull = kBVEmpty + 2,       // [2 tiles] scores in TMEM: MMA commit
    kBPFull = kBSFull + 2,        // [2 tiles] P written, O rescaled: 4 warps
    kBODone = kBPFull + 2,        // every product done: MMA commit
    kBQ = kBODone + 1,            // Q operands written: 8 warps
    kBRawFull = kBQ + 1,          // [3] V codes landed: 32 cp.async arrivals and lane 0's own
    kBRawEmpty = kBRawFull + kRawSlots,  // [3] V codes converted: 4 warps
    kBCount = kBRawEmpty + kRawSlots
};
constexpr uint32_t kPrOffMisc = kPrOffBar + kBCount * 8;
constexpr uint32_t kPrSmem = kPrOffMisc + 16;
static_assert(kPrSmem <= 232448, "shared memory budget");

struct PromptArgs {
    View c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    float scale_log2;
    int heads, group;
    int least;        // requests with at least this many packed rows
    long long slots;  // row-block slots over all requests (upper bound)
    int parts;        // CTAs that contexts may be cut over, 0: they are not cut
    int4 *meta;       // [parts]: (request, head, row block, 2 parts) of the context that the CTA begins
    float *ml;        // [parts][256][2]
    float *part;      // [parts][256][D]
};

// What a CTA works on: row block `nth` of a request and head, part `part` of the
// `parts` that its context is cut into, `chunk` token tiles each.
struct Piece {
    int req, h, nth, part, parts, chunk;
};

// With fewer row blocks N than CTAs C, contexts are cut into pieces of
// chunk = ceil(tiles / (C - N)) tiles: at most tiles / chunk + N <= C of them.
// Called by the whole CTA; false: there are row blocks enough, nothing is cut.
__device__ __forceinline__ bool find_piece(const PromptArgs &a, Piece &o)
{
    constexpr int WARPS = kPrThreads / 32;
    __shared__ long long s_n[WARPS], s_t[WARPS];
    __shared__ int s_req;
    __shared__ long long s_at;
    const View &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto shape = [&](int i, int &B, int &T) {
        const Request q = load_request(c, i, false);
        const int rows = q.n * a.group;
        B = rows >= a.least ? (rows + kPrRows - 1) / kPrRows : 0;
        T = max(1, (q.ctx + kPrTok - 1) / kPrTok);
    };
    long long n = 0, t = 0;
    int B, T;
    for (int i = tid; i < c.bs; i += kPrThreads) {
        shape(i, B, T);
        n += (long long)c.H * B;
        t += (long long)c.H * B * T;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
        n += __shfl_xor_sync(kFull, n, k);
        t += __shfl_xor_sync(kFull, t, k);
    }
    if (lane == 0) {
        s_n[warp] = n;
        s_t[warp] = t;
    }
    __syncthreads();
    n = t = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
        n += s_n[k];
        t += s_t[k];
    }
    if (n >= a.parts)
        return false;
    const long long u = blockIdx.x, room = a.parts - n;
    const int chunk = (int)max((long long)kLeastPart, (t + room - 1) / room);
    o.parts = 0;
    if (tid == 0)
        s_req = -1;
    long long base = 0;
    for (int i0 = 0; u < a.parts && i0 < c.bs; i0 += kPrThreads) {
        const int i = i0 + tid;
        long long mine = 0;
        if (i < c.bs) {
            shape(i, B, T);
            mine = (long long)c.H * B * ((T + chunk - 1) / chunk);
        }
        long long inc = mine;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const long long y = __shfl_up_sync(kFull, inc, k);
            if (lane >= k)
                inc += y;
        }
        __syncthreads();
        if (lane == 31)
            s_n[warp] = inc;
        __syncthreads();
        long long lo = base + inc - mine, all = 0;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            if (k < warp)
                lo += s_n[k];
            all += s_n[k];
        }
        if (lo <= u && u < lo + mine) {
            s_req = i;
            s_at = u - lo;
        }
        base += all;
        if (base > u)
            break;  // the same for every thread
    }
    __syncthreads();
    if (s_req < 0)
        return true;  // no piece for this CTA (parts = 0)
    o.req = s_req;
    shape(o.req, B, T);
    o.parts = (T + chunk - 1) / chunk;
    o.chunk = (T + o.parts - 1) / o.parts;  // pieces of one context are alike
    long long y = s_at;
    o.part = (int)(y % o.parts);
    y /= o.parts;
    o.nth = (int)(y % B);
    o.h = (int)(y / B);
    return true;
}

// First row-block slot of request i (see the append kernel's first_slot).
__device__ __forceinline__ long long first_block(const PromptArgs &a, int i)
{
    return (long long)max(__ldg(a.c.row_begin + i), 0) * a.group / kPrRows + i;
}

// Row blocks of request i that see at least x token tiles (its last ones): some row
// of the block must see slot 128 (x - 1).
__device__ __forceinline__ int blocks_from(const PromptArgs &a, int i, int x)
{
    const Request q = load_request(a.c, i, false);
    const int rows = q.n * a.group, B = rows >= a.least ? (rows + kPrRows - 1) / kPrRows : 0;
    const long long j = (long long)(x - 1) * kPrTok - (q.ctx - q.n);  // the first row that sees it
    if (x <= 0 || j <= 0)
        return B;
    return j * a.group >= rows ? 0 : B - (int)(j * a.group / kPrRows);
}

// The u-th row block in the order of falling length (then by request, block, head):
// a long one started late is waited for (two prompts among decoding requests: 69 us,
// in the order of the rows 73; by one warp, whose result the others read: in every
// warp it costs the loops below registers, 482 us instead of 427 on 6415 rows of 32
// heads). Called by a whole warp; false: u is past the last.
__device__ __forceinline__ bool ranked_block(const PromptArgs &a, long long u, Piece &o)
{
    const View &c = a.c;
    const int lane = threadIdx.x & 31;
    auto count = [&](int x) {
        long long n = 0;
        for (int i = lane; i < c.bs; i += 32)
            n += blocks_from(a, i, x);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1)
            n += __shfl_xor_sync(kFull, n, k);
        return n * c.H;
    };
    if (u >= count(0))
        return false;
    int lo = 0, hi = 0;  // count(lo) > u >= count(hi)
    for (int i = lane; i < c.bs; i += 32)
        hi = max(hi, clamp_ctx(c, i, false));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        hi = max(hi, __shfl_xor_sync(kFull, hi, k));
    hi = (hi + kPrTok - 1) / kPrTok + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (count(mid) > u)
            lo = mid;
        else
            hi = mid;
    }
    long long at = u - count(hi);  // among the blocks of `lo` tiles
    for (int i0 = 0; i0 < c.bs; i0 += 32) {
        const int i = i0 + lane;
        const int from = i < c.bs ? blocks_from(a, i, lo) : 0;
        const int mine = i < c.bs ? (from - blocks_from(a, i, hi)) * c.H : 0;
        int inc = mine;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, k);
            if (lane >= k)
                inc += y;
        }
        const uint32_t over = __ballot_sync(kFull, inc > at);
        if (over) {
            const int who = __ffs(over) - 1;
            const int first = __shfl_sync(kFull, inc - mine, who);
            o.req = i0 + who;
            const int k = (int)at - first;
            o.nth = blocks_from(a, o.req, 0) - __shfl_sync(kFull, from, who) + k / c.H;
            o.h = k % c.H;
            o.part = 0;
            o.parts = 1;
            return true;
        }
        at -= __shfl_sync(kFull, inc, 31);
    }
    return false;
}

// Byte of (row r, 16-byte chunk c) in a 128-byte-row operand, 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int r, int c)
{
    return (uint32_t)(r * 128) + (uint32_t)((c ^ (r & 7)) << 4);
}

// D[tmem] (+)= A[tmem] * B[smem], f16 inputs, fp32 accumulation, one CTA.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 consecutive TMEM columns of this thread's lane from registers.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t scale_f16x2(uint32_t x, float f)
{
    return pack_f16x2(__half2float(__ushort_as_half((unsigned short)(x & 0xFFFFu))) * f,
                      __half2float(__ushort_as_half((unsigned short)(x >> 16))) * f);
}

// How the scores of a tile are read. kEven: every token counts and each 32 of
// them share one scale that is not negative (a block that covers them, or equal
// scales); kWhole: every token counts, a scale each; kMasked: tokens that do not
// exist (mask words) or lie behind the row's last slot `lim` are -inf.
enum { kEven, kWhole, kMasked };

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// (d0, d1) = (a0, a1) * b + c with b and c pairs held in 64 bits.
__device__ __forceinline__ void ffma2_to(float &d0, float &d1, float a0, float a1, uint64_t b, uint64_t c)
{
    asm("{\n\t.reg .b64 ra, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\t"
        "fma.rn.f32x2 rd, ra, %4, %5;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "l"(b), "l"(c));
}

__device__ __forceinline__ uint64_t pair(float x)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}

// The largest scaled score of this thread's row (128 columns from tS), of tokens with a
// scale each or masked. The loops over column chunks stay rolled: unrolled, the two passes
// and their forms outgrow the instruction cache (882 us against 543, before later steps, on
// 6415 rows of 32 heads).
template <int HOW>
__device__ __forceinline__ float row_max(uint32_t tS, const float *ks, uint32_t tb, int lim)
{
    static_assert(HOW != kEven, "equal scales are read as single ones");
    float top = -INFINITY;
#pragma unroll 1
    for (int cc = 0; cc < 4; ++cc) {
        uint32_t r[32];
        tmem_ld32(tS + 32u * cc, r);
        const uint32_t have = HOW == kMasked ? lds32(tb + 4u * cc) : 0u;
        tmem_ld_wait();
        reg_fence_cols<32>(r);
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int z = 0; z < 32; z += 4) {
            float y[4];
            const float4 k = *reinterpret_cast<const float4 *>(ks + 32 * cc + z);
            fmul2(y[0], y[1], __uint_as_float(r[z]), __uint_as_float(r[z + 1]), k.x, k.y);
            fmul2(y[2], y[3], __uint_as_float(r[z + 2]), __uint_as_float(r[z + 3]), k.z, k.w);
            if constexpr (HOW == kMasked) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = (have >> (z + e) & 1u) && 32 * cc + z + e <= lim ? y[e] : -INFINITY;
            }
            t0 = max3(t0, y[0], y[1]);
            t1 = max3(t1, y[2], y[3]);
        }
        top = fmaxf(top, fmaxf(t0, t1));
    }
    return top;
}

// p = 2^(y rc + ms) of the row's 128 columns as f16 pairs; returns their sum.
// The next 32 columns load while these are worked on.
template <int HOW>
__device__ __forceinline__ float weights(uint32_t tS, const float *ks, uint32_t tb, int lim, float rc, float ms,
                                         uint32_t (&p)[64])
{
    float l0 = 0.0f, l1 = 0.0f;
    const uint64_t m2 = pair(ms);
    uint64_t r2 = pair(rc);
    uint32_t r[2][32];
    tmem_ld32(tS, r[0]);
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
        const uint32_t have = HOW == kMasked ? lds32(tb + 4u * cc) : 0u;
        if constexpr (HOW == kEven)
            r2 = pair(ks[32 * cc] * rc);
        tmem_ld_wait();
        reg_fence_cols<32>(r[cc & 1]);
        if (cc < 3)
            tmem_ld32(tS + 32u * (cc + 1), r[(cc + 1) & 1]);
#pragma unroll
        for (int z = 0; z < 32; z += 4) {
            float y[4], x[4];
            if constexpr (HOW == kEven) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = __uint_as_float(r[cc & 1][z + e]);
            } else {
                const float4 k = *reinterpret_cast<const float4 *>(ks + 32 * cc + z);
                fmul2(y[0], y[1], __uint_as_float(r[cc & 1][z]), __uint_as_float(r[cc & 1][z + 1]), k.x, k.y);
                fmul2(y[2], y[3], __uint_as_float(r[cc & 1][z + 2]), __uint_as_float(r[cc & 1][z + 3]), k.z, k.w);
            }
            ffma2_to(x[0], x[1], y[0], y[1], r2, m2);
            ffma2_to(x[2], x[3], y[2], y[3], r2, m2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (HOW == kMasked)  // after the product: c_row may be 0
                    x[e] = (have >> (z + e) & 1u) && 32 * cc + z + e <= lim ? x[e] : -INFINITY;
                x[e] = ex2_approx(x[e]);
            }
            fadd2(l0, l1, x[0], x[1]);
            fadd2(l0, l1, x[2], x[3]);
            p[16 * cc + z / 2] = pack_f16x2(x[0], x[1]);
            p[16 * cc + z / 2 + 1] = pack_f16x2(x[2], x[3]);
        }
    }
    return l0 + l1;
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1) cache_prompt_kernel(const __grid_constant__ PromptArgs a)
{
    constexpr int CH = D / 16;  // 16-byte chunks of a cached row
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    const View &c = a.c;
    const int G = a.group;
    griddep_launch_dependents();  // the few-row kernel fills the SMs that run out of rows
    if (G > kShortRows && blockIdx.x == 0)
        report_requests(c);  // no few-row kernel follows

    // ------------------------------------------------------------ which rows
    Piece pc{0, 0, 0, 0, 1, 0};
    const bool cut = a.parts > 0 && find_piece(a, pc);
    if (!cut && c.bs <= kRankedRequests) {
        __shared__ int s_pc[4];
        if (warp == 0) {
            const bool any = ranked_block(a, blockIdx.x, pc);
            if (lane == 0) {
                s_pc[0] = pc.req;
                s_pc[1] = pc.h;
                s_pc[2] = pc.nth;
                s_pc[3] = any ? 1 : 0;
            }
        }
        __syncthreads();
        pc = Piece{s_pc[0], s_pc[1], s_pc[2], 0, s_pc[3], 0};
    } else if (!cut) {
        // slots run from the last to the first: a request's last rows see the most tokens
        const long long item = a.slots * c.H - 1 - blockIdx.x;
        const long long slot = max(item, 0ll) / c.H;
        int lo = 0, len = c.bs;
        while (len > 1) {
            const int step = (len + 31) >> 5;
            const int at = lo + lane * step;
            const uint32_t le = __ballot_sync(kFull, lane * step < len && first_block(a, at) <= slot);
            const int k = max(__popc(le) - 1, 0);
            lo += k * step;
            len = min(step, len - k * step);
        }
        const long long nth = slot - first_block(a, lo);
        const bool mine = item >= 0 && nth >= 0 && nth * kPrRows < 0x7FFFFFFFll;
        pc = Piece{lo, (int)(max(item, 0ll) - slot * c.H), mine ? (int)nth : 0, 0, mine ? 1 : 0, 0};
    }
    if (a.parts > 0 && tid == 0 && blockIdx.x < a.parts)
        a.meta[blockIdx.x] = pc.parts > 1 && pc.part == 0 ? make_int4(pc.req, pc.h, pc.nth, 2 * pc.parts)
                                                          : make_int4(0, 0, 0, 0);
    if (pc.parts == 0)
        return;  // the same for the whole CTA
    const int req = pc.req, h = pc.h;
    const Request q = load_request(c, req, h == 0 && tid == 0);
    const int rows_all = q.n * G;
    if (rows_all < a.least || (long long)pc.nth * kPrRows >= rows_all)
        return;
    const int R0 = pc.nth * kPrRows;
    const int nrow = min(kPrRows, rows_all - R0);
    const bool two = nrow > 128;
    const int first_tok = q.ctx - q.n;  // slot of query token 0
    const int end = max(0, first_tok + (R0 + nrow - 1) / G + 1);  // tokens that some row sees
    const int tiles = (end + kPrTok - 1) / kPrTok;
    const int t_0 = pc.part * pc.chunk;  // the piece's first tile, and its number of them
    const int T = pc.parts > 1 ? max(0, min(tiles - t_0, pc.chunk)) : tiles;

    if (sbase & 1023u) {
        if (tid == 0)
            atomicOr(c.status, (uint32_t)PMQA_DEV_INTERNAL);
        return;
    }
    uint64_t *const bar = reinterpret_cast<uint64_t *>(smem + kPrOffBar);
    uint32_t *const misc = reinterpret_cast<uint32_t *>(smem + kPrOffMisc);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    if (tid == 0) {
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(&bar[kBKFull + s], 33);
            mbar_init(&bar[kBKEmpty + s], 5);
        }
        for (int s = 0; s < kRawSlots; ++s) {
            mbar_init(&bar[kBRawFull + s], 33);
            mbar_init(&bar[kBRawEmpty + s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[kBVFull + s], 4);
            mbar_init(&bar[kBVEmpty + s], 1);
            mbar_init(&bar[kBSFull + s], 1);
            mbar_init(&bar[kBPFull + s], 4);
        }
        mbar_init(&bar[kBODone], 1);
        mbar_init(&bar[kBQ], 8);
        misc[1] = 0;
        mbar_init_fence();
    }
    if (warp == 12)
        tmem_alloc(misc, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];
    // columns: S (then P) of tile 0, 1 at 0, 128; O of tile 0, 1 at 256, 384
    auto fail = [&]() {
        atomicOr(c.status, (uint32_t)PMQA_DEV_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp < 8) {
        // -------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");  // 2 x 192 + 2 x 64 = 4 x 128
        const int tile = warp >> 2;
        const int row = (warp & 3) * 32 + lane;     // TMEM lane
        const int R = R0 + tile * 128 + row;
        const bool has = tile * 128 + row < nrow;
        const int j = R / G, g = R - j * G;
        const long long rh = (long long)(q.r0 + j) * a.heads + h * G + g;
        const int lim = has ? first_tok + j : 0x7FFFFFFF;  // last slot that the row sees
        float rc;
        {
            // the row's q as two terms, K-major in the 128-byte swizzle
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + rh * D);
            uint4 u[D / 8];
#pragma unroll
            for (int k = 0; k < D / 8; ++k)
                u[k] = has ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const uint32_t e[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(e[z] << 16)),
                                           fabsf(__uint_as_float(e[z] & 0xFFFF0000u))));
            }
            const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 127, -119), 127);
            // a negative scale goes into q, so that c_row >= 0 keeps the order of the scores
            const float up = copysignf(__uint_as_float((uint32_t)(7 - e2 + 127) << 23), a.scale_log2);
            rc = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(e2 - 7 + 127) << 23);
            const uint32_t qd = sbase + kPrOffQ + (uint32_t)tile * 2 * kTileBytes;
            // an infinite or NaN q would saturate: its scores become NaN through c_row
            if (!(top < INFINITY))
                rc = __int_as_float(0x7FFFFFFF);
            bool nan = false;
#pragma unroll
            for (int k = 0; k < D / 8; k += 2) {
                uint32_t hi[4], lw[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint4 &uu = u[k + (y >> 1)];
                    const uint32_t e0 = (y & 1) ? uu.z : uu.x, e1 = (y & 1) ? uu.w : uu.y;
                    const float f0 = __uint_as_float(e0 << 16) * up, f1 = __uint_as_float(e0 & 0xFFFF0000u) * up;
                    const float f2 = __uint_as_float(e1 << 16) * up, f3 = __uint_as_float(e1 & 0xFFFF0000u) * up;
                    nan |= f0 != f0 || f1 != f1 || f2 != f2 || f3 != f3;
                    split_terms(f0, f1, f2, f3, hi[y], lw[y]);
                }
                sts128(qd + sw128(row, k >> 1), hi[0], hi[1], hi[2], hi[3]);
                sts128(qd + kTileBytes + sw128(row, k >> 1), lw[0], lw[1], lw[2], lw[3]);
            }
            if (nan)
                rc = __int_as_float(0x7FFFFFFF);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[kBQ]);
        }
        float m = -INFINITY, l = 0.0f, vref = 0.0f;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + (uint32_t)tile * 128u + lane_off;
        const uint32_t tO = tmem + 256u + (uint32_t)tile * 128u + lane_off;
        bool ok = true;
        if (tile == 0 || two) {
            for (int t = 0; t < T; ++t) {
                const uint32_t vph = (uint32_t)(t >> 1) & 1u;
                ok = ok && mbar_wait(&bar[kBSFull + tile], (uint32_t)t & 1u, abort_flag) &&
                     mbar_wait(&bar[kBVFull + (t & 1)], vph, abort_flag);
                if (!__all_sync(kFull, ok)) {
                    ok = false;
                    fail();
                    break;
                }
                tc_fence_after_sync();
                const float *const ksp = reinterpret_cast<const float *>(smem + kPrOffKs + (t % kMeta) * 512);
                const uint32_t tb = sbase + kPrOffTile + (uint32_t)(t % kMeta) * 32u;
                const uint4 mw = lds128(tb);
                const float vfac = __uint_as_float(lds32(tb + 16u));
                vref = __uint_as_float(lds32(tb + 20u));
                const uint32_t even = lds32(tb + 24u);
                const int past = lim - (t_0 + t) * kPrTok;
                // nothing of the tile is masked for any row of this warp
                const bool whole = (mw.x & mw.y & mw.z & mw.w) == 0xFFFFFFFFu &&
                                   __all_sync(kFull, past >= kPrTok - 1);
                const int how = !whole ? kMasked : even == 0x01010101u ? kEven : kWhole;
                // m is the largest score of the first tile that the row saw, and
                // moves again only when a tile's weights sum to more than 2^15:
                // till then every p fits f16, so the scores are read once and
                // the tile's maximum is not taken.
                float alpha = vfac, sum;
                uint32_t p[64];
                bool fix = __any_sync(kFull, m == -INFINITY);
#pragma unroll 1
                for (int round = 0;; ++round) {
                    if (fix) {
                        const float top = rc * (how == kMasked ? row_max<kMasked>(tS, ksp, tb, past)
                                                               : row_max<kWhole>(tS, ksp, tb, past));
                        if (top > m && (round > 0 || m == -INFINITY)) {
                            const float f = ex2_approx(m - top);
                            alpha *= f;
                            l *= f;
                            m = top;
                        }
                    }
                    const float ms = m == -INFINITY ? 0.0f : -m;
                    sum = how == kEven    ? weights<kEven>(tS, ksp, tb, past, rc, ms, p)
                          : how == kWhole ? weights<kWhole>(tS, ksp, tb, past, rc, ms, p)
                                          : weights<kMasked>(tS, ksp, tb, past, rc, ms, p);
                    fix = __any_sync(kFull, sum > 32768.0f);
                    if (!fix || round > 0)
                        break;
                }
                l += sum;
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
                    tmem_st16(tS + 16u * cc, p + 16 * cc);
                if (t > 0 && __any_sync(kFull, alpha != 1.0f)) {
                    // O holds tiles before this one: PV of tile t - 1 is done (SFull)
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; ++cc) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * cc, o);
                        tmem_ld_wait();
                        reg_fence_cols<32>(o);
#pragma unroll
                        for (int z = 0; z < 32; ++z)
                            o[z] = __float_as_uint(__uint_as_float(o[z]) * alpha);
                        tmem_st32(tO + 32u * cc, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[kBPFull + tile]);
            }
            // -------------------------------------------------------- output
            ok = ok && mbar_wait(&bar[kBODone], 0u, abort_flag);
            if (__all_sync(kFull, ok)) {
                tc_fence_after_sync();
                const float f = l == 0.0f ? 0.0f : vref * (1.0f / kVUp) / (pc.parts > 1 ? 1.0f : l);
                const long long at = (long long)blockIdx.x * kPrRows + tile * 128 + row;  // of a part
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[32];
                    if (T > 0) {
                        tmem_ld32(tO + 32u * cc, o);
                        tmem_ld_wait();
                        reg_fence_cols<32>(o);
                    }
                    if (has && pc.parts > 1) {
                        float4 *dst = reinterpret_cast<float4 *>(a.part + at * D + 32 * cc);
#pragma unroll
                        for (int z = 0; z < 8; ++z) {
                            float y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = l == 0.0f ? 0.0f : __uint_as_float(o[4 * z + e]) * f;
                            dst[z] = make_float4(y[0], y[1], y[2], y[3]);
                        }
                    } else if (has) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + rh * D + 32 * cc);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            uint32_t b[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const float f0 = l == 0.0f ? 0.0f : __uint_as_float(o[8 * z + 2 * y]) * f;
                                const float f1 = l == 0.0f ? 0.0f : __uint_as_float(o[8 * z + 2 * y + 1]) * f;
                                b[y] = __bfloat16_as_ushort(__float2bfloat16_rn(f0)) |
                                       (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f1)) << 16;
                            }
                            dst[z] = make_uint4(b[0], b[1], b[2], b[3]);
                        }
                    }
                }
                if (has && pc.parts > 1)
                    *reinterpret_cast<float2 *>(a.ml + at * 2) = make_float2(m, l);
                else if (has && a.lse)
                    a.lse[rh] = l == 0.0f ? -INFINITY : (m == -INFINITY ? l : (m + log2f(l)) * kLn2);
            } else {
                fail();
            }
        }
    } else if (warp < 12) {
        // -------------------------------------------------------- V conversion
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const int lt = tid - 256, lw = lt >> 5;
        float *const red = reinterpret_cast<float *>(smem + kPrOffRed);
        float vref = 0.0f;
        bool ok = true;
        int raw_slot = 0;
        uint32_t raw_ph = 0;
        for (int t = 0; t < T; ++t) {
            ok = ok && mbar_wait(&bar[kBKFull + t % kKStages], (uint32_t)(t / kKStages) & 1u, abort_flag) &&
                 mbar_wait(&bar[kBRawFull + raw_slot], raw_ph, abort_flag) &&
                 mbar_wait(&bar[kBVEmpty + (t & 1)], ((uint32_t)(t >> 1) & 1u) ^ 1u, abort_flag);
            const float *const ksp = reinterpret_cast<const float *>(smem + kPrOffKs + (t % kMeta) * 512);
            const float *const vsp = reinterpret_cast<const float *>(smem + kPrOffVs + (t % kMeta) * 512);
            const uint32_t tb = sbase + kPrOffTile + (uint32_t)(t % kMeta) * 32u;
            // vref: the largest |scale| so far; and do the warp's 32 tokens share one
            // key scale that is not negative?
            const float kmine = ksp[lt];
            // the largest and the smallest scale but 0 of the warp's 32 (a NaN counts as 0), as bits
            uint32_t vbits = __float_as_uint(vsp[lt]) & 0x7FFFFFFFu;
            vbits = vbits > 0x7F800000u ? 0u : vbits;
            const uint32_t top = __reduce_max_sync(kFull, vbits);
            const uint32_t least = __reduce_min_sync(kFull, vbits ? vbits : 0x7F800000u);
            const bool pow2 = __all_sync(kFull, (vbits & 0x7FFFFFu) == 0);
            const float klead = __shfl_sync(kFull, kmine, 0);
            const bool even = __all_sync(kFull, kmine >= 0.0f && kmine == klead);
            if (lane == 0) {
                red[8 * (t & 1) + lw] = __uint_as_float(top);
                red[8 * (t & 1) + 4 + lw] = pow2 ? __uint_as_float(least) : 0.0f;
                asm volatile("st.shared.u8 [%0], %1;" ::"r"(tb + 24u + (uint32_t)lw), "r"(even ? 1u : 0u) : "memory");
            }
            if (!named_bar_and(1, 128, ok)) {
                fail();
                break;
            }
            const float4 r4 = *reinterpret_cast<const float4 *>(red + 8 * (t & 1));
            const float4 s4 = *reinterpret_cast<const float4 *>(red + 8 * (t & 1) + 4);
            const float vmax = fmaxf(fmaxf(r4.x, r4.y), fmaxf(r4.z, r4.w));
            const float vmin = fminf(fminf(s4.x, s4.y), fminf(s4.z, s4.w));
            const float vnew = vmax > vref && vmax > 1e-36f ? vmax : vref;
            const float vfac = vnew > vref ? vref / vnew : 1.0f;
            vref = vnew;
            const float vinv = vref > 0.0f ? kVUp / vref : 0.0f;
            if (lt == 0)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tb + 16u), "r"(__float_as_uint(vfac)),
                             "r"(__float_as_uint(vref)) : "memory");
            const uint8_t *const raw = smem + kPrOffRaw + raw_slot * kTileBytes;
            uint8_t *const vd = smem + kPrOffV + (t & 1) * 2 * kTileBytes;
            // a thread converts 16 codes of a token at a time; the lanes of the upper
            // value columns take the neighbouring token, which spreads the stores
            // of both column blocks over all banks
            const int ch = lt % CH, flip = D == 128 ? ch >> 2 : 0;
            if (vmin < vref * 0x1p-30f || (__float_as_uint(vref) & 0x7FFFFFu) != 0) {
                // factors that f16 does not hold (a quotient that is no power of two, or too
                // small a one): products in fp32, rounded once. The choice is the tile's, the
                // loop rolled: 0.3 % on 6415 rows of 32 heads (unrolled 1.5 %, a choice per
                // token 4 to 7 %, for the instructions that are fetched or passed over).
#pragma unroll 1
                for (int k = 0; k < 4 * CH; ++k) {
                    // four codes of a thread's 16, of its k / 4-th token
                    const int tok = ((k >> 2) * (128 / CH) + lt / CH) ^ flip, col = 16 * ch + 4 * (k & 3);
                    const float f = vsp[tok] * vinv;
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2(*reinterpret_cast<const uint32_t *>(raw + tok * 128 + col), lo, hi);
                    *reinterpret_cast<uint2 *>(vd + (col >> 6) * kTileBytes + sw128(tok, (col & 63) >> 3) + 2 * (col & 4)) =
                        make_uint2(scale_f16x2(lo, f), scale_f16x2(hi, f));
                }
            } else {
#pragma unroll
                for (int k0 = 0; k0 < CH; k0 += 4) {
                    uint4 u[4];
                    float f[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = ((k0 + k) * (128 / CH) + lt / CH) ^ flip;
                        u[k] = *reinterpret_cast<const uint4 *>(raw + tok * 128 + ch * 16);
                        f[k] = vsp[tok] * vinv;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tok = ((k0 + k) * (128 / CH) + lt / CH) ^ flip;
                        const uint32_t f2 = pack_f16x2(f[k], f[k]);
                        uint32_t o[8];
                        e4m3x4_to_f16x2(u[k].x, o[0], o[1]);
                        e4m3x4_to_f16x2(u[k].y, o[2], o[3]);
                        e4m3x4_to_f16x2(u[k].z, o[4], o[5]);
                        e4m3x4_to_f16x2(u[k].w, o[6], o[7]);
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[y]) : "r"(f2));
                        // value columns 16 ch .. 16 ch + 15: chunks 2 ch, 2 ch + 1 of 8 columns each
                        uint8_t *const blk = vd + (ch >> 2) * kTileBytes;
                        const int c0 = (2 * ch) & 7;
                        *reinterpret_cast<uint4 *>(blk + sw128(tok, c0)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(blk + sw128(tok, c0 + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[kBVFull + (t & 1)]);
                mbar_arrive(&bar[kBRawEmpty + raw_slot]);
                mbar_arrive(&bar[kBKEmpty + t % kKStages]);
            }
            if (++raw_slot == kRawSlots) {
                raw_slot = 0;
                raw_ph ^= 1u;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 12 && lane == 0) {
        // -------------------------------------------------------- products
        constexpr uint32_t idq = idesc_e4m3_f32(128, 128);
        constexpr uint32_t idv = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | (8u << 24);
        const int tiles = two ? 2 : 1;
        auto scores = [&](int t, int tile) {
            const uint32_t qd = sbase + kPrOffQ + (uint32_t)tile * 2 * kTileBytes;
            const uint64_t kd = sw128_kmajor_desc(sbase + kPrOffK + (uint32_t)(t % kKStages) * kTileBytes);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
                const uint64_t ad = sw128_kmajor_desc(qd + (uint32_t)term * kTileBytes);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    umma_e4m3(tmem + (uint32_t)tile * 128u, ad + 2u * k, kd + 2u * k, term ? idq | kIdescAE5m2 : idq,
                              (term | k) ? 1u : 0u);
            }
            umma_commit(&bar[kBSFull + tile]);
        };
        bool ok = T == 0 || (mbar_wait(&bar[kBQ], 0u, abort_flag) && mbar_wait(&bar[kBKFull], 0u, abort_flag));
        if (ok && T > 0) {
            fence_proxy_async_smem();
            tc_fence_after_sync();
            for (int tile = 0; tile < tiles; ++tile)
                scores(0, tile);
            umma_commit(&bar[kBKEmpty]);
        }
        for (int t = 0; ok && t < T; ++t) {
            const bool more = t + 1 < T;
            ok = mbar_wait(&bar[kBVFull + (t & 1)], (uint32_t)(t >> 1) & 1u, abort_flag);
            if (more)
                ok = ok && mbar_wait(&bar[kBKFull + (t + 1) % kKStages], (uint32_t)((t + 1) / kKStages) & 1u, abort_flag);
            if (!ok)
                break;
            fence_proxy_async_smem();
            for (int tile = 0; ok && tile < tiles; ++tile) {
                ok = mbar_wait(&bar[kBPFull + tile], (uint32_t)t & 1u, abort_flag);
                if (!ok)
                    break;
                tc_fence_after_sync();
                const uint32_t vd = sbase + kPrOffV + (uint32_t)(t & 1) * 2 * kTileBytes;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_f16_ts(tmem + 256u + (uint32_t)tile * 128u, tmem + (uint32_t)tile * 128u + 8u * k,
                                sw128_mnmajor_desc(vd + (uint32_t)k * 2048u, kTileBytes, 1024u), idv,
                                (t | k) ? 1u : 0u);
                if (tile == tiles - 1)
                    umma_commit(&bar[kBVEmpty + (t & 1)]);
                if (more)
                    scores(t + 1, tile);
                if (more && tile == tiles - 1)
                    umma_commit(&bar[kBKEmpty + (t + 1) % kKStages]);
            }
        }
        if (!ok)
            fail();
        umma_commit(&bar[kBODone]);
        if (!mbar_wait(&bar[kBODone], 0u, nullptr))
            atomicOr(c.status, (uint32_t)PMQA_DEV_TIMEOUT);
        } else if (warp == 13 || warp == 14) {
            // ---------------------------------------------------- loaders
            // warp 13: K rows, both scales and the mask; warp 14: V codes. A lane
            // looks up tokens lane, lane + 32, ... of the tile, one tile ahead.
            const bool is_k = warp == 13;
            const uint8_t *const pool = is_k ? c.k : c.v;
            const int32_t *const bt = c.bt + (long long)req * c.W;
            constexpr uint32_t kNone = 0xFFFFFFFFu;
            constexpr int PER = 32 / CH;  // rows an instruction copies
            const int ch = lane % CH;
            int page[4];
            auto look_up = [&](int t) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = (t_0 + t) * kPrTok + 32 * k + lane;
                    page[k] = t < T && tok < end ? __ldg(bt + c.page_of(tok)) : -1;
                }
            };
            look_up(0);
            bool ok = true;
            int slot_i = 0;
            uint32_t ph = 1;
            const int slots = is_k ? kKStages : kRawSlots;
            for (int t = 0; t < T; ++t) {
                uint32_t phys[4], row[4];  // block * H + h, and row of the pool
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = (t_0 + t) * kPrTok + 32 * k + lane;
                    phys[k] = row[k] = kNone;
                    if (tok < end) {
                        if (page[k] < 0 || (long long)page[k] >= c.nb) {
                            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
                        } else {
                            phys[k] = (uint32_t)page[k] * (uint32_t)c.H + (uint32_t)h;
                            row[k] = phys[k] * (uint32_t)c.P + (uint32_t)(tok - c.page_of(tok) * c.P);
                        }
                    }
                }
                look_up(t + 1);
                ok = mbar_wait(&bar[(is_k ? kBKEmpty : kBRawEmpty) + slot_i], ph, abort_flag);
                ok = __all_sync(kFull, ok);
                if (!ok) {
                    fail();
                    break;
                }
                const uint32_t dst = sbase + (is_k ? kPrOffK : kPrOffRaw) + (uint32_t)slot_i * kTileBytes;
                if (is_k) {
                    const uint32_t meta = (uint32_t)(t % kMeta);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t at = meta * 512u + (uint32_t)(32 * k + lane) * 4u;
                        const uint32_t mask = __ballot_sync(kFull, phys[k] != kNone);
                        if (lane == 0)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + kPrOffTile + meta * 32u + 4u * k),
                                         "r"(mask) : "memory");
                        if (phys[k] != kNone) {
                            cp_async_4(sbase + kPrOffKs + at, c.ks + phys[k]);
                            cp_async_4(sbase + kPrOffVs + at, c.vs + phys[k]);
                        } else {
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + kPrOffKs + at), "r"(0) : "memory");
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + kPrOffVs + at), "r"(0) : "memory");
                        }
                    }
                }
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const uint32_t mine = k & 2 ? (k & 1 ? row[3] : row[2]) : k & 1 ? row[1] : row[0];
#pragma unroll
                    for (int y = 0; y < CH; ++y) {
                        const int rr = y * PER + lane / CH, rt = 32 * k + rr;
                        const uint32_t src = __shfl_sync(kFull, mine, rr);
                        cp_async_16(dst + (is_k ? sw128(rt, ch) : (uint32_t)(rt * 128 + ch * 16)),
                                    pool + (src == kNone ? 0ull : (unsigned long long)src * D) + ch * 16,
                                    src == kNone ? 0u : 16u);
                    }
                }
                uint64_t *const full = &bar[(is_k ? kBKFull : kBRawFull) + slot_i];
                cp_async_arrive_noinc(full);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full);  // releases the plain stores (masks, zero scales)
                if (++slot_i == slots) {
                    slot_i = 0;
                    ph ^= 1u;
                }
            }
            cp_async_wait_all();
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Requests with at least `least` packed rows (rows * group).
// parts: CTAs that contexts may be cut over (launch_attn_join follows), or 0.
cudaError_t launch_attn_prompt(AttnCall &q, int least, int parts, cudaStream_t st)
{
    PromptArgs a{};
    a.c = q.c;
    a.q = static_cast<const uint16_t *>(q.q);
    a.out = static_cast<uint16_t *>(q.out);
    a.lse = q.lse;
    a.scale_log2 = q.sm_scale * kLog2e;
    a.heads = q.heads;
    a.group = q.heads / q.c.H;
    a.least = least;
    a.slots = (long long)q.c.rows * a.group / kPrRows + q.c.bs;
    a.parts = parts;
    a.meta = reinterpret_cast<int4 *>(q.ws + kWsPromptMeta);
    a.ml = reinterpret_cast<float *>(q.ws + kWsPromptMl);
    a.part = reinterpret_cast<float *>(q.ws + kWsPromptPart);
    const long long grid = a.slots * q.c.H + parts;
    if (grid > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> done64{0}, done128{0};
    cudaError_t e = q.c.D == 128 ? allow_smem(cache_prompt_kernel<128>, (int)kPrSmem, done128)
                                 : allow_smem(cache_prompt_kernel<64>, (int)kPrSmem, done64);
    if (e != cudaSuccess)
        return e;
    if (q.c.D == 128)
        cache_prompt_kernel<128><<<(unsigned)grid, kPrThreads, kPrSmem, st>>>(a);
    else
        cache_prompt_kernel<64><<<(unsigned)grid, kPrThreads, kPrSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace pmqa
