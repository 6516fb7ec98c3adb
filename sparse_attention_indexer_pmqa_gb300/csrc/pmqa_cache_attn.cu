// pmqa_cache_attn.cu -- attention over the paged 8-bit K/V cache for requests
// with few query rows (decode, speculative verify), and the kernel that joins
// split contexts.
//
// For query row j of request i and query head hq (kv head h = hq / group):
//   x_t = sm_scale log2(e) ks_t (q . K_t),  p_t = 2^(x_t - m),  l = sum p_t,
//   out = sum_t p_t vs_t V_t / l,           lse = (m + log2 l) ln 2,
// one pass over the tokens with a running m (a row's maximum, moved only when a
// token exceeds it by more than 2^8).
//
// Bound by HBM: each token and kv head costs 2 D bytes and 4 D flops per query
// row, so with R rows per kv head the arithmetic is 2 R flops a byte; at R <=
// 32 that is far below the ridge. The layout follows from that:
//   * the items (request, kv head, block of 8 NT rows, tile of 128 tokens) are
//     flattened and split evenly over the CTAs, so contexts of any mix of
//     lengths finish together; a context cut between CTAs leaves (O, m, l)
//     parts in the workspace and the second kernel joins them;
//   * every warp takes 32 of a tile's 128 tokens through its own ring of cp.async
//     stages and never waits for another warp inside a context. Two blocks of 16
//     tokens in flight hide the products' latency better than more warps do (16
//     tokens, and three CTAs per SM where registers allow: 127 us instead of 102
//     for 32 contexts of 32 k tokens, 2 kv heads and 16 rows; 188 instead of 154
//     with 32 rows; 96 instead of 94 with 8);
//   * products run as S^T = K Q^T and O^T = V^T P^T, so the 16 rows of the
//     m16n8k16 shape are tokens (then value columns) and the 8 columns are
//     query rows: a group of 8 wastes nothing, the softmax weights of a thread
//     stay in its registers (one movmatrix makes the second product's
//     operand), and O costs 32 registers per 8 rows at D = 128;
//   * e4m3 to f16 is exact; q is scaled by a power of two per row so that its
//     largest value lies in [2^14, 2^15) (bf16 values within 2^-31 of it
//     exactly representable in f16); p is rounded to f16 (2^-12 relative), the
//     only rounding before the bf16 output; sums, m, l and O are fp32.
// 64 contexts of 4 to 32 k tokens, 64 query heads over 8: 380 us, 94 % of the
// measured copy rate. With 16 rows 5.3 TB/s and with 32 rows 3.5 TB/s are left (32
// contexts of 32 k): there the products (8 cycles each and scheduler) and their
// latencies bind, O of 32 rows leaves room for two warps per scheduler only.
#include <algorithm>
#include <cmath>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace cache {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kTok = 32;  // tokens of a warp's step
constexpr int kTile = kAttnWarps * kTok;
constexpr float kSlack = 8.0f;    // p <= 2^8 before the maximum moves
constexpr int kPad = 2;           // what a context's start and end cost, in tiles: 16 requests
                                  // of 1 to 4096 tokens take 22 us with it, 31 without
constexpr int kLeastTiles = 2;    // fewest tiles a CTA takes (small problems)
// Joining one more part, in tiles: with it 60000 tokens of one kv head take 25 us (8
// rows) and 37 us (32), cut over every CTA 70 and 54.
constexpr float kJoinCost = 0.15f;
constexpr int kWholeTokens = 640;

struct AttnArgs {
    View c;
    const uint16_t *q;   // bf16 [rows, heads, D]
    uint16_t *out;       // bf16 [rows, heads, D]
    float *lse;          // [rows, heads] or null
    float scale_log2;    // sm_scale log2(e)
    int heads, group;
    int least, most;     // requests with least <= n group <= most are this kernel's
    int whole;           // contexts are short: none is cut between CTAs
    int4 *meta;          // per CTA: (i, h, b, 2 parts + (slot & 1)) of the context it leaves open
    float *ml;           // [2 CTAs][8 NT][2]
    float *part;         // [2 CTAs][8 NT][D]
};

// A warp's stage: 32 K rows, 32 V rows, 32 + 32 scales, the mask of tokens
// that exist. 16-byte chunk c of row r is stored at a place that spreads both
// access patterns (8 tokens x 4 chunks for K, 4 tokens x 2 chunks for V) over
// all banks.
template <int D>
struct Stage {
    static constexpr uint32_t kRows = kTok * D;
    static constexpr uint32_t kOffKs = 2 * kRows, kOffVs = kOffKs + 4 * kTok, kOffMask = kOffVs + 4 * kTok;
    static constexpr uint32_t kBytes = kOffMask + 16;
    __device__ static __forceinline__ uint32_t at(int r, int c)
    {
        if constexpr (D == 128)
            return (uint32_t)(r * 128 + ((c ^ ((((r >> 1) & 3) << 1) ^ ((r & 1) << 2))) << 4));
        else
            return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (((r >> 1) & 3) << 1)) << 4));
    }
};

template <int D, int NT>
struct AttnShape {
    static constexpr int kStages = D == 64 ? 3 : 2;  // what leaves room for kOcc CTAs per SM
    static constexpr int kRows = 8 * NT;
    static constexpr int kPitch = D + 4;  // floats per row of the merge buffer
    static constexpr uint32_t kRing = kAttnWarps * kStages * Stage<D>::kBytes;
    static constexpr uint32_t kOffMerge = kRing;
    static constexpr uint32_t kOffMl = kOffMerge + kAttnWarps * 8 * kPitch * 4;
    static constexpr uint32_t kOffQ = kOffMl + kAttnWarps * kRows * 8;
    // 32 rows: q's operand in shared memory, the registers go to O. Every warp writes
    // the same values there; a context's end has all of them wait for one another.
    static constexpr bool kQShared = NT == 4;
    static constexpr uint32_t kOffRows = kOffQ + (kQShared ? (D / 16) * NT * 32 * 8 : 0u);
    static constexpr uint32_t kSmem = kOffRows + (kQShared ? kRows * 8 : 0u);  // a factor, a last slot
    static constexpr int kOcc = D == 64 && NT < 4 ? 3 : 2;
};

template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<D, NT>::kOcc)
    cache_attn_kernel(const __grid_constant__ AttnArgs a)
{
    using Sh = AttnShape<D, NT>;
    using St = Stage<D>;
    constexpr int S = Sh::kStages;
    constexpr int ROWS = Sh::kRows;
    constexpr int KS = D / 16;   // k steps of the first product
    constexpr int MT = D / 16;   // 16-column tiles of the second
    constexpr int U = kTok / 16;  // m16 blocks of a step
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const View &c = a.c;
    const int G = a.group;
    griddep_launch_dependents();

    Range rg;
    Walk w;
    find_range<kTile, ROWS, kPad, kAttnThreads>(c, G, a.least, a.most, kLeastTiles, kJoinCost, rg, w);
    if (rg.x0 >= rg.x1) {
        if (tid == 0)
            a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
        griddep_wait();
        return;
    }
    long long x = rg.x0;
    if (w.t >= w.T || (a.whole && w.t > 0)) {
        // the range starts behind a context's tiles; or (uncut) a context belongs to
        // the CTA whose range holds its first tile
        x += w.T + kPad - w.t;
        w.t = w.T - 1;
        if (x < rg.x1)
            w.template next<kTile, ROWS, kPad>(c, G, a.least, a.most);
    }
    if (x >= rg.x1) {
        if (tid == 0)
            a.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
        griddep_wait();
        return;
    }
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * S) * St::kBytes;
    float *const merge = reinterpret_cast<float *>(smem + Sh::kOffMerge);
    float2 *const mls = reinterpret_cast<float2 *>(smem + Sh::kOffMl);

    // tokens of request q that some row of row block b sees
    auto seen_end = [&](const Request &q, int b) {
        const int last = min(q.n - 1, (b * ROWS + ROWS - 1) / G);
        return max(0, q.ctx - q.n + last + 1);
    };

    // ---------------------------------------------------------- producer state
    // `pw` is the item whose table entry is loaded (pend_*); its copies are
    // issued one step later.
    Walk pw = w;
    long long p_x = x;          // its index
    bool p_more = true;         // it is one of this CTA's
    int p_end = seen_end(pw.q, pw.b);
    int pend_page = -1, pend_off = 0, pend_h = 0;
    bool pend_in = false;       // this lane's token is one that a row sees
    auto look_up = [&]() {
        pend_in = false;
        if (p_more) {
            const int tok = pw.t * kTile + warp * kTok + lane;
            pend_in = tok < p_end;
            const int pg = c.page_of(tok);
            pend_off = tok - pg * c.P;
            pend_h = pw.h;
            if (pend_in)
                pend_page = __ldg(c.bt + (long long)pw.i * c.W + pg);
            ++p_x;
            if (pw.t + 1 < pw.T) {
                ++pw.t;
                p_more = p_x < rg.x1 || a.whole;
            } else {
                p_x += kPad;
                p_more = p_x < rg.x1;
                if (p_more) {
                    pw.template next<kTile, ROWS, kPad>(c, G, a.least, a.most);
                    p_end = seen_end(pw.q, pw.b);
                }
            }
        }
    };
    constexpr int CH = D / 16, PER = 32 / CH;  // chunks a row, rows an instruction
    const int ch = lane % CH;
    const bool one_block = (c.P & 15) == 0;  // 16 tokens never leave a block
    int p_slot = 0;
    auto issue = [&]() {
        const uint32_t st = ring + (uint32_t)p_slot * St::kBytes;
        if (++p_slot == S)
            p_slot = 0;
        bool ok = pend_in;
        if (ok && (uint32_t)pend_page >= (uint32_t)min(c.nb, 0x7FFFFFFFll)) {
            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
            ok = false;
        }
        const uint32_t mask = __ballot_sync(kFull, ok);
        if (lane == 0)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + St::kOffMask), "r"(mask) : "memory");
        if (mask) {
            // block * H + head, and the row of the pool (both below 2^32)
            const uint32_t phys = ok ? (uint32_t)pend_page * (uint32_t)c.H + (uint32_t)pend_h : 0u;
            const uint32_t row = phys * (uint32_t)c.P + (uint32_t)pend_off;
            const uint32_t sdst = st + (uint32_t)lane * 4u;
            if (ok) {
                cp_async_4(sdst + St::kOffKs, c.ks + phys);
                cp_async_4(sdst + St::kOffVs, c.vs + phys);
            } else {
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sdst + St::kOffKs), "r"(0) : "memory");
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sdst + St::kOffVs), "r"(0) : "memory");
            }
            if (one_block) {
                // of 16 tokens the first exists if any does: rows on end from its own
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint64_t src = (uint64_t)__shfl_sync(kFull, row, 16 * u) * D + (uint32_t)lane * 16u;
                    const uint8_t *const ks = c.k + src, *const vs = c.v + src;
#pragma unroll
                    for (int k = 0; k < 16 / PER; ++k) {
                        const int r = 16 * u + k * PER + lane / CH;
                        const uint32_t nb = (mask >> r) & 1u ? 16u : 0u;
                        cp_async_16(st + St::at(r, ch), ks + k * 512, nb);
                        cp_async_16(st + St::kRows + St::at(r, ch), vs + k * 512, nb);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < kTok / PER; ++k) {
                    const int r = k * PER + lane / CH;
                    const uint32_t nb = (mask >> r) & 1u ? 16u : 0u;
                    const uint32_t rr = __shfl_sync(kFull, row, r);
                    const uint64_t src = (uint64_t)(nb ? rr : 0u) * D + (uint32_t)ch * 16u;
                    cp_async_16(st + St::at(r, ch), c.k + src, nb);
                    cp_async_16(st + St::kRows + St::at(r, ch), c.v + src, nb);
                }
            }
        }
        cp_async_commit();
    };

    look_up();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) {
        issue();
        look_up();
    }

    // ---------------------------------------------------------- consumer state
    float acc[NT][MT][4];
    constexpr int NQ = Sh::kQShared ? 1 : NT;
    uint32_t qb[NQ][KS][2];
    uint2 *const qsm = reinterpret_cast<uint2 *>(smem + Sh::kOffQ) + lane;
    float m[NT][2], l[NT][2], rc[NQ][2];
    int lim[NQ][2];               // last slot that the row sees, -1 for padding
    float2 *const rows_c = reinterpret_cast<float2 *>(smem + Sh::kOffRows);
    int2 *const rows_lim = reinterpret_cast<int2 *>(rows_c + ROWS / 2);
    float vref = 0.0f, vinv = 0.0f, vtop = 0.0f;
    int seg = -1, end = 0, c_slot = 0;
    const long long x_first = x;
    int4 open = make_int4(0, 0, 0, 0);
    bool fresh = true;
#pragma unroll 1
    for (;;) {
        if (fresh) {
            fresh = false;
            ++seg;
            end = seen_end(w.q, w.b);
            vref = vinv = vtop = 0.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // this thread's part of query row g of the block: 16 dims of each 64
                const int R = w.b * ROWS + nt * 8 + g;
                const bool has = R < w.q.n * G;
                const uint16_t *src =
                    a.q + ((long long)(w.q.r0 + R / G) * a.heads + w.h * G + R % G) * D + 16 * t4;
                uint4 u[D / 32];
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    u[k] = has ? __ldg(reinterpret_cast<const uint4 *>(src + (k >> 1) * 64 + (k & 1) * 8))
                               : make_uint4(0, 0, 0, 0);
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint32_t e[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(e[z] << 16)),
                                               fabsf(__uint_as_float(e[z] & 0xFFFF0000u))));
                }
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
                const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 127, -112), 127);
                const float up = __uint_as_float((uint32_t)(14 - e2 + 127) << 23);
                const float down = __uint_as_float((uint32_t)(e2 - 14 + 127) << 23);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint32_t e[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        // dims 8 (k & 1) + 2 z of this thread's 16: k step (k >> 1) * 4 + (k & 1) * 2 + z / 2
                        const float lo = __uint_as_float(e[z] << 16) * up;
                        const float hi = __uint_as_float(e[z] & 0xFFFF0000u) * up;
                        qb[Sh::kQShared ? 0 : nt][(k >> 1) * 4 + (k & 1) * 2 + (z >> 1)][z & 1] = pack_f16x2(lo, hi);
                    }
                }
                if constexpr (Sh::kQShared) {
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        qsm[(nt * KS + k) * 32] = make_uint2(qb[0][k][0], qb[0][k][1]);
                }
                // an infinite value would leave its row the tokens of score -inf: NaN instead
                const float mine = top < INFINITY ? a.scale_log2 * down : __int_as_float(0x7FFFFFFF);
                constexpr auto at = [](int k) { return Sh::kQShared ? 0 : k; };
                rc[at(nt)][0] = __shfl_sync(kFull, mine, 8 * t4);
                rc[at(nt)][1] = __shfl_sync(kFull, mine, 8 * t4 + 4);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int Re = w.b * ROWS + nt * 8 + 2 * t4 + e;
                    lim[at(nt)][e] = Re < w.q.n * G ? w.q.ctx - w.q.n + Re / G : -1;
                    m[nt][e] = -INFINITY;
                    l[nt][e] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[nt][j][e] = 0.0f;
                if constexpr (Sh::kQShared) {
                    rows_c[nt * 4 + t4] = make_float2(rc[0][0], rc[0][1]);
                    rows_lim[nt * 4 + t4] = make_int2(lim[0][0], lim[0][1]);
                }
            }
        }
        cp_async_wait_group<S - 2>();
        __syncwarp();
        issue();
        look_up();
        const uint32_t st = ring + (uint32_t)c_slot * St::kBytes;
        if (++c_slot == S)
            c_slot = 0;
        const int base = w.t * kTile + warp * kTok;
        const uint32_t mask = base < end ? lds32(st + St::kOffMask) : 0u;
        if (mask) {
            float s[U][NT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[u][nt][e] = 0.0f;
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 ka = lds128(st + St::at(16 * u + g, half * 4 + t4));
                    const uint4 kb = lds128(st + St::at(16 * u + g + 8, half * 4 + t4));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16x2(wa[z], a0, a2);
                        e4m3x4_to_f16x2(wb[z], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (Sh::kQShared) {
                                const uint2 b = qsm[(nt * KS + half * 4 + z) * 32];
                                mma_f16(s[u][nt], a0, a1, a2, a3, b.x, b.y);
                            } else {
                                mma_f16(s[u][nt], a0, a1, a2, a3, qb[nt][half * 4 + z][0], qb[nt][half * 4 + z][1]);
                            }
                        }
                    }
                }
            // scales of tokens 16 u + g and 16 u + g + 8
            float ks[U][2], vs[U][2], vmax = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t at = st + 4u * (uint32_t)(16 * u + 8 * y + g);
                    ks[u][y] = __uint_as_float(lds32(at + St::kOffKs));
                    vs[u][y] = __uint_as_float(lds32(at + St::kOffVs));
                    vmax = fmaxf(vmax, fabsf(vs[u][y]));
                }
            // every row sees every token of the chunk (no mask to apply)
            const bool whole = mask == kFull && base + kTok - 1 <= w.q.ctx - w.q.n;
            bool exceed = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 f = Sh::kQShared ? rows_c[nt * 4 + t4]
                                              : make_float2(rc[nt % NQ][0], rc[nt % NQ][1]);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][nt][0] *= ks[u][0] * f.x;
                    s[u][nt][1] *= ks[u][0] * f.y;
                    s[u][nt][2] *= ks[u][1] * f.x;
                    s[u][nt][3] *= ks[u][1] * f.y;
                    if (!whole) {
                        const int2 end2 = Sh::kQShared ? rows_lim[nt * 4 + t4]
                                                       : make_int2(lim[nt % NQ][0], lim[nt % NQ][1]);
                        const int r = 16 * u + g;
                        const bool k0 = (mask >> r) & 1u, k1 = (mask >> (r + 8)) & 1u;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (!k0 || base + r > (e ? end2.y : end2.x))
                                s[u][nt][e] = -INFINITY;
                            if (!k1 || base + r + 8 > (e ? end2.y : end2.x))
                                s[u][nt][2 + e] = -INFINITY;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float top = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
                    top = fmaxf(top, fmaxf(s[U - 1][nt][e], s[U - 1][nt][2 + e]));
                    exceed |= top > m[nt][e] + kSlack;
                }
            }
            if (__any_sync(kFull, exceed)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
                        top = fmaxf(top, fmaxf(s[U - 1][nt][e], s[U - 1][nt][2 + e]));
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
                        if (top > m[nt][e]) {
                            const float alpha = ex2_approx(m[nt][e] - top);
                            m[nt][e] = top;
                            l[nt][e] *= alpha;
#pragma unroll
                            for (int j = 0; j < MT; ++j) {
                                acc[nt][j][e] *= alpha;
                                acc[nt][j][2 + e] *= alpha;
                            }
                        }
                    }
            }
            // O is held in units of vref; p takes the token's scale over vref.
            // vref moves when the chunk's largest scale leaves [2^-5, 2^5] vref
            // (not to scales under 2^-60 of the largest seen: blocks of zeros).
            if (__any_sync(kFull, vmax > 32.0f * vref) || __all_sync(kFull, 32.0f * vmax < vref)) {
                vmax = fmaxf(vmax, __shfl_xor_sync(kFull, vmax, 4));
                vmax = fmaxf(vmax, __shfl_xor_sync(kFull, vmax, 8));
                vmax = fmaxf(vmax, __shfl_xor_sync(kFull, vmax, 16));
                if (vmax > 1e-36f && vmax >= vtop * 8.6736174e-19f) {
                    const float f = vref / vmax;
                    vref = vmax;
                    vinv = 1.0f / vmax;
                    vtop = fmaxf(vtop, vmax);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < MT; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[nt][j][e] *= f;
                }
            }
            uint32_t pb[U][NT][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float rv0 = vs[u][0] * vinv, rv1 = vs[u][1] * vinv;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
                    const float m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
                    const float p0 = ex2_approx(s[u][nt][0] - m0), p1 = ex2_approx(s[u][nt][1] - m1);
                    const float p2 = ex2_approx(s[u][nt][2] - m0), p3 = ex2_approx(s[u][nt][3] - m1);
                    l[nt][0] += p0 + p2;
                    l[nt][1] += p1 + p3;
                    pb[u][nt][0] = transpose8x8(pack_f16x2(p0 * rv0, p1 * rv0));
                    pb[u][nt][1] = transpose8x8(pack_f16x2(p2 * rv1, p3 * rv1));
                }
            }
            // value columns: D = 128, thread g holds dims 16 g .. 16 g + 15; D = 64, 8 g .. 8 g + 7
            constexpr int VW = D / 32;  // 32-bit words per token and thread
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t v[4][VW];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 16 * u + 2 * t4 + (k & 1) + (k >> 1) * 8;
                    if constexpr (D == 128) {
                        const uint4 y = lds128(st + St::kRows + St::at(r, g));
                        v[k][0] = y.x;
                        v[k][1] = y.y;
                        v[k][2] = y.z;
                        v[k][3] = y.w;
                    } else {
                        const uint32_t ad = st + St::kRows + St::at(r, g >> 1) + (uint32_t)(g & 1) * 8u;
                        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[k][0]), "=r"(v[k][1]) : "r"(ad));
                    }
                }
#pragma unroll
                for (int z = 0; z < VW; ++z) {
                    uint32_t f[2][2], h[2][2];
                    e4m3x4_to_f16x2(__byte_perm(v[0][z], v[1][z], 0x5140), f[0][0], f[0][1]);
                    e4m3x4_to_f16x2(__byte_perm(v[2][z], v[3][z], 0x5140), h[0][0], h[0][1]);
                    e4m3x4_to_f16x2(__byte_perm(v[0][z], v[1][z], 0x7362), f[1][0], f[1][1]);
                    e4m3x4_to_f16x2(__byte_perm(v[2][z], v[3][z], 0x7362), h[1][0], h[1][1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            mma_f16(acc[nt][2 * z + y], f[y][0], f[y][1], h[y][0], h[y][1], pb[u][nt][0],
                                    pb[u][nt][1]);
                }
            }
        }
        ++x;
        if (w.t + 1 < w.T && (x < rg.x1 || a.whole)) {
            ++w.t;
            continue;
        }

        // ------------------------------------------- the end of a context (or of this CTA's part)
        // thread (g, t4) holds rows 2 t4, 2 t4 + 1 of each 8 and D / 8 value columns from g D / 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(kFull, sum, 4);
                sum += __shfl_xor_sync(kFull, sum, 8);
                sum += __shfl_xor_sync(kFull, sum, 16);
                if (g == 0)
                    mls[warp * ROWS + nt * 8 + 2 * t4 + e] = make_float2(m[nt][e], sum);
            }
        __syncthreads();
        const bool starts = x - x_first > w.t;  // the context's first tile was this CTA's too
        const bool ends = w.t + 1 == w.T;
        const int slot = 2 * (int)blockIdx.x + (seg > 0 ? 1 : 0);
        const bool split = !(starts && ends);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * t4 + e;
                float M = -INFINITY;
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k)
                    M = fmaxf(M, mls[k * ROWS + row].x);
                const float f = m[nt][e] == -INFINITY ? 0.0f : ex2_approx(m[nt][e] - M) * vref;
                float *dst = merge + (warp * 8 + 2 * t4 + e) * Sh::kPitch + g * (D / 8);
                // a NaN sum keeps its NaN: weight 0 is only for a warp without tokens
#pragma unroll
                for (int j = 0; j < MT; j += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * j) =
                        make_float4(acc[nt][j][e] * f, acc[nt][j][2 + e] * f, acc[nt][j + 1][e] * f,
                                    acc[nt][j + 1][2 + e] * f);
            }
            __syncthreads();
            constexpr int TPR = D / 4;                    // threads per row
            constexpr int RPP = kAttnThreads / TPR;       // rows per pass
#pragma unroll
            for (int r8 = tid / TPR; r8 < 8; r8 += RPP) {
                const int row = nt * 8 + r8, col = (tid % TPR) * 4;
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k)
                    M = fmaxf(M, mls[k * ROWS + row].x);
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kAttnWarps; ++k) {
                    const float2 q2 = mls[k * ROWS + row];
                    L += q2.x == -INFINITY ? q2.y : q2.y * ex2_approx(q2.x - M);
                    const float4 u = *reinterpret_cast<const float4 *>(merge + (k * 8 + r8) * Sh::kPitch + col);
                    o.x += u.x;
                    o.y += u.y;
                    o.z += u.z;
                    o.w += u.w;
                }
                if (split) {
                    __stcg(reinterpret_cast<float4 *>(a.part + ((long long)slot * ROWS + row) * D + col), o);
                    if (col == 0)
                        __stcg(reinterpret_cast<float2 *>(a.ml + ((long long)slot * ROWS + row) * 2),
                               make_float2(M, L));
                } else {
                    const int R = w.b * ROWS + row;
                    if (R < w.q.n * G) {
                        const long long rh = (long long)(w.q.r0 + R / G) * a.heads + w.h * G + R % G;
                        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                        uint2 b;
                        b.x = __bfloat16_as_ushort(__float2bfloat16_rn(o.x * inv)) |
                              (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(o.y * inv)) << 16;
                        b.y = __bfloat16_as_ushort(__float2bfloat16_rn(o.z * inv)) |
                              (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(o.w * inv)) << 16;
                        *reinterpret_cast<uint2 *>(a.out + rh * D + col) = b;
                        if (a.lse && col == 0)
                            a.lse[rh] = L == 0.0f ? -INFINITY : (M == -INFINITY ? L : (M + log2f(L)) * kLn2);
                    }
                }
            }
            __syncthreads();
        }
        if (starts && !ends) {
            // this CTA is the first of several: it names the parts for the joining kernel
            const long long last = x - 1 + (w.T - 1 - w.t);
            const int cta = (int)(((last + 1) * rg.C - 1) / rg.total);
            open = make_int4(w.i, w.h, w.b, 2 * (cta - (int)blockIdx.x + 1) + (slot & 1));
        }
        x += kPad;
        if (x >= rg.x1)
            break;
        fresh = true;
        w.template next<kTile, ROWS, kPad>(c, G, a.least, a.most);
    }
    cp_async_wait_all();
    if (tid == 0)
        a.meta[blockIdx.x] = open;
    // behind the many-row kernel this one starts early; it ends after it
    griddep_wait();
}

// Joins the parts of the contexts that a kernel cut: block (c, y) takes 4 rows at a
// time of the context that CTA c began and left open. Each row's weights 2^(m_k - M)
// are worked out once, then every thread adds its 4 columns over the parts. ROWS:
// rows of a part; SLOTS: parts that a CTA may leave.
template <int D, int ROWS, int SLOTS>
__global__ void __launch_bounds__(D) cache_attn_join_kernel(const __grid_constant__ AttnArgs a)
{
    __shared__ float s_w[4][kMaxCtas];
    __shared__ float s_M[4], s_L[4];
    griddep_wait();
    const int4 meta = a.meta[blockIdx.x];
    const int parts = meta.w >> 1;
    if (parts == 0)
        return;
    const int h = meta.y, b = meta.z;
    const Request q = load_request(a.c, meta.x, false);
    // part k in the first slot of CTA c + k, part 0 where CTA c put it
    auto slot_of = [&](int k) { return SLOTS * ((int)blockIdx.x + k) + (k == 0 ? meta.w & 1 : 0); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int y = (int)blockIdx.y * 4; y < ROWS && b * ROWS + y < q.n * a.group; y += 4 * (int)gridDim.y) {
        for (int r = warp; r < 4; r += D / 32) {
            const int row = y + r;
            float M = -INFINITY;
            for (int k = lane; k < parts; k += 32)
                M = fmaxf(M, a.ml[((long long)slot_of(k) * ROWS + row) * 2]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
            float L = 0.0f;
            for (int k = lane; k < parts; k += 32) {
                const float2 p = *reinterpret_cast<const float2 *>(a.ml + ((long long)slot_of(k) * ROWS + row) * 2);
                const float f = p.x == -INFINITY ? (p.y == 0.0f ? 0.0f : 1.0f) : ex2_approx(p.x - M);
                s_w[r][k] = f;
                L += f * p.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                L += __shfl_xor_sync(kFull, L, o);
            if (lane == 0) {
                s_M[r] = M;
                s_L[r] = L;
            }
        }
        __syncthreads();
        const int r = threadIdx.x / (D / 4), col = (threadIdx.x % (D / 4)) * 4;
        const int row = y + r, R = b * ROWS + row;
        if (R < q.n * a.group) {
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
                const float f = s_w[r][k];
                const float4 u =
                    *reinterpret_cast<const float4 *>(a.part + ((long long)slot_of(k) * ROWS + row) * D + col);
                o.x += f * u.x;
                o.y += f * u.y;
                o.z += f * u.z;
                o.w += f * u.w;
            }
            const float M = s_M[r], L = s_L[r], inv = L == 0.0f ? 0.0f : 1.0f / L;
            const long long rh = (long long)(q.r0 + R / a.group) * a.heads + h * a.group + R % a.group;
            uint2 bb;
            bb.x = __bfloat16_as_ushort(__float2bfloat16_rn(o.x * inv)) |
                   (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(o.y * inv)) << 16;
            bb.y = __bfloat16_as_ushort(__float2bfloat16_rn(o.z * inv)) |
                   (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(o.w * inv)) << 16;
            *reinterpret_cast<uint2 *>(a.out + rh * D + col) = bb;
            if (a.lse && col == 0)
                a.lse[rh] = L == 0.0f ? -INFINITY : (M == -INFINITY ? L : (M + log2f(L)) * kLn2);
        }
        __syncthreads();
    }
}

template <int D, int NT>
static cudaError_t launch_rows(AttnArgs &a, uint8_t *ws, int sms, bool early, cudaStream_t st)
{
    using Sh = AttnShape<D, NT>;
    const int grid = std::min(sms * Sh::kOcc, NT == 4 ? kMaxWide : kMaxCtas);
    a.meta = reinterpret_cast<int4 *>(ws + kWsMeta);
    a.ml = reinterpret_cast<float *>(ws + kWsMl);
    a.part = reinterpret_cast<float *>(ws + kWsPart);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(cache_attn_kernel<D, NT>, (int)Sh::kSmem, done);
    if (e != cudaSuccess)
        return e;
    e = launch_early(cache_attn_kernel<D, NT>, dim3((unsigned)grid), kAttnThreads, Sh::kSmem, early, st, a);
    if (e != cudaSuccess || a.whole)
        return e;
    return launch_early(cache_attn_join_kernel<D, Sh::kRows, 2>, dim3((unsigned)grid, 2 * NT), D, 0, true, st, a);
}

static AttnArgs arguments(const AttnCall &q)
{
    AttnArgs a{};
    a.c = q.c;
    a.q = static_cast<const uint16_t *>(q.q);
    a.out = static_cast<uint16_t *>(q.out);
    a.lse = q.lse;
    a.scale_log2 = q.sm_scale * kLog2e;
    a.heads = q.heads;
    a.group = q.heads / q.c.H;
    return a;
}

// Joins what the many-row kernel cut (`parts` as in its launch). Every kernel
// between the two ends after that one.
cudaError_t launch_attn_join(AttnCall &q, int parts, cudaStream_t st)
{
    AttnArgs a = arguments(q);
    a.meta = reinterpret_cast<int4 *>(q.ws + kWsPromptMeta);
    a.ml = reinterpret_cast<float *>(q.ws + kWsPromptMl);
    a.part = reinterpret_cast<float *>(q.ws + kWsPromptPart);
    const dim3 grid((unsigned)parts, 16);
    return q.c.D == 128
               ? launch_early(cache_attn_join_kernel<128, kPromptRows, 1>, grid, 128, 0, true, st, a)
               : launch_early(cache_attn_join_kernel<64, kPromptRows, 1>, grid, 64, 0, true, st, a);
}

// Requests with least <= rows * group <= most. early: the kernel before this one
// in the stream is the many-row kernel of the same call.
cudaError_t launch_attn_rows(AttnCall &q, int least, int most, int sms, bool early, cudaStream_t st)
{
    AttnArgs a = arguments(q);
    a.least = least;
    a.most = most;
    // A table of at most kWholeTokens tokens: uncut, one CTA reads 500 tokens in
    // 9.7 us and 640 in 11.0; cut and joined, 9.9 and 10.4 us and a second launch,
    // which costs the host about 4 us. (The CTA that writes the last part as the joining
    // one saves that launch, but 4000 tokens then take 18 us instead of 15, and
    // 60000 take 58 instead of 38.)
    a.whole = (long long)q.c.P * q.c.W <= kWholeTokens;
    // 8, 16 or 32 rows a block: what the longest request needs, or (when longer
    // ones go elsewhere or take several blocks) what one row of every head needs
    const long long need = (long long)q.c.max_rows * a.group;
    const int rows = need <= 32 ? (int)need : a.group;
    if (q.c.D == 128)
        return rows <= 8 ? launch_rows<128, 1>(a, q.ws, sms, early, st)
               : rows <= 16 ? launch_rows<128, 2>(a, q.ws, sms, early, st)
                            : launch_rows<128, 4>(a, q.ws, sms, early, st);
    return rows <= 8 ? launch_rows<64, 1>(a, q.ws, sms, early, st)
           : rows <= 16 ? launch_rows<64, 2>(a, q.ws, sms, early, st)
                        : launch_rows<64, 4>(a, q.ws, sms, early, st);
}

}  // namespace cache
}  // namespace pmqa
