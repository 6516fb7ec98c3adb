// pmqa_latent_wide.cu -- attention to all latent tokens for requests with more than
// 64 packed rows (query tokens x heads): many heads, prompts.
//
// 128 packed rows to a block, tokens in tiles of 64. Two CTAs take a block, each one
// half of the value columns (a block's output is 128 x 512 fp32, all of one SM's
// tensor memory):
//   S = Q K^T    kind::f8f6f4, M = 128 rows, N = 64 tokens, Q's 512 latent values in tensor
//                memory (its 64 rotary ones in shared memory: there are no columns left)
//   p = 2^(x - m), a row to a thread; two fp8 terms, to tensor memory
//   O += P V     M = 128 rows, N = 256 value columns, both terms into one accumulator
// Neither these nor P pass through shared memory, whose 128 bytes a cycle bound the
// narrow kernel: a tile of 64 tokens costs 36 KB written, 36 read for the scores and
// 2 x 16 for the output (832 cycles) against 1088 cycles of products. The price is that
// both CTAs form the scores: 576 + 576 + 2 * 512 fp8 multiplications a row and token.
// Roles of the 16 warps: 0-3 copy rows (five slots of 64), 4-11 softmax and output, 12
// and 14 issue the products, 13 looks tokens up. S has one buffer (the scores of the next tile
// are formed while the softmax works on registers), P two (with one, each output update
// waited for the one before through four warps: 1830 cycles a tile).
#include <algorithm>

#include "pmqa_latent_attn.cuh"

namespace pmqa {
namespace latent {

// The block of the scores' products behind which the output update may be issued: its
// warp wakes and issues in 200 cycles, about the time until the scores are done (by graph batch
// decode 246 us after block 2, 239 after 3, prompt chunks 1943 and 1888).
constexpr int kTurnAt = 3;

struct Wide {
    static constexpr int kTile = 64;                      // tokens per tile
    static constexpr int kStages = 5;                     // slots of a tile's rows
    static constexpr int kAhead = 2;                      // tiles that the planner is ahead of the producers
    // A tile's description is read by both softmax groups, but its output waits for the one that
    // works on it: the other has read it when the next tile's output, which is its own, is done.
    static constexpr int kSpare = 1;
    static constexpr int kTiles = kStages + kAhead + kSpare, kPieces = 10;
    // The output of tile t waits for the scores of t + 2. Those of t + 6 need the slot of
    // tile t + 1 and so this wait's end: with four barriers no phase is passed over (two
    // could be, by the scores of t + 4: they need the slot of t - 1 alone).
    static constexpr int kTurns = 4;
    // A softmax group waits for the output of the tile two before its own, and where m moved, and
    // at a block's end, for that of the tile it does not work on. Four barriers: each such wait begins
    // when the phase before its own, four tiles back, is over. With two, that rested on one output's
    // end being reported before the next one's.
    static constexpr int kOuts = 4;
    static constexpr float kAim = 0.0f;  // a weight that moves m up (at 1 prompt chunks 1935 us, at 0 1907)
    static constexpr int kRows = 128, kThreads = 512;
    static constexpr int kMmaWarp = 12, kPlanWarp = 13, kOutWarp = 14;
    static constexpr uint32_t kVBytes = kTile / 8 * kVGroup, kRBytes = kTile / 8 * kRGroup;
    static constexpr uint32_t kColO = 0, kColQ = 256, kColP = 384, kColS = 448;  // tensor memory, P twice 32

    static constexpr uint32_t kOffV = 0;
    static constexpr uint32_t kOffR = kOffV + kStages * kVBytes;
    static constexpr uint32_t kOffQR = kOffR + kStages * kRBytes;       // the queries' rotary part
    static constexpr uint32_t kOffRows = kOffQR + kRows / 8 * kRGroup;  // [kAhead][64]
    static constexpr uint32_t kOffInfo = kOffRows + kAhead * kTile * 4; // [kTiles] Tile
    static constexpr uint32_t kOffPiece = kOffInfo + kTiles * 32;       // [kPieces] Piece
    static constexpr uint32_t kOffRange = kOffPiece + kPieces * 32;     // Range
    static constexpr uint32_t kOffRed = kOffRange + 128;                // [2][128]
    static constexpr uint32_t kOffM = kOffRed + 2 * kRows * 4;          // [128]: -m
    static constexpr uint32_t kOffLeast = kOffM + kRows * 4;            // [128]: the least -m of the block so far
    static constexpr uint32_t kOffBar = kOffLeast + kRows * 4;
    static constexpr int kBInfo = 0;                    // [kTiles] tile described: the planner
    static constexpr int kBUsed = kBInfo + kTiles;      // [kTiles] its slot is free, its rows read: 4 producer warps
    static constexpr int kBReady = kBUsed + kTiles;     // [stages] rows landed: 128 cp.async arrivals
    static constexpr int kBVEmpty = kBReady + kStages;  // [stages] rows read by both products: MMA commit
    // (pairs by the tile's parity: a softmax group waits on every second tile alone)
    static constexpr int kBSFull = kBVEmpty + kStages;  // [2] scores in tensor memory: MMA commit
    static constexpr int kBSFree = kBSFull + 2;         // scores read: 4 softmax warps
    static constexpr int kBPFull = kBSFree + 1;         // [2] P written, O rescaled: 4 softmax warps
    static constexpr int kBPEmpty = kBPFull + 2;        // [kOuts] P read: MMA commit
    static constexpr int kBM = kBPEmpty + kOuts;        // [2] m published: 4 softmax warps
    static constexpr int kBQFull = kBM + 2;             // a block's queries in tensor memory: 8 softmax warps
    static constexpr int kBTurn = kBQFull + 1;          // [kTurns] scores issued: the scores' warp
    static constexpr int kBDrain = kBTurn + kTurns;
    static constexpr int kBars = kBDrain + 2;           // both product warps
    static constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
    static constexpr uint32_t kSmem = kOffMisc + 16;
    static_assert(kSmem <= 232448 && kOffBar % 8 == 0 && kOffQR % 1024 == 0 && sizeof(Range) <= 128, "shared memory");

    static constexpr uint32_t kIdescQK = idesc_e4m3_f32(kRows, kTile);
    static constexpr uint32_t kIdescPV = idesc_e4m3_f32(kRows, 256) | (1u << 16);  // B MN-major
    static constexpr uint32_t kIdescPVLo = kIdescPV | cache::kIdescAE5m2;
};

// D[tmem] (+)= A[tmem] * B[smem]^T, 8-bit inputs, fp32 accumulation, one CTA.
__device__ __forceinline__ void umma_f8_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two 16-byte neighbours u, v of this lane's row (row `lane` from p on, `stride`
// elements apart) to memory, 32 bytes of a row at a time: neighbouring lanes trade, so
// that each store of the pair goes to one row.
template <typename T>
__device__ __forceinline__ void store_pair(T *p, int stride, int rows, const uint4 &u, const uint4 &v)
{
    const int lane = threadIdx.x & 31, odd = lane & 1;
    const uint4 send = odd ? u : v;
    const uint4 got = make_uint4(__shfl_xor_sync(kFull, send.x, 1), __shfl_xor_sync(kFull, send.y, 1),
                                 __shfl_xor_sync(kFull, send.z, 1), __shfl_xor_sync(kFull, send.w, 1));
    T *const at = p + (long long)(lane & ~1) * stride + odd * (int)(16 / sizeof(T));
    if ((lane & ~1) < rows)
        __stcg(reinterpret_cast<uint4 *>(at), odd ? got : u);
    if ((lane | 1) < rows)
        __stcg(reinterpret_cast<uint4 *>(at + stride), odd ? v : got);
}

__global__ void __launch_bounds__(Wide::kThreads, 1) latent_wide_kernel(const __grid_constant__ Args a)
{
    using K = Wide;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    const int g = blockIdx.x / 2, vh = blockIdx.x & 1;

    if (vh == 0 && tid == 0)
        a.meta[g] = make_int4(0, 0, 0, 0);
    Range *const range = reinterpret_cast<Range *>(smem + K::kOffRange);
    find_range<K::kThreads>(a, g, reinterpret_cast<long long *>(smem), range);
    griddep_launch_dependents();
    if (!range->any)
        return;  // the same for the whole CTA
    if (sbase & 1023u) {
        if (tid == 0)
            atomicOr(a.c.status, (uint32_t)PMQA_DEV_INTERNAL);
        return;
    }
    uint64_t *const bar = reinterpret_cast<uint64_t *>(smem + K::kOffBar);
    uint32_t *const misc = reinterpret_cast<uint32_t *>(smem + K::kOffMisc);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    if (tid == 0) {
        for (int s = 0; s < K::kStages; ++s) {
            mbar_init(&bar[K::kBReady + s], 128);
            mbar_init(&bar[K::kBVEmpty + s], 1);
        }
        for (int s = 0; s < K::kTiles; ++s) {
            mbar_init(&bar[K::kBInfo + s], 1);
            mbar_init(&bar[K::kBUsed + s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[K::kBSFull + s], 1);
            mbar_init(&bar[K::kBPFull + s], 4);
            mbar_init(&bar[K::kBM + s], 4);
        }
        for (int s = 0; s < K::kOuts; ++s)
            mbar_init(&bar[K::kBPEmpty + s], 1);
        for (int s = 0; s < K::kTurns; ++s)
            mbar_init(&bar[K::kBTurn + s], 1);
        mbar_init(&bar[K::kBSFree], 4);
        mbar_init(&bar[K::kBQFull], 8);
        mbar_init(&bar[K::kBDrain], 1);
        mbar_init(&bar[K::kBDrain + 1], 1);
        misc[1] = 0;
        mbar_init_fence();
    }
    if (warp == K::kMmaWarp)
        tmem_alloc(misc, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];

    if (warp < 4) {
        // ------------------------------------------------------------ producer
        // Warp w copies the rows of tokens 16 w .. 16 w + 15, one row per instruction
        // (lane = 16-byte chunk).
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");  // 2 x 192 + 2 x 64 = 4 x 128
        int vs = 0, e = 0;
        uint32_t vph = 0, eph = 0;
        for (int it = 0;; ++it) {
            if (!__all_sync(kFull, wait_for(&bar[K::kBInfo + e], eph, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
            const uint32_t flags = (reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e)->flags;
            const uint32_t srow = reinterpret_cast<const uint32_t *>(
                smem + K::kOffRows)[it % K::kAhead * K::kTile + warp * 16 + (lane & 15)];
            if (!__all_sync(kFull, wait_for(&bar[K::kBVEmpty + vs], vph ^ 1u, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
            if (lane == 0)
                mbar_arrive(&bar[K::kBUsed + e]);
            const uint32_t vdst = sbase + K::kOffV + (uint32_t)vs * K::kVBytes;
            const uint32_t rdst = sbase + K::kOffR + (uint32_t)vs * K::kRBytes;
#pragma unroll 8
            for (int tt = 0; tt < 16; ++tt) {
                const uint32_t sr = __shfl_sync(kFull, srow, tt);
                const bool is = sr != paged::kNoRow;
                cp_async_16(vdst + v_offset(warp * 16 + tt, lane), a.kv + (is ? (unsigned long long)sr * kDim : 0ull) + 16 * lane,
                            is ? 16u : 0u);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int tt = k * 8 + (lane >> 2), cc = lane & 3;
                const uint32_t sr = __shfl_sync(kFull, srow, tt);
                const bool is = sr != paged::kNoRow;
                cp_async_16(rdst + r_offset(warp * 16 + tt, cc),
                            a.kv + (is ? (unsigned long long)sr * kDim : 0ull) + kVDim + 16 * cc, is ? 16u : 0u);
            }
            cp_async_arrive_noinc(&bar[K::kBReady + vs]);
            if (flags & kEnd)
                break;
            if (++vs == K::kStages) {
                vs = 0;
                vph ^= 1u;
            }
            if (++e == K::kTiles) {
                e = 0;
                eph ^= 1u;
            }
        }
        cp_async_wait_all();
    } else if (warp < K::kMmaWarp) {
        // ------------------------------------------------------------ softmax
        // The two groups take the tiles in turn, a row to a thread, so that one's waits
        // and conversions run beside the other's (both on every tile, half a row each:
        // 2400 cycles a tile, most of them waits). m is theirs in common: it goes from tile
        // to tile, published before a tile's weights are formed. A warp whose wait failed
        // takes part in one more barrier, at which all leave.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int wg = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
        float *const red = reinterpret_cast<float *>(smem + K::kOffRed);  // [2][128]
        float *const shared_m = reinterpret_cast<float *>(smem + K::kOffM);  // [128]: -m
        float *const least = reinterpret_cast<float *>(smem + K::kOffLeast);  // [128]
        // the output of tile t is done
        auto out_done = [&](int t) {
            static_assert(K::kOuts == 4, "a shift: tiles before the first have the phase before the first");
            return mbar_wait(&bar[K::kBPEmpty + (t & (K::kOuts - 1))], (uint32_t)(t >> 2) & 1u, abort_flag);
        };
        float l = 0.0f, mneg = kUnseen, need = 0.0f;
        int seg = -1, vs = 0, e = 0, lim = 0;
        uint32_t eph = 0;
        for (int it = 0;; ++it) {
            const uint32_t now = (uint32_t)it & 1u, was = now ^ 1u;  // parity of this tile and the one before,
            const uint32_t ph = (uint32_t)(it >> 1) & 1u, wph = (uint32_t)((it - 1) >> 1) & 1u;  // and their phases
            if (!__all_sync(kFull, mbar_wait(&bar[K::kBInfo + e], eph, abort_flag))) {
                fail(a, abort_flag);
                named_bar_and(1, 256, false);
                break;
            }
            const Tile *const tile = reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e;
            const uint32_t flags = tile->flags;
            const bool first = flags & kFirst;
            if (first) {
                // the row's queries, to tensor memory (the scores of the block before are done)
                ++seg;
                const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
                const bool is = row < piece->rows;
                const uint4 *const src = reinterpret_cast<const uint4 *>(a.q + (piece->first + (is ? row : 0)) * kDim);
                uint4 u[18];
#pragma unroll
                for (int k = 0; k < 18; ++k)
                    u[k] = is ? __ldg(src + (k < 16 ? 16 * wg + k : 32 + 2 * wg + k - 16)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tmem_st16(lanes + K::kColQ + 64u * wg + 16u * k, &u[4 * k].x);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    sts128(sbase + K::kOffQR + r_offset(row, 2 * wg + k), u[16 + k].x, u[16 + k].y, u[16 + k].z, u[16 + k].w);
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBQFull]);
                l = 0.0f;
                mneg = kUnseen;
                need = 0.0f;
                if (now == (uint32_t)wg)
                    least[row] = kUnseen;
                // rows that do not exist see everything: no mask for their sake
                lim = is ? piece->last + row / a.heads : 0x7FFFFFFF;
            }
            if (now == (uint32_t)wg) {
                // what does not wait for the scores comes before them: m as the tile before
                // left it, the tokens that the row sees
                if (!first && !__all_sync(kFull, mbar_wait(&bar[K::kBM + was], wph, abort_flag))) {
                    fail(a, abort_flag);
                    named_bar_and(1, 256, false);
                    break;
                }
                if (!first) {
                    const float m = shared_m[row];
                    if (m != mneg) {
                        l = finite(l) * ex2_approx(m - mneg);
                        mneg = m;
                    }
                }
                uint32_t sees[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int past = lim - tile->tok - 32 * half;
                    sees[half] = tile->have[half] & (past >= 31 ? kFull : past < 0 ? 0u : (2u << past) - 1u);
                }
                const bool whole = __all_sync(kFull, (sees[0] & sees[1]) == kFull);
                if (!__all_sync(kFull, mbar_wait(&bar[K::kBSFull + now], ph, abort_flag))) {
                    fail(a, abort_flag);
                    named_bar_and(1, 256, false);
                    break;
                }
                uint32_t sr[64];
                tc_fence_after_sync();
                tmem_ld32(lanes + K::kColS, sr);
                tmem_ld32(lanes + K::kColS + 32u, sr + 32);
                tmem_ld_wait();
                reg_fence16(sr);
                reg_fence16(sr + 16);
                reg_fence16(sr + 32);
                reg_fence16(sr + 48);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBSFree]);
                bool cleaned = false;
                if (!whole) {
                    const uint32_t never = __float_as_uint(a.c_log2 > 0.0f ? -INFINITY : INFINITY);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t nan = 0u;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float x = __uint_as_float(sr[32 * half + k]);
                            nan |= x != x ? 1u << k : 0u;
                            sr[32 * half + k] = sees[half] >> k & 1u ? sr[32 * half + k] : never;
                        }
                        nan = __reduce_or_sync(kFull, nan);
                        cleaned |= nan != 0u;
                        // in the queries, or in a token's row: then out of its values
                        for (; nan; nan &= nan - 1u) {
                            const uint32_t v = sbase + K::kOffV + (uint32_t)vs * K::kVBytes + v_offset(32 * half + __ffs(nan) - 1, lane);
                            const uint4 w = lds128(v);
                            sts128(v, without_nan(w.x), without_nan(w.y), without_nan(w.z), without_nan(w.w));
                        }
                    }
                }
                // the row's largest score here, and m (l and need are of this group's tiles)
                float x;
                {
                    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 64; k += 8)
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float y0 = __uint_as_float(sr[k + 2 * z]), y1 = __uint_as_float(sr[k + 2 * z + 1]);
                            t[z] = a.c_log2 > 0.0f ? fmaxf(t[z], fmaxf(y0, y1)) : fmaxf(t[z], fmaxf(-y0, -y1));
                        }
                    x = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * fabsf(a.c_log2);
                }
                float alpha = 1.0f;
                need += kEnough * K::kTile;
                if (x + mneg > kTop || l < need) {
                    bool is_short;
                    const float low = least[row], to = moved_to(K::kAim, mneg, x, l, need, is_short, low + kReach);
                    least[row] = fminf(low, to);
                    alpha = ex2_approx(to - mneg);  // 0 where no score was seen before
                    mneg = to;
                    l = finite(l) * alpha;
                }
                if (first || alpha != 1.0f)
                    shared_m[row] = mneg;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBM + now]);
                // the weights, their sum and their two terms
                uint32_t hi[16], lo[16];
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float p0, p1, p2, p3;
                    ffma2_of(p0, p1, sr[4 * k], sr[4 * k + 1], a.c_log2, mneg, mneg);
                    ffma2_of(p2, p3, sr[4 * k + 2], sr[4 * k + 3], a.c_log2, mneg, mneg);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                    p2 = ex2_approx(p2);
                    p3 = ex2_approx(p3);
                    fadd2(s0, s1, p0, p1);
                    fadd2(s0, s1, p2, p3);
                    uint32_t h0, h1, d0, d1;
                    split2<true>(cache::pack_f16x2(p0, p1), h0, d0);
                    split2<true>(cache::pack_f16x2(p2, p3), h1, d1);
                    hi[k] = h0 | h1 << 16;
                    lo[k] = d0 | d1 << 16;
                }
                l += s0 + s1;
                // this buffer of P is free
                if (!__all_sync(kFull, out_done(it - 2))) {
                    fail(a, abort_flag);
                    named_bar_and(1, 256, false);
                    break;
                }
                if (!first && __any_sync(kFull, alpha != 1.0f)) {
                    // O: the output of the tile before is done
                    if (!__all_sync(kFull, out_done(it - 1))) {
                        fail(a, abort_flag);
                        named_bar_and(1, 256, false);
                        break;
                    }
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[64];
                        const uint32_t ta = lanes + K::kColO + 64u * k;
                        tmem_ld32(ta, o);
                        tmem_ld32(ta + 32u, o + 32);
                        tmem_ld_wait();
                        reg_fence16(o);
                        reg_fence16(o + 16);
                        reg_fence16(o + 32);
                        reg_fence16(o + 48);
#pragma unroll
                        for (int z = 0; z < 64; ++z)
                            o[z] = __float_as_uint(__uint_as_float(o[z]) * alpha);
                        tmem_st32(ta, o);
                        tmem_st32(ta + 32u, o + 32);
                    }
                }
                tc_fence_after_sync();
                tmem_st16(lanes + K::kColP + 32u * now, hi);
                tmem_st16(lanes + K::kColP + 32u * now + 16u, lo);
                tmem_st_wait();
                if (cleaned)
                    fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBPFull + now]);
            }
            if (++vs == K::kStages)
                vs = 0;
            if (++e == K::kTiles) {
                e = 0;
                eph ^= 1u;
            }
            if (!(flags & kLast))
                continue;

            // ------------------------------------------------ end of a block
            // (the last two tiles': one of them is of the other group)
            if (!named_bar_and(1, 256, __all_sync(kFull, (it == 0 || out_done(it - 1)) && out_done(it)))) {
                fail(a, abort_flag);
                break;
            }
            tc_fence_after_sync();
            {
                const float m = shared_m[row];
                red[wg * K::kRows + row] = finite(l) * ex2_approx(m - mneg);
                mneg = m;
            }
            named_bar_sync(1, 256);
            const float L = red[row] + red[K::kRows + row];
            const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
            const bool sole = piece->sole != 0;
            const int rows = piece->rows - w4 * 32;  // from the warp's first on
            const long long at = (long long)piece->slot * K::kRows + row;
            if (wg == 0 && vh == 0 && lane < rows) {
                if (!sole) {
                    __stcg(a.ml + at * 2, -mneg);
                    __stcg(a.ml + at * 2 + 1, finite(L));
                } else {
                    if (too_far(mneg))
                        atomicOr(a.c.status, (uint32_t)PMQA_DEV_SCORE_RANGE);
                    if (a.lse)
                        a.lse[piece->first + row] = L == 0.0f ? -INFINITY : (log2f(L) - mneg) * cache::kLn2;
                }
            }
            const float f = L == 0.0f ? 0.0f : a.kv_scale / L;
            const int col = vh * 256 + wg * 128;
            uint16_t *const out = a.out + (piece->first + w4 * 32) * kVDim + col;
            float *const part = a.part + (at - lane) * kVDim + col;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                uint32_t o[32];
                tmem_ld32(lanes + K::kColO + 128u * wg + 32u * k, o);
                tmem_ld_wait();
                reg_fence_cols<32>(o);
                if (sole) {
#pragma unroll
                    for (int z = 0; z < 32; z += 16) {
                        uint32_t b[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) {
                            const float y0 = f == 0.0f ? 0.0f : __uint_as_float(o[z + 2 * y]) * f;
                            const float y1 = f == 0.0f ? 0.0f : __uint_as_float(o[z + 2 * y + 1]) * f;
                            b[y] = __bfloat16_as_ushort(__float2bfloat16_rn(y0)) |
                                   (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(y1)) << 16;
                        }
                        store_pair(out + 32 * k + z, kVDim, rows, make_uint4(b[0], b[1], b[2], b[3]),
                                   make_uint4(b[4], b[5], b[6], b[7]));
                    }
                } else {
#pragma unroll
                    for (int z = 0; z < 32; z += 8)
                        store_pair(part + 32 * k + z, kVDim, rows, make_uint4(o[z], o[z + 1], o[z + 2], o[z + 3]),
                                   make_uint4(o[z + 4], o[z + 5], o[z + 6], o[z + 7]));
                }
            }
            tc_fence_before_sync();
            if (flags & kEnd)
                break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == K::kPlanWarp) {
            plan_tiles<K>(a, smem, bar, range, g, vh == 0, abort_flag);
        } else if (warp == K::kMmaWarp || warp == K::kOutWarp) {
            // -------------------------------------------------------- products
            // One warp for the scores, one for the output updates: between two issues a
            // warp takes 500 to 650 cycles over its waits and its instructions' way past
            // the softmax's, and one warp's is the other's tensor time (one warp for both:
            // 1830 cycles a tile). One elected lane of the converged warp issues; the
            // scores' loop is rolled for the instruction caches' sake.
            const bool out = warp == K::kOutWarp;
            const Tile *const tiles = reinterpret_cast<const Tile *>(smem + K::kOffInfo);
            int seg = 0, vs = 0, e = 0;
            uint32_t vph = 0, eph = 0;
            bool ok = true;
            auto wait = [&](int barrier, uint32_t parity) {
                ok = ok && __all_sync(kFull, wait_for(&bar[barrier], parity, abort_flag));
                return ok;
            };
            const uint64_t kd = sw128_kmajor_desc_sbo(sbase + K::kOffV, kVGroup);
            const uint64_t vd = sw128_mnmajor_desc(sbase + K::kOffV + (uint32_t)vh * 2048u, 1024u, kVGroup);
            const uint64_t rd = sw64_kmajor_desc(sbase + K::kOffR, kRGroup), qrd = sw64_kmajor_desc(sbase + K::kOffQR, kRGroup);
            for (int it = 0;; ++it) {
                const uint32_t now = (uint32_t)it & 1u;
                if (!wait(K::kBInfo + e, eph))
                    break;
                const uint32_t flags = tiles[e].flags;
                if (!out) {
                    if (!wait(K::kBReady + vs, vph) || ((flags & kFirst) && !wait(K::kBQFull, (uint32_t)seg & 1u)) ||
                        !wait(K::kBSFree, now ^ 1u))
                        break;
                    if (flags & kFirst)
                        ++seg;
                    fence_proxy_async_smem();  // cp.async writes -> tensor-core reads
                    tc_fence_after_sync();
                    const uint64_t bk = kd + (((uint32_t)vs * K::kVBytes) >> 4), br = rd + (((uint32_t)vs * K::kRBytes) >> 4);
                    if (elect_one()) {
#pragma unroll 1
                        for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                umma_f8_ts(tmem + K::kColS, tmem + K::kColQ + 32u * kb + 8u * k, bk + 64u * kb + 2u * k, K::kIdescQK,
                                           (kb | k) ? 1u : 0u);
                            if (kb == kTurnAt)
                                mbar_arrive(&bar[K::kBTurn + ((uint32_t)it & (K::kTurns - 1u))]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            umma_e4m3(tmem + K::kColS, qrd + 2u * k, br + 2u * k, K::kIdescQK, 1u);
                        umma_commit(&bar[K::kBSFull + now]);
                    }
                } else {
                    // behind the scores of two tiles on, so that these are worked on while S
                    // waits to be read; a piece's last two tiles do not wait
                    if (!wait(K::kBPFull + now, (uint32_t)(it >> 1) & 1u) ||
                        ((flags & kSteady) && !wait(K::kBTurn + (((uint32_t)it + 2u) & (K::kTurns - 1u)), (((uint32_t)it + 2u) >> 2) & 1u)))
                        break;
                    fence_proxy_async_smem();  // cp.async writes -> tensor-core reads
                    tc_fence_after_sync();
                    const uint64_t bv = vd + (((uint32_t)vs * K::kVBytes) >> 4);
                    const uint32_t ap = tmem + K::kColP + 32u * now;
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int term = 0; term < 2; ++term)
                                umma_f8_ts(tmem + K::kColO, ap + 16u * term + 8u * ks, bv + (((uint32_t)ks * 4u * kVGroup) >> 4),
                                           term ? K::kIdescPVLo : K::kIdescPV, ((flags & kFirst) && ks == 0 && term == 0) ? 0u : 1u);
                        umma_commit(&bar[K::kBVEmpty + vs]);
                        umma_commit(&bar[K::kBPEmpty + ((uint32_t)it & (K::kOuts - 1u))]);
                    }
                }
                __syncwarp();
                if (flags & kEnd)
                    break;
                if (++vs == K::kStages) {
                    vs = 0;
                    vph ^= 1u;
                }
                if (++e == K::kTiles) {
                    e = 0;
                    eph ^= 1u;
                }
            }
            if (!ok)
                fail(a, abort_flag);
            if (elect_one()) {
                uint64_t *const drain = &bar[K::kBDrain + (out ? 1 : 0)];
                umma_commit(drain);
                if (!mbar_wait(drain, 0u, nullptr))
                    atomicOr(a.c.status, (uint32_t)PMQA_DEV_TIMEOUT);
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == K::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

cudaError_t launch_wide(Args &a, int sms, cudaStream_t st)
{
    a.tile = Wide::kTile;
    a.N = Wide::kRows;
    a.pad = 4;
    a.least = 4;
    a.toks = 1;
    while (2 * a.toks * a.heads <= Wide::kRows && 2 * a.toks <= Wide::kTile)
        a.toks *= 2;
    a.ranges = std::max(1, std::min(sms, kMaxCtas) / 2);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cache::allow_smem(latent_wide_kernel, (int)Wide::kSmem, done);
    if (e != cudaSuccess)
        return e;
    latent_wide_kernel<<<(unsigned)(a.ranges * 2), Wide::kThreads, Wide::kSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace latent
}  // namespace pmqa
