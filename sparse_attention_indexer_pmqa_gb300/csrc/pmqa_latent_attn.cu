// pmqa_latent_attn.cu -- attention of every row to all the tokens that it sees of
// the latent cache, and its C ABI (pmqa_latent_attention).
//
//   out[r][h] = sum_t softmax_t(sm_scale * q_h . k_t) * v_t,   v_t = k_t[0..511]
//
// Rows of one request are packed as (query token, head), up to N = 16, 32 or 64 to
// a block. A CTA walks the token tiles (128 tokens) of its blocks:
//   * one warp walks the tiles ahead of the others, looks their tokens up in the block
//     table and says what each tile is (Tile, Piece);
//   * four warps copy the latent rows (576 bytes) by cp.async straight into the operand
//     layout (pmqa_latent.cuh);
//   * one thread issues S^T = K Q^T (kind::f8f6f4, M = 128 tokens, N packed rows,
//     K = 576) into TMEM;
//   * the softmax threads, one per token and 16 or 32 packed rows, form p = 2^(x - m)
//     with an m for each row that moves when a weight passes 2^8, or when the row's sum (looked
//     at before tiles 2, 4, 8, ... for those up to the next of them, and where an m moves) is too
//     small for the terms' steps, and write p as two 8-bit terms, p_hi = e4m3(p) and p_lo, the
//     remainder;
//   * the thread issues O^T += V^T P^T (M = 128 value columns, four blocks, K = 128
//     tokens) from the SAME tile as an MN-major operand. With N = 64 both terms add
//     into one accumulator (576 + 2 * 512 fp8 multiplications a row and token; p_lo is
//     e5m2); with fewer rows p_lo is e4m3 times 16 in N more columns, since there the
//     cost is the read of V.
// The flattened sequence of (block, tile) is split evenly over the CTAs; a block
// that is cut leaves its parts (O, m, l) in the workspace and a second kernel joins
// them. (More packed rows: pmqa_latent_wide.cu.)
//
// A NaN in a token's row makes all its scores NaN. Where some rows do not see the
// token, its thread sets the row's values to zero before they are multiplied by
// the weights (0 for those rows, and for the others a NaN in the sum l, which makes
// all of their output NaN).
#include <algorithm>
#include <cmath>

#include "pmqa_latent_attn.cuh"

namespace pmqa {
namespace latent {

constexpr int kTile = 128;      // tokens per tile

// ------------------------------------------------------------- kernel

template <int N>
struct Cfg {
    static constexpr int kGroups = N == 16 ? 1 : 2;       // softmax warpgroups
    static constexpr int kRowsG = N / kGroups;            // packed rows of each
    static constexpr int kStages = N == 16 ? 3 : 2;       // value ring
    // N = 64: two idle warps complete the products' warpgroup, so that registers can
    // move to the softmax (2 x 192 + 64 + 64 = 4 x 128). Spilled registers cost more than
    // their instructions: the L1 cache beside so much shared memory holds 28 KB, and rows
    // pass through it (80 registers, 16 rows a thread: 434 us against 288).
    static constexpr bool kSplit = N == 64;
    static constexpr int kTile = latent::kTile, kPieces = 8;
    static constexpr int kThreads = 128 + 128 * kGroups + (kSplit ? 128 : 64);
    static constexpr int kAhead = N == 16 ? 1 : 2;        // tiles that the planner is ahead of the producers
    static constexpr int kTiles = kStages + kAhead;       // tiles that are described at a time
    static constexpr int kMmaWarp = 4 + 4 * kGroups, kPlanWarp = kMmaWarp + 1;
    static constexpr int kTerms = N == 64 ? 1 : 2;        // accumulators of a value block
    static constexpr int kOCols = kTerms * N;             // its output columns
    static constexpr float kAim = 1.0f;                   // a weight that moves m up (verify of 64 rows 185 us, at 2 188)
    static constexpr float kLo = N == 64 ? 1.0f : 16.0f;  // p_lo holds kLo (p - p_hi)
    // P: a row of 64 bytes per token, two terms of N rows. N = 64: a buffer of 128 rows for
    // each term; N = 16: both stages share a row, 32 bytes each.
    static constexpr uint32_t kPTerm = 128u * 64u;
    static constexpr uint32_t kPStage = N == 64 ? 2 * kPTerm : N == 32 ? kPTerm : 32u;
    static constexpr uint32_t kPBytes = N == 16 ? kPTerm : 2 * kPStage;
    static constexpr uint32_t kColS = 0;                  // 2 x N score columns
    static constexpr uint32_t kColO = 128;                // 4 x kOCols output columns
    static constexpr uint32_t kTmem = N == 64 ? 512 : N == 32 ? 512 : 256;

    static constexpr uint32_t kOffV = 0;
    static constexpr uint32_t kOffR = kOffV + kStages * kVStage;
    static constexpr uint32_t kOffQV = kOffR + 2 * kRStage;
    static constexpr uint32_t kOffQR = kOffQV + (N / 8) * kVGroup;
    static constexpr uint32_t kOffP = kOffQR + ((N / 8) * kRGroup + 1023) / 1024 * 1024;
    // 1 KB for each softmax warp's output; N = 16 has room for it only where P was
    static constexpr uint32_t kOffOut = N == 16 ? kOffP : kOffP + kPBytes;
    static constexpr uint32_t kOffRows = N == 16 ? kOffP + kPBytes : kOffOut + 4096 * kGroups;  // [kAhead][128]
    static constexpr uint32_t kOffInfo = kOffRows + kAhead * 512;       // [kTiles] Tile
    static constexpr uint32_t kOffPiece = kOffInfo + kTiles * 32;       // [kPieces] Piece
    static constexpr uint32_t kOffRange = kOffPiece + kPieces * 32;     // Range
    static constexpr uint32_t kOffLim = kOffRange + 128;                // [N] ints
    static constexpr uint32_t kOffM = kOffLim + N * 4;                  // [N] floats: -m       
    static constexpr uint32_t kOffAlpha = kOffM + N * 4;                // [N]
    static constexpr uint32_t kOffRed = kOffAlpha + N * 4;              // [4][N]
    static constexpr uint32_t kOffShort = kOffRed + 4 * N * 4;          // [kGroups]
    static constexpr uint32_t kOffBar = kOffShort + 8;
    static constexpr int kBInfo = 0;                        // [kTiles] tile described: the planner
    static constexpr int kBUsed = kBInfo + kTiles;          // [kTiles] its slot is free, its rows read: 4 producer warps
    static constexpr int kBReady = kBUsed + kTiles;        // [stages] rows landed: 128 cp.async arrivals
    static constexpr int kBVEmpty = kBReady + kStages;      // [stages][4] values of 32 tokens read: MMA commit
    static constexpr int kBREmpty = kBVEmpty + 4 * kStages;    // [2] rotary columns read: MMA commit
    static constexpr int kBSFull = kBREmpty + 2;            // [2] scores in TMEM: MMA commit
    static constexpr int kBSFree = kBSFull + 2;             // [2] scores read: softmax warps
    static constexpr int kBPFull = kBSFree + 2;             // [2] P written, O rescaled: softmax warps
    static constexpr int kBPEmpty = kBPFull + 2;            // [2] P read: MMA commit
    static constexpr int kBQEmpty = kBPEmpty + 2;           // queries read: MMA commit
    static constexpr int kBDrain = kBQEmpty + 1;
    static constexpr int kBars = kBDrain + 1;
    static constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
    static constexpr uint32_t kSmem = kOffMisc + 16;
    static_assert(kSmem <= 232448 && sizeof(Range) <= 128, "shared memory");
    static_assert(kOffP % 1024 == 0 && kOffBar % 8 == 0, "alignment");

    static constexpr uint32_t kIdescQK = idesc_e4m3_f32(128, N);
    // A and B MN-major (bits 15 and 16)
    static constexpr uint32_t kIdescPV = idesc_e4m3_f32(128, kOCols) | kIdescAMnMajor | (1u << 16);
    static constexpr uint32_t kIdescPVLo = kIdescPV | cache::kIdescBE5m2;  // N = 64
};

// Shared-memory matrix descriptor, MN-major with the 64-byte swizzle: one row of 64
// bytes per K index, 16-byte chunk c of row k at chunk c ^ ((k >> 1) & 3), groups of
// 8 rows 512 bytes apart; up to 64 elements along N.
__device__ __forceinline__ uint64_t sw64_mnmajor_desc(uint32_t smem_addr)
{
    return sw64_kmajor_desc(smem_addr, 512u);
}

// Sums or maxima of NR values over the warp's lanes: lane gets the result of value
// lane (NR = 32) or lane >> 1 (NR = 16).
template <bool MAX, int NR>
__device__ __forceinline__ float reduce_scatter(float (&v)[NR], int lane)
{
    auto op = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
    int bit = 16;
#pragma unroll
    for (int n = NR / 2; n > 0; n >>= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
            v[k] = op(keep, __shfl_xor_sync(kFull, send, bit));
        }
        bit >>= 1;
    }
    return NR == 32 ? v[0] : op(v[0], __shfl_xor_sync(kFull, v[0], 1));
}

template <int N>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1) latent_attn_kernel(const __grid_constant__ Args a)
{
    using K = Cfg<N>;
    constexpr int RG = K::kRowsG;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    const int g = blockIdx.x;

    if (tid == 0)
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
            for (int w = 0; w < 4; ++w)
                mbar_init(&bar[K::kBVEmpty + 4 * s + w], 1);
        }
        for (int s = 0; s < K::kTiles; ++s) {
            mbar_init(&bar[K::kBInfo + s], 1);
            mbar_init(&bar[K::kBUsed + s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar[K::kBREmpty + s], 1);
            mbar_init(&bar[K::kBSFull + s], 1);
            mbar_init(&bar[K::kBSFree + s], 4 * K::kGroups);
            mbar_init(&bar[K::kBPFull + s], 4 * K::kGroups);
            mbar_init(&bar[K::kBPEmpty + s], 1);
        }
        mbar_init(&bar[K::kBQEmpty], 1);
        mbar_init(&bar[K::kBDrain], 1);
        misc[1] = 0;
        mbar_init_fence();
    }
    if (warp == K::kMmaWarp)
        tmem_alloc(misc, K::kTmem);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];

    if (warp < 4) {
        // ------------------------------------------------------------ producer
        if constexpr (K::kSplit)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // Warp w copies the rows of tokens 32 w .. 32 w + 31, one row per instruction
        // (lane = 16-byte chunk).
        int vs = 0, seg = -1, e = 0;
        uint32_t vph = 0, eph = 0;
        for (int it = 0;; ++it) {
            const int rs = it & 1;
            const uint32_t rph = (uint32_t)(it >> 1) & 1u;
            if (!__all_sync(kFull, mbar_wait(&bar[K::kBInfo + e], eph, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
            const Tile *const tile = reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e;
            const uint32_t flags = tile->flags, srow = reinterpret_cast<const uint32_t *>(smem + K::kOffRows)[it % K::kAhead * 128 + tid];
            if (flags & kFirst) {
                // one query buffer: free once the last scores of the block before are done
                ++seg;
                if (!__all_sync(kFull, mbar_wait(&bar[K::kBQEmpty], ((uint32_t)seg & 1u) ^ 1u, abort_flag))) {
                    fail(a, abort_flag);
                    break;
                }
                const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
                const uint8_t *const src = a.q + piece->first * kDim;
                const int rows = piece->rows;
                for (int k = tid; k < N * kChunks; k += 128) {
                    const int r = k / kChunks, ch = k - r * kChunks;
                    const uint32_t dst = ch < 32 ? sbase + K::kOffQV + v_offset(r, ch)
                                                 : sbase + K::kOffQR + r_offset(r, ch - 32);
                    cp_async_16(dst, src + (r < rows ? r * kDim + ch * 16 : 0), r < rows ? 16u : 0u);
                }
            }
            // this warp's 32 tokens of the slot
            if (!__all_sync(kFull, mbar_wait(&bar[K::kBVEmpty + 4 * vs + warp], vph ^ 1u, abort_flag) &&
                                       mbar_wait(&bar[K::kBREmpty + rs], rph ^ 1u, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
            if (lane == 0)
                mbar_arrive(&bar[K::kBUsed + e]);
            const uint32_t vdst = sbase + K::kOffV + (uint32_t)vs * kVStage;
            const uint32_t rdst = sbase + K::kOffR + (uint32_t)rs * kRStage;
#pragma unroll 8
            for (int tt = 0; tt < 32; ++tt) {
                const uint32_t sr = __shfl_sync(kFull, srow, tt);
                const bool is = sr != paged::kNoRow;
                cp_async_16(vdst + v_offset(warp * 32 + tt, lane), a.kv + (is ? (unsigned long long)sr * kDim : 0ull) + 16 * lane,
                            is ? 16u : 0u);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tt = k * 8 + (lane >> 2), cc = lane & 3;
                const uint32_t sr = __shfl_sync(kFull, srow, tt);
                const bool is = sr != paged::kNoRow;
                cp_async_16(rdst + r_offset(warp * 32 + tt, cc),
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
        if constexpr (K::kSplit)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // Thread s of a group owns token s (TMEM lane s) and the group's RG packed
        // rows. Exits are uniform over the group: a failed wait clears `ok`, and the
        // group leaves together at its next barrier.
        const int wg = (warp - 4) >> 2, s = (tid - 128) & 127, w4 = s >> 5;
        const uint32_t lane_off = (uint32_t)(w4 * 32) << 16;
        const uint32_t barrier = 1u + wg;
        float *const mneg = reinterpret_cast<float *>(smem + K::kOffM) + wg * RG;
        float *const alpha = reinterpret_cast<float *>(smem + K::kOffAlpha) + wg * RG;
        float *const red = reinterpret_cast<float *>(smem + K::kOffRed) + wg * RG;  // [4][N]
        uint32_t *const any_short = reinterpret_cast<uint32_t *>(smem + K::kOffShort) + wg;
        int *const lims = reinterpret_cast<int *>(smem + K::kOffLim) + wg * RG;
        float l[RG];
        int seg = -1, vs = 0, e = 0, seen_by_all = 0;  // last slot that every row of the block sees
        int tiles = 0, look = 0;  // tiles of the piece so far, and at how many the sums are looked at next
        uint32_t eph = 0;
        bool ok = true;
        for (int it = 0;; ++it) {
            const int stage = it & 1;
            const uint32_t kph = (uint32_t)(it >> 1) & 1u;
            ok = ok && mbar_wait(&bar[K::kBInfo + e], eph, abort_flag);
            ok = __all_sync(kFull, ok);
            const Tile *const tile = reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e;
            const uint32_t flags = ok ? tile->flags : 0u;
            const bool first = flags & kFirst;
            if (first) {
                // every warp writes the same (no barrier: a failed wait must not part them)
                ++seg;
                tiles = 0;
                look = 2;
#pragma unroll
                for (int h = 0; h < RG; ++h)
                    l[h] = 0.0f;
                const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
                seen_by_all = piece->last;
                if (lane < RG) {
                    const int r = wg * RG + lane;
                    mneg[lane] = kUnseen;
                    // rows that do not exist see everything: no mask for their sake
                    lims[lane] = r < piece->rows ? seen_by_all + r / a.heads : 0x7FFFFFFF;
                }
                __syncwarp();
            }
            ok = ok && mbar_wait(&bar[K::kBSFull + stage], kph, abort_flag) &&
                 mbar_wait(&bar[K::kBPEmpty + stage], kph ^ 1u, abort_flag);
            ok = __all_sync(kFull, ok);
            const bool masked = (tile->have[0] & tile->have[1] & tile->have[2] & tile->have[3]) != kFull ||
                                tile->tok + kTile - 1 > seen_by_all;
            // the token's scores; those of rows that do not see it become what c_log2
            // turns into -inf
            uint32_t sr[RG];
            auto load_scores = [&]() {
                tmem_ld_cols<RG>(tmem + K::kColS + (uint32_t)(stage * N + wg * RG) + lane_off, sr);
                tmem_ld_wait();
                reg_fence_cols<RG>(sr);
                if (masked) {
                    const bool there = tile->have[w4] >> lane & 1u;
                    const int tok = tile->tok + s;
                    const uint32_t never = __float_as_uint(a.c_log2 > 0.0f ? -INFINITY : INFINITY);
                    bool nan = false;
#pragma unroll
                    for (int h = 0; h < RG; ++h) {
                        const float x = __uint_as_float(sr[h]);
                        nan |= x != x;
                        sr[h] = there && tok <= lims[h] ? sr[h] : never;
                    }
                    if (nan) {
                        // in the queries, or in the token's row: then out of its values
                        const uint32_t v = sbase + K::kOffV + (uint32_t)vs * kVStage;
#pragma unroll 1
                        for (int ch = 0; ch < 32; ++ch) {
                            const uint4 u = lds128(v + v_offset(s, ch));
                            sts128(v + v_offset(s, ch), without_nan(u.x), without_nan(u.y), without_nan(u.z), without_nan(u.w));
                        }
                    }
                }
            };
            // the weights, in fp32 and as f16 pairs; returns whether one passes 2^kTop
            float p[RG];
            uint32_t ph[RG / 2];
            auto weights = [&]() -> bool {
                uint32_t top = 0u;
#pragma unroll
                for (int h = 0; h < RG; h += 4) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(mneg + h);
                    ffma2_of(p[h], p[h + 1], sr[h], sr[h + 1], a.c_log2, m4.x, m4.y);
                    ffma2_of(p[h + 2], p[h + 3], sr[h + 2], sr[h + 3], a.c_log2, m4.z, m4.w);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[h + e] = ex2_approx(p[h + e]);
                    ph[h / 2] = cache::pack_f16x2(p[h], p[h + 1]);
                    ph[h / 2 + 1] = cache::pack_f16x2(p[h + 2], p[h + 3]);
                    asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(ph[h / 2]));
                    asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(ph[h / 2 + 1]));
                }
                // halves compare as whole numbers: none is negative (0x5C00: 2^8)
                return (top & 0xFFFFu) > 0x5C00u || (top >> 16) > 0x5C00u;
            };
            bool over = true;
            ++tiles;
            if (ok) {
                tc_fence_after_sync();
                load_scores();
                over = weights();
            }
            bool resc = false;
            over = named_bar_or(barrier, 128, over);
            const bool due = tiles == look;
            if (over || due) {
                // the rows' sums; most often that is all there is to a look
                if (ok && tiles > 1) {
                    float v[RG];
#pragma unroll
                    for (int h = 0; h < RG; ++h)
                        v[h] = l[h];
                    red[w4 * N + (RG == 32 ? lane : lane >> 1)] = reduce_scatter<false, RG>(v, lane);
                }
                if (!named_bar_and(barrier, 128, ok)) {
                    fail(a, abort_flag);
                    break;
                }
                if (due)
                    look = 2 * tiles;
                const float need = kEnough * kTile * (float)(look - 1);
                float L = 0.0f;
                if (w4 == 0 && lane < RG) {
                    if (tiles > 1)
                        L = (red[lane] + red[N + lane]) + (red[2 * N + lane] + red[3 * N + lane]);
                    const bool is_short = __any_sync(RG == 32 ? kFull : 0xFFFFu, L < need);
                    if (lane == 0)
                        *any_short = is_short;
                }
                named_bar_sync(barrier, 128);
                if (over || *any_short) {
                    load_scores();
                    float v[RG];
#pragma unroll
                    for (int h = 0; h < RG; ++h)
                        v[h] = __uint_as_float(sr[h]) * a.c_log2;
                    red[w4 * N + (RG == 32 ? lane : lane >> 1)] = reduce_scatter<true, RG>(v, lane);
                    named_bar_sync(barrier, 128);
                    if (w4 == 0 && lane < RG) {
                        const float x = fmaxf(fmaxf(red[lane], red[N + lane]), fmaxf(red[2 * N + lane], red[3 * N + lane]));
                        const float m = mneg[lane];
                        bool is_short;
                        const float to = moved_to(K::kAim, m, x, L, need, is_short);
                        alpha[lane] = ex2_approx(to - m);  // 0 where no score was seen before
                        mneg[lane] = to;
                        is_short = __any_sync(RG == 32 ? kFull : 0xFFFFu, is_short);
                        if (lane == 0)
                            *any_short = is_short;
                    }
                    named_bar_sync(barrier, 128);
                    if (*any_short)
                        look = tiles + 1;
#pragma unroll
                    for (int h = 0; h < RG; ++h) {
                        const float f = alpha[h];
                        resc |= f != 1.0f;
                        l[h] = finite(l[h]) * f;
                    }
                    if (resc)
                        weights();
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[K::kBSFree + stage]);
            // their sum and their two terms
            uint32_t hi[RG / 4], lo[RG / 4];
#pragma unroll
            for (int h = 0; h < RG; h += 4) {
                fadd2(l[h], l[h + 1], p[h], p[h + 1]);
                fadd2(l[h + 2], l[h + 3], p[h + 2], p[h + 3]);
                uint32_t h0, l0, h1, l1;
                split2<N == 64>(ph[h / 2], h0, l0);
                split2<N == 64>(ph[h / 2 + 1], h1, l1);
                hi[h / 4] = h0 | h1 << 16;
                lo[h / 4] = l0 | l1 << 16;
            }
            {
                // token s: one row of 64 bytes, 64-byte swizzle
                const uint32_t pb = sbase + K::kOffP + (N == 16 ? 0u : (uint32_t)stage * K::kPStage) + (uint32_t)s * 64u;
                const uint32_t x = (uint32_t)(s >> 1) & 3u;
#pragma unroll
                for (int k = 0; k < RG / 16; ++k) {
                    const uint32_t ch = (uint32_t)(N == 64 ? 2 * wg + k : N == 32 ? wg : 2 * stage);
                    const uint32_t cl = N == 64 ? ch : N == 32 ? ch + 2 : ch + 1;
                    sts128(pb + ((ch ^ x) << 4), hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                    sts128(pb + (N == 64 ? K::kPTerm : 0u) + ((cl ^ x) << 4), lo[4 * k], lo[4 * k + 1], lo[4 * k + 2],
                           lo[4 * k + 3]);
                }
            }
            if (resc && !first) {
                // O holds the block's earlier tiles, up to it - 1
                ok = ok && mbar_wait(&bar[K::kBPEmpty + (stage ^ 1)], (uint32_t)((it - 1) >> 1) & 1u, abort_flag);
                ok = __all_sync(kFull, ok);
                if (ok) {
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int k = 0; k < 4 * K::kTerms; ++k) {
                        uint32_t o[RG];
                        const uint32_t ta = tmem + K::kColO + (uint32_t)((k & 3) * K::kOCols + (k >> 2) * N + RG * wg) + lane_off;
                        tmem_ld_cols<RG>(ta, o);
                        tmem_ld_wait();
                        reg_fence_cols<RG>(o);
#pragma unroll
                        for (int e = 0; e < RG; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[e]);
                        if constexpr (RG == 32)
                            tmem_st32(ta, o);
                        else
                            tmem_st16(ta, o);
                    }
                    tmem_st_wait();
                }
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[K::kBPFull + stage]);
            if (++vs == K::kStages)
                vs = 0;
            if (++e == K::kTiles) {
                e = 0;
                eph ^= 1u;
            }
            if (!(flags & kLast))
                continue;

            // ------------------------------------------------ end of a block
            ok = ok && mbar_wait(&bar[K::kBPEmpty + stage], kph, abort_flag);
            ok = __all_sync(kFull, ok);
            const float wl = reduce_scatter<false, RG>(l, lane);
            red[w4 * N + (RG == 32 ? lane : lane >> 1)] = wl;
            if (!named_bar_and(barrier, 128, ok)) {
                fail(a, abort_flag);
                break;
            }
            tc_fence_after_sync();
            const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
            const bool sole = piece->sole != 0;
            const int slot = piece->slot, rows = piece->rows - wg * RG;  // rows of this group
            const long long out_row = piece->first + wg * RG;
            const uint32_t turn = sbase + K::kOffOut + (uint32_t)(warp - 4) * 1024u;
            float *const pp = a.part + ((long long)slot * N + wg * RG) * kVDim;
            if (s < RG && s < rows) {
                const float L = (red[s] + red[N + s]) + (red[2 * N + s] + red[3 * N + s]);
                if (sole) {
                    if (too_far(mneg[s]))
                        atomicOr(a.c.status, (uint32_t)PMQA_DEV_SCORE_RANGE);
                    if (a.lse)
                        a.lse[out_row + s] = L == 0.0f ? -INFINITY : (log2f(L) - mneg[s]) * cache::kLn2;
                } else {
                    __stcg(a.ml + ((long long)slot * N + wg * RG + s) * 2, -mneg[s]);
                    __stcg(a.ml + ((long long)slot * N + wg * RG + s) * 2 + 1, finite(L));
                }
                alpha[s] = L == 0.0f ? 0.0f : a.kv_scale / L;
            }
            named_bar_sync(barrier, 128);
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                uint32_t o[RG], o2[RG];
                const uint32_t ta = tmem + K::kColO + (uint32_t)(k * K::kOCols + RG * wg) + lane_off;
                tmem_ld_cols<RG>(ta, o);
                if (K::kTerms > 1)
                    tmem_ld_cols<RG>(ta + N, o2);
                tmem_ld_wait();
                reg_fence_cols<RG>(o);
                if (K::kTerms > 1) {
                    reg_fence_cols<RG>(o2);
#pragma unroll
                    for (int h = 0; h < RG; ++h)
                        o[h] = __float_as_uint(__uint_as_float(o[h]) + __uint_as_float(o2[h]) * (1.0f / K::kLo));
                }
                // 32 columns of the warp, turned in its own kilobyte so that 16 bytes are
                // stored at a time (2-byte stores: 20 cycles each, 21000 a block)
                if (sole) {
#pragma unroll
                    for (int q = 0; q < RG; q += 16) {
#pragma unroll
                        for (int h = 0; h < 16; ++h) {
                            const float f = alpha[q + h], y = f == 0.0f ? 0.0f : __uint_as_float(o[q + h]) * f;
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + 64u * h + 2u * lane),
                                         "h"(__bfloat16_as_ushort(__float2bfloat16_rn(y))) : "memory");
                        }
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            const int r = j + (lane >> 2);
                            const uint4 v = lds128(turn + 64u * r + 16u * (lane & 3));
                            if (q + r < rows)
                                *reinterpret_cast<uint4 *>(a.out + (out_row + q + r) * kVDim + k * 128 + w4 * 32 + 8 * (lane & 3)) = v;
                        }
                        __syncwarp();
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < RG; q += 8) {
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(turn + 128u * h + 4u * lane), "r"(o[q + h]) : "memory");
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            const int r = j + (lane >> 3);
                            const uint4 v = lds128(turn + 128u * r + 16u * (lane & 7));
                            if (q + r < rows)
                                __stcg(reinterpret_cast<uint4 *>(pp + (q + r) * kVDim + k * 128 + w4 * 32 + 4 * (lane & 7)), v);
                        }
                        __syncwarp();
                    }
                }
            }
            tc_fence_before_sync();
            if (flags & kEnd)
                break;
            // mneg and alpha (and P, where N = 16) are written anew only after every thread read them
            named_bar_sync(barrier, 128);
        }
    } else {
        if constexpr (K::kSplit)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == K::kPlanWarp) {
            plan_tiles<K>(a, smem, bar, range, g, true, abort_flag);
        } else if (warp == K::kMmaWarp) {
        // ------------------------------------------------------------ products
        // Two streams, each issued as soon as its inputs are ready: the scores of tile nq and the output update of tile np. The
        // whole warp walks them, so that descriptors stay in uniform registers; one
        // elected lane issues. The update goes 32 tokens at a time over all value
        // columns, and each 32 tokens' values are free for the loads when it is done.
        const Tile *const tiles = reinterpret_cast<const Tile *>(smem + K::kOffInfo);
        int nq = 0, np = 0, idle = 0;
        bool more_q = true, more_p = true;
        int qv = 0, pv = 0, qe = 0, pe = 0;  // value slots and descriptions of tiles nq and np
        uint32_t qvph = 0, qeph = 0;
        uint64_t idle_since = 0;
        bool ok = true;
        const uint64_t kd = sw128_kmajor_desc_sbo(sbase + K::kOffV, kVGroup), qd = sw128_kmajor_desc_sbo(sbase + K::kOffQV, kVGroup);
        const uint64_t rd = sw64_kmajor_desc(sbase + K::kOffR, kRGroup), qrd = sw64_kmajor_desc(sbase + K::kOffQR, kRGroup);
        const uint64_t vd = sw128_mnmajor_desc(sbase + K::kOffV, 1024u, kVGroup), pd = sw64_mnmajor_desc(sbase + K::kOffP);
        while (more_p) {
            bool prog = false;
            if (np < nq) {
                const int sb = np & 1;
                if (__all_sync(kFull, mbar_test(&bar[K::kBPFull + sb], (uint32_t)(np >> 1) & 1u))) {
                    const uint32_t flags = tiles[pe].flags;
                    const bool first = flags & kFirst;
                    tc_fence_after_sync();
                    const uint64_t av = vd + (((uint32_t)pv * kVStage) >> 4), bv = pd + (((uint32_t)sb * K::kPStage) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
                            for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                                for (int term = 0; term < (N == 64 ? 2 : 1); ++term)
                                    umma_e4m3(tmem + K::kColO + (uint32_t)(kb * K::kOCols),
                                              av + (((uint32_t)kb * 1024u + (uint32_t)ks * 4u * kVGroup) >> 4),
                                              bv + (((uint32_t)term * K::kPTerm + (uint32_t)ks * 2048u) >> 4),
                                              term ? K::kIdescPVLo : K::kIdescPV, (first && ks == 0 && term == 0) ? 0u : 1u);
                            umma_commit(&bar[K::kBVEmpty + 4 * pv + ks]);
                        }
                        umma_commit(&bar[K::kBPEmpty + sb]);
                    }
                    __syncwarp();
                    if (++pv == K::kStages)
                        pv = 0;
                    if (++pe == K::kTiles)
                        pe = 0;
                    ++np;
                    more_p = !(flags & kEnd);
                    prog = true;
                }
            }
            if (more_q) {
                const int sb = nq & 1;
                const uint32_t ph = (uint32_t)(nq >> 1) & 1u;
                if (__all_sync(kFull, mbar_test(&bar[K::kBReady + qv], qvph) && mbar_test(&bar[K::kBInfo + qe], qeph) &&
                                             mbar_test(&bar[K::kBSFree + sb], ph ^ 1u))) {
                    fence_proxy_async_smem();  // cp.async writes -> tensor-core reads
                    tc_fence_after_sync();
                    const uint32_t flags = tiles[qe].flags;
                    ++nq;
                    more_q = !(flags & kEnd);
                    const uint64_t av = kd + (((uint32_t)qv * kVStage) >> 4), ar = rd + (((uint32_t)sb * kRStage) >> 4);
                    const uint32_t dS = tmem + K::kColS + (uint32_t)(sb * N);
                    if (elect_one()) {
#pragma unroll
                        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) {
                                const uint32_t k = (uint32_t)kb * 1024u + (uint32_t)ks * 32u;
                                umma_e4m3(dS, av + (k >> 4), qd + (k >> 4), K::kIdescQK, (kb | ks) != 0 ? 1u : 0u);
                            }
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
                            umma_e4m3(dS, ar + 2u * ks, qrd + 2u * ks, K::kIdescQK, 1u);
                        umma_commit(&bar[K::kBSFull + sb]);
                        umma_commit(&bar[K::kBREmpty + sb]);
                        if (flags & kLast)
                            umma_commit(&bar[K::kBQEmpty]);
                    }
                    __syncwarp();
                    if (++qv == K::kStages) {
                        qv = 0;
                        qvph ^= 1u;
                    }
                    if (++qe == K::kTiles) {
                        qe = 0;
                        qeph ^= 1u;
                    }
                    prog = true;
                }
            }
            if (prog) {
                idle = 0;
                idle_since = 0;
                continue;
            }
            // nothing ready: sleep on what comes next for a moment, so that the polls
            // take no issue slots from the softmax; every 64 times the abort flag and
            // the clock
            if (np < nq)
                mbar_try_wait_sleep(&bar[K::kBPFull + (np & 1)], (uint32_t)(np >> 1) & 1u, 64u);
            else
                mbar_try_wait_sleep(&bar[K::kBReady + qv], qvph, 64u);
            if (++idle < 64)
                continue;
            idle = 0;
            const uint64_t now = __shfl_sync(kFull, global_timer_ns(), 0);
            if (idle_since == 0) {
                idle_since = now;
            } else if (__any_sync(kFull, *abort_flag != 0) || now - idle_since > kWaitLimitNs) {
                ok = false;
                break;
            }
        }
        if (!ok)
            fail(a, abort_flag);
        if (elect_one()) {
            umma_commit(&bar[K::kBDrain]);
            if (!mbar_wait(&bar[K::kBDrain], 0u, nullptr))
                atomicOr(a.c.status, (uint32_t)PMQA_DEV_TIMEOUT);
        }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == K::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, K::kTmem);
    }
}

// The parts of every unit that was cut, joined: block (g, y) takes packed row y of the unit
// that range g begins and later ranges go on with; a thread four columns. Bound by the
// latency of a chain of loads (what there is, the parts), about 5 us behind 32 contexts: each
// step rescales what the steps before gave, so that maxima and values are loaded
// together (looking the request up and reading the maxima first: batch decode 6 us more by graph,
// verify 2). Two or four rows to a block, or a warp a row: equal.
__global__ void __launch_bounds__(128) latent_join_kernel(const __grid_constant__ Args a)
{
    griddep_wait();
    const int g = blockIdx.x, at = threadIdx.x, row = blockIdx.y;
    const int4 m = __ldcg(a.meta + g);
    if (row >= m.y)
        return;
    constexpr int U = 4;  // parts of a step
    float M = -INFINITY, L = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int k0 = 0; k0 < m.z; k0 += U) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            ml[k] = make_float2(-INFINITY, 0.0f);
            o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k0 + k < m.z) {
                const long long slot = (long long)(2 * (g + k0 + k) + (k0 + k == 0 ? 1 : 0)) * a.N + row;
                ml[k] = __ldcg(reinterpret_cast<const float2 *>(a.ml + slot * 2));
                o[k] = __ldcg(reinterpret_cast<const float4 *>(a.part + slot * kVDim) + at);
            }
        }
        const float top = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x))), old = ex2_approx(M - top);
        M = top;
        L *= old;
        acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const float w = ex2_approx(ml[k].x - top);
            L += w * ml[k].y;
            acc.x += w * o[k].x;
            acc.y += w * o[k].y;
            acc.z += w * o[k].z;
            acc.w += w * o[k].w;
        }
    }
    const float f = L == 0.0f ? 0.0f : a.kv_scale / L;
    const float y[4] = {acc.x, acc.y, acc.z, acc.w};
    uint32_t b[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        b[k] = __bfloat16_as_ushort(__float2bfloat16_rn(f == 0.0f ? 0.0f : y[2 * k] * f)) |
               (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f == 0.0f ? 0.0f : y[2 * k + 1] * f)) << 16;
    *reinterpret_cast<uint2 *>(a.out + ((long long)m.x + row) * kVDim + 4 * at) = make_uint2(b[0], b[1]);
    if (at == 0 && too_far(-M))
        atomicOr(a.c.status, (uint32_t)PMQA_DEV_SCORE_RANGE);
    if (a.lse && at == 0)
        a.lse[m.x + row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * cache::kLn2;
}

template <int N>
cudaError_t launch(Args &a, int sms, cudaStream_t st)
{
    a.tile = kTile;
    a.N = N;
    a.pad = 2;
    a.least = 1;  // 500 tokens of one row by graph: 1 us less than with 2
    a.toks = 1;
    while (2 * a.toks * a.heads <= N)
        a.toks *= 2;
    a.ranges = std::max(1, std::min(sms, kMaxCtas));
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cache::allow_smem(latent_attn_kernel<N>, (int)Cfg<N>::kSmem, done);
    if (e != cudaSuccess)
        return e;
    latent_attn_kernel<N><<<(unsigned)a.ranges, Cfg<N>::kThreads, Cfg<N>::kSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace latent
}  // namespace pmqa

using namespace pmqa;
using namespace pmqa::latent;

extern "C" size_t pmqa_latent_workspace_bytes(void) { return kWorkspace; }

extern "C" int pmqa_latent_attention(const pmqa_paged_rows *p, const void *q, const void *kv_cache, int32_t heads,
                                     float q_scale, float kv_scale, float sm_scale, void *out, float *lse, void *ws,
                                     size_t ws_bytes, pmqa_stream_t stream)
{
    int rc = paged::check_rows(p, true, ws, ws_bytes, kWorkspace);
    if (rc != PMQA_OK)
        return rc;
    const double factor = (double)sm_scale * (double)q_scale * (double)kv_scale * 1.4426950408889634;
    if (heads < 1 || !std::isfinite(kv_scale) || !std::isfinite(factor))
        return PMQA_ERR_INVALID_ARG;
    if (std::fabs(factor) > kMaxFactor)
        return PMQA_ERR_UNSUPPORTED;
    if (heads > kMaxHeads || (long long)p->rows * heads > 0x7FFFFFFFll)
        return PMQA_ERR_UNSUPPORTED;
    if (p->bs == 0 || p->rows == 0)
        return PMQA_OK;
    if (cache::missing(q, 16) || cache::missing(kv_cache, 16) || cache::missing(out, 16) || !cache::aligned(lse, 4))
        return PMQA_ERR_INVALID_ARG;
    int sms = 0;
    if ((rc = cache::sm_count(&sms)) != PMQA_OK)
        return rc;
    Args a{};
    a.c = paged::view(p, ws);
    a.q = static_cast<const uint8_t *>(q);
    a.kv = static_cast<const uint8_t *>(kv_cache);
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    // 0: all scores alike; the kernel's masks need a factor that an infinity keeps
    a.c_log2 = std::fabs(factor) < 1e-37 ? 1e-37f : (float)factor;
    a.kv_scale = kv_scale;
    a.heads = heads;
    a.whole = (long long)p->block_size * p->max_blocks_per_seq <= kWhole ? 1 : 0;
    uint8_t *const wsb = static_cast<uint8_t *>(ws);
    a.meta = reinterpret_cast<int4 *>(wsb + kWsMeta);
    a.ml = reinterpret_cast<float *>(wsb + kWsMl);
    a.part = reinterpret_cast<float *>(wsb + kWsPart);
    // packed rows of a block: as many as a request can have, up to 64
    const long long most = std::min<long long>(p->max_rows, p->rows) * heads;
    const cudaStream_t st = cache::cuda(stream);
    cudaError_t e = most <= 16   ? launch<16>(a, sms, st)
                    : most <= 32 ? launch<32>(a, sms, st)
                    : most <= 64 ? launch<64>(a, sms, st)
                                 : launch_wide(a, sms, st);
    if (e == cudaSuccess && !a.whole)
        e = cache::launch_early(latent_join_kernel, dim3((unsigned)a.ranges, (unsigned)a.N), 128, 0, true, st, a);
    return cache::code_of(e);
}
