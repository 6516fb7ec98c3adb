// pmqa_latent_wide.cu -- attention to all latent tokens for requests with more than
// 64 packed rows (query tokens x heads): many heads, prompts.
//
// 128 packed rows to a block, tokens in tiles of 64. Two CTAs take a block, each one
// half of the value columns (a block's output is 128 x 512 fp32, all of one SM's
// tensor memory):
//   S = Q K^T    kind::f8f6f4, M = 128 rows, N = 64 tokens, Q (128 x 576) in tensor memory
//   p = 2^(x - m), one row to a thread pair; two fp8 terms, to tensor memory
//   O += P V     M = 128 rows, N = 256 value columns, both terms into one accumulator
// Neither Q nor P passes through shared memory, whose 128 bytes a cycle bound the
// narrow kernel: a tile of 64 tokens costs 36 KB written, 36 read for the scores and
// 2 x 16 for the output (832 cycles) against 1088 cycles of products. The price is that
// both CTAs form the scores: 576 + 576 + 2 * 512 fp8 multiplications a row and token.
// Roles of the 16 warps: 0-3 copy rows (six slots of 64), 4-11 softmax and output, 12
// issues the products, 13 looks tokens up. S and P have one buffer each: the scores of
// the next tile are formed while the softmax works on registers.
#include <algorithm>

#include "pmqa_latent_attn.cuh"

namespace pmqa {
namespace latent {

struct Wide {
    static constexpr int kTile = 64;                      // tokens per tile
    static constexpr int kStages = 6;                     // slots of a tile's rows
    static constexpr int kAhead = 2;                      // tiles that the planner is ahead of the producers
    static constexpr int kTiles = kStages + kAhead, kPieces = 16;
    static constexpr int kRows = 128, kThreads = 512;
    static constexpr int kMmaWarp = 12, kPlanWarp = 13;
    static constexpr uint32_t kVBytes = kTile / 8 * kVGroup, kRBytes = kTile / 8 * kRGroup;
    static constexpr uint32_t kColO = 0, kColQ = 256, kColP = 400, kColS = 448;  // tensor memory

    static constexpr uint32_t kOffV = 0;
    static constexpr uint32_t kOffR = kOffV + kStages * kVBytes;
    static constexpr uint32_t kOffOut = kOffR + kStages * kRBytes;      // 1 KB for each softmax warp's output
    static constexpr uint32_t kOffRows = kOffOut + 8 * 1024;            // [kAhead][64]
    static constexpr uint32_t kOffInfo = kOffRows + kAhead * kTile * 4; // [kTiles] Tile
    static constexpr uint32_t kOffPiece = kOffInfo + kTiles * 32;       // [kPieces] Piece
    static constexpr uint32_t kOffRange = kOffPiece + kPieces * 32;     // Range
    static constexpr uint32_t kOffRed = kOffRange + 128;                // [2][128]
    static constexpr uint32_t kOffBar = kOffRed + 2 * kRows * 4;
    static constexpr int kBInfo = 0;                    // [kTiles] tile described: the planner
    static constexpr int kBUsed = kBInfo + kTiles;      // [kTiles] its slot is free, its rows read: 4 producer warps
    static constexpr int kBReady = kBUsed + kTiles;     // [stages] rows landed: 128 cp.async arrivals
    static constexpr int kBVEmpty = kBReady + kStages;  // [stages] rows read by both products: MMA commit
    static constexpr int kBSFull = kBVEmpty + kStages;  // scores in tensor memory: MMA commit
    static constexpr int kBSFree = kBSFull + 1;         // scores read: 8 softmax warps
    static constexpr int kBPFull = kBSFree + 1;         // P written, O rescaled: 8 softmax warps
    static constexpr int kBPEmpty = kBPFull + 1;        // P read: MMA commit
    static constexpr int kBQFull = kBPEmpty + 1;        // a block's queries in tensor memory: 8 softmax warps
    static constexpr int kBDrain = kBQFull + 1;
    static constexpr int kBars = kBDrain + 1;
    static constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
    static constexpr uint32_t kSmem = kOffMisc + 16;
    static_assert(kSmem <= 232448 && kOffBar % 8 == 0 && sizeof(Range) <= 128, "shared memory");

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

// 8 consecutive TMEM columns of this thread's lane from registers.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
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
        mbar_init(&bar[K::kBSFull], 1);
        mbar_init(&bar[K::kBSFree], 8);
        mbar_init(&bar[K::kBPFull], 8);
        mbar_init(&bar[K::kBPEmpty], 1);
        mbar_init(&bar[K::kBQFull], 8);
        mbar_init(&bar[K::kBDrain], 1);
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
            if (!__all_sync(kFull, mbar_wait(&bar[K::kBInfo + e], eph, abort_flag))) {
                fail(a, abort_flag);
                break;
            }
            const uint32_t flags = (reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e)->flags;
            const uint32_t srow = reinterpret_cast<const uint32_t *>(
                smem + K::kOffRows)[it % K::kAhead * K::kTile + warp * 16 + (lane & 15)];
            if (!__all_sync(kFull, mbar_wait(&bar[K::kBVEmpty + vs], vph ^ 1u, abort_flag))) {
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
        // Thread (group wg, row): the row's scores of tokens 32 wg .. 32 wg + 31. Both
        // threads of a row hold the same m. Exits are uniform over both groups: a failed
        // wait clears `ok`, and they leave together at the next barrier.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int wg = (warp - 4) >> 2, w4 = warp & 3, row = w4 * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(w4 * 32) << 16);
        float *const red = reinterpret_cast<float *>(smem + K::kOffRed);  // [2][128]
        const uint32_t turn = sbase + K::kOffOut + (uint32_t)(warp - 4) * 1024u;
        float l0 = 0.0f, l1 = 0.0f, mneg = kUnseen;
        int seg = -1, vs = 0, e = 0, lim = 0;
        uint32_t eph = 0;
        bool ok = true;
        for (int it = 0;; ++it) {
            const uint32_t ph = (uint32_t)it & 1u;
            ok = ok && mbar_wait(&bar[K::kBInfo + e], eph, abort_flag);
            ok = __all_sync(kFull, ok);
            const Tile *const tile = reinterpret_cast<const Tile *>(smem + K::kOffInfo) + e;
            const uint32_t flags = ok ? tile->flags : 0u;
            const bool first = flags & kFirst;
            if (first) {
                // the row's queries, to tensor memory (the scores of the block before are done)
                ++seg;
                const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
                const bool is = row < piece->rows;
                const uint4 *const src = reinterpret_cast<const uint4 *>(a.q + (piece->first + (is ? row : 0)) * kDim) + 20 * wg;
                uint4 u[20];
#pragma unroll
                for (int k = 0; k < 20; ++k)
                    u[k] = is && (wg == 0 || k < 16) ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 5; ++k)
                    if (wg == 0 || k < 4)
                        tmem_st16(lanes + K::kColQ + 80u * wg + 16u * k, &u[4 * k].x);
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBQFull]);
                l0 = l1 = 0.0f;
                mneg = kUnseen;
                // rows that do not exist see everything: no mask for their sake
                lim = is ? piece->last + row / a.heads : 0x7FFFFFFF;
            }
            ok = ok && mbar_wait(&bar[K::kBSFull], ph, abort_flag);
            ok = __all_sync(kFull, ok);
            uint32_t sr[32];
            float p[32];
            uint32_t q[16];  // the weights as f16 pairs
            bool cleaned = false;
            auto weights = [&]() -> bool {
                uint32_t top = 0u;
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    ffma2_of(p[k], p[k + 1], sr[k], sr[k + 1], a.c_log2, mneg, mneg);
                    p[k] = ex2_approx(p[k]);
                    p[k + 1] = ex2_approx(p[k + 1]);
                    q[k / 2] = cache::pack_f16x2(p[k], p[k + 1]);
                    asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(q[k / 2]));
                }
                // halves compare as whole numbers: none is negative (0x5C00: 2^8)
                return (top & 0xFFFFu) > 0x5C00u || (top >> 16) > 0x5C00u;
            };
            bool over = true;
            if (ok) {
                tc_fence_after_sync();
                tmem_ld32(lanes + K::kColS + 32u * wg, sr);
                tmem_ld_wait();
                reg_fence_cols<32>(sr);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bar[K::kBSFree]);
                // tokens that are there and that the row sees
                const int past = lim - tile->tok - 32 * wg;
                const uint32_t sees = tile->have[wg] & (past >= 31 ? kFull : past < 0 ? 0u : (2u << past) - 1u);
                if (!__all_sync(kFull, sees == kFull)) {
                    const uint32_t never = __float_as_uint(a.c_log2 > 0.0f ? -INFINITY : INFINITY);
                    uint32_t nan = 0u;
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float x = __uint_as_float(sr[k]);
                        nan |= x != x ? 1u << k : 0u;
                        sr[k] = sees >> k & 1u ? sr[k] : never;
                    }
                    nan = __reduce_or_sync(kFull, nan);
                    cleaned = nan != 0u;
                    // in the queries, or in a token's row: then out of its values
                    for (; nan; nan &= nan - 1u) {
                        const uint32_t v = sbase + K::kOffV + (uint32_t)vs * K::kVBytes + v_offset(32 * wg + __ffs(nan) - 1, lane);
                        const uint4 w = lds128(v);
                        sts128(v, without_nan(w.x), without_nan(w.y), without_nan(w.z), without_nan(w.w));
                    }
                }
                over = weights();
            }
            float alpha = 1.0f;
            if (named_bar_or(1, 256, over)) {
                float x = -INFINITY;
                if (ok) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        x = fmaxf(x, __uint_as_float(sr[k]) * a.c_log2);
                    red[wg * K::kRows + row] = x;
                }
                if (!named_bar_and(1, 256, ok)) {
                    fail(a, abort_flag);
                    break;
                }
                x = fmaxf(x, red[(wg ^ 1) * K::kRows + row]);
                if (x + mneg > kTop) {
                    alpha = ex2_approx(-x - mneg);  // 0 where no score was seen before
                    mneg = -x;
                    l0 *= alpha;
                    l1 *= alpha;
                }
                weights();
            }
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                fadd2(l0, l1, p[k], p[k + 1]);
                fadd2(l0, l1, p[k + 2], p[k + 3]);
                uint32_t h0, h1, d0, d1;
                split2<true>(q[k / 2], h0, d0);
                split2<true>(q[k / 2 + 1], h1, d1);
                hi[k / 4] = h0 | h1 << 16;
                lo[k / 4] = d0 | d1 << 16;
            }
            // P, and O where m moved: the output of the tile before is done
            ok = ok && mbar_wait(&bar[K::kBPEmpty], ph ^ 1u, abort_flag);
            ok = __all_sync(kFull, ok);
            if (ok) {
                tc_fence_after_sync();
                if (!first && __any_sync(kFull, alpha != 1.0f)) {
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[32];
                        const uint32_t ta = lanes + K::kColO + 128u * wg + 32u * k;
                        tmem_ld32(ta, o);
                        tmem_ld_wait();
                        reg_fence_cols<32>(o);
#pragma unroll
                        for (int z = 0; z < 32; ++z)
                            o[z] = __float_as_uint(__uint_as_float(o[z]) * alpha);
                        tmem_st32(ta, o);
                    }
                }
                tmem_st8(lanes + K::kColP + 8u * wg, hi);
                tmem_st8(lanes + K::kColP + 16u + 8u * wg, lo);
                tmem_st_wait();
            }
            if (cleaned)
                fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar[K::kBPFull]);
            if (++vs == K::kStages)
                vs = 0;
            if (++e == K::kTiles) {
                e = 0;
                eph ^= 1u;
            }
            if (!(flags & kLast))
                continue;

            // ------------------------------------------------ end of a block
            ok = ok && mbar_wait(&bar[K::kBPEmpty], ph, abort_flag);
            ok = __all_sync(kFull, ok);
            red[wg * K::kRows + row] = l0 + l1;
            if (!named_bar_and(1, 256, ok)) {
                fail(a, abort_flag);
                break;
            }
            tc_fence_after_sync();
            const float L = red[row] + red[K::kRows + row];
            const Piece *const piece = reinterpret_cast<const Piece *>(smem + K::kOffPiece) + seg % K::kPieces;
            const bool sole = piece->sole != 0;
            const int rows = piece->rows - w4 * 32;  // from the warp's first on
            const long long at = (long long)piece->slot * K::kRows + row;
            if (wg == 0 && vh == 0 && lane < rows) {
                if (!sole) {
                    __stcg(a.ml + at * 2, -mneg);
                    __stcg(a.ml + at * 2 + 1, L);
                } else if (a.lse) {
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
                // turned in the warp's kilobyte, so that rows are stored 32 bytes at a time
                const uint32_t mine = turn + 32u * lane, flip = (uint32_t)(lane >> 2) & 1u;
                const int r0 = lane >> 1, half = lane & 1;
                const uint32_t other = turn + 32u * r0 + 16u * ((uint32_t)half ^ ((uint32_t)(r0 >> 2) & 1u));
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
                        sts128(mine + 16u * flip, b[0], b[1], b[2], b[3]);
                        sts128(mine + 16u * (flip ^ 1u), b[4], b[5], b[6], b[7]);
                        __syncwarp();
                        const uint4 v0 = lds128(other), v1 = lds128(other + 512u);
                        if (r0 < rows)
                            *reinterpret_cast<uint4 *>(out + r0 * kVDim + 32 * k + z + 8 * half) = v0;
                        if (r0 + 16 < rows)
                            *reinterpret_cast<uint4 *>(out + (r0 + 16) * kVDim + 32 * k + z + 8 * half) = v1;
                        __syncwarp();
                    }
                } else {
#pragma unroll
                    for (int z = 0; z < 32; z += 8) {
                        sts128(mine + 16u * flip, o[z], o[z + 1], o[z + 2], o[z + 3]);
                        sts128(mine + 16u * (flip ^ 1u), o[z + 4], o[z + 5], o[z + 6], o[z + 7]);
                        __syncwarp();
                        const uint4 v0 = lds128(other), v1 = lds128(other + 512u);
                        if (r0 < rows)
                            __stcg(reinterpret_cast<uint4 *>(part + r0 * kVDim + 32 * k + z + 4 * half), v0);
                        if (r0 + 16 < rows)
                            __stcg(reinterpret_cast<uint4 *>(part + (r0 + 16) * kVDim + 32 * k + z + 4 * half), v1);
                        __syncwarp();
                    }
                }
            }
            tc_fence_before_sync();
            if (flags & kEnd)
                break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == K::kPlanWarp) {
            plan_tiles<K>(a, smem, bar, range, g, 0, vh == 0, abort_flag);
        } else if (warp == K::kMmaWarp) {
            // -------------------------------------------------------- products
            // The scores of tile nq as soon as its rows are there and the scores before
            // were read, the output update of tile np as soon as its weights are there;
            // one elected lane of the converged warp issues.
            const Tile *const tiles = reinterpret_cast<const Tile *>(smem + K::kOffInfo);
            int nq = 0, np = 0, seg = 0, idle = 0;
            bool more_q = true, more_p = true, ok = true;
            int qv = 0, pv = 0, qe = 0, pe = 0;  // slots and descriptions of tiles nq and np
            uint32_t qvph = 0, qeph = 0;
            uint64_t idle_since = 0;
            const uint64_t kd = sw128_kmajor_desc_sbo(sbase, kVGroup), vd = sw128_mnmajor_desc(sbase, 1024u, kVGroup);
            const uint64_t rd = sw64_kmajor_desc(sbase, kRGroup);
            while (more_p) {
                bool prog = false;
                if (np < nq && __all_sync(kFull, mbar_test(&bar[K::kBPFull], (uint32_t)np & 1u))) {
                    const uint32_t flags = tiles[pe].flags;
                    const bool first = flags & kFirst;
                    tc_fence_after_sync();
                    const uint64_t bv = vd + ((K::kOffV + (uint32_t)pv * K::kVBytes + (uint32_t)vh * 2048u) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int term = 0; term < 2; ++term)
                                umma_f8_ts(tmem + K::kColO, tmem + K::kColP + 16u * term + 8u * ks,
                                           bv + (((uint32_t)ks * 4u * kVGroup) >> 4), term ? K::kIdescPVLo : K::kIdescPV,
                                           (first && ks == 0 && term == 0) ? 0u : 1u);
                        umma_commit(&bar[K::kBVEmpty + pv]);
                        umma_commit(&bar[K::kBPEmpty]);
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
                if (more_q && __all_sync(kFull, mbar_test(&bar[K::kBInfo + qe], qeph) && mbar_test(&bar[K::kBReady + qv], qvph) &&
                                                    mbar_test(&bar[K::kBSFree], ((uint32_t)nq & 1u) ^ 1u))) {
                    const uint32_t flags = tiles[qe].flags;
                    if (!(flags & kFirst) || __all_sync(kFull, mbar_test(&bar[K::kBQFull], (uint32_t)seg & 1u))) {
                        if (flags & kFirst)
                            ++seg;
                        fence_proxy_async_smem();  // cp.async writes -> tensor-core reads
                        tc_fence_after_sync();
                        const uint64_t bk = kd + ((K::kOffV + (uint32_t)qv * K::kVBytes) >> 4);
                        const uint64_t br = rd + ((K::kOffR + (uint32_t)qv * K::kRBytes) >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                umma_f8_ts(tmem + K::kColS, tmem + K::kColQ + 8u * k,
                                           bk + (((uint32_t)(k >> 2) * 1024u + (uint32_t)(k & 3) * 32u) >> 4), K::kIdescQK,
                                           k ? 1u : 0u);
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                umma_f8_ts(tmem + K::kColS, tmem + K::kColQ + 128u + 8u * k, br + 2u * k, K::kIdescQK, 1u);
                            umma_commit(&bar[K::kBSFull]);
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
                        ++nq;
                        more_q = !(flags & kEnd);
                        prog = true;
                    }
                }
                if (prog) {
                    idle = 0;
                    idle_since = 0;
                    continue;
                }
                // nothing ready: every 64 polls the abort flag and the clock
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
        tmem_dealloc(tmem, 512);
    }
}

cudaError_t launch_wide(Args &a, int sms, cudaStream_t st)
{
    a.tile = Wide::kTile;
    a.N = Wide::kRows;
    a.pad = 4;
    a.least = 4;
    a.hb = 1;
    a.peers = 2;
    a.toks = 1;
    while (2 * a.toks * a.heads <= Wide::kRows && 2 * a.toks <= Wide::kTile)
        a.toks *= 2;
    a.ranges = std::max(1, std::min(sms, kMaxCtas) / a.peers);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = cache::allow_smem(latent_wide_kernel, (int)Wide::kSmem, done);
    if (e != cudaSuccess)
        return e;
    latent_wide_kernel<<<(unsigned)(a.ranges * a.peers), Wide::kThreads, Wide::kSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace latent
}  // namespace pmqa
