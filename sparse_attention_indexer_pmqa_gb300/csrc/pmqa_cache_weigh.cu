// pmqa_cache_weigh.cu -- the attention weight that each cached token receives
// from a call's query rows, added to a running total per request and kv head:
//   mass_out[i][h][t] = mass_in[i][h][t] +
//       sum over rows j and heads hq of kv head h that see t of
//       exp(sm_scale q_(j,hq) . k_t - lse[j][hq]).
//
// Reads K once (D bytes per token and kv head) and nothing of V; every token
// belongs to one warp, so there are no atomics and the sums are the same on
// every run. Products run as S = K Q^T (tokens are the 16 rows of the
// m16n8k16 shape, query rows the 8 columns): a thread adds the weights of its
// own query rows in registers and four threads join theirs by two shuffles.
// Bound by HBM: one row of 32 requests of 4 to 16 k tokens, 32 query heads over 8,
// takes 64 us, 81 % of the measured copy rate.
#include <algorithm>
#include <cmath>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace cache {

constexpr int kWeighWarps = 4;
constexpr int kWeighThreads = 32 * kWeighWarps;
constexpr int kWarpTok = 32;
constexpr int kWeighTile = kWarpTok * kWeighWarps;
constexpr int kWeighStages = 3;
constexpr int kWeighPad = 1;  // what a context's start costs, in tiles: 16 requests of 1 to
                              // 4096 tokens and 32 rows take 20 us with it, 25 without

struct WeighArgs {
    View c;
    const uint16_t *q;
    const float *lse;      // [rows, heads]
    const float *mass_in;  // [bs, H, width] or null
    float *mass_out;
    long long width;
    float scale_log2;
    int heads, group;
    int least, most;
};

template <int D>
struct WeighStage {
    static constexpr uint32_t kRows = kWarpTok * D;
    static constexpr uint32_t kOffKs = kRows, kOffMass = kOffKs + 128, kOffMask = kOffMass + 128;
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
__global__ void __launch_bounds__(kWeighThreads, 3)
    cache_weigh_kernel(const __grid_constant__ WeighArgs a)
{
    using St = WeighStage<D>;
    constexpr int S = kWeighStages;
    constexpr int KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const View &c = a.c;
    const int G = a.group;
    Range rg;
    Walk w;
    find_range<kWeighTile, 0, kWeighPad, kWeighThreads>(c, G, a.least, a.most, 1, 0.0f, rg, w);
    if (rg.x0 >= rg.x1) {
        griddep_wait();
        return;
    }
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * S) * St::kBytes;

    if (w.t >= w.T) {  // the range starts behind a context's tiles
        rg.x0 += w.T + kWeighPad - w.t;
        w.t = w.T - 1;
        if (rg.x0 < rg.x1)
            w.template next<kWeighTile, 0, kWeighPad>(c, G, a.least, a.most);
    }
    if (rg.x0 >= rg.x1) {
        griddep_wait();
        return;
    }
    Walk pw = w;
    long long p_x = rg.x0;
    int pend_page = -1, pend_off = 0, pend_tok = 0, pend_h = 0, pend_i = 0;
    bool pend_in = false;
    bool pend_rows = false;  // the request has rows; otherwise its keys are not read
    auto look_up = [&]() {
        pend_in = false;
        if (p_x < rg.x1) {
            pend_tok = pw.t * kWeighTile + warp * kWarpTok + lane;
            pend_h = pw.h;
            pend_i = pw.i;
            pend_in = pend_tok < pw.q.ctx && pend_tok < a.width;
            pend_rows = pw.q.n > 0;
            const int pg = c.page_of(pend_tok);
            pend_off = pend_tok - pg * c.P;
            if (pend_in)
                pend_page = __ldg(c.bt + (long long)pw.i * c.W + pg);
            ++p_x;
            if (pw.t + 1 < pw.T) {
                ++pw.t;
            } else {
                p_x += kWeighPad;
                if (p_x < rg.x1)
                    pw.template next<kWeighTile, 0, kWeighPad>(c, G, a.least, a.most);
            }
        }
    };
    constexpr int CH = D / 16, PER = 32 / CH;
    const int ch = lane % CH;
    const bool one_block = (c.P & (kWarpTok - 1)) == 0;  // 32 tokens never leave a block
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
        // no mask bit for a token that no row sees: its weight is 0 whatever its key is
        ok = ok && pend_rows;
        const uint32_t mask = __ballot_sync(kFull, ok);
        const uint32_t here = __ballot_sync(kFull, pend_in);
        if (lane == 0)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + St::kOffMask), "r"(mask) : "memory");
        if (here) {
            const uint32_t phys = ok ? (uint32_t)pend_page * (uint32_t)c.H + (uint32_t)pend_h : 0u;
            const uint32_t row = phys * (uint32_t)c.P + (uint32_t)pend_off;
            if (ok)
                cp_async_4(st + St::kOffKs + (uint32_t)lane * 4u, c.ks + phys);
            if (pend_in && a.mass_in)
                cp_async_4(st + St::kOffMass + (uint32_t)lane * 4u,
                           a.mass_in + ((long long)pend_i * c.H + pend_h) * a.width + pend_tok);
            // 32 tokens of one block follow one another (token 0 exists if any does)
            const uint8_t *const lead =
                c.k + (uint64_t)(mask ? __shfl_sync(kFull, row, 0) : 0u) * D + (uint32_t)lane * 16u;
#pragma unroll
            for (int k = 0; k < kWarpTok / PER; ++k) {
                const int r = k * PER + lane / CH;
                const uint32_t nb = (mask >> r) & 1u ? 16u : 0u;
                const uint8_t *src = lead + k * 512;
                if (!one_block) {
                    const uint32_t rr = __shfl_sync(kFull, row, r);
                    src = c.k + (uint64_t)(nb ? rr : 0u) * D + (uint32_t)ch * 16u;
                }
                cp_async_16(st + St::at(r, ch), nb ? src : c.k, nb);
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

    uint32_t qb[NT][KS][2];
    float rc[NT][2], rl[NT][2];  // scale and lse (base 2) of rows 2 t4, 2 t4 + 1 of each 8
    int lim[NT][2];
    // the query rows of the current request and head into registers (at most 8 NT of them)
    auto load_rows = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int R = nt * 8 + g;
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
                    const float lo = __uint_as_float(e[z] << 16) * up;
                    const float hi = __uint_as_float(e[z] & 0xFFFF0000u) * up;
                    qb[nt][(k >> 1) * 4 + (k & 1) * 2 + (z >> 1)][z & 1] = pack_f16x2(lo, hi);
                }
            }
            // an infinite value would leave its row the tokens of score -inf: NaN instead
            const float mine = top < INFINITY ? a.scale_log2 * down : __int_as_float(0x7FFFFFFF);
            rc[nt][0] = __shfl_sync(kFull, mine, 8 * t4);
            rc[nt][1] = __shfl_sync(kFull, mine, 8 * t4 + 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int Re = nt * 8 + 2 * t4 + e;
                const bool row = Re < w.q.n * G;
                lim[nt][e] = row ? w.q.ctx - w.q.n + Re / G : -1;
                rl[nt][e] = row ? __ldg(a.lse + (long long)(w.q.r0 + Re / G) * a.heads + w.h * G + Re % G) * kLog2e
                                : INFINITY;
            }
        }
    };
    int c_slot = 0;
    bool fresh = true;
#pragma unroll 1
    for (long long x = rg.x0; x < rg.x1;) {
        if (fresh) {
            load_rows();
            fresh = false;
        }
        cp_async_wait_group<S - 2>();
        __syncwarp();
        issue();
        look_up();
        const uint32_t st = ring + (uint32_t)c_slot * St::kBytes;
        if (++c_slot == S)
            c_slot = 0;
        const int base = w.t * kWeighTile + warp * kWarpTok;
        if (base < w.q.ctx) {
            const uint32_t mask = lds32(st + St::kOffMask);
            float s[2][NT][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[u][nt][e] = 0.0f;
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint4 u0 = lds128(st + St::at(g + 16 * u, half * 4 + t4));
                    const uint4 u1 = lds128(st + St::at(g + 16 * u + 8, half * 4 + t4));
                    const uint32_t wa[4] = {u0.x, u0.y, u0.z, u0.w}, wb[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_f16x2(wa[z], a0, a2);
                        e4m3x4_to_f16x2(wb[z], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(s[u][nt], a0, a1, a2, a3, qb[nt][half * 4 + z][0], qb[nt][half * 4 + z][1]);
                    }
                }
            // every row sees every token of the chunk (rows that do not exist weigh 0)
            const bool whole = mask == kFull && base + kWarpTok - 1 <= w.q.ctx - w.q.n;
            float sum[4];  // of tokens g, g + 8, g + 16, g + 24
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int tok = g + 8 * v;
                const float ks = __uint_as_float(lds32(st + St::kOffKs + 4u * (uint32_t)tok));
                const bool have = (mask >> tok) & 1u;
                float t = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float y = ex2_approx(s[v >> 1][nt][2 * (v & 1) + e] * (ks * rc[nt][e]) - rl[nt][e]);
                        t += whole || (have && base + tok <= lim[nt][e]) ? y : 0.0f;
                    }
                t += __shfl_xor_sync(kFull, t, 1);
                sum[v] = t + __shfl_xor_sync(kFull, t, 2);
            }
            // lane (g, t4) writes token g + 8 t4
            const int tok = g + 8 * t4, slot = base + tok;
            if (slot < w.q.ctx && slot < a.width) {
                const float got = t4 == 0 ? sum[0] : t4 == 1 ? sum[1] : t4 == 2 ? sum[2] : sum[3];
                const float had =
                    a.mass_in ? __uint_as_float(lds32(st + St::kOffMass + 4u * (uint32_t)tok)) : 0.0f;
                a.mass_out[((long long)w.i * c.H + w.h) * a.width + slot] = had + got;
            }
        }
        ++x;
        if (w.t + 1 < w.T) {
            ++w.t;
            continue;
        }
        x += kWeighPad;
        if (x < rg.x1) {
            w.template next<kWeighTile, 0, kWeighPad>(c, G, a.least, a.most);
            fresh = true;
        }
    }
    cp_async_wait_all();
    griddep_wait();  // this kernel may start before the many-row one is done; it ends after it
}

template <int D, int NT>
static cudaError_t launch(const WeighArgs &a, int sms, bool early, cudaStream_t st)
{
    const int smem = (int)(kWeighWarps * kWeighStages * WeighStage<D>::kBytes);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(cache_weigh_kernel<D, NT>, smem, done);
    if (e != cudaSuccess)
        return e;
    return launch_early(cache_weigh_kernel<D, NT>, dim3(3u * (unsigned)sms), kWeighThreads, smem, early, st, a);
}

// Requests with least <= rows * group <= most. early: the kernel before this one
// in the stream is the many-row kernel of the same call.
cudaError_t launch_weigh_rows(const WeighCall &q, int least, int most, int sms, bool early, cudaStream_t st)
{
    WeighArgs a{};
    a.c = q.c;
    a.q = static_cast<const uint16_t *>(q.q);
    a.lse = q.lse;
    a.mass_in = q.mass_in;
    a.mass_out = q.mass_out;
    a.width = q.width;
    a.scale_log2 = q.sm_scale * kLog2e;
    a.heads = q.heads;
    a.group = q.heads / q.c.H;
    a.least = least;
    a.most = most;
    const long long need = std::min<long long>((long long)q.c.max_rows * a.group, most);
    if (q.c.D == 128)
        return need <= 8 ? launch<128, 1>(a, sms, early, st)
               : need <= 16 ? launch<128, 2>(a, sms, early, st)
                            : launch<128, 4>(a, sms, early, st);
    return need <= 8 ? launch<64, 1>(a, sms, early, st)
           : need <= 16 ? launch<64, 2>(a, sms, early, st)
                        : launch<64, 4>(a, sms, early, st);
}

}  // namespace cache
}  // namespace pmqa
