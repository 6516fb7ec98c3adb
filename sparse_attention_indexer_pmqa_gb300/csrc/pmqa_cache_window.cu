// pmqa_cache_window.cu -- the attention weight of cached tokens (see
// pmqa_cache_weigh.cu) for requests with many query rows: the rows of a prompt
// chunk, or of an observation window before an eviction.
//
// S^T = K Q^T on the tensor cores (kind::f8f6f4): the cached codes as they are
// are the M = 128 tokens, q (an e4m3 and an e5m2 term, exact for bf16 values from
// 2^-13 of their row's largest on: split_terms) the N = 128 packed rows
// R = j * group + g. A thread then owns one token and adds the weights of its 128
// columns in registers,
//   w_t = sum_R 2^(S ks_t c_R - lse_R log2 e),
// so there is no reduction over lanes and no atomic.
//
// A CTA keeps 256 packed rows of one (request, kv head) as operands and streams
// token tiles past them; more rows are further rounds over the same tiles. Tiles
// of all requests are split evenly over the CTAs, weighted by their rounds. A tile of
// 256 rows takes about 3200 cycles: its products 1050 (D / 32 * 2 of 66 cycles per 128
// rows), the weights 1560 issue slots of each scheduler (6.1 instructions a score and
// lane, all of the kernel's counted). Windows of 64 rows of 4 requests of 16 to 32 k
// tokens (32 query heads over 8) take 75 us, 33 % of the measured bf16 rate counted for
// one product: a row tile's scores, sums and hand-back follow one another, and four warps
// a scheduler overlap them at 49 % of the issue slots. K comes row by row: tensor copies
// of whole blocks were no faster (89 us against 86).
#include <algorithm>
#include <cmath>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace cache {

constexpr int kWnRows = 256;
constexpr int kWnTok = 128;
constexpr int kWnThreads = 18 * 32;  // warps 0-15: four warpgroups of sums; 16: products; 17: K rows
constexpr int kWnStages = 4;
constexpr uint32_t kWnTile = 128 * 128;

constexpr uint32_t kWnOffQ = 0;                                // [2 tiles][hi, lo]
constexpr uint32_t kWnOffK = kWnOffQ + 4 * kWnTile;
constexpr uint32_t kWnOffRow = kWnOffK + kWnStages * kWnTile;  // [256] c_R, [256] -lse log2 e, [256] last slot
constexpr uint32_t kWnOffKs = kWnOffRow + 3 * kWnRows * 4;     // [stages][128]: key scale, NaN bits for no token
constexpr uint32_t kWnOffHave = kWnOffKs + kWnStages * 512;    // [stages][4] mask words
constexpr uint32_t kWnOffSum = kWnOffHave + kWnStages * 16;    // [2 buffers][2][128] the second row tile's sums
constexpr uint32_t kWnOffMin = kWnOffSum + 4 * 512;            // [8] smallest last slot of each 32 rows
constexpr uint32_t kWnOffBar = kWnOffMin + 32;
enum {
    kWKFull = 0,                       // [4] K rows landed: 32 cp.async arrivals and lane 0's own
    kWKEmpty = kWKFull + kWnStages,    // [4] products done (commit), scales read (8 warps)
    kWSFull = kWKEmpty + kWnStages,    // [2 buffers][2 row tiles] scores: commit
    kWSEmpty = kWSFull + 4,            // [2][2] scores read: 4 warps
    kWDrain = kWSEmpty + 4,            // every product done, before the columns are freed: commit
    kWCount = kWDrain + 1
};
constexpr uint32_t kWnOffMisc = kWnOffBar + kWCount * 8;
constexpr uint32_t kWnSmem = kWnOffMisc + 16;
static_assert(kWnSmem <= 232448, "shared memory budget");

struct WindowArgs {
    View c;
    const uint16_t *q;
    const float *lse;
    const float *mass_in;
    float *mass_out;
    long long width;
    float scale_log2;
    int heads, group;
    int least;
};

__device__ __forceinline__ uint32_t wn_sw128(int r, int c)
{
    return (uint32_t)(r * 128) + (uint32_t)((c ^ (r & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kWnThreads, 1) cache_window_kernel(const __grid_constant__ WindowArgs a)
{
    constexpr int CH = D / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_units;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);
    const View &c = a.c;
    const int G = a.group;
    uint64_t *const bar = reinterpret_cast<uint64_t *>(smem + kWnOffBar);
    uint32_t *const misc = reinterpret_cast<uint32_t *>(smem + kWnOffMisc);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    griddep_launch_dependents();  // the few-row kernel fills the SMs that run out of tiles
    if (sbase & 1023u) {
        if (tid == 0)
            atomicOr(c.status, (uint32_t)PMQA_DEV_INTERNAL);
        return;
    }

    // ------------------------------------------------------------ this CTA's share
    // units: (request, head, tile, round), rounds fastest; a tile belongs to the
    // CTA whose range holds its first unit
    auto units = [&](const Request &q, int &T, int &B) -> long long {
        T = (q.ctx + kWnTok - 1) / kWnTok;
        B = q.n * G >= a.least ? (q.n * G + kWnRows - 1) / kWnRows : 0;
        return (long long)c.H * T * B;
    };
    if (tid == 0)
        s_units = 0;
    __syncthreads();
    {
        long long mine = 0;
        int T, B;
        for (int i = tid; i < c.bs; i += kWnThreads)
            mine += units(load_request(c, i, blockIdx.x == 0), T, B);
        if (mine)
            atomicAdd(reinterpret_cast<unsigned long long *>(&s_units), (unsigned long long)mine);
    }
    __syncthreads();
    const long long total = s_units;
    if (total == 0)
        return;
    const long long x0 = blockIdx.x * total / gridDim.x, x1 = (blockIdx.x + 1) * total / gridDim.x;
    if (x0 >= x1)
        return;

    if (tid == 0) {
        for (int s = 0; s < kWnStages; ++s) {
            mbar_init(&bar[kWKFull + s], 33);
            mbar_init(&bar[kWKEmpty + s], 9);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&bar[kWSFull + s], 1);
            mbar_init(&bar[kWSEmpty + s], 4);
        }
        mbar_init(&bar[kWDrain], 1);
        misc[1] = 0;
        mbar_init_fence();
    }
    if (warp == 16)
        tmem_alloc(misc, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = misc[0];  // buffer b, row tile r: columns 256 b + 128 r
    auto fail = [&]() {
        atomicOr(c.status, (uint32_t)PMQA_DEV_TIMEOUT);
        *abort_flag = 1;
    };

    // Every role walks the same segments (request, head, tiles [t0, t1)) and
    // rounds; `n` counts the tiles of the CTA over all of them.
    int n = 0;
    bool ok = true;
    long long before = 0;
#pragma unroll 1
    for (int i = 0; i < c.bs && before < x1; ++i) {
        const Request q = load_request(c, i, false);
        int T, B;
        const long long all = units(q, T, B);
        if (before + all <= x0) {
            before += all;
            continue;
        }
        // tiles (over the heads) whose first unit lies in [x0, x1)
        const long long y0 = x0 > before ? (x0 - before + B - 1) / B : 0;
        const long long y1 = x1 < before + all ? (x1 - before + B - 1) / B : (long long)c.H * T;
        before += all;
#pragma unroll 1
        for (long long y = y0; y < y1;) {
            const int h = (int)(y / T), t0 = (int)(y - (long long)h * T);
            const int t1 = (int)min((long long)T, t0 + (y1 - y));
            y += t1 - t0;
#pragma unroll 1
            for (int round = 0; round < B; ++round) {
                const int R0 = round * kWnRows, nrow = min(kWnRows, q.n * G - R0);
                const bool two = nrow > 128;
                // ---------------------------------------- the rows as operands
                // (every warp is done with the previous round's)
                __syncthreads();
                if (warp < 8) {
                    const int row = tid;  // 0 .. 255
                    const int R = R0 + row, j = R / G, g = R - j * G;
                    const bool has = row < nrow;
                    const long long rh = (long long)(q.r0 + j) * a.heads + h * G + g;
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + rh * D);
                    float top = 0.0f;
                    bool nan = false;
                    // the row is read twice (its largest value, then the terms): registers are few
#pragma unroll 4
                    for (int k = 0; k < D / 8; ++k) {
                        const uint4 u = has ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
                        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float f0 = __uint_as_float(e[z] << 16), f1 = __uint_as_float(e[z] & 0xFFFF0000u);
                            nan |= !(fabsf(f0) < INFINITY) || !(fabsf(f1) < INFINITY);
                            top = fmaxf(top, fmaxf(fabsf(f0), fabsf(f1)));
                        }
                    }
                    const int e2 = min(max((int)(__float_as_uint(top) >> 23) - 127, -119), 127);
                    const float up = __uint_as_float((uint32_t)(7 - e2 + 127) << 23);
                    const uint32_t qd = sbase + kWnOffQ + (uint32_t)(row >> 7) * 2 * kWnTile;
#pragma unroll 2
                    for (int k = 0; k < D / 8; k += 2) {
                        uint32_t hi[4], lw[4];
                        const uint4 ua = has ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
                        const uint4 ub = has ? __ldg(src + k + 1) : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint4 &uu = z < 2 ? ua : ub;
                            const uint32_t e0 = (z & 1) ? uu.z : uu.x, e1 = (z & 1) ? uu.w : uu.y;
                            const float f0 = __uint_as_float(e0 << 16) * up, f1 = __uint_as_float(e0 & 0xFFFF0000u) * up;
                            const float f2 = __uint_as_float(e1 << 16) * up, f3 = __uint_as_float(e1 & 0xFFFF0000u) * up;
                            split_terms(f0, f1, f2, f3, hi[z], lw[z]);
                        }
                        sts128(qd + wn_sw128(row & 127, k >> 1), hi[0], hi[1], hi[2], hi[3]);
                        sts128(qd + kWnTile + wn_sw128(row & 127, k >> 1), lw[0], lw[1], lw[2], lw[3]);
                    }
                    // a row that does not exist: c = 0 and -inf, so its weights are 0
                    float *const rowv = reinterpret_cast<float *>(smem + kWnOffRow);
                    const int last = has ? q.ctx - q.n + j : 0x7FFFFFFF;
                    rowv[row] = !has ? 0.0f
                                : nan ? __int_as_float(0x7FFFFFFF)
                                      : a.scale_log2 * __uint_as_float((uint32_t)(e2 - 7 + 127) << 23);
                    rowv[kWnRows + row] = has ? -__ldg(a.lse + rh) * kLog2e : -INFINITY;
                    reinterpret_cast<int *>(rowv)[2 * kWnRows + row] = last;
                    int low = last;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        low = min(low, __shfl_xor_sync(kFull, low, o));
                    if (lane == 0)
                        reinterpret_cast<int *>(smem + kWnOffMin)[warp] = low;
                    fence_proxy_async_smem();
                }
                if (tid == kWnThreads - 1)
                    misc[2] = (uint32_t)*abort_flag;
                __syncthreads();
                if (misc[2]) {  // the same for every thread: no barrier is left half full
                    n += t1 - t0;
                    continue;
                }
                if (warp < 16) {
                    // ------------------------------------ sums: buffer b, row tile r
                    const int b = warp >> 3, r = (warp >> 2) & 1;
                    const int tok = (warp & 3) * 32 + lane;  // TMEM lane
                    const int *const lows = reinterpret_cast<const int *>(smem + kWnOffMin) + 4 * r;
                    const int low = min(min(lows[0], lows[1]), min(lows[2], lows[3]));
                    const float *const rc = reinterpret_cast<const float *>(smem + kWnOffRow) + 128 * r;
                    const float *const nl = rc + kWnRows;
                    const int *const last = reinterpret_cast<const int *>(rc) + 2 * kWnRows;
                    const uint32_t tS = tmem + 256u * b + 128u * r + ((uint32_t)((warp & 3) * 32) << 16);
                    for (int t = t0; t < t1; ++t) {
                        const int k = n + (t - t0);
                        if ((k & 1) != b)
                            continue;
                        const int st = k % kWnStages;
                        ok = ok && mbar_wait(&bar[kWSFull + 2 * b + r], (uint32_t)(k >> 1) & 1u, abort_flag) &&
                             mbar_wait(&bar[kWKFull + st], (uint32_t)(k / kWnStages) & 1u, abort_flag);
                        ok = __all_sync(kFull, ok);
                        if (!ok)
                            fail();
                        const int slot = t * kWnTok + tok;
                        const bool in = slot < q.ctx && slot < a.width;
                        const bool have = lds32(sbase + kWnOffHave + (uint32_t)(st * 16 + 4 * (warp & 3))) >> lane & 1u;
                        const float ks = have ? reinterpret_cast<const float *>(smem + kWnOffKs)[st * 128 + tok] : 0.0f;
                        float *const dst = a.mass_out + ((long long)i * c.H + h) * a.width + slot;
                        float had = 0.0f;
                        if (r == 0 && in) {
                            if (round > 0)
                                had = *dst;
                            else if (a.mass_in)
                                had = a.mass_in[((long long)i * c.H + h) * a.width + slot];
                        }
                        float s0 = 0.0f, s1 = 0.0f;
                        if (ok && (r == 0 || two)) {
                            tc_fence_after_sync();
                            const bool whole = __all_sync(kFull, slot <= low);
                            // 16 columns are worked on while the next 16 load
                            uint32_t v[2][16];
                            tmem_ld16(tS, v[0]);
#pragma unroll 1
                            for (int cc = 0; cc < 8; cc += 2) {
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int col = 16 * (cc + y);
                                    tmem_ld_wait();
                                    reg_fence_cols<16>(v[y]);
                                    if (y == 0 || cc < 6)
                                        tmem_ld16(tS + (uint32_t)(col + 16), v[y ^ 1]);
#pragma unroll
                                    for (int z = 0; z < 16; z += 4) {
                                        const float4 c4 = *reinterpret_cast<const float4 *>(rc + col + z);
                                        const float4 l4 = *reinterpret_cast<const float4 *>(nl + col + z);
                                        float y0, y1, y2, y3, w0 = l4.x, w1 = l4.y, w2 = l4.z, w3 = l4.w;
                                        fmul2(y0, y1, __uint_as_float(v[y][z]), __uint_as_float(v[y][z + 1]), c4.x, c4.y);
                                        fmul2(y2, y3, __uint_as_float(v[y][z + 2]), __uint_as_float(v[y][z + 3]), c4.z, c4.w);
                                        ffma2(w0, w1, y0, y1, ks, ks);
                                        ffma2(w2, w3, y2, y3, ks, ks);
                                        w0 = ex2_approx(w0);
                                        w1 = ex2_approx(w1);
                                        w2 = ex2_approx(w2);
                                        w3 = ex2_approx(w3);
                                        if (!whole) {
                                            const int4 e = *reinterpret_cast<const int4 *>(last + col + z);
                                            w0 = slot <= e.x ? w0 : 0.0f;
                                            w1 = slot <= e.y ? w1 : 0.0f;
                                            w2 = slot <= e.z ? w2 : 0.0f;
                                            w3 = slot <= e.w ? w3 : 0.0f;
                                        }
                                        fadd2(s0, s1, w0, w1);
                                        fadd2(s0, s1, w2, w3);
                                    }
                                }
                            }
                            tc_fence_before_sync();
                        }
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bar[kWSEmpty + 2 * b + r]);
                            mbar_arrive(&bar[kWKEmpty + st]);
                        }
                        const float sum = have ? s0 + s1 : 0.0f;
                        // row tile 1 hands its sums to row tile 0, which writes
                        float *const ex = reinterpret_cast<float *>(smem + kWnOffSum) + (2 * b + ((k >> 1) & 1)) * 128;
                        if (two) {
                            if (r == 1)
                                ex[tok] = sum;
                            named_bar_sync(1 + b, 256);
                        }
                        if (r == 0 && in && ok)
                            *dst = had + (two ? sum + ex[tok] : sum);
                    }
                } else if (warp == 16) {
                    // ------------------------------------ products
                    if (lane == 0) {
                        const uint32_t id = idesc_e4m3_f32(128, 128);
                        for (int t = t0; ok && t < t1; ++t) {
                            const int k = n + (t - t0), st = k % kWnStages, b = k & 1;
                            ok = mbar_wait(&bar[kWKFull + st], (uint32_t)(k / kWnStages) & 1u, abort_flag);
                            if (!ok)
                                break;
                            fence_proxy_async_smem();
                            const uint64_t kd = sw128_kmajor_desc(sbase + kWnOffK + (uint32_t)st * kWnTile);
#pragma unroll 1
                            for (int r = 0; ok && r < 2; ++r) {
                                ok = mbar_wait(&bar[kWSEmpty + 2 * b + r], ((uint32_t)(k >> 1) & 1u) ^ 1u, abort_flag);
                                if (!ok)
                                    break;
                                tc_fence_after_sync();
                                const uint64_t qd = sw128_kmajor_desc(sbase + kWnOffQ + (uint32_t)r * 2 * kWnTile);
                                if (r == 0 || two) {
#pragma unroll
                                    for (int z = 0; z < D / 16; ++z)
                                        umma_e4m3(tmem + 256u * b + 128u * r, kd + 2u * (z % (D / 32)),
                                                  qd + (uint64_t)((z / (D / 32)) * (kWnTile >> 4)) + 2u * (z % (D / 32)),
                                                  z < D / 32 ? id : id | kIdescBE5m2, z ? 1u : 0u);
                                }
                                umma_commit(&bar[kWSFull + 2 * b + r]);
                            }
                            if (!ok)
                                break;
                            umma_commit(&bar[kWKEmpty + st]);
                        }
                        if (!ok)
                            fail();
                    }
                    ok = __shfl_sync(kFull, ok ? 1 : 0, 0);
                } else {
                    // ------------------------------------ K rows and scales
                    const int32_t *const bt = c.bt + (long long)i * c.W;
                    constexpr uint32_t kNone = 0xFFFFFFFFu;
                    constexpr int PER = 32 / CH;
                    const int ch = lane % CH;
                    int page[4];
                    auto look_up = [&](int t) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tk = t * kWnTok + 32 * k + lane;
                            page[k] = t < t1 && tk < q.ctx ? __ldg(bt + c.page_of(tk)) : -1;
                        }
                    };
                    look_up(t0);
                    for (int t = t0; t < t1; ++t) {
                        const int k0 = n + (t - t0), st = k0 % kWnStages;
                        uint32_t phys[4], row[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tk = t * kWnTok + 32 * k + lane;
                            phys[k] = row[k] = kNone;
                            if (tk < q.ctx) {
                                if (page[k] < 0 || (long long)page[k] >= c.nb) {
                                    atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
                                } else {
                                    phys[k] = (uint32_t)page[k] * (uint32_t)c.H + (uint32_t)h;
                                    row[k] = phys[k] * (uint32_t)c.P + (uint32_t)(tk - c.page_of(tk) * c.P);
                                }
                            }
                        }
                        look_up(t + 1);
                        ok = ok && mbar_wait(&bar[kWKEmpty + st], ((uint32_t)(k0 / kWnStages) & 1u) ^ 1u, abort_flag);
                        ok = __all_sync(kFull, ok);
                        if (!ok) {
                            fail();
                            break;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t mask = __ballot_sync(kFull, phys[k] != kNone);
                            if (lane == 0)
                                asm volatile("st.shared.b32 [%0], %1;" ::"r"(sbase + kWnOffHave + (uint32_t)(st * 16 + 4 * k)),
                                             "r"(mask) : "memory");
                            if (phys[k] != kNone)
                                cp_async_4(sbase + kWnOffKs + (uint32_t)(st * 512 + (32 * k + lane) * 4), c.ks + phys[k]);
                        }
                        const uint32_t dst = sbase + kWnOffK + (uint32_t)st * kWnTile;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int y2 = 0; y2 < CH; ++y2) {
                                const int rr = y2 * PER + lane / CH, rt = 32 * k + rr;
                                const uint32_t src = __shfl_sync(kFull, row[k], rr);
                                cp_async_16(dst + wn_sw128(rt, ch),
                                            c.k + (src == kNone ? 0ull : (unsigned long long)src * D) + ch * 16,
                                            src == kNone ? 0u : 16u);
                            }
                        cp_async_arrive_noinc(&bar[kWKFull + st]);
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&bar[kWKFull + st]);
                    }
                }
                n += t1 - t0;
            }
        }
    }
    cp_async_wait_all();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 16) {
        // products still in flight after a failure end before their columns are freed
        if (lane == 0) {
            umma_commit(&bar[kWDrain]);
            if (!mbar_wait(&bar[kWDrain], 0u, nullptr))
                atomicOr(c.status, (uint32_t)PMQA_DEV_TIMEOUT);
        }
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Requests with at least `least` packed rows (rows * group).
cudaError_t launch_weigh_window(const WeighCall &q, int least, int sms, cudaStream_t st)
{
    WindowArgs a{};
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
    static std::atomic<uint64_t> done64{0}, done128{0};
    cudaError_t e = q.c.D == 128 ? allow_smem(cache_window_kernel<128>, (int)kWnSmem, done128)
                                 : allow_smem(cache_window_kernel<64>, (int)kWnSmem, done64);
    if (e != cudaSuccess)
        return e;
    if (q.c.D == 128)
        cache_window_kernel<128><<<sms, kWnThreads, kWnSmem, st>>>(a);
    else
        cache_window_kernel<64><<<sms, kWnThreads, kWnSmem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace cache
}  // namespace pmqa
