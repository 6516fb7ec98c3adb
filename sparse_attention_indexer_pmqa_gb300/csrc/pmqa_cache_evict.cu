// pmqa_cache_evict.cu -- eviction from the paged 8-bit K/V cache by accumulated
// attention weight: per request and kv head, the tokens to keep, then their
// keys and values moved into fewer blocks.
//
// Selection. A request with ctx <= keep keeps everything. Otherwise the first
// `sinks` and the last `recent` tokens stay, and of the ones between the
// keep - sinks - recent with the largest mass (equal masses: the lower slot; a
// NaN counts as the lowest). One cluster per (request, kv head): each CTA holds
// its slice of the masses as order-preserving 32-bit keys in shared memory
// (read once from HBM), three histogram passes of 11 + 11 + 10 bits find the
// threshold key, each pass joined over the cluster through distributed shared
// memory, and a count over warps turns the kept flags into positions in slot
// order. Everything is integer arithmetic: the result does not depend on the
// order of the atomics.
//
// Move. A unit (request, head, new block, pool) gathers its rows through the
// kept list and the old table, takes the largest |code * scale| for the new
// block's power-of-two scale, and writes the codes rounded to it: 2 D bytes in
// and out per kept token and head.
//
// 16 requests of 2 to 64 k tokens and 8 kv heads cut to 4096 tokens take 115 us back to
// back. The selection takes 57 us in one cold launch (of a CTA's 27: 9 for the masses and
// the first histogram, 10 for the other passes and their joins, 8 for the places; smaller
// CTAs, two of them per SM, take 1.1 to 1.4 times as long), bound by the instructions and
// latencies of its passes at 56 % of the issue slots. The move takes 65 us at 3.5 TB/s:
// the look-ups and conversions of a row bind it, at 87 % of the issue slots. One request of
// 1500 tokens: 13.5 us back to back.
#include <cooperative_groups.h>

#include <algorithm>

#include "pmqa_cache_host.cuh"

namespace cg = cooperative_groups;

namespace pmqa {
namespace cache {

constexpr int kSelThr = 1024;
constexpr int kSelWarps = kSelThr / 32;
constexpr int kBins = 2048;
constexpr int kKeysMax = 48 * 1024;  // keys of a CTA's slice kept in shared memory (192 KB)
constexpr int kMoveThreads = 128;

struct EvictArgs {
    View c;
    const float *mass;
    long long width;
    int keep, sinks, recent;
    const int32_t *new_bt;
    int new_w;
    int32_t *kept, *lens_out;
    float *mass_out;
    int cs;        // CTAs per cluster
    int key_cap;   // keys of a slice that fit the shared memory given
    int pages;     // new blocks per request (upper bound)
    int ranked;    // requests are taken in the order of falling length
};

// Larger floats get larger keys; both zeros the same one; NaN the lowest.
__device__ __forceinline__ uint32_t mass_key(float x)
{
    if (x != x)
        return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One more key in `bin` of a histogram, for every lane with `in`: the lanes that
// share the first one's bin (masses pile up at zero) add up first.
__device__ __forceinline__ void count_key(uint32_t *hist, uint32_t bin, bool in, int lane)
{
    const uint32_t act = __ballot_sync(kFull, in);
    if (act == 0)
        return;
    const int lead = __ffs(act) - 1;
    const uint32_t first = __shfl_sync(kFull, bin, lead);
    const uint32_t same = __ballot_sync(kFull, in && bin == first);
    if (lane == lead)
        atomicAdd(&hist[bin], (uint32_t)__popc(same));
    else if (in && !(same >> lane & 1u))
        atomicAdd(&hist[bin], 1u);
}

__global__ void __launch_bounds__(kSelThr, 1) cache_evict_select_kernel(const __grid_constant__ EvictArgs a)
{
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[2][kBins];
    __shared__ uint32_t s_warp[kSelWarps];
    __shared__ uint32_t s_cnt[2];             // this slice's keys above and at the threshold
    __shared__ uint32_t s_gt[kSelWarps], s_eq[kSelWarps];
    __shared__ uint32_t s_pick[2];            // bin chosen, rank left within it
    cg::cluster_group cl = cg::this_cluster();
    const View &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cl.block_rank();
    long long pair = blockIdx.x / a.cs;
    int i = (int)(pair / c.H);
    griddep_launch_dependents();
    if (a.ranked) {
        // the request with i longer ones (of equal ones, the first come first)
        __shared__ int s_req;
        if (tid < c.bs) {
            const int mine = __ldg(c.ctx + tid);
            int before = 0;
            for (int j = 0; j < c.bs; ++j) {
                const int other = __ldg(c.ctx + j);
                before += other > mine || (other == mine && j < tid);
            }
            if (before == i)
                s_req = tid;
        }
        __syncthreads();
        pair += (long long)(s_req - i) * c.H;
        i = s_req;
    }
    int ctx = clamp_ctx(c, i, rank == 0 && tid == 0 && pair % c.H == 0);
    if (ctx > a.width) {
        if (rank == 0 && tid == 0)
            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);
        ctx = (int)a.width;
    }
    const int len = min(ctx, a.keep);
    const float *const mass = a.mass + pair * a.width;
    float *const mass_out = a.mass_out ? a.mass_out + pair * a.width : nullptr;
    int32_t *const kept = a.kept + pair * a.keep;
    if (rank == 0 && tid == 0 && pair % c.H == 0)
        a.lens_out[i] = len;
    // what lies behind the kept tokens
    const int all = a.cs * kSelThr, at = rank * kSelThr + tid;
    for (long long p = (long long)len + at; p < a.keep; p += all)
        kept[p] = -1;
    if (mass_out)
        for (long long p = (long long)len + at; p < a.width; p += all)
            mass_out[p] = 0.0f;
    if (ctx <= a.keep) {
        for (int p = at; p < ctx; p += all) {
            kept[p] = p;
            if (mass_out)
                mass_out[p] = __ldg(mass + p);
        }
        return;  // the same for the whole cluster
    }
    // slice [lo, hi) of the slots, a warp's span of it, in slot order
    const int chunk = ((ctx + a.cs - 1) / a.cs + 1023) & ~1023;
    const int lo = min(rank * chunk, ctx), hi = min(lo + chunk, ctx);
    const int mid0 = a.sinks, mid1 = ctx - a.recent;  // slots that compete
    auto key_of = [&](int t) -> uint32_t {
        return t - lo < a.key_cap ? keys[t - lo] : mass_key(__ldg(mass + t));
    };
    for (int b = tid; b < 2 * kBins; b += kSelThr)
        (&hist[0][0])[b] = 0u;
    __syncthreads();
    // keys into shared memory, and the first histogram (top 11 bits)
    for (int t0 = lo; t0 < hi; t0 += 4 * kSelThr) {
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = t0 + k * kSelThr + tid;
            f[k] = t < hi ? __ldg(mass + t) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = t0 + k * kSelThr + tid;
            const uint32_t key = mass_key(f[k]);
            if (t < hi && t - lo < a.key_cap)
                keys[t - lo] = key;
            count_key(hist[0], key >> 21, t < hi && t >= mid0 && t < mid1, lane);
        }
    }
    uint32_t want = (uint32_t)(a.keep - a.sinks - a.recent);  // rank (from the top) of the last kept key
    uint32_t prefix = 0;  // bits of the threshold found so far
    const bool any = want > 0;
#pragma unroll 1
    for (int pass = 0; pass < 3 && any; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const int bins = pass == 2 ? 1024 : kBins;
        uint32_t *const h = hist[pass & 1];
        cl.sync();  // every CTA's histogram of this pass is complete
        // thread owns bins 2 tid, 2 tid + 1, counted from the top
        uint32_t n0 = 0, n1 = 0;
        const int b0 = bins - 1 - 2 * tid;  // the larger bin of the two
        if (b0 > 0)
            for (int r = 0; r < a.cs; ++r) {
                const uint32_t *o = cl.map_shared_rank(h, r);
                n0 += o[b0];
                n1 += o[b0 - 1];
            }
        uint32_t inc = n0 + n1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o)
                inc += y;
        }
        if (lane == 31)
            s_warp[warp] = inc;
        __syncthreads();
        uint32_t before = inc - n0 - n1;
        for (int k = 0; k < warp; ++k)
            before += s_warp[k];
        if (before < want && want <= before + n0 + n1) {
            const bool second = want > before + n0;
            s_pick[0] = (uint32_t)(second ? b0 - 1 : b0);
            s_pick[1] = want - before - (second ? n0 : 0u);
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        want = s_pick[1];
        if (pass == 2)
            break;
        // the next pass counts the keys that share the bits found so far; its
        // histogram is the other buffer, cleared before the last cluster barrier
        uint32_t *const hn = hist[(pass + 1) & 1];
        const int nshift = pass == 0 ? 10 : 0;
        const uint32_t nmask = pass == 0 ? 2047u : 1023u;
        const int ms = shift;
        for (int t = lo + tid; t - tid < hi; t += kSelThr) {
            const bool mid = t < hi && t >= mid0 && t < mid1;
            const uint32_t key = mid ? key_of(t) : 0u;
            count_key(hn, (key >> nshift) & nmask, mid && (key >> ms) == (prefix >> ms), lane);
        }
        if (pass == 0) {
            // pass 2 counts into hist[0] again: clear it once every CTA has read it
            cl.sync();
            for (int b = tid; b < kBins; b += kSelThr)
                hist[0][b] = 0u;
            __syncthreads();
        }
    }
    const uint32_t thr = any ? prefix : 0xFFFFFFFFu;  // no key is all ones
    const uint32_t ties = any ? want : 0u;            // keys at the threshold that are kept
    // kept: outside the middle, above the threshold, or one of the first `ties` at it
    const int span = chunk / kSelWarps;  // a multiple of 32
    const int w0 = min(lo + warp * span, hi), w1 = min(w0 + span, hi);
    uint32_t gt = 0, eq = 0;
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        const bool in = t < w1;
        const bool mid = in && t >= mid0 && t < mid1;
        const uint32_t key = mid ? key_of(t) : 0u;
        gt += __popc(__ballot_sync(kFull, (in && !mid) || (mid && key > thr)));
        eq += __popc(__ballot_sync(kFull, mid && key == thr));
    }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int k = 0; k < kSelWarps; ++k) {
            g += s_gt[k];
            e += s_eq[k];
        }
        s_cnt[0] = g;
        s_cnt[1] = e;
    }
    cl.sync();
    uint32_t gb = 0, eb = 0;  // kept above and ties before this warp's span
    for (int r = 0; r < rank; ++r) {
        const uint32_t *o = cl.map_shared_rank(s_cnt, r);
        gb += o[0];
        eb += o[1];
    }
    for (int k = 0; k < warp; ++k) {
        gb += s_gt[k];
        eb += s_eq[k];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int t = w0 + lane; t - lane < w1; t += 32) {
        const bool in = t < w1;
        const bool mid = in && t >= mid0 && t < mid1;
        const uint32_t key = mid ? key_of(t) : 0u;
        const bool up = (in && !mid) || (mid && key > thr), tie = mid && key == thr;
        const uint32_t bu = __ballot_sync(kFull, up), bt = __ballot_sync(kFull, tie);
        const uint32_t e = eb + __popc(bt & below);
        if (up || (tie && e < ties)) {
            const uint32_t p = gb + __popc(bu & below) + min(e, ties);
            kept[p] = t;
            if (mass_out)
                mass_out[p] = __ldg(mass + t);
        }
        gb += __popc(bu);
        eb += __popc(bt);
    }
    cl.sync();  // no CTA leaves while others read its shared memory
}

// HOLD: 16-byte pieces of rows that a thread keeps in registers. The three
// dependent look-ups of a row (kept slot, block, data) are made for all HOLD
// rows at a time.
template <int D, int WARPS, int HOLD>
__global__ void __launch_bounds__(kMoveThreads) cache_evict_move_kernel(const __grid_constant__ EvictArgs a)
{
    constexpr int UNITS = kMoveThreads / (32 * WARPS);
    constexpr int TPR = D / 16;             // threads per row (16 codes each)
    constexpr int RPP = 32 * WARPS / TPR;   // rows per pass
    __shared__ float s_top[kMoveThreads / 32];
    const View &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ut = tid % (32 * WARPS);
    const long long u = (long long)blockIdx.x * UNITS + warp / WARPS;
    if (u >= (long long)c.bs * c.H * a.pages * 2)
        return;
    const bool is_v = u & 1;
    long long y = u >> 1;
    const int b = (int)(y % a.pages);
    y /= a.pages;  // (request, head)
    const int i = (int)(y / c.H), h = (int)(y - (long long)i * c.H);
    const int ctx = min((long long)clamp_ctx(c, i, false), a.width);
    const int len = min(ctx, a.keep);
    const int p0 = b * c.P, n = min(c.P, len - p0);
    if (n <= 0) {
        griddep_wait();  // all CTAs wait: this grid must not end before the selection does
        return;
    }
    const int dpage = __ldg(a.new_bt + (long long)i * a.new_w + b);
    if (dpage < 0 || (long long)dpage >= c.nb) {
        if (ut == 0)
            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
        griddep_wait();
        return;
    }
    griddep_wait();  // the kept lists are complete
    const uint8_t *const pool = is_v ? c.v : c.k;
    float *const scale = is_v ? c.vs : c.ks;
    const int32_t *const kept = a.kept + y * a.keep + p0;
    const int col = (ut % TPR) * 16, r0 = ut / TPR;
    float top = 0.0f;
    uint4 x[HOLD];
    float s[HOLD];
    // rows rb + k RPP of the new block: codes and scales (zeros for none)
    auto fetch = [&](int rb) {
        int t[HOLD], page[HOLD];
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            t[k] = rb + k * RPP < n ? __ldcg(kept + rb + k * RPP) : -1;
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            page[k] = t[k] >= 0 ? __ldg(c.bt + (long long)i * c.W + c.page_of(t[k])) : 0;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const bool ok = t[k] >= 0 && page[k] >= 0 && (long long)page[k] < c.nb;
            bad |= t[k] >= 0 && !ok;
            x[k] = make_uint4(0, 0, 0, 0);
            s[k] = 0.0f;
            if (ok) {
                const long long phys = (long long)page[k] * c.H + h;
                x[k] = __ldg(reinterpret_cast<const uint4 *>(
                    pool + (phys * c.P + (t[k] - c.page_of(t[k]) * c.P)) * D + col));
                s[k] = __ldg(scale + phys);
            }
        }
        if (bad)
            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
    };
    auto widen = [&]() {
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const uint32_t e[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                float f0, f1, f2, f3;
                e4m3x2_to_f32x2(e[z] & 0xFFFFu, f0, f1);
                e4m3x2_to_f32x2(e[z] >> 16, f2, f3);
                const float m = fmaxf(fmaxf(fabsf(f0), fabsf(f1)), fmaxf(fabsf(f2), fabsf(f3))) * s[k];
                top = fmaxf(top, m < INFINITY ? m : 0.0f);
            }
        }
    };
    // blocks longer than the registers hold are read twice: for the maximum, and to move
    const bool once = n <= HOLD * RPP;
    for (int rb = r0; rb < n; rb += HOLD * RPP) {
        fetch(rb);
        widen();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if constexpr (WARPS > 1) {
        if (lane == 0)
            s_top[warp] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WARPS; ++k)
            top = fmaxf(top, s_top[k]);
    }
    const float sn = pow2_scale(top), inv = 1.0f / sn;  // a power of two: exact
    const long long dphys = (long long)dpage * c.H + h;
    uint8_t *const dst = (is_v ? c.v : c.k) + dphys * c.P * D;
    if (ut == 0)
        scale[dphys] = sn;
    for (int rb = r0; rb < n; rb += HOLD * RPP) {
        if (!once)
            fetch(rb);
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            const int r = rb + k * RPP;
            if (r >= n)
                break;
            const uint32_t e[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t o[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                float f0, f1, f2, f3;
                e4m3x2_to_f32x2(e[z] & 0xFFFFu, f0, f1);
                e4m3x2_to_f32x2(e[z] >> 16, f2, f3);
                o[z] = f32x4_to_e4m3x4(f0 * s[k] * inv, f1 * s[k] * inv, f2 * s[k] * inv, f3 * s[k] * inv);
            }
            *reinterpret_cast<uint4 *>(dst + (long long)r * D + col) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <int D>
static cudaError_t launch_move(const EvictArgs &a, long long pairs, cudaStream_t st)
{
    // a warp's pass covers 512 / D rows: up to 4 passes of one warp, else of four warps
    const int P = a.c.P, pass = 512 / D;
    const bool one = P <= 4 * pass;
    const long long units = pairs * a.pages * 2;
    const long long grid = one ? (units + 3) / 4 : units;
    if (grid > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    const dim3 g((unsigned)grid);
    if (one)
        return launch_early(cache_evict_move_kernel<D, 1, 4>, g, kMoveThreads, 0, true, st, a);
    return P <= 16 * pass ? launch_early(cache_evict_move_kernel<D, 4, 4>, g, kMoveThreads, 0, true, st, a)
                          : launch_early(cache_evict_move_kernel<D, 4, 8>, g, kMoveThreads, 0, true, st, a);
}

cudaError_t launch_evict(const EvictCall &q, int sms, cudaStream_t st)
{
    EvictArgs a{};
    a.c = q.c;
    a.mass = q.mass;
    a.width = q.width;
    a.keep = q.keep;
    a.sinks = q.sinks;
    a.recent = q.recent;
    a.new_bt = q.new_bt;
    a.new_w = q.new_w;
    a.kept = q.kept;
    a.lens_out = q.lens_out;
    a.mass_out = q.mass_out;
    // new blocks that a request can fill: of `keep` tokens, or of its longest context
    // (keep may be up to 2^31 - 1)
    const long long most = std::min({(long long)q.keep, (long long)q.c.P * q.c.W, (long long)kMaxContext});
    a.pages = (int)((most + q.c.P - 1) / q.c.P);
    const long long pairs = (long long)q.c.bs * q.c.H;
    // CTAs per cluster: enough for the longest row's keys to stay in shared
    // memory, and (few pairs) enough to use the GPU; 8 is the portable most
    int cs = 1;
    while (cs < 8 && (q.width > (long long)cs * kKeysMax ||
                      (pairs * cs <= sms && q.width > (long long)cs * 4096)))
        cs *= 2;
    a.cs = cs;
    // more CTAs than SMs: long requests start first (selection of the batch above: 55 us
    // instead of 70), unless ranking them would take longer than it gains
    a.ranked = pairs * cs > sms && q.c.bs <= 128;
    const long long chunk = ((std::min<long long>(q.width, 0x7FFFFF00ll) + cs - 1) / cs + 1023) & ~1023ll;
    a.key_cap = (int)std::min<long long>(chunk, kKeysMax);
    const int smem = a.key_cap * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(cache_evict_select_kernel, kKeysMax * 4, done);
    if (e != cudaSuccess)
        return e;
    if (pairs * cs > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.gridDim = dim3((unsigned)(pairs * cs));
    cfg.blockDim = dim3(kSelThr);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, cache_evict_select_kernel, a);
    if (e != cudaSuccess)
        return e;
    return q.c.D == 128 ? launch_move<128>(a, pairs, st) : launch_move<64>(a, pairs, st);
}

}  // namespace cache
}  // namespace pmqa
