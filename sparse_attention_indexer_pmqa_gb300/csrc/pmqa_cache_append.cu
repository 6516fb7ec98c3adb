// pmqa_cache_append.cu -- the write into the paged 8-bit K/V cache: a step's new
// keys and values, quantised with one power-of-two scale per block and kv head.
//
// A block's scale is e(a) = 2^ceil(log2(a / 448)) of the largest finite new
// value a, or the scale that it already has where that is larger and the block
// holds earlier tokens; when the scale grows, the earlier codes are rounded
// again to the new one. Power-of-two scales make that rounding exact but for
// values that fall below e4m3's normal range, and make x / s exact.
//
// Bound by HBM for prompts (2 D bytes read and D written per token, head and
// pool) and by latency for single tokens. A unit (block, head, pool) belongs to
// one warp, or to four where blocks receive more than a warp can keep in
// registers: the rows are read once, reduced to their largest value, and
// written from the registers. 15730 new tokens of 8 kv heads take 20.5 us in one cold
// launch (97 MB, 70 % of the measured copy rate) and 17.4 us back to back, 64 single
// tokens 2.6 us back to back. Units of a request are found by a 32-way search over
// row_begin, so that ragged batches need no list made by the host.
#include <algorithm>

#include "pmqa_cache_host.cuh"

namespace pmqa {
namespace cache {

constexpr int kAppendThreads = 128;
constexpr int kHold = 8;  // 16-byte pieces of new rows that a thread keeps in registers

struct AppendArgs {
    View c;
    const uint16_t *k, *v;  // bf16 [rows, H, D]
    int slots;              // block slots over all requests (upper bound)
    int single;             // every request has at most one row: slot = request
};

// First block slot of request i: row_begin[i] / P + 2 i leaves room for the at
// most floor(n / P) + 2 blocks that n rows touch, whatever the first offset.
__device__ __forceinline__ long long first_slot(const View &c, int i)
{
    return (long long)(max(__ldg(c.row_begin + i), 0) / c.P) + 2ll * i;
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a < INFINITY ? a : 0.0f;  // NaN and infinities do not set the scale
}

template <int D, int WARPS>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int UNITS = kAppendThreads / (32 * WARPS);  // units per CTA
    constexpr int TPR = D / 8;                            // threads per row (8 values each)
    constexpr int RPP = 32 * WARPS / TPR;                 // rows per pass
    __shared__ float s_top[kAppendThreads / 32];
    const View &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ut = tid % (32 * WARPS);  // thread within the unit
    // where row_begin falls, the search below may pass a request over: the last CTA,
    // whose slots are seldom in use, reports for all of them
    if (!a.single && blockIdx.x == gridDim.x - 1)
        report_requests(c);
    const long long u = (long long)blockIdx.x * UNITS + warp / WARPS;
    const long long n_units = (long long)a.slots * c.H * 2;
    if (u >= n_units)
        return;
    const bool is_v = u & 1;
    const long long sh = u >> 1;
    const long long slot = sh / c.H;
    const int h = (int)(sh - slot * c.H);
    int i;
    long long kth = 0;
    if (a.single) {
        i = (int)slot;
    } else {
        int lo = 0, len = c.bs;
        while (len > 1) {
            const int step = (len + 31) >> 5;
            const int at = lo + lane * step;
            const uint32_t le = __ballot_sync(kFull, lane * step < len && first_slot(c, at) <= slot);
            const int k = max(__popc(le) - 1, 0);
            lo += k * step;
            len = min(step, len - k * step);
        }
        i = lo;
        kth = slot - first_slot(c, i);
    }
    const Request q = load_request(c, i, u == 2 * slot * c.H && ut == 0);
    if (q.n == 0 || kth < 0)
        return;
    // A row's slot comes from the lengths as they are given: rows that the arrays or
    // the table have no place for are dropped, and no other row moves over tokens
    // that are already there.
    const int rb = __ldg(c.row_begin + i);
    const long long given = (long long)__ldg(c.row_begin + i + 1) - rb;
    const long long first = (long long)__ldg(c.ctx + i) - given + (q.r0 - (long long)rb);  // slot of row r0
    const long long cap = min((long long)c.P * c.W, (long long)kMaxContext);
    const long long from = max(first, 0ll), to = min(first + q.n, cap);  // slots written
    if (first < 0 && ut == 0)
        atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_CONTEXT);  // rows before slot 0 are not kept
    if (from >= to)
        return;
    const long long bl = c.page_of((int)from) + kth;
    if (bl * c.P >= to)
        return;
    const int b = (int)bl, lo = (int)max(from, bl * c.P);
    const int hi = (int)min(to, (bl + 1) * c.P);
    const int held = lo - b * c.P, nrow = hi - lo;
    const int page = __ldg(c.bt + (long long)i * c.W + b);
    if (page < 0 || (long long)page >= c.nb) {
        if (ut == 0)
            atomicOr(c.status, (uint32_t)PMQA_DEV_BAD_BLOCK_ID);
        return;
    }
    const long long phys = (long long)page * c.H + h;
    float *const scale = (is_v ? c.vs : c.ks) + phys;
    uint8_t *const dst = (is_v ? c.v : c.k) + phys * c.P * D;
    const uint16_t *const src = (is_v ? a.v : a.k) + ((long long)(q.r0 + lo - first) * c.H + h) * D;
    const long long pitch = (long long)c.H * D;  // values between rows
    const float s_old = held > 0 ? *scale : 0.0f;

    const int col = (ut % TPR) * 8, r0 = ut / TPR;
    uint4 x[kHold];
    // the largest |value|, as the larger of two bf16 patterns without their signs
    uint32_t big = 0;
    auto widen = [&](const uint4 &w) {
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                     __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int r = r0 + k * RPP;
        x[k] = r < nrow ? __ldcs(reinterpret_cast<const uint4 *>(src + r * pitch + col)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kHold; ++k)
        widen(x[k]);
    // rows beyond what the registers hold: read here for the maximum, and again below
    for (int r = r0 + kHold * RPP; r < nrow; r += RPP)
        widen(__ldg(reinterpret_cast<const uint4 *>(src + r * pitch + col)));
    float top = fmaxf(__uint_as_float(big << 16), __uint_as_float(big & 0xFFFF0000u));
    if (big << 16 >= 0x7F800000u || big >= 0x7F800000u) {
        // a NaN or an infinity among them: the largest of the others (rare)
        top = 0.0f;
        for (int r = r0; r < nrow; r += RPP) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + r * pitch + col));
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int z = 0; z < 4; ++z)
                top = fmaxf(top, fmaxf(finite_abs(__uint_as_float(e[z] << 16)),
                                       finite_abs(__uint_as_float(e[z] & 0xFFFF0000u))));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if constexpr (WARPS > 1) {
        if (lane == 0)
            s_top[warp] = top;
        __syncthreads();  // also: every thread has read the old scale
#pragma unroll
        for (int k = 0; k < WARPS; ++k)
            top = fmaxf(top, s_top[k]);
    } else {
        __syncwarp();  // every lane has read the old scale
    }
    float s = pow2_scale(top);
    if (held > 0)
        s = fmaxf(s, s_old);
    if (ut == 0 && !(held > 0 && s == s_old))
        *scale = s;
    if (held > 0 && s != s_old) {
        // s is a power of two here: 1 / s is exact
        const float inv = 1.0f / s;
        for (int w = ut; w < held * (D / 4); w += 32 * WARPS) {
            uint32_t *p = reinterpret_cast<uint32_t *>(dst) + w;
            const uint32_t old = *p;
            float f[4];
            e4m3x2_to_f32x2(old & 0xFFFFu, f[0], f[1]);
            e4m3x2_to_f32x2(old >> 16, f[2], f[3]);
#pragma unroll
            for (int z = 0; z < 4; ++z)
                f[z] = f[z] * s_old * inv;
            *p = f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]);
        }
    }
    const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    const float inv = 1.0f / s;
    auto put = [&](int r, const uint4 &w) {
        const uint32_t e[4] = {w.x, w.y, w.z, w.w};
        float f[8];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            f[2 * z] = __uint_as_float(e[z] << 16);
            f[2 * z + 1] = __uint_as_float(e[z] & 0xFFFF0000u);
        }
        if (pow2) {
#pragma unroll
            for (int z = 0; z < 8; z += 2)
                fmul2(f[z], f[z + 1], f[z], f[z + 1], inv, inv);
        } else {
            // a scale that append did not make: the nearest code of x / s itself
#pragma unroll
            for (int z = 0; z < 8; ++z)
                f[z] = __fdiv_rn(f[z], s);
        }
        *reinterpret_cast<uint2 *>(dst + (long long)(held + r) * D + col) =
            make_uint2(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]));
    };
#pragma unroll
    for (int k = 0; k < kHold; ++k)
        if (r0 + k * RPP < nrow)
            put(r0 + k * RPP, x[k]);
    for (int r = r0 + kHold * RPP; r < nrow; r += RPP)
        put(r, __ldg(reinterpret_cast<const uint4 *>(src + r * pitch + col)));
}

template <int D>
static cudaError_t launch(const AppendArgs &a, cudaStream_t st)
{
    // one warp holds kHold * 256 / D rows; four warps share blocks that get more
    const bool wide = std::min(a.c.P, a.c.max_rows) > kHold * 256 / D;
    const long long units = (long long)a.slots * a.c.H * 2;
    const long long grid = wide ? units : (units + 3) / 4;
    if (grid > 0x7FFFFFFFll)
        return cudaErrorInvalidConfiguration;
    if (wide)
        cache_append_kernel<D, 4><<<(unsigned)grid, kAppendThreads, 0, st>>>(a);
    else
        cache_append_kernel<D, 1><<<(unsigned)grid, kAppendThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_append(const View &c, const void *k, const void *v, cudaStream_t st)
{
    AppendArgs a{};
    a.c = c;
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.single = c.max_rows == 1;
    a.slots = a.single ? c.bs : c.rows / c.P + 2 * c.bs;
    return c.D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace cache
}  // namespace pmqa
