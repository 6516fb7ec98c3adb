// pmqa_latent_rows.cu -- the latent cache written, and the queries beside it:
// pmqa_latent_append.
//
// Per row one latent row (512 values, layer or RMS norm, and 64 rotary ones) of 576
// codes into the row's slot, and `heads` query rows of the same form. One scale for
// all: no value waits for another but in the key's norm. Bound by memory: 1728 bytes
// a query head. A warp takes four heads at a time, 16-byte loads of eight values a
// lane: eight for their latent values and one for their rotary ones, eight
// lanes a head. 15.7 k rows of 16 heads (462 MB): 79.7 us, 85 % of the copy rate.
#include <algorithm>

#include "pmqa_latent.cuh"
#include "pmqa_paged.cuh"

namespace pmqa {
namespace paged {

using mla::kDim;
using mla::kVDim;

constexpr int kPe = kDim - kVDim;
constexpr int kLatentThreads = 128;

struct LatentArgs {
    View c;
    Rotary r;
    Norm n;
    uint8_t *kv;
    const uint16_t *k_c, *k_pe, *q_c, *q_pe;
    uint8_t *q_out;
    long long c_row, pe_row, q_c_row, q_c_head, q_pe_row, q_pe_head;
    int heads;
    float kv_inv, q_inv;
};

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        x += __shfl_xor_sync(kFull, x, k);
    return x;
}

// Eight rotary values of a head, whose eight lanes are next to each other; the
// whole warp takes part.
__device__ __forceinline__ void rotate8(const Rotary &r, const Turn &turn, const uint4 &u, float (&y)[8])
{
    float other[8];
    unpack8(u, y);
    if (r.dim && !r.interleaved) {
        const int from = ((threadIdx.x & 31) + turn.partner) & 31;
        const uint4 p = make_uint4(__shfl_sync(kFull, u.x, from), __shfl_sync(kFull, u.y, from),
                                   __shfl_sync(kFull, u.z, from), __shfl_sync(kFull, u.w, from));
        unpack8(p, other);
    }
    turn.apply(r.interleaved, y, other);
}

__device__ __forceinline__ void write_key(const LatentArgs &a, const Turn &turn, long long r, uint32_t dst)
{
    const int lane = threadIdx.x & 31;
    const uint16_t *const src = a.k_c + r * a.c_row + 8 * lane;
    const uint4 u0 = load_input(src), u1 = load_input(src + 256);
    const uint4 up = lane < 8 ? load_input(a.k_pe + r * a.pe_row + 8 * lane) : make_uint4(0, 0, 0, 0);
    float y[2][8], pe[8];
    unpack8(u0, y[0]);
    unpack8(u1, y[1]);
    if (a.n.kind != PMQA_NORM_NONE) {
        if (a.n.kind == PMQA_NORM_LAYER) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                s += y[e >> 3][e & 7];
            const float mean = warp_sum(s) * (1.0f / kVDim);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                y[e >> 3][e & 7] -= mean;
        }
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            s += y[e >> 3][e & 7] * y[e >> 3][e & 7];
        const float f = rsqrtf(warp_sum(s) * (1.0f / kVDim) + a.n.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int d = (e >> 3) * 256 + 8 * lane + (e & 7);
            y[e >> 3][e & 7] = y[e >> 3][e & 7] * f * (a.n.weight ? __ldg(a.n.weight + d) : 1.0f) +
                               (a.n.bias ? __ldg(a.n.bias + d) : 0.0f);
        }
    }
    rotate8(a.r, turn, up, pe);
    if (dst == kNoRow)
        return;
    uint8_t *const p = a.kv + (unsigned long long)dst * kDim + 8 * lane;
    *reinterpret_cast<uint2 *>(p) = codes8(y[0], a.kv_inv);
    *reinterpret_cast<uint2 *>(p + 256) = codes8(y[1], a.kv_inv);
    if (lane < 8)
        *reinterpret_cast<uint2 *>(p + kVDim) = codes8(pe, a.kv_inv);
}

// Heads h0 .. h0 + 3 of row r.
__device__ __forceinline__ void write_queries(const LatentArgs &a, const Turn &turn, long long r, int h0)
{
    const int lane = threadIdx.x & 31, n = min(4, a.heads - h0);
    const uint16_t *const c = a.q_c + r * a.q_c_row + h0 * a.q_c_head + 8 * lane;
    uint8_t *const out = a.q_out + (r * a.heads + h0) * kDim + 8 * lane;
    uint4 u[8], up = make_uint4(0, 0, 0, 0);
    if (lane >> 3 < n)
        up = load_input(a.q_pe + r * a.q_pe_row + (h0 + (lane >> 3)) * a.q_pe_head + 8 * (lane & 7));
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k >> 1 < n)
            u[k] = load_input(c + (k >> 1) * a.q_c_head + (k & 1) * 256);
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k >> 1 < n) {
            unpack8(u[k], y);
            *reinterpret_cast<uint2 *>(out + (k >> 1) * kDim + (k & 1) * 256) = codes8(y, a.q_inv);
        }
    rotate8(a.r, turn, up, y);
    if (lane >> 3 < n)
        *reinterpret_cast<uint2 *>(a.q_out + (r * a.heads + h0 + (lane >> 3)) * kDim + kVDim + 8 * (lane & 7)) =
            codes8(y, a.q_inv);
}

// CTAs on an SM: many rows, five (with 76 bytes of spilled registers all the same 79.7 us for
// 15.7 k rows of 16 heads; four 82.0, six 84.4); few, where they do not fill the SMs, as many
// as come without spills (4.8 us for 128 rows by graph, 5.2).
template <int ROWS>
__global__ void __launch_bounds__(kLatentThreads, ROWS == 1 ? 4 : 5) latent_append_kernel(const __grid_constant__ LatentArgs a)
{
    __shared__ RowTable<ROWS, kPe> t;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * ROWS;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        cache::report_requests(a.c);
    load_turns(t, a.r);
    load_rows(t, a.c, a.r, row0, a.k_c != nullptr);
    const int groups = (a.heads + 3) / 4, all = groups + (a.k_c ? 1 : 0);
    int row_now = -1;
    Turn turn;
    for (int v = (int)blockIdx.y * (kLatentThreads / 32) + warp; v < ROWS * all; v += (int)gridDim.y * (kLatentThreads / 32)) {
        const int row = ROWS == 1 ? 0 : v / all, g = v - row * all;
        if (!t.place[row].valid)
            continue;
        if (row != row_now) {
            row_now = row;
            turn.load(a.r, t.cs[row], lane & 7);
        }
        if (g == groups)
            write_key(a, turn, row0 + row, t.place[row].row);
        else
            write_queries(a, turn, row0 + row, 4 * g);
    }
}

}  // namespace paged
}  // namespace pmqa

using namespace pmqa;
using namespace pmqa::paged;

extern "C" int pmqa_latent_append(const pmqa_paged_rows *p, void *kv_cache, const pmqa_latent_rows *x,
                                  const pmqa_norm *norm, const pmqa_rotary *rotary, void *ws, size_t ws_bytes,
                                  pmqa_stream_t stream)
{
    int rc = check_rows(p, true, ws, ws_bytes, cache::kStatusBytes);
    if (rc != PMQA_OK)
        return rc;
    LatentArgs a{};
    if (!x || (rc = check_norm(norm, &a.n)) != PMQA_OK || (rc = check_rotary(rotary, kPe, false, &a.r)) != PMQA_OK)
        return x ? rc : PMQA_ERR_INVALID_ARG;
    a.kv_inv = 1.0f / x->kv_scale;
    a.q_inv = 1.0f / x->q_scale;
    if ((x->c && !(std::isfinite(x->kv_scale) && std::isfinite(a.kv_inv))) ||
        (x->q_c && (x->heads < 1 || !(std::isfinite(x->q_scale) && std::isfinite(a.q_inv)))))
        return PMQA_ERR_INVALID_ARG;
    if (x->q_c && (x->heads > kMaxHeads || (long long)x->heads * p->rows > 0x7FFFFFFFll))
        return PMQA_ERR_UNSUPPORTED;
    if (p->bs == 0 || p->rows == 0 || (!x->c && !x->q_c))
        return PMQA_OK;
    if (x->c && (cache::missing(kv_cache, 8) || bad_rows(x->c, 16, p->rows, x->c_row) || bad_rows(x->k_pe, 16, p->rows, x->pe_row)))
        return PMQA_ERR_INVALID_ARG;
    if (x->q_c && (bad_rows(x->q_c, 16, p->rows, x->q_c_row, x->heads, x->q_c_head) ||
                   bad_rows(x->q_pe, 16, p->rows, x->q_pe_row, x->heads, x->q_pe_head) ||
                   cache::missing(x->q_out, 8)))
        return PMQA_ERR_INVALID_ARG;
    a.c = view(p, ws);
    a.kv = static_cast<uint8_t *>(kv_cache);
    a.k_c = static_cast<const uint16_t *>(x->c);
    a.k_pe = static_cast<const uint16_t *>(x->k_pe);
    a.q_c = static_cast<const uint16_t *>(x->q_c);
    a.q_pe = static_cast<const uint16_t *>(x->q_pe);
    a.q_out = static_cast<uint8_t *>(x->q_out);
    a.c_row = x->c_row;
    a.pe_row = x->pe_row;
    a.q_c_row = x->q_c_row;
    a.q_c_head = x->q_c_head;
    a.q_pe_row = x->q_pe_row;
    a.q_pe_head = x->q_pe_head;
    a.heads = x->q_c ? x->heads : 0;
    int sms = 0;
    if ((rc = cache::sm_count(&sms)) != PMQA_OK)
        return rc;
    const int rows = p->rows;
    const cudaStream_t st = cache::cuda(stream);
    if (rows >= 16 * sms)
        latent_append_kernel<4><<<(unsigned)((rows + 3ll) / 4), kLatentThreads, 0, st>>>(a);
    else  // few rows: a row's heads over several CTAs, up to 8 per SM
        latent_append_kernel<1><<<dim3(rows, std::max(1, std::min((a.heads + 15) / 16, 8 * sms / rows))), kLatentThreads, 0, st>>>(a);
    return cache::code_of(cudaGetLastError());
}
