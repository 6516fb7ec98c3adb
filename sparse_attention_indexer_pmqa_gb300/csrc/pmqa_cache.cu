// pmqa_cache.cu -- C ABI of the operators on the paged 8-bit K/V cache
// (include/pmqa.h): argument checks, the device view of a problem, the choice
// of kernels. No allocation, no synchronisation, no state between calls.
#include <algorithm>
#include <cmath>

#include "pmqa_cache_host.cuh"

using namespace pmqa;
using namespace pmqa::cache;

namespace {

enum { kNeedRows = 1, kNeedValues = 2 };

// Sizes first, then what is out of the kernels' range, then (when there is
// anything to do) the pointers.
int check(const pmqa_cache_problem *p, int need, const void *ws, size_t ws_bytes)
{
    if (!p)
        return PMQA_ERR_INVALID_ARG;
    if (p->bs < 0 || p->kv_heads < 1 || p->head_dim < 1 || p->block_size < 1 ||
        p->max_blocks_per_seq < 1 || p->num_blocks < 1)
        return PMQA_ERR_INVALID_ARG;
    if ((need & kNeedRows) && (p->rows < 0 || p->max_rows < 1))
        return PMQA_ERR_INVALID_ARG;
    if ((p->head_dim != 64 && p->head_dim != 128) || p->block_size > kMaxBlock || p->kv_heads > 65535)
        return PMQA_ERR_UNSUPPORTED;
    // rows of a pool are counted in 32 bits
    if (p->num_blocks > 0xFFFFFFFEll / ((long long)p->kv_heads * p->block_size))
        return PMQA_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256))
        return PMQA_ERR_INVALID_ARG;
    if (ws_bytes < kWorkspace)
        return PMQA_ERR_WORKSPACE;
    if (p->bs == 0)
        return PMQA_OK;
    if (missing(p->k_cache, 16) || missing(p->k_scale, 4) || missing(p->block_tables, 4) ||
        missing(p->context_lens, 4))
        return PMQA_ERR_INVALID_ARG;
    if ((need & kNeedValues) && (missing(p->v_cache, 16) || missing(p->v_scale, 4)))
        return PMQA_ERR_INVALID_ARG;
    if ((need & kNeedRows) && missing(p->row_begin, 4))
        return PMQA_ERR_INVALID_ARG;
    return PMQA_OK;
}

// heads query heads over the cache's kv heads
int check_heads(const pmqa_cache_problem *p, int32_t heads, float sm_scale)
{
    if (heads < 1 || heads % p->kv_heads != 0 || !std::isfinite(sm_scale * kLog2e))
        return PMQA_ERR_INVALID_ARG;
    if (heads / p->kv_heads > kMaxGroup || (long long)p->max_rows * heads > 0x7FFFFFFFll)
        return PMQA_ERR_UNSUPPORTED;
    return PMQA_OK;
}

View view(const pmqa_cache_problem *p, void *ws)
{
    View c{};
    c.k = static_cast<uint8_t *>(p->k_cache);
    c.v = static_cast<uint8_t *>(p->v_cache);
    c.ks = p->k_scale;
    c.vs = p->v_scale;
    c.bt = p->block_tables;
    c.ctx = p->context_lens;
    c.row_begin = p->row_begin;
    c.bs = p->bs;
    c.H = p->kv_heads;
    c.D = p->head_dim;
    c.P = p->block_size;
    c.W = p->max_blocks_per_seq;
    c.rows = p->rows;
    c.max_rows = p->max_rows;
    c.p_inv = c.P == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / (uint32_t)c.P);
    c.nb = p->num_blocks;
    c.status = static_cast<uint32_t *>(ws);
    return c;
}

}  // namespace

extern "C" size_t pmqa_cache_workspace_bytes(void) { return kWorkspace; }

extern "C" int pmqa_cache_append(const pmqa_cache_problem *p, const void *k, const void *v, void *ws,
                                 size_t ws_bytes, pmqa_stream_t stream)
{
    int rc = check(p, kNeedRows | kNeedValues, ws, ws_bytes);
    if (rc != PMQA_OK)
        return rc;
    if (p->bs == 0 || p->rows == 0)
        return PMQA_OK;
    if (missing(k, 16) || missing(v, 16))
        return PMQA_ERR_INVALID_ARG;
    if ((long long)p->rows / p->block_size + 2ll * p->bs > 0x7FFFFFFFll)
        return PMQA_ERR_UNSUPPORTED;
    return code_of(launch_append(view(p, ws), k, v, cuda(stream)));
}

extern "C" int pmqa_cache_attention(const pmqa_cache_problem *p, const void *q, int32_t heads,
                                    float sm_scale, void *out, float *lse, void *ws, size_t ws_bytes,
                                    pmqa_stream_t stream)
{
    int rc = check(p, kNeedRows | kNeedValues, ws, ws_bytes);
    if (rc == PMQA_OK)
        rc = check_heads(p, heads, sm_scale);
    if (rc != PMQA_OK)
        return rc;
    if (p->bs == 0 || p->rows == 0)
        return PMQA_OK;
    if (missing(q, 16) || missing(out, 16) || (lse && !aligned(lse, 4)))
        return PMQA_ERR_INVALID_ARG;
    int sms = 0;
    if ((rc = sm_count(&sms)) != PMQA_OK)
        return rc;
    AttnCall a{view(p, ws), q, out, lse, sm_scale, heads, static_cast<uint8_t *>(ws)};
    // requests with up to kShortRows packed rows split their context over the
    // GPU; longer ones keep the tensor cores busy with their rows
    const long long most = (long long)p->max_rows * (heads / p->kv_heads);
    cudaError_t e = cudaSuccess;
    // fewer row blocks than SMs: their contexts are cut too
    const int ctas = std::min(sms, kMaxParts);
    const long long blocks = (long long)p->rows * (heads / p->kv_heads) / kPromptRows * p->kv_heads;
    const int parts = most > kShortRows && blocks < ctas ? ctas : 0;
    if (most > kShortRows)
        e = launch_attn_prompt(a, kShortRows + 1, parts, cuda(stream));
    if (e == cudaSuccess && heads / p->kv_heads <= kShortRows)
        e = launch_attn_rows(a, 1, kShortRows, sms, most > kShortRows, cuda(stream));
    if (e == cudaSuccess && parts > 0)
        e = launch_attn_join(a, parts, cuda(stream));
    return code_of(e);
}

extern "C" int pmqa_cache_weigh(const pmqa_cache_problem *p, const void *q, int32_t heads,
                                float sm_scale, const float *lse, const float *mass_in,
                                float *mass_out, int64_t mass_width, void *ws, size_t ws_bytes,
                                pmqa_stream_t stream)
{
    int rc = check(p, kNeedRows, ws, ws_bytes);
    if (rc == PMQA_OK)
        rc = check_heads(p, heads, sm_scale);
    if (rc != PMQA_OK)
        return rc;
    if (mass_width < 1)
        return PMQA_ERR_INVALID_ARG;
    if (p->bs == 0)
        return PMQA_OK;
    if (missing(mass_out, 4) || (mass_in && !aligned(mass_in, 4)) ||
        (p->rows > 0 && (missing(q, 16) || missing(lse, 4))))
        return PMQA_ERR_INVALID_ARG;
    // in place or apart: shifted, sums would be read as other tokens' earlier masses
    const long long n = 4ll * p->bs * p->kv_heads * mass_width;
    if (mass_in && mass_in != mass_out && overlap(mass_in, n, mass_out, n))
        return PMQA_ERR_INVALID_ARG;
    int sms = 0;
    if ((rc = sm_count(&sms)) != PMQA_OK)
        return rc;
    WeighCall a{view(p, ws), q, lse, mass_in, mass_out, mass_width, sm_scale, heads};
    const long long most = (long long)p->max_rows * (heads / p->kv_heads);
    cudaError_t e = cudaSuccess;
    if (most > kShortRows)
        e = launch_weigh_window(a, kShortRows + 1, sms, cuda(stream));
    if (e == cudaSuccess)
        e = launch_weigh_rows(a, 0, kShortRows, sms, most > kShortRows, cuda(stream));
    return code_of(e);
}

extern "C" int pmqa_cache_evict(const pmqa_cache_problem *p, const float *mass, int64_t mass_width,
                                int32_t keep, int32_t sinks, int32_t recent,
                                const int32_t *new_tables, int32_t new_blocks_per_seq, int32_t *kept,
                                int32_t *lens_out, float *mass_out, void *ws, size_t ws_bytes,
                                pmqa_stream_t stream)
{
    int rc = check(p, kNeedValues, ws, ws_bytes);
    if (rc != PMQA_OK)
        return rc;
    if (mass_width < 1 || keep < 1 || sinks < 0 || recent < 0 || (long long)sinks + recent > keep ||
        new_blocks_per_seq < 1 || (long long)new_blocks_per_seq * p->block_size < keep)
        return PMQA_ERR_INVALID_ARG;
    if (p->bs == 0)
        return PMQA_OK;
    if (missing(mass, 4) || missing(new_tables, 4) || missing(kept, 4) || missing(lens_out, 4) ||
        (mass_out && !aligned(mass_out, 4)))
        return PMQA_ERR_INVALID_ARG;
    // lengths and masses are read while the new ones are written
    const long long n = 4ll * p->bs * p->kv_heads * mass_width;
    if (overlap(lens_out, 4ll * p->bs, p->context_lens, 4ll * p->bs) ||
        (mass_out && overlap(mass_out, n, mass, n)))
        return PMQA_ERR_INVALID_ARG;
    int sms = 0;
    if ((rc = sm_count(&sms)) != PMQA_OK)
        return rc;
    EvictCall a{view(p, ws), mass, mass_width, keep, sinks, recent, new_tables, new_blocks_per_seq,
                kept, lens_out, mass_out};
    return code_of(launch_evict(a, sms, cuda(stream)));
}
