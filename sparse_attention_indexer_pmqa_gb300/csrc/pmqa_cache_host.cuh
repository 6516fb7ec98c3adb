// pmqa_cache_host.cuh -- host side of the cache operators: the calls that the
// C ABI hands to the kernels' translation units.
#pragma once

#include <atomic>

#include "pmqa_cache.cuh"

namespace pmqa {
namespace cache {

// The kernel's shared-memory limit, raised once per device and kernel (a
// property of the loaded code; setting it costs several microseconds of host
// time, more than the launch). `done` is one word per kernel, a bit per device.
template <typename K>
inline cudaError_t allow_smem(K *kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (bit & done.load(std::memory_order_relaxed))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A launch that, where `early`, may start once every CTA of the kernel before it
// has started: it waits for that kernel (griddep_wait) before it needs what it
// wrote, and in any case before it ends.
template <typename A>
inline cudaError_t launch_early(void (*kernel)(A), dim3 grid, int threads, size_t smem, bool early,
                                cudaStream_t st, const A &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

constexpr int kShortRows = 32;  // packed rows (rows * group) of the short-row kernels

// Workspace: status | open contexts, one per CTA | (m, l) and O of two parts per CTA,
// 32 rows of 128 (or 16 rows and more CTAs) | the same of the many-row kernel, one
// part of 256 rows per CTA
constexpr size_t kPartRows = (size_t)2 * kMaxWide * 32;
static_assert(kPartRows >= (size_t)2 * kMaxCtas * 16, "parts of 16 rows");
constexpr size_t kWsMeta = kStatusBytes;
constexpr size_t kWsMl = kWsMeta + kMaxCtas * 16;
constexpr size_t kWsPart = kWsMl + kPartRows * 2 * 4;
constexpr size_t kWsPromptMeta = kWsPart + kPartRows * 128 * 4;
constexpr size_t kWsPromptMl = kWsPromptMeta + kMaxParts * 16;
constexpr size_t kWsPromptPart = kWsPromptMl + (size_t)kMaxParts * kPromptRows * 2 * 4;
constexpr size_t kWorkspace = kWsPromptPart + (size_t)kMaxParts * kPromptRows * 128 * 4;

struct AttnCall {
    View c;
    const void *q;
    void *out;
    float *lse;
    float sm_scale;
    int heads;
    uint8_t *ws;
};

struct WeighCall {
    View c;
    const void *q;
    const float *lse;
    const float *mass_in;
    float *mass_out;
    long long width;
    float sm_scale;
    int heads;
};

struct EvictCall {
    View c;
    const float *mass;
    long long width;
    int keep, sinks, recent;
    const int32_t *new_bt;  // [bs, new_w]
    int new_w;
    int32_t *kept;          // [bs, H, keep]
    int32_t *lens_out;      // [bs]
    float *mass_out;        // [bs, H, width] or null
};

cudaError_t launch_append(const View &c, const void *k, const void *v, cudaStream_t st);
cudaError_t launch_attn_rows(AttnCall &q, int least, int most, int sms, bool early, cudaStream_t st);
cudaError_t launch_attn_prompt(AttnCall &q, int least, int parts, cudaStream_t st);
cudaError_t launch_attn_join(AttnCall &q, int parts, cudaStream_t st);
cudaError_t launch_weigh_rows(const WeighCall &q, int least, int most, int sms, bool early, cudaStream_t st);
cudaError_t launch_weigh_window(const WeighCall &q, int least, int sms, cudaStream_t st);
cudaError_t launch_evict(const EvictCall &q, int sms, cudaStream_t st);

}  // namespace cache
}  // namespace pmqa
