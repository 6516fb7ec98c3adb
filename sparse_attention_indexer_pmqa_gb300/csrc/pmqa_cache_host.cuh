// pmqa_cache_host.cuh -- host side of the cache operators: the calls that the
// C ABI hands to the kernels' translation units.
#pragma once

#include "pmqa_cache.cuh"

namespace pmqa {
namespace cache {

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
cudaError_t launch_attn_rows(AttnCall &q, int least, int most, int sms, cudaStream_t st);
cudaError_t launch_weigh_rows(const WeighCall &q, int least, int most, int sms, cudaStream_t st);
cudaError_t launch_evict(const EvictCall &q, int sms, cudaStream_t st);

}  // namespace cache
}  // namespace pmqa
