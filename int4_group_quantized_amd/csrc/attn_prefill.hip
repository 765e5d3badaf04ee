// Attention of prompt tokens over the paged cache: the kernels of attn_prefill.hpp
// for the cache's widths.
#include "attn_prefill.hpp"

namespace q4 {

int64_t attn_prefill_workspace(int64_t tokens, int64_t count, int heads, int kv_heads, int dim, int dim_v,
                               int64_t max_length, int64_t max_new) {
    const int splits = prefill_plan(tokens, count, heads, kv_heads, dim, dim_v, max_length, max_new).splits;
    // The counters of the decode call come first, so that both can share one.
    return splits == 1 ? 0 : ((int64_t)splits * tokens * heads * (dim_v + 2) + kAttnCounters) * (int64_t)sizeof(float);
}

hipError_t launch_attn_prefill(const AttnArgs& a, const DeviceInfo& dev, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_prefill_attn<64>(a, dev, st);
        case 96: return launch_prefill_attn<96>(a, dev, st);
        case 128: return launch_prefill_attn<128>(a, dev, st);
        case 192: return launch_prefill_attn<192>(a, dev, st);
        case 256: return launch_prefill_attn<256>(a, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
