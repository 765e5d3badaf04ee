// Attention of prompt tokens over keys and values expanded from latent rows: the
// kernels of attn_prefill.hpp with keys wider than values, by their rotary part.
//
// 4,096 tokens of 64 heads (192 and 128 columns, 344 GFLOP): 370 us, 930 TFLOP/s.  Two
// waves for 32 rows, as at dim 192 with values as wide, took 470.
#include "attn_prefill.hpp"

namespace q4 {

hipError_t launch_latent_prefill(const AttnArgs& a, const DeviceInfo& dev, hipStream_t st) {
    switch (a.c.dim) {
        case 128: return launch_prefill_attn<128, 64>(a, dev, st);
        case 192: return launch_prefill_attn<192, 128>(a, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
