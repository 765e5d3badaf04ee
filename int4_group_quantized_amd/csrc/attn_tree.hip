// Attention of drafted tokens over the paged cache (gfx950): the prompt kernel
// (attn_prefill.hpp) with masks, which say what the last positions of a sequence see
// of each other.
//
// A cached position costs 4 * dim bytes per kv head for every 128 rows (a tree's tokens
// times the heads of the group); the workgroups of further rows find it in L2 (16 trees of
// 64 tokens, 256 rows each, fetch 1.08 GB of a cache of 1.07).  Few rows are bound by
// latency, many by the matrix cores and the softmax, as prompts are.  What a row sees of
// a tile is one 64-bit word (seen_word), formed only for tiles that hold drafted
// positions or a window's edge.
//
// A kernel of its own after the decode call's, every wave with keys and values of its
// own straight from memory into registers, for 16, 32 or 64 rows, was slower in all but
// the largest calls: 16 sequences of 8 tokens of 16 heads (4 kv heads of 128) on up
// to 4,000 positions 36 us, 21 here; one of 16 tokens on 8,000 24 and 16; 16 of 64 on
// 16,384 (32 heads on 8) 574 and 352; 64 sequences of 16 tokens on 8,192 196 and 206.
#include "attn_prefill.hpp"

namespace q4 {

hipError_t launch_attn_tree(const AttnArgs& a, const DeviceInfo& dev, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_prefill_attn<64, 64, true>(a, dev, st);
        case 96: return launch_prefill_attn<96, 96, true>(a, dev, st);
        case 128: return launch_prefill_attn<128, 128, true>(a, dev, st);
        case 192: return launch_prefill_attn<192, 192, true>(a, dev, st);
        case 256: return launch_prefill_attn<256, 256, true>(a, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
