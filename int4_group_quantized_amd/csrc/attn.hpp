// Paged key-value cache shared by the append and attention kernels: host-side
// launch arguments and the device-side addressing.  Arguments reaching the
// launchers have been validated by the C ABI.
#pragma once

#include "launch.hpp"
#include "q4_device.hpp"

namespace q4 {

// Attention's kernels treat 64 positions as one tile.
constexpr int kTileKeys = 64;
// Counters at the start of an attention workspace.
constexpr int kAttnCounters = 1024;

struct KvCache {
    uint16_t* k;        // [pages][kv_heads][page][dim]
    uint16_t* v;        // [pages][kv_heads][dim][page]
    const int* table;   // [sequences][cols]
    long k_stride;      // elements from page to page
    long v_stride;
    int pages;
    int sequences;
    int cols;
    int kv_heads;
    int dim;
    int shift;          // log2(page)
};

struct AppendArgs {
    const float* qkv;
    long ld;
    int tokens;
    int heads;
    KvCache c;
    const int* seq;        // or NULL: token t is of sequence t
    const int* positions;
    const float* inv_freq;
    int rot;
    int interleaved;
    float mscale;
    const uint16_t* q_norm;  // or NULL
    const uint16_t* k_norm;  // or NULL
    float eps;
    uint16_t* q;
};

struct AttnArgs {
    const uint16_t* q;
    KvCache c;
    const int* lengths;
    int max_length;
    int rows;              // decode: batch; prompt: tokens
    int heads;
    int group;             // heads per kv head
    float scale;
    float softcap;         // 0: none
    int window;            // 0: none
    const float* slopes;   // or NULL
    uint16_t* out;
    float* workspace;
    // prompt only
    const int* q_starts;
    const int* prefix;     // or NULL
    int count;             // sequences
    int tile;              // tokens of a workgroup
    float inv_tile;        // 1 / tile
    int splits;            // parts that the positions are cut into
    float inv_group;       // 1 / group
    int images;            // tiles that fit into the launch's LDS, 2 to 4
};

// Widths the attention kernels are compiled for.
inline bool attn_dim_supported(int dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 192 || dim == 256; }

hipError_t launch_rope_append(const AppendArgs& a, hipStream_t st);
hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t st);
int64_t attn_decode_workspace(int64_t batch, int heads, int dim);
hipError_t launch_attn_prefill(const AttnArgs& a, const DeviceInfo& dev, hipStream_t st);
int64_t attn_prefill_workspace(int64_t tokens, int64_t count, int heads, int kv_heads, int dim, int64_t max_length);

// The table's page for a position of sequence `row`, or -1 when the page is
// absent.  pos must lie below cols << shift.
__device__ __forceinline__ int page_of(const KvCache& c, const int* __restrict__ row, int pos) {
    const int id = row[pos >> c.shift];
    return (unsigned)id < (unsigned)c.pages ? id : -1;
}

// Inclusive prefix sum over the wave's 64 lanes, and its last value.
struct LaneScan {
    int upto;
    int last;
};
__device__ __forceinline__ LaneScan lane_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 of a row to the next row, rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
    return {v, __builtin_amdgcn_readlane(v, 63)};
}

}  // namespace q4
