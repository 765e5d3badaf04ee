// Latent attention: one row of latent + 64 halves per cached position, shared by
// all heads.  The first `latent` columns are key and value at once, the last 64 are
// the rotary part of the key.  Arguments reaching the launchers have been validated
// by the C ABI.
#pragma once

#include "attn_new.hpp"

namespace q4 {

constexpr int kRot = 64;  // rotary columns of a latent row

// As a cache without V, of one kv head: k the rows, dim = latent + 64.
inline bool latent_supported(int latent) { return latent == 128 || latent == 256 || latent == 512; }

struct LatentAppendArgs {
    const float* kv;         // [tokens][ld]: latent, rotary part
    long ld;
    int tokens;
    KvCache c;
    const int* seq;          // or NULL: token t is of sequence t
    const int* positions;
    const int* slots;
    const float* inv_freq;   // [32], or NULL
    int interleaved;
    float mscale;
    const uint16_t* norm;    // [latent], or NULL
    float eps;
    // queries: q[t][h] = (q_main[t][h], turned q_rot[t][h]), or heads 0
    const float* q_main;
    long main_ld, main_head; // elements from token to token, head to head
    int main;                // columns
    const float* q_rot;
    long rot_ld, rot_head;
    int heads;
    uint16_t* q;
};

// Latent rows to keys and values; `to` has value + 64 columns of K (dim) and value
// of V (dim_v) per head (kv_heads).
struct ExpandArgs {
    KvCache c;
    const int* lengths;
    const int* firsts;       // or NULL: all positions
    int max_length;
    int count;               // sequences
    const uint8_t* packed;   // [heads * 2 value][latent / 2]
    const uint16_t* scales;
    const uint16_t* mins;
    KvCache to;
};

inline bool value_supported(int value) { return value == 64 || value == 128; }

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t st);
hipError_t launch_latent_attn(const NewArgs& x, const DeviceInfo& dev, hipStream_t st);
hipError_t launch_latent_expand(const ExpandArgs& a, const DeviceInfo& dev, hipStream_t st);
int64_t latent_attn_workspace(int heads, int latent, long max_new);

}  // namespace q4
