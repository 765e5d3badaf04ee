// New tokens' latent rows into the cache, and their queries (gfx950).
//
// Cache row of a token:  (x_l * weight / sqrt(mean(x_l^2) + eps)  (norm optional),
// its last 64 columns with each pair turned by position * inv_freq[pair] and scaled by
// mscale), rounded once to fp16.  Query of a token and head: its main part as it
// is, its rotary part turned alike.
//
// Memory bound: reads fp32, writes as many fp16 values: 4,001 tokens with queries of
// 128 heads of 192 (604 MB) take 107 to 111 us, 5.5 TB/s; one token with 16 heads 4.5,
// the launch and a chain of reads.  Angles as in the append of
// heads: formed in turns in 64 bits and reduced before they become floats.
//
// One launch, two kinds of workgroups:
//  * cache rows: a wave each.
//  * queries: a workgroup owns one token and `hb` heads, so that sines and cosines
//    are formed once for them, in LDS; its threads take units of eight columns of
//    the main part or 16 of the rotary part, 16 or two times 16 bytes written.
#include "latent.hpp"

namespace q4 {

constexpr int kLatentAppendThreads = 256;
constexpr int kPairs = kRot / 2;
constexpr double kInvTurn = 0.15915494309189533577;
// Queries' units of a workgroup: as many heads as make about this many.
constexpr int kQueryUnits = 1024;

// Sine and cosine, times mscale, of pair i at a position; nothing is turned or
// scaled without frequencies.
__device__ __forceinline__ float2 latent_angle(const LatentAppendArgs& a, int position, int i) {
    if (!a.inv_freq) return {0.0f, 1.0f};
    const double turns = (double)position * kInvTurn * (double)a.inv_freq[i];
    float s, c;
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
    return {s * a.mscale, c * a.mscale};
}

__device__ __forceinline__ uint32_t two_halves(float a, float b) { return as_u32((h2){(_Float16)a, (_Float16)b}); }

// The wave's token's row into the cache.
template <int L>
__device__ __forceinline__ void append_row(const LatentAppendArgs& a, int t) {
    constexpr int PER = L / 64;  // columns of a lane: 2, 4 or 8
    const int lane = threadIdx.x & 63;
    const int s = a.seq ? a.seq[t] : t, pos = a.slots[t];
    int page = -1;
    if ((unsigned)s < (unsigned)a.c.sequences && pos >= 0 && (pos >> a.c.shift) < a.c.cols)
        page = page_of(a.c, a.c.table + (size_t)s * a.c.cols, pos);
    if (page < 0) return;
    const float* x = a.kv + (size_t)t * a.ld;
    uint16_t* out = a.c.k + (size_t)page * a.c.k_stride + (size_t)(pos & ((1 << a.c.shift) - 1)) * (L + kRot);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
        const float2 w = *reinterpret_cast<const float2*>(x + PER * lane + i);
        v[i] = w.x;
        v[i + 1] = w.y;
    }
    float2 lo = {0, 0};
    if (lane < kPairs) {
        const int i0 = a.interleaved ? 2 * lane : lane, i1 = a.interleaved ? 2 * lane + 1 : lane + kPairs;
        lo = {x[L + i0], x[L + i1]};
    }
    if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
        const float r = rsqrtf(reduce_lanes<64>(ss) * (1.0f / L) + a.eps);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] *= r * f16_bits_to_f32(a.norm[PER * lane + i]);
    }
#pragma unroll
    for (int i = 0; i < PER; i += 2) *reinterpret_cast<uint32_t*>(out + PER * lane + i) = two_halves(v[i], v[i + 1]);
    if (lane < kPairs) {
        const float2 sc = latent_angle(a, a.positions[t], lane);
        const float y0 = lo.x * sc.y - lo.y * sc.x, y1 = lo.y * sc.y + lo.x * sc.x;
        if (a.interleaved) {
            *reinterpret_cast<uint32_t*>(out + L + 2 * lane) = two_halves(y0, y1);
        } else {
            out[L + lane] = __builtin_bit_cast(uint16_t, (_Float16)y0);
            out[L + kPairs + lane] = __builtin_bit_cast(uint16_t, (_Float16)y1);
        }
    }
}

template <int L>
__global__ void __launch_bounds__(kLatentAppendThreads) latent_append_kernel(LatentAppendArgs a, int row_blocks, int hb) {
    constexpr int WAVES = kLatentAppendThreads / 64;
    if ((int)blockIdx.x < row_blocks) {
        const int t = blockIdx.x * WAVES + (threadIdx.x >> 6);
        if (t < a.tokens) append_row<L>(a, t);
        return;
    }
    __shared__ float2 angle[kPairs];
    const int chunks = (a.heads + hb - 1) / hb, block = blockIdx.x - row_blocks;
    const int t = block / chunks, h0 = (block - t * chunks) * hb, heads = min(hb, a.heads - h0);
    if (threadIdx.x < kPairs) angle[threadIdx.x] = latent_angle(a, a.positions[t], threadIdx.x);
    __syncthreads();
    const int wide = a.main / 8, units = wide + kRot / 16;
    const float* from = a.q_main + (size_t)t * a.main_ld + (size_t)h0 * a.main_head;
    const float* turn = a.q_rot + (size_t)t * a.rot_ld + (size_t)h0 * a.rot_head;
    uint16_t* out = a.q + ((size_t)t * a.heads + h0) * (a.main + kRot);
    // Unit u of head h; each step takes the workgroup's threads further.
    int h = threadIdx.x / units, u = threadIdx.x % units;
    const int dh = kLatentAppendThreads / units, du = kLatentAppendThreads % units;
    for (; h < heads; h += dh, u += du, h += u >= units, u -= u >= units ? units : 0) {
        uint16_t* to = out + (size_t)h * (a.main + kRot);
        if (u < wide) {
            const f4* x = reinterpret_cast<const f4*>(from + (size_t)h * a.main_head + 8 * u);
            const f4 v = x[0], w = x[1];
            *reinterpret_cast<u4*>(to + 8 * u) =
                (u4){two_halves(v[0], v[1]), two_halves(v[2], v[3]), two_halves(w[0], w[1]), two_halves(w[2], w[3])};
            continue;
        }
        // Eight pairs: 16 columns next to each other, or two times eight.
        const int p0 = 8 * (u - wide), at0 = a.interleaved ? 2 * p0 : p0, at1 = a.interleaved ? 2 * p0 + 8 : p0 + kPairs;
        const float* x = turn + (size_t)h * a.rot_head;
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const f4 v = *reinterpret_cast<const f4*>(x + at0 + i), w = *reinterpret_cast<const f4*>(x + at1 + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[i + e] = v[e];
                hi[i + e] = w[e];
            }
        }
        uint32_t first[4], second[4];
        if (a.interleaved) {
            // Pair i is columns 2i and 2i + 1 of both halves in order.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 s0 = angle[p0 + i], s1 = angle[p0 + 4 + i];
                first[i] = two_halves(lo[2 * i] * s0.y - lo[2 * i + 1] * s0.x, lo[2 * i + 1] * s0.y + lo[2 * i] * s0.x);
                second[i] = two_halves(hi[2 * i] * s1.y - hi[2 * i + 1] * s1.x, hi[2 * i + 1] * s1.y + hi[2 * i] * s1.x);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 s0 = angle[p0 + 2 * i], s1 = angle[p0 + 2 * i + 1];
                first[i] = two_halves(lo[2 * i] * s0.y - hi[2 * i] * s0.x, lo[2 * i + 1] * s1.y - hi[2 * i + 1] * s1.x);
                second[i] = two_halves(hi[2 * i] * s0.y + lo[2 * i] * s0.x, hi[2 * i + 1] * s1.y + lo[2 * i + 1] * s1.x);
            }
        }
        *reinterpret_cast<u4*>(to + a.main + at0) = (u4){first[0], first[1], first[2], first[3]};
        *reinterpret_cast<u4*>(to + a.main + at1) = (u4){second[0], second[1], second[2], second[3]};
    }
}

template <int L>
static hipError_t launch_append_rows(const LatentAppendArgs& a, hipStream_t st) {
    constexpr int WAVES = kLatentAppendThreads / 64;
    const int units = a.main / 8 + kRot / 16;
    int hb = kQueryUnits / units;
    if (hb < 1) hb = 1;
    const long row_blocks = ((long)a.tokens + WAVES - 1) / WAVES;
    const long grid = row_blocks + (a.heads > 0 ? (long)a.tokens * ((a.heads + hb - 1) / hb) : 0);
    // A launch takes at most 2^32 - 1 threads.
    if (grid > (1L << 24) - 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL((latent_append_kernel<L>), dim3((unsigned)grid), dim3(kLatentAppendThreads), 0, st, a, (int)row_blocks, hb);
    return hipGetLastError();
}

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t st) {
    switch (a.c.dim - kRot) {
        case 128: return launch_append_rows<128>(a, st);
        case 256: return launch_append_rows<256>(a, st);
        case 512: return launch_append_rows<512>(a, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
