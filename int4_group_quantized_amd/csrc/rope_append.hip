// Head norm, rotary position and cache write of new tokens (gfx950).
//
// For each query and key head of a token (x = its fp32 columns of the fused
// projection's row):  x *= weight / sqrt(mean(x^2) + eps)  (optional), then
// each pair (lo, hi) of the first `rot` dimensions is turned by the angle
// position * inv_freq[pair] and scaled by mscale; the result is rounded once
// to fp16.  Values are rounded and written only.
//
// Memory bound: a token reads (heads + 2 kv_heads) * dim fp32 values and writes
// as many fp16 ones.  8,192 tokens of 48 heads of 128 (302 MB) take 62.6 us, 4.8
// TB/s; a 4 GiB copy runs at 4.6.  One token takes 2.6 us a launch among others of
// a graph (3.2 from start to end in a kernel trace), bound by the launch.
//
// Angles: position * inv_freq is formed in turns in 64 bits and reduced to
// [-1/2, 1/2] before it becomes a float.  In fp32 the product alone is off by
// position * 2^-24 radians (0.008 at position 131,072); the 64-bit product
// costs one multiplication per pair and token because a team keeps its sines
// and cosines for all the heads it serves.
//
// One launch, two kinds of workgroups:
//  * query / key rows: a team of LR lanes (LR the power of two >= dim / 4) owns
//    one token and HB consecutive heads.  A lane holds four dimensions: two
//    pairs with either pair layout, so that no value crosses lanes except for
//    the norm's sum.
//  * values: up to 64 tokens of one kv head go through LDS and leave transposed,
//    eight positions of one dimension per 16-byte store where the eight tokens
//    sit on an aligned run of one page (a prompt from position 3 takes 3% longer
//    than from position 0; with unaligned runs stored one by one 10%).
#include "attn.hpp"

namespace q4 {

constexpr int kAppendThreads = 256;
constexpr int kValueTokens = 64;
constexpr int kAppendAhead = 4;      // heads whose rows a team requests together
// Waves beyond which a team serves more heads (2, 4 or 8 of one token), so that
// sines and cosines are formed less often, and the most heads.  40 query and key
// heads, one per team against as chosen: 8,192 tokens of 128 100 and 66 us (4
// heads 66, 16 68, 32 82), 700 of 128 13.7 and 10.7, 1,404 of 256 56 and 32; a
// limit of 2,048 waves takes 300 of 256 from 9.9 to 10.9, one of 16,384 to 13.1.
constexpr long kAppendWaves = 4096;
constexpr int kAppendMost = 8;
constexpr int kValuePitch = kValueTokens + 10;  // halves; 37 dwords, so a token's dimensions fall on different banks
// Tokens per workgroup of values: kValueTokens, halved to kValueFew at least while
// that gives fewer than kValueBlocks workgroups (one token of each of 64
// sequences: 3.7 us with 8, 5.2 with 16, 9.0 with 64; 4,000 tokens of 40 heads of
// 128: 37.3 with 64, 46.6 with 8; 1,000 tokens of 24 heads of 64: 6.7 with 16, 7.9
// with 8, 8.9 with 64).
constexpr int kValueFew = 8;
constexpr long kValueBlocks = 256;
constexpr double kInvTwoPi = 0.15915494309189533577;

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const h2 v = {(_Float16)a, (_Float16)b};
    return as_u32(v);
}

// Page and offset of token t, or page -1.
__device__ __forceinline__ int append_slot(const AppendArgs& a, int t, int& off) {
    const int s = a.seq ? a.seq[t] : t;
    const int pos = a.positions[t];
    off = pos & ((1 << a.c.shift) - 1);
    if ((unsigned)s >= (unsigned)a.c.sequences || pos < 0 || (pos >> a.c.shift) >= a.c.cols) return -1;
    return page_of(a.c, a.c.table + (size_t)s * a.c.cols, pos);
}

// `vt` tokens (a multiple of 8 up to kValueTokens) of one kv head.
template <int D>
__device__ __forceinline__ void append_values(const AppendArgs& a, int tile, int vt, int head, uint16_t* lds) {
    __shared__ int slot_page[kValueTokens];
    __shared__ int slot_off[kValueTokens];
    __shared__ int run[kValueTokens / 8 + 1];
    const int tid = threadIdx.x;
    const int t0 = tile * vt;
    const int nt = min(vt, a.tokens - t0);
    if (tid < nt) {
        int off;
        slot_page[tid] = append_slot(a, t0 + tid, off);
        slot_off[tid] = off;
    }
    // Columns are shifted by the first position's place in its run of eight, so
    // that a prompt's aligned runs start at multiples of eight columns wherever
    // it starts.
    const int shift = a.positions[t0] & 7;
    const float* src = a.qkv + (size_t)t0 * a.ld + (size_t)(a.heads + a.c.kv_heads + head) * D;
    for (int i = tid; i < nt * (D / 4); i += kAppendThreads) {
        const int t = i / (D / 4), d = i % (D / 4) * 4;
        const f4 v = *reinterpret_cast<const f4*>(src + (size_t)t * a.ld + d);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            lds[(d + e) * kValuePitch + t + shift] = __builtin_bit_cast(uint16_t, (_Float16)v[e]);
    }
    __syncthreads();
    const int groups = (nt + shift + 7) / 8;
    if (tid < groups) {
        const int t = 8 * tid - shift;  // token of the group's first column
        int ok = t >= 0 && t + 8 <= nt;
        if (ok) {
            const int p = slot_page[t], o = slot_off[t];
            ok = p >= 0 && (o & 7) == 0;
            for (int e = 1; e < 8; ++e) ok = ok && slot_page[t + e] == p && slot_off[t + e] == o + e;
        }
        run[tid] = ok;
    }
    __syncthreads();
    const int P = 1 << a.c.shift;
    for (int i = tid; i < groups * D; i += kAppendThreads) {
        const int g = i % groups, d = i / groups, t = 8 * g - shift;
        const uint16_t* col = lds + d * kValuePitch + 8 * g;
        const size_t base = ((size_t)head * D + d) * P;
        if (run[g]) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(col);
            *reinterpret_cast<u4*>(a.c.v + (size_t)slot_page[t] * a.c.v_stride + base + slot_off[t]) =
                (u4){w[0], w[1], w[2], w[3]};
        } else {
            for (int e = max(0, -t); e < 8 && t + e < nt; ++e) {
                const int p = slot_page[t + e];
                if (p >= 0) a.c.v[(size_t)p * a.c.v_stride + base + slot_off[t + e]] = col[e];
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(AppendArgs a, int value_blocks, int vt, int hb) {
    __shared__ uint16_t lds[D * kValuePitch];
    if ((int)blockIdx.x < value_blocks) {
        append_values<D>(a, blockIdx.x / a.c.kv_heads, vt, blockIdx.x % a.c.kv_heads, lds);
        return;
    }
    constexpr int LR = D <= 64 ? 16 : D <= 128 ? 32 : 64;
    constexpr int TEAMS = kAppendThreads / LR;
    const int lane = threadIdx.x % LR;
    const int rows = a.heads + a.c.kv_heads;  // query and key heads
    const int blocks_of_heads = (rows + hb - 1) / hb;
    const long team = (long)(blockIdx.x - value_blocks) * TEAMS + threadIdx.x / LR;
    const bool live = team < (long)a.tokens * blocks_of_heads;
    const int t = live ? (int)(team / blocks_of_heads) : 0;
    const int h0 = (int)(team % blocks_of_heads) * hb;
    const int h1 = live ? min(rows, h0 + hb) : h0;
    // Lanes past the last dimension (dim 96 and 192) hold zeros and stay with
    // their team for the norm's sum.
    const bool wide = 4 * lane < D;

    // Dimensions of the lane: oa, oa + 1 and ob, ob + 1.
    const bool turned = 4 * lane < a.rot;  // rot <= D, so such a lane is not past the end
    const bool split = turned && !a.interleaved;
    const int oa = split ? 2 * lane : 4 * lane;
    const int ob = split ? a.rot / 2 + 2 * lane : 4 * lane + 2;
    float c0 = 1.0f, s0 = 0.0f, c1 = 1.0f, s1 = 0.0f;
    int page = -1, off = 0;
    if (live) {
        page = append_slot(a, t, off);
        if (turned) {
            const double pos = (double)a.positions[t] * kInvTwoPi;
            const double ta = pos * (double)a.inv_freq[2 * lane], tb = pos * (double)a.inv_freq[2 * lane + 1];
            sincospif(2.0f * (float)(ta - __builtin_rint(ta)), &s0, &c0);
            sincospif(2.0f * (float)(tb - __builtin_rint(tb)), &s1, &c1);
            c0 *= a.mscale; s0 *= a.mscale; c1 *= a.mscale; s1 *= a.mscale;
        }
    }
    float wq[4] = {1.0f, 1.0f, 1.0f, 1.0f}, wk[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if (wide && a.q_norm) {
        wq[0] = f16_bits_to_f32(a.q_norm[oa]);
        wq[1] = f16_bits_to_f32(a.q_norm[oa + 1]);
        wq[2] = f16_bits_to_f32(a.q_norm[ob]);
        wq[3] = f16_bits_to_f32(a.q_norm[ob + 1]);
    }
    if (wide && a.k_norm) {
        wk[0] = f16_bits_to_f32(a.k_norm[oa]);
        wk[1] = f16_bits_to_f32(a.k_norm[oa + 1]);
        wk[2] = f16_bits_to_f32(a.k_norm[ob]);
        wk[3] = f16_bits_to_f32(a.k_norm[ob + 1]);
    }
    const float* src = a.qkv + (size_t)t * a.ld;
    uint16_t* qrow = a.q + (size_t)t * a.heads * D;
    uint16_t* krow = a.c.k + (size_t)max(page, 0) * a.c.k_stride + (size_t)off * D;
    for (int h = h0; h < h1; h += kAppendAhead) {
        // The rows of several heads are requested together.
        float2 us[kAppendAhead], ws[kAppendAhead];
#pragma unroll
        for (int j = 0; j < kAppendAhead; ++j) {
            us[j] = ws[j] = {0.0f, 0.0f};
            if (wide && h + j < h1) {
                const float* x = src + (size_t)(h + j) * D;
                us[j] = *reinterpret_cast<const float2*>(x + oa);
                ws[j] = *reinterpret_cast<const float2*>(x + ob);
            }
        }
#pragma unroll
        for (int j = 0; j < kAppendAhead; ++j) {
            if (h + j >= h1) break;
            const bool is_q = h + j < a.heads;
            float2 u = us[j], w = ws[j];
            if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
                const float ss = reduce_lanes<LR>(u.x * u.x + u.y * u.y + (w.x * w.x + w.y * w.y));
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
                u.x *= r * (is_q ? wq[0] : wk[0]);
                u.y *= r * (is_q ? wq[1] : wk[1]);
                w.x *= r * (is_q ? wq[2] : wk[2]);
                w.y *= r * (is_q ? wq[3] : wk[3]);
            }
            float2 y = u, z = w;
            if (split) {
                y.x = u.x * c0 - w.x * s0;
                z.x = w.x * c0 + u.x * s0;
                y.y = u.y * c1 - w.y * s1;
                z.y = w.y * c1 + u.y * s1;
            } else if (turned) {
                y.x = u.x * c0 - u.y * s0;
                y.y = u.y * c0 + u.x * s0;
                z.x = w.x * c1 - w.y * s1;
                z.y = w.y * c1 + w.x * s1;
            }
            if (!wide || (!is_q && page < 0)) continue;
            uint16_t* dst = is_q ? qrow + (size_t)(h + j) * D : krow + ((size_t)(h + j - a.heads) << a.c.shift) * D;
            *reinterpret_cast<uint32_t*>(dst + oa) = pack_f16(y.x, y.y);
            *reinterpret_cast<uint32_t*>(dst + ob) = pack_f16(z.x, z.y);
        }
    }
}

template <int D>
static hipError_t launch_append(const AppendArgs& a, hipStream_t st) {
    constexpr int TEAMS = kAppendThreads / (D <= 64 ? 16 : D <= 128 ? 32 : 64);
    const int rows = a.heads + a.c.kv_heads;
    int hb = 1;
    constexpr long SLOTS = kAppendWaves * 64 * TEAMS / kAppendThreads;
    while ((long)a.tokens * ((rows + hb - 1) / hb) > SLOTS && hb < rows && hb < kAppendMost) hb *= 2;
    int vt = kValueTokens;
    while (vt > kValueFew && ((long)a.tokens + vt - 1) / vt * a.c.kv_heads < kValueBlocks) vt /= 2;
    const long value_blocks = ((long)a.tokens + vt - 1) / vt * a.c.kv_heads;
    const long teams = (long)a.tokens * ((rows + hb - 1) / hb);
    const long grid = value_blocks + (teams + TEAMS - 1) / TEAMS;
    // A launch takes at most 2^32 - 1 threads; rows and queries for more than that
    // would take over 288 GB.
    if (grid > (1L << 24) - 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rope_append_kernel<D>), dim3((unsigned)grid), dim3(kAppendThreads), 0, st, a,
                       (int)value_blocks, vt, hb);
    return hipGetLastError();
}

hipError_t launch_rope_append(const AppendArgs& a, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_append<64>(a, st);
        case 96: return launch_append<96>(a, st);
        case 128: return launch_append<128>(a, st);
        case 192: return launch_append<192>(a, st);
        case 256: return launch_append<256>(a, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
