// Score and softmax arithmetic shared by the decode and prompt attention
// kernels, and the join of partial results over parts of the cache.
//
// Softmax runs in base 2: scores carry the factor log2(e), so that each
// exponential is one v_exp_f32.  Every part keeps, per query row, the largest
// score m (-inf: nothing seen), the sum l of 2^(s - m) and the unnormalised
// output O = sum 2^(s - m) v; two parts join exactly as
//   m = max(m1, m2),  l = l1 2^(m1-m) + l2 2^(m2-m),  O likewise.
#pragma once

#include "attn.hpp"

namespace q4 {

constexpr float kLog2e = 1.44269504088896340736f;
#define Q4_NEG_INF (-__builtin_inff())

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Kernels without options form 2^(score - base) from a dot product in one multiply-add,
// whose product is not rounded, while the base is a maximum that is.  They are apart by
// 2^-24 of the score, which is a power of two common to a row's weights and so no error,
// until it takes them out of fp16's range: bases of 2^29 leave infinities or nothing.
// Rows that meet a base beyond 2^26 (a power of 4 at most) are started again, one
// position after the other, with scores rounded as the maximum is.  In the loop over
// tiles, rounding where the base asks for it cost 1 to 2% of 1,000 prompt tokens' time and
// of absorbed attention's with 64 rows, though no row asked.
__device__ __forceinline__ bool far_base(float m) {
    constexpr uint32_t FAR = 0x4C800000u, INF = 0x7F800000u;  // 2^26; neither infinities nor NaN are far
    return (__builtin_bit_cast(uint32_t, m) & 0x7FFFFFFFu) - FAR - 1 < INF - FAR - 1;
}

// 2^(m - top), 0 for an empty part; top is the joint maximum.
__device__ __forceinline__ float part_weight(float m, float top) {
    return m == Q4_NEG_INF ? 0.0f : exp2_hw(m - top);
}

// The larger of two, NaN if either is: one instruction for two or three operands,
// where fmaxf first passes each matrix result through one of its own to quieten
// signalling NaN (35 more for the 32 scores of a lane).
__device__ __forceinline__ float top_of(float a, float b) {
    return __builtin_elementwise_maximum(a, b);
}

// The maximum of lanes i and i ^ 32, and of i and i ^ 16, in registers.
__device__ __forceinline__ float top_of_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return top_of(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float top_of_rows(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return top_of(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}

// Partial results pass between workgroups that may run on different XCDs, whose
// L2 caches are not coherent with each other: they are written through to and
// read from memory (agent scope).  A workgroup publishes them by waiting for its
// own stores before it counts itself as finished (parts_done).  Fences of agent
// scope would instead write back and invalidate whole caches for every
// workgroup: decode over 16 sequences of up to 4,096 positions took 32 us with
// them and 18.6 us with this.
__device__ __forceinline__ void share_store(float* p, float x, float y) {
    const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, x) | (uint64_t)__builtin_bit_cast(uint32_t, y) << 32;
    __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float2 share_load(const float* p) {
    const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    return {__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32))};
}

// Called by every thread of a workgroup after its last share_store.  True in
// the workgroup that finishes last of `parts`; the counter is then zero again.
__device__ __forceinline__ bool parts_done(int* counter, int parts) {
    __shared__ int last;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0) {
        last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
        if (last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return last != 0;
}

// A query row over some of its positions, held by a wave: lane l has the pairs
// of dimensions 2 (l + 64 i) of the unnormalised output; m and l in all lanes.
template <int D>
struct JoinedRow {
    static constexpr int PER = (D + 127) / 128;
    float2 o[PER];
    float m, l;
};

// Joins the parts of a row in order: part p has its output at po + p * stride * D
// and (m, l) at ml + p * stride * 2.  Up to kJoin parts at a time are requested
// together, lane p holding part p's statistics; part after part waited for each
// time took 3.3 us for 8 parts.  AGENT: the parts come from workgroups of the
// same launch.
constexpr int kJoin = 16;
template <int D, bool AGENT>
__device__ __forceinline__ JoinedRow<D> join_parts(const float* po, const float* ml, long stride, int parts) {
    const int lane = threadIdx.x & 63;
    auto get = [](const float* p) { return AGENT ? share_load(p) : *reinterpret_cast<const float2*>(p); };
    constexpr int PER = JoinedRow<D>::PER;
    JoinedRow<D> r;
#pragma unroll
    for (int i = 0; i < PER; ++i) r.o[i] = {0.0f, 0.0f};
    r.m = Q4_NEG_INF;
    r.l = 0.0f;
    for (int p0 = 0; p0 < parts; p0 += kJoin) {
        float2 v[kJoin][PER];
        float2 st = {Q4_NEG_INF, 0.0f};
        if (lane < kJoin && p0 + lane < parts) st = get(ml + (long)(p0 + lane) * stride * 2);
#pragma unroll
        for (int p = 0; p < kJoin; ++p) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int d = 2 * (lane + 64 * i);
                v[p][i] = {0.0f, 0.0f};
                if (p0 + p < parts && d < D) v[p][i] = get(po + (long)(p0 + p) * stride * D + d);
            }
        }
        float t = st.x;
#pragma unroll
        for (int d = kJoin / 2; d >= 1; d >>= 1) t = fmaxf(t, __shfl_xor(t, d, 64));
        t = fmaxf(r.m, __shfl(t, 0, 64));
        const float f0 = part_weight(r.m, t), w = part_weight(st.x, t);
        float s1 = st.y * w;
#pragma unroll
        for (int d = kJoin / 2; d >= 1; d >>= 1) s1 += __shfl_xor(s1, d, 64);
        r.l = r.l * f0 + __shfl(s1, 0, 64);
        r.m = t;
#pragma unroll
        for (int i = 0; i < PER; ++i) r.o[i] = {r.o[i].x * f0, r.o[i].y * f0};
#pragma unroll
        for (int p = 0; p < kJoin; ++p) {
            const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), p));
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                r.o[i].x += v[p][i].x * f;
                r.o[i].y += v[p][i].y * f;
            }
        }
    }
    return r;
}

template <int D>
__device__ __forceinline__ void store_joined(const JoinedRow<D>& r, uint16_t* out) {
    const float inv = r.l > 0.0f || r.l != r.l ? 1.0f / r.l : 0.0f;
#pragma unroll
    for (int i = 0; i < JoinedRow<D>::PER; ++i) {
        const int d = 2 * ((threadIdx.x & 63) + 64 * i);
        if (d < D)
            *reinterpret_cast<uint32_t*>(out + d) = as_u32((h2){(_Float16)(r.o[i].x * inv), (_Float16)(r.o[i].y * inv)});
    }
}

// The kernels' instantiations by what their scores need: scale only, a cap or a
// bias, a large cap (and perhaps a bias).
constexpr int kNoOptions = 0, kOptions = 1, kLargeCapOptions = 2;
constexpr float kLargeCap = 64.0f;  // see capped
inline int attn_options(const AttnArgs& a) {
    return a.softcap > kLargeCap ? kLargeCapOptions : a.softcap > 0.0f || a.slopes ? kOptions : kNoOptions;
}

// A dot product as a base-2 score: scale * log2(e) * dot, or with the options'
// cap and bias.
struct ScoreParams {
    float scale2;  // scale * log2(e)
    float cap_in;  // 2 log2(e) * scale / softcap, finite
    float cap2;    // softcap * log2(e)
    float slope2;  // slope * log2(e)
};

template <int OPTIONS>
__device__ __forceinline__ ScoreParams score_params(const AttnArgs& a, int head) {
    ScoreParams p;
    p.scale2 = a.scale * kLog2e;
    // Held finite, so that under the smallest caps a product of zero stays zero;
    // without a cap unused.
    p.cap_in = OPTIONS != kNoOptions ? fminf(2.0f * kLog2e * a.scale / a.softcap, __FLT_MAX__) : 0.0f;
    p.cap2 = a.softcap * kLog2e;
    p.slope2 = OPTIONS != kNoOptions && a.slopes ? a.slopes[head] * kLog2e : 0.0f;
    return p;
}

// softcap tanh(x) log2(e), x = scale dot / softcap, from tanh(x) = 1 - 2 / (e^(2x)
// + 1): off by a few 2^-23 whatever x is, so the score by softcap times that,
// 2.3e-5 under a cap of 64, a twentieth of the weights' rounding.  Under larger
// caps it would pass the scores themselves (0.1 under a cap of 10^6), so LARGE
// takes the series x - x^3/3 + 2x^5/15 below |2 log2(e) x| = 0.33, off by 2^-22 of x
// there; above, the first form is off by less than 2^-18 of x.  Both forms for every
// cap: 4,096 tokens of 16 heads of 128 148 us, of 64 127; one 121 and 93.  Chosen in
// the kernel instead of by its instantiation: with a bias only 123 and 111 us.
template <bool LARGE>
__device__ __forceinline__ float capped(float dot, const ScoreParams& p) {
    const float z = dot * p.cap_in;
    const float far = __builtin_fmaf(-2.0f * p.cap2, __builtin_amdgcn_rcpf(exp2_hw(z) + 1.0f), p.cap2);
    if constexpr (!LARGE) return far;
    constexpr float A = 1.0f / (3.0f * 4.0f * kLog2e * kLog2e);
    constexpr float B = 2.0f / (15.0f * 16.0f * kLog2e * kLog2e * kLog2e * kLog2e);
    const float y = dot * p.scale2, t = z * z;
    return __builtin_fabsf(z) < 0.33f ? __builtin_fmaf(y, t * __builtin_fmaf(t, B, -A), y) : far;
}

// distance = key position - query position
template <int OPTIONS>
__device__ __forceinline__ float score(float dot, const ScoreParams& p, int distance) {
    if constexpr (OPTIONS == kNoOptions) return dot * p.scale2;
    constexpr bool LARGE = OPTIONS == kLargeCapOptions;
    const float s = LARGE || p.cap2 > 0.0f ? capped<LARGE>(dot, p) : dot * p.scale2;
    return __builtin_fmaf(p.slope2, (float)distance, s);
}

}  // namespace q4
