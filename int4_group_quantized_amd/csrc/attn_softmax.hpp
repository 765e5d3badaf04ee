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

// 2^(m - top), 0 for an empty part; top is the joint maximum.
__device__ __forceinline__ float part_weight(float m, float top) {
    return m == Q4_NEG_INF ? 0.0f : exp2_hw(m - top);
}

// A dot product as a base-2 score.  EXTRA: with the options' cap and bias;
// tanh(x) = 1 - 2 / (e^(2x) + 1), absolute error about 2^-23, so the score's
// is about softcap * 2^-23.
struct ScoreParams {
    float scale2;     // scale * log2(e); EXTRA: unused
    float scale;      // EXTRA: scale, or with a cap scale / softcap * 2 log2(e)
    float softcap;
    float slope;
};

template <bool EXTRA>
__device__ __forceinline__ ScoreParams score_params(const AttnArgs& a, int head) {
    ScoreParams p;
    p.scale2 = a.scale * kLog2e;
    p.scale = a.softcap > 0.0f ? a.scale / a.softcap * (2.0f * kLog2e) : a.scale;
    p.softcap = a.softcap;
    p.slope = EXTRA && a.slopes ? a.slopes[head] : 0.0f;
    return p;
}

// distance = key position - query position
template <bool EXTRA>
__device__ __forceinline__ float score(float dot, const ScoreParams& p, int distance) {
    if constexpr (!EXTRA) return dot * p.scale2;
    float s = dot * p.scale;
    if (p.softcap > 0.0f) s = p.softcap - p.softcap * 2.0f * __builtin_amdgcn_rcpf(exp2_hw(s) + 1.0f);
    return (s + p.slope * (float)distance) * kLog2e;
}

}  // namespace q4
