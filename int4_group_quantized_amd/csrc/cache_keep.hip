// The accepted tokens of each sequence's draft moved together in the cache
// (gfx950): position starts[s] + keep[i] to starts[s] + i.
//
// A workgroup moves one sequence's tokens of one kv head, kKeepTokens at a time:
// all of them are read before any is written, and since keep ascends (keep[i] >=
// i) later ones lie behind what has been written.  Keys go as 16-byte chunks of
// their rows; values, whose positions are next to each other for one dimension, as
// single halves with the tokens of one dimension in neighbouring lanes, so that
// they share memory lines.
//
// Bound by the launch and a chain of three reads (bounds, pages, rows): one sequence
// with 5 kept tokens takes 3.7 us (4 kv heads of 128; 3.9 with 8), 256 sequences of 8 kv
// heads with up to 12 each 10.7 to 12.4 us for 14 MB read and written (the values in two
// to three times as much, whole lines), with 12 each 18.5.  Numbering the values over
// the tokens that there are, not over 32 with most lanes idle, took the call with up to
// 12 from 20 us.
#include "attn.hpp"

namespace q4 {

constexpr int kKeepThreads = 256;
constexpr int kKeepTokens = 32;

// i / n for i < 2^13, n <= 32: (i + 1/2) / n keeps 1 / (2 n) from every whole number,
// 500 times its rounding error.
__device__ __forceinline__ int quotient(int i, float inv_n) { return (int)(((float)i + 0.5f) * inv_n); }

// D: columns of a key, or of a latent row (a cache without V).
template <int D>
__global__ void __launch_bounds__(kKeepThreads) cache_keep_kernel(KeepArgs a) {
    constexpr int C = D / 8;                                      // 16-byte chunks of a key
    constexpr int KEYS = (kKeepTokens * C + kKeepThreads - 1) / kKeepThreads;  // chunks of a thread
    constexpr int VALUES = D <= 256 ? kKeepTokens * D / kKeepThreads : 1;      // and halves
    __shared__ int from_page[kKeepTokens], from_off[kKeepTokens], to_page[kKeepTokens], to_off[kKeepTokens];
    const int s = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
    const int pmask = (1 << a.c.shift) - 1;
    const int* row = a.c.table + (size_t)s * a.c.cols;
    const int ks = a.keep_starts[s], ke = a.keep_starts[s + 1];
    const long start = a.starts[s], end = (long)a.c.cols << a.c.shift;
    const int first = min(max(ks, 0), a.total), last = min(max(ke, first), a.total);
    for (int i0 = first; i0 < last; i0 += kKeepTokens) {
        const int n = min(kKeepTokens, last - i0);
        const float inv_n = 1.0f / (float)n;
        __syncthreads();
        if (tid < n) {
            const long from = start + a.keep[i0 + tid], to = start + (i0 - first + tid);
            int p = -1;
            // A token that stays where it is is not moved, nor one that has no place.
            if (from != to && from >= 0 && from < end && to >= 0 && to < end) {
                p = page_of(a.c, row, (int)from);
                to_page[tid] = page_of(a.c, row, (int)to);
                if (to_page[tid] < 0) p = -1;
                from_off[tid] = (int)from & pmask;
                to_off[tid] = (int)to & pmask;
            }
            from_page[tid] = p;
        }
        __syncthreads();
        u4 k[KEYS];
        uint16_t v[VALUES];
#pragma unroll
        for (int j = 0; j < KEYS; ++j) {
            const int i = j * kKeepThreads + tid, e = i / C, c = i % C;
            if (e < n && from_page[e] >= 0)
                k[j] = *reinterpret_cast<const u4*>(a.c.k + (size_t)from_page[e] * a.c.k_stride +
                                                    (((size_t)head << a.c.shift) + from_off[e]) * D + 8 * c);
        }
        if (D <= 256 && a.c.v) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                if (j * kKeepThreads >= n * D) break;
                const int i = j * kKeepThreads + tid, d = quotient(i, inv_n), e = i - d * n;
                if (d < D && from_page[e] >= 0)
                    v[j] = a.c.v[(size_t)from_page[e] * a.c.v_stride + ((size_t)(head * D + d) << a.c.shift) + from_off[e]];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KEYS; ++j) {
            const int i = j * kKeepThreads + tid, e = i / C, c = i % C;
            if (e < n && from_page[e] >= 0)
                *reinterpret_cast<u4*>(a.c.k + (size_t)to_page[e] * a.c.k_stride +
                                       (((size_t)head << a.c.shift) + to_off[e]) * D + 8 * c) = k[j];
        }
        if (D <= 256 && a.c.v) {
#pragma unroll
            for (int j = 0; j < VALUES; ++j) {
                if (j * kKeepThreads >= n * D) break;
                const int i = j * kKeepThreads + tid, d = quotient(i, inv_n), e = i - d * n;
                if (d < D && from_page[e] >= 0)
                    a.c.v[(size_t)to_page[e] * a.c.v_stride + ((size_t)(head * D + d) << a.c.shift) + to_off[e]] = v[j];
            }
        }
    }
}

template <int D>
static hipError_t launch_keep(const KeepArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((cache_keep_kernel<D>), dim3((unsigned)a.count, (unsigned)a.c.kv_heads), dim3(kKeepThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_cache_keep(const KeepArgs& a, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_keep<64>(a, st);
        case 96: return launch_keep<96>(a, st);
        case 128: return launch_keep<128>(a, st);
        case 192: return launch_keep<192>(a, st);
        case 256: return launch_keep<256>(a, st);
        case 320: return launch_keep<320>(a, st);
        case 576: return launch_keep<576>(a, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
