// Attention of one new token per sequence over the paged cache (gfx950).
//
//   out[b][h] = sum_j softmax_j(s(q[b][h] . k_j)) v_j  over the positions j that
//   the query at lengths[b] - 1 sees.
//
// Memory bound: every cached position costs 4 * dim bytes per kv head and
// 4 * dim flops per head that reads it; the matrix cores' work (query rows
// padded to 16) is a twentieth of what they can do in the time the bytes take.
//
// A wave takes 64 positions (a tile) at a time, keys and values straight from
// memory into registers in the operand layout of v_mfma_f32_16x16x32_f16:
//   S^T[key][row] = K Q^T     A = K rows as stored, B = the query rows
//   O^T[dim][row] = V^T P^T   A = V pages' rows as stored, B = P^T
// The result layout of the first product (lane: row = lane & 15, keys 4g + i of
// each 16-key subtile, g = lane >> 4) becomes the operand layout of the second
// (keys 8g + j of a 32-key block) without moving a value across lanes, because
// subtile t's row r loads key 32 (t/2) + 8 (r/4) + 4 (t%2) + r%4.  A query row's
// maximum and sum cross lanes twice per tile (lanes xor 16 and xor 32).
//
// Split: the visible tiles of all sequences are cut into parts of one length,
// computed on the device from the lengths so that uneven batches stay
// balanced: every workgroup gets one part of one sequence and kv head (4 waves
// take its tiles in turn), parts of a sequence are joined in order by a second
// launch.  A sequence of one part is written directly.
#include "attn_softmax.hpp"

namespace q4 {

constexpr int kDecodeWaves = 4;
constexpr int kDecodeThreads = 64 * kDecodeWaves;
constexpr int kDecodeSlots = 512;   // workgroups wanted per launch: two per CU
constexpr int kDecodeMinTiles = 4;  // tiles per part at least: one per wave

// First visible tile and the number of tiles of sequence b.
__device__ __forceinline__ int decode_tiles(const AttnArgs& a, int b, int& first, int& len) {
    len = min(max(a.lengths[b], 0), a.max_length);
    first = a.window > 0 && len > a.window ? (len - a.window) / kTileKeys : 0;
    return (len + kTileKeys - 1) / kTileKeys - first;
}

struct DecodePart {
    int b;        // sequence, or -1: no such part
    int part;     // of the sequence
    int parts;    // parts of the sequence
    int slot;     // workspace slot of the sequence's first part
    int chunk;    // tiles per part
};

// Tiles per part; each wave computes it for itself.  target: parts wanted per
// kv head and row block.
__device__ __forceinline__ int decode_chunk(const AttnArgs& a, int target) {
    const int lane = threadIdx.x & 63;
    long total = 0;
    for (int b0 = 0; b0 < a.rows; b0 += 64) {
        int first, len;
        int n = b0 + lane < a.rows ? decode_tiles(a, b0 + lane, first, len) : 0;
        for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, 64);
        total += n;
    }
    const long want = (total + target - 1) / target;
    return (int)(want > kDecodeMinTiles ? want : kDecodeMinTiles);
}

// The part with number `item`; parts are numbered sequence by sequence.
__device__ __forceinline__ DecodePart decode_part(const AttnArgs& a, int item, int target) {
    const int lane = threadIdx.x & 63;
    DecodePart r;
    r.chunk = decode_chunk(a, target);
    r.b = -1;
    r.part = r.parts = r.slot = 0;
    int before = 0;  // parts of earlier sequences
    for (int b0 = 0; b0 < a.rows; b0 += 64) {
        int first, len, n = 0;
        if (b0 + lane < a.rows) {
            n = (decode_tiles(a, b0 + lane, first, len) + r.chunk - 1) / r.chunk;
            n = n > 0 ? n : 1;  // an empty sequence has a part that writes zeros
        }
        int upto = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d, 64);
            if (lane >= d) upto += o;
        }
        const uint64_t hit = __ballot(n > 0 && item < before + upto && item >= before + upto - n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            r.b = b0 + l;
            r.parts = __builtin_amdgcn_readlane(n, l);
            r.slot = before + __builtin_amdgcn_readlane(upto, l) - r.parts;
            r.part = item - r.slot;
            return r;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return r;
}

__host__ __device__ inline int decode_target(int pairs) {
    const int t = kDecodeSlots / pairs;
    return t > 0 ? t : 1;
}

__device__ __forceinline__ h8 load_h8(const uint16_t* p) {
    return __builtin_bit_cast(h8, *reinterpret_cast<const u4*>(p));
}

template <int D, bool EXTRA>
__global__ void __launch_bounds__(kDecodeThreads) attn_decode_kernel(AttnArgs a, int target) {
    constexpr int OP = D + 4;  // pitch of a row of partial outputs in LDS
    __shared__ float part_o[kDecodeWaves][16][OP];
    __shared__ float part_m[kDecodeWaves][16], part_l[kDecodeWaves][16];
    const int row_blocks = (a.group + 15) / 16;
    const int kvh = blockIdx.y / row_blocks;
    const int row0 = (blockIdx.y % row_blocks) * 16;   // first head of the group in this workgroup
    const int nrows = min(16, a.group - row0);
    const DecodePart it = decode_part(a, blockIdx.x, target);
    if (it.b < 0) return;
    int first, len;
    const int tiles = decode_tiles(a, it.b, first, len);
    const int t_begin = first + it.part * it.chunk;
    const int t_end = min(first + tiles, t_begin + it.chunk);
    const int start = a.window > 0 && len > a.window ? len - a.window : 0;  // first visible position

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int P = 1 << a.c.shift, pmask = P - 1;
    const int* row = a.c.table + (size_t)it.b * a.c.cols;
    const int head0 = kvh * a.group + row0;

    h8 qf[D / 32];
    {
        const uint16_t* qp = a.q + ((size_t)it.b * a.heads + head0 + (n < nrows ? n : 0)) * D + 8 * g;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            qf[s] = load_h8(qp + 32 * s);
            if (n >= nrows) qf[s] = (h8)(_Float16)0.0f;
        }
    }
    const ScoreParams sp = score_params<EXTRA>(a, head0 + (n < nrows ? n : 0));

    f4 acc[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] = (f4){0, 0, 0, 0};
    float m = Q4_NEG_INF, l = 0.0f;

    for (int t = t_begin + wave; t < t_end; t += kDecodeWaves) {
        const int kb = t * kTileKeys;
        // Pages of the two 8-key groups this lane's values and scores belong to,
        // and of its keys' groups.  Positions past the end read the last one's page.
        int vp[2], kp[2];
        bool whole = kb >= start && kb + kTileKeys <= len;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            vp[h] = page_of(a.c, row, min(kb + 32 * h + 8 * g, len - 1));
            kp[h] = page_of(a.c, row, min(kb + 32 * h + 8 * (n >> 2), len - 1));
            whole = whole && vp[h] >= 0;
        }
        whole = __all(whole);
        f4 s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int key = kb + 32 * (u >> 1) + 8 * (n >> 2) + 4 * (u & 1) + (n & 3);
            const int page = max(kp[u >> 1], 0);
            const uint16_t* p = a.c.k + (size_t)page * a.c.k_stride + ((size_t)kvh * P + (key & pmask)) * D + 8 * g;
            s[u] = (f4){0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
                s[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(load_h8(p + 32 * d), qf[d], s[u], 0, 0, 0);
        }
        // Scores; masked ones are -inf.
        float top = Q4_NEG_INF;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = kb + 32 * (u >> 1) + 8 * g + 4 * (u & 1) + i;
                float x = score<EXTRA>(s[u][i], sp, key - (len - 1));
                if (!whole) x = key >= start && key < len && vp[u >> 1] >= 0 ? x : Q4_NEG_INF;
                s[u][i] = x;
                top = fmaxf(top, x);
            }
        }
        top = fmaxf(top, lane_swap16(top));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float m_new = fmaxf(m, top);
        const float base = m_new == Q4_NEG_INF ? 0.0f : m_new;
        const float f = exp2_hw(m - base);
        h8 pf[2];
        float sum = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = exp2_hw(s[u][i] - base);
                sum += p;
                pf[u >> 1][4 * (u & 1) + i] = (_Float16)p;
            }
        }
        l = l * f + sum;
        m = m_new;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            acc[d] *= f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = kb + 32 * h + 8 * g;
                const uint16_t* p = a.c.v + (size_t)max(vp[h], 0) * a.c.v_stride +
                                    ((size_t)(kvh * D + 16 * d + n) << a.c.shift) + (key & pmask);
                u4 v = *reinterpret_cast<const u4*>(p);
                if (!whole) {
                    // A masked position has weight zero, but zero times what an
                    // unwritten slot holds may be NaN: such values are cleared.
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool seen = key + e >= start && key + e < len && vp[h] >= 0;
                        if (!seen) w[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                    }
                    v = (u4){w[0], w[1], w[2], w[3]};
                }
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, v), pf[h], acc[d], 0, 0, 0);
            }
        }
    }
    l += lane_swap16(l);
    l += __shfl_xor(l, 32, 64);

    // Join the four waves in order.
    if (g == 0) {
        part_m[wave][n] = m;
        part_l[wave][n] = l;
    }
    if (n < nrows) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f4*>(&part_o[wave][n][16 * d + 4 * g]) = acc[d];
    }
    __syncthreads();
    const long slot = (long)it.slot + it.part;
    float* ws_o = a.workspace;
    float* ws_ml = a.workspace + (long)(target + a.rows) * a.heads * D;
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kDecodeThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = part_m[0][r];
#pragma unroll
        for (int w = 1; w < kDecodeWaves; ++w) top = fmaxf(top, part_m[w][r]);
        f4 o = {0, 0, 0, 0};
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kDecodeWaves; ++w) {
            const float f = part_weight(part_m[w][r], top);
            sum += part_l[w][r] * f;
            o += *reinterpret_cast<const f4*>(&part_o[w][r][d]) * f;
        }
        if (it.parts == 1) {
            const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            uint2 w;
            w.x = as_u32((h2){(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)});
            w.y = as_u32((h2){(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)});
            *reinterpret_cast<uint2*>(a.out + ((size_t)it.b * a.heads + head0 + r) * D + d) = w;
        } else {
            *reinterpret_cast<f4*>(ws_o + (slot * a.heads + head0 + r) * D + d) = o;
            if (d == 0) {
                ws_ml[(slot * a.heads + head0 + r) * 2] = top;
                ws_ml[(slot * a.heads + head0 + r) * 2 + 1] = sum;
            }
        }
    }
}

// Join of the parts of one sequence and head: one workgroup, each wave sums
// every fourth part, the waves are summed in order.
template <int D>
__global__ void __launch_bounds__(kDecodeThreads) attn_decode_join_kernel(AttnArgs a, int target) {
    __shared__ float acc[kDecodeWaves][D];
    __shared__ float sums[kDecodeWaves];
    const int b = blockIdx.x, head = blockIdx.y;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    // The sequence's parts; those of earlier sequences have the lower numbers.
    const int chunk = decode_chunk(a, target);
    int slot = 0, parts = 1;
    for (int b0 = 0; b0 <= b; b0 += 64) {
        int first, len, n = 0;
        if (b0 + lane <= b) {
            n = (decode_tiles(a, b0 + lane, first, len) + chunk - 1) / chunk;
            n = n > 0 ? n : 1;
        }
        if (b0 + 64 > b) parts = __shfl(n, b - b0, 64);
        for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d, 64);
        slot += n;
    }
    slot -= parts;
    if (parts == 1) return;
    const float* ws_o = a.workspace;
    const float* ws_ml = a.workspace + (long)(target + a.rows) * a.heads * D;
    float top = Q4_NEG_INF;
    for (int p = lane; p < parts; p += 64) top = fmaxf(top, ws_ml[((long)(slot + p) * a.heads + head) * 2]);
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    constexpr int PER = (D + 63) / 64;
    float o[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = 0.0f;
    float sum = 0.0f;
    for (int p = wave; p < parts; p += kDecodeWaves) {
        const long at = (long)(slot + p) * a.heads + head;
        const float f = part_weight(ws_ml[at * 2], top);
        sum += ws_ml[at * 2 + 1] * f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int d = lane + 64 * i;
            if (d < D) o[i] += ws_o[at * D + d] * f;
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lane + 64 * i < D) acc[wave][lane + 64 * i] = o[i];
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kDecodeThreads) {
        const float all = sums[0] + sums[1] + sums[2] + sums[3];
        const float inv = all > 0.0f || all != all ? 1.0f / all : 0.0f;
        const float v = (acc[0][d] + acc[1][d] + acc[2][d] + acc[3][d]) * inv;
        a.out[((size_t)b * a.heads + head) * D + d] = __builtin_bit_cast(uint16_t, (_Float16)v);
    }
}

int64_t attn_decode_workspace(int64_t batch, int heads, int dim) {
    // Parts: at most the wanted number and one more per sequence.
    return ((int64_t)kDecodeSlots + batch) * heads * (dim + 2) * (int64_t)sizeof(float);
}

template <int D>
static hipError_t launch_decode(const AttnArgs& a, hipStream_t st) {
    const int pairs = a.c.kv_heads * ((a.group + 15) / 16);
    const int target = decode_target(pairs);
    const long most = ((long)a.max_length + kTileKeys * kDecodeMinTiles - 1) / (kTileKeys * kDecodeMinTiles);
    const long grid = (long)target + a.rows < most * a.rows ? (long)target + a.rows : most * a.rows;
    const bool extra = a.softcap > 0.0f || a.slopes;
    if (extra)
        hipLaunchKernelGGL((attn_decode_kernel<D, true>), dim3((unsigned)grid, pairs), dim3(kDecodeThreads), 0, st, a,
                           target);
    else
        hipLaunchKernelGGL((attn_decode_kernel<D, false>), dim3((unsigned)grid, pairs), dim3(kDecodeThreads), 0, st, a,
                           target);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || most == 1) return e;
    hipLaunchKernelGGL((attn_decode_join_kernel<D>), dim3((unsigned)a.rows, a.heads), dim3(kDecodeThreads), 0, st, a,
                       target);
    return hipGetLastError();
}

hipError_t launch_attn_decode(const AttnArgs& a, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_decode<64>(a, st);
        case 96: return launch_decode<96>(a, st);
        case 128: return launch_decode<128>(a, st);
        case 192: return launch_decode<192>(a, st);
        case 256: return launch_decode<256>(a, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
