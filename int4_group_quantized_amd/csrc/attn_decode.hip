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
// Schedule: a wave has one tile's values and the next tile's keys on their way
// while it computes (32 KB per wave, two waves per SIMD up to dim 128).  With
// keys and values requested only when needed 64 sequences of 16,384 positions
// (2.15 GB) took 499 us, with this 357 us (6.0 TB/s); its read-only twin, the
// same loads without the arithmetic, takes 358 us, a one-shot read of such a pool
// runs at 7.0 TB/s.  One sequence of 2,000 positions takes 7.5 us, bound by the
// chain of dependent loads (lengths, table, keys, parts).
//
// Split: the visible tiles of all sequences are cut into parts of one length,
// computed on the device from the lengths so that uneven batches stay
// balanced: every workgroup gets one part of one sequence and kv head, its four
// waves take its tiles in turn.  512 parts (two workgroups per CU) measured
// best: 256 ran 1.3 times as long, 768 and 1,024 2% longer on that case and 20%
// on 16 uneven sequences.  The last part of a sequence to finish joins them in
// order; a second launch for that cost 2 to 3 us more.
#include "attn_softmax.hpp"

namespace q4 {

constexpr int kDecodeWaves = 4;
constexpr int kDecodeThreads = 64 * kDecodeWaves;
constexpr int kDecodeSlots = 512;   // workgroups wanted per launch: two per CU
static_assert(2 * kDecodeSlots <= kAttnCounters, "a counter for each sequence of several parts, and for each group");
// Parts of a sequence beyond which groups of kJoin are joined first: 128 parts of
// 131,072 positions 58.8 us without groups, 54.3 with them (75.1 and 56.9 for 64
// heads on one kv head); 32 parts of 8,000 positions 11.2 and 12.3.
constexpr int kDecodeGroups = 2 * kJoin;
constexpr int kDecodeGridY = 32768;  // parts per layer of the grid

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
    int split;    // sequences of several parts before this one
    int group;    // groups of kJoin parts before this sequence's
    int chunk;    // tiles per part
};

__host__ __device__ constexpr int decode_least(int dim) { return dim <= 128 ? 2 : 1; }

// Tiles per part: the total over `target`, the parts wanted per kv head and row
// block, rounded up, so that there are at most target + rows parts; and at least
// one tile per wave, except that where sequences average 3 to 32 tiles (above
// dim 128, 64) and CUs are idle they are cut finer (least: 2, above dim 128 1),
// which shortens the loads of a CU by more than the longer join costs: one
// sequence of 2,000 positions 7.4 us with two tiles per part, 8.7 with four; 2,772
// of dim 256 10.3 with one, 12.9 with four; eight of up to 300 7.4 and 8.9; but one
// of 130 6.4 with two, 5.8 with four, one of 8,000 of dim 64 15.8 and 11.2.
__device__ __forceinline__ int decode_chunk(int64_t total, int rows, int target, int least) {
    if (total > target || total <= 4 || total < 3 * (int64_t)rows || total > 64 / least * (int64_t)rows)
        least = kDecodeWaves;
    const float quotient = (float)total / (float)target;
    if (quotient > (float)(1 << 22)) return 1 << 26;  // more than any sequence has: one part each
    int c = max((int)quotient - 1, least);            // at most two below
    while ((int64_t)c * target < total) ++c;
    return c;
}

// Long parts, more than kDecodeLong tiles each: a sequence's shorter last part
// would leave more parts than workgroups that run at once, so parts are made
// longer until there are no more than `target` (the second try is nearly always
// enough), and a sequence's are then made alike.  Uneven sequences of up to 8,192
// positions, 64 of them: 113 us, 128 without, 119 made alike only; of dim 256 215
// and 241; 20 of up to 20,000 164 and 187.  With shorter parts it costs more than
// it gives: 16 of up to 4,096 17.1 us without, 17.5 with.
constexpr int kDecodeLong = 8;

// The part with number `item`; parts are numbered sequence by sequence.  Each
// wave computes it for itself.
__device__ __forceinline__ DecodePart decode_part(const AttnArgs& a, int item, int target, int least) {
    const int lane = threadIdx.x & 63;
    DecodePart r;
    r.b = -1;
    r.part = r.parts = r.slot = r.split = r.group = 0;
    if (a.rows == 1) {
        int first, len;
        const int n = decode_tiles(a, 0, first, len);
        r.chunk = decode_chunk(n, 1, target, least);
        r.parts = n > r.chunk ? (n + r.chunk - 1) / r.chunk : 1;
        r.part = item;
        if (item < r.parts) r.b = 0;
        return r;
    }
    int64_t total = 0;
    for (int b0 = 0; b0 < a.rows; b0 += 64) {
        int first, len;
        total += lane_scan(b0 + lane < a.rows ? decode_tiles(a, b0 + lane, first, len) : 0).last;
    }
    r.chunk = decode_chunk(total, a.rows, target, least);
    const bool even = total > kDecodeLong * (int64_t)target && 2 * a.rows <= target;
    for (int k = 0; even && k < 2; ++k) {
        int parts = 0;
        for (int b0 = 0; b0 < a.rows; b0 += 64) {
            int first, len, n = 0;
            if (b0 + lane < a.rows) n = max((decode_tiles(a, b0 + lane, first, len) + r.chunk - 1) / r.chunk, 1);
            parts += lane_scan(n).last;
        }
        if (parts <= target) break;
        r.chunk = (int)((int64_t)r.chunk * parts / target) + 1;
    }
    int before = 0;  // parts of earlier sequences
    for (int b0 = 0; b0 < a.rows; b0 += 64) {
        int first, len, tiles = 0, n = 0;
        if (b0 + lane < a.rows) {
            tiles = decode_tiles(a, b0 + lane, first, len);
            n = (tiles + r.chunk - 1) / r.chunk;
            n = n > 0 ? n : 1;  // an empty sequence has a part that writes zeros
        }
        const LaneScan s = lane_scan(n);
        const int groups = n > kDecodeGroups ? (n + kJoin - 1) / kJoin : 0;
        const LaneScan gs = lane_scan(groups);
        const uint64_t hit = __ballot(n > 0 && item < before + s.upto && item >= before + s.upto - n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            r.b = b0 + l;
            r.parts = __builtin_amdgcn_readlane(n, l);
            r.slot = before + __builtin_amdgcn_readlane(s.upto, l) - r.parts;
            r.part = item - r.slot;
            if (even) r.chunk = (__builtin_amdgcn_readlane(tiles, l) + r.parts - 1) / r.parts;
            r.split += __builtin_popcountll(__ballot(n > 1 && lane < l));
            r.group += __builtin_amdgcn_readlane(gs.upto - groups, l);
            return r;
        }
        r.split += __builtin_popcountll(__ballot(n > 1));
        r.group += gs.last;
        before += s.last;
    }
    return r;
}

__host__ __device__ inline int decode_target(int pairs) {
    const int t = kDecodeSlots / pairs;
    return t > 0 ? t : 1;
}

// Counters of finished parts, then partial outputs [parts][heads][dim], their
// maxima and sums [parts][heads][2].  A sequence of several parts has at least
// two tiles and more than total / target, so there are fewer than `target` of
// them, and target times the kv heads and row blocks is at most kDecodeSlots: the counters have
// one place whatever the shape, so calls of all shapes can share a workspace.
// Sequences of more than kDecodeGroups parts join them in groups of kJoin, a
// tenth as many as parts, with counters of their own.
struct DecodeWorkspace {
    float* o;
    float* ml;
    int* counters;
};

__device__ __forceinline__ DecodeWorkspace decode_workspace(const AttnArgs& a, int dim, int target) {
    const long slots = (long)(target + a.rows) * a.heads;
    DecodeWorkspace w;
    w.counters = reinterpret_cast<int*>(a.workspace);
    w.o = a.workspace + kAttnCounters;
    w.ml = w.o + slots * dim;
    return w;
}

// Four dimensions of an output row: o / sum in fp16, zeros where nothing was seen.
__device__ __forceinline__ void store_row(uint16_t* p, f4 o, float sum) {
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    uint2 w;
    w.x = as_u32((h2){(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)});
    w.y = as_u32((h2){(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)});
    *reinterpret_cast<uint2*>(p) = w;
}

__device__ __forceinline__ h8 load_h8(const uint16_t* p) {
    return __builtin_bit_cast(h8, *reinterpret_cast<const u4*>(p));
}

template <int D, int OPTIONS>
__global__ void __launch_bounds__(kDecodeThreads, D <= 128 ? 2 : 1) attn_decode_kernel(AttnArgs a, int target) {
    constexpr int OP = D + 4;  // pitch of a row of partial outputs in LDS
    __shared__ float part_o[kDecodeWaves][16][OP];
    __shared__ float part_m[kDecodeWaves][16], part_l[kDecodeWaves][16];
    // Kv heads and row blocks first, so that neighbouring workgroups read
    // neighbouring parts of the same pages at the same time.
    const int row_blocks = (a.group + 15) / 16;
    const int pairs = gridDim.x, pair = blockIdx.x;
    const int kvh = row_blocks == 1 ? pair : pair / row_blocks;
    const int row0 = (pair - kvh * row_blocks) * 16;   // first head of the group in this workgroup
    const int nrows = min(16, a.group - row0);
    const DecodePart it = decode_part(a, blockIdx.y + blockIdx.z * kDecodeGridY, target, decode_least(D));
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
    const ScoreParams sp = score_params<OPTIONS>(a, head0 + (n < nrows ? n : 0));

    f4 acc[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) acc[i] = (f4){0, 0, 0, 0};
    float m = Q4_NEG_INF, l = 0.0f;

    // Operands of one tile: K as A of the first product, V as A of the second.
    u4 kr[4][D / 32], vr[D / 16][2];
    // Pages of the 8-key groups that this lane's values and scores belong to
    // (vp) and that its keys belong to (kp), per 32-key block.  Positions past
    // the end take the last one's page.
    struct Ids {
        int v[2], k[2];
    };
    auto ids = [&](int t) {
        Ids r;
        const int kb = t * kTileKeys;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            r.v[h] = page_of(a.c, row, min(kb + 32 * h + 8 * g, len - 1));
            r.k[h] = page_of(a.c, row, min(kb + 32 * h + 8 * (n >> 2), len - 1));
        }
        return r;
    };
    auto load_k = [&](int t, const Ids& id) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int key = t * kTileKeys + 32 * (u >> 1) + 8 * (n >> 2) + 4 * (u & 1) + (n & 3);
            const uint16_t* p = a.c.k + (size_t)max(id.k[u >> 1], 0) * a.c.k_stride +
                                ((size_t)kvh * P + (key & pmask)) * D + 8 * g;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) kr[u][d] = *reinterpret_cast<const u4*>(p + 32 * d);
        }
    };
    auto load_v = [&](int t, const Ids& id) {
        // Both halves of a 128-byte line (a page of 64) are requested back to back.
        const uint16_t* p[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            p[h] = a.c.v + (size_t)max(id.v[h], 0) * a.c.v_stride + ((size_t)(kvh * D + n) << a.c.shift) +
                   ((t * kTileKeys + 32 * h + 8 * g) & pmask);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
#pragma unroll
            for (int h = 0; h < 2; ++h) vr[d][h] = *reinterpret_cast<const u4*>(p[h] + ((size_t)(16 * d) << a.c.shift));
        }
    };
    // One tile; K is in kr.  `next` requests the next tile's K as soon as kr is
    // free, so that it travels during the softmax and the second product.
    auto tile = [&](int t, const Ids& id, auto next) {
        const int kb = t * kTileKeys;
        load_v(t, id);
        __builtin_amdgcn_sched_barrier(0);
        f4 s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = (f4){0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < D / 32; ++d)
                s[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, kr[u][d]), qf[d], s[u], 0, 0, 0);
        }
        next();
        __builtin_amdgcn_sched_barrier(0);
        const bool whole = __all(kb >= start && kb + kTileKeys <= len && id.v[0] >= 0 && id.v[1] >= 0);
        // Scores; masked ones are -inf.
        float top = Q4_NEG_INF;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = kb + 32 * (u >> 1) + 8 * g + 4 * (u & 1) + i;
                float x = score<OPTIONS>(s[u][i], sp, key - (len - 1));
                if (!whole) x = key >= start && key < len && id.v[u >> 1] >= 0 ? x : Q4_NEG_INF;
                s[u][i] = x;
                top = top_of(top, x);
            }
        }
        top = top_of_halves(top_of_rows(top));
        const float m_new = fmaxf(m, top);
        const float base = m_new == Q4_NEG_INF ? 0.0f : m_new;
        const float f = exp2_hw(m - base);
        // The weights are summed as they enter the second product, rounded: they then
        // sum to one, and the mean of equal values is that value.
        h8 pf[2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pf[u >> 1][4 * (u & 1) + i] = (_Float16)exp2_hw(s[u][i] - base);
        }
        const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
        float sum = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum = __builtin_amdgcn_fdot2((h2){pf[h][2 * e], pf[h][2 * e + 1]}, one, sum, false);
        l = l * f + sum;
        m = m_new;
        if (!whole) {
            // A masked position has weight zero, but zero times what an unwritten
            // slot holds may be NaN: such values are cleared.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k0 = kb + 32 * h + 8 * g;
                const int from = id.v[h] < 0 ? 8 : start - k0, to = len - k0;
                uint32_t keep[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    keep[e] = (2 * e >= from && 2 * e < to ? 0x0000FFFFu : 0u) |
                              (2 * e + 1 >= from && 2 * e + 1 < to ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int d = 0; d < D / 16; ++d) vr[d][h] &= (u4){keep[0], keep[1], keep[2], keep[3]};
            }
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
            acc[d] *= f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, vr[d][h]), pf[h], acc[d], 0, 0, 0);
        }
    };

    int t = t_begin + wave;
    if (t < t_end) {
        Ids id = ids(t);
        load_k(t, id);
        for (; t + kDecodeWaves < t_end; t += kDecodeWaves) {
            const Ids after = ids(t + kDecodeWaves);
            tile(t, id, [&] { load_k(t + kDecodeWaves, after); });
            id = after;
        }
        tile(t, id, [] {});
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
    const DecodeWorkspace ws = decode_workspace(a, D, target);
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
            store_row(a.out + ((size_t)it.b * a.heads + head0 + r) * D + d, o, sum);
        } else {
            float* wo = ws.o + (slot * a.heads + head0 + r) * D + d;
            share_store(wo, o[0], o[1]);
            share_store(wo + 2, o[2], o[3]);
            if (d == 0) share_store(ws.ml + (slot * a.heads + head0 + r) * 2, top, sum);
        }
    }
    if (it.parts == 1) return;

    // The last workgroup of a sequence and row block to finish joins its parts,
    // in order, whichever it is.  It leaves the counter at zero for the next call.
    const long row_at = (long)it.slot * a.heads + head0;  // of the first part
    int parts = it.parts;
    long stride = a.heads;  // rows from part to part
    if (parts > kDecodeGroups) {
        // Many parts: groups of kJoin are joined first, each by its last workgroup,
        // into the place of the group's first part.
        const int first_part = it.part / kJoin * kJoin;
        if (!parts_done(ws.counters + kDecodeSlots + (it.group + it.part / kJoin) * pairs + pair,
                        min(kJoin, parts - first_part)))
            return;
        for (int r = wave; r < nrows; r += kDecodeWaves) {
            const long at = row_at + (long)first_part * a.heads + r;
            const JoinedRow<D> j = join_parts<D, true>(ws.o + at * D, ws.ml + at * 2, a.heads, min(kJoin, parts - first_part));
#pragma unroll
            for (int i = 0; i < JoinedRow<D>::PER; ++i) {
                const int d = 2 * (lane + 64 * i);
                if (d < D) share_store(ws.o + at * D + d, j.o[i].x, j.o[i].y);
            }
            if (lane == 0) share_store(ws.ml + at * 2, j.m, j.l);
        }
        parts = (parts + kJoin - 1) / kJoin;
        stride *= kJoin;
    }
    if (!parts_done(ws.counters + it.split * pairs + pair, parts)) return;
    for (int r = wave; r < nrows; r += kDecodeWaves)
        store_joined(join_parts<D, true>(ws.o + (row_at + r) * D, ws.ml + (row_at + r) * 2, stride, parts),
                     a.out + ((size_t)it.b * a.heads + head0 + r) * D);
}

int64_t attn_decode_workspace(int64_t batch, int heads, int dim) {
    // Parts: at most the wanted number and one more per sequence.
    return (((int64_t)kDecodeSlots + batch) * heads * (dim + 2) + kAttnCounters) * (int64_t)sizeof(float);
}

template <int D>
static hipError_t launch_decode(const AttnArgs& a, hipStream_t st) {
    const int pairs = a.c.kv_heads * ((a.group + 15) / 16);
    const int target = decode_target(pairs);
    const long most = ((long)a.max_length + kTileKeys * decode_least(D) - 1) / (kTileKeys * decode_least(D));
    const long grid = (long)target + a.rows < most * a.rows ? (long)target + a.rows : most * a.rows;
    const dim3 blocks(pairs, (unsigned)(grid < kDecodeGridY ? grid : kDecodeGridY),
                      (unsigned)((grid + kDecodeGridY - 1) / kDecodeGridY));
    const int options = attn_options(a);
    auto kernel = options == kNoOptions ? &attn_decode_kernel<D, kNoOptions>
                  : options == kOptions ? &attn_decode_kernel<D, kOptions>
                                        : &attn_decode_kernel<D, kLargeCapOptions>;
    hipLaunchKernelGGL(kernel, blocks, dim3(kDecodeThreads), 0, st, a, target);
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
