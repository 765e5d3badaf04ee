// New tokens over a cache: what they see, for the latent attention (latent_attn.hip)
// and that of drafted tokens (attn_tree.hip), and how the cached positions are shared
// out to the workgroups of the former.
//
// The n new tokens of a sequence are its last n cached positions, base .. base +
// n - 1.  Without masks token i sees every position up to base + i.  With masks it
// sees every position below base, and position base + k where bit k of its mask
// is set; its place is then base + (bits set) - 1, at least base, which for a tree of
// drafted tokens is base + its depth; windows and distances go by places.
#pragma once

#include "attn_softmax.hpp"

namespace q4 {

constexpr int kMaskTokens = 64;   // tokens that a mask can name

struct NewArgs {
    AttnArgs a;             // rows: new tokens of all sequences
    const uint64_t* masks;  // [rows], or NULL
    int max_new;            // most new tokens of a sequence that are served
    int target;             // parts wanted per row block
    int pairs;              // row blocks of a sequence, at most
};

struct NewSeq {
    int s;      // sequence, or -1
    int row;    // its first row
    int n;      // its rows
    int len;    // cached positions
    int base;   // position of its first new token (may be negative)
};

__device__ __forceinline__ NewSeq new_seq(const NewArgs& x, int s, int first, int last, int len) {
    NewSeq r;
    r.s = s;
    r.row = min(max(first, 0), x.a.rows);
    r.n = min(max(last, r.row), x.a.rows) - r.row;
    r.len = min(max(len, 0), x.a.max_length);
    r.base = r.len - r.n;
    return r;
}

// Its tiles of positions.
__device__ __forceinline__ int new_tiles(const NewSeq& q) { return q.n > 0 ? (q.len + kTileKeys - 1) / kTileKeys : 0; }

__device__ __forceinline__ int bits_of(uint64_t v) { return __builtin_popcountll(v); }

// Place of a token with this mask.
__device__ __forceinline__ int place_of(const NewSeq& q, uint64_t mask) { return q.base + max(bits_of(mask), 1) - 1; }

// What a row sees: positions lo <= j < hi, and base + k for the bits k of mask.
struct SeenRow {
    uint64_t mask;
    int lo, hi;
    int place;
};

// The first n bits.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0 : n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1;
}

__device__ __forceinline__ SeenRow seen_row(const uint64_t* masks, int window, const NewSeq& q, int token) {
    SeenRow r = {0, 0, 0, 0};
    if (token >= q.n) return r;
    if (masks) {
        const uint64_t* mine = masks + q.row;
        const uint64_t valid = low_bits(q.n);
        r.mask = mine[token] & valid;
        r.place = place_of(q, r.mask);
        r.hi = max(q.base, 0);
        if (window > 0 && window <= kMaskTokens) {
            // places differ by 63 at most
            for (int k = 0; k < min(q.n, kMaskTokens); ++k)
                if (place_of(q, mine[k] & valid) <= r.place - window) r.mask &= ~((uint64_t)1 << k);
        }
    } else {
        r.place = q.base + token;
        r.hi = max(r.place + 1, 0);
    }
    r.lo = window > 0 ? max(r.place + 1 - window, 0) : 0;
    return r;
}

// Which of the 64 positions from kb on the row sees.
__device__ __forceinline__ uint64_t seen_word(const SeenRow& r, int kb, int base) {
    uint64_t w = low_bits(r.hi - kb) & ~low_bits(r.lo - kb);
    const int d = kb - base;  // bit d of the mask is position kb
    if (d >= 0 && d < 64) w |= r.mask >> d;
    if (d < 0 && d > -64) w |= r.mask << -d;
    return w;
}

// A workgroup's part of one sequence's tiles, for one block of its rows.
struct NewPart {
    NewSeq q;
    int part;     // of the sequence
    int parts;    // parts of the sequence
    int slot;     // workspace slot of its first part, if it has several
    int block;    // of the sequence's rows
    int t_begin, t_end;
};

// Tiles of a part: the total over `target`, rounded up, so that there are at most
// target + (sequences of several parts) parts of such sequences.
__device__ __forceinline__ int new_chunk(int64_t total, int target) {
    const float quotient = (float)total / (float)target;
    if (quotient > (float)(1 << 22)) return 1 << 26;  // more than any sequence has
    int c = max((int)quotient - 1, 1);                // at most two below
    while ((int64_t)c * target < total) ++c;
    return c;
}

// Parts and row blocks of a sequence.  One with new tokens but no positions has a part,
// which writes zeros.  A sequence of several parts has more than total / target tiles,
// so there are fewer than `target` of them, with fewer than 2 target parts.
struct NewShare {
    int parts, blocks;
};
__device__ __forceinline__ NewShare new_share(const NewArgs& x, const NewSeq& q, int chunk, int rows) {
    NewShare r;
    r.parts = q.n == 0 ? 0 : max((new_tiles(q) + chunk - 1) / chunk, 1);
    r.blocks = (min(q.n, x.max_new) * x.a.heads + rows - 1) / rows;
    return r;
}

// Workgroups are dealt to the eight XCDs in turn.  Of `total` items each XCD takes a
// run, so that neighbours, the row blocks of one part, share an L2.  -1: none left.
__device__ __forceinline__ int new_item(int total) {
    const int g = (int)(blockIdx.x + blockIdx.y * gridDim.x), per = (total + 7) / 8, item = (g & 7) * per + (g >> 3);
    return (g >> 3) < per && item < total ? item : -1;
}

// The sequences of a call, 64 at a time, one per lane; the first 64 are read once.
struct NewSeqs {
    const NewArgs& x;
    NewSeq first;
    __device__ __forceinline__ NewSeq read(int s) const {
        NewSeq q = {-1, 0, 0, 0, 0};
        if (s < x.a.count) q = new_seq(x, s, x.a.q_starts[s], x.a.q_starts[s + 1], x.a.lengths[s]);
        return q;
    }
    __device__ __forceinline__ explicit NewSeqs(const NewArgs& args) : x(args), first(read(threadIdx.x & 63)) {}
    __device__ __forceinline__ NewSeq operator()(int s0) const { return s0 == 0 ? first : read(s0 + (int)(threadIdx.x & 63)); }
    // Tiles of a part.
    __device__ __forceinline__ int chunk() const {
        int64_t total = 0;
        for (int s0 = 0; s0 < x.a.count; s0 += 64) total += lane_scan(new_tiles((*this)(s0))).last;
        return new_chunk(total, x.target);
    }
};

__device__ __forceinline__ NewSeq new_seq_of(const NewSeq& q, int l) {
    const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
    return {of(q.s), of(q.row), of(q.n), of(q.len), of(q.base)};
}

// What the workgroup does, in blocks of `rows` rows; each wave computes it for itself.
// Items are numbered sequence by sequence, part by part, row block by row block.
__device__ __forceinline__ NewPart new_part(const NewArgs& x, int rows) {
    const AttnArgs& a = x.a;
    NewPart r;
    r.q.s = -1;
    r.part = r.parts = r.slot = r.block = r.t_begin = r.t_end = 0;
    const auto set = [&](const NewSeq& q, const NewShare& s, int number) {
        r.q = q;
        r.parts = s.parts;
        r.part = number / s.blocks;
        r.block = number - r.part * s.blocks;
        // Alike parts: the last one is no shorter than it has to be.
        const int tiles = new_tiles(q), per = (tiles + r.parts - 1) / r.parts;
        r.t_begin = r.part * per;
        r.t_end = min(tiles, r.t_begin + per);
    };
    if (a.count == 1) {
        const auto of = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        const int first = of(a.q_starts[0]), last = of(a.q_starts[1]), len = of(a.lengths[0]);
        const NewSeq q = new_seq(x, 0, first, last, len);
        const NewShare s = new_share(x, q, new_chunk(new_tiles(q), x.target), rows);
        const int item = new_item(s.parts * s.blocks);
        if (item >= 0) set(q, s, item);
        return r;
    }
    const NewSeqs seqs(x);
    const int chunk = seqs.chunk();
    const auto items_of = [&](const NewSeq& q) {
        const NewShare s = new_share(x, q, chunk, rows);
        return s.parts * s.blocks;
    };
    const LaneScan scan0 = lane_scan(items_of(seqs.first));
    int total = scan0.last;
    for (int s0 = 64; s0 < a.count; s0 += 64) total += lane_scan(items_of(seqs(s0))).last;
    const int item = new_item(total);
    if (item < 0) return r;
    int before = 0;  // items of earlier sequences
    for (int s0 = 0; s0 < a.count; s0 += 64) {
        const NewSeq q = seqs(s0);
        const NewShare s = new_share(x, q, chunk, rows);
        const int n = s.parts * s.blocks;
        const LaneScan scan = s0 == 0 ? scan0 : lane_scan(n), several = lane_scan(s.parts > 1 ? s.parts : 0);
        const uint64_t hit = __ballot(n > 0 && item < before + scan.upto && item >= before + scan.upto - n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            r.slot += of(several.upto - (s.parts > 1 ? s.parts : 0));
            set(new_seq_of(q, l), {of(s.parts), of(s.blocks)}, item - (before + of(scan.upto - n)));
            return r;
        }
        r.slot += several.last;
        before += scan.last;
    }
    return r;
}

// For the second launch: a sequence of several parts, and the workgroup's first row of
// it, `each` rows a workgroup.  q.s is -1 where there is nothing to do.
struct NewParts {
    NewSeq q;
    int parts, slot, row0;
};
__device__ __forceinline__ NewParts new_parts(const NewArgs& x, int each) {
    const AttnArgs& a = x.a;
    NewParts r;
    r.q.s = -1;
    r.parts = r.slot = r.row0 = 0;
    const int item = (int)(blockIdx.x + blockIdx.y * gridDim.x);
    const NewSeqs seqs(x);
    const int chunk = seqs.chunk();
    int before = 0;
    for (int s0 = 0; s0 < a.count; s0 += 64) {
        const NewSeq q = seqs(s0);
        const NewShare s = new_share(x, q, chunk, each);
        const int n = s.parts > 1 ? s.blocks : 0;
        const LaneScan scan = lane_scan(n), several = lane_scan(s.parts > 1 ? s.parts : 0);
        const uint64_t hit = __ballot(n > 0 && item < before + scan.upto && item >= before + scan.upto - n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            r.q = new_seq_of(q, l);
            r.parts = of(s.parts);
            r.slot += of(several.upto - (s.parts > 1 ? s.parts : 0));
            r.row0 = (item - (before + of(scan.upto - n))) * each;
            return r;
        }
        r.slot += several.last;
        before += scan.last;
    }
    return r;
}

// Workgroups of the two launches, at most: row blocks of all sequences, and of those in
// several parts for each part.
inline long new_blocks(const NewArgs& x, int rows) {
    const long most = ((long)x.max_new * x.a.heads + rows - 1) / rows * x.a.count;  // every sequence as long as it may be
    const long all = (long)x.a.rows * x.a.heads / rows + x.a.count;
    return most < all ? most : all;
}
inline long new_items(const NewArgs& x, int rows, long tiles) {
    const long most = ((long)x.target + x.a.count < tiles * x.a.count ? (long)x.target + x.a.count : tiles * x.a.count) * x.pairs;
    const long all = new_blocks(x, rows) + (x.target > 1 ? 2L * x.target * x.pairs : 0);
    return most < all ? most : all;
}
inline dim3 new_grid(long n) {
    constexpr long X = 1 << 20;
    n = (n + 7) / 8 * 8;
    return dim3((unsigned)(n < X ? n : X), (unsigned)((n + X - 1) / X));
}

// Partial results: outputs [slots][pairs][R][dim], their maxima and sums
// [slots][pairs][R][2], R rows of a workgroup, behind the counters of the decode call
// (so that both can share a workspace).  There are fewer than 2 target slots; with a
// target of one nothing is split.
struct NewWorkspace {
    float* o;
    float* ml;
};

__host__ __device__ inline long new_slots(int target) { return target > 1 ? 2 * (long)target : 0; }

__device__ __forceinline__ NewWorkspace new_workspace(const NewArgs& x, int pairs, int rows, int dim) {
    NewWorkspace w;
    w.o = x.a.workspace + kAttnCounters;
    w.ml = w.o + new_slots(x.target) * pairs * rows * dim;
    return w;
}

inline int64_t new_workspace_bytes(int target, long pairs, int rows, int dim) {
    return (new_slots(target) * pairs * rows * (dim + 2) + kAttnCounters) * (int64_t)sizeof(float);
}

// Join, by a second launch: a workgroup for RW rows of one sequence, of `rows` in all.  Weights first, a thread for each row and part, then four columns of a
// row for each thread, all of its parts' requested together; where that leaves
// threads, several take parts of one four.
//   at(slot, row): place of the row in part `slot`; stride: from part to part, rows
//   out(q, row): the output row
constexpr int kJoinThreads = 256;
// PARTS: most parts of a sequence, the launch's target and one.
template <int D, int RW, int PARTS>
struct JoinShared {
    static constexpr int ITEMS = RW * (D / 4);
    static constexpr int GROUPS = ITEMS >= kJoinThreads ? 1 : kJoinThreads / ITEMS;
    float2 ml[RW][PARTS];  // maxima and sums; then weights
    float sum[RW];
    f4 part[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? ITEMS : 1];
};
template <int D, int RW, int PARTS, class At, class Out>
__device__ __forceinline__ void join_rows(JoinShared<D, RW, PARTS>& sh, const NewWorkspace& ws, const NewParts& p, int rows, long stride,
                                          At at, Out out) {
    using Shared = JoinShared<D, RW, PARTS>;
    constexpr int ITEMS = Shared::ITEMS, GROUPS = Shared::GROUPS, PER = (ITEMS + kJoinThreads - 1) / kJoinThreads;
    const int tid = threadIdx.x, parts = p.parts, row0 = p.row0;
    const int n = min(RW, rows - row0);
    for (int i = tid; i < n * parts; i += kJoinThreads) {
        const int r = i / parts, k = i % parts;
        sh.ml[r][k] = *reinterpret_cast<const float2*>(ws.ml + (at(p.slot, row0 + r) + k * stride) * 2);
    }
    __syncthreads();
    for (int r = tid >> 6; r < n; r += kJoinThreads / 64) {
        const int lane = tid & 63;
        float top = Q4_NEG_INF, sum = 0.0f;
        for (int k = lane; k < parts; k += 64) top = fmaxf(top, sh.ml[r][k].x);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        for (int k = lane; k < parts; k += 64) {
            const float2 v = sh.ml[r][k];
            const float w = part_weight(v.x, top);
            sum += v.y * w;
            sh.ml[r][k].x = w;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (lane == 0) sh.sum[r] = sum;
    }
    __syncthreads();
    const int group = GROUPS > 1 ? tid / ITEMS : 0, first = GROUPS > 1 ? tid % ITEMS : tid;
    f4 acc[PER];
    const float* from[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int item = first + j * kJoinThreads, r = min(item / (D / 4), n - 1);
        acc[j] = (f4){0, 0, 0, 0};
        from[j] = ws.o + at(p.slot, row0 + r) * D + item % (D / 4) * 4;
    }
    constexpr int UNROLL = PER >= 4 ? 2 : 8;
    if (group < GROUPS) {
        for (int k0 = group; k0 < parts; k0 += GROUPS * UNROLL) {
            f4 v[UNROLL][PER];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int k = k0 + u * GROUPS;
                    v[u][j] = (f4){0, 0, 0, 0};
                    if (k < parts) v[u][j] = *reinterpret_cast<const f4*>(from[j] + k * stride * D);
                }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int k = k0 + u * GROUPS, r = min((first + j * kJoinThreads) / (D / 4), n - 1);
                    if (k < parts) acc[j] += v[u][j] * sh.ml[r][k].x;
                }
        }
    }
    if constexpr (GROUPS > 1) {
        if (group < GROUPS) sh.part[group][first] = acc[0];
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) acc[0] += sh.part[g][first];
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int item = first + j * kJoinThreads, r = item / (D / 4);
        if (r >= n) continue;
        const float sum = sh.sum[r], inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        uint2 w;
        w.x = as_u32((h2){(_Float16)(acc[j][0] * inv), (_Float16)(acc[j][1] * inv)});
        w.y = as_u32((h2){(_Float16)(acc[j][2] * inv), (_Float16)(acc[j][3] * inv)});
        *reinterpret_cast<uint2*>(out(p.q, row0 + r) + item % (D / 4) * 4) = w;
    }
}

// Rows of a workgroup of the second launch: as many as leave two workgroups per CU.
inline int join_rows_per_group(long rows) { return rows >= 16 * 512 ? 16 : rows >= 4 * 512 ? 4 : 1; }

// Whether there may be parts to join at all.
inline bool new_second(const NewArgs& x, long tiles) { return x.target > 1 && tiles > 1; }

}  // namespace q4
