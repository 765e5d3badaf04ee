// Attention of prompt tokens over the paged cache (gfx950).
//
//   out[t][h] = sum_j softmax_j(s(q[t][h] . k_j)) v_j  over the positions j that
//   token t sees: causal, its own sequence only, optionally within a window or
//   with a prefix that every token sees.
//
// A workgroup of four or eight waves serves 128 query rows of one kv head, or 64
// where that leaves CUs idle: the tokens of one tile times the heads of the group
// (row = token * group + head), so that every key and value read serves the whole
// group.  One pass over the
// visible tiles of 64 positions keeps the running maximum and sum of the
// softmax; scores and outputs stay in registers.
//
// Products with v_mfma_f32_32x32x16_f16, 32 rows per wave:
//   S^T[key][row] = K Q^T     A = K rows from LDS, B = the query rows, in registers
//   O^T[dim][row] = V^T P^T   A = V pages' rows from LDS, B = P^T
// The result of the first (lane: row = lane & 31, h = lane >> 5, register r:
// matrix row 4h + r%4 + 8(r/4)) is the operand of the second (k = 8h + j of
// each 16) as it stands when matrix row m of a 32-key block loads key
// 16(m/16) + 8(m/4%2) + 4(m/8%2) + m%4: register r then is key 16(r/8) + 8h + r%8.
//
// Dimensions 192 and 256: one wave's outputs and queries of 32 rows take most of
// the registers, so two waves share the rows (SHARE = 2); so they do in
// workgroups of 64 rows, to be done sooner.  Each takes half of a tile's keys in the first product and half of the output
// dimensions in the second; between them the weights meet in LDS, with the
// maximum they were taken from.  4,096 tokens of 16 heads of 256 (4 kv heads)
// take 191 us, with one wave per SIMD 214; 3,044 tokens of five sequences, 8
// heads on one kv head, with a distance bias, 46 and 85.  128 rows by eight waves
// at dim 64 and 128, one workgroup per CU: 5 to 15% slower than by four.
//
// Bound by the matrix cores and the softmax's vector work together: 8,192 tokens
// of 32 heads of 128 (8 kv heads, 550 GFLOP) take 555 us call after call, 990
// TFLOP/s (580 to 670 in the first calls after a pause, while the clock settles);
// a counter run had the matrix cores busy 53% of the cycles.  Without either
// product, the loads or the exponentials it would be 2 to 15% less, with half of
// the LDS operand reads 3%.  Few tokens are bound by latency: 34 tokens take 6.4 us.
//
// Tiles go straight from memory into LDS images, one ahead with two images (two
// workgroups per CU) and up to three ahead with four (one per CU, where there are
// not more); staged through registers the case above took 2,020 us.  A wave's
// loads are spread over the first product, where a tile lies in one page: at
// once they hold it up for 400 to 700 cycles (2 to 4% of a prompt's time).  LDS
// rows are swizzled so that an operand load's rows fall on different banks
// (k_chunk).
//
// Few tokens on a long cache leave most CUs idle, so the visible tiles are
// then cut into equal splits joined by a second launch (prefill_split).
#include "attn_softmax.hpp"

#include <cmath>
#include <type_traits>

namespace q4 {

typedef float f16v __attribute__((ext_vector_type(16)));

// Waves that share 32 of a workgroup's rows, and threads of a workgroup.
__host__ __device__ constexpr int prefill_share(int dim, int rows) { return dim > 128 || rows == 64 ? 2 : 1; }
__host__ __device__ constexpr int prefill_threads(int dim, int rows) { return 2 * rows * prefill_share(dim, rows); }
constexpr int kPrefillAlone = 256;      // workgroups that have a CU to themselves
constexpr double kSecondLaunch = 4.0;   // us, launch and join of short partial results
constexpr double kJoinRound = 1.0;      // us, each further kJoin of them
// Tokens per workgroup.
static int prefill_tokens(int rows, int group) { return rows / group; }

static long prefill_tiles(long tokens, long count, int rows, int group) {
    const int tb = prefill_tokens(rows, group);
    const long a = tokens / tb + count;  // sum of ceil(n_s / tb) at most
    return a < tokens ? a : tokens;      // each tile has a token
}

// How a call is cut up.
struct PrefillPlan {
    int rows;     // query rows of a workgroup
    int splits;   // of the positions
    double time;  // estimate, us
};

// Splits of the positions.  A workgroup alone on its CU takes a time c per tile
// (1.1, 1.4 and 2.3 us at dim 64, 128 and 256; 85% of that with 64 rows); n
// splits of L tiles take c L / n, the second launch, its rounds of kJoin parts
// and n times what writing and reading one partial output per row costs (v, at
// about 4 TB/s): least at n = sqrt(c L / v), or where the last round is full.
// Measured, dim 128, 16 heads: 34 tokens on 8,000 positions 20.7 us with 32
// splits, 23.9 with 63, 25.1 with 16; 300 tokens on 720 19.8 with 4, 22.1 with
// 8, 28.5 whole; 20 tokens on 740 22.3 whole, 14.4 with 3, 12.0 with 6; 40
// tokens of 8 heads on 8,000 18.6 with 42, 16.4 with 32.  A second launch taken
// for 5 us left 100 tokens on 300 whole (13.2 us, 11.5 split), for 3 it split
// 1,000 tokens (30.3 us, 24.1 whole).
static PrefillPlan prefill_split(int rows, long blocks, long length, long tokens, int heads, int dim) {
    // Beyond dim 128 a CU's LDS holds one workgroup: 128 tokens of 16 heads of 256 on
    // 4,000 positions take 33 us in 256 workgroups, 44 in 512.
    const long room = (dim > 128 ? 1 : 2) * kPrefillAlone / blocks, most = room < length ? room : length;
    const double c = (0.6 + dim / 150.0) * (rows == 64 ? 0.85 : 1.0), v = 8e-6 / 4.0 * (double)tokens * heads * dim;
    PrefillPlan plan = {rows, 1, c * (double)length};
    if (most < 2) return plan;
    long n = (long)(std::sqrt(c * (double)length / v) + 0.5);
    n = n < 1 ? 1 : n > most ? most : n;
    for (const long want : {n, (n - 1) / kJoin * kJoin}) {
        if (want < 2) continue;
        const long per = (length + want - 1) / want;
        const long made = (length + per - 1) / per;  // as many as that many tiles each make
        const double time =
            c * (double)per + v * (double)made + kSecondLaunch + kJoinRound * (double)((made - 1) / kJoin);
        if (time < plan.time) plan = {rows, (int)made, time};
    }
    return plan;
}

// 64 or 128 rows.  Where workgroups of 64 rows have a CU each, a tile takes them
// less time than those of 128 (two waves share 32 rows instead of one): 1,000
// tokens of 16 heads of 128 23.7 against 27.7 us, 34 tokens 6.5 against 7.4.
// They read the keys and values twice as often, and leave room for fewer
// splits: 200 tokens of 32 heads on 4,000 positions 38.3 against 34.0.  So a
// call that would be split takes them only with up to 64 workgroups (16 tokens
// on 16,000 positions 19.9 against 21.3; 34 tokens of 32 heads on 4 kv heads
// on 8,000 24.0 against 27.2).
static PrefillPlan prefill_plan(long tokens, long count, int heads, int kv_heads, int dim, long max_length) {
    const int group = heads / kv_heads;
    const long length = (max_length + kTileKeys - 1) / kTileKeys;
    const long large = prefill_tiles(tokens, count, 128, group) * kv_heads;
    const long small = prefill_tiles(tokens, count, 64, group) * kv_heads;
    const PrefillPlan plan = prefill_split(128, large, length, tokens, heads, dim);
    if (dim == 96 || small > (plan.splits > 1 ? kPrefillAlone / 4 : kPrefillAlone)) return plan;
    return prefill_split(64, small, length, tokens, heads, dim);
}

int64_t attn_prefill_workspace(int64_t tokens, int64_t count, int heads, int kv_heads, int dim, int64_t max_length) {
    const int splits = prefill_plan(tokens, count, heads, kv_heads, dim, max_length).splits;
    // The counters of the decode call come first, so that both can share one.
    return splits == 1 ? 0 : ((int64_t)splits * tokens * heads * (dim + 2) + kAttnCounters) * (int64_t)sizeof(float);
}

struct PrefillTile {
    int s;       // sequence, or -1
    int token;   // first token of the tile (row of q)
    int n;       // tokens in the tile
    int pos;     // position of the first token (may be negative)
    int len;     // positions of the sequence
    int prefix;  // positions that all of its tokens see
};

// x / a.tile rounded up, x < 2^21: the quotient of x - 1/2 keeps 1 / 256 from
// every whole number, four times its error.
__device__ __forceinline__ int prefill_tiles_of(const AttnArgs& a, int x) {
    return (int)(((float)(x + a.tile) - 0.5f) * a.inv_tile);
}

// Tile t of the `tiles` of sequence s, whose rows are first .. last - 1.  A
// sequence's last tokens, which see the most positions, come first.
__device__ __forceinline__ PrefillTile prefill_tile_of(const AttnArgs& a, int s, int first, int last, int len,
                                                       int prefix, int tiles, int t) {
    const int at = (tiles - 1 - t) * a.tile;
    PrefillTile r;
    r.s = s;
    r.token = first + at;
    r.n = min(a.tile, last - r.token);
    r.len = min(max(len, 0), a.max_length);
    r.pos = r.len - (last - first) + at;
    r.prefix = prefix;
    return r;
}

// Tile number `item`.  A sequence's length and prefix are read with its rows,
// not after them (readfirstlane and the empty assembly keep the compiler from
// moving the reads to where they are needed: 0.1 to 0.3 us).
__device__ __forceinline__ PrefillTile prefill_tile(const AttnArgs& a, int item) {
    const int lane = threadIdx.x & 63;
    PrefillTile none;
    none.s = -1;
    none.token = none.n = none.pos = none.len = none.prefix = 0;
    if (a.count == 1) {
        const auto of = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        const int first = of(a.q_starts[0]), last = of(a.q_starts[1]), len = of(a.lengths[0]);
        const int prefix = a.prefix ? of(a.prefix[0]) : 0;
        const int st = min(max(first, 0), a.rows), en = min(max(last, st), a.rows);
        const int n = prefill_tiles_of(a, en - st);
        return item < n ? prefill_tile_of(a, 0, st, en, len, prefix, n, item) : none;
    }
    int before = 0;
    for (int s0 = 0; s0 < a.count; s0 += 64) {
        int st = 0, en = 0, len = 0, prefix = 0;
        if (s0 + lane < a.count) {
            st = a.q_starts[s0 + lane];
            en = a.q_starts[s0 + lane + 1];
            len = a.lengths[s0 + lane];
            if (a.prefix) prefix = a.prefix[s0 + lane];
        }
        asm volatile("" : "+v"(st), "+v"(en), "+v"(len), "+v"(prefix));
        st = min(max(st, 0), a.rows);
        en = min(max(en, st), a.rows);
        const int n = prefill_tiles_of(a, en - st);
        const LaneScan c = lane_scan(n);
        const uint64_t hit = __ballot(n > 0 && item < before + c.upto && item >= before + c.upto - n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            return prefill_tile_of(a, s0 + l, of(st), of(en), of(len), of(prefix), of(n),
                                   item - (before + of(c.upto) - of(n)));
        }
        before += c.last;
    }
    return none;
}

// Chunk of 16 bytes (eight halves) c of K row `key`, and of V row `dim`, in a
// tile's LDS image: K [64][D / 8], V [D][8] behind it.  LDS serves 16 lanes of a
// 16-byte read at a time from 64 banks, so the 16 rows n .. n + 15 of an operand
// (n: matrix row, see above) have to fall on different sixteenths of 256 bytes:
// the part of n that the row pitch does not already spread is exclusive-ored
// into the chunk.  With the permutation over 128 bytes only, half of the LDS
// cycles were conflicts.
template <int D>
__device__ __forceinline__ int k_chunk(int key, int c) {
    const int n = (key & 3) | ((key >> 1) & 4) | ((key << 1) & 8);  // matrix row, low four bits
    constexpr int SHIFT = D % 128 == 0 ? 0 : D % 64 == 0 ? 1 : 2;   // pitch 256 or 512, 128 or 384, 192 bytes
    return key * (D / 8) + (c ^ (n >> SHIFT));
}
template <int D>
__device__ __forceinline__ int v_chunk(int dim, int c) {
    return kTileKeys * (D / 8) + dim * (kTileKeys / 8) + (c ^ ((dim >> 1) & 7));
}

__device__ __forceinline__ h8 as_h8(u4 v) { return __builtin_bit_cast(h8, v); }

// Halves of a dword whose exponent is all ones (infinite or NaN), as bits 0 and 16.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return (((w & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u;
}

// Token `tok` of a tile sees positions lo <= j < hi.
struct Seen {
    int lo, hi;
};
__device__ __forceinline__ Seen prefill_sees(const AttnArgs& a, const PrefillTile& it, int prefix, int tok) {
    const int pos = it.pos + tok;
    if (tok >= it.n || pos < 0) return {0, 0};
    return {a.window > 0 ? max(pos + 1 - a.window, 0) : 0, min(max(pos + 1, prefix), it.len)};
}

// Row r of a tile, r < 128.  Rows that the tile does not have are not live.
struct PrefillRow {
    int token, head, pos;
    Seen see;
    bool live;
};

// r / group: the quotient of r + 1/2 keeps 1 / 128 from every whole number.
__device__ __forceinline__ int prefill_token_of(const AttnArgs& a, int r) {
    return (int)(((float)r + 0.5f) * a.inv_group);
}

__device__ __forceinline__ PrefillRow prefill_row(const AttnArgs& a, const PrefillTile& it, int prefix, int kvh, int r) {
    PrefillRow q;
    const int tok = prefill_token_of(a, r);
    q.live = tok < it.n;
    q.head = kvh * a.group + (q.live ? r - tok * a.group : 0);
    q.token = it.token + (q.live ? tok : 0);
    q.pos = it.pos + tok;
    q.see = prefill_sees(a, it, prefix, tok);
    return q;
}

// A wave's 32 rows over positions [k_begin, k_end), one position after the
// other, never touching what a row does not see: for tiles that hold infinities
// or NaN in masked places, where the matrix products would multiply them by
// zero.  Lanes n and n + 32 share row n, half the dimensions each (waves that share
// it split the output dimensions too).  Far slower; all waves of a workgroup that
// has met such a tile start their rows again here, after the fast loop and with
// nothing of it live, because the same handling inside that loop cost it 100
// registers (8,192 tokens of 32 heads: 865 us with it inside, 740 us with it here).
template <int D, int OPTIONS, int SHARE>
__device__ __forceinline__ void prefill_rows_one_by_one(const AttnArgs& a, const PrefillTile& it, int prefix,
                                                        int split, int kvh, int wave, int k_begin, int k_end) {
    constexpr int OUT = D / (2 * SHARE);  // output dimensions of a lane
    const int lane = threadIdx.x & 63, n = lane & 31, d0 = (lane >> 5) * (D / 2);
    const int o0 = (2 * (wave % SHARE) + (lane >> 5)) * OUT;
    const PrefillRow q = prefill_row(a, it, prefix, kvh, wave / SHARE * 32 + n);
    const ScoreParams sp = score_params<OPTIONS>(a, q.head);
    const _Float16* qp = reinterpret_cast<const _Float16*>(a.q) + ((size_t)q.token * a.heads + q.head) * D + d0;
    const int* row = a.c.table + (size_t)it.s * a.c.cols;
    const int pmask = (1 << a.c.shift) - 1;
    float acc[OUT];
#pragma unroll
    for (int i = 0; i < OUT; ++i) acc[i] = 0.0f;
    float m = Q4_NEG_INF, l = 0.0f;
    for (int key = k_begin; key < min(k_end, it.len); ++key) {
        const int page = page_of(a.c, row, key);
        if (page < 0) continue;
        const _Float16* kp = reinterpret_cast<const _Float16*>(a.c.k) + (size_t)page * a.c.k_stride +
                             (((size_t)kvh << a.c.shift) + (key & pmask)) * D + d0;
        const _Float16* vp = reinterpret_cast<const _Float16*>(a.c.v) + (size_t)page * a.c.v_stride +
                             ((size_t)(kvh * D + o0) << a.c.shift) + (key & pmask);
        float dot = 0.0f;
#pragma unroll 4
        for (int i = 0; i < D / 2; ++i) dot = __builtin_fmaf((float)qp[i], (float)kp[i], dot);
        dot += __shfl_xor(dot, 32, 64);
        if (key < q.see.lo || key >= q.see.hi) continue;
        const float s = score<OPTIONS>(dot, sp, key - q.pos);
        const float m_new = fmaxf(m, s), base = m_new == Q4_NEG_INF ? 0.0f : m_new;
        const float f = exp2_hw(m - base), p = exp2_hw(s - base);
        l = l * f + p;
        m = m_new;
#pragma unroll
        for (int i = 0; i < OUT; ++i) acc[i] = acc[i] * f + p * (float)vp[(size_t)i << a.c.shift];
    }
    if (!q.live) return;
    const long at = ((long)split * a.rows + q.token) * a.heads + q.head;
    float* po = a.workspace + kAttnCounters + at * D + o0;
    _Float16* op = reinterpret_cast<_Float16*>(a.out) + ((size_t)q.token * a.heads + q.head) * D + o0;
    const bool partial = a.splits > 1;
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
        if (partial) po[i] = acc[i];
        else op[i] = (_Float16)(acc[i] * inv);
    }
    if (partial && o0 == 0) {
        float* ml = a.workspace + kAttnCounters + (long)a.splits * a.rows * a.heads * D + at * 2;
        ml[0] = m;
        ml[1] = l;
    }
}

// 16 bytes per lane from memory into LDS: lane i's to byte `to` + 16 i.  In
// assembly because the compiler, which sees that images follow each other in
// one array, would let every LDS read wait for all such loads under way; the
// waits are wait_and_meet's.  The instruction has no destination register.  m0, a
// reserved register, cannot be declared as overwritten; nothing else in these
// kernels uses it, which tests/test_attention_assembly.py checks.
// First form: from base + the lane's offset in bytes, base the same in all lanes.
// A vector instruction may have written base just before (a value read from a
// lane, a spilled one too), and the compiler does not look into the assembly: the
// five wait states that a memory operation then needs are the move's and the
// no-operation's.  They cost 0.3% of 8,192 tokens' time, 1.6% at dim 64.
__device__ __forceinline__ void load_lds(const uint16_t* base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(offset), "s"(base)
                 : "memory");
}
// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint16_t* uniform(const uint16_t* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint16_t*)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void load_lds(const uint16_t* p, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(to), "v"(p) : "memory");
}

// Waits until at most NEWER of this wave's vector memory operations (which
// complete in order) and none of its LDS operations are under way, then for the
// workgroup.
template <int NEWER>
__device__ __forceinline__ void wait_and_meet() {
    static_assert(NEWER < 64, "the counter has six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((NEWER & 15) | 0x70 | (NEWER >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// LDS of a workgroup behind its images.
template <int WAVES, bool SHARED>
struct PrefillShared {
    u4 weights[SHARED ? WAVES : 0][2][64];  // a wave's half of a tile's weights, as operands
    float base[SHARED ? WAVES : 0][32];     // and the maximum that they were taken from
    float sum[SHARED ? WAVES : 0][32];      // a wave's share of the rows' sums
    int found[WAVES];                       // a wave has seen infinities or NaN where a row is masked
};

// The same for LDS operations only.
__device__ __forceinline__ void lds_meet() {
    asm volatile("" ::: "memory");
    lds_barrier();
    asm volatile("" ::: "memory");
}

template <int D, int OPTIONS, int ROWS>
__global__ void __launch_bounds__(prefill_threads(D, ROWS), D > 128 && ROWS == 64 ? 1 : 2)
    attn_prefill_kernel(AttnArgs a, int tile0) {
    constexpr int SHARE = prefill_share(D, ROWS), THREADS = prefill_threads(D, ROWS), WAVES = THREADS / 64;
    constexpr bool EXTRA = OPTIONS != kNoOptions;
    constexpr int KEYS = 2 / SHARE;                 // blocks of 32 keys of a wave
    constexpr int DIMS = D / (32 * SHARE);          // and of 32 output dimensions
    constexpr int C = D / 8;                        // 16-byte chunks of a K row
    constexpr int STAGE = kTileKeys * C / THREADS;  // chunks per thread and tile, for K and for V
    constexpr int IMAGE = 2 * kTileKeys * C;        // chunks of a tile's image
    extern __shared__ u4 lds[];                     // a.images of them, used in turn, and PrefillShared
    const int splits = a.splits;
    const int kvh = blockIdx.x, split = blockIdx.y;
    // One sequence's first table entries, requested before anything else is known.
    int ids = -1, ids_first = -64;
    if (a.count == 1) {
        ids = a.c.table[min((int)(threadIdx.x & 63), a.c.cols - 1)];
        ids_first = 0;
    }
    const PrefillTile it = prefill_tile(a, tile0 + blockIdx.z);
    if (it.s < 0) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int n = lane & 31, h = lane >> 5;
    const int part = wave % SHARE, rows0 = wave / SHARE * 32;
    auto& shared = *reinterpret_cast<PrefillShared<WAVES, (SHARE > 1)>*>(lds + a.images * IMAGE);

    const int prefix = it.prefix;
    const PrefillRow q = prefill_row(a, it, prefix, kvh, rows0 + n);
    const int head = q.head, token = q.token, qpos = q.pos, hi = q.see.hi, lo = q.see.lo;
    const bool live = q.live;
    // What a token sees starts and ends no earlier than what the one before it
    // sees: all of the wave's rows see [all_lo, all_hi), none sees from any_hi on.
    const int tok0 = __builtin_amdgcn_readfirstlane(prefill_token_of(a, rows0));
    const int tok1 = min(__builtin_amdgcn_readfirstlane(prefill_token_of(a, rows0 + 31)), it.n - 1);
    const int all_hi = prefill_sees(a, it, prefix, tok0).hi;
    const Seen most = prefill_sees(a, it, prefix, tok1);
    const int any_hi = tok0 < it.n ? most.hi : 0, all_lo = most.lo;

    // All of the workgroup's rows see [seen_lo, seen_hi).
    const int seen_hi = prefill_sees(a, it, prefix, 0).hi, seen_lo = prefill_sees(a, it, prefix, it.n - 1).lo;

    // Tiles of the workgroup: the first token sees the lowest position, the last
    // (or the prefix) the highest.
    const int last = it.pos + it.n - 1;
    const int wg_hi = last >= 0 ? min(max(last + 1, prefix), it.len) : 0;
    const int wg_lo = a.window > 0 ? max(it.pos + 1 - a.window, 0) : 0;
    const int first_tile = wg_lo / kTileKeys;
    const int tiles = max((wg_hi + kTileKeys - 1) / kTileKeys - first_tile, 0);
    const int per = splits == 1 ? tiles : (tiles + splits - 1) / splits;
    const int t_begin = first_tile + split * per;
    const int t_end = min(t_begin + per, first_tile + tiles);

    h8 qf[D / 16];
    {
        const u4* qp = reinterpret_cast<const u4*>(a.q + ((size_t)token * a.heads + head) * D + 8 * h);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            qf[s] = as_h8(qp[2 * s]);
            if (!live) qf[s] = (h8)(_Float16)0.0f;
        }
    }
    const ScoreParams sp = score_params<OPTIONS>(a, head);
    const int pmask = (1 << a.c.shift) - 1;
    const int* row = a.c.table + (size_t)it.s * a.c.cols;

    // Pages of a tile's four quarters (16 positions each); positions past the end
    // take the last one's.  Uniform over the workgroup.
    struct Pages {
        int p0, p1, p2, p3;
        __device__ int gone() const {  // bit i: quarter i has no page
            return (p0 < 0 ? 1 : 0) | (p1 < 0 ? 2 : 0) | (p2 < 0 ? 4 : 0) | (p3 < 0 ? 8 : 0);
        }
        __device__ size_t of(int quarter) const {
            const int even = quarter & 2 ? p2 : p0, odd = quarter & 2 ? p3 : p1;
            return (size_t)max(quarter & 1 ? odd : even, 0);
        }
    };
    // Table entries [ids_first, ids_first + 64), one per lane: an entry read when
    // its tile is requested would wait for all tiles under way, because loads
    // complete in order.
    const int last_entry = max(it.len - 1, 0) >> a.c.shift;
    ids = (unsigned)ids < (unsigned)a.c.pages ? ids : -1;
    auto page_at = [&](int pos) {
        const int e = min(pos, it.len - 1) >> a.c.shift;
        if (e >= ids_first + 64) {
            ids_first = e;
            ids = row[min(e + lane, last_entry)];
            ids = (unsigned)ids < (unsigned)a.c.pages ? ids : -1;
        }
        return __builtin_amdgcn_readlane(ids, e - ids_first);
    };
    auto pages_of = [&](int t) {
        Pages r;
        r.p0 = page_at(t * kTileKeys);
        r.p1 = r.p2 = r.p3 = r.p0;
        if (a.c.shift < 6) {
            r.p1 = page_at(t * kTileKeys + 16);
            r.p2 = page_at(t * kTileKeys + 32);
            r.p3 = page_at(t * kTileKeys + 48);
        }
        return r;
    };
    // A tile straight into an image, 16 bytes per lane: LDS takes a wave's lanes
    // in order, so each lane fetches the chunk that the swizzle puts at its place:
    // of K, load j of thread tid is place x = THREADS j + tid, row x / C; of V,
    // dimension THREADS / 8 j + tid / 8, whose swizzle is the same for all j.
    const int v_c = v_chunk<D>(tid >> 3, tid & 7) & 7;
    uint32_t k_at[STAGE];  // byte offset from the tile's first row
#pragma unroll
    for (int j = 0; j < STAGE; ++j) {
        const int x = THREADS * j + tid, key = x / C;
        k_at[j] = 2 * (key * D + 8 * (k_chunk<D>(key, x % C) - key * C));
    }
    const uint32_t v_at = 2 * (((uint32_t)(tid >> 3) << a.c.shift) + 8 * v_c);
    const uint32_t lds_at =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u4*)lds + 1024 * wave);
    // A tile within one page.
    struct Whole {
        const uint16_t *k, *v;
        uint32_t to;
    };
    auto whole = [&](int t, const Pages& pg, int image) {
        const int off = (t * kTileKeys) & pmask;
        const size_t p = (size_t)max(pg.p0, 0);
        Whole w;
        w.k = uniform(a.c.k + p * a.c.k_stride + (((size_t)kvh << a.c.shift) + off) * D);
        w.v = uniform(a.c.v + p * a.c.v_stride + ((size_t)(kvh * D) << a.c.shift) + off);
        w.to = lds_at + image * (IMAGE * 16);
        return w;
    };
    auto load_piece = [&](const Whole& w, int j) {  // 0 <= j < 2 STAGE
        if (j < STAGE) load_lds(w.k, k_at[j], w.to + 16 * THREADS * j);
        else load_lds(w.v + ((size_t)(THREADS / 8 * (j - STAGE)) << a.c.shift), v_at, w.to + 16 * THREADS * j);
    };
    auto load = [&](int t, const Pages& pg, int image) {
        const int kb = t * kTileKeys;
        const uint32_t to = lds_at + image * (IMAGE * 16);
        if (a.c.shift >= 6) {
            const Whole w = whole(t, pg, image);
#pragma unroll
            for (int j = 0; j < 2 * STAGE; ++j) load_piece(w, j);
        } else {
            // Quarters of 16 positions, each in a page of its own or shared.
            const size_t vpage = pg.of(v_c >> 1);
            const uint16_t* vp = a.c.v + vpage * a.c.v_stride + ((size_t)(kvh * D + (tid >> 3)) << a.c.shift) +
                                 ((kb + 8 * v_c) & pmask);
#pragma unroll
            for (int j = 0; j < STAGE; ++j) {
                const int x = THREADS * j + tid, key = x / C;
                load_lds(a.c.k + pg.of(key >> 4) * a.c.k_stride + (((size_t)kvh << a.c.shift) + ((kb + key) & pmask)) * D +
                             8 * (k_chunk<D>(key, x % C) - key * C),
                         to + 16 * THREADS * j);
                load_lds(vp + ((size_t)(THREADS / 8 * j) << a.c.shift), to + kTileKeys * C * 16 + 16 * THREADS * j);
            }
        }
    };

    f16v acc[DIMS];
#pragma unroll
    for (int i = 0; i < DIMS; ++i) acc[i] = (f16v)0.0f;
    float m = Q4_NEG_INF, l = 0.0f;
    int t_use = t_begin;
    // Key of this lane's K row, in its wave's blocks.
    const int km = 32 * KEYS * part + 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
    const int dm = 32 * DIMS * part + n;  // first dimension of this lane's V rows

    const int ahead = a.images - 1;  // tiles requested ahead
    // Bit i of pages.gone() for the tiles under way, four bits each, oldest first.
    uint32_t gone_bits = 0;
    uint32_t bad = 0;  // nonzero: a tile with masked positions holds infinities or NaN
    Pages pg = {};
    if (t_begin < t_end) pg = pages_of(t_begin);
    int t_load = t_begin, slot_load = 0;  // next tile to request, and its image
    auto requested = [&] {
        gone_bits |= (uint32_t)pg.gone() << (4 * (t_load - t_use));
        slot_load = slot_load == ahead ? 0 : slot_load + 1;
        ++t_load;
        if (t_load < t_end) pg = pages_of(t_load);
    };
    auto request = [&] {
        load(t_load, pg, slot_load);
        requested();
    };
    for (int i = 0; i < ahead && t_load < t_end; ++i) request();
    auto follow = [&](float m_new) {
        const float f = part_weight(m, m_new);
        l *= f;
#pragma unroll
        for (int d = 0; d < DIMS; ++d) acc[d] *= f;
        m = m_new;
    };
    int slot = 0;
    // SPREAD: another tile, in one page, is requested piece by piece during the
    // first product.  At once its loads hold the wave up for a time each.
    auto tile = [&](auto spread) {
        constexpr bool SPREAD = decltype(spread)::value;
        const int kb = t_use * kTileKeys, gone = gone_bits & 15;
        u4* im = lds + slot * IMAGE;
        slot = slot == ahead ? 0 : slot + 1;
        // This tile's loads are done (2 STAGE operations per newer tile may be
        // under way), and everyone has read the image that the next request
        // overwrites.
        if (t_load - t_use == 3) wait_and_meet<4 * STAGE>();
        else if (t_load - t_use == 2) wait_and_meet<2 * STAGE>();
        else wait_and_meet<0>();
        Whole next;
        if constexpr (SPREAD) {
            next = whole(t_load, pg, slot_load);
            requested();
        } else {
            if (t_load < t_end) request();
        }
        if (gone || kb + kTileKeys > it.len) {
            // Values past the end and of absent pages are cleared: their weight is
            // zero, but zero times what an unwritten slot holds may be NaN.
            for (int i = tid; i < D * (kTileKeys / 8); i += THREADS) {
                const int dim = i >> 3, vc = i & 7;
                const int keep = (gone >> (vc >> 1)) & 1 ? 0 : min(max(it.len - (kb + 8 * vc), 0), 8);
                u4 mask;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mask[e] = (2 * e < keep ? 0x0000FFFFu : 0u) | (2 * e + 1 < keep ? 0xFFFF0000u : 0u);
                im[v_chunk<D>(dim, vc)] &= mask;
            }
            lds_meet();
        }
        if (gone || kb < seen_lo || kb + kTileKeys > seen_hi) {
            // Masked for some row.  A weight of zero hides a masked value only if the
            // value is finite: each wave looks at its share of the values.
#pragma unroll
            for (int i = 0; i < D * (kTileKeys / 8); i += THREADS) {
                const u4 v = im[kTileKeys * C + i + tid];
                bad |= odd_halves(v.x) | odd_halves(v.y) | odd_halves(v.z) | odd_halves(v.w);
            }
        }
        if (kb >= any_hi) {
            if constexpr (SPREAD) {
#pragma unroll
                for (int j = 0; j < 2 * STAGE; ++j) load_piece(next, j);
            }
            if constexpr (SHARE > 1) lds_meet();
        } else {
            // Operand reads run ahead of the products: KW steps of K, and VW of V before
            // the softmax, as many as registers hold without spilling (a spilled
            // register's reload would wait for the tiles under way).
            constexpr int STEPS = D / 16, KW = STEPS == 4 || (D > 192 && EXTRA) ? 2 : STEPS == 6 ? 3 : 4;
            constexpr int VW = (SHARE > 1 ? D <= 192 : !EXTRA) ? 2 : 1;
            u4 kf[KW][KEYS];
#pragma unroll
            for (int d = 0; d < KW; ++d)
#pragma unroll
                for (int b = 0; b < KEYS; ++b) kf[d][b] = im[k_chunk<D>(32 * b + km, 2 * d + h)];
            __builtin_amdgcn_sched_barrier(0);
            f16v s[KEYS];
#pragma unroll
            for (int b = 0; b < KEYS; ++b) s[b] = (f16v)0.0f;
#pragma unroll
            for (int d = 0; d < STEPS; ++d) {
#pragma unroll
                for (int b = 0; b < KEYS; ++b) {
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(kf[d % KW][b]), qf[d], s[b], 0, 0, 0);
                    if (d + KW < STEPS) kf[d % KW][b] = im[k_chunk<D>(32 * b + km, 2 * (d + KW) + h)];
                }
                if constexpr (SPREAD) {
                    constexpr int EVERY = STEPS / (2 * STAGE);
                    if (d % EVERY == 0) load_piece(next, d / EVERY);
                }
            }
            // V operands in the order of use: the wave's own keys first.
            const auto v_of = [&](int d, int kk) {
                const int c = SHARE == 1 ? 2 * kk + h : 4 * (part ^ (kk >> 1)) + 2 * (kk & 1) + h;
                return im[v_chunk<D>(32 * d + dm, c)];
            };
            u4 vf[VW][DIMS];
#pragma unroll
            for (int w = 0; w < VW; ++w)
#pragma unroll
                for (int d = 0; d < DIMS; ++d) vf[w][d] = v_of(d, w);
            __builtin_amdgcn_sched_barrier(0);
            const int kw = kb + 32 * KEYS * part;  // first position of the wave's blocks
            const bool masked = gone || kb < all_lo || kb + kTileKeys > all_hi;
            // Without options the running maximum is that of the plain products
            // (scale > 0), and scale and maximum enter the exponent in one
            // multiply-add.
            if constexpr (EXTRA) {
                if (OPTIONS == kLargeCapOptions || a.softcap > 0.0f) {
#pragma unroll
                    for (int b = 0; b < KEYS; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[b][i] = capped<OPTIONS == kLargeCapOptions>(s[b][i], sp);
                } else {
#pragma unroll
                    for (int b = 0; b < KEYS; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i) s[b][i] *= sp.scale2;
                }
                if (a.slopes) {
                    const float bias = sp.slope2 * (float)(kw + 8 * h - qpos);
#pragma unroll
                    for (int b = 0; b < KEYS; ++b)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            s[b][i] += __builtin_fmaf(sp.slope2, (float)(32 * b + 16 * (i >> 3) + (i & 7)), bias);
                }
            }
            if (masked) {
                // seen: lo <= key < hi, as one unsigned comparison
                const int from = kw + 8 * h - lo;
                const unsigned count = (unsigned)max(hi - lo, 0);
#pragma unroll
                for (int b = 0; b < KEYS; ++b) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[b][i] = (unsigned)(from + 32 * b + 16 * (i >> 3) + (i & 7)) < count ? s[b][i] : Q4_NEG_INF;
                }
                if (gone) {
#pragma unroll
                    for (int b = 0; b < KEYS; ++b) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if ((gone >> (2 * (KEYS * part + b) + (i >> 3))) & 1) s[b][i] = Q4_NEG_INF;
                    }
                }
            }
            // Four chains, of three operands an instruction.
            float tops[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const auto v = [&](int i) { return s[i / 4][4 * (i % 4) + c]; };
                tops[c] = v(0);
#pragma unroll
                for (int i = 1; i + 1 < 4 * KEYS; i += 2) tops[c] = top_of(top_of(tops[c], v(i)), v(i + 1));
                tops[c] = top_of(tops[c], v(4 * KEYS - 1));
            }
            float top = top_of_halves(top_of(top_of(tops[0], tops[1]), top_of(tops[2], tops[3])));
            if constexpr (!EXTRA) top *= sp.scale2;
            // The maximum that the exponents are taken from follows the true one only
            // when it is more than 2^8 behind: weights then stay below 2^8, and the
            // outputs are rarely rescaled after the first tiles.
            if (__any(top > m + 8.0f)) {
                // A pair's two maxima meet after the weights are rounded: whole ones
                // differ by a power of two, which changes no digit.
                follow(fmaxf(m, SHARE > 1 ? ceilf(top) : top));
            }
            const float base = m == Q4_NEG_INF ? 0.0f : m;
            // The weights are summed as they enter the second product, rounded.
            const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
            float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            h8 pf[2 * KEYS];
#pragma unroll
            for (int b = 0; b < KEYS; ++b) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = exp2_hw(EXTRA ? s[b][i] - base : __builtin_fmaf(s[b][i], sp.scale2, -base));
                    pf[2 * b + (i >> 3)][i & 7] = (_Float16)p;
                }
            }
#pragma unroll
            for (int i = 0; i < 2 * KEYS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sums[e] = __builtin_amdgcn_fdot2((h2){pf[i][2 * e], pf[i][2 * e + 1]}, one, sums[e], false);
            l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
            if constexpr (SHARE > 1) {
                shared.weights[wave][0][lane] = __builtin_bit_cast(u4, pf[0]);
                shared.weights[wave][1][lane] = __builtin_bit_cast(u4, pf[1]);
                if (h == 0) shared.base[wave][n] = m;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                if constexpr (SHARE > 1) {
                    if (kk == 2) {
                        // The other wave's weights, brought to the higher maximum.
                        lds_meet();
                        const float theirs = shared.base[wave ^ 1][n];
                        pf[0] = as_h8(shared.weights[wave ^ 1][0][lane]);
                        pf[1] = as_h8(shared.weights[wave ^ 1][1][lane]);
                        if (__any(theirs != m)) {
                            follow(fmaxf(m, theirs));
                            // In two factors: weights reach 2^8, so that under a single one, which
                            // fp16 ends at 2^-24, weights of up to 2^-17 would be lost while their
                            // sum stays.  Where nothing is seen the weights are zeros.
                            const float apart = theirs == Q4_NEG_INF ? 0.0f : theirs - m;
                            const float near = fmaxf(apart, -14.0f);
                            const _Float16 f = (_Float16)exp2_hw(near), f2 = (_Float16)exp2_hw(apart - near);
                            pf[0] = pf[0] * f * f2;
                            pf[1] = pf[1] * f * f2;
                        }
                    }
                }
#pragma unroll
                for (int d = 0; d < DIMS; ++d) {
                    acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(as_h8(vf[kk % VW][d]), pf[kk % (2 * KEYS)], acc[d], 0, 0, 0);
                    if (kk + VW < 4) vf[kk % VW][d] = v_of(d, kk + VW);
                }
            }
        }
        ++t_use;
        gone_bits >>= 4;
    };
    if (a.c.shift >= 6)
        while (t_load < t_end) tile(std::true_type{});
    while (t_use < t_end) tile(std::false_type{});
    l += __shfl_xor(l, 32, 64);
    const bool found = __any(bad != 0);
    if (lane == 0) shared.found[wave] = found;
    if constexpr (SHARE > 1) {
        if (h == 0) shared.sum[wave][n] = l;
    }
    __syncthreads();
    int any_found = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) any_found |= shared.found[w];
    if (any_found) {
        prefill_rows_one_by_one<D, OPTIONS, SHARE>(a, it, prefix, split, kvh, wave, t_begin * kTileKeys, t_end * kTileKeys);
        return;
    }
    if constexpr (SHARE > 1) l += shared.sum[wave ^ 1][n];

    if (!live) return;
    if (splits == 1) {
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        uint16_t* op = a.out + ((size_t)token * a.heads + head) * D + 32 * DIMS * part;
#pragma unroll
        for (int d = 0; d < DIMS; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint2 w;
                w.x = as_u32((h2){(_Float16)(acc[d][4 * i] * inv), (_Float16)(acc[d][4 * i + 1] * inv)});
                w.y = as_u32((h2){(_Float16)(acc[d][4 * i + 2] * inv), (_Float16)(acc[d][4 * i + 3] * inv)});
                *reinterpret_cast<uint2*>(op + 32 * d + 8 * i + 4 * h) = w;
            }
        }
    } else {
        const long at = ((long)split * a.rows + token) * a.heads + head;
        float* op = a.workspace + kAttnCounters + at * D + 32 * DIMS * part;
#pragma unroll
        for (int d = 0; d < DIMS; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4*>(op + 32 * d + 8 * i + 4 * h) =
                    (f4){acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
        }
        if (h == 0 && part == 0) {
            float* ml = a.workspace + kAttnCounters + (long)splits * a.rows * a.heads * D + at * 2;
            ml[0] = m;
            ml[1] = l;
        }
    }
}

// Join of the splits of one query row, one wave each, in order.
template <int D>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(AttnArgs a) {
    const int splits = a.splits;
    const long rows = (long)a.rows * a.heads;
    const long r = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= rows) return;
    // Tokens outside every sequence have no parts.
    const int token = (int)(r / a.heads);
    if (token < a.q_starts[0] || token >= a.q_starts[a.count]) return;
    const float* part = a.workspace + kAttnCounters;
    store_joined(join_parts<D, false>(part + r * D, part + (long)splits * rows * D + r * 2, rows, splits), a.out + r * D);
}

template <int D, int OPTIONS, int ROWS>
static hipError_t launch_tiles(AttnArgs a, const DeviceInfo& dev, hipStream_t st) {
    constexpr size_t image = 2 * kTileKeys * D * sizeof(uint16_t);
    constexpr size_t behind = sizeof(PrefillShared<prefill_threads(D, ROWS) / 64, (prefill_share(D, ROWS) > 1)>);
    // Two workgroups of four waves per CU hide each other's waits where there are
    // enough of them; fewer workgroups, and those of eight waves, get as many
    // images as a CU's LDS holds, up to four (three tiles ahead).
    const long tiles = prefill_tiles(a.rows, a.count, ROWS, a.group);
    const bool two = prefill_threads(D, ROWS) == 256 && tiles * a.c.kv_heads * a.splits > dev.num_cu;
    const int fit = (int)(((two ? dev.max_lds / 2 : dev.max_lds) - behind) / image);
    a.images = fit < 2 ? 2 : fit > 4 ? 4 : fit;
    auto kernel = &attn_prefill_kernel<D, OPTIONS, ROWS>;
    std::atomic<int>& ready = PerDevice<&attn_prefill_kernel<D, OPTIONS, ROWS>>::value[dev.device];
    if (!ready.load(std::memory_order_acquire)) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)dev.max_lds);
        if (e != hipSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    // Kv heads are next to each other, so that with a multiple of eight of them
    // each XCD's L2 holds its own heads' keys and values.
    const long most = 65535;  // of a grid's third dimension
    for (long t = 0; t < tiles; t += most) {
        const dim3 grid(a.c.kv_heads, a.splits, (unsigned)(tiles - t < most ? tiles - t : most));
        hipLaunchKernelGGL((attn_prefill_kernel<D, OPTIONS, ROWS>), grid, dim3(prefill_threads(D, ROWS)), a.images * image + behind,
                           st, a, (int)t);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int D, int OPTIONS>
static hipError_t launch_rows(const AttnArgs& a, int rows, const DeviceInfo& dev, hipStream_t st) {
    if constexpr (D != 96) {  // three blocks of 32 dimensions do not share out
        if (rows == 64) return launch_tiles<D, OPTIONS, 64>(a, dev, st);
    }
    return launch_tiles<D, OPTIONS, 128>(a, dev, st);
}

template <int D>
static hipError_t launch_prefill_attn(AttnArgs a, const DeviceInfo& dev, hipStream_t st) {
    a.inv_group = 1.0f / (float)a.group;
    PrefillPlan plan = prefill_plan(a.rows, a.count, a.heads, a.c.kv_heads, D, a.max_length);
    // A window leaves a workgroup fewer positions: 34 tokens on 8,000 with a window of
    // 128 take 9.3 us planned for those, 13.6 for all.  The workspace is for all.
    const long span = (long)a.window + prefill_tokens(128, a.group) + kTileKeys;
    if (a.window > 0 && span < a.max_length) {
        const int most = plan.splits;
        plan = prefill_plan(a.rows, a.count, a.heads, a.c.kv_heads, D, span);
        if (plan.splits > most) plan.splits = most;
    }
    a.splits = plan.splits;
    a.tile = prefill_tokens(plan.rows, a.group);
    a.inv_tile = 1.0f / (float)a.tile;
    hipError_t e = hipSuccess;
    switch (attn_options(a)) {
        case kNoOptions: e = launch_rows<D, kNoOptions>(a, plan.rows, dev, st); break;
        case kOptions: e = launch_rows<D, kOptions>(a, plan.rows, dev, st); break;
        case kLargeCapOptions: e = launch_rows<D, kLargeCapOptions>(a, plan.rows, dev, st); break;
    }
    if (e != hipSuccess || a.splits == 1) return e;
    const long rows = (long)a.rows * a.heads;
    hipLaunchKernelGGL((attn_prefill_join_kernel<D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_attn_prefill(const AttnArgs& a, const DeviceInfo& dev, hipStream_t st) {
    switch (a.c.dim) {
        case 64: return launch_prefill_attn<64>(a, dev, st);
        case 96: return launch_prefill_attn<96>(a, dev, st);
        case 128: return launch_prefill_attn<128>(a, dev, st);
        case 192: return launch_prefill_attn<192>(a, dev, st);
        case 256: return launch_prefill_attn<256>(a, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
