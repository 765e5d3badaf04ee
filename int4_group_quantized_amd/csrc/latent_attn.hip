// Attention over latent rows, in the absorbed form (gfx950).
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . c_j) c_j[:L]
// over the positions j that token t sees (attn_new.hpp), c_j the cached row of L +
// 64 columns: key with all of them, value with the first L.  All heads share the
// rows, so a position is read once for R = 16, 32 or 64 query rows (row = token *
// heads + head): 2 (L + 64) bytes for 2 R (2 L + 64) flops.  Memory bound up to about
// 64 rows in all, from there on bound by the matrix cores and what feeds them.
//
// A workgroup of four waves takes 64 positions (a tile) at a time, which go straight
// from memory into one of two LDS images while the other is worked on.
//   S^T[key][row] = C Q^T     16 and 32 rows: wave w takes keys 16w .. 16w + 15;
//                             64 rows: half of the keys for half of the rows
//   O^T[dim][row] = C^T P^T   wave w takes dims w L/4 .. for all keys and rows; the
//                             operand is read transposed (ds_read_b64_tr_b16: of 16
//                             lanes that name 4 rows of 16 columns each gets one
//                             column's 4 rows)
// with v_mfma_f32_16x16x32_f16, 64 rows with v_mfma_f32_32x32x16_f16.  Queries and
// outputs stay in registers, the weights pass through LDS.
//
// 64 sequences of 8,192 positions (0.6 GB): 16 heads 115 us (5.2 TB/s), 64 heads 139,
// 128 heads 203 to 211 (146 GFLOP, 690 to 720 TFLOP/s; the join 12 to 14 of it).  The
// last has its matrix cores busy 35 to 40% of the cycles: one wave per SIMD, whose
// registers hold queries and outputs, goes through products, softmax and barriers in
// turn.  64 rows by eight waves of 32 each, whose registers leave no room for reading
// operands ahead, took 262; a tile's first product beside the last one's second, in
// tiles of 32 positions, 214.  Few rows are bound by latency: one sequence of 2,000
// positions and 16 heads takes 16 us, 5 of them the join.
//
// R and the number of parts follow max_new, not the rows that there are: the first and
// the last of the 64-sequence calls take 290 and 296 us when it is 64 instead of 1.
//
// A wave takes its weights from the maximum that all had after the last tile, or from
// its own where that is 2^8 above; the waves' maxima meet with the weights.  Whole
// ones: bringing the weights from one to another changes no digit.
//
// LDS rows are a multiple of 128 bytes apart, an odd one; the low bits of a row's
// chunk numbers are exclusive-ored with some of the row's (swizzle) so that the 16
// rows of a key operand and the rows of a transposed read fall on different banks.
//
// The positions are cut into parts (attn_new.hpp), which a second launch joins.
#include "latent.hpp"
#include "lds_loads.hpp"

#include <type_traits>

namespace q4 {

typedef float f16s __attribute__((ext_vector_type(16)));

constexpr int kLatentThreads = 256;
constexpr int kLatentTarget = 256;    // workgroups wanted per launch: one per CU
constexpr int kWeightPitch = 72;      // halves of a row of weights in LDS: 9 chunks, so 16 rows differ in banks

template <int L, int R>
struct LatentShared {
    static constexpr int D = L + kRot;
    uint16_t image[2][kTileKeys * D];
    uint16_t weights[R * kWeightPitch];
    float base[4][R];  // what a wave's weights were taken from
    int found[2][4];   // a wave has found infinities or NaN where a row is masked
};
// After the tiles its place holds the outputs, a row's dims in order.
template <int L, int R>
struct LatentResult {
    static constexpr int PITCH = L + 4;
    float o[R][PITCH];
    float l[4][R];
    float m[R], sum[R];
};

// Exclusive-ored into the low three bits of a row's chunk numbers.  A transposed
// read of 32 lanes takes rows 0 to 3 and 8 to 11 (of 16) of two chunks each for the
// small product, rows 0 to 3 of four chunks for the large one.
template <bool WIDE>
__device__ __forceinline__ int latent_swizzle(int row) {
    return WIDE ? (row & 2) << 1 | ((row >> 1) & 2) | ((row >> 3) & 1) : (row & 2) | ((row >> 1) & 4) | ((row >> 2) & 1);
}

// Halves of a dword whose exponent is all ones (infinite or NaN), as bits 0 and 16.
__device__ __forceinline__ uint32_t odd_halves_in(uint32_t w) {
    return (((w & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u;
}

typedef short s4v __attribute__((ext_vector_type(4)));

// A row of the workgroup over one tile that the fast loop has left out, or has scores far
// from zero in, one position after the other, on top of its results in LDS.
template <int L>
__device__ __forceinline__ void latent_row_one_by_one(const NewArgs& x, const NewSeq& q, int token, int head, int kb, float* o, float& m,
                                      float& sum) {
    constexpr int D = L + kRot, PER = L / 64;
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 63, end = min(kb + kTileKeys, q.len), pmask = (1 << a.c.shift) - 1;
    const SeenRow see = seen_row(x.masks, 0, q, token);
    const _Float16* qp = reinterpret_cast<const _Float16*>(a.q) + ((size_t)(q.row + token) * a.heads + head) * D;
    float acc[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = o[lane + 64 * i];
    for (int key = kb; key < end; ++key) {
        const int page = page_of(a.c, a.c.table + (size_t)q.s * a.c.cols, key);
        if (page < 0 || !(seen_word(see, key, q.base) & 1)) continue;
        const _Float16* c = reinterpret_cast<const _Float16*>(a.c.k) + (size_t)page * a.c.k_stride + (size_t)(key & pmask) * D;
        float dot = (float)qp[L + lane] * (float)c[L + lane], v[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = (float)c[lane + 64 * i];
            dot = __builtin_fmaf((float)qp[lane + 64 * i], v[i], dot);
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
        const float s = dot * (a.scale * kLog2e), m_new = fmaxf(m, s), from = m_new == Q4_NEG_INF ? 0.0f : m_new;
        const float f = exp2_hw(m - from), p = exp2_hw(s - from);
        sum = sum * f + p;
        m = m_new;
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = acc[i] * f + p * v[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) o[lane + 64 * i] = acc[i];
}

// What a workgroup works on.
struct LatentWork {
    NewPart it;
    int r0, nrows;  // first row of the sequence's, rows
    int t_end;      // tiles end
    int all_hi;     // every row sees [0, all_hi)
};

__device__ __forceinline__ LatentWork latent_work(const NewArgs& x, int rows) {
    LatentWork w;
    w.it = new_part(x, rows);
    w.r0 = w.it.block * rows;
    w.nrows = w.it.q.s < 0 ? 0 : min(rows, min(w.it.q.n, x.max_new) * x.a.heads - w.r0);
    if (w.nrows <= 0) return w;
    const int base = w.it.q.base;
    // Without masks the rows' last token sees most, the first least.
    const int last_token = (w.r0 + w.nrows - 1) / x.a.heads;
    w.t_end = x.masks ? w.it.t_end : min(w.it.t_end, (max(base + last_token + 1, 0) + kTileKeys - 1) / kTileKeys);
    w.all_hi = x.masks ? base : base + w.r0 / x.a.heads + 1;
    return w;
}

// A wave's share of the loads: 16 rows of a tile, which lie in one page and follow
// each other there.  LDS takes a wave's lanes in order, so each lane fetches the
// chunk that the swizzle puts at its place: load j of a lane is place 64 j + lane, row
// place / C, and only the low three bits of the place differ from the chunk fetched.
template <int L, bool WIDE>
struct LatentLoads {
    static constexpr int D = L + kRot, C = D / 8;
    static constexpr int LOADS = 16 * C / 64;  // of a tile
    static constexpr uint32_t IMAGE = 2 * kTileKeys * D;
    const KvCache& c;
    const int* table;
    const int len, wave, lane;
    // Table entries [ids_first, ids_first + 64), one per lane: an entry read when its
    // tile is requested would wait for the tile under way, because loads complete in
    // order.
    int ids = -1, ids_first = -64;
    const uint16_t* source;
    uint32_t to;         // the wave's place in the first image
    int page_next = 0;   // of the wave's rows of the tile aimed at
    int gone_next = 0;   // bit i: quarter i of it has no page

    // first: latent_entry's.
    __device__ __forceinline__ LatentLoads(const KvCache& cache, const NewSeq& q, int w, int l, const u4* lds, bool one, int first)
        : c(cache), table(cache.table + (size_t)q.s * cache.cols), len(q.len), wave(w), lane(l), source(cache.k) {
        if (one) {
            ids = (unsigned)first < (unsigned)c.pages ? first : -1;
            ids_first = 0;
        }
        to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u4*)lds + 32 * D * wave);
    }
    __device__ __forceinline__ void aim(int t) {
        const int p = t * kTileKeys + 16 * wave, e0 = min(t * kTileKeys, len - 1) >> c.shift;
        if (e0 + 3 >= ids_first + 64 || ids_first < 0) {
            ids_first = e0;
            ids = table[min(e0 + lane, max(len - 1, 0) >> c.shift)];
            ids = (unsigned)ids < (unsigned)c.pages ? ids : -1;
        }
        gone_next = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int id = __builtin_amdgcn_readlane(ids, (min(t * kTileKeys + 16 * i, len - 1) >> c.shift) - ids_first);
            gone_next |= id < 0 ? 1 << i : 0;
            if (i == wave) page_next = id;
        }
        source = uniform(c.k + (size_t)max(page_next, 0) * c.k_stride + (size_t)(p & ((1 << c.shift) - 1)) * D);
    }
    static __device__ __forceinline__ uint32_t offset(int place) {
        return 16 * (place ^ latent_swizzle<WIDE>(place / C));
    }
    __device__ __forceinline__ void piece(int slot, int j, uint32_t off) const {
        load_lds(source, off, to + slot * IMAGE + 1024 * j);
    }
    // A masked position has weight zero, but zero times what it holds may be NaN.
    // The wave's rows past the end and of an absent page are cleared.  A tile with
    // infinities or NaN in other rows, which some query rows may see, is left for
    // later (true): they are cleared too, and no one sees the tile.
    __device__ __forceinline__ bool clear(uint8_t* image, int kb, int page) const {
        const int keep = page < 0 ? 0 : min(max(len - (kb + 16 * wave), 0), 16);
        uint32_t odd = 0;
#pragma unroll 1
        for (int i = lane; i < 16 * C; i += 64) {
            u4* p = reinterpret_cast<u4*>(image) + 16 * C * wave + i;
            const u4 v = *p;
            const uint32_t here = odd_halves_in(v.x) | odd_halves_in(v.y) | odd_halves_in(v.z) | odd_halves_in(v.w);
            if (i / C >= keep || here) *p = (u4){0, 0, 0, 0};
            if (i / C < keep) odd |= here;
        }
        return __any(odd != 0);
    }
};

// A value operand: this lane's four keys of two blocks of four, at byte offsets in
// an image.
__device__ __forceinline__ h8 latent_values(const uint8_t* image, uint32_t first, uint32_t second) {
    const auto part = [&](uint32_t off) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s4v*)(__attribute__((address_space(3))) uint8_t*)(image + off));
    };
    return __builtin_bit_cast(h8, __builtin_shufflevector(part(first), part(second), 0, 1, 2, 3, 4, 5, 6, 7));
}

// Weights brought from one maximum to another.  In two factors: weights reach 2^8, so
// that under a single one, which fp16 ends at 2^-24, weights of up to 2^-17 would be
// lost while their sum stays.  Where nothing is seen they are zeros.
__device__ __forceinline__ h8 latent_moved(h8 p, float from, float to) {
    const float apart = from == Q4_NEG_INF ? 0.0f : from - to, near = fmaxf(apart, -14.0f);
    return p * (_Float16)exp2_hw(near) * (_Float16)exp2_hw(apart - near);
}

// x *= f for an output in an accumulation register.  In assembly, because the compiler
// would otherwise move all outputs to other registers and back for every tile, whether
// they are rescaled or not.  The last product that wrote x lies a whole first product
// back, and wait states stand between the last of these and the next product.
__device__ __forceinline__ void latent_scale(float& x, float f) {
    float v;
    asm volatile("v_accvgpr_read_b32 %1, %0\n\tv_mul_f32 %1, %1, %2\n\tv_accvgpr_write_b32 %0, %1" : "+a"(x), "=&v"(v) : "v"(f));
}

// From the results in LDS (o, m, sum) to the outputs, or the parts' places.  far: a base
// was (far_base), so that all tiles are taken again.
template <int L, int R>
__device__ __forceinline__ void latent_finish(const NewArgs& x, const LatentWork& w, int left_from, int left_to, bool far,
                                              LatentResult<L, R>& res) {
    constexpr int D = L + kRot, WAVES = kLatentThreads / 64;
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, pmask = (1 << a.c.shift) - 1;
    const NewSeq& q = w.it.q;
    const auto out_row = [&](int r) { return (size_t)q.row * a.heads + w.r0 + r; };
    if (far) {
        left_from = w.it.t_begin;
        left_to = w.t_end;
    }
    if (left_to > 0) {
        // The same tiles in every wave; each takes rows of its own.
        for (int r = wave; r < w.nrows; r += WAVES) {
            const int token = (w.r0 + r) / a.heads, head = w.r0 + r - token * a.heads;
            float mr = far ? Q4_NEG_INF : res.m[r], sum = far ? 0.0f : res.sum[r];
            if (far)
                for (int i = lane; i < L; i += 64) res.o[r][i] = 0.0f;
            for (int t = left_from; t < left_to; ++t) {
                // Whether the fast loop left it out.  It looks at tiles that some row does
                // not see whole or that lack a page, and finds nothing in rows without one.
                uint32_t odd = 0;
                bool whole = !far && t * kTileKeys + kTileKeys <= w.all_hi;
                for (int key = t * kTileKeys; key < min((t + 1) * kTileKeys, q.len) && !far; ++key) {
                    const int p = page_of(a.c, a.c.table + (size_t)q.s * a.c.cols, key);
                    if (p < 0) {
                        whole = false;
                        continue;
                    }
                    const uint32_t* c =
                        reinterpret_cast<const uint32_t*>(a.c.k + (size_t)p * a.c.k_stride + (size_t)(key & pmask) * D);
                    for (int i = lane; i < D / 2; i += 64) odd |= odd_halves_in(c[i]);
                }
                if (far || (!whole && __any(odd != 0))) latent_row_one_by_one<L>(x, q, token, head, t * kTileKeys, res.o[r], mr, sum);
            }
            if (lane == 0) {
                res.m[r] = mr;
                res.sum[r] = sum;
            }
        }
        __syncthreads();
    }
    const NewWorkspace ws = new_workspace(x, x.pairs, R, L);
    const long first = ((long)(w.it.slot + w.it.part) * x.pairs + w.it.block) * R;
    for (int i = tid; i < w.nrows * (L / 4); i += kLatentThreads) {
        const int r = i / (L / 4), d = i % (L / 4) * 4;
        const f4 o = *reinterpret_cast<const f4*>(&res.o[r][d]);
        const float sum = res.sum[r];
        if (w.it.parts == 1) {
            const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            uint2 v;
            v.x = as_u32((h2){(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)});
            v.y = as_u32((h2){(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)});
            *reinterpret_cast<uint2*>(a.out + out_row(r) * L + d) = v;
        } else {
            *reinterpret_cast<f4*>(ws.o + (first + r) * L + d) = o;
            if (d == 0) *reinterpret_cast<float2*>(ws.ml + (first + r) * 2) = {res.m[r], sum};
        }
    }
}

// One sequence's first table entries, requested before anything else is known.
__device__ __forceinline__ int latent_entry(const AttnArgs& a) {
    return a.count == 1 ? a.c.table[min((int)(threadIdx.x & 63), a.c.cols - 1)] : -1;
}

// 16 RB rows.
template <int L, int RB>
__global__ void __launch_bounds__(kLatentThreads, 1) latent_attn_kernel(NewArgs x) {
    constexpr int R = 16 * RB;
    using Loads = LatentLoads<L, false>;
    constexpr int D = Loads::D, LOADS = Loads::LOADS, STEPS = D / 32;
    constexpr int DT = L / 64;  // blocks of 16 dims of a wave
    static_assert(LOADS <= STEPS, "a load a step");
    extern __shared__ u4 lds[];
    auto& sh = *reinterpret_cast<LatentShared<L, R>*>(lds);
    const AttnArgs& a = x.a;
    const int entry = latent_entry(a);
    const LatentWork work = latent_work(x, R);
    if (work.nrows <= 0) return;
    const int nrows = work.nrows, r0 = work.r0, t_end = work.t_end, base = work.it.q.base;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int n = lane & 15, g = lane >> 4;
    h8 qf[RB][STEPS];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int r = 16 * b + n;
        const bool live = r < nrows;
        const u4* qp = reinterpret_cast<const u4*>(a.q + ((size_t)work.it.q.row * a.heads + r0 + (live ? r : 0)) * D + 8 * g);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            qf[b][s] = __builtin_bit_cast(h8, qp[4 * s]);
            if (!live) qf[b][s] = (h8)(_Float16)0.0f;
        }
    }
    const float scale2 = a.scale * kLog2e;
    Loads loads(a.c, work.it.q, wave, lane, lds, a.count == 1, entry);
    // Byte offsets in an image of the lane's operands: of step 0's keys, and of dims
    // 0's values, the first 4 of the 8 keys.  Further ones differ by whole rows and
    // 128 bytes, and by exclusive-ors below that.
    const uint32_t k_at = (16 * wave + n) * (2 * D) + 16 * (g ^ latent_swizzle<false>(n));
    const int v_key = 8 * g + (n >> 2);
    const uint32_t v_at = v_key * (2 * D) + 16 * ((wave * (L / 32) + ((n >> 1) & 1)) ^ latent_swizzle<false>(v_key)) + 8 * (n & 1);

    f4 acc[RB][DT];
    float m[RB], l[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        m[b] = Q4_NEG_INF;
        l[b] = 0.0f;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[b][i] = (f4){0, 0, 0, 0};
    }
    int left_from = 1 << 30, left_to = 0;  // tiles left for later
    uint32_t far = 0;                      // nonzero: a base of the lane's rows was, in any wave
    uint32_t at[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) at[j] = Loads::offset(64 * j + lane);
    int t = work.it.t_begin;
    if (t < t_end) {
        loads.aim(t);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) loads.piece(0, j, at[j]);
    }
    for (int slot = 0; t < t_end; ++t, slot ^= 1) {
        const int kb = t * kTileKeys, page = loads.page_next, gone = loads.gone_next;
        uint8_t* image = reinterpret_cast<uint8_t*>(sh.image[slot]);
        wait_for_loads<0>();
        const bool more = t + 1 < t_end;
        if (more) loads.aim(t + 1);
        // Seen whole by every row; the same in all waves.
        const bool whole = kb + kTileKeys <= work.all_hi && gone == 0;
        if (!whole) {
            const int bad = loads.clear(image, kb, page);
            if (lane == 0) sh.found[slot][wave] = bad;
        }
        // Every wave's loads of the tile are there, and the other image has been read.
        lds_meet();
        uint32_t seen = 0;  // bit 4b + i: the lane's row of block b sees key 16 wave + 4g + i
        if (!whole) {
            if (__any(sh.found[slot][lane & 3] != 0)) {
                left_from = min(left_from, t);
                left_to = t + 1;
            } else if (page >= 0) {
                // Formed again for each such tile: kept, it would take 20 registers.
#pragma unroll 1
                for (int b = 0; b < RB; ++b) {
                    const SeenRow see = seen_row(x.masks, 0, work.it.q, (r0 + min(16 * b + n, nrows - 1)) / a.heads);
                    seen |= ((uint32_t)(seen_word(see, kb, base) >> (16 * wave + 4 * g)) & 15) << (4 * b);
                }
            }
        }
        // Keys times queries, the next tile's loads between them.
        f4 s[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = (f4){0, 0, 0, 0};
        constexpr int AHEAD = 4;  // operands read ahead of the products
        h8 kf[AHEAD];
        const auto key_of = [&](int d) { return *reinterpret_cast<const h8*>(image + (k_at ^ 64 * (d & 1)) + 128 * (d >> 1)); };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) kf[d] = key_of(d);
        const auto products = [&](auto load) {
#pragma unroll
            for (int d = 0; d < STEPS; ++d) {
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[d % AHEAD], qf[b][d], s[b], 0, 0, 0);
                if (d + AHEAD < STEPS) kf[d % AHEAD] = key_of(d + AHEAD);
                if (decltype(load)::value && d < LOADS) loads.piece(slot ^ 1, d, at[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (more) products(std::true_type{});
        else products(std::false_type{});
        float sums[RB], mine[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[b][i] = seen >> (4 * b + i) & 1 ? s[b][i] : Q4_NEG_INF;
            }
            float top = top_of(top_of(s[b][0], s[b][1]), top_of(s[b][2], s[b][3]));
            top = top_of_halves(top_of_rows(top)) * scale2;
            // Follows the true maximum only when it is more than 2^8 behind.
            mine[b] = top > m[b] + 8.0f ? ceilf(top) : m[b];
            const float from = mine[b] == Q4_NEG_INF ? 0.0f : mine[b];
            const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
            h2 p[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i >> 1][i & 1] = (_Float16)exp2_hw(__builtin_fmaf(s[b][i], scale2, -from));
            // The weights are summed as they enter the second product, rounded.
            sums[b] = __builtin_amdgcn_fdot2(p[0], one, __builtin_amdgcn_fdot2(p[1], one, 0.0f, false), false);
            uint2 v;
            v.x = as_u32(p[0]);
            v.y = as_u32(p[1]);
            *reinterpret_cast<uint2*>(sh.weights + (16 * b + n) * kWeightPitch + 16 * wave + 4 * g) = v;
            if (g == 0) sh.base[wave][16 * b + n] = mine[b];
        }
        lds_meet();  // the weights are there
        // Whether the waves' maxima differ from each other or the last one.
        bool apart = false;
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int w = 0; w < 4; ++w) apart = apart || sh.base[w][16 * b + n] != m[b];
        const bool moved = __any(apart);
        if (moved) {
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                float common = Q4_NEG_INF;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float theirs = sh.base[w][16 * b + n];
                    common = fmaxf(common, theirs);
                    far |= far_base(theirs);
                }
                const float f = part_weight(m[b], common);
                l[b] *= f;
                sums[b] *= part_weight(mine[b], common);
#pragma unroll
                for (int d = 0; d < DT; ++d) acc[b][d] *= f;
                m[b] = common;
            }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) l[b] += sums[b];
        const auto value_of = [&](int i) {  // block i % DT of dims, 32 keys i / DT
            const int d = i % DT, kk = i / DT;
            const uint32_t off = (v_at ^ 32 * (d & 3)) + 64 * kk * D + 128 * (d >> 2);
            return latent_values(image, off, (off ^ 16) + 8 * D);
        };
        constexpr int VALUES = DT < 2 ? 2 : 4;  // operands read ahead of the products
        h8 vf[VALUES], pf[RB];
#pragma unroll
        for (int i = 0; i < VALUES; ++i) vf[i] = value_of(i);
#pragma unroll
        for (int i = 0; i < 2 * DT; ++i) {
            const int d = i % DT, kk = i / DT;
            if (d == 0) {
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    const int r = 16 * b + n;
                    pf[b] = *reinterpret_cast<const h8*>(sh.weights + r * kWeightPitch + 32 * kk + 8 * g);
                    if (moved) pf[b] = latent_moved(pf[b], sh.base[2 * kk + (g >> 1)][r], m[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < RB; ++b)
                acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i % VALUES], pf[b], acc[b][d], 0, 0, 0);
            if (i + VALUES < 2 * DT) vf[i % VALUES] = value_of(i + VALUES);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    lds_meet();  // the images have been read

    // Outputs and sums into LDS, where the images were.
    auto& res = *reinterpret_cast<LatentResult<L, R>*>(lds);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        l[b] += lane_swap16(l[b]);
        l[b] += __shfl_xor(l[b], 32, 64);
        const int r = 16 * b + n;
        if (g == 0) res.l[wave][r] = l[b];
        if (g == 0 && wave == 0) res.m[r] = m[b];
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<f4*>(&res.o[r][wave * (L / 4) + 16 * d + 4 * g]) = acc[b][d];
    }
    __syncthreads();
    if (tid < R) res.sum[tid] = (res.l[0][tid] + res.l[1][tid]) + (res.l[2][tid] + res.l[3][tid]);
    __syncthreads();
    latent_finish<L, R>(x, work, left_from, left_to, __any(far != 0), res);
}

// 64 rows.  Matrix row i of 32 keys loads key 16(i/16) + 8(i/4%2) + 4(i/8%2) + i%4,
// so that a lane (row = lane & 31, h = lane >> 5) holds keys 8h .. 8h + 7 of each 16.
template <int L>
__global__ void __launch_bounds__(kLatentThreads, 1) latent_attn_wide_kernel(NewArgs x) {
    constexpr int R = 64;
    using Loads = LatentLoads<L, true>;
    constexpr int D = Loads::D, LOADS = Loads::LOADS, STEPS = D / 16;
    constexpr int DT = L / 128;  // blocks of 32 dims of a wave
    static_assert(2 * LOADS <= STEPS, "a load every second step");
    extern __shared__ u4 lds[];
    auto& sh = *reinterpret_cast<LatentShared<L, R>*>(lds);
    const AttnArgs& a = x.a;
    const int entry = latent_entry(a);
    const LatentWork work = latent_work(x, R);
    if (work.nrows <= 0) return;
    const int nrows = work.nrows, r0 = work.r0, t_end = work.t_end, base = work.it.q.base;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int n = lane & 31, h = lane >> 5;
    const int kh = wave & 1, rh = wave >> 1;  // half of the keys, of the rows
    h8 qf[STEPS];
    {
        const int r = 32 * rh + n;
        const bool live = r < nrows;
        const u4* qp = reinterpret_cast<const u4*>(a.q + ((size_t)work.it.q.row * a.heads + r0 + (live ? r : 0)) * D + 8 * h);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            qf[s] = __builtin_bit_cast(h8, qp[2 * s]);
            if (!live) qf[s] = (h8)(_Float16)0.0f;
        }
    }
    const float scale2 = a.scale * kLog2e;
    Loads loads(a.c, work.it.q, wave, lane, lds, a.count == 1, entry);
    const int k_row = 32 * kh + 16 * (n >> 4) + 8 * ((n >> 2) & 1) + 4 * ((n >> 3) & 1) + (n & 3);
    const uint32_t k_at = k_row * (2 * D) + 16 * (h ^ latent_swizzle<true>(k_row));
    // Values: 16 lanes take 16 dims of 4 keys; lanes 16 and up the next 16 dims, 32 and
    // up 8 keys on.
    const int i16 = lane & 15, v_key = 8 * h + (i16 >> 2);
    const uint32_t v_at =
        v_key * (2 * D) + 16 * ((wave * (L / 32) + 2 * ((lane >> 4) & 1) + ((i16 >> 1) & 1)) ^ latent_swizzle<true>(v_key)) + 8 * (i16 & 1);

    f16s acc[2][DT];
    float m[2] = {Q4_NEG_INF, Q4_NEG_INF}, l = 0.0f;  // of all rows; of the wave's
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[b][i] = (f16s)0.0f;
    int left_from = 1 << 30, left_to = 0;  // tiles left for later
    uint32_t far = 0;                      // nonzero: a base of the lane's rows was, in any wave
    uint32_t at[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) at[j] = Loads::offset(64 * j + lane);
    int t = work.it.t_begin;
    if (t < t_end) {
        loads.aim(t);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) loads.piece(0, j, at[j]);
    }
    for (int slot = 0; t < t_end; ++t, slot ^= 1) {
        const int kb = t * kTileKeys, page = loads.page_next, gone = loads.gone_next;
        uint8_t* image = reinterpret_cast<uint8_t*>(sh.image[slot]);
        wait_for_loads<0>();
        const bool more = t + 1 < t_end;
        if (more) loads.aim(t + 1);
        // Seen whole by every row; the same in all waves.
        const bool whole = kb + kTileKeys <= work.all_hi && gone == 0;
        if (!whole) {
            const int bad = loads.clear(image, kb, page);
            if (lane == 0) sh.found[slot][wave] = bad;
        }
        // Every wave's loads of the tile are there, and the other image has been read.
        lds_meet();
        uint32_t seen = 0;  // bit i: the lane's row sees the key of its register i
        if (!whole) {
            if (__any(sh.found[slot][lane & 3] != 0)) {
                left_from = min(left_from, t);
                left_to = t + 1;
            } else {
                const SeenRow see = seen_row(x.masks, 0, work.it.q, (r0 + min(32 * rh + n, nrows - 1)) / a.heads);
                uint32_t word = (uint32_t)(seen_word(see, kb, base) >> (32 * kh));
                if (gone >> (2 * kh) & 1) word &= 0xFFFF0000u;
                if (gone >> (2 * kh) & 2) word &= 0x0000FFFFu;
                seen = (word >> (8 * h) & 0xFF) | (word >> (16 + 8 * h) & 0xFF) << 8;
            }
        }
        // Keys times queries, the next tile's loads between them.
        f16s s = (f16s)0.0f;
        constexpr int AHEAD = 6;  // operands read ahead of the products
        h8 kf[AHEAD];
        const auto key_of = [&](int d) { return *reinterpret_cast<const h8*>(image + (k_at ^ 32 * (d & 3)) + 128 * (d >> 2)); };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) kf[d] = key_of(d);
        const auto products = [&](auto load) {
#pragma unroll
            for (int d = 0; d < STEPS; ++d) {
                s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[d % AHEAD], qf[d], s, 0, 0, 0);
                if (d + AHEAD < STEPS) kf[d % AHEAD] = key_of(d + AHEAD);
                if (decltype(load)::value && d % 2 == 0 && d / 2 < LOADS) loads.piece(slot ^ 1, d / 2, at[d / 2]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (more) products(std::true_type{});
        else products(std::false_type{});
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = seen >> i & 1 ? s[i] : Q4_NEG_INF;
        }
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) tops[c] = top_of(top_of(s[c], s[4 + c]), top_of(s[8 + c], s[12 + c]));
        const float top = top_of_halves(top_of(top_of(tops[0], tops[1]), top_of(tops[2], tops[3]))) * scale2;
        // Follows the true maximum only when it is more than 2^8 behind.
        const float held = rh ? m[1] : m[0], mine = top > held + 8.0f ? ceilf(top) : held;
        const float from = mine == Q4_NEG_INF ? 0.0f : mine;
        const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
        h8 p[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i >> 3][i & 7] = (_Float16)exp2_hw(__builtin_fmaf(s[i], scale2, -from));
        // The weights are summed as they enter the second product, rounded.
        float sums[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sums[i] = __builtin_amdgcn_fdot2((h2){p[i][2 * e], p[i][2 * e + 1]}, one, sums[i], false);
        float sum = sums[0] + sums[1];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<h8*>(sh.weights + (32 * rh + n) * kWeightPitch + 32 * kh + 16 * i + 8 * h) = p[i];
        if (h == 0) sh.base[kh][32 * rh + n] = mine;
        const auto value_of = [&](int i) {  // block i % DT of dims, 16 keys i / DT
            const int d = i % DT, kk = i / DT;
            const uint32_t off = (v_at ^ 64 * (d & 1)) + 32 * kk * D + 128 * (d >> 1);
            return latent_values(image, off, (off ^ 32) + 8 * D);
        };
        constexpr int VALUES = 4;  // operands read ahead of the products
        h8 vf[VALUES];
#pragma unroll
        for (int i = 0; i < VALUES; ++i) vf[i] = value_of(i);
        lds_meet();  // the weights are there
        h8 pf[2][2];
        const auto weights_of = [&](int b, int kk) {
            return *reinterpret_cast<const h8*>(sh.weights + (32 * b + n) * kWeightPitch + 16 * kk + 8 * h);
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) pf[0][b] = weights_of(b, 0);
        // Whether the waves' maxima differ from each other or the last one.
        float theirs[2][2];
        bool apart = false;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                theirs[b][k] = sh.base[k][32 * b + n];
                apart = apart || theirs[b][k] != m[b];
            }
        const bool moved = __any(apart);
        if (moved) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float common = fmaxf(theirs[b][0], theirs[b][1]), f = part_weight(m[b], common);
                far |= far_base(theirs[b][0]) || far_base(theirs[b][1]);
                if (b == rh) {
                    l *= f;
                    sum *= part_weight(mine, common);
                }
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float o = acc[b][d][i];
                        latent_scale(o, f);
                        acc[b][d][i] = o;
                    }
                m[b] = common;
            }
            asm volatile("s_nop 7");
        }
        l += sum;
#pragma unroll
        for (int i = 0; i < 4 * DT; ++i) {
            const int d = i % DT, kk = i / DT;
            if (d == 0) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (kk + 1 < 4) pf[(kk + 1) & 1][b] = weights_of(b, kk + 1);
                    if (moved) pf[kk & 1][b] = latent_moved(pf[kk & 1][b], theirs[b][kk >> 1], m[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
                acc[b][d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[i % VALUES], pf[kk & 1][b], acc[b][d], 0, 0, 0);
            if (i + VALUES < 4 * DT) vf[i % VALUES] = value_of(i + VALUES);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    lds_meet();  // the images have been read

    // Outputs and sums into LDS, where the images were.
    auto& res = *reinterpret_cast<LatentResult<L, R>*>(lds);
    l += __shfl_xor(l, 32, 64);
    if (h == 0) res.l[kh][32 * rh + n] = l;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (h == 0 && wave == 0) res.m[32 * b + n] = m[b];
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4*>(&res.o[32 * b + n][wave * (L / 4) + 32 * d + 8 * i + 4 * h]) =
                    (f4){acc[b][d][4 * i], acc[b][d][4 * i + 1], acc[b][d][4 * i + 2], acc[b][d][4 * i + 3]};
    }
    __syncthreads();
    if (tid < R) res.sum[tid] = res.l[0][tid] + res.l[1][tid];
    __syncthreads();
    latent_finish<L, R>(x, work, left_from, left_to, __any(far != 0), res);
}

// Rows of a workgroup for `rows` query rows of a sequence.
static int latent_rows(long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

static int latent_target(long pairs) {
    const long t = kLatentTarget / pairs;
    return t > 0 ? (int)t : 1;
}

int64_t latent_attn_workspace(int heads, int latent, long max_new) {
    const long rows = max_new * heads;
    const int r = latent_rows(rows);
    const long pairs = (rows + r - 1) / r;
    return new_workspace_bytes(latent_target(pairs), pairs, r, latent);
}

template <int L, int RW>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(NewArgs x, int rows) {
    __shared__ JoinShared<L, RW, kLatentTarget + 1> sh;
    const AttnArgs& a = x.a;
    const NewParts p = new_parts(x, RW);
    if (p.q.s < 0) return;
    join_rows(
        sh, new_workspace(x, x.pairs, rows, L), p, min(p.q.n, x.max_new) * a.heads, (long)x.pairs * rows,
        [&](int slot, int row) { return ((long)slot * x.pairs + row / rows) * rows + row % rows; },
        [&](const NewSeq& q, int row) { return a.out + ((size_t)q.row * a.heads + row) * L; });
}

template <int L, auto Kernel, int R>
static hipError_t launch_latent_rows(NewArgs x, const DeviceInfo& dev, hipStream_t st) {
    constexpr size_t images = sizeof(LatentShared<L, R>), result = sizeof(LatentResult<L, R>);
    constexpr size_t bytes = images > result ? images : result;
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    const long rows = (long)x.max_new * x.a.heads, pairs = (rows + R - 1) / R;
    x.target = latent_target(pairs);
    const long tiles = ((long)x.a.max_length + kTileKeys - 1) / kTileKeys;
    x.pairs = (int)pairs;
    std::atomic<int>& ready = PerDevice<Kernel>::value[dev.device];
    if (!ready.load(std::memory_order_acquire)) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)bytes);
        if (e != hipSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    hipLaunchKernelGGL(Kernel, new_grid(new_items(x, R, tiles)), dim3(kLatentThreads), bytes, st, x);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !new_second(x, tiles)) return e;
    const int rw = join_rows_per_group((long)x.a.rows * x.a.heads);
    auto join = rw == 16 ? &latent_join_kernel<L, 16> : rw == 4 ? &latent_join_kernel<L, 4> : &latent_join_kernel<L, 1>;
    hipLaunchKernelGGL(join, new_grid(new_blocks(x, rw)), dim3(kJoinThreads), 0, st, x, R);
    return hipGetLastError();
}

template <int L>
static hipError_t launch_latent(const NewArgs& x, const DeviceInfo& dev, hipStream_t st) {
    switch (latent_rows((long)x.max_new * x.a.heads)) {
        case 16: return launch_latent_rows<L, &latent_attn_kernel<L, 1>, 16>(x, dev, st);
        case 32: return launch_latent_rows<L, &latent_attn_kernel<L, 2>, 32>(x, dev, st);
    }
    return launch_latent_rows<L, &latent_attn_wide_kernel<L>, 64>(x, dev, st);
}

hipError_t launch_latent_attn(const NewArgs& x, const DeviceInfo& dev, hipStream_t st) {
    switch (x.a.c.dim - kRot) {
        case 128: return launch_latent<128>(x, dev, st);
        case 256: return launch_latent<256>(x, dev, st);
        case 512: return launch_latent<512>(x, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
