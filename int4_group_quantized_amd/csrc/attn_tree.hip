// Attention of drafted tokens over the paged cache (gfx950).
//
//   out[t][h] = sum_j softmax_j(s(q[t][h] . k_j)) v_j  over the positions j that
//   token t sees: the committed ones and, of its sequence's drafted tokens, those
//   that its mask names (see attn_new.hpp).
//
// Memory bound: every cached position costs 4 * dim bytes per kv head, once for
// all of a tree's tokens and all heads of the group.  A workgroup takes 16, 32 or
// 64 of these query rows (RB row blocks of 16; row = token * group + head).
//
// A wave takes 64 positions (or 32, tree_halves) at a time, keys and values straight from
// memory into registers in the operand layout of v_mfma_f32_16x16x32_f16, and uses
// each operand for all row blocks:
//   S^T[key][row] = K Q^T     A = K rows as stored, B = the query rows
//   O^T[dim][row] = V^T P^T   A = V pages' rows as stored, B = P^T
// The result layout of the first product (lane: row = lane & 15, keys 4g + i of
// each 16-key subtile, g = lane >> 4) is the operand layout of the second (keys 8g
// + j of a 32-key block) because subtile t's row r loads key 32 (t/2) + 8 (r/4) +
// 4 (t%2) + r%4.
//
// What a row sees of 64 positions is one 64-bit word; it is formed only for those that
// hold drafted positions or a window's edge.
//
// The visible tiles of all sequences are cut into parts of one length, computed on
// the device from the lengths; a second launch joins them in order.
#include "attn_new.hpp"

namespace q4 {

constexpr int kTreeWaves = 4;
constexpr int kTreeThreads = 64 * kTreeWaves;
constexpr int kTreeGridY = 32768;  // parts, or sequences, per layer of the grid
constexpr int kTreeTarget = 512;   // most workgroups wanted per launch: two per CU

// Workgroups per CU that registers and LDS leave room for.
__host__ __device__ constexpr int tree_per_cu(int dim, int rb) { return dim <= 128 && rb == 1 ? 2 : 1; }

// Blocks of 32 positions that a wave takes at a time: one where two would not fit
// the registers.
__host__ __device__ constexpr int tree_halves(int dim, int rb) { return dim * rb > 256 && rb > 1 ? 1 : 2; }

// Row blocks of a workgroup for `rows` query rows of a sequence and kv head.
// Beyond dim 128 four row blocks' outputs and queries do not fit the registers.
static int tree_row_blocks(int rows, int dim) { return rows <= 16 ? 1 : rows <= 32 || dim > 128 ? 2 : 4; }

static int tree_target(long pairs, int dim, int rb) {
    const long t = kTreeTarget / 2 * tree_per_cu(dim, rb) / pairs;
    return t > 0 ? (int)t : 1;
}

__device__ __forceinline__ h8 tree_load(const uint16_t* p) { return __builtin_bit_cast(h8, *reinterpret_cast<const u4*>(p)); }

// Halves of a dword whose exponent is all ones (infinite or NaN), as bits 0 and 16.
__device__ __forceinline__ uint32_t odd_halves_of(uint32_t w) {
    return (((w & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u;
}

// Eight halves, each all ones where its bit is set.
__device__ __forceinline__ u4 halves_of(uint32_t bits) {
    u4 k;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        k[e] = (bits >> (2 * e) & 1 ? 0x0000FFFFu : 0u) | (bits >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
    return k;
}

// A wave's step of 32 H positions that the fast loop has left out, if it was: one
// where rows are masked and values that are there hold infinities or NaN, which
// the matrix products would multiply by zero.  Row after row and position after
// position, never touching what a row does not see, on top of the wave's results
// (outputs, maxima and sums) in LDS.  Far slower.
template <int D, int OPTIONS, int H>
__device__ void tree_step_one_by_one(const NewArgs& x, const NewSeq& q, int kvh, int r0, int nrows, int kb,
                                                  int all_lo, int all_hi, float* o, int pitch, float* ms, float* ls) {
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 63, end = min(kb + 32 * H, q.len), pmask = (1 << a.c.shift) - 1;
    const int* row = a.c.table + (size_t)q.s * a.c.cols;
    // The same decision as the fast loop's.
    bool whole = kb >= all_lo && kb + 32 * H <= all_hi;
    uint32_t bad = 0;
    for (int key = kb; key < end; ++key) {
        const int page = page_of(a.c, row, key);
        whole = whole && page >= 0;
        if (page < 0) continue;
        const uint16_t* v = a.c.v + (size_t)page * a.c.v_stride + ((size_t)(kvh * D) << a.c.shift) + (key & pmask);
        for (int d = lane; d < D; d += 64) bad |= odd_halves_of(v[(size_t)d << a.c.shift]);
    }
    if (whole || !__any(bad != 0)) return;
    constexpr int PER = (D + 63) / 64;
    for (int r = 0; r < nrows; ++r) {
        const int token = (r0 + r) / a.group, head = kvh * a.group + (r0 + r - token * a.group);
        const SeenRow see = seen_row(x, q, token);
        const ScoreParams sp = score_params<OPTIONS>(a, head);
        const _Float16* qp = reinterpret_cast<const _Float16*>(a.q) + ((size_t)(q.row + token) * a.heads + head) * D;
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = lane + 64 * i < D ? o[r * pitch + lane + 64 * i] : 0.0f;
        float m = ms[r], l = ls[r];
        for (int key = kb; key < end; ++key) {
            const int page = page_of(a.c, row, key);
            if (page < 0 || !(seen_word(see, key, q.base) & 1)) continue;
            const _Float16* k = reinterpret_cast<const _Float16*>(a.c.k) + (size_t)page * a.c.k_stride +
                                (((size_t)kvh << a.c.shift) + (key & pmask)) * D;
            const _Float16* v = reinterpret_cast<const _Float16*>(a.c.v) + (size_t)page * a.c.v_stride +
                                ((size_t)(kvh * D) << a.c.shift) + (key & pmask);
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 64 * i < D) dot = __builtin_fmaf((float)qp[lane + 64 * i], (float)k[lane + 64 * i], dot);
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d, 64);
            int at = key;
            if (x.masks && key >= q.base) {
                const int k0 = key - q.base;  // seen, so that a mask names it
                at = place_of(q, x.masks[q.row + k0] & low_bits(q.n));
            }
            const float s = score<OPTIONS>(dot, sp, at - see.place);
            const float m_new = fmaxf(m, s), from = m_new == Q4_NEG_INF ? 0.0f : m_new;
            const float f = exp2_hw(m - from), p = exp2_hw(s - from);
            l = l * f + p;
            m = m_new;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (lane + 64 * i < D) acc[i] = acc[i] * f + p * (float)v[(size_t)(lane + 64 * i) << a.c.shift];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < D) o[r * pitch + lane + 64 * i] = acc[i];
        if (lane == 0) {
            ms[r] = m;
            ls[r] = l;
        }
    }
}

template <int D, int OPTIONS, int RB>
__global__ void __launch_bounds__(kTreeThreads, tree_per_cu(D, RB)) attn_tree_kernel(NewArgs x, int least) {
    constexpr int R = 16 * RB;  // rows of a workgroup
    constexpr int OP = D + 4;   // pitch of a row of partial outputs in LDS
    constexpr bool EXTRA = OPTIONS != kNoOptions;
    constexpr int H = tree_halves(D, RB), STEP = 32 * H;
    __shared__ float part_o[kTreeWaves][R][OP];
    __shared__ float part_m[kTreeWaves][R], part_l[kTreeWaves][R];
    __shared__ int places[EXTRA ? kMaskTokens : 1];  // of the drafted tokens
    const AttnArgs& a = x.a;
    // Kv heads and row blocks first, so that neighbouring workgroups read
    // neighbouring parts of the same pages at the same time.
    const int pairs = gridDim.x, pair = blockIdx.x, kvh = pair % a.c.kv_heads;
    const int r0 = pair / a.c.kv_heads * R;  // first row of the sequence's in this workgroup
    const NewPart it = new_part(x, blockIdx.y + blockIdx.z * kTreeGridY, least);
    if (it.q.s < 0) return;
    const int nrows = min(R, min(it.q.n, x.max_new) * a.group - r0);
    if (nrows <= 0) return;
    const int base = it.q.base, len = it.q.len;

    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int n = lane & 15, g = lane >> 4;
    const int P = 1 << a.c.shift, pmask = P - 1;
    const int* row = a.c.table + (size_t)it.q.s * a.c.cols;

    // Token and head of row r of the workgroup.
    const auto token_of = [&](int r) { return (r0 + r) / a.group; };
    const auto out_row = [&](int r) {
        const int token = token_of(r);
        return (size_t)(it.q.row + token) * a.heads + kvh * a.group + (r0 + r - token * a.group);
    };
    h8 qf[RB][D / 32];
    SeenRow see[RB];
    ScoreParams sp[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int r = 16 * b + n;
        const bool live = r < nrows;
        const uint16_t* qp = a.q + out_row(live ? r : 0) * D + 8 * g;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
            qf[b][s] = tree_load(qp + 32 * s);
            if (!live) qf[b][s] = (h8)(_Float16)0.0f;
        }
        const int token = token_of(live ? r : 0);
        see[b] = seen_row(x, it.q, token);
        sp[b] = score_params<OPTIONS>(a, kvh * a.group + (r0 + (live ? r : 0) - token * a.group));
    }
    if constexpr (EXTRA) {
        if (a.slopes) {
            for (int k = threadIdx.x; k < kMaskTokens; k += kTreeThreads)
                places[k] = x.masks && k < it.q.n ? place_of(it.q, x.masks[it.q.row + k] & low_bits(it.q.n)) : base + k;
            __syncthreads();
        }
    }
    // Every row of every workgroup sees [all_lo, all_hi).
    const int all_hi = base, all_lo = a.window > 0 ? max(base + it.q.n - a.window, 0) : 0;

    f4 acc[RB][D / 16];
    float m[RB], l[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        m[b] = Q4_NEG_INF;
        l[b] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) acc[b][i] = (f4){0, 0, 0, 0};
    }

    // Operands of one tile: K as A of the first product, V as A of the second.
    u4 kr[2 * H][D / 32], vr[D / 16][H];
    // Pages of the 8-key groups that this lane's values and scores belong to
    // (v) and that its keys belong to (k), per 32-key block.  Positions past
    // the end take the last one's page.
    struct Ids {
        int v[H], k[H];
    };
    auto ids = [&](int t) {
        Ids r;
        const int kb = t * STEP;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            r.v[h] = page_of(a.c, row, min(kb + 32 * h + 8 * g, len - 1));
            r.k[h] = page_of(a.c, row, min(kb + 32 * h + 8 * (n >> 2), len - 1));
        }
        return r;
    };
    auto load_k = [&](int t, const Ids& id) {
#pragma unroll
        for (int u = 0; u < 2 * H; ++u) {
            const int key = t * STEP + 32 * (u >> 1) + 8 * (n >> 2) + 4 * (u & 1) + (n & 3);
            const uint16_t* p = a.c.k + (size_t)max(id.k[u >> 1], 0) * a.c.k_stride +
                                ((size_t)kvh * P + (key & pmask)) * D + 8 * g;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) kr[u][d] = *reinterpret_cast<const u4*>(p + 32 * d);
        }
    };
    auto load_v = [&](int t, const Ids& id) {
        // Both halves of a 128-byte line (a page of 64) are requested back to back.
        const uint16_t* p[H];
#pragma unroll
        for (int h = 0; h < H; ++h)
            p[h] = a.c.v + (size_t)max(id.v[h], 0) * a.c.v_stride + ((size_t)(kvh * D + n) << a.c.shift) +
                   ((t * STEP + 32 * h + 8 * g) & pmask);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
#pragma unroll
            for (int h = 0; h < H; ++h) vr[d][h] = *reinterpret_cast<const u4*>(p[h] + ((size_t)(16 * d) << a.c.shift));
        }
    };
    // Positions from which to which tiles were left for later.
    int left_from = it.q.len + kTileKeys, left_to = 0;
    // One tile; K is in kr.  `next` requests the next tile's K as soon as kr is
    // free, so that it travels during the softmax and the second product.
    auto tile = [&](int t, const Ids& id, auto next) {
        const int kb = t * STEP;
        load_v(t, id);
        __builtin_amdgcn_sched_barrier(0);
        f4 s[RB][2 * H];
#pragma unroll
        for (int u = 0; u < 2 * H; ++u) {
#pragma unroll
            for (int b = 0; b < RB; ++b) s[b][u] = (f4){0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    s[b][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, kr[u][d]), qf[b][d], s[b][u], 0, 0, 0);
            }
        }
        next();
        __builtin_amdgcn_sched_barrier(0);
        const bool whole = __all(kb >= all_lo && kb + STEP <= all_hi && id.v[0] >= 0 && id.v[H - 1] >= 0);
        h8 pf[RB][H];
        float sums[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            uint32_t seen[H];  // bits of this lane's keys, 8g .. 8g + 7 of each block of 32
            if (!whole) {
                const uint64_t word = seen_word(see[b], kb, base);
#pragma unroll
                for (int h = 0; h < H; ++h) seen[h] = id.v[h] < 0 ? 0 : (uint32_t)(word >> (32 * h)) >> (8 * g) & 0xFF;
            }
            float top = Q4_NEG_INF;
#pragma unroll
            for (int u = 0; u < 2 * H; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = 4 * (u & 1) + i, key = kb + 32 * (u >> 1) + 8 * g + e;
                    int distance = 0;
                    if constexpr (EXTRA) {
                        distance = key - see[b].place;
                        if (a.slopes && !whole && key >= base)
                            distance = places[min(key - base, kMaskTokens - 1)] - see[b].place;
                    }
                    float v = score<OPTIONS>(s[b][u][i], sp[b], distance);
                    if (!whole) v = seen[u >> 1] >> e & 1 ? v : Q4_NEG_INF;
                    s[b][u][i] = v;
                    top = top_of(top, v);
                }
            }
            top = top_of_halves(top_of_rows(top));
            // The maximum that the exponents are taken from follows the true one only
            // when it is more than 2^8 behind: weights then stay below 2^8, and the
            // outputs are rarely rescaled after the first tiles.
            if (__any(top > m[b] + 8.0f)) {
                const float m_new = fmaxf(m[b], top), f = part_weight(m[b], m_new);
                l[b] *= f;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) acc[b][d] *= f;
                m[b] = m_new;
            }
            const float from = m[b] == Q4_NEG_INF ? 0.0f : m[b];
            // The weights are summed as they enter the second product, rounded.
#pragma unroll
            for (int u = 0; u < 2 * H; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) pf[b][u >> 1][4 * (u & 1) + i] = (_Float16)exp2_hw(s[b][u][i] - from);
            }
            const h2 one = {(_Float16)1.0f, (_Float16)1.0f};
            sums[b] = 0.0f;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sums[b] = __builtin_amdgcn_fdot2((h2){pf[b][h][2 * e], pf[b][h][2 * e + 1]}, one, sums[b], false);
        }
        if (!whole) {
            // A masked position has weight zero, but zero times what it holds may be
            // NaN.  Positions past the end and of absent pages are cleared; a tile with
            // infinities or NaN elsewhere, which some rows may see, is left for later.
            uint32_t bad = 0;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const u4 keep = halves_of(id.v[h] < 0 ? 0u : (uint32_t)low_bits(len - (kb + 32 * h + 8 * g)));
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    vr[d][h] &= keep;
                    // One after the other: all at once took 60 registers more.
                    asm volatile("" : "+v"(vr[d][h]));
                    bad |= odd_halves_of(vr[d][h].x) | odd_halves_of(vr[d][h].y) | odd_halves_of(vr[d][h].z) |
                           odd_halves_of(vr[d][h].w);
                    asm volatile("" : "+v"(bad));
                }
            }
            if (__any(bad != 0)) {
                left_to = kb + STEP;
                left_from = min(left_from, kb);
                return;
            }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) l[b] += sums[b];
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, vr[d][h]), pf[b][h], acc[b][d], 0, 0, 0);
            }
        }
    };

    constexpr int STEPS = kTileKeys / STEP;  // of a tile
    const int t_end = it.t_end * STEPS;
    int t = it.t_begin * STEPS + wave;
    if (t < t_end) {
        Ids id = ids(t);
        load_k(t, id);
        for (; t + kTreeWaves < t_end; t += kTreeWaves) {
            const Ids after = ids(t + kTreeWaves);
            tile(t, id, [&] { load_k(t + kTreeWaves, after); });
            id = after;
        }
        tile(t, id, [] {});
    }

    // Join the four waves in order.
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        l[b] += lane_swap16(l[b]);
        l[b] += __shfl_xor(l[b], 32, 64);
        if (g == 0) {
            part_m[wave][16 * b + n] = m[b];
            part_l[wave][16 * b + n] = l[b];
        }
        if (16 * b + n < nrows) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f4*>(&part_o[wave][16 * b + n][16 * d + 4 * g]) = acc[b][d];
        }
    }
    for (int kb = left_from; kb < left_to; kb += STEP * kTreeWaves)
        tree_step_one_by_one<D, OPTIONS, H>(x, it.q, kvh, r0, nrows, kb, all_lo, all_hi, &part_o[wave][0][0], OP, part_m[wave],
                                            part_l[wave]);
    __syncthreads();
    const NewWorkspace ws = new_workspace(x, pairs, R, D);
    const long slot = ((long)(it.slot + it.part) * pairs + pair) * R;
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kTreeThreads) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = part_m[0][r];
#pragma unroll
        for (int w = 1; w < kTreeWaves; ++w) top = fmaxf(top, part_m[w][r]);
        f4 o = {0, 0, 0, 0};
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kTreeWaves; ++w) {
            const float f = part_weight(part_m[w][r], top);
            sum += part_l[w][r] * f;
            o += *reinterpret_cast<const f4*>(&part_o[w][r][d]) * f;
        }
        if (it.parts == 1) {
            const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            uint2 w;
            w.x = as_u32((h2){(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)});
            w.y = as_u32((h2){(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)});
            *reinterpret_cast<uint2*>(a.out + out_row(r) * D + d) = w;
        } else {
            *reinterpret_cast<f4*>(ws.o + (slot + r) * D + d) = o;
            if (d == 0) *reinterpret_cast<float2*>(ws.ml + (slot + r) * 2) = {top, sum};
        }
    }
}

// Row `row` of a sequence is token row / heads, head row % heads.
template <int D, int RW>
__global__ void __launch_bounds__(kJoinThreads) attn_tree_join_kernel(NewArgs x, int least, int rows) {
    __shared__ JoinShared<D, RW, kTreeTarget + 1> sh;
    const AttnArgs& a = x.a;
    const NewParts p = new_parts(x, blockIdx.y + blockIdx.z * kTreeGridY, least);
    const int row0 = blockIdx.x * RW, all = min(p.q.n, x.max_new) * a.heads;
    if (p.parts < 2 || row0 >= all) return;
    join_rows(
        sh, new_workspace(x, x.pairs, rows, D), p, row0, all, (long)x.pairs * rows,
        [&](int slot, int row) {
            const int token = row / a.heads, head = row - token * a.heads, kvh = head / a.group;
            const int r = token * a.group + head - kvh * a.group;  // of the kv head's
            return ((long)slot * x.pairs + r / rows * a.c.kv_heads + kvh) * rows + r % rows;
        },
        [&](const NewSeq& q, int row) { return a.out + ((size_t)q.row * a.heads + row) * D; });
}

static int tree_blocks(int kv_heads, int group, int max_new, int dim, int* rb) {
    const long rows = (long)max_new * group;
    *rb = tree_row_blocks(rows > 64 ? 64 : (int)rows, dim);
    return (int)((rows + 16 * *rb - 1) / (16 * *rb)) * kv_heads;
}

// Whether the prompt kernel serves a call: from this many rows of a sequence and kv
// head on, where its tiles, which all waves of a workgroup share, cost less than
// every wave's own loads; options are this file's.
constexpr int kPromptRows = 64;
static bool by_prompt(int max_new, int group) { return max_new * group >= kPromptRows; }

int64_t attn_tree_workspace(int64_t tokens, int64_t count, int heads, int kv_heads, int dim, int max_new,
                            int64_t max_length) {
    int rb;
    const int pairs = tree_blocks(kv_heads, heads / kv_heads, max_new, dim, &rb);
    const int64_t own = new_workspace_bytes(tree_target(pairs, dim, rb), pairs, 16 * rb, dim);
    if (!by_prompt(max_new, heads / kv_heads)) return own;
    const int64_t prompt = attn_prefill_workspace(tokens, count, heads, kv_heads, dim, dim, max_length);
    return prompt > own ? prompt : own;
}

template <int D, int RB>
static hipError_t launch_tree_rows(NewArgs x, int pairs, hipStream_t st) {
    x.target = tree_target(pairs, D, RB);
    x.pairs = pairs;
    const int least = D <= 128 ? 2 : 1;
    const long tiles = ((long)x.a.max_length + kTileKeys - 1) / kTileKeys, most = (tiles + least - 1) / least * x.a.count;
    const long grid = (long)x.target + x.a.count < most ? (long)x.target + x.a.count : most;
    const dim3 blocks(pairs, (unsigned)(grid < kTreeGridY ? grid : kTreeGridY), (unsigned)((grid + kTreeGridY - 1) / kTreeGridY));
    const int options = attn_options(x.a);
    auto kernel = options == kNoOptions ? &attn_tree_kernel<D, kNoOptions, RB>
                  : options == kOptions ? &attn_tree_kernel<D, kOptions, RB>
                                        : &attn_tree_kernel<D, kLargeCapOptions, RB>;
    hipLaunchKernelGGL(kernel, blocks, dim3(kTreeThreads), 0, st, x, least);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !new_second(x, tiles)) return e;
    const int rw = join_rows_per_group((long)x.a.rows * x.a.heads);
    const dim3 groups((unsigned)(((long)x.max_new * x.a.heads + rw - 1) / rw),
                      (unsigned)(x.a.count < kTreeGridY ? x.a.count : kTreeGridY),
                      (unsigned)((x.a.count + kTreeGridY - 1) / kTreeGridY));
    auto join = rw == 16  ? &attn_tree_join_kernel<D, 16>
                : rw == 4 ? &attn_tree_join_kernel<D, 4>
                          : &attn_tree_join_kernel<D, 1>;
    hipLaunchKernelGGL(join, groups, dim3(kJoinThreads), 0, st, x, least, 16 * RB);
    return hipGetLastError();
}

template <int D>
static hipError_t launch_tree(const NewArgs& x, hipStream_t st) {
    int rb;
    const int pairs = tree_blocks(x.a.c.kv_heads, x.a.group, x.max_new, D, &rb);
    if (rb == 1) return launch_tree_rows<D, 1>(x, pairs, st);
    if constexpr (D <= 128) {
        if (rb == 4) return launch_tree_rows<D, 4>(x, pairs, st);
    }
    return launch_tree_rows<D, 2>(x, pairs, st);
}

hipError_t launch_attn_tree(const NewArgs& x, const DeviceInfo& dev, hipStream_t st) {
    if (by_prompt(x.max_new, x.a.group) && attn_options(x.a) == kNoOptions && x.a.window == 0) {
        AttnArgs a = x.a;
        a.masks = x.masks;
        a.max_new = x.max_new;
        return launch_prefill_tree(a, dev, st);
    }
    switch (x.a.c.dim) {
        case 64: return launch_tree<64>(x, st);
        case 96: return launch_tree<96>(x, st);
        case 128: return launch_tree<128>(x, st);
        case 192: return launch_tree<192>(x, st);
        case 256: return launch_tree<256>(x, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
