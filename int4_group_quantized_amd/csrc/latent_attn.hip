// Attention over latent rows, in the absorbed form (gfx950).
//
//   out[t][h] = sum_j softmax_j(scale q[t][h] . c_j) c_j[:L]
// over the positions j that token t sees (attn_new.hpp), c_j the cached row of L +
// 64 columns: key with all of them, value with the first L.  All heads share the
// rows, so a position is read once for R = 16, 32 or 64 query rows (row = token *
// heads + head): 2 (L + 64) bytes for 2 R (2 L + 64) flops.  Memory bound up to about
// 64 rows in all, from there on bound by the matrix cores and what feeds them.
//
// A workgroup of G = 1 or 2 groups of four waves takes 64 positions (a tile) at a
// time, which go straight from memory into one of two LDS images while the other is
// worked on.  A group has 16 RB rows of its own; wave w of it takes
//   S^T[key][row] = C Q^T     keys 16w .. 16w + 15 for these rows
//   O^T[dim][row] = C^T P^T   dims w L/4 .. for all keys; the operand is read
//                             transposed (ds_read_b64_tr_b16: of 16 lanes that name
//                             4 rows of 16 columns each gets one column's 4 rows)
// with v_mfma_f32_16x16x32_f16; an operand from LDS serves RB products.  Queries
// and outputs stay in registers (64 rows by four waves took more of them than there
// are), the weights pass through LDS.  A wave takes its weights from the maximum that all had after the last tile, or from its own where
// that is 2^8 above; the waves' maxima meet with the weights.  Whole ones: bringing
// the weights from one to another changes no digit.
//
// LDS rows are a multiple of 128 bytes apart, an odd one; the chunk's low bits are
// exclusive-ored with the row's (swizzle) so that the 16 rows of a key operand and
// the 8 rows of a transposed read fall on different banks.
//
// The positions are cut into parts as for drafted tokens (attn_new.hpp).
#include "latent.hpp"
#include "lds_loads.hpp"

namespace q4 {

constexpr int kLatentGridY = 32768;   // parts per layer of the grid
constexpr int kWeightPitch = 72;      // halves of a row of weights in LDS: 9 chunks, so 16 rows differ in banks

template <int L, int RB, int G>
struct LatentShared {
    static constexpr int D = L + kRot, R = 16 * RB * G;
    uint16_t image[2][kTileKeys * D];
    uint16_t weights[R * kWeightPitch];
    float base[4][R];  // what a wave's weights were taken from
    int found[2][4 * G];  // a wave has found infinities or NaN where a row is masked
};
// After the tiles its place holds the outputs, a row's dims in order.
template <int L, int RB, int G>
struct LatentResult {
    static constexpr int R = 16 * RB * G, PITCH = L + 4;
    float o[R][PITCH];
    float l[4][R];
    float m[R], sum[R];
};

// Exclusive-ored into the low three bits of a row's chunk numbers.
__device__ __forceinline__ int latent_swizzle(int row) { return (row & 2) | ((row >> 1) & 4) | ((row >> 2) & 1); }

// Halves of a dword whose exponent is all ones (infinite or NaN), as bits 0 and 16.
__device__ __forceinline__ uint32_t odd_halves_in(uint32_t w) {
    return (((w & 0x7C007C00u) + 0x04000400u) >> 15) & 0x00010001u;
}

typedef short s4v __attribute__((ext_vector_type(4)));

// A row of the workgroup over one tile that the fast loop has left out, one
// position after the other, on top of its results in LDS.
template <int L>
__device__ __forceinline__ void latent_row_one_by_one(const NewArgs& x, const NewSeq& q, int token, int head, int kb, float* o, float& m,
                                      float& sum) {
    constexpr int D = L + kRot, PER = L / 64;
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 63, end = min(kb + kTileKeys, q.len), pmask = (1 << a.c.shift) - 1;
    const SeenRow see = seen_row(x, q, token);
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

template <int L, int RB, int G>
__global__ void __launch_bounds__(256 * G, G) latent_attn_kernel(NewArgs x) {
    constexpr int D = L + kRot, C = D / 8;   // columns and 16-byte chunks of a row
    constexpr int THREADS = 256 * G, WAVES = 4 * G;
    constexpr int R = 16 * RB * G, STEPS = D / 32;
    constexpr int LOADS = 16 * C / 64 / G;   // of a wave and tile, 64 chunks each
    constexpr int DT = L / 64;               // blocks of 16 dims of a wave
    using Shared = LatentShared<L, RB, G>;
    using Result = LatentResult<L, RB, G>;
    extern __shared__ u4 lds[];
    Shared& sh = *reinterpret_cast<Shared*>(lds);
    const AttnArgs& a = x.a;
    const int pairs = gridDim.x, pair = blockIdx.x, r0 = pair * R;
    const NewPart it = new_part(x, blockIdx.y + blockIdx.z * kLatentGridY, 1);
    if (it.q.s < 0) return;
    const int nrows = min(R, min(it.q.n, x.max_new) * a.heads - r0);
    if (nrows <= 0) return;
    const int base = it.q.base, len = it.q.len;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int n = lane & 15, g = lane >> 4;
    const int kw = wave & 3, rows0 = wave / 4 * 16 * RB;  // the wave's keys and dims, and rows
    const int pmask = (1 << a.c.shift) - 1;
    const int* table = a.c.table + (size_t)it.q.s * a.c.cols;

    const auto out_row = [&](int r) { return (size_t)it.q.row * a.heads + r0 + r; };
    h8 qf[RB][STEPS];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int r = rows0 + 16 * b + n;
        const bool live = r < nrows;
        const u4* qp = reinterpret_cast<const u4*>(a.q + out_row(live ? r : 0) * D + 8 * g);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            qf[b][s] = __builtin_bit_cast(h8, qp[4 * s]);
            if (!live) qf[b][s] = (h8)(_Float16)0.0f;
        }
    }
    // Without masks the rows' last token sees most.
    const int last_token = (r0 + nrows - 1) / a.heads;
    const int t_end = x.masks ? it.t_end : min(it.t_end, (max(base + last_token + 1, 0) + kTileKeys - 1) / kTileKeys);
    // Every row of the workgroup sees [0, all_hi).
    const int all_hi = x.masks ? base : base + r0 / a.heads + 1;
    const float scale2 = a.scale * kLog2e;

    // Table entries [ids_first, ids_first + 64), one per lane: an entry read when
    // its tile is requested would wait for the tile under way, because loads
    // complete in order.
    const int last_entry = max(len - 1, 0) >> a.c.shift;
    int ids = -1, ids_first = -64;
    auto page_at = [&](int pos) {
        const int e = min(pos, len - 1) >> a.c.shift;
        if (e >= ids_first + 64 || ids_first < 0) {
            ids_first = e;
            ids = table[min(e + lane, last_entry)];
            ids = (unsigned)ids < (unsigned)a.c.pages ? ids : -1;
        }
        return __builtin_amdgcn_readlane(ids, e - ids_first);
    };
    // 16 rows of a tile lie in one page and follow each other there; the waves with
    // the same keys share their loads.  LDS takes a wave's lanes in order, so each
    // lane fetches the chunk that the swizzle puts at its place.  Load j of a lane is
    // place place0 + 64 j, row place / C; only the low three bits of the place differ
    // from the chunk fetched.
    const int place0 = wave / 4 * (64 * LOADS) + lane;
    // Bytes of LDS: the images come first.
    const uint32_t lds_at =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u4*)lds + 32 * D * kw +
                                       wave / 4 * (1024 * LOADS));
    constexpr uint32_t IMAGE = 2 * kTileKeys * D;
    const uint16_t* source = a.c.k;
    int page = 0, page_next = 0;  // of the wave's rows in this tile and the one requested
    auto aim = [&](int t) {
        const int p = t * kTileKeys + 16 * kw;
        page_next = page_at(p);
        source = uniform(a.c.k + (size_t)max(page_next, 0) * a.c.k_stride + (size_t)(p & pmask) * D);
    };
    auto load_piece = [&](int slot, int j, int place) {
        load_lds(source, 16 * ((place + 64 * j) ^ latent_swizzle((place + 64 * j) / C)), lds_at + slot * IMAGE + 1024 * j);
    };

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

    int t = it.t_begin;
    if (t < t_end) {
        aim(t);
#pragma unroll
        for (int j = 0; j < LOADS; ++j) load_piece(0, j, place0);
    }
    for (int slot = 0; t < t_end; ++t, slot ^= 1) {
        const int kb = t * kTileKeys;
        uint8_t* image = reinterpret_cast<uint8_t*>(sh.image[slot]);
        // What follows from the lane's number is formed for every tile: kept, it would
        // push queries out of the registers.
        int ln = lane;
        asm volatile("" : "+v"(ln));
        const int n = ln & 15, g = ln >> 4;
        // Byte offset in an image of the lane's operand of step 0's keys.
        const uint32_t k_at = (16 * kw + n) * (2 * D) + 16 * (g ^ latent_swizzle(n));
        page = page_next;
        wait_for_loads<0>();
        const bool more = t + 1 < t_end;
        if (more) aim(t + 1);
        const bool whole = kb + kTileKeys <= all_hi && page >= 0;
        int bad = 0;
        uint32_t seen = 0;  // bit 4b + i: the lane's row of block b sees key 16 kw + 4g + i
        if (!whole) {
            // A masked position has weight zero, but zero times what it holds may be
            // NaN.  What the wave has loaded past the end and of an absent page is
            // cleared.  A tile with infinities or NaN in other rows, which some rows may
            // see, is left for later: they are cleared too, and no one sees the tile.
            const int keep = page < 0 ? 0 : min(max(len - (kb + 16 * kw), 0), 16);
            uint32_t odd = 0;
#pragma unroll 1
            for (int i = place0; i < place0 + 64 * LOADS; i += 64) {
                u4* p = reinterpret_cast<u4*>(image) + 16 * C * kw + i;
                const u4 v = *p;
                uint32_t here = odd_halves_in(v.x) | odd_halves_in(v.y) | odd_halves_in(v.z) | odd_halves_in(v.w);
                if (i / C >= keep || here) *p = (u4){0, 0, 0, 0};
                if (i / C < keep) odd |= here;
            }
            bad = __any(odd != 0);
            if (page >= 0) {
                // Formed again for each such tile: kept, it would take 20 registers.
#pragma unroll 1
                for (int b = 0; b < RB; ++b) {
                    const SeenRow see = seen_row(x, it.q, (r0 + min(rows0 + 16 * b + n, nrows - 1)) / a.heads);
                    seen |= ((uint32_t)(seen_word(see, kb, base) >> (16 * kw + 4 * g)) & 15) << (4 * b);
                }
            }
        }
        if (lane == 0) sh.found[slot][wave] = bad;
        // Every wave's loads of the tile are there, and the other image has been read.
        lds_meet();
        if (__any(sh.found[slot][lane & (WAVES - 1)] != 0)) {
            left_from = min(left_from, t);
            left_to = t + 1;
            seen = 0;
        }
        // Keys times queries, the next tile's loads between them.
        f4 s[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) s[b] = (f4){0, 0, 0, 0};
        constexpr int AHEAD = G > 1 ? 2 : 3;  // operands read ahead of the products
        h8 kf[AHEAD];
        const auto key_of = [&](int d) { return *reinterpret_cast<const h8*>(image + (k_at ^ 64 * (d & 1)) + 128 * (d >> 1)); };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) kf[d] = key_of(d);
#pragma unroll
        for (int d = 0; d < STEPS; ++d) {
#pragma unroll
            for (int b = 0; b < RB; ++b) s[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[d % AHEAD], qf[b][d], s[b], 0, 0, 0);
            if (d + AHEAD < STEPS) kf[d % AHEAD] = key_of(d + AHEAD);
            if (d < LOADS && more) load_piece(slot ^ 1, d, wave / 4 * (64 * LOADS) + ln);
            __builtin_amdgcn_sched_barrier(0);
        }
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
            uint2 w;
            w.x = as_u32(p[0]);
            w.y = as_u32(p[1]);
            *reinterpret_cast<uint2*>(sh.weights + (rows0 + 16 * b + n) * kWeightPitch + 16 * kw + 4 * g) = w;
            if (g == 0) sh.base[kw][rows0 + 16 * b + n] = mine[b];
        }
        lds_meet();  // the weights are there
        {
            asm volatile("" : "+v"(ln));
            const int n = ln & 15, g = ln >> 4;
            // Byte offset of the operand of dims 0's values, the first 4 of the 8 keys.
            const int key = 8 * g + (n >> 2);
            const uint32_t v_at = key * (2 * D) + 16 * ((kw * (L / 32) + ((n >> 1) & 1)) ^ latent_swizzle(key)) + 8 * (n & 1);
            // Whether the waves' maxima differ from each other or the last one.
            bool apart = false;
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int w = 0; w < 4; ++w) apart = apart || sh.base[w][rows0 + 16 * b + n] != m[b];
            const bool moved = __any(apart);
            if (moved) {
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    float common = sh.base[0][rows0 + 16 * b + n];
#pragma unroll
                    for (int w = 1; w < 4; ++w) common = fmaxf(common, sh.base[w][rows0 + 16 * b + n]);
                    const float f = part_weight(m[b], common);
                    l[b] *= f;
                    sums[b] *= part_weight(mine[b], common);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        acc[b][d] *= f;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    m[b] = common;
                }
            }
#pragma unroll
            for (int b = 0; b < RB; ++b) l[b] += sums[b];
            const auto value_of = [&](int i) {  // operand of block i % DT of dims, 32 keys i / DT
                const int d = i % DT, kk = i / DT;
                s4v part[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t off = (v_at ^ (32 * (d & 3) + 16 * h)) + 8 * h * D + 64 * kk * D + 128 * (d >> 2);
                    part[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s4v*)(__attribute__((address_space(3))) uint8_t*)(image + off));
                }
                return __builtin_bit_cast(h8, __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7));
            };
            constexpr int VALUES = 2;  // operands read ahead of the products
            h8 vf[VALUES], pf[RB];
#pragma unroll
            for (int i = 0; i < VALUES; ++i) vf[i] = value_of(i);
#pragma unroll
            for (int i = 0; i < 2 * DT; ++i) {
                const int d = i % DT, kk = i / DT;
                if (d == 0) {
#pragma unroll
                    for (int b = 0; b < RB; ++b) {
                        const int r = rows0 + 16 * b + n;
                        pf[b] = *reinterpret_cast<const h8*>(sh.weights + r * kWeightPitch + 32 * kk + 8 * g);
                        if (moved) {
                            // In two factors: weights reach 2^8, so that under a single one,
                            // which fp16 ends at 2^-24, weights of up to 2^-17 would be lost
                            // while their sum stays.  Where nothing is seen they are zeros.
                            const float from = sh.base[2 * kk + (g >> 1)][r];
                            const float apart = from == Q4_NEG_INF ? 0.0f : from - m[b];
                            const float near = fmaxf(apart, -14.0f);
                            pf[b] = pf[b] * (_Float16)exp2_hw(near) * (_Float16)exp2_hw(apart - near);
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < RB; ++b)
                    acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf[i % VALUES], pf[b], acc[b][d], 0, 0, 0);
                if (i + VALUES < 2 * DT) vf[i % VALUES] = value_of(i + VALUES);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    lds_meet();  // the images have been read

    // Outputs and sums into LDS, where the images were.
    Result& res = *reinterpret_cast<Result*>(lds);
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        l[b] += lane_swap16(l[b]);
        l[b] += __shfl_xor(l[b], 32, 64);
        const int r = rows0 + 16 * b + n;
        if (g == 0) res.l[kw][r] = l[b];
        if (g == 0 && kw == 0) res.m[r] = m[b];
#pragma unroll
        for (int d = 0; d < DT; ++d) *reinterpret_cast<f4*>(&res.o[r][kw * (L / 4) + 16 * d + 4 * g]) = acc[b][d];
    }
    __syncthreads();
    if (tid < R) res.sum[tid] = (res.l[0][tid] + res.l[1][tid]) + (res.l[2][tid] + res.l[3][tid]);
    __syncthreads();
    if (left_to > 0) {
        // The same tiles in every wave; each takes rows of its own.
        for (int r = wave; r < nrows; r += WAVES) {
            const int token = (r0 + r) / a.heads, head = r0 + r - token * a.heads;
            float mr = res.m[r], sum = res.sum[r];
            for (int tt = left_from; tt < left_to; ++tt) {
                // Whether the fast loop left it out.  It looks at tiles that some row does
                // not see whole, and finds nothing in rows of absent pages.
                if (tt * kTileKeys + kTileKeys <= all_hi) continue;
                uint32_t odd = 0;
                for (int key = tt * kTileKeys; key < min((tt + 1) * kTileKeys, len); ++key) {
                    const int p = page_of(a.c, table, key);
                    if (p < 0) continue;
                    const uint32_t* c =
                        reinterpret_cast<const uint32_t*>(a.c.k + (size_t)p * a.c.k_stride + (size_t)(key & pmask) * D);
                    for (int i = lane; i < D / 2; i += 64) odd |= odd_halves_in(c[i]);
                }
                if (__any(odd != 0)) latent_row_one_by_one<L>(x, it.q, token, head, tt * kTileKeys, res.o[r], mr, sum);
            }
            if (lane == 0) {
                res.m[r] = mr;
                res.sum[r] = sum;
            }
        }
        __syncthreads();
    }
    const NewWorkspace ws = new_workspace(x, pairs, R, L);
    const long first = ((long)(it.slot + it.part) * pairs + pair) * R;
    for (int i = tid; i < nrows * (L / 4); i += THREADS) {
        const int r = i / (L / 4), d = i % (L / 4) * 4;
        const f4 o = *reinterpret_cast<const f4*>(&res.o[r][d]);
        const float sum = res.sum[r];
        if (it.parts == 1) {
            const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
            uint2 w;
            w.x = as_u32((h2){(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)});
            w.y = as_u32((h2){(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)});
            *reinterpret_cast<uint2*>(a.out + out_row(r) * L + d) = w;
        } else {
            float* wo = ws.o + (first + r) * L + d;
            share_store(wo, o[0], o[1]);
            share_store(wo + 2, o[2], o[3]);
            if (d == 0) share_store(ws.ml + (first + r) * 2, res.m[r], sum);
        }
    }
    if (it.parts == 1) return;
    join_new_parts<L>(it, ws, pairs, pair, R, nrows,
                      [&](int r, const JoinedRow<L>& j) { store_joined(j, a.out + out_row(r) * L); });
}

// Rows of a workgroup for `rows` query rows of a sequence.
static int latent_rows(long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

static int latent_target(long pairs) {
    const long t = 256 / pairs;  // one workgroup per CU
    return t > 0 ? (int)t : 1;
}

int64_t latent_attn_workspace(int heads, int latent, long max_new) {
    const long rows = max_new * heads;
    const int r = latent_rows(rows);
    const long pairs = (rows + r - 1) / r;
    return new_workspace_bytes(latent_target(pairs), pairs, r, latent);
}

template <int L, int RB, int G>
static hipError_t launch_latent_rows(NewArgs x, const DeviceInfo& dev, hipStream_t st) {
    constexpr size_t images = sizeof(LatentShared<L, RB, G>), result = sizeof(LatentResult<L, RB, G>);
    constexpr size_t bytes = images > result ? images : result;
    static_assert(bytes <= 160 * 1024, "LDS of a CU");
    const long pairs = ((long)x.max_new * x.a.heads + 16 * RB * G - 1) / (16 * RB * G);
    x.target = latent_target(pairs);
    const long tiles = ((long)x.a.max_length + kTileKeys - 1) / kTileKeys * x.a.count;
    const long grid = (long)x.target + x.a.count < tiles ? (long)x.target + x.a.count : tiles;
    std::atomic<int>& ready = PerDevice<&latent_attn_kernel<L, RB, G>>::value[dev.device];
    if (!ready.load(std::memory_order_acquire)) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&latent_attn_kernel<L, RB, G>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    const dim3 blocks((unsigned)pairs, (unsigned)(grid < kLatentGridY ? grid : kLatentGridY),
                      (unsigned)((grid + kLatentGridY - 1) / kLatentGridY));
    hipLaunchKernelGGL((latent_attn_kernel<L, RB, G>), blocks, dim3(256 * G), bytes, st, x);
    return hipGetLastError();
}

template <int L>
static hipError_t launch_latent(const NewArgs& x, const DeviceInfo& dev, hipStream_t st) {
    switch (latent_rows((long)x.max_new * x.a.heads)) {
        case 16: return launch_latent_rows<L, 1, 1>(x, dev, st);
        case 32: return launch_latent_rows<L, 2, 1>(x, dev, st);
    }
    return launch_latent_rows<L, 2, 2>(x, dev, st);
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
