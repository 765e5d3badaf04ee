// Keys and values of every head from latent rows, by int4 weights (gfx950).
//
//   k[j][h] = (W_k[h] c_j, r_j),  v[j][h] = W_v[h] c_j
// c_j the L latent columns and r_j the 64 rotary ones of position j, W the weights
// dequantised to fp16 with one rounding, into the pages that the prompt attention
// reads: K [page][head][position][V + 64], V [page][head][dim][position].
//
// The weights stay: a workgroup of four waves owns one head, waves 0 and 1 its key
// rows, 2 and 3 its value rows, V / 2 each, dequantised once into registers as
// operands, and walks over tiles of 64 positions, which go straight from memory
// into one of two LDS images while the other is worked on.  An operand from LDS
// serves V / 64 products of v_mfma_f32_32x32x16_f16.  Keys are computed as
// [dim][position] and values as [position][dim], so that a lane holds neighbours of
// what it stores, eight once the halves of the wave have swapped theirs.
//
// 4,096 positions of 64 heads of 128 (latent 512, 69 GFLOP, 168 MB written) take 84 to
// 94 us, 1,000 of 128 heads 47 to 50, 1,900 of 16 heads 18 to 20, 4,096 of 96 heads, which
// leave 64 of 256 CUs without work, 140 to 144.  Matrix cores are busy 36% of the first
// one's cycles: one wave per SIMD, whose registers hold the weights, goes through
// products and stores in turn.  Where it took 84, results stored in halves as the
// products leave them, 8 bytes at a time, took 92, stored between the next tile's products
// 90.  The weights are read and turned to fp16 once per workgroup: codes and the fp16
// results leave no other rounding than theirs and the sums' own.
#include "latent.hpp"
#include "lds_loads.hpp"

#include <type_traits>

namespace q4 {

typedef float f16r __attribute__((ext_vector_type(16)));

constexpr int kExpandThreads = 256;

// Exclusive-ored into the low three bits of an LDS row's chunk numbers, so that 16
// rows at a pitch of an odd multiple of 128 bytes differ in banks.
__device__ __forceinline__ int expand_swizzle(int row) { return (row >> 1) & 7; }

// Eight weights in order: fp16(code * scale + min) of a dword of codes.
__device__ __forceinline__ h8 weights_of(uint32_t q, h2 s, h2 m, const DequantConsts& kc) {
    h2 c[4];
    dequant_dword(q, kc, c);  // (0, 4), (1, 5), (2, 6), (3, 7)
    h2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_elementwise_fma(c[i], s, m);
    return (h8){w[0][0], w[1][0], w[2][0], w[3][0], w[0][1], w[1][1], w[2][1], w[3][1]};
}

template <int L, int V>
__global__ void __launch_bounds__(kExpandThreads, 1) latent_expand_kernel(ExpandArgs a, int ranges) {
    constexpr int D = L + kRot, C = D / 8, K = V + kRot;
    constexpr int STEPS = L / 16, NB = V / 64;  // steps of a product, blocks of 32 weight rows of a wave
    constexpr int LOADS = 16 * C / 64;          // of a wave and tile, 64 chunks each
    static_assert(LOADS <= STEPS, "a load a step");
    extern __shared__ u4 lds[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int n = lane & 31, h = lane >> 5;
    const int head = blockIdx.x;
    const int pmask = (1 << a.c.shift) - 1;

    // Tiles of a sequence, from the one that holds its first position to expand.
    const auto bounds = [&](int s, int& from, int& to) {
        to = min(max(a.lengths[s], 0), a.max_length);
        from = a.firsts ? min(max(a.firsts[s], 0), to) : 0;
        return from < to ? (to + kTileKeys - 1) / kTileKeys - from / kTileKeys : 0;
    };
    int64_t total = 0;
    for (int s0 = 0; s0 < a.count; s0 += 64) {
        int from, to;
        total += lane_scan(s0 + lane < a.count ? bounds(s0 + lane, from, to) : 0).last;
    }
    const int64_t per = (total + ranges - 1) / ranges, begin = per * blockIdx.y, end = min(begin + per, total);
    if (begin >= end) return;
    // Looks up the tile with number `item` of all: its sequence, number, positions.
    int next_s = 0, next_tile = 0, next_from = 0, next_to = 0;
    const auto find = [&](int64_t item) {
        int64_t before = 0;
        for (int s0 = 0; s0 < a.count; s0 += 64) {
            int from = 0, to = 0;
            const int tiles = s0 + lane < a.count ? bounds(s0 + lane, from, to) : 0;
            const LaneScan c = lane_scan(tiles);
            const uint64_t hit = __ballot(tiles > 0 && item < before + c.upto && item >= before + c.upto - tiles);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
                next_s = s0 + l;
                next_from = of(from);
                next_to = of(to);
                next_tile = next_from / kTileKeys + (int)(item - (before + of(c.upto) - of(tiles)));
                return;
            }
            before += c.last;
        }
    };

    // Weights: rows of the head's 2 V, 32 a block.  A lane reads 32 codes at a time, the
    // upper half of the wave those behind the lower half's; of every two dwords (a
    // step's codes) they then swap the one that belongs to the other.
    h8 w[NB][STEPS];
    {
        const DequantConsts kc = make_dequant_consts();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const size_t row = (size_t)head * (2 * V) + (wave * NB + b) * 32 + n;
            const u4* q = reinterpret_cast<const u4*>(a.packed + row * (L / 2)) + h;
            const _Float16* sp = reinterpret_cast<const _Float16*>(a.scales) + row * (L / 128);
            const _Float16* mp = reinterpret_cast<const _Float16*>(a.mins) + row * (L / 128);
#pragma unroll
            for (int c = 0; c < L / 64; ++c) {
                const u4 v = q[2 * c];
                const h2 s = {sp[c / 2], sp[c / 2]}, m = {mp[c / 2], mp[c / 2]};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // Lower half: dwords 2i, 2i + 1 of the first 32 codes; upper: of the second.
                    const auto r = __builtin_amdgcn_permlane32_swap(v[2 * i], v[2 * i + 1], false, false);
                    w[b][4 * c + i] = weights_of(r[0], s, m, kc);
                    w[b][4 * c + 2 + i] = weights_of(r[1], s, m, kc);
                }
            }
        }
    }

    const uint32_t lds_at =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u4*)lds + 32 * D * wave);
    constexpr uint32_t IMAGE = 2 * kTileKeys * D;
    // The tile requested: where it lies, and where its keys and values go.  Lane i
    // holds the pages of the tile's quarter i % 4.
    const uint16_t* source = a.c.k;
    int page_to = -1;
    // Table entries [first, first + 64) of either cache, one per lane: an entry read for
    // its tile alone would hold up every tile.
    int ids = -1, ids_first = 0, to_ids = -1, to_first = 0;
    const auto refill = [&](const KvCache& c, int entry, int& first) {
        first = entry;
        const int e = entry + lane, id = e < c.cols ? c.table[(size_t)next_s * c.cols + e] : -1;
        return (unsigned)id < (unsigned)c.pages ? id : -1;
    };
    auto aim = [&](int64_t item) {
        const bool same = item > begin && (next_tile + 1) * kTileKeys < next_to;
        if (same) ++next_tile;
        else find(item);
        const int kb = next_tile * kTileKeys;
        if (!same || ((kb + 63) >> a.c.shift) >= ids_first + 64) ids = refill(a.c, kb >> a.c.shift, ids_first);
        if (!same || ((kb + 63) >> a.to.shift) >= to_first + 64) to_ids = refill(a.to, kb >> a.to.shift, to_first);
        page_to = -1;
        int mine = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = kb + 16 * i;
            const int page = __builtin_amdgcn_readlane(ids, (at >> a.c.shift) - ids_first);
            const int to = __builtin_amdgcn_readlane(to_ids, (at >> a.to.shift) - to_first);
            if (i == wave) mine = page;
            if ((lane & 3) == i && page >= 0) page_to = to;
        }
        source = uniform(a.c.k + (size_t)max(mine, 0) * a.c.k_stride + (size_t)((kb + 16 * wave) & pmask) * D);
    };
    uint32_t at[LOADS];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) at[j] = 16 * ((64 * j + lane) ^ expand_swizzle((64 * j + lane) / C));
    auto load_piece = [&](int slot, int j) { load_lds(source, at[j], lds_at + slot * IMAGE + 1024 * j); };

    const bool keys = wave < 2;
    const int d0 = (wave & 1) * (32 * NB);  // first of the wave's dims
    const int tp = (1 << a.to.shift) - 1;
    constexpr int ROT_CHUNKS = kTileKeys * (kRot / 8) / kExpandThreads;
    // A tile's results, kept until the next one's loads have been waited for, so that
    // the stores have a whole tile's time before anything waits for them.
    f16r acc[2][NB];
    u4 rot[ROT_CHUNKS];
    struct Done {
        int kb, from, to, page;
    } done = {0, 0, 0, -1};
    // Eight neighbours of one row of results: registers 8 j .. 8 j + 7 of a block hold,
    // in a lane's lower and upper partner, two runs of eight by halves; of each pair of
    // dwords the partners swap the one that belongs to the other.  The lane's run is
    // number 2 j + h.
    const auto run_of = [&](const f16r& x, int j) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lo[e] = as_u32((h2){(_Float16)x[8 * j + 2 * e], (_Float16)x[8 * j + 2 * e + 1]});
            hi[e] = as_u32((h2){(_Float16)x[8 * j + 4 + 2 * e], (_Float16)x[8 * j + 5 + 2 * e]});
        }
        const auto r0 = __builtin_amdgcn_permlane32_swap(lo[0], hi[0], false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(lo[1], hi[1], false, false);
        return (u4){r0[0], r1[0], r0[1], r1[1]};
    };
    auto store = [&] {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (keys) {
                const int pos = done.kb + 32 * p + n, page = __shfl(done.page, 2 * p + (n >> 4), 64);
                const bool live = page >= 0 && pos >= done.from && pos < done.to;
                uint16_t* to = a.to.k + (size_t)max(page, 0) * a.to.k_stride + (((size_t)head << a.to.shift) + (pos & tp)) * K + d0;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const u4 v = run_of(acc[p][b], j);
                        if (live) *reinterpret_cast<u4*>(to + 32 * b + 16 * j + 8 * h) = v;
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int pos = done.kb + 32 * p + 16 * j + 8 * h, page = __builtin_amdgcn_readlane(done.page, 2 * p + j);
                    const bool all = pos >= done.from && pos + 7 < done.to;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const u4 v = run_of(acc[p][b], j);
                        if (page < 0) continue;
                        uint16_t* to = a.to.v + (size_t)page * a.to.v_stride +
                                       ((size_t)(head * V + d0 + 32 * b + n) << a.to.shift) + (pos & tp);
                        if (all) {
                            *reinterpret_cast<u4*>(to) = v;
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (pos + e >= done.from && pos + e < done.to) to[e] = (uint16_t)(v[e >> 1] >> 16 * (e & 1));
                        }
                    }
                }
            }
        }
        // The rotary part of the keys.
#pragma unroll
        for (int i = 0; i < ROT_CHUNKS; ++i) {
            const int row = (tid + i * kExpandThreads) >> 3, c = tid & 7, pos = done.kb + row, page = __shfl(done.page, row >> 4, 64);
            if (page >= 0 && pos >= done.from && pos < done.to)
                *reinterpret_cast<u4*>(a.to.k + (size_t)page * a.to.k_stride +
                                       (((size_t)head << a.to.shift) + (pos & tp)) * K + V + 8 * c) = rot[i];
        }
    };
    aim(begin);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load_piece(0, j);
    int slot = 0;
    for (int64_t item = begin; item < end; ++item, slot ^= 1) {
        wait_for_loads<0>();
        lds_meet();  // all waves' loads are there, and the other image has been read
        const int kb = next_tile * kTileKeys, from = next_from, upto = next_to, page = page_to;
        const bool more = item + 1 < end;
        if (more) aim(item + 1);
        if (item > begin) store();
        done = {kb, from, upto, page};
        const uint8_t* image = reinterpret_cast<const uint8_t*>(lds) + slot * IMAGE;
#pragma unroll
        for (int i = 0; i < ROT_CHUNKS; ++i) {
            const int row = (tid + i * kExpandThreads) >> 3, c = tid & 7;
            rot[i] = *reinterpret_cast<const u4*>(image + row * (2 * D) + 16 * ((L / 8 + c) ^ expand_swizzle(row)));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[p][b] = (f16r)0.0f;
        constexpr int AHEAD = 3;  // operands read ahead of the products
        h8 c[AHEAD][2];
        const auto row_of = [&](int p, int s) {
            const int row = 32 * p + n;
            return *reinterpret_cast<const h8*>(image + row * (2 * D) + 16 * ((2 * s + h) ^ expand_swizzle(row)));
        };
        const auto products = [&](auto load, auto of_keys) {
#pragma unroll
            for (int s = 0; s < AHEAD; ++s)
#pragma unroll
                for (int p = 0; p < 2; ++p) c[s][p] = row_of(p, s);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
                        acc[p][b] = decltype(of_keys)::value
                                        ? __builtin_amdgcn_mfma_f32_32x32x16_f16(w[b][s], c[s % AHEAD][p], acc[p][b], 0, 0, 0)
                                        : __builtin_amdgcn_mfma_f32_32x32x16_f16(c[s % AHEAD][p], w[b][s], acc[p][b], 0, 0, 0);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (s + AHEAD < STEPS) c[s % AHEAD][p] = row_of(p, s + AHEAD);
                if (decltype(load)::value && s < LOADS) load_piece(slot ^ 1, s);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (more) {
            if (keys) products(std::true_type{}, std::true_type{});
            else products(std::true_type{}, std::false_type{});
        } else {
            if (keys) products(std::false_type{}, std::true_type{});
            else products(std::false_type{}, std::false_type{});
        }
    }
    store();
}

template <int L, int V>
static hipError_t launch_expand(const ExpandArgs& a, const DeviceInfo& dev, hipStream_t st) {
    constexpr size_t bytes = 2 * 2 * kTileKeys * (L + kRot);
    // As many workgroups as CUs, each with an equal range of all tiles.
    const long tiles = ((long)a.max_length + kTileKeys - 1) / kTileKeys * a.count;
    long ranges = dev.num_cu / a.to.kv_heads;
    ranges = ranges < 1 ? 1 : ranges > tiles ? tiles : ranges;
    std::atomic<int>& ready = PerDevice<&latent_expand_kernel<L, V>>::value[dev.device];
    if (!ready.load(std::memory_order_acquire)) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&latent_expand_kernel<L, V>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e != hipSuccess) return e;
        ready.store(1, std::memory_order_release);
    }
    hipLaunchKernelGGL((latent_expand_kernel<L, V>), dim3((unsigned)a.to.kv_heads, (unsigned)ranges), dim3(kExpandThreads),
                       bytes, st, a, (int)ranges);
    return hipGetLastError();
}

template <int L>
static hipError_t launch_expand_latent(const ExpandArgs& a, const DeviceInfo& dev, hipStream_t st) {
    return a.to.dim_v == 64 ? launch_expand<L, 64>(a, dev, st) : launch_expand<L, 128>(a, dev, st);
}

hipError_t launch_latent_expand(const ExpandArgs& a, const DeviceInfo& dev, hipStream_t st) {
    switch (a.c.dim - kRot) {
        case 128: return launch_expand_latent<128>(a, dev, st);
        case 256: return launch_expand_latent<256>(a, dev, st);
        case 512: return launch_expand_latent<512>(a, dev, st);
    }
    return hipErrorInvalidValue;  // widths are validated before
}

}  // namespace q4
