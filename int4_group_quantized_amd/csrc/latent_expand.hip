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
// [dim][position] and values as [position][dim], so that a lane holds four
// neighbours of what it stores.
#include "latent.hpp"
#include "lds_loads.hpp"

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

    // Weights: rows of the head's 2 V, 32 a block.
    h8 w[NB][STEPS];
    {
        const DequantConsts kc = make_dequant_consts();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const size_t row = (size_t)head * (2 * V) + (wave * NB + b) * 32 + n;
            const uint32_t* q = reinterpret_cast<const uint32_t*>(a.packed + row * (L / 2)) + h;
            const _Float16* sp = reinterpret_cast<const _Float16*>(a.scales) + row * (L / 128);
            const _Float16* mp = reinterpret_cast<const _Float16*>(a.mins) + row * (L / 128);
#pragma unroll
            for (int g = 0; g < L / 128; ++g) {
                const h2 s = {sp[g], sp[g]}, m = {mp[g], mp[g]};
#pragma unroll
                for (int i = 0; i < 8; ++i) w[b][8 * g + i] = weights_of(q[2 * (8 * g + i)], s, m, kc);
            }
        }
    }

    const uint32_t lds_at =
        __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) u4*)lds + 32 * D * wave);
    constexpr uint32_t IMAGE = 2 * kTileKeys * D;
    const uint16_t* source = a.c.k;
    int gone_next = 0;  // bit i: quarter i has no latent page
    auto aim = [&](int64_t item) {
        find(item);
        const int* row = a.c.table + (size_t)next_s * a.c.cols;
        const int last = next_to - 1, kb = next_tile * kTileKeys;
        const int page = page_of(a.c, row, min(kb + 16 * (lane & 3), last));
        gone_next = (int)(__ballot(page < 0) & 15);
        const int mine = max(__builtin_amdgcn_readlane(page, wave), 0);
        source = uniform(a.c.k + (size_t)mine * a.c.k_stride + (size_t)((kb + 16 * wave) & pmask) * D);
    };
    auto load_piece = [&](int slot, int j) {
        const int place = 64 * j + lane;
        load_lds(source, 16 * (place ^ expand_swizzle(place / C)), lds_at + slot * IMAGE + 1024 * j);
    };

    const bool keys = wave < 2;
    const int d0 = (wave & 1) * (32 * NB);  // first of the wave's dims
    aim(begin);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) load_piece(0, j);
    int slot = 0;
    for (int64_t item = begin; item < end; ++item, slot ^= 1) {
        const int seq = next_s, kb = next_tile * kTileKeys, from = next_from, upto = next_to, gone = gone_next;
        wait_for_loads<0>();
        lds_meet();  // all waves' loads are there, and the other image has been read
        const bool more = item + 1 < end;
        // Where this tile's keys and values go: pages by quarter.
        int to_page;
        {
            const int* row = a.to.table + (size_t)seq * a.to.cols;
            const int at = kb + 16 * (lane & 3);
            const bool in = (at >> a.to.shift) < a.to.cols;
            to_page = in ? page_of(a.to, row, at) : -1;
            if (gone >> (lane & 3) & 1) to_page = -1;
        }
        const auto page_to = [&](int quarter) { return __shfl(to_page, quarter, 64); };
        if (more) aim(item + 1);
        const uint8_t* image = reinterpret_cast<const uint8_t*>(lds) + slot * IMAGE;
        f16r acc[2][NB];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[p][b] = (f16r)0.0f;
        const auto row_of = [&](int p, int s) {
            const int row = 32 * p + n;
            return *reinterpret_cast<const h8*>(image + row * (2 * D) + 16 * ((2 * s + h) ^ expand_swizzle(row)));
        };
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const h8 c[2] = {row_of(0, s), row_of(1, s)};
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    acc[p][b] = keys ? __builtin_amdgcn_mfma_f32_32x32x16_f16(w[b][s], c[p], acc[p][b], 0, 0, 0)
                                     : __builtin_amdgcn_mfma_f32_32x32x16_f16(c[p], w[b][s], acc[p][b], 0, 0, 0);
            if (more && s < LOADS) load_piece(slot ^ 1, s);
        }
        const int tp = (1 << a.to.shift) - 1;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (keys) {
                const int pos = kb + 32 * p + n, page = page_to(2 * p + (n >> 4));
                if (page >= 0 && pos >= from && pos < upto) {
                    uint16_t* to = a.to.k + (size_t)page * a.to.k_stride + (((size_t)head << a.to.shift) + (pos & tp)) * K + d0;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint2 v;
                            v.x = as_u32((h2){(_Float16)acc[p][b][4 * i], (_Float16)acc[p][b][4 * i + 1]});
                            v.y = as_u32((h2){(_Float16)acc[p][b][4 * i + 2], (_Float16)acc[p][b][4 * i + 3]});
                            *reinterpret_cast<uint2*>(to + 32 * b + 8 * i + 4 * h) = v;
                        }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = kb + 32 * p + 8 * i + 4 * h, page = __builtin_amdgcn_readlane(to_page, 2 * p + (i >> 1));
                    if (page < 0 || pos + 3 < from || pos >= upto) continue;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint16_t* to = a.to.v + (size_t)page * a.to.v_stride +
                                       ((size_t)(head * V + d0 + 32 * b + n) << a.to.shift) + (pos & tp);
                        uint16_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = __builtin_bit_cast(uint16_t, (_Float16)acc[p][b][4 * i + e]);
                        if (pos >= from && pos + 3 < upto) {
                            *reinterpret_cast<uint2*>(to) = {(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (pos + e >= from && pos + e < upto) to[e] = v[e];
                        }
                    }
                }
            }
        }
        // The rotary part of the keys.
#pragma unroll
        for (int i = tid; i < kTileKeys * (kRot / 8); i += kExpandThreads) {
            const int row = i >> 3, c = i & 7, pos = kb + row, page = page_to(row >> 4);
            if (page >= 0 && pos >= from && pos < upto) {
                const u4 v = *reinterpret_cast<const u4*>(image + row * (2 * D) + 16 * ((L / 8 + c) ^ expand_swizzle(row)));
                *reinterpret_cast<u4*>(a.to.k + (size_t)page * a.to.k_stride +
                                       (((size_t)head << a.to.shift) + (pos & tp)) * K + V + 8 * c) = v;
            }
        }
    }
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
