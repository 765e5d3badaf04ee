// C ABI of the int4 group-128 library: argument validation (host only, no
// HIP call before it passes), per-device properties, dispatch to the kernel
// launchers and status reporting.
#include "q4g128.h"

#include <float.h>
#include <hip/hip_runtime.h>

#include <algorithm>
#include <mutex>
#include <utility>
#include <vector>

#include "latent.hpp"
#include "launch.hpp"

namespace {

thread_local int32_t g_last_hip_error = 0;

constexpr int kMaxDevices = q4::kMaxDevices;
q4::DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

q4_status device_error(hipError_t e) {
    g_last_hip_error = (int32_t)e;
    (void)hipGetLastError();  // clear the sticky per-thread error for the caller
    return Q4_EDEVICE;
}

// Properties of the current device, queried once per device.
q4_status current_device(q4::DeviceInfo* out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return device_error(e);
    if (dev < 0 || dev >= kMaxDevices) return device_error(hipErrorInvalidDevice);
    std::lock_guard<std::mutex> lock(g_dev_mu);
    q4::DeviceInfo& d = g_dev[dev];
    if (d.device != dev) {
        int cu = 0, lds = 0, lds_optin = 0;
        e = hipDeviceGetAttribute(&cu, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess) return device_error(e);
        e = hipDeviceGetAttribute(&lds, hipDeviceAttributeMaxSharedMemoryPerBlock, dev);
        if (e != hipSuccess) return device_error(e);
        if (hipDeviceGetAttribute(&lds_optin, hipDeviceAttributeSharedMemPerBlockOptin, dev) != hipSuccess) {
            (void)hipGetLastError();
            lds_optin = 0;
        }
        d.num_cu = cu;
        d.max_lds = (size_t)(lds_optin > lds ? lds_optin : lds);
        d.device = dev;
    }
    *out = d;
    return Q4_OK;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// End of [p, p + bytes), saturated at the top of the address space.
uintptr_t end_of(const void* p, size_t bytes) {
    const uintptr_t a = (uintptr_t)p;
    return bytes > UINTPTR_MAX - a ? UINTPTR_MAX : a + bytes;
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    return (uintptr_t)a < end_of(b, nb) && (uintptr_t)b < end_of(a, na);
}

q4_status check_nk(int64_t n, int64_t k) {
    if (n <= 0) return Q4_EINVAL;
    if (k < Q4G128_GROUP || k % Q4G128_GROUP != 0 || k > Q4G128_MAX_K) return Q4_ESHAPE;
    if (n > Q4G128_MAX_N) return Q4_ESHAPE;
    return Q4_OK;
}

// Shared checks of the three product entry points; `rows` = B or M.
q4_status check_product(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                        const uint16_t* X, const float* Y, int64_t n, int64_t k, int64_t rows) {
    if (!packed || !scales || !mins || !X || !Y) return Q4_EINVAL;
    q4_status s = check_nk(n, k);
    if (s != Q4_OK) return s;
    if (rows > Q4G128_MAX_N) return Q4_ESHAPE;
    if (!aligned(packed, 16) || !aligned(X, 16) || !aligned(scales, 2) || !aligned(mins, 2) ||
        !aligned(Y, 4))
        return Q4_EALIGN;
    const size_t g = (size_t)(k / Q4G128_GROUP);
    // rows and n are below 2^31, so their product fits; its byte count may not.
    const uint64_t yelems = (uint64_t)rows * (uint64_t)n;
    if (yelems > UINT64_MAX / sizeof(float)) return Q4_ESHAPE;
    const size_t ybytes = (size_t)yelems * sizeof(float);
    if (overlaps(Y, ybytes, packed, (size_t)n * (size_t)k / 2) ||
        overlaps(Y, ybytes, scales, (size_t)n * g * 2) || overlaps(Y, ybytes, mins, (size_t)n * g * 2) ||
        overlaps(Y, ybytes, X, (size_t)rows * (size_t)k * 2))
        return Q4_EINVAL;
    return Q4_OK;
}

q4::GemvArgs make_args(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                       const uint16_t* x, float* y, int64_t n, int64_t k) {
    q4::GemvArgs a;
    a.packed = packed;
    a.scales = scales;
    a.mins = mins;
    a.x = x;
    a.y = y;
    a.n = (int)n;
    a.k = (int)k;
    return a;
}

// Checks the cache descriptor and fills the kernels' form of it.
q4_status check_cache(const q4g128_kv_cache* c, int64_t heads, q4::KvCache* out) {
    if (!c || !c->k || !c->v || !c->table) return Q4_EINVAL;
    if (c->pages < 1 || c->sequences < 1 || c->table_cols < 1 || c->kv_heads < 1 || heads < 1) return Q4_EINVAL;
    if (!q4::attn_dim_supported(c->dim)) return Q4_ESHAPE;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0) return Q4_ESHAPE;
    if (heads > Q4G128_MAX_HEADS || heads % c->kv_heads != 0 || heads / c->kv_heads > Q4G128_MAX_GROUP)
        return Q4_ESHAPE;
    if (c->pages > Q4G128_MAX_N || c->sequences > Q4G128_MAX_N || c->table_cols > Q4G128_MAX_N / c->page)
        return Q4_ESHAPE;
    const int64_t per_page = (int64_t)c->kv_heads * c->page * c->dim;
    if (c->k_stride < per_page || c->v_stride < per_page || c->k_stride % 8 != 0 || c->v_stride % 8 != 0 ||
        c->k_stride > INT64_MAX / 4 / c->pages || c->v_stride > INT64_MAX / 4 / c->pages)
        return Q4_ESHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4)) return Q4_EALIGN;
    out->k = c->k;
    out->v = c->v;
    out->table = c->table;
    out->k_stride = c->k_stride;
    out->v_stride = c->v_stride;
    out->pages = (int)c->pages;
    out->sequences = (int)c->sequences;
    out->cols = (int)c->table_cols;
    out->kv_heads = c->kv_heads;
    out->dim = out->dim_v = c->dim;
    out->shift = __builtin_ctz((unsigned)c->page);
    return Q4_OK;
}

// Checks a cache of expanded keys (value + 64 columns) and values, one kv head per
// head: dim is the values' width.
q4_status check_expanded(const q4g128_kv_cache* c, q4::KvCache* out) {
    if (!c || !c->k || !c->v || !c->table) return Q4_EINVAL;
    if (c->pages < 1 || c->sequences < 1 || c->table_cols < 1 || c->kv_heads < 1) return Q4_EINVAL;
    if (!q4::value_supported(c->dim) || c->kv_heads > Q4G128_MAX_HEADS) return Q4_ESHAPE;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0) return Q4_ESHAPE;
    if (c->pages > Q4G128_MAX_N || c->sequences > Q4G128_MAX_N || c->table_cols > Q4G128_MAX_N / c->page)
        return Q4_ESHAPE;
    const int64_t cell = (int64_t)c->kv_heads * c->page;
    if (c->k_stride < cell * (c->dim + q4::kRot) || c->v_stride < cell * c->dim || c->k_stride % 8 != 0 ||
        c->v_stride % 8 != 0 || c->k_stride > INT64_MAX / 4 / c->pages || c->v_stride > INT64_MAX / 4 / c->pages)
        return Q4_ESHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4)) return Q4_EALIGN;
    out->k = c->k;
    out->v = c->v;
    out->table = c->table;
    out->k_stride = c->k_stride;
    out->v_stride = c->v_stride;
    out->pages = (int)c->pages;
    out->sequences = (int)c->sequences;
    out->cols = (int)c->table_cols;
    out->kv_heads = c->kv_heads;
    out->dim = c->dim + q4::kRot;
    out->dim_v = c->dim;
    out->shift = __builtin_ctz((unsigned)c->page);
    return Q4_OK;
}

// Bytes from the first to past the last element of a pool of rows `dim` wide.
size_t pool_bytes(const q4::KvCache& c, long stride, int dim) {
    return ((size_t)(c.pages - 1) * (size_t)stride + ((size_t)c.kv_heads * (size_t)dim << c.shift)) * 2;
}
size_t k_bytes(const q4::KvCache& c) { return pool_bytes(c, c.k_stride, c.dim); }
size_t v_bytes(const q4::KvCache& c) { return c.v ? pool_bytes(c, c.v_stride, c.dim_v) : 0; }
size_t table_bytes(const q4::KvCache& c) { return (size_t)c.sequences * (size_t)c.cols * 4; }

// Pages of one pool: `cell` bytes each, `stride` bytes from one to the next, `bytes` in all.
struct Pool {
    const void* p;
    size_t stride, cell, bytes;
};
Pool k_pool(const q4::KvCache& c) {
    return {c.k, (size_t)c.k_stride * 2, ((size_t)c.kv_heads * (size_t)c.dim << c.shift) * 2, k_bytes(c)};
}
Pool v_pool(const q4::KvCache& c) {
    return {c.v, (size_t)c.v_stride * 2, ((size_t)c.kv_heads * (size_t)c.dim_v << c.shift) * 2, v_bytes(c)};
}

// Whether two pools share an element.  Pools whose pages interleave (parts of one
// larger pool) overlap as ranges without sharing any.
bool pools_meet(const Pool& a, const Pool& b) {
    if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.stride != b.stride) return true;
    const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p, stride = a.stride;
    // How far a page of b begins behind one of a.
    const uintptr_t behind = q >= p ? (q - p) % stride : (stride - (p - q) % stride) % stride;
    return behind < a.cell || behind > stride - b.cell;
}
bool pools_meet(const q4::KvCache& c) { return pools_meet(k_pool(c), v_pool(c)); }

// Whether [p, p + bytes) meets one of the cache's pools or its table.
bool hits_cache(const q4::KvCache& c, const void* p, size_t bytes) {
    return overlaps(p, bytes, c.k, k_bytes(c)) || (c.v && overlaps(p, bytes, c.v, v_bytes(c))) ||
           overlaps(p, bytes, c.table, table_bytes(c));
}

// Shared checks of the two attention calls; `rows` = batch or tokens.
q4_status check_attention(const uint16_t* q, const q4g128_kv_cache* cache, const int32_t* lengths, int64_t max_length,
                          int64_t rows, int64_t sequences, int64_t heads, const q4g128_attn_options* o, uint16_t* out,
                          void* workspace, int64_t workspace_bytes, int64_t workspace_needed, q4::AttnArgs* a,
                          bool expanded = false) {
    if (!q || !lengths || !o || !out || rows < 1 || sequences < 1 || max_length < 1) return Q4_EINVAL;
    q4_status s = expanded ? check_expanded(cache, &a->c) : check_cache(cache, heads, &a->c);
    if (s != Q4_OK) return s;
    if (rows > Q4G128_MAX_TOKENS || sequences > Q4G128_MAX_SEQUENCES || sequences > cache->sequences ||
        max_length > cache->table_cols * cache->page)
        return Q4_ESHAPE;
    // written so that NaN fails
    if (!(o->scale > 0.0f && o->scale <= FLT_MAX) || !(o->softcap >= 0.0f && o->softcap <= FLT_MAX) || o->window < 0 ||
        (o->prefix && o->window > 0))
        return Q4_EINVAL;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(o->slopes, 4) ||
        !aligned(o->prefix, 4) || !aligned(workspace, 16))
        return Q4_EALIGN;
    if (workspace_needed > 0 && (!workspace || workspace_bytes < workspace_needed)) return Q4_EINVAL;
    const size_t qbytes = (size_t)rows * (size_t)heads * (size_t)a->c.dim * 2;
    const size_t obytes = (size_t)rows * (size_t)heads * (size_t)a->c.dim_v * 2;
    const size_t seqbytes = (size_t)sequences * 4, wsbytes = (size_t)workspace_needed;
    if (hits_cache(a->c, out, obytes) || overlaps(out, obytes, q, qbytes) || overlaps(out, obytes, lengths, seqbytes) ||
        (o->slopes && overlaps(out, obytes, o->slopes, (size_t)heads * 4)) ||
        (o->prefix && overlaps(out, obytes, o->prefix, seqbytes)))
        return Q4_EINVAL;
    if (wsbytes > 0 &&
        (hits_cache(a->c, workspace, wsbytes) || overlaps(workspace, wsbytes, q, qbytes) ||
         overlaps(workspace, wsbytes, out, obytes) || overlaps(workspace, wsbytes, lengths, seqbytes) ||
         (o->slopes && overlaps(workspace, wsbytes, o->slopes, (size_t)heads * 4)) ||
         (o->prefix && overlaps(workspace, wsbytes, o->prefix, seqbytes))))
        return Q4_EINVAL;
    a->q = q;
    a->lengths = lengths;
    a->max_length = (int)max_length;
    a->rows = (int)rows;
    a->heads = (int)heads;
    a->group = (int)(heads / cache->kv_heads);
    a->scale = o->scale;
    a->softcap = o->softcap;
    // A window of max_length positions or more hides nothing.
    a->window = o->window >= max_length ? 0 : (int)o->window;
    a->slopes = o->slopes;
    a->prefix = o->prefix;
    a->out = out;
    a->workspace = (float*)workspace;
    a->q_starts = nullptr;
    a->masks = nullptr;
    a->max_new = (int)rows;
    a->count = (int)sequences;
    return Q4_OK;
}

// Checks a latent cache and fills the kernels' form of it: a cache without V, of
// one kv head.
q4_status check_latent(const q4g128_latent_cache* c, q4::KvCache* out) {
    if (!c || !c->rows || !c->table) return Q4_EINVAL;
    if (c->pages < 1 || c->sequences < 1 || c->table_cols < 1) return Q4_EINVAL;
    if (!q4::latent_supported(c->latent)) return Q4_ESHAPE;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0) return Q4_ESHAPE;
    if (c->pages > Q4G128_MAX_N || c->sequences > Q4G128_MAX_N || c->table_cols > Q4G128_MAX_N / c->page)
        return Q4_ESHAPE;
    const int dim = c->latent + q4::kRot;
    if (c->stride < (int64_t)c->page * dim || c->stride % 8 != 0 || c->stride > INT64_MAX / 4 / c->pages) return Q4_ESHAPE;
    if (!aligned(c->rows, 16) || !aligned(c->table, 4)) return Q4_EALIGN;
    out->k = c->rows;
    out->v = nullptr;
    out->table = c->table;
    out->k_stride = c->stride;
    out->v_stride = 0;
    out->pages = (int)c->pages;
    out->sequences = (int)c->sequences;
    out->cols = (int)c->table_cols;
    out->kv_heads = 1;
    out->dim = out->dim_v = dim;
    out->shift = __builtin_ctz((unsigned)c->page);
    return Q4_OK;
}

// Row numbers and masks of new tokens, against what a call writes.
q4_status check_new(const int32_t* q_starts, const uint64_t* masks, int64_t tokens, int64_t count, const void* out,
                    size_t outbytes, const void* workspace, size_t wsbytes) {
    if (!aligned(q_starts, 4) || !aligned(masks, 8)) return Q4_EALIGN;
    const size_t sbytes = (size_t)(count + 1) * 4, mbytes = (size_t)tokens * 8;
    if (overlaps(out, outbytes, q_starts, sbytes) || overlaps(workspace, wsbytes, q_starts, sbytes) ||
        (masks && (overlaps(out, outbytes, masks, mbytes) || overlaps(workspace, wsbytes, masks, mbytes))))
        return Q4_EINVAL;
    return Q4_OK;
}

// The rest of the two keep calls' checks, and their launch.  a->c is filled.
q4_status keep_tokens(q4::KeepArgs* a, const int32_t* starts, const int32_t* keep_starts, const int32_t* keep,
                      int64_t total, int64_t count, void* stream) {
    if (!starts || !keep_starts || (!keep && total > 0) || total < 0 || count < 1) return Q4_EINVAL;
    if (count > Q4G128_MAX_SEQUENCES || count > a->c.sequences || total > Q4G128_MAX_TOKENS) return Q4_ESHAPE;
    if (!aligned(starts, 4) || !aligned(keep_starts, 4) || !aligned(keep, 4)) return Q4_EALIGN;
    const size_t kbytes = k_bytes(a->c), vbytes = v_bytes(a->c), tbytes = table_bytes(a->c);
    const void* in[] = {a->c.table, starts, keep_starts, keep};
    const size_t inbytes[] = {tbytes, (size_t)count * 4, (size_t)(count + 1) * 4, (size_t)total * 4};
    for (int i = 0; i < 4; ++i)
        if (in[i] && (overlaps(a->c.k, kbytes, in[i], inbytes[i]) ||
                      (vbytes > 0 && overlaps(a->c.v, vbytes, in[i], inbytes[i]))))
            return Q4_EINVAL;
    if (a->c.v && pools_meet(a->c)) return Q4_EINVAL;
    if (total == 0) return Q4_OK;
    a->starts = starts;
    a->keep_starts = keep_starts;
    a->keep = keep;
    a->total = (int)total;
    a->count = (int)count;
    hipError_t e = q4::launch_cache_keep(*a, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

}  // namespace

extern "C" {

q4_status q4g128_pack(const uint8_t* codes, uint8_t* packed, int64_t n, int64_t k, void* stream) {
    if (!codes || !packed) return Q4_EINVAL;
    q4_status s = check_nk(n, k);
    if (s != Q4_OK) return s;
    if (!aligned(codes, 16) || !aligned(packed, 16)) return Q4_EALIGN;
    if (overlaps(packed, (size_t)n * (size_t)k / 2, codes, (size_t)n * (size_t)k)) return Q4_EINVAL;
    hipError_t e = q4::launch_pack(codes, packed, n, k, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_quantize(const float* W, uint8_t* packed, uint16_t* scales, uint16_t* mins, int64_t n,
                          int64_t k, void* stream) {
    if (!W || !packed || !scales || !mins) return Q4_EINVAL;
    q4_status s = check_nk(n, k);
    if (s != Q4_OK) return s;
    const size_t groups = (size_t)n * (size_t)(k / Q4G128_GROUP);
    if (groups > (size_t)q4::kQuantizeMaxGroups) return Q4_ESHAPE;
    if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales, 2) || !aligned(mins, 2)) return Q4_EALIGN;
    const size_t wbytes = (size_t)n * (size_t)k * 4, pbytes = (size_t)n * (size_t)k / 2, gbytes = groups * 2;
    if (overlaps(packed, pbytes, W, wbytes) || overlaps(scales, gbytes, W, wbytes) ||
        overlaps(mins, gbytes, W, wbytes) || overlaps(packed, pbytes, scales, gbytes) ||
        overlaps(packed, pbytes, mins, gbytes) || overlaps(scales, gbytes, mins, gbytes))
        return Q4_EINVAL;
    hipError_t e = q4::launch_quantize(W, packed, scales, mins, n, k, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemv(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                      const uint16_t* x, float* y, int64_t n, int64_t k, void* stream) {
    q4_status s = check_product(packed, scales, mins, x, y, n, k, 1);
    if (s != Q4_OK) return s;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_gemv(make_args(packed, scales, mins, x, y, n, k), dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemv_grouped(const q4g128_gemv_desc* descs, int64_t count, void* stream) {
    if (!descs || count < 1 || count > Q4G128_MAX_GROUPED) return Q4_EINVAL;
    std::vector<q4::GemvArgs> list((size_t)count);
    // Outputs must be pairwise disjoint and disjoint from every input.
    std::vector<std::pair<uintptr_t, uintptr_t>> outs((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        const q4g128_gemv_desc& d = descs[i];
        q4_status s = check_product(d.packed, d.scales, d.mins, d.x, d.y, d.n, d.k, 1);
        if (s != Q4_OK) return s;
        list[(size_t)i] = make_args(d.packed, d.scales, d.mins, d.x, d.y, d.n, d.k);
        outs[(size_t)i] = {(uintptr_t)d.y, end_of(d.y, (size_t)d.n * sizeof(float))};
    }
    std::sort(outs.begin(), outs.end());
    for (size_t i = 1; i < outs.size(); ++i)
        if (outs[i - 1].second > outs[i].first) return Q4_EINVAL;
    // The only output that can overlap [lo, hi) is the last one starting below hi.
    auto hits_output = [&](const void* p, size_t bytes) {
        const uintptr_t lo = (uintptr_t)p, hi = end_of(p, bytes);
        auto it = std::lower_bound(outs.begin(), outs.end(), std::make_pair(hi, (uintptr_t)0));
        if (it == outs.begin()) return false;
        --it;
        return it->second > lo;
    };
    for (int64_t i = 0; i < count; ++i) {
        const q4g128_gemv_desc& d = descs[i];
        const size_t g = (size_t)(d.k / Q4G128_GROUP);
        if (hits_output(d.packed, (size_t)d.n * (size_t)d.k / 2) || hits_output(d.scales, (size_t)d.n * g * 2) ||
            hits_output(d.mins, (size_t)d.n * g * 2) || hits_output(d.x, (size_t)d.k * 2))
            return Q4_EINVAL;
    }
    q4::DeviceInfo dev;
    q4_status s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_gemv_group(list.data(), (int)count, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemm_small_batch(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                                  const uint16_t* X, float* Y, int64_t n, int64_t k, int64_t b,
                                  void* stream) {
    if (b < 1 || b > Q4G128_MAX_BATCH) return Q4_EINVAL;
    q4_status s = check_product(packed, scales, mins, X, Y, n, k, b);
    if (s != Q4_OK) return s;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_small_batch(make_args(packed, scales, mins, X, Y, n, k), X, Y, (int)b, dev,
                                          (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemm_prefill(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                              const uint16_t* X, float* Y, int64_t n, int64_t k, int64_t m,
                              void* stream) {
    if (m < 1) return Q4_EINVAL;
    q4_status s = check_product(packed, scales, mins, X, Y, n, k, m);
    if (s != Q4_OK) return s;
    if (((n + 63) / 64) * ((m + 15) / 16) > 0x7FFFFFFFLL) return Q4_ESHAPE;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_prefill(make_args(packed, scales, mins, X, Y, n, k), X, Y, (int)m, dev,
                                      (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemm_prefill_epilogue(const uint8_t* packed, const uint16_t* scales, const uint16_t* mins,
                                       const uint16_t* X, float* Y, int64_t n, int64_t k, int64_t m,
                                       void* stream) {
    if (m < 1) return Q4_EINVAL;
    q4_status s = check_product(packed, scales, mins, X, Y, n, k, m);
    if (s != Q4_OK) return s;
    if ((size_t)m * (size_t)n > (size_t)0x7FFFFFFFFFFFLL) return Q4_ESHAPE;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_prefill_epilogue(make_args(packed, scales, mins, X, Y, n, k), X, Y, (int)m, dev,
                                               (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_gemv_int8(const int8_t* q, const uint16_t* scales, const uint16_t* x, float* y, int64_t n,
                           int64_t k, void* stream) {
    if (!q || !scales || !x || !y) return Q4_EINVAL;
    if (n <= 0) return Q4_EINVAL;
    if (k < Q4G128_GROUP || k % Q4G128_GROUP != 0 || k > Q4G128_INT8_MAX_K || n > Q4G128_MAX_N) return Q4_ESHAPE;
    if (!aligned(q, 16) || !aligned(x, 16) || !aligned(scales, 2) || !aligned(y, 4)) return Q4_EALIGN;
    const size_t ybytes = (size_t)n * sizeof(float);
    if (overlaps(y, ybytes, q, (size_t)n * (size_t)k) || overlaps(y, ybytes, scales, (size_t)n * 2) ||
        overlaps(y, ybytes, x, (size_t)k * 2))
        return Q4_EINVAL;
    q4::DeviceInfo dev;
    q4_status s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_head_int8(q, scales, x, y, n, k, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_rope_append(const float* qkv, int64_t ld, int64_t tokens, int32_t heads,
                             const q4g128_kv_cache* cache, const int32_t* seq, const int32_t* positions,
                             const float* inv_freq, int32_t rot, int32_t interleaved, float mscale,
                             const uint16_t* q_norm, const uint16_t* k_norm, float eps, uint16_t* q, void* stream) {
    return q4g128_rope_append_slots(qkv, ld, tokens, heads, cache, seq, positions, positions, inv_freq, rot,
                                    interleaved, mscale, q_norm, k_norm, eps, q, stream);
}

q4_status q4g128_rope_append_slots(const float* qkv, int64_t ld, int64_t tokens, int32_t heads,
                                   const q4g128_kv_cache* cache, const int32_t* seq, const int32_t* positions,
                                   const int32_t* slots, const float* inv_freq, int32_t rot, int32_t interleaved,
                                   float mscale, const uint16_t* q_norm, const uint16_t* k_norm, float eps, uint16_t* q,
                                   void* stream) {
    if (!qkv || !positions || !slots || !q || tokens < 1) return Q4_EINVAL;
    q4::AppendArgs a;
    q4_status s = check_cache(cache, heads, &a.c);
    if (s != Q4_OK) return s;
    const int64_t dim = cache->dim, columns = ((int64_t)heads + 2 * (int64_t)cache->kv_heads) * dim;
    if (rot < 0 || rot > dim || rot % 4 != 0 || tokens > Q4G128_MAX_TOKENS || ld < columns || ld % 4 != 0 ||
        ld > INT64_MAX / 8 / tokens)
        return Q4_ESHAPE;
    if ((rot > 0 && !inv_freq) || !(eps >= 0.0f)) return Q4_EINVAL;  // written so that NaN fails
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(seq, 4) || !aligned(positions, 4) || !aligned(slots, 4) ||
        !aligned(inv_freq, 4) || !aligned(q_norm, 2) || !aligned(k_norm, 2))
        return Q4_EALIGN;
    const size_t qbytes = (size_t)tokens * (size_t)heads * (size_t)dim * 2, nbytes = (size_t)dim * 2;
    const void* in[] = {qkv, seq, positions, slots, inv_freq, q_norm, k_norm};
    const size_t inbytes[] = {((size_t)(tokens - 1) * (size_t)ld + (size_t)columns) * 4, (size_t)tokens * 4,
                              (size_t)tokens * 4, (size_t)tokens * 4, (size_t)rot * 2, nbytes, nbytes};
    if (pools_meet(a.c)) return Q4_EINVAL;
    const size_t kbytes = k_bytes(a.c), vbytes = v_bytes(a.c);
    const size_t tbytes = table_bytes(a.c);
    if (hits_cache(a.c, q, qbytes) || overlaps(a.c.k, kbytes, a.c.table, tbytes) ||
        overlaps(a.c.v, vbytes, a.c.table, tbytes))
        return Q4_EINVAL;
    for (int i = 0; i < 7; ++i)
        if (in[i] && (overlaps(q, qbytes, in[i], inbytes[i]) || overlaps(a.c.k, kbytes, in[i], inbytes[i]) ||
                      overlaps(a.c.v, vbytes, in[i], inbytes[i])))
            return Q4_EINVAL;
    a.qkv = qkv;
    a.ld = ld;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.seq = seq;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.mscale = mscale;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.eps = eps;
    a.q = q;
    hipError_t e = q4::launch_rope_append(a, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_cache_keep(const q4g128_kv_cache* cache, const int32_t* starts, const int32_t* keep_starts,
                            const int32_t* keep, int64_t total, int64_t count, void* stream) {
    q4::KeepArgs a;
    q4_status s = check_cache(cache, cache ? cache->kv_heads : 0, &a.c);
    if (s != Q4_OK) return s;
    return keep_tokens(&a, starts, keep_starts, keep, total, count, stream);
}

int64_t q4g128_attn_decode_workspace(int64_t batch, int32_t heads, int32_t dim) {
    if (batch < 1 || heads < 1) return Q4_EINVAL;
    if (batch > Q4G128_MAX_SEQUENCES || heads > Q4G128_MAX_HEADS || !q4::attn_dim_supported(dim)) return Q4_ESHAPE;
    return q4::attn_decode_workspace(batch, heads, dim);
}

q4_status q4g128_attn_decode(const uint16_t* q, const q4g128_kv_cache* cache, const int32_t* lengths,
                             int64_t max_length, int64_t batch, int32_t heads, const q4g128_attn_options* options,
                             uint16_t* out, void* workspace, int64_t workspace_bytes, void* stream) {
    q4::AttnArgs a;
    const int64_t need = cache ? q4g128_attn_decode_workspace(batch, heads, cache->dim) : Q4_EINVAL;
    if (need < 0) return (q4_status)need;
    if (options && options->prefix) return Q4_EINVAL;
    q4_status s = check_attention(q, cache, lengths, max_length, batch, batch, heads, options, out, workspace,
                                  workspace_bytes, need, &a);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_attn_decode(a, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

int64_t q4g128_attn_prefill_workspace(int64_t tokens, int64_t count, int32_t heads, int32_t kv_heads, int32_t dim,
                                      int64_t max_length) {
    if (tokens < 1 || count < 1 || heads < 1 || kv_heads < 1 || max_length < 1) return Q4_EINVAL;
    if (tokens > Q4G128_MAX_TOKENS || count > Q4G128_MAX_SEQUENCES || heads > Q4G128_MAX_HEADS ||
        heads % kv_heads != 0 || heads / kv_heads > Q4G128_MAX_GROUP || !q4::attn_dim_supported(dim) ||
        max_length > Q4G128_MAX_N)
        return Q4_ESHAPE;
    return q4::attn_prefill_workspace(tokens, count, heads, kv_heads, dim, dim, max_length);
}

q4_status q4g128_attn_prefill(const uint16_t* q, const q4g128_kv_cache* cache, const int32_t* q_starts,
                              const int32_t* lengths, int64_t max_length, int64_t tokens, int64_t count, int32_t heads,
                              const q4g128_attn_options* options, uint16_t* out, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    q4::AttnArgs a;
    if (!q_starts) return Q4_EINVAL;
    const int64_t need =
        cache ? q4g128_attn_prefill_workspace(tokens, count, heads, cache->kv_heads, cache->dim, max_length) : Q4_EINVAL;
    if (need < 0) return (q4_status)need;
    q4_status s = check_attention(q, cache, lengths, max_length, tokens, count, heads, options, out, workspace,
                                  workspace_bytes, need, &a);
    if (s != Q4_OK) return s;
    if (!aligned(q_starts, 4)) return Q4_EALIGN;
    const size_t sbytes = (size_t)(count + 1) * 4;
    if (overlaps(out, (size_t)tokens * (size_t)heads * (size_t)cache->dim * 2, q_starts, sbytes) ||
        (need > 0 && overlaps(workspace, (size_t)need, q_starts, sbytes)))
        return Q4_EINVAL;
    a.q_starts = q_starts;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_attn_prefill(a, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

int64_t q4g128_attn_tree_workspace(int64_t tokens, int64_t count, int32_t heads, int32_t kv_heads, int32_t dim,
                                   int64_t max_new, int64_t max_length) {
    if (tokens < 1 || count < 1 || heads < 1 || kv_heads < 1 || max_new < 1 || max_length < 1) return Q4_EINVAL;
    if (tokens > Q4G128_MAX_TOKENS || count > Q4G128_MAX_SEQUENCES || max_length > Q4G128_MAX_N || heads > Q4G128_MAX_HEADS || heads % kv_heads != 0 || heads / kv_heads > Q4G128_MAX_GROUP ||
        !q4::attn_dim_supported(dim) || max_new > Q4G128_MAX_DRAFT)
        return Q4_ESHAPE;
    return q4::attn_prefill_workspace(tokens, count, heads, kv_heads, dim, dim, max_length, max_new);
}

q4_status q4g128_attn_tree(const uint16_t* q, const q4g128_kv_cache* cache, const int32_t* q_starts,
                           const int32_t* lengths, const uint64_t* masks, int64_t max_new, int64_t max_length,
                           int64_t tokens, int64_t count, int32_t heads, const q4g128_attn_options* options,
                           uint16_t* out, void* workspace, int64_t workspace_bytes, void* stream) {
    q4::AttnArgs a;
    if (!q_starts) return Q4_EINVAL;
    const int64_t need = cache ? q4g128_attn_tree_workspace(tokens, count, heads, cache->kv_heads, cache->dim, max_new,
                                                            max_length)
                               : Q4_EINVAL;
    if (need < 0) return (q4_status)need;
    if (options && options->prefix) return Q4_EINVAL;
    q4_status s = check_attention(q, cache, lengths, max_length, tokens, count, heads, options, out, workspace,
                                  workspace_bytes, need, &a);
    if (s != Q4_OK) return s;
    s = check_new(q_starts, masks, tokens, count, out, (size_t)tokens * (size_t)heads * (size_t)cache->dim * 2,
                  workspace, (size_t)need);
    if (s != Q4_OK) return s;
    a.q_starts = q_starts;
    a.masks = masks;
    a.max_new = (int)max_new;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_attn_tree(a, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_latent_append(const float* kv, int64_t ld, int64_t tokens, const q4g128_latent_cache* cache,
                               const int32_t* seq, const int32_t* positions, const int32_t* slots,
                               const float* inv_freq, int32_t interleaved, float mscale, const uint16_t* norm, float eps,
                               const float* q_main, int64_t main_ld, int64_t main_head, int32_t main,
                               const float* q_rot, int64_t rot_ld, int64_t rot_head, int32_t heads, uint16_t* q,
                               void* stream) {
    if (!kv || !positions || !slots || tokens < 1 || heads < 0 || (heads > 0 && (!q_main || !q_rot || !q)))
        return Q4_EINVAL;
    q4::LatentAppendArgs a;
    q4_status s = check_latent(cache, &a.c);
    if (s != Q4_OK) return s;
    const int64_t row = a.c.dim, wide = (int64_t)main + q4::kRot;
    if (tokens > Q4G128_MAX_TOKENS || ld < row || ld % 4 != 0 || ld > INT64_MAX / 8 / tokens || heads > Q4G128_MAX_HEADS)
        return Q4_ESHAPE;
    if (heads > 0) {
        if (main < 8 || main > Q4G128_LATENT_MAX_MAIN || main % 8 != 0) return Q4_ESHAPE;
        // Strides are of views of one tensor, in either order of tokens and heads.
        const int64_t most = INT64_MAX / 16 / tokens / heads;
        if (main_ld < main || main_head < main || rot_ld < q4::kRot || rot_head < q4::kRot || main_ld % 4 != 0 ||
            main_head % 4 != 0 || rot_ld % 4 != 0 || rot_head % 4 != 0 || main_ld > most || main_head > most ||
            rot_ld > most || rot_head > most)
            return Q4_ESHAPE;
    }
    if (!(eps >= 0.0f)) return Q4_EINVAL;  // written so that NaN fails
    if (!aligned(kv, 16) || !aligned(seq, 4) || !aligned(positions, 4) || !aligned(slots, 4) || !aligned(inv_freq, 4) ||
        !aligned(norm, 2) || (heads > 0 && (!aligned(q_main, 16) || !aligned(q_rot, 16) || !aligned(q, 16))))
        return Q4_EALIGN;
    const size_t n = (size_t)tokens, h = (size_t)heads, rows = k_bytes(a.c);
    const size_t qbytes = n * h * (size_t)wide * 2;
    const void* in[] = {kv, seq, positions, slots, inv_freq, norm, heads ? q_main : nullptr, heads ? q_rot : nullptr};
    const size_t inbytes[] = {((n - 1) * (size_t)ld + (size_t)row) * 4, n * 4, n * 4, n * 4, (size_t)q4::kRot * 2,
                              (size_t)cache->latent * 2,
                              heads ? ((n - 1) * (size_t)main_ld + (h - 1) * (size_t)main_head + (size_t)main) * 4 : 0,
                              heads ? ((n - 1) * (size_t)rot_ld + (h - 1) * (size_t)rot_head + q4::kRot) * 4 : 0};
    if (overlaps(a.c.k, rows, a.c.table, table_bytes(a.c)) ||
        (heads > 0 && hits_cache(a.c, q, qbytes)))
        return Q4_EINVAL;
    for (int i = 0; i < 8; ++i)
        if (in[i] && (overlaps(a.c.k, rows, in[i], inbytes[i]) || (heads > 0 && overlaps(q, qbytes, in[i], inbytes[i]))))
            return Q4_EINVAL;
    a.kv = kv;
    a.ld = ld;
    a.tokens = (int)tokens;
    a.seq = seq;
    a.positions = positions;
    a.slots = slots;
    a.inv_freq = inv_freq;
    a.interleaved = interleaved != 0;
    a.mscale = mscale;
    a.norm = norm;
    a.eps = eps;
    a.q_main = q_main;
    a.main_ld = main_ld;
    a.main_head = main_head;
    a.main = heads > 0 ? main : 0;
    a.q_rot = q_rot;
    a.rot_ld = rot_ld;
    a.rot_head = rot_head;
    a.heads = heads;
    a.q = q;
    hipError_t e = q4::launch_latent_append(a, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_latent_keep(const q4g128_latent_cache* cache, const int32_t* starts, const int32_t* keep_starts,
                             const int32_t* keep, int64_t total, int64_t count, void* stream) {
    q4::KeepArgs a;
    q4_status s = check_latent(cache, &a.c);
    if (s != Q4_OK) return s;
    return keep_tokens(&a, starts, keep_starts, keep, total, count, stream);
}

int64_t q4g128_latent_attn_workspace(int32_t heads, int32_t latent, int64_t max_new) {
    if (heads < 1 || max_new < 1) return Q4_EINVAL;
    if (heads > Q4G128_MAX_HEADS || !q4::latent_supported(latent) || max_new > Q4G128_MAX_TOKENS) return Q4_ESHAPE;
    return q4::latent_attn_workspace(heads, latent, max_new);
}

q4_status q4g128_latent_attn(const uint16_t* q, const q4g128_latent_cache* cache, const int32_t* q_starts,
                             const int32_t* lengths, const uint64_t* masks, int64_t max_new, int64_t max_length,
                             int64_t tokens, int64_t count, int32_t heads, float scale, uint16_t* out, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    if (!q || !q_starts || !lengths || !out || tokens < 1 || count < 1 || max_length < 1) return Q4_EINVAL;
    q4::NewArgs x;
    q4_status s = check_latent(cache, &x.a.c);
    if (s != Q4_OK) return s;
    const int64_t need = q4g128_latent_attn_workspace(heads, cache->latent, max_new);
    if (need < 0) return (q4_status)need;
    if (tokens > Q4G128_MAX_TOKENS || count > Q4G128_MAX_SEQUENCES || count > cache->sequences ||
        max_length > cache->table_cols * cache->page || (masks && max_new > Q4G128_MAX_DRAFT))
        return Q4_ESHAPE;
    if (!(scale > 0.0f && scale <= FLT_MAX)) return Q4_EINVAL;  // written so that NaN fails
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(workspace, 16)) return Q4_EALIGN;
    if (!workspace || workspace_bytes < need) return Q4_EINVAL;
    const size_t rows = (size_t)tokens * (size_t)heads;
    const size_t qbytes = rows * (size_t)x.a.c.dim * 2, obytes = rows * (size_t)cache->latent * 2;
    const size_t lbytes = (size_t)count * 4, wsbytes = (size_t)need;
    if (hits_cache(x.a.c, out, obytes) || overlaps(out, obytes, q, qbytes) || overlaps(out, obytes, lengths, lbytes) ||
        hits_cache(x.a.c, workspace, wsbytes) || overlaps(workspace, wsbytes, q, qbytes) ||
        overlaps(workspace, wsbytes, out, obytes) || overlaps(workspace, wsbytes, lengths, lbytes))
        return Q4_EINVAL;
    s = check_new(q_starts, masks, tokens, count, out, obytes, workspace, wsbytes);
    if (s != Q4_OK) return s;
    x.a.q = q;
    x.a.lengths = lengths;
    x.a.max_length = (int)max_length;
    x.a.rows = (int)tokens;
    x.a.heads = heads;
    x.a.group = heads;
    x.a.scale = scale;
    x.a.softcap = 0.0f;
    x.a.window = 0;
    x.a.slopes = nullptr;
    x.a.prefix = nullptr;
    x.a.out = out;
    x.a.workspace = (float*)workspace;
    x.a.q_starts = q_starts;
    x.a.count = (int)count;
    x.masks = masks;
    x.max_new = (int)max_new;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_latent_attn(x, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

q4_status q4g128_latent_expand(const q4g128_latent_cache* cache, const int32_t* lengths, const int32_t* firsts,
                               int64_t max_length, int64_t count, const uint8_t* packed, const uint16_t* scales,
                               const uint16_t* mins, const q4g128_kv_cache* expanded, void* stream) {
    if (!lengths || !packed || !scales || !mins || count < 1 || max_length < 1) return Q4_EINVAL;
    q4::ExpandArgs a;
    q4_status s = check_latent(cache, &a.c);
    if (s != Q4_OK) return s;
    s = check_expanded(expanded, &a.to);
    if (s != Q4_OK) return s;
    if (count > Q4G128_MAX_SEQUENCES || count > cache->sequences || count > expanded->sequences ||
        max_length > cache->table_cols * cache->page || max_length > expanded->table_cols * expanded->page)
        return Q4_ESHAPE;
    if (!aligned(lengths, 4) || !aligned(firsts, 4) || !aligned(packed, 16) || !aligned(scales, 2) || !aligned(mins, 2))
        return Q4_EALIGN;
    const size_t n = (size_t)expanded->kv_heads * 2 * (size_t)expanded->dim, l = (size_t)cache->latent;
    const size_t kbytes = k_bytes(a.to), vbytes = v_bytes(a.to);
    const void* in[] = {lengths, firsts, packed, scales, mins, a.c.table, a.to.table};
    const size_t inbytes[] = {(size_t)count * 4, (size_t)count * 4, n * l / 2, n * (l / 128) * 2, n * (l / 128) * 2,
                              table_bytes(a.c), table_bytes(a.to)};
    for (int i = 0; i < 7; ++i)
        if (in[i] && (overlaps(a.to.k, kbytes, in[i], inbytes[i]) || overlaps(a.to.v, vbytes, in[i], inbytes[i])))
            return Q4_EINVAL;
    const Pool rows = k_pool(a.c);
    if (pools_meet(a.to) || pools_meet(rows, k_pool(a.to)) || pools_meet(rows, v_pool(a.to))) return Q4_EINVAL;
    a.lengths = lengths;
    a.firsts = firsts;
    a.max_length = (int)max_length;
    a.count = (int)count;
    a.packed = packed;
    a.scales = scales;
    a.mins = mins;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_latent_expand(a, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

int64_t q4g128_latent_prefill_workspace(int64_t tokens, int64_t count, int32_t heads, int32_t value, int64_t max_length) {
    if (tokens < 1 || count < 1 || heads < 1 || max_length < 1) return Q4_EINVAL;
    if (tokens > Q4G128_MAX_TOKENS || count > Q4G128_MAX_SEQUENCES || heads > Q4G128_MAX_HEADS ||
        !q4::value_supported(value) || max_length > Q4G128_MAX_N)
        return Q4_ESHAPE;
    return q4::attn_prefill_workspace(tokens, count, heads, heads, value + q4::kRot, value, max_length);
}

q4_status q4g128_latent_prefill(const uint16_t* q, const q4g128_kv_cache* expanded, const int32_t* q_starts,
                                const int32_t* lengths, int64_t max_length, int64_t tokens, int64_t count, float scale,
                                uint16_t* out, void* workspace, int64_t workspace_bytes, void* stream) {
    q4::AttnArgs a;
    if (!q_starts) return Q4_EINVAL;
    const int32_t heads = expanded ? expanded->kv_heads : 0;
    const int64_t need = expanded ? q4g128_latent_prefill_workspace(tokens, count, heads, expanded->dim, max_length)
                                  : Q4_EINVAL;
    if (need < 0) return (q4_status)need;
    const q4g128_attn_options options = {scale, 0.0f, 0, nullptr, nullptr};
    q4_status s = check_attention(q, expanded, lengths, max_length, tokens, count, heads, &options, out, workspace,
                                  workspace_bytes, need, &a, true);
    if (s != Q4_OK) return s;
    s = check_new(q_starts, nullptr, tokens, count, out, (size_t)tokens * (size_t)heads * (size_t)expanded->dim * 2,
                  workspace, (size_t)need);
    if (s != Q4_OK) return s;
    a.q_starts = q_starts;
    q4::DeviceInfo dev;
    s = current_device(&dev);
    if (s != Q4_OK) return s;
    hipError_t e = q4::launch_latent_prefill(a, dev, (hipStream_t)stream);
    return e == hipSuccess ? Q4_OK : device_error(e);
}

const char* q4g128_status_string(q4_status status) {
    switch (status) {
        case Q4_OK: return "Q4_OK: success";
        case Q4_EINVAL: return "Q4_EINVAL: null pointer, non-positive size, batch outside 1..16, invalid option, short workspace or overlapping output";
        case Q4_ESHAPE: return "Q4_ESHAPE: K must be a multiple of 128 in [128, 32768], a cache's dim, page and heads among the supported ones; sizes must fit the kernels' index range";
        case Q4_EALIGN: return "Q4_EALIGN: packed/codes/activations/float weights, caches, queries and workspaces need 16-byte, scales/mins/norms 2-byte, masks 8-byte, other arrays 4-byte alignment";
        case Q4_EDEVICE: return "Q4_EDEVICE: the HIP runtime reported an error (see q4g128_last_hip_error)";
    }
    return "unknown q4g128 status";
}

int32_t q4g128_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
