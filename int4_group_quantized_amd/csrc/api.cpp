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

#include "attn.hpp"
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
    out->dim = c->dim;
    out->shift = __builtin_ctz((unsigned)c->page);
    return Q4_OK;
}

// Bytes from the first to past the last element of a pool.
size_t pool_bytes(const q4::KvCache& c, long stride) {
    return ((size_t)(c.pages - 1) * (size_t)stride + ((size_t)c.kv_heads * (size_t)c.dim << c.shift)) * 2;
}

// Whether the two pools share an element.  Pools whose pages interleave (parts
// of one larger pool) overlap as ranges without sharing any.
bool pools_meet(const q4::KvCache& c) {
    if (!overlaps(c.k, pool_bytes(c, c.k_stride), c.v, pool_bytes(c, c.v_stride))) return false;
    if (c.k_stride != c.v_stride) return true;
    const uintptr_t k = (uintptr_t)c.k, v = (uintptr_t)c.v;
    const uintptr_t stride = (uintptr_t)c.k_stride * 2, page = ((uintptr_t)c.kv_heads * c.dim << c.shift) * 2;
    const uintptr_t apart = (k > v ? k - v : v - k) % stride;
    return apart < page || apart > stride - page;
}

// Whether [p, p + bytes) meets one of the cache's pools or its table.
bool hits_cache(const q4::KvCache& c, const void* p, size_t bytes) {
    return overlaps(p, bytes, c.k, pool_bytes(c, c.k_stride)) || overlaps(p, bytes, c.v, pool_bytes(c, c.v_stride)) ||
           overlaps(p, bytes, c.table, (size_t)c.sequences * (size_t)c.cols * 4);
}

// Shared checks of the two attention calls; `rows` = batch or tokens.
q4_status check_attention(const uint16_t* q, const q4g128_kv_cache* cache, const int32_t* lengths, int64_t max_length,
                          int64_t rows, int64_t sequences, int64_t heads, const q4g128_attn_options* o, uint16_t* out,
                          void* workspace, int64_t workspace_bytes, int64_t workspace_needed, q4::AttnArgs* a) {
    if (!q || !lengths || !o || !out || rows < 1 || sequences < 1 || max_length < 1) return Q4_EINVAL;
    q4_status s = check_cache(cache, heads, &a->c);
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
    const size_t qbytes = (size_t)rows * (size_t)heads * (size_t)cache->dim * 2;
    const size_t seqbytes = (size_t)sequences * 4, wsbytes = (size_t)workspace_needed;
    if (hits_cache(a->c, out, qbytes) || overlaps(out, qbytes, q, qbytes) || overlaps(out, qbytes, lengths, seqbytes) ||
        (o->slopes && overlaps(out, qbytes, o->slopes, (size_t)heads * 4)) ||
        (o->prefix && overlaps(out, qbytes, o->prefix, seqbytes)))
        return Q4_EINVAL;
    if (wsbytes > 0 &&
        (hits_cache(a->c, workspace, wsbytes) || overlaps(workspace, wsbytes, q, qbytes) ||
         overlaps(workspace, wsbytes, out, qbytes) || overlaps(workspace, wsbytes, lengths, seqbytes) ||
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
    a->count = (int)sequences;
    return Q4_OK;
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
    if (!qkv || !positions || !q || tokens < 1) return Q4_EINVAL;
    q4::AppendArgs a;
    q4_status s = check_cache(cache, heads, &a.c);
    if (s != Q4_OK) return s;
    const int64_t dim = cache->dim, columns = ((int64_t)heads + 2 * (int64_t)cache->kv_heads) * dim;
    if (rot < 0 || rot > dim || rot % 4 != 0 || tokens > Q4G128_MAX_TOKENS || ld < columns || ld % 4 != 0 ||
        ld > INT64_MAX / 8 / tokens)
        return Q4_ESHAPE;
    if ((rot > 0 && !inv_freq) || !(eps >= 0.0f)) return Q4_EINVAL;  // written so that NaN fails
    if (!aligned(qkv, 16) || !aligned(q, 16) || !aligned(seq, 4) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
        !aligned(q_norm, 2) || !aligned(k_norm, 2))
        return Q4_EALIGN;
    const size_t qbytes = (size_t)tokens * (size_t)heads * (size_t)dim * 2, nbytes = (size_t)dim * 2;
    const void* in[] = {qkv, seq, positions, inv_freq, q_norm, k_norm};
    const size_t inbytes[] = {((size_t)(tokens - 1) * (size_t)ld + (size_t)columns) * 4, (size_t)tokens * 4,
                              (size_t)tokens * 4, (size_t)rot * 2, nbytes, nbytes};
    if (pools_meet(a.c)) return Q4_EINVAL;
    const size_t kbytes = pool_bytes(a.c, a.c.k_stride), vbytes = pool_bytes(a.c, a.c.v_stride);
    const size_t tbytes = (size_t)a.c.sequences * (size_t)a.c.cols * 4;
    if (hits_cache(a.c, q, qbytes) || overlaps(a.c.k, kbytes, a.c.table, tbytes) ||
        overlaps(a.c.v, vbytes, a.c.table, tbytes))
        return Q4_EINVAL;
    for (int i = 0; i < 6; ++i)
        if (in[i] && (overlaps(q, qbytes, in[i], inbytes[i]) || overlaps(a.c.k, kbytes, in[i], inbytes[i]) ||
                      overlaps(a.c.v, vbytes, in[i], inbytes[i])))
            return Q4_EINVAL;
    a.qkv = qkv;
    a.ld = ld;
    a.tokens = (int)tokens;
    a.heads = heads;
    a.seq = seq;
    a.positions = positions;
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
    return q4::attn_prefill_workspace(tokens, count, heads, kv_heads, dim, max_length);
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

const char* q4g128_status_string(q4_status status) {
    switch (status) {
        case Q4_OK: return "Q4_OK: success";
        case Q4_EINVAL: return "Q4_EINVAL: null pointer, non-positive size, batch outside 1..16, invalid option, short workspace or overlapping output";
        case Q4_ESHAPE: return "Q4_ESHAPE: K must be a multiple of 128 in [128, 32768], a cache's dim, page and heads among the supported ones; sizes must fit the kernels' index range";
        case Q4_EALIGN: return "Q4_EALIGN: packed/codes/activations/float weights, caches, queries and workspaces need 16-byte, scales/mins/norms 2-byte, other arrays 4-byte alignment";
        case Q4_EDEVICE: return "Q4_EDEVICE: the HIP runtime reported an error (see q4g128_last_hip_error)";
    }
    return "unknown q4g128 status";
}

int32_t q4g128_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
