// Python binding of the cache and attention calls (module _binding): checks
// tensor devices, types, shapes and contiguity, and passes pointers, sizes and
// the current stream to the C ABI of include/q4g128.h.
//
// Compiled, unlike the ctypes binding of the products, because these calls take
// up to a dozen tensors and the kernels of a small step run for 3 to 9 us: the
// same checks in Python and ctypes took 13 us more per call (one token appended:
// 18.3 us a call with them, 5.2 us here).
//
// Every function takes its arguments by position (the Python wrappers give the
// defaults) and returns the output tensor, or the library's status as an int
// when that is not Q4_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <map>
#include <string>
#include <utility>

#include "q4g128.h"

namespace {

template <class... A>
[[noreturn]] void type_error(const char* format, A... a) {
    PyErr_Format(PyExc_TypeError, format, a...);
    throw python_error();
}

template <class... A>
[[noreturn]] void value_error(const char* format, A... a) {
    PyErr_Format(PyExc_ValueError, format, a...);
    throw python_error();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error("%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

void on_gpu(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) value_error("%s must live on a GPU (got %s)", name, t.device().str().c_str());
}

void of_type(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type)
        type_error("%s must be %s (got %s)", name, c10::toString(type), c10::toString(t.scalar_type()));
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    on_gpu(t, name);
    of_type(t, name, type);
    if (t.sizes() != shape)
        value_error("%s must have shape %s (got %s)", name, shape_text(shape).c_str(),
                                shape_text(t.sizes()).c_str());
    if (!t.is_contiguous()) value_error("%s must be contiguous", name);
}

// One call's tensors have to share a device.
struct SameDevice {
    at::Device device;
    explicit SameDevice(const at::Tensor& t) : device(t.device()) {}
    void add(const at::Tensor& t) const {
        if (t.device() != device) value_error("all tensors must be on the same GPU");
    }
};

// The pointer of an optional tensor argument (None: NULL).
template <class T>
const T* optional(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const SameDevice& dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    check(t, name, type, shape);
    dev.add(t);
    return static_cast<const T*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

// An int32 argument; values outside its range become -1, which every call refuses.
int32_t small_integer(PyObject* o) {
    const int64_t v = integer(o);
    return v < 0 || v > INT32_MAX ? -1 : (int32_t)v;
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

hipStream_t current_stream(const at::Device& d) {
    return at::hip::getCurrentHIPStreamMasqueradingAsCUDA(d.index()).stream();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& d) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(d));
}

// An output given by the caller, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, const SameDevice& dev) {
    if (o == Py_None) return empty(shape, at::kHalf, dev.device);
    const at::Tensor& t = tensor(o, name);
    check(t, name, at::kHalf, shape);
    dev.add(t);
    return t;
}

// Whether the elements of a page follow each other.  The stride of a size of one
// means nothing.
bool page_contiguous(const at::Tensor& t) {
    int64_t next = 1;
    for (int i = 3; i >= 1; --i) {
        if (t.size(i) != 1 && t.stride(i) != next) return false;
        next *= t.size(i);
    }
    return true;
}

// The cache descriptor.  Pages may be strided (a slice of a larger pool); each
// page itself is contiguous.
q4g128_kv_cache cache_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table) {
    for (const auto& p : {std::make_pair(&k, "k_cache"), std::make_pair(&v, "v_cache")}) {
        on_gpu(*p.first, p.second);
        of_type(*p.first, p.second, at::kHalf);
        if (p.first->dim() != 4)
            value_error(
                "k_cache must be [pages][kv_heads][page][dim], v_cache [pages][kv_heads][dim][page]");
    }
    const int64_t pages = k.size(0), heads = k.size(1), page = k.size(2), dim = k.size(3);
    if (v.size(0) != pages || v.size(1) != heads || v.size(2) != dim || v.size(3) != page)
        value_error("v_cache must have shape %s (got %s)", shape_text({pages, heads, dim, page}).c_str(),
                                shape_text(v.sizes()).c_str());
    if (!page_contiguous(k) || !page_contiguous(v))
        value_error("each page of k_cache and v_cache must be contiguous");
    if (table.dim() != 2) value_error("table must be [sequences][table_cols]");
    check(table, "table", at::kInt, table.sizes());
    if (heads > INT32_MAX || dim > INT32_MAX || page > INT32_MAX) value_error("cache too large");
    q4g128_kv_cache c;
    c.k = static_cast<uint16_t*>(k.data_ptr());
    c.v = static_cast<uint16_t*>(v.data_ptr());
    c.table = static_cast<const int32_t*>(table.data_ptr());
    c.pages = pages;
    // One page has no next page: any stride will do.
    c.k_stride = pages > 1 ? k.stride(0) : heads * page * dim;
    c.v_stride = pages > 1 ? v.stride(0) : heads * page * dim;
    c.sequences = table.size(0);
    c.table_cols = table.size(1);
    c.kv_heads = (int32_t)heads;
    c.dim = (int32_t)dim;
    c.page = (int32_t)page;
    return c;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) type_error("expected %d arguments (got %d)", (int)want, (int)got);
}

PyObject* answer(q4_status status, const at::Tensor& out) {
    return status == Q4_OK ? THPVariable_Wrap(out) : PyLong_FromLong(status);
}

// rope_append(qkv, k_cache, v_cache, table, positions, inv_freq, heads, seq,
//             q_norm, k_norm, eps, interleaved, mscale, q, slots)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 15);
    const at::Tensor &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache"), &table = tensor(a[3], "table");
    const at::Tensor& qkv = tensor(a[0], "qkv");
    const q4g128_kv_cache c = cache_of(k, v, table);
    if (qkv.dim() != 2) value_error("qkv must be [T][columns]");
    on_gpu(qkv, "qkv");
    of_type(qkv, "qkv", at::kFloat);
    const SameDevice dev(qkv);
    dev.add(k), dev.add(v), dev.add(table);
    const int32_t heads = small_integer(a[6]);
    const int64_t tokens = qkv.size(0), columns = qkv.size(1), need = (heads + 2 * (int64_t)c.kv_heads) * c.dim;
    if (heads < 1) value_error("heads must be positive");
    if (columns < need)
        value_error("qkv has %lld columns, fewer than (heads + 2 kv_heads) dim", (long long)columns);
    if (qkv.stride(1) != 1) value_error("rows of qkv must be contiguous");
    const at::Tensor& positions = tensor(a[4], "positions");
    check(positions, "positions", at::kInt, {tokens});
    dev.add(positions);
    int64_t pairs = 0;
    if (a[5] != Py_None) {
        const at::Tensor& f = tensor(a[5], "inv_freq");
        if (f.dim() != 1) value_error("inv_freq must be [rot / 2]");
        pairs = f.size(0);
    }
    const float* freq = optional<float>(a[5], "inv_freq", at::kFloat, {pairs}, dev);
    const int32_t* seq = optional<int32_t>(a[7], "seq", at::kInt, {tokens}, dev);
    const uint16_t* q_norm = optional<uint16_t>(a[8], "q_norm", at::kHalf, {c.dim}, dev);
    const uint16_t* k_norm = optional<uint16_t>(a[9], "k_norm", at::kHalf, {c.dim}, dev);
    const int32_t* pos = static_cast<const int32_t*>(positions.data_ptr());
    const int32_t* slots = optional<int32_t>(a[14], "slots", at::kInt, {tokens}, dev);
    const float eps = real(a[10]), mscale = real(a[12]);
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw python_error();
    const c10::DeviceGuard guard(dev.device);
    const at::Tensor q = output(a[13], "q", {tokens, heads, c.dim}, dev);
    // One row has no next row: any stride will do.
    const int64_t ld = tokens > 1 ? qkv.stride(0) : (columns + 3) / 4 * 4;
    const int32_t rot = pairs > INT32_MAX / 2 ? -1 : (int32_t)(2 * pairs);
    return answer(q4g128_rope_append_slots(static_cast<const float*>(qkv.data_ptr()), ld, tokens, heads, &c, seq, pos,
                                           slots ? slots : pos, freq, rot, interleaved, mscale, q_norm, k_norm, eps,
                                           static_cast<uint16_t*>(q.data_ptr()), current_stream(dev.device)),
                  q);
    END_HANDLE_TH_ERRORS
}

// Workspaces of calls that are given none: one per device and stream (calls on
// one stream run one after the other), grown as needed, counters zeroed once.
// A call in a graph capture gets memory of its own, since a graph may be
// replayed on any stream.  Never destroyed: at exit the device may be gone.
// counted: whether the call uses the counters.
at::Tensor kept_workspace(int64_t need, const at::Device& d, hipStream_t stream, bool counted) {
    static auto* kept = new std::map<std::pair<int, hipStream_t>, at::Tensor>;
    hipStreamCaptureStatus status = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(stream, &status) != hipSuccess) {
        (void)hipGetLastError();  // the null stream while another one is captured: not a capture itself
        status = hipStreamCaptureStatusNone;
    }
    const bool capturing = status != hipStreamCaptureStatusNone;
    at::Tensor fresh;
    at::Tensor& t = capturing ? fresh : (*kept)[{d.index(), stream}];
    if (!t.defined() || t.numel() < need) {
        t = empty({need}, at::kByte, d);
        if (capturing && !counted) return t;
        t.narrow(0, 0, Q4G128_ATTN_COUNTER_BYTES).zero_();
    }
    return t;
}

at::Tensor workspace_of(PyObject* o, int64_t need, const SameDevice& dev, hipStream_t stream, bool counted = false) {
    if (o == Py_None) return need > 0 ? kept_workspace(need, dev.device, stream, counted) : at::Tensor();
    const at::Tensor& t = tensor(o, "workspace");
    on_gpu(t, "workspace");
    dev.add(t);
    if (t.scalar_type() != at::kByte || t.dim() != 1 || !t.is_contiguous())
        value_error("workspace must be a contiguous uint8 vector");
    return t;
}

struct Attention {
    const at::Tensor &q, &k, &v, &table, &lengths;
    q4g128_kv_cache c;
    SameDevice dev;
    int64_t rows, count, max_length;
    int32_t heads;
    q4g128_attn_options o;

    // count < 0: one sequence per row
    Attention(PyObject* q_, PyObject* k_, PyObject* v_, PyObject* table_, PyObject* lengths_, int64_t count_,
              PyObject* scale, PyObject* softcap, PyObject* window, PyObject* slopes, PyObject* prefix,
              PyObject* max_length_)
        : q(tensor(q_, "q")), k(tensor(k_, "k_cache")), v(tensor(v_, "v_cache")), table(tensor(table_, "table")),
          lengths(tensor(lengths_, "lengths")), c(cache_of(k, v, table)), dev(k) {
        if (q.dim() != 3) value_error("q must be [rows][heads][dim]");
        rows = q.size(0);
        if (q.size(1) > INT32_MAX) value_error("q has too many heads");
        heads = (int32_t)q.size(1);
        check(q, "q", at::kHalf, {rows, heads, c.dim});
        count = count_ < 0 ? rows : count_;
        check(lengths, "lengths", at::kInt, {count});
        dev.add(q), dev.add(v), dev.add(table), dev.add(lengths);
        if (count > c.sequences)
            value_error("table has %lld sequences, fewer than %lld", (long long)c.sequences,
                                    (long long)count);
        o.scale = scale == Py_None ? 1.0f / std::sqrt((float)c.dim) : real(scale);
        o.softcap = real(softcap);
        o.window = integer(window);
        o.slopes = optional<float>(slopes, "slopes", at::kFloat, {heads}, dev);
        o.prefix = optional<int32_t>(prefix, "prefix", at::kInt, {count}, dev);
        max_length = max_length_ == Py_None ? c.table_cols * c.page : integer(max_length_);
    }
    const uint16_t* qp() const { return static_cast<const uint16_t*>(q.data_ptr()); }
    const int32_t* lp() const { return static_cast<const int32_t*>(lengths.data_ptr()); }
};

// attn_decode(q, k_cache, v_cache, table, lengths, scale, softcap, window,
//             slopes, max_length, out, workspace)
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 12);
    const Attention t(a[0], a[1], a[2], a[3], a[4], -1, a[5], a[6], a[7], a[8], Py_None, a[9]);
    const int64_t need = q4g128_attn_decode_workspace(t.rows, t.heads, t.c.dim);
    if (need < 0) return PyLong_FromLongLong(need);
    const c10::DeviceGuard guard(t.dev.device);
    const hipStream_t stream = current_stream(t.dev.device);
    const at::Tensor out = output(a[10], "out", t.q.sizes(), t.dev);
    const at::Tensor ws = workspace_of(a[11], need, t.dev, stream, true);
    return answer(q4g128_attn_decode(t.qp(), &t.c, t.lp(), t.max_length, t.rows, t.heads, &t.o,
                                     static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(), ws.numel(), stream),
                  out);
    END_HANDLE_TH_ERRORS
}

// attn_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale, softcap,
//              window, slopes, prefix, max_length, out, workspace)
PyObject* attn_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);
    const at::Tensor& lengths = tensor(a[5], "lengths");
    if (lengths.dim() != 1) value_error("lengths must be [sequences]");
    const Attention t(a[0], a[1], a[2], a[3], a[5], lengths.size(0), a[6], a[7], a[8], a[9], a[10], a[11]);
    const at::Tensor& starts = tensor(a[4], "q_starts");
    check(starts, "q_starts", at::kInt, {t.count + 1});
    t.dev.add(starts);
    const int64_t need =
        q4g128_attn_prefill_workspace(t.rows, t.count, t.heads, t.c.kv_heads, t.c.dim, t.max_length);
    if (need < 0) return PyLong_FromLongLong(need);
    const c10::DeviceGuard guard(t.dev.device);
    const hipStream_t stream = current_stream(t.dev.device);
    const at::Tensor out = output(a[12], "out", t.q.sizes(), t.dev);
    const at::Tensor ws = workspace_of(a[13], need, t.dev, stream);
    return answer(q4g128_attn_prefill(t.qp(), &t.c, static_cast<const int32_t*>(starts.data_ptr()), t.lp(),
                                      t.max_length, t.rows, t.count, t.heads, &t.o,
                                      static_cast<uint16_t*>(out.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                                      ws.defined() ? ws.numel() : 0, stream),
                  out);
    END_HANDLE_TH_ERRORS
}

// attn_tree(q, k_cache, v_cache, table, q_starts, lengths, masks, scale, softcap,
//           window, slopes, max_new, max_length, out, workspace)
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 15);
    const at::Tensor& lengths = tensor(a[5], "lengths");
    if (lengths.dim() != 1) value_error("lengths must be [sequences]");
    const Attention t(a[0], a[1], a[2], a[3], a[5], lengths.size(0), a[7], a[8], a[9], a[10], Py_None, a[12]);
    const at::Tensor& starts = tensor(a[4], "q_starts");
    check(starts, "q_starts", at::kInt, {t.count + 1});
    t.dev.add(starts);
    const uint64_t* masks = optional<uint64_t>(a[6], "masks", at::kLong, {t.rows}, t.dev);
    const int64_t max_new = a[11] == Py_None ? std::min<int64_t>(t.rows, Q4G128_MAX_DRAFT) : integer(a[11]);
    const int64_t need = q4g128_attn_tree_workspace(t.rows, t.count, t.heads, t.c.kv_heads, t.c.dim, max_new, t.max_length);
    if (need < 0) return PyLong_FromLongLong(need);
    const c10::DeviceGuard guard(t.dev.device);
    const hipStream_t stream = current_stream(t.dev.device);
    const at::Tensor out = output(a[13], "out", t.q.sizes(), t.dev);
    const at::Tensor ws = workspace_of(a[14], need, t.dev, stream);
    return answer(q4g128_attn_tree(t.qp(), &t.c, static_cast<const int32_t*>(starts.data_ptr()), t.lp(), masks, max_new,
                                   t.max_length, t.rows, t.count, t.heads, &t.o,
                                   static_cast<uint16_t*>(out.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                                   ws.defined() ? ws.numel() : 0, stream),
                  out);
    END_HANDLE_TH_ERRORS
}

// Numbers of accepted tokens: (starts, keep_starts, keep).
struct Keep {
    const at::Tensor &starts, &keep_starts, &keep;
    int64_t count, total;
    Keep(PyObject* s, PyObject* ks, PyObject* k, const SameDevice& dev)
        : starts(tensor(s, "starts")), keep_starts(tensor(ks, "keep_starts")), keep(tensor(k, "keep")) {
        if (starts.dim() != 1) value_error("starts must be [sequences]");
        if (keep.dim() != 1) value_error("keep must be a vector");
        count = starts.size(0);
        total = keep.size(0);
        check(starts, "starts", at::kInt, {count});
        check(keep_starts, "keep_starts", at::kInt, {count + 1});
        check(keep, "keep", at::kInt, {total});
        dev.add(starts), dev.add(keep_starts), dev.add(keep);
    }
    static const int32_t* p(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
};

// cache_keep(k_cache, v_cache, table, starts, keep_starts, keep)
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 6);
    const at::Tensor &k = tensor(a[0], "k_cache"), &v = tensor(a[1], "v_cache"), &table = tensor(a[2], "table");
    const q4g128_kv_cache c = cache_of(k, v, table);
    const SameDevice dev(k);
    dev.add(v), dev.add(table);
    const Keep t(a[3], a[4], a[5], dev);
    const c10::DeviceGuard guard(dev.device);
    return PyLong_FromLong(q4g128_cache_keep(&c, t.p(t.starts), t.p(t.keep_starts), t.p(t.keep), t.total, t.count,
                                             current_stream(dev.device)));
    END_HANDLE_TH_ERRORS
}

// The descriptor of a latent cache.  Pages may be strided.
q4g128_latent_cache latent_of(const at::Tensor& rows, const at::Tensor& table) {
    on_gpu(rows, "cache");
    of_type(rows, "cache", at::kHalf);
    if (rows.dim() != 3) value_error("cache must be [pages][page][latent + 64]");
    const int64_t pages = rows.size(0), page = rows.size(1), dim = rows.size(2);
    if ((dim != 1 && rows.stride(2) != 1) || (page != 1 && rows.stride(1) != dim))
        value_error("each page of cache must be contiguous");
    if (table.dim() != 2) value_error("table must be [sequences][table_cols]");
    check(table, "table", at::kInt, table.sizes());
    if (dim > INT32_MAX || page > INT32_MAX || dim < Q4G128_LATENT_ROT) value_error("cache must be [pages][page][latent + 64]");
    q4g128_latent_cache c;
    c.rows = static_cast<uint16_t*>(rows.data_ptr());
    c.table = static_cast<const int32_t*>(table.data_ptr());
    c.pages = pages;
    c.stride = pages > 1 ? rows.stride(0) : page * dim;
    c.sequences = table.size(0);
    c.table_cols = table.size(1);
    c.latent = (int32_t)(dim - Q4G128_LATENT_ROT);
    c.page = (int32_t)page;
    return c;
}

// One part of the queries, fp32 [tokens][heads][columns] with strides of its own.
struct Part {
    const float* p;
    int64_t ld, head, columns;
    Part(PyObject* o, const char* name, int64_t tokens, int64_t heads, const SameDevice& dev) {
        const at::Tensor& t = tensor(o, name);
        on_gpu(t, name);
        of_type(t, name, at::kFloat);
        dev.add(t);
        if (t.dim() != 3 || t.size(0) != tokens || (heads >= 0 && t.size(1) != heads))
            value_error("%s must be [T][heads][columns] (got %s)", name, shape_text(t.sizes()).c_str());
        if (t.size(2) != 1 && t.stride(2) != 1) value_error("rows of %s must be contiguous", name);
        p = static_cast<const float*>(t.data_ptr());
        columns = t.size(2);
        // A size of one has no next: any stride will do.
        const int64_t any = (columns + 3) / 4 * 4;
        ld = t.size(0) > 1 ? t.stride(0) : any;
        head = t.size(1) > 1 ? t.stride(1) : any;
    }
};

// latent_append(kv, cache, table, positions, inv_freq, seq, slots, norm, eps,
//               interleaved, mscale, q_main, q_rot, q)
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);
    const at::Tensor &kv = tensor(a[0], "kv"), &rows = tensor(a[1], "cache"), &table = tensor(a[2], "table");
    const q4g128_latent_cache c = latent_of(rows, table);
    on_gpu(kv, "kv");
    of_type(kv, "kv", at::kFloat);
    if (kv.dim() != 2) value_error("kv must be [T][columns]");
    const int64_t tokens = kv.size(0), columns = kv.size(1);
    if (columns < c.latent + Q4G128_LATENT_ROT) value_error("kv has %lld columns, fewer than latent + 64", (long long)columns);
    if (kv.stride(1) != 1) value_error("rows of kv must be contiguous");
    const SameDevice dev(kv);
    dev.add(rows), dev.add(table);
    const at::Tensor& positions = tensor(a[3], "positions");
    check(positions, "positions", at::kInt, {tokens});
    dev.add(positions);
    const int32_t* pos = static_cast<const int32_t*>(positions.data_ptr());
    const float* freq = optional<float>(a[4], "inv_freq", at::kFloat, {Q4G128_LATENT_ROT / 2}, dev);
    const int32_t* seq = optional<int32_t>(a[5], "seq", at::kInt, {tokens}, dev);
    const int32_t* slots = optional<int32_t>(a[6], "slots", at::kInt, {tokens}, dev);
    const uint16_t* norm = optional<uint16_t>(a[7], "norm", at::kHalf, {c.latent}, dev);
    const float eps = real(a[8]), mscale = real(a[10]);
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) throw python_error();
    const int64_t ld = tokens > 1 ? kv.stride(0) : (columns + 3) / 4 * 4;
    const c10::DeviceGuard guard(dev.device);
    if ((a[11] == Py_None) != (a[12] == Py_None)) value_error("q_main and q_rot go together");
    if (a[11] == Py_None) {
        const q4_status status = q4g128_latent_append(
            static_cast<const float*>(kv.data_ptr()), ld, tokens, &c, seq, pos, slots ? slots : pos, freq, interleaved, mscale,
            norm, eps, nullptr, 0, 0, 0, nullptr, 0, 0, 0, nullptr, current_stream(dev.device));
        if (status != Q4_OK) return PyLong_FromLong(status);
        Py_RETURN_NONE;
    }
    const Part main(a[11], "q_main", tokens, -1, dev);
    const int64_t heads = tensor(a[11], "q_main").size(1);
    const Part rot(a[12], "q_rot", tokens, heads, dev);
    if (rot.columns != Q4G128_LATENT_ROT) value_error("q_rot must have 64 columns");
    if (heads < 1 || heads > Q4G128_MAX_HEADS || main.columns > Q4G128_LATENT_MAX_MAIN) return PyLong_FromLong(Q4_ESHAPE);
    const at::Tensor q = output(a[13], "q", {tokens, heads, main.columns + Q4G128_LATENT_ROT}, dev);
    return answer(q4g128_latent_append(static_cast<const float*>(kv.data_ptr()), ld, tokens, &c, seq, pos,
                                       slots ? slots : pos, freq, interleaved, mscale, norm, eps, main.p, main.ld, main.head,
                                       (int32_t)main.columns, rot.p, rot.ld, rot.head, (int32_t)heads,
                                       static_cast<uint16_t*>(q.data_ptr()), current_stream(dev.device)),
                  q);
    END_HANDLE_TH_ERRORS
}

// latent_keep(cache, table, starts, keep_starts, keep)
PyObject* latent_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 5);
    const at::Tensor &rows = tensor(a[0], "cache"), &table = tensor(a[1], "table");
    const q4g128_latent_cache c = latent_of(rows, table);
    const SameDevice dev(rows);
    dev.add(table);
    const Keep t(a[2], a[3], a[4], dev);
    const c10::DeviceGuard guard(dev.device);
    return PyLong_FromLong(q4g128_latent_keep(&c, t.p(t.starts), t.p(t.keep_starts), t.p(t.keep), t.total, t.count,
                                              current_stream(dev.device)));
    END_HANDLE_TH_ERRORS
}

// latent_attn(q, cache, table, q_starts, lengths, scale, masks, max_new,
//             max_length, out, workspace)
PyObject* latent_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    const at::Tensor &q = tensor(a[0], "q"), &rows = tensor(a[1], "cache"), &table = tensor(a[2], "table");
    const q4g128_latent_cache c = latent_of(rows, table);
    if (q.dim() != 3) value_error("q must be [T][heads][latent + 64]");
    const int64_t tokens = q.size(0), heads = q.size(1);
    check(q, "q", at::kHalf, {tokens, heads, c.latent + Q4G128_LATENT_ROT});
    const SameDevice dev(rows);
    const at::Tensor &starts = tensor(a[3], "q_starts"), &lengths = tensor(a[4], "lengths");
    if (lengths.dim() != 1) value_error("lengths must be [sequences]");
    const int64_t count = lengths.size(0);
    check(lengths, "lengths", at::kInt, {count});
    check(starts, "q_starts", at::kInt, {count + 1});
    dev.add(q), dev.add(table), dev.add(starts), dev.add(lengths);
    if (count > c.sequences)
        value_error("table has %lld sequences, fewer than %lld", (long long)c.sequences, (long long)count);
    const uint64_t* masks = optional<uint64_t>(a[6], "masks", at::kLong, {tokens}, dev);
    const int64_t most = masks ? Q4G128_MAX_DRAFT : Q4G128_MAX_TOKENS;
    const int64_t max_new = a[7] == Py_None ? std::min(tokens, most) : integer(a[7]);
    const int64_t max_length = a[8] == Py_None ? c.table_cols * c.page : integer(a[8]);
    const int32_t h = heads > INT32_MAX ? -1 : (int32_t)heads;
    const int64_t need = q4g128_latent_attn_workspace(h, c.latent, max_new);
    if (need < 0) return PyLong_FromLongLong(need);
    const float scale = real(a[5]);
    const c10::DeviceGuard guard(dev.device);
    const hipStream_t stream = current_stream(dev.device);
    const at::Tensor out = output(a[9], "out", {tokens, heads, c.latent}, dev);
    const at::Tensor ws = workspace_of(a[10], need, dev, stream);
    return answer(q4g128_latent_attn(static_cast<const uint16_t*>(q.data_ptr()), &c,
                                     static_cast<const int32_t*>(starts.data_ptr()),
                                     static_cast<const int32_t*>(lengths.data_ptr()), masks, max_new, max_length, tokens,
                                     count, h, scale, static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(), ws.numel(),
                                     stream),
                  out);
    END_HANDLE_TH_ERRORS
}

// The descriptor of a cache of expanded keys and values.
q4g128_kv_cache expanded_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table) {
    for (const auto& p : {std::make_pair(&k, "k_cache"), std::make_pair(&v, "v_cache")}) {
        on_gpu(*p.first, p.second);
        of_type(*p.first, p.second, at::kHalf);
        if (p.first->dim() != 4)
            value_error("k_cache must be [pages][heads][page][value + 64], v_cache [pages][heads][value][page]");
    }
    const int64_t pages = k.size(0), heads = k.size(1), page = k.size(2), dim = k.size(3) - Q4G128_LATENT_ROT;
    if (dim < 0 || v.size(0) != pages || v.size(1) != heads || v.size(2) != dim || v.size(3) != page)
        value_error("v_cache must have shape %s (got %s)", shape_text({pages, heads, dim, page}).c_str(),
                    shape_text(v.sizes()).c_str());
    if (!page_contiguous(k) || !page_contiguous(v))
        value_error("each page of k_cache and v_cache must be contiguous");
    if (table.dim() != 2) value_error("table must be [sequences][table_cols]");
    check(table, "table", at::kInt, table.sizes());
    if (heads > INT32_MAX || dim > INT32_MAX || page > INT32_MAX) value_error("cache too large");
    q4g128_kv_cache c;
    c.k = static_cast<uint16_t*>(k.data_ptr());
    c.v = static_cast<uint16_t*>(v.data_ptr());
    c.table = static_cast<const int32_t*>(table.data_ptr());
    c.pages = pages;
    c.k_stride = pages > 1 ? k.stride(0) : heads * page * (dim + Q4G128_LATENT_ROT);
    c.v_stride = pages > 1 ? v.stride(0) : heads * page * dim;
    c.sequences = table.size(0);
    c.table_cols = table.size(1);
    c.kv_heads = (int32_t)heads;
    c.dim = (int32_t)dim;
    c.page = (int32_t)page;
    return c;
}

// latent_expand(cache, table, lengths, packed, scales, mins, k_cache, v_cache,
//               expanded_table, firsts, max_length); no result
PyObject* latent_expand(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    const at::Tensor &rows = tensor(a[0], "cache"), &table = tensor(a[1], "table"), &lengths = tensor(a[2], "lengths");
    const q4g128_latent_cache c = latent_of(rows, table);
    const at::Tensor &k = tensor(a[6], "k_cache"), &v = tensor(a[7], "v_cache"), &to = tensor(a[8], "expanded_table");
    const q4g128_kv_cache e = expanded_of(k, v, to);
    const SameDevice dev(rows);
    if (lengths.dim() != 1) value_error("lengths must be [sequences]");
    const int64_t count = lengths.size(0), wide = (int64_t)e.kv_heads * 2 * e.dim;
    check(lengths, "lengths", at::kInt, {count});
    dev.add(table), dev.add(lengths), dev.add(k), dev.add(v), dev.add(to);
    if (count > c.sequences || count > e.sequences) value_error("a table has fewer than %lld sequences", (long long)count);
    const uint8_t* packed = optional<uint8_t>(a[3], "packed", at::kByte, {wide, c.latent / 2}, dev);
    const uint16_t* scales = optional<uint16_t>(a[4], "scales", at::kHalf, {wide, c.latent / Q4G128_GROUP}, dev);
    const uint16_t* mins = optional<uint16_t>(a[5], "mins", at::kHalf, {wide, c.latent / Q4G128_GROUP}, dev);
    const int32_t* firsts = optional<int32_t>(a[9], "firsts", at::kInt, {count}, dev);
    const int64_t held = std::min((int64_t)c.table_cols * c.page, (int64_t)e.table_cols * e.page);
    const int64_t max_length = a[10] == Py_None ? held : integer(a[10]);
    const c10::DeviceGuard guard(dev.device);
    return PyLong_FromLong(q4g128_latent_expand(&c, static_cast<const int32_t*>(lengths.data_ptr()), firsts, max_length, count,
                                                packed, scales, mins, &e, current_stream(dev.device)));
    END_HANDLE_TH_ERRORS
}

// latent_prefill(q, k_cache, v_cache, table, q_starts, lengths, scale,
//                max_length, out, workspace)
PyObject* latent_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 10);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache"),
                     &table = tensor(a[3], "table"), &starts = tensor(a[4], "q_starts"), &lengths = tensor(a[5], "lengths");
    const q4g128_kv_cache c = expanded_of(k, v, table);
    const SameDevice dev(k);
    if (q.dim() != 3) value_error("q must be [T][heads][value + 64]");
    const int64_t tokens = q.size(0);
    check(q, "q", at::kHalf, {tokens, c.kv_heads, c.dim + Q4G128_LATENT_ROT});
    if (lengths.dim() != 1) value_error("lengths must be [sequences]");
    const int64_t count = lengths.size(0);
    check(lengths, "lengths", at::kInt, {count});
    check(starts, "q_starts", at::kInt, {count + 1});
    dev.add(q), dev.add(v), dev.add(table), dev.add(starts), dev.add(lengths);
    if (count > c.sequences)
        value_error("table has %lld sequences, fewer than %lld", (long long)c.sequences, (long long)count);
    const float scale = real(a[6]);
    const int64_t max_length = a[7] == Py_None ? (int64_t)c.table_cols * c.page : integer(a[7]);
    const int64_t need = q4g128_latent_prefill_workspace(tokens, count, c.kv_heads, c.dim, max_length);
    if (need < 0) return PyLong_FromLongLong(need);
    const c10::DeviceGuard guard(dev.device);
    const hipStream_t stream = current_stream(dev.device);
    const at::Tensor out = output(a[8], "out", {tokens, c.kv_heads, c.dim}, dev);
    const at::Tensor ws = workspace_of(a[9], need, dev, stream);
    return answer(q4g128_latent_prefill(static_cast<const uint16_t*>(q.data_ptr()), &c,
                                        static_cast<const int32_t*>(starts.data_ptr()),
                                        static_cast<const int32_t*>(lengths.data_ptr()), max_length, tokens, count, scale,
                                        static_cast<uint16_t*>(out.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                                        ws.defined() ? ws.numel() : 0, stream),
                  out);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, nullptr},
    {"attn_decode", (PyCFunction)(void (*)(void))attn_decode, METH_FASTCALL, nullptr},
    {"attn_prefill", (PyCFunction)(void (*)(void))attn_prefill, METH_FASTCALL, nullptr},
    {"attn_tree", (PyCFunction)(void (*)(void))attn_tree, METH_FASTCALL, nullptr},
    {"cache_keep", (PyCFunction)(void (*)(void))cache_keep, METH_FASTCALL, nullptr},
    {"latent_append", (PyCFunction)(void (*)(void))latent_append, METH_FASTCALL, nullptr},
    {"latent_keep", (PyCFunction)(void (*)(void))latent_keep, METH_FASTCALL, nullptr},
    {"latent_attn", (PyCFunction)(void (*)(void))latent_attn, METH_FASTCALL, nullptr},
    {"latent_expand", (PyCFunction)(void (*)(void))latent_expand, METH_FASTCALL, nullptr},
    {"latent_prefill", (PyCFunction)(void (*)(void))latent_prefill, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
