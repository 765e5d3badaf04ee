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
//             q_norm, k_norm, eps, interleaved, mscale, q)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 14);
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
    const float eps = real(a[10]), mscale = real(a[12]);
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) throw python_error();
    const c10::DeviceGuard guard(dev.device);
    const at::Tensor q = output(a[13], "q", {tokens, heads, c.dim}, dev);
    // One row has no next row: any stride will do.
    const int64_t ld = tokens > 1 ? qkv.stride(0) : (columns + 3) / 4 * 4;
    const int32_t rot = pairs > INT32_MAX / 2 ? -1 : (int32_t)(2 * pairs);
    return answer(q4g128_rope_append(static_cast<const float*>(qkv.data_ptr()), ld, tokens, heads, &c, seq,
                                     static_cast<const int32_t*>(positions.data_ptr()), freq, rot, interleaved, mscale,
                                     q_norm, k_norm, eps, static_cast<uint16_t*>(q.data_ptr()),
                                     current_stream(dev.device)),
                  q);
    END_HANDLE_TH_ERRORS
}

// Workspaces of calls that are given none: one per device and stream (calls on
// one stream run one after the other), grown as needed, counters zeroed once.
// A call in a graph capture gets memory of its own, since a graph may be
// replayed on any stream.  Never destroyed: at exit the device may be gone.
at::Tensor kept_workspace(int64_t need, const at::Device& d, hipStream_t stream) {
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
        t.narrow(0, 0, Q4G128_ATTN_COUNTER_BYTES).zero_();
    }
    return t;
}

at::Tensor workspace_of(PyObject* o, int64_t need, const SameDevice& dev, hipStream_t stream) {
    if (o == Py_None) return need > 0 ? kept_workspace(need, dev.device, stream) : at::Tensor();
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
    const at::Tensor ws = workspace_of(a[11], need, t.dev, stream);
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

PyMethodDef methods[] = {
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, nullptr},
    {"attn_decode", (PyCFunction)(void (*)(void))attn_decode, METH_FASTCALL, nullptr},
    {"attn_prefill", (PyCFunction)(void (*)(void))attn_prefill, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
