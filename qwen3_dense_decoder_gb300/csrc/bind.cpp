// bind.cpp -- the Python side of the asynchronous operators: arguments checked,
// outputs allocated and the C entry point called in one step.  For a few rows their
// kernels take 3 to 20 us, and the same steps written in Python took 12 to 15 us of
// host time beside the launch (a call that appends 32 rows: 21.2 us, 7.5 from here;
// one row's decode attention 16.0 and 3.8).
//
// The module has one function an operator, called positionally by the documented
// wrappers of __init__.py.  init() hands over the entry points of libq3.so and the
// function that raises for a return code.
#include <Python.h>

#include <climits>
#include <initializer_list>
#include <optional>
#include <string>

#include <ATen/Context.h>
#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <ATen/record_function.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "q3.h"

namespace {

decltype(&q3_op_kv4_append) p_append;
decltype(&q3_op_kv4_decode_attention) p_decode;
decltype(&q3_op_kv4_prefill_attention) p_prefill;
decltype(&q3_kv4_prefill_workspace) p_workspace;
decltype(&q3_op_token_logprobs) p_logprobs;
decltype(&q3_op_i8_quantize) p_i8_quantize;
decltype(&q3_op_i8_norm) p_i8_norm;
decltype(&q3_op_i8_swiglu) p_i8_swiglu;
decltype(&q3_op_i8_matmul) p_i8_matmul;
decltype(&q3_i8_matmul_workspace_used) p_i8_workspace;
PyObject* g_check;

struct Refusal { std::string what; };        // becomes a ValueError
struct Raised {};                            // a Python error is set

// Allocating may wait for the device and a launch for room in its queue: other Python
// threads run meanwhile.  No tensor that Python knows is copied or let go here.
class Unlocked {
public:
    Unlocked() : state_(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state_); }
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;

private:
    PyThreadState* state_;
};

#define Q3_BEGIN HANDLE_TH_ERRORS try {
#define Q3_END                                                  \
    }                                                           \
    catch (const Refusal& r) {                                  \
        PyErr_SetString(PyExc_ValueError, r.what.c_str());      \
        return nullptr;                                         \
    }                                                           \
    catch (const Raised&) { return nullptr; }                   \
    END_HANDLE_TH_ERRORS

// The arguments of a call
struct Args {
    const char* name;
    PyObject* const* a;

    Args(const char* name, PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : name(name), a(a) {
        if (n != want) refuse("takes " + std::to_string(want) + " arguments");
    }
    [[noreturn]] void refuse(const std::string& what) const { throw Refusal{std::string(name) + ": " + what}; }
    const at::Tensor& tensor(int i) const {
        if (!THPVariable_Check(a[i])) refuse("a tensor is expected, not " + std::string(Py_TYPE(a[i])->tp_name));
        return THPVariable_Unpack(a[i]);
    }
    const at::Tensor* maybe(int i) const { return a[i] == Py_None ? nullptr : &tensor(i); }
    int num(int i) const {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) throw Raised{};
        if (v < INT_MIN || v > INT_MAX) refuse("a number is out of range");
        return (int)v;
    }
    int size(const at::Tensor& t, int d) const {
        if (t.size(d) > INT_MAX) refuse("a tensor is too large");
        return (int)t.size(d);
    }
};

int type_of(const at::Tensor& t)             // Q3_TYPE_*, or -1
{
    switch (t.scalar_type()) {
    case at::kFloat: return Q3_TYPE_F32;
    case at::kHalf: return Q3_TYPE_F16;
    case at::kBFloat16: return Q3_TYPE_BF16;
    default: return -1;
    }
}

void* ptr(const at::Tensor& t) { return t.data_ptr(); }
void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T> T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T> T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

std::string text(at::IntArrayRef shape)
{
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

void int32(const Args& c, const char* what, const at::Tensor& t, at::IntArrayRef shape)
{
    if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_contiguous())
        c.refuse(std::string(what) + " must be contiguous int32 " + text(shape));
}

void pool(const Args& c, const at::Tensor& kv, const at::Tensor& tables, const at::Tensor* status)
{
    if (kv.scalar_type() != at::kByte || kv.dim() != 4 || kv.size(1) != 2 || kv.size(3) != Q3_KV4_TILE_BYTES || !kv.is_contiguous())
        c.refuse("kv must be contiguous uint8 [n_blocks, 2, n_kv, " + std::to_string(Q3_KV4_TILE_BYTES) + "]");
    if (tables.scalar_type() != at::kInt || tables.dim() != 2 || !tables.is_contiguous())
        c.refuse("tables must be contiguous int32 [n_slots, max_blocks]");
    if (status) int32(c, "status", *status, {1});
}

void q_rows(const Args& c, const at::Tensor& q, bool f32)
{
    if ((q.scalar_type() != at::kHalf && !(f32 && q.scalar_type() == at::kFloat)) || q.dim() != 3 || q.size(2) != 128 || q.stride(2) != 1 ||
        (q.stride(1) != 128 && q.size(1) > 1))
        c.refuse(std::string("q must be [T, n_q, 128], ") + (f32 ? "f32 or fp16" : "fp16") + ", with contiguous rows");
}

// The device and stream of a call.  Outputs are memory of the stream that writes
// them, so that none of their earlier uses can still be running; on a stream other
// than the current one the caller's tensors are kept from reuse until it is done.
class Where {
public:
    // launch: whether a kernel will run (else the tensors may be anywhere)
    Where(const Args& c, std::initializer_list<const at::Tensor*> tensors, PyObject* stream, bool launch) : device_((*tensors.begin())->device())
    {
        if (!launch) return;
        const int dev = (*tensors.begin())->get_device();
        for (const at::Tensor* t : tensors)
            if (t && (!t->is_cuda() || t->get_device() != dev)) c.refuse("tensors must be on one CUDA device");
        guard_.emplace((c10::DeviceIndex)dev);
        const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
        raw_ = now.stream();
        if (stream == Py_None) return;
        const long long index = number(stream, "device_index");
        if (index != dev) c.refuse("the stream is another device's");
        raw_ = reinterpret_cast<cudaStream_t>(number(stream, "cuda_stream"));
        if (raw_ == now.stream()) return;
        other_.emplace(c10::cuda::getStreamFromExternal(raw_, (c10::DeviceIndex)dev));
        set_.emplace(*other_);
        for (const at::Tensor* t : tensors)
            if (t) t->record_stream(*other_);
    }
    // On the call's device straight from its allocator, for the current stream: by way
    // of the dispatcher a call that makes two outputs takes 4.6 us of host time, not 3.9.
    at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        if (!direct()) return at::empty(shape, at::TensorOptions().dtype(type).device(device_));
        return at::Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                    type, std::nullopt));
    }
    // rows of k elements, `stride` apart
    at::Tensor rows(int64_t t, int64_t k, int64_t stride, at::ScalarType type) const {
        if (!direct()) return at::empty_strided({t, k}, {stride, 1}, at::TensorOptions().dtype(type).device(device_));
        return at::Tensor(at::detail::empty_strided_generic({t, k}, {stride, 1}, c10::cuda::CUDACachingAllocator::get(),
                                                            c10::DispatchKeySet(c10::DispatchKey::CUDA), type));
    }
    // a caller's tensor, checked, or none yet
    static at::Tensor given(const Args& c, const at::Tensor* t, at::IntArrayRef shape, at::ScalarType type) {
        if (!t) return {};
        check(c, *t, shape, type);
        return *t;
    }
    static void check(const Args& c, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type) {
        if (t.sizes() != shape || t.scalar_type() != type || !t.is_contiguous())
            c.refuse(std::string("outputs must be contiguous ") + c10::toString(type) + " " + text(shape));
    }
    void* stream() const { return raw_; }

private:
    // Whether nothing but the allocator has a part in making a tensor: not the filling
    // of new memory, a mode or transform of this thread, or a profiler
    bool direct() const {
        if (!guard_ || at::hasCallbacks()) return false;
        const at::Context& now = at::globalContext();
        if (now.deterministicAlgorithms() && now.deterministicFillUninitializedMemory()) return false;
        return (c10::impl::tls_local_dispatch_key_set().included_ - c10::default_included_set).empty();
    }
    static long long number(PyObject* o, const char* what) {
        PyObject* v = PyObject_GetAttrString(o, what);
        if (!v) throw Raised{};
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred()) throw Raised{};
        return x;
    }
    c10::Device device_;
    cudaStream_t raw_ = nullptr;
    std::optional<c10::cuda::CUDAGuard> guard_;
    std::optional<c10::cuda::CUDAStream> other_;
    std::optional<c10::cuda::CUDAStreamGuard> set_;
};

void check(int rc)
{
    if (rc == 0) return;
    PyObject* r = PyObject_CallFunction(g_check, "i", rc);
    Py_XDECREF(r);
    if (!r) throw Raised{};
}

// (qkv, q_gain, k_gain, rope, row_pos, row_slot, tables, kv, n_q, eps, q_out, kv_out, status, stream)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_kv4_append", a, n, 14);
    const at::Tensor &qkv = c.tensor(0), &qg = c.tensor(1), &kg = c.tensor(2), &rope = c.tensor(3), &pos = c.tensor(4), &slot = c.tensor(5),
                     &tables = c.tensor(6), &kv = c.tensor(7);
    const at::Tensor *q_given = c.maybe(10), *kv_out = c.maybe(11), *status = c.maybe(12);
    pool(c, kv, tables, status);
    const int n_q = c.num(8), n_kv = c.size(kv, 2), type = type_of(qkv);
    const double eps = PyFloat_AsDouble(a[9]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const int64_t width = ((int64_t)n_q + 2ll * n_kv) * 128;
    if (type < 0 || qkv.dim() != 2 || qkv.size(1) != width || qkv.stride(1) != 1)
        c.refuse("qkv must be f32, fp16 or bf16 [T, (n_q + 2 n_kv) * 128]");
    const int T = c.size(qkv, 0);
    for (const at::Tensor* g : {&qg, &kg})
        if (g->scalar_type() != at::kBFloat16 || g->dim() != 1 || g->size(0) != 128 || !g->is_contiguous()) c.refuse("gains must be bf16 [128]");
    if (rope.scalar_type() != at::kFloat || rope.dim() != 3 || rope.size(1) != 64 || rope.size(2) != 2 || !rope.is_contiguous())
        c.refuse("rope must be f32 [n, 64, 2]");
    int32(c, "row_pos", pos, {T});
    int32(c, "row_slot", slot, {T});
    const Where w(c, {&qkv, &qg, &kg, &rope, &pos, &slot, &tables, &kv, q_given, kv_out, status}, a[13], T > 0);
    if (kv_out) Where::check(c, *kv_out, {T, 2, n_kv, 128}, at::kHalf);
    at::Tensor q = Where::given(c, q_given, {T, n_q, 128}, at::kHalf);
    int rc = 0;
    {
        const Unlocked other_threads_run;
        if (!q.defined()) q = w.make({T, n_q, 128}, at::kHalf);
        if (T > 0)
            rc = p_append(ptr(qkv), type, T > 1 ? qkv.stride(0) : width, ptr(qg), ptr(kg), (float)eps, ptr<float>(rope), c.size(rope, 0),
                          ptr<int32_t>(pos), ptr<int32_t>(slot), T, n_q, n_kv, ptr<int32_t>(tables), c.size(tables, 0), c.size(tables, 1),
                          ptr(kv), c.size(kv, 0), ptr(q), ptr(kv_out), ptr<int32_t>(status), w.stream());
    }
    check(rc);
    return THPVariable_Wrap(q);
    Q3_END
}

// (q, row_pos, row_slot, tables, kv, max_ctx, out, status, stream)
PyObject* kv4_decode_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_kv4_decode_attention", a, n, 9);
    const at::Tensor &q = c.tensor(0), &pos = c.tensor(1), &slot = c.tensor(2), &tables = c.tensor(3), &kv = c.tensor(4);
    const at::Tensor *given = c.maybe(6), *status = c.maybe(7);
    const int max_ctx = c.num(5);
    pool(c, kv, tables, status);
    q_rows(c, q, true);
    const int T = c.size(q, 0), n_q = c.size(q, 1);
    int32(c, "row_pos", pos, {T});
    int32(c, "row_slot", slot, {T});
    const Where w(c, {&q, &pos, &slot, &tables, &kv, given, status}, a[8], T > 0);
    at::Tensor out = Where::given(c, given, {T, n_q, 128}, given && given->scalar_type() == at::kFloat ? at::kFloat : at::kHalf);
    int rc = 0;
    {
        const Unlocked other_threads_run;
        if (!out.defined()) out = w.make({T, n_q, 128}, at::kHalf);
        if (T > 0)
            rc = p_decode(ptr(q), type_of(q), T > 1 ? q.stride(0) : n_q * 128ll, ptr<int32_t>(pos), ptr<int32_t>(slot), T, n_q, c.size(kv, 2),
                          ptr<int32_t>(tables), c.size(tables, 0), c.size(tables, 1), max_ctx, ptr(kv), c.size(kv, 0), ptr(out), type_of(out),
                          ptr<int32_t>(status), w.stream());
    }
    check(rc);
    return THPVariable_Wrap(out);
    Q3_END
}

// (q, seq_rows, seq_pos, tables, kv, seq_slot, out, workspace, status, stream)
PyObject* kv4_prefill_attention(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_kv4_prefill_attention", a, n, 10);
    const at::Tensor &q = c.tensor(0), &rows = c.tensor(1), &pos = c.tensor(2), &tables = c.tensor(3), &kv = c.tensor(4);
    const at::Tensor *slot = c.maybe(5), *given = c.maybe(6), *space = c.maybe(7), *status = c.maybe(8);
    pool(c, kv, tables, status);
    q_rows(c, q, false);
    const int T = c.size(q, 0), n_q = c.size(q, 1), n_kv = c.size(kv, 2), n_blocks = c.size(kv, 0);
    if (pos.dim() != 1) c.refuse("seq_pos must be int32 [sequences]");
    const int ns = c.size(pos, 0), n_slots = c.size(tables, 0), max_blocks = c.size(tables, 1);
    int32(c, "seq_rows", rows, {ns + 1ll});
    int32(c, "seq_pos", pos, {ns});
    if (slot) int32(c, "seq_slot", *slot, {ns});
    const bool launch = T > 0 && ns > 0;
    const Where w(c, {&q, &rows, &pos, &tables, &kv, slot, given, space, status}, a[9], launch);
    int64_t need = 0;
    if (launch) {
        check(p_workspace(ns, T, n_q, n_kv, max_blocks, n_blocks, &need));
        if (space && (space->scalar_type() != at::kByte || !space->is_contiguous() || space->numel() < need))
            c.refuse("workspace must be contiguous uint8, at least " + std::to_string(need) + " bytes");
    }
    at::Tensor out = Where::given(c, given, {T, n_q, 128}, at::kHalf), ws;
    if (space) ws = *space;
    int rc = 0;
    {
        const Unlocked other_threads_run;
        if (!out.defined()) out = w.make({T, n_q, 128}, at::kHalf);
        if (launch) {
            if (!ws.defined()) ws = w.make({need}, at::kByte);
            rc = p_prefill(ptr(q), T > 1 ? q.stride(0) : n_q * 128ll, ptr<int32_t>(rows), ptr<int32_t>(pos), ptr<int32_t>(slot), ns, T, n_q,
                           n_kv, ptr<int32_t>(tables), n_slots, max_blocks, ptr(kv), n_blocks, ptr(out), ptr(ws), ws.numel(),
                           ptr<int32_t>(status), w.stream());
        }
    }
    check(rc);
    return THPVariable_Wrap(out);
    Q3_END
}

// (logits, targets, top_k, status, stream)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_token_logprobs", a, n, 5);
    const at::Tensor& x = c.tensor(0);
    const at::Tensor *targets = c.maybe(1), *status = c.maybe(3);
    const int top = c.num(2), type = type_of(x);
    if (type < 0 || x.dim() != 2 || (x.stride(1) != 1 && x.size(1) > 1)) c.refuse("logits must be f32, fp16 or bf16 [N, V] with contiguous rows");
    const int N = c.size(x, 0), V = c.size(x, 1);
    if (targets) int32(c, "targets", *targets, {N});
    if (status) int32(c, "status", *status, {1});
    if (top < 0) c.refuse("top_k must not be negative");
    const Where w(c, {&x, targets, status}, a[4], N > 0);
    at::Tensor lp, entropy, ids, values;
    int rc = 0;
    {
        const Unlocked other_threads_run;
        if (targets) lp = w.make({N}, at::kFloat);
        entropy = w.make({N}, at::kFloat);
        ids = w.make({N, top}, at::kInt);
        values = w.make({N, top}, at::kFloat);
        if (N > 0)
            rc = p_logprobs(ptr(x), type, N > 1 ? x.stride(0) : V, N, V, ptr<int32_t>(targets), top, targets ? ptr<float>(lp) : nullptr,
                            ptr<float>(entropy), ptr<int32_t>(ids), ptr<float>(values), ptr<int32_t>(status), w.stream());
    }
    check(rc);
    PyObject* r = PyTuple_New(4);
    if (!r) throw Raised{};
    if (targets) PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(lp));
    else PyTuple_SET_ITEM(r, 0, Py_NewRef(Py_None));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(entropy));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(ids));
    PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(values));
    return r;
    Q3_END
}

// ---------------------------------------------------------------- 8-bit integer rows

// rows of f32, fp16 or bf16 values
int i8_values(const Args& c, const char* what, const at::Tensor& t)
{
    const int type = type_of(t);
    if (type < 0 || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1)) c.refuse(std::string(what) + " must be f32, fp16 or bf16 rows, each contiguous");
    return type;
}
// elements between rows; one row has no next
int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// int8 rows that begin on 16-byte boundaries
void i8_codes(const Args& c, const char* what, const at::Tensor& t)
{
    if (t.scalar_type() != at::kChar || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) % 16) ||
        reinterpret_cast<uintptr_t>(t.data_ptr()) % 16)
        c.refuse(std::string(what) + " must be int8 rows that begin on 16-byte boundaries");
}
int64_t code_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : (t.size(1) + 15) / 16 * 16; }

void f32(const Args& c, const char* what, const at::Tensor& t, int64_t n)
{
    if (t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        c.refuse(std::string(what) + " must be contiguous f32 [" + std::to_string(n) + "]");
}

// codes, scales and values of the three writers, checked or made
struct I8Out {
    at::Tensor codes, scales;
    const at::Tensor* values;
    int T, K;

    I8Out(const Args& c, int T, int K, const at::Tensor* codes_given, const at::Tensor* scales_given, const at::Tensor* values, const at::Tensor* status)
        : values(values), T(T), K(K)
    {
        if (K < 1) c.refuse("rows must have at least one value");
        if (codes_given) {
            i8_codes(c, "codes", *codes_given);
            if (codes_given->size(0) != T || codes_given->size(1) != K) c.refuse("codes must be [" + std::to_string(T) + ", " + std::to_string(K) + "]");
            codes = *codes_given;
        }
        if (scales_given) {
            f32(c, "scales", *scales_given, T);
            scales = *scales_given;
        }
        if (values && (type_of(*values) < 0 || values->sizes() != at::IntArrayRef({T, K}) || !values->is_contiguous()))
            c.refuse("values must be contiguous f32, fp16 or bf16 [" + std::to_string(T) + ", " + std::to_string(K) + "]");
        if (status) int32(c, "status", *status, {1});
    }
    void make(const Where& w) {                  // no tensor of the caller's is touched
        if (!codes.defined()) {
            codes = w.rows(T, K, (K + 15ll) / 16 * 16, at::kChar);
        }
        if (!scales.defined()) scales = w.make({T}, at::kFloat);
    }
    int values_type() const { return values ? type_of(*values) : 0; }
};

PyObject* i8_pair(const I8Out& o, const at::Tensor* third = nullptr)
{
    PyObject* r = PyTuple_New(third ? 3 : 2);
    if (!r) throw Raised{};
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(o.codes));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(o.scales));
    if (third) PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(*third));
    return r;
}

// (x, codes, scales, values, status, stream)
PyObject* i8_rows(const char* name, PyObject* const* a, Py_ssize_t n, int parts, decltype(p_i8_quantize) entry)
{
    const Args c(name, a, n, 6);
    const at::Tensor& x = c.tensor(0);
    const at::Tensor *codes = c.maybe(1), *scales = c.maybe(2), *values = c.maybe(3), *status = c.maybe(4);
    const int type = i8_values(c, "x", x), T = c.size(x, 0), width = c.size(x, 1);
    if (width % parts) c.refuse("x must be [T, 2 F], gate then up");
    const int K = width / parts;
    I8Out o(c, T, K, codes, scales, values, status);
    const Where w(c, {&x, codes, scales, values, status}, a[5], T > 0);
    int rc = 0;
    {
        const Unlocked other_threads_run;
        o.make(w);
        if (T > 0)
            rc = entry(ptr(x), type, row_stride(x), T, K, ptr<int8_t>(o.codes), code_stride(o.codes), ptr<float>(o.scales), ptr(values),
                       o.values_type(), ptr<int32_t>(status), w.stream());
    }
    check(rc);
    return i8_pair(o);
}

PyObject* i8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    return i8_rows("op_i8_quantize", a, n, 1, p_i8_quantize);
    Q3_END
}

PyObject* i8_swiglu(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    return i8_rows("op_i8_swiglu", a, n, 2, p_i8_swiglu);
    Q3_END
}

// (x, gain, eps, delta, sum_out, codes, scales, values, status, stream)
PyObject* i8_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_i8_norm", a, n, 10);
    const at::Tensor &x = c.tensor(0), &gain = c.tensor(1);
    const double eps = PyFloat_AsDouble(a[2]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const at::Tensor *delta = c.maybe(3), *sum_given = c.maybe(4), *codes = c.maybe(5), *scales = c.maybe(6), *values = c.maybe(7),
                     *status = c.maybe(8);
    const int type = i8_values(c, "x", x), T = c.size(x, 0), K = c.size(x, 1);
    if (gain.scalar_type() != at::kBFloat16 || gain.dim() != 1 || gain.size(0) != K || !gain.is_contiguous())
        c.refuse("gain must be contiguous bf16 [" + std::to_string(K) + "]");
    const int delta_type = delta ? i8_values(c, "delta", *delta) : 0;
    if (delta && delta->sizes() != x.sizes()) c.refuse("delta must be " + text(x.sizes()));
    if (sum_given && !delta) c.refuse("sum_out is for calls with delta");
    if (sum_given && (i8_values(c, "sum_out", *sum_given) != type || sum_given->sizes() != x.sizes())) c.refuse("sum_out must be of x's type and size");
    I8Out o(c, T, K, codes, scales, values, status);
    const Where w(c, {&x, &gain, delta, sum_given, codes, scales, values, status}, a[9], T > 0);
    at::Tensor sum;
    if (!delta) sum = x;
    else if (sum_given) sum = *sum_given;
    int rc = 0;
    {
        const Unlocked other_threads_run;
        o.make(w);
        if (!sum.defined()) sum = w.make({T, K}, x.scalar_type());
        if (T > 0)
            rc = p_i8_norm(ptr(x), type, row_stride(x), ptr(delta), delta_type, delta ? row_stride(*delta) : 0, delta ? ptr(sum) : nullptr,
                           delta ? row_stride(sum) : 0, ptr(gain), (float)eps, T, K, ptr<int8_t>(o.codes), code_stride(o.codes),
                           ptr<float>(o.scales), ptr(values), o.values_type(), ptr<int32_t>(status), w.stream());
    }
    check(rc);
    return i8_pair(o, &sum);
    Q3_END
}

// (x, x_scales, w, w_scales, out, dtype, workspace, status, stream)
PyObject* i8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    Q3_BEGIN
    const Args c("op_i8_matmul", a, n, 9);
    const at::Tensor &x = c.tensor(0), &xs = c.tensor(1), &wt = c.tensor(2), &ws = c.tensor(3);
    const at::Tensor *given = c.maybe(4), *space = c.maybe(6), *status = c.maybe(7);
    i8_codes(c, "x", x);
    i8_codes(c, "w", wt);
    const int T = c.size(x, 0), K = c.size(x, 1), M = c.size(wt, 0);
    if (wt.size(1) != K) c.refuse("w must be [M, " + std::to_string(K) + "]");
    f32(c, "x_scales", xs, T);
    f32(c, "w_scales", ws, M);
    at::ScalarType type = at::kHalf;
    if (a[5] != Py_None) {
        if (!THPDtype_Check(a[5])) c.refuse("dtype must be a torch.dtype");
        type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    }
    if (type != at::kFloat && type != at::kHalf && type != at::kBFloat16) c.refuse("dtype must be f32, fp16 or bf16");
    if (given) {
        i8_values(c, "out", *given);
        if (given->size(0) != T || given->size(1) != M || (a[5] != Py_None && given->scalar_type() != type))
            c.refuse("out must be [" + std::to_string(T) + ", " + std::to_string(M) + "], of dtype where that is given");
    }
    if (status) int32(c, "status", *status, {1});
    const Where w(c, {&x, &xs, &wt, &ws, given, space, status}, a[8], T > 0);
    int64_t need = 0;
    if (T > 0) {
        check(p_i8_workspace(T, M, K, &need));
        if (space && (space->scalar_type() != at::kByte || !space->is_contiguous() || space->numel() < need))
            c.refuse("workspace must be contiguous uint8, at least " + std::to_string(need) + " bytes");
    }
    at::Tensor out, room;
    if (given) out = *given;
    if (space) room = *space;
    int rc = 0;
    {
        const Unlocked other_threads_run;
        if (!out.defined()) out = w.make({T, M}, type);
        if (T > 0) {
            if (need && !room.defined()) room = w.make({need}, at::kByte);
            rc = p_i8_matmul(ptr<int8_t>(x), code_stride(x), ptr<float>(xs), ptr<int8_t>(wt), code_stride(wt), ptr<float>(ws), T, M, K, ptr(out),
                             type_of(out), row_stride(out), need ? ptr(room) : nullptr, need ? room.numel() : 0, ptr<int32_t>(status), w.stream());
        }
    }
    check(rc);
    return THPVariable_Wrap(out);
    Q3_END
}

// (check, addresses of the entry points)
PyObject* init(PyObject*, PyObject* args)
{
    PyObject* f;
    unsigned long long p[10];
    if (!PyArg_ParseTuple(args, "OKKKKKKKKKK", &f, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5], &p[6], &p[7], &p[8], &p[9])) return nullptr;
    Py_INCREF(f);
    Py_XDECREF(g_check);
    g_check = f;
    p_append = reinterpret_cast<decltype(p_append)>(p[0]);
    p_decode = reinterpret_cast<decltype(p_decode)>(p[1]);
    p_prefill = reinterpret_cast<decltype(p_prefill)>(p[2]);
    p_workspace = reinterpret_cast<decltype(p_workspace)>(p[3]);
    p_logprobs = reinterpret_cast<decltype(p_logprobs)>(p[4]);
    p_i8_quantize = reinterpret_cast<decltype(p_i8_quantize)>(p[5]);
    p_i8_norm = reinterpret_cast<decltype(p_i8_norm)>(p[6]);
    p_i8_swiglu = reinterpret_cast<decltype(p_i8_swiglu)>(p[7]);
    p_i8_matmul = reinterpret_cast<decltype(p_i8_matmul)>(p[8]);
    p_i8_workspace = reinterpret_cast<decltype(p_i8_workspace)>(p[9]);
    Py_RETURN_NONE;
}

#define Q3_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {Q3_FAST(kv4_append), Q3_FAST(kv4_decode_attention), Q3_FAST(kv4_prefill_attention), Q3_FAST(token_logprobs),
                         Q3_FAST(i8_quantize), Q3_FAST(i8_norm), Q3_FAST(i8_swiglu), Q3_FAST(i8_matmul),
                         {"init", init, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops() { return PyModule_Create(&module_def); }
