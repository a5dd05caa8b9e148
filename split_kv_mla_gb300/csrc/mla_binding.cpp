// mla_binding.cpp -- argument checks and output tensors of the cache and
// shared-prefix entry points, for mla.py.
//
// A small call spends more of the host's time on its arguments than on its
// launches when they are checked in Python and passed through ctypes: eleven
// tensors' types, devices, strides and addresses are forty-four method calls.
// Here they are field reads.  Nothing is computed: each function checks, allocates
// the outputs that the caller did not give, and makes one call of the C ABI on the
// current stream, through the addresses that bind() was given, so it calls the very
// library that mla.py has loaded.  (Measured with a GB300's Grace host, µs of the
// host's time per call, these checks in Python and ctypes / here: shared-prefix
// decode at B=4, P=1024 24 / 11.6; append of 8 tokens 21 / 11.0; fork of two
// requests of 700 18 / 10.9; compaction of 8192 rows 19 / 13.3, two launches.)
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "mla_decode.h"

namespace {

struct BadArgument {
    std::string what;
};

[[noreturn]] void bad(const std::string& what) { throw BadArgument{what}; }

decltype(&mla_prefix_decode) prefix_decode_fn;
decltype(&mla_cache_append) append_fn;
decltype(&mla_cache_fork) fork_fn;
decltype(&mla_cache_compact) compact_fn;
PyObject* mla_error;   // the exception of a status other than MLA_OK

const char* type_name(at::ScalarType t)
{
    switch (t) {
    case at::kInt: return "torch.int32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}

// The tensor behind an argument; undefined for None.
const at::Tensor& tensor(PyObject* o, const char* name)
{
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor& given(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.defined()) bad(std::string(name) + " must be given");
    return t;
}

// The CUDA device of a call's first tensor, which must be the current one (the
// library launches on the current device).
int call_device(const at::Tensor& t)
{
    if (!t.is_cuda()) bad("tensors must be CUDA tensors");
    const int dev = t.get_device(), now = c10::cuda::current_device();
    if (dev != now)
        bad("the tensors are on cuda:" + std::to_string(dev) + ", but the current device is cuda:" +
            std::to_string(now));
    return dev;
}

void on_device(const at::Tensor& t, const char* name, int dev)
{
    if (!t.is_cuda() || t.get_device() != dev)
        bad(std::string(name) + " must be on cuda:" + std::to_string(dev) + ", got " +
            t.device().str());
}

// Address of a contiguous tensor of the type on device dev; NULL if undefined.
void* address(const at::Tensor& t, const char* name, at::ScalarType type, int dev)
{
    if (!t.defined()) return nullptr;
    if (t.scalar_type() != type)
        bad(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    on_device(t, name, dev);
    if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

const int32_t* table(const at::Tensor& t, const char* name, int dev)
{
    return static_cast<const int32_t*>(address(t, name, at::kInt, dev));
}

// The pool, [rows, row_bytes] or [rows, 1, row_bytes], of bytes.
void check_pool(const at::Tensor& t, int dev)
{
    if (t.element_size() != 1 || !(t.dim() == 2 || (t.dim() == 3 && t.size(1) == 1)))
        bad("pool must hold one byte per element, [rows, row_bytes]");
    on_device(t, "pool", dev);
    if (!t.is_contiguous()) bad("pool must be contiguous");
}

// A bf16 tensor whose rows are contiguous.
void check_rows(const at::Tensor& t, const char* name, int64_t dims, int dev)
{
    if (t.scalar_type() != at::kBFloat16)
        bad(std::string(name) + " must be torch.bfloat16, got " + type_name(t.scalar_type()));
    on_device(t, name, dev);
    if (t.dim() != dims) bad(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
    if (t.stride(-1) != 1 && t.size(-1) > 1) bad(std::string(name) + " must have contiguous rows");
}

at::Tensor allocate(at::IntArrayRef shape, at::ScalarType type, int dev)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int32_t integer32(PyObject* o, const char* name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " is out of range");
    return static_cast<int32_t>(v);
}

float real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void* current_stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

// The status of a C call as an exception, if it is one.
void check(int status, const char* where)
{
    if (status == MLA_OK) return;
    PyObject* e = PyObject_CallFunction(mla_error, "is", status, where);
    if (e != nullptr) {
        PyErr_SetObject(mla_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

int size32(int64_t n)
{
    if (n > INT32_MAX) bad("a size is out of range");
    return static_cast<int>(n);
}

// What a caller gets back: the tensor that it gave, or the new one.
PyObject* output(PyObject* passed, const at::Tensor& t)
{
    if (passed != Py_None) {
        Py_INCREF(passed);
        return passed;
    }
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* pair(PyObject* a, PyObject* b)
{
    PyObject* r = a != nullptr && b != nullptr ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f)
{
    HANDLE_TH_ERRORS
    try {
        if (got != want) bad("wrong number of arguments");
        return f();
    } catch (const BadArgument& e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(prefix_decode, append, fork, compact, MlaError): addresses of the library's
// entry points, and the exception to raise.
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject* {
        prefix_decode_fn = reinterpret_cast<decltype(prefix_decode_fn)>(integer(v[0]));
        append_fn = reinterpret_cast<decltype(append_fn)>(integer(v[1]));
        fork_fn = reinterpret_cast<decltype(fork_fn)>(integer(v[2]));
        compact_fn = reinterpret_cast<decltype(compact_fn)>(integer(v[3]));
        Py_XSETREF(mla_error, Py_NewRef(v[4]));
        Py_RETURN_NONE;
    });
}

// prefix_decode(plan address, q_lat, q_pe, pool, prefix_indices, seq_lens, kv_indices,
// kv_indptr, scale, kv_scale, prefix_len, o, lse, workspace, return_lse)
PyObject* prefix_decode(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded(n, 15, [&]() -> PyObject* {
        const auto* plan = reinterpret_cast<const mla_prefix_plan_t*>(integer(v[0]));
        const at::Tensor& q_lat = given(v[1], "q_lat");
        const at::Tensor& q_pe = given(v[2], "q_pe");
        const at::Tensor& pool = given(v[3], "pool");
        const at::Tensor& prefix = given(v[4], "prefix_indices");
        const at::Tensor& lens = given(v[5], "seq_lens");
        const at::Tensor& indices = given(v[6], "kv_indices");
        const at::Tensor& indptr = given(v[7], "kv_indptr");
        const at::Tensor& prefix_len = tensor(v[10], "prefix_len");
        at::Tensor o = tensor(v[11], "o"), lse = tensor(v[12], "lse");
        const at::Tensor& ws = given(v[13], "workspace");
        const int dev = call_device(q_lat);
        check_pool(pool, dev);
        if (q_lat.dim() != 3 || q_pe.dim() != 3 || lens.dim() != 1)
            bad("q_lat and q_pe must have three dimensions, seq_lens one");
        const int64_t R = q_lat.size(0), H = q_lat.size(1), batch = lens.size(0);
        const int64_t q_len = batch > 0 ? R / batch : plan->own.q_len;
        if (R != batch * q_len || q_lat.size(2) != 512 || q_pe.size(0) != R || q_pe.size(1) != H ||
            q_pe.size(2) != 64 || pool.size(-1) != 576 || indptr.numel() != batch + 1)
            bad("q_lat [B * q_len, H, 512], q_pe [B * q_len, H, 64], pool [N, 576] and "
                "kv_indptr [B + 1] must agree");
        if (prefix.numel() != plan->prefix_cap || indices.numel() != plan->own.total_keys)
            bad("prefix_indices and kv_indices must have the plan's entries");
        if (prefix_len.defined() && prefix_len.numel() != 1) bad("prefix_len must have one entry");
        if (!o.defined()) o = allocate({R, H, 512}, at::kBFloat16, dev);
        else if (o.sizes() != q_lat.sizes()) bad("o must have q_lat's shape");
        if (lse.defined() ? lse.numel() != R * H : false) bad("lse must be [B * q_len, H]");
        if (!lse.defined() && truth(v[14])) lse = allocate({R, H}, at::kFloat, dev);
        const void* q0 = address(q_lat, "q_lat", at::kBFloat16, dev);
        const void* q1 = address(q_pe, "q_pe", at::kBFloat16, dev);
        const int32_t* pi = table(prefix, "prefix_indices", dev);
        const int32_t* pl = table(prefix_len, "prefix_len", dev);
        const int32_t* sl = table(lens, "seq_lens", dev);
        const int32_t* ki = table(indices, "kv_indices", dev);
        const int32_t* kp = table(indptr, "kv_indptr", dev);
        void* po = address(o, "o", at::kBFloat16, dev);
        float* pz = static_cast<float*>(address(lse, "lse", at::kFloat, dev));
        void* pw = address(ws, "workspace", at::kByte, dev);
        const float scale = real(v[8]), kv_scale = real(v[9]);
        void* stream = current_stream(dev);
        const int b = size32(batch), ql = size32(q_len), h = size32(H);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = prefix_decode_fn(plan, q0, q1, pool.data_ptr(), pool.size(0), pi, pl, sl, ki, kp,
                                  b, ql, h, scale, kv_scale, po, pz, pw, ws.numel(), stream);
        Py_END_ALLOW_THREADS
        check(status, "mla_prefix_decode");
        return pair(output(v[11], o), output(v[12], lse));
    });
}

// cache_append(kv, slots, pool, positions, cos_sin, kv_scale, q, kv_weight, kv_norm_cols,
// q_weight, q_norm, eps, half_split, q_nope, q_pe, workspace)
PyObject* cache_append(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded(n, 16, [&]() -> PyObject* {
        const at::Tensor& kv = tensor(v[0], "kv");
        const at::Tensor& slots = tensor(v[1], "slots");
        const at::Tensor& pool = tensor(v[2], "pool");
        const at::Tensor& positions = given(v[3], "positions");
        const at::Tensor& cos_sin = given(v[4], "cos_sin");
        const at::Tensor& q = tensor(v[6], "q");
        const at::Tensor& kv_weight = tensor(v[7], "kv_weight");
        const at::Tensor& q_weight = tensor(v[9], "q_weight");
        at::Tensor q_nope = tensor(v[13], "q_nope"), q_pe = tensor(v[14], "q_pe");
        if (!kv.defined() && !q.defined()) bad("kv or q must be given");
        const at::Tensor& ws = given(v[15], "workspace");
        const at::Tensor& first = kv.defined() ? kv : q;
        const int dev = call_device(first);
        const int64_t T = first.dim() > 0 ? first.size(0) : 0;
        const int32_t norm_cols = integer32(v[8], "kv_norm_cols");
        int64_t pool_rows = 0, width = 0, H = 0, cols = 0;
        const int32_t* ps = nullptr;
        if (kv.defined()) {
            if (!slots.defined() || !pool.defined()) bad("slots and pool must be given with kv");
            check_pool(pool, dev);
            pool_rows = pool.size(0);
            width = pool.size(-1);
            check_rows(kv, "kv", 2, dev);
            if (kv.size(1) != width)
                bad("kv must be [T, " + std::to_string(width) + "], the pool's row width");
            if (slots.numel() != T) bad("slots must have one entry per token");
            if (kv_weight.defined() && kv_weight.numel() != norm_cols)
                bad("kv_weight must have kv_norm_cols entries");
            ps = table(slots, "slots", dev);
        }
        if (positions.numel() != T) bad("positions must have one entry per token");
        if (cos_sin.dim() != 2 || cos_sin.size(1) != 64) bad("cos_sin must be [max_positions, 64]");
        if (q.defined()) {
            check_rows(q, "q", 3, dev);
            if (q.size(0) != T) bad("q must be [T, H, q_cols]");
            H = q.size(1);
            cols = q.size(2);
            if (q_weight.defined() && q_weight.numel() != cols) bad("q_weight must have q_cols entries");
            if (!q_nope.defined() && cols > 64) q_nope = allocate({T, H, cols - 64}, at::kBFloat16, dev);
            if (!q_pe.defined()) q_pe = allocate({T, H, 64}, at::kBFloat16, dev);
            if (q_pe.numel() != T * H * 64 || (cols > 64 && q_nope.numel() != T * H * (cols - 64)))
                bad("q_nope and q_pe must be [T, H, q_cols - 64] and [T, H, 64]");
        }
        const void* kw = address(kv_weight, "kv_weight", at::kBFloat16, dev);
        const void* qw = address(q_weight, "q_weight", at::kBFloat16, dev);
        void* qn = address(q_nope, "q_nope", at::kBFloat16, dev);
        void* qp = address(q_pe, "q_pe", at::kBFloat16, dev);
        const int32_t* pp = table(positions, "positions", dev);
        const float* cs = static_cast<const float*>(address(cos_sin, "cos_sin", at::kFloat, dev));
        void* pw = address(ws, "workspace", at::kByte, dev);
        const float kv_scale = real(v[5]), eps = real(v[11]);
        const int q_norm = truth(v[10]) ? 1 : 0, half = truth(v[12]) ? 1 : 0;
        void* stream = current_stream(dev);
        const void* kvp = kv.defined() ? kv.data_ptr() : nullptr;
        void* pool_p = kv.defined() ? pool.data_ptr() : nullptr;
        const void* qd = q.defined() ? q.data_ptr() : nullptr;
        const int64_t kvs = kv.defined() ? kv.stride(0) : 0;
        const int64_t qts = q.defined() ? q.stride(0) : 0, qhs = q.defined() ? q.stride(1) : 0;
        const int w = size32(width), c = size32(cols), t = size32(T), h = size32(H);
        const int64_t most = cos_sin.size(0);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = append_fn(kvp, kvs, kw, norm_cols, ps, pool_p, pool_rows, w, kv_scale, qd, qts, qhs,
                           qw, q_norm, c, qn, qp, pp, cs, most, half, eps, t, h, pw, ws.numel(),
                           stream);
        Py_END_ALLOW_THREADS
        check(status, "mla_cache_append");
        return pair(output(v[13], q_nope), output(v[14], q_pe));
    });
}

// cache_fork(pool, kv_indices, kv_indptr, parents, keep, child_indptr, total, fresh,
// fresh_indptr, table, workspace)
PyObject* cache_fork(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded(n, 11, [&]() -> PyObject* {
        const at::Tensor& pool = given(v[0], "pool");
        const at::Tensor& indices = given(v[1], "kv_indices");
        const at::Tensor& indptr = given(v[2], "kv_indptr");
        const at::Tensor& parents = given(v[3], "parents");
        const at::Tensor& keep = given(v[4], "keep");
        const at::Tensor& child = given(v[5], "child_indptr");
        const at::Tensor& fresh = given(v[7], "fresh");
        const at::Tensor& fresh_indptr = given(v[8], "fresh_indptr");
        at::Tensor out = tensor(v[9], "table");
        const at::Tensor& ws = given(v[10], "workspace");
        const int dev = call_device(pool);
        check_pool(pool, dev);
        const int64_t total = integer(v[6]), F = parents.numel();
        if (keep.numel() != F || child.numel() != F + 1 || fresh_indptr.numel() != F + 1)
            bad("keep, child_indptr and fresh_indptr must match parents");
        if (total < 0) bad("total must not be negative");
        if (!out.defined()) out = allocate({total}, at::kInt, dev);
        else if (out.numel() < total) bad("table must have total entries");
        const int32_t* ki = table(indices, "kv_indices", dev);
        const int32_t* kp = table(indptr, "kv_indptr", dev);
        const int32_t* pa = table(parents, "parents", dev);
        const int32_t* ke = table(keep, "keep", dev);
        const int32_t* ci = table(child, "child_indptr", dev);
        const int32_t* fr = table(fresh, "fresh", dev);
        const int32_t* fi = table(fresh_indptr, "fresh_indptr", dev);
        int32_t* to = static_cast<int32_t*>(address(out, "table", at::kInt, dev));
        void* pw = address(ws, "workspace", at::kByte, dev);
        void* stream = current_stream(dev);
        const int w = size32(pool.size(-1)), f = size32(F);
        const int np = size32(indptr.numel() > 0 ? indptr.numel() - 1 : 0);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = fork_fn(pool.data_ptr(), pool.size(0), w, ki, indices.numel(), kp, np, pa, ke, ci, f,
                         fr, fresh.numel(), fi, to, total, pw, ws.numel(), stream);
        Py_END_ALLOW_THREADS
        check(status, "mla_cache_fork");
        return output(v[9], out);
    });
}

// cache_compact(pool, kv_indices, new_indices, live, workspace)
PyObject* cache_compact(PyObject*, PyObject* const* v, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject* {
        const at::Tensor& pool = given(v[0], "pool");
        const at::Tensor& indices = given(v[1], "kv_indices");
        at::Tensor out = tensor(v[2], "new_indices"), live = tensor(v[3], "live");
        const at::Tensor& ws = given(v[4], "workspace");
        const int dev = call_device(pool);
        check_pool(pool, dev);
        const int32_t* ki = table(indices, "kv_indices", dev);
        if (!out.defined()) out = allocate(indices.sizes(), at::kInt, dev);
        else if (out.numel() != indices.numel()) bad("new_indices must match kv_indices");
        if (!live.defined()) live = allocate({1}, at::kInt, dev);
        else if (live.numel() < 1) bad("live must have an entry");
        int32_t* to = static_cast<int32_t*>(address(out, "new_indices", at::kInt, dev));
        int32_t* pl = static_cast<int32_t*>(address(live, "live", at::kInt, dev));
        void* pw = address(ws, "workspace", at::kByte, dev);
        void* stream = current_stream(dev);
        const int w = size32(pool.size(-1));
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = compact_fn(pool.data_ptr(), pool.size(0), w, ki, indices.numel(), to, pl, pw,
                            ws.numel(), stream);
        Py_END_ALLOW_THREADS
        check(status, "mla_cache_compact");
        return pair(output(v[2], out), output(v[3], live));
    });
}

#define MLA_METHOD(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MLA_METHOD(bind),       MLA_METHOD(prefix_decode), MLA_METHOD(cache_append),
                         MLA_METHOD(cache_fork), MLA_METHOD(cache_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "mla_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mla_binding() { return PyModule_Create(&module); }
