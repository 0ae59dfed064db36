// py_calls.cpp -- argument marshalling of the calls around the verify, as a CPython module over the C ABI of
// libsmcsd.so: the tensors' checks, the missing outputs and the call itself in one step, because a small call's
// time is its issue (on the Grace CPU the same marshalling through ctypes takes 15 to 25 us, here about 4).
// The module holds no code of the operators: `bind` is given the addresses of the library's entry points, and the
// functions here return what the entry points write. Wrong types raise TypeError, wrong shapes and devices
// ValueError, and a status other than SMCSD_OK calls the error function that `bind` was given.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/TensorOptions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "smcsd.h"

namespace {

struct Refused {
    PyObject* type;
    std::string what;
};
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
struct Raised {};  // a Python exception is set

decltype(&kv_slot_map) f_slot_map;
decltype(&kv_append) f_append;
decltype(&tree_mask) f_tree_mask;
decltype(&tree_attention) f_attention;
decltype(&logits_process) f_logits;
PyObject* f_error;  // error(status, where) raises

// One call's positional arguments.
class Args {
   public:
    Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
        if (n != want) type_error("wrong number of arguments");
    }
    const at::Tensor* tensor() {
        PyObject* o = a_[i_++];
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) type_error("expected a tensor");
        return &THPVariable_Unpack(o);
    }
    const at::Tensor& some() {
        const at::Tensor* t = tensor();
        if (!t) type_error("expected a tensor, not None");
        return *t;
    }
    long long integer() {
        const long long v = PyLong_AsLongLong(a_[i_++]);
        if (v == -1 && PyErr_Occurred()) throw Raised{};
        return v;
    }
    int size() {
        const long long v = integer();
        if (v < INT32_MIN || v > INT32_MAX) value_error("size out of range");
        return (int)v;
    }
    double real() {
        const double v = PyFloat_AsDouble(a_[i_++]);
        if (v == -1.0 && PyErr_Occurred()) throw Raised{};
        return v;
    }
    bool none() {
        if (a_[i_] != Py_None) return false;
        ++i_;
        return true;
    }

   private:
    PyObject* const* a_;
    Py_ssize_t i_ = 0;
};

// Address of a contiguous CUDA tensor of one type, or null.
void* address(const at::Tensor* t, at::ScalarType type) {
    if (!t) return nullptr;
    if (t->scalar_type() != type)
        type_error(std::string("tensor must be ") + c10::toString(type) + ", not " + c10::toString(t->scalar_type()));
    if (!t->is_cuda()) value_error("tensor must be on the CUDA device");
    if (!t->is_contiguous()) value_error("tensor must be contiguous");
    return t->data_ptr();
}
int32_t* i32(const at::Tensor* t) { return static_cast<int32_t*>(address(t, at::kInt)); }
float* f32(const at::Tensor* t) { return static_cast<float*>(address(t, at::kFloat)); }

void at_least(const at::Tensor* t, int64_t n, const char* what) {
    if (t && t->numel() < n) value_error(std::string(what) + " is too small");
}

// n rows of `row` elements, one behind the other: a flat tensor, or one whose inner dimensions make up a row (of rows longer
// than the call takes them for, all but the first would be met at the wrong place).
void rows_of(const at::Tensor* t, int64_t n, int64_t row, const char* what) {
    if (!t) return;
    at_least(t, n * row, what);
    if (t->dim() < 2 || t->numel() == row) return;
    int64_t inner = 1;
    for (int64_t k = t->dim() - 1; k > 0; --k)
        if ((inner *= t->size(k)) == row) return;
    value_error(std::string(what) + " has rows of another size");
}

// An output: the given tensor, or a new one.
at::Tensor output(const at::Tensor* t, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (!t) return at::empty(shape, like.options().dtype(type));
    int64_t row = 1;
    for (size_t i = 1; i < shape.size(); ++i) row *= shape[i];
    if (shape.size() > 1)
        rows_of(t, shape[0], row, "an output");
    else
        at_least(t, shape[0], "an output");
    return *t;
}

// Whatever is given of these is where `like` is.
void one_device(const at::Tensor& like, std::initializer_list<const at::Tensor*> list) {
    for (const at::Tensor* t : list)
        if (t && t->device() != like.device()) value_error("tensors must be on one device");
}

int dtype_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kFloat) return SMCSD_F32;
    if (t.scalar_type() == at::kBFloat16) return SMCSD_BF16;
    type_error(std::string("tensor must be float32 or bfloat16, not ") + c10::toString(t.scalar_type()));
}

// A [rows, heads, D] tensor whose rows are contiguous: elements from one row to the next.
int64_t row_stride(const at::Tensor& t) {
    if (t.dim() != 3 || !t.is_cuda()) value_error("tensor must be [rows, heads, D] on the CUDA device");
    // the stride of a dimension of one is never used and may be anything
    if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
        value_error("the heads of a row must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

void check_caches(const at::Tensor& k, const at::Tensor& v, const at::Tensor& like) {
    if (k.dim() != 4 || !k.sizes().equals(v.sizes())) value_error("caches must be [num_pages, Hkv, page_size, D], both alike");
    if (k.scalar_type() != like.scalar_type() || v.scalar_type() != like.scalar_type())
        type_error("caches and rows must have one type");
}

int dim(int64_t n) {
    if (n > INT32_MAX) value_error("size out of range");
    return (int)n;
}

// The last two arguments of every call, workspace address and size, and the current stream.
struct Tail {
    void* ws;
    size_t bytes;
    void* stream;
    Tail(Args& a, const at::Tensor& like) {
        ws = reinterpret_cast<void*>((uintptr_t)a.integer());
        bytes = (size_t)a.integer();
        if (!like.is_cuda()) value_error("tensor must be on the CUDA device");
        stream = (void*)c10::cuda::getCurrentCUDAStream(like.get_device()).stream();
    }
};

void check(int status, const char* where) {
    if (status == SMCSD_OK) return;
    PyObject* r = PyObject_CallFunction(f_error, "is", status, where);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, status);
    throw Raised{};
}

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* tuple(std::initializer_list<at::Tensor> list) {
    PyObject* t = PyTuple_New((Py_ssize_t)list.size());
    if (!t) throw Raised{};
    Py_ssize_t i = 0;
    for (const at::Tensor& x : list) {
        PyObject* o = x.defined() ? THPVariable_Wrap(x) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(t);
            throw Raised{};
        }
        PyTuple_SET_ITEM(t, i++, o);
    }
    return t;
}

PyObject* py_bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 6);
        f_slot_map = reinterpret_cast<decltype(f_slot_map)>((uintptr_t)a.integer());
        f_append = reinterpret_cast<decltype(f_append)>((uintptr_t)a.integer());
        f_tree_mask = reinterpret_cast<decltype(f_tree_mask)>((uintptr_t)a.integer());
        f_attention = reinterpret_cast<decltype(f_attention)>((uintptr_t)a.integer());
        f_logits = reinterpret_cast<decltype(f_logits)>((uintptr_t)a.integer());
        Py_XDECREF(f_error);
        f_error = Py_NewRef(args[5]);
        Py_RETURN_NONE;
    });
}

// kv_slot_map(ctx_len, table_in, refcount_in, S, T, page_size, new_offsets, rows, table_out, refcount_out, slots,
//             copy_src, copy_dst, ws, bytes)
PyObject* py_slot_map(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 15);
        const at::Tensor &ctx = a.some(), &table = a.some(), &ref = a.some();
        const int S = a.size(), T = a.size(), page = a.size();
        const at::Tensor* off = a.tensor();
        const bool fixed = a.none();
        const int R = fixed ? dim((int64_t)S * T) : a.size();
        if (off && fixed) value_error("ragged tokens need rows");
        if (table.dim() != 2 || table.size(0) != S) value_error("table_in must be [S, pages_per_seq]");
        at_least(&ctx, S, "ctx_len");
        at_least(off, (int64_t)S + 1, "new_offsets");
        const int pages = dim(ref.numel());
        if (!table.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(table.device());
        const at::Tensor table_out = output(a.tensor(), table.sizes(), at::kInt, table);
        const at::Tensor ref_out = output(a.tensor(), {pages}, at::kInt, table);
        const at::Tensor slots = output(a.tensor(), {R}, at::kLong, table);
        const at::Tensor src = output(a.tensor(), {S}, at::kInt, table);
        const at::Tensor dst = output(a.tensor(), {S}, at::kInt, table);
        one_device(table, {&ctx, &ref, off, &table_out, &ref_out, &slots, &src, &dst});
        const Tail t(a, table);
        check(f_slot_map(i32(&ctx), i32(off), S, T, R, i32(&table), i32(&table_out), dim(table.size(1)), page, i32(&ref), i32(&ref_out),
                         pages, static_cast<int64_t*>(address(&slots, at::kLong)), i32(&src), i32(&dst), t.ws, t.bytes, t.stream),
              "kv_slot_map");
        return tuple({table_out, ref_out, slots, src, dst});
    });
}

// kv_append(k_new, v_new, slots, k_cache, v_cache, ctx_len, copy_src, copy_dst, ws, bytes)
PyObject* py_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 10);
        const at::Tensor &k = a.some(), &v = a.some(), &slots = a.some(), &kc = a.some(), &vc = a.some();
        const at::Tensor *ctx = a.tensor(), *src = a.tensor(), *dst = a.tensor();
        check_caches(kc, vc, k);
        const int64_t stride = row_stride(k);
        if (v.scalar_type() != k.scalar_type() || !v.sizes().equals(k.sizes()) || row_stride(v) != stride)
            value_error("keys and values must be alike");
        if (k.size(1) != kc.size(1) || k.size(2) != kc.size(3)) value_error("rows and caches must have the same heads");
        at_least(&slots, k.size(0), "slots");
        const int S = src ? dim(src->numel()) : 0;
        at_least(dst, S, "copy_dst");
        at_least(ctx, S, "ctx_len");
        one_device(kc, {&k, &v, &slots, &vc, ctx, src, dst});
        const Tail t(a, kc);
        const c10::cuda::CUDAGuard guard(kc.device());
        check(f_append(k.data_ptr(), v.data_ptr(), dtype_code(k), dim(k.size(0)), dim(kc.size(1)), dim(kc.size(3)), stride,
                       static_cast<int64_t*>(address(&slots, at::kLong)), i32(src), i32(dst), S ? i32(ctx) : nullptr, S,
                       address(&kc, k.scalar_type()), address(&vc, k.scalar_type()), dim(kc.size(2)), dim(kc.size(0)), t.ws, t.bytes,
                       t.stream),
              "kv_append");
        Py_RETURN_NONE;
    });
}

// tree_mask(parents, S, T, node_offsets, mask, ws, bytes)
PyObject* py_tree_mask(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 7);
        const at::Tensor& parents = a.some();
        const int S = a.size(), T = a.size(), R = dim(parents.numel());
        const at::Tensor* off = a.tensor();
        at_least(off, (int64_t)S + 1, "node_offsets");
        if (!parents.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(parents.device());
        const at::Tensor mask = output(a.tensor(), {R, ((int64_t)T + 31) / 32}, at::kInt, parents);
        one_device(parents, {off, &mask});
        const Tail t(a, parents);
        check(f_tree_mask(i32(&parents), i32(off), S, T, R, reinterpret_cast<uint32_t*>(i32(&mask)), t.ws, t.bytes, t.stream), "tree_mask");
        return THPVariable_Wrap(mask);
    });
}

// tree_attention(q, k_cache, v_cache, table, ctx_len, S, T, scale, N, node_offsets, mask, out, lse, with_lse, ws,
//                bytes)
PyObject* py_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 16);
        const at::Tensor &q = a.some(), &kc = a.some(), &vc = a.some(), &table = a.some(), &ctx = a.some();
        const int S = a.size(), T = a.size();
        const double scale = a.real();
        const int N = a.size();
        const at::Tensor *off = a.tensor(), *mask = a.tensor();
        check_caches(kc, vc, q);
        const int64_t stride = row_stride(q);
        const int R = dim(q.size(0)), Hq = dim(q.size(1)), D = dim(kc.size(3));
        if (q.size(2) != D) value_error("rows and caches must have the same head size");
        if (table.dim() != 2 || table.size(0) != S) value_error("table must be [S, pages_per_seq]");
        at_least(&ctx, S, "ctx_len");
        at_least(off, (int64_t)S + 1, "node_offsets");
        rows_of(mask, R, ((int64_t)T + 31) / 32, "mask");
        const c10::cuda::CUDAGuard guard(q.device());
        const at::Tensor out = output(a.tensor(), {R, Hq, D}, q.scalar_type(), q);
        const at::Tensor* lse_in = a.tensor();
        at::Tensor lse;
        if (a.integer() || lse_in) lse = output(lse_in, {R, Hq}, at::kFloat, q);
        one_device(q, {&kc, &vc, &table, &ctx, off, mask, &out, lse_in});
        const Tail t(a, q);
        const at::ScalarType type = q.scalar_type();
        check(f_attention(q.data_ptr(), stride, address(&kc, type), address(&vc, type), dtype_code(q), dim(kc.size(0)), dim(kc.size(2)),
                          i32(&table), dim(table.size(1)), i32(&ctx), i32(off), S, N, T, R, reinterpret_cast<const uint32_t*>(i32(mask)),
                          Hq, dim(kc.size(1)), D, (float)scale, address(&out, type), lse.defined() ? f32(&lse) : nullptr, t.ws, t.bytes,
                          t.stream),
              "tree_attention");
        return tuple({out, lse});
    });
}

// logits_process(logits, S, T, V, node_offsets, node_tokens, mask, hist_tokens, hist_offsets, repetition, presence,
//                frequency, bias_tokens, bias_values, bias_offsets, allowed, out, ws, bytes)
PyObject* py_logits(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 19);
        const at::Tensor& z = a.some();
        const int S = a.size(), T = a.size(), V = a.size();
        if (V <= 0) value_error("V must be positive");
        const int R = dim(z.numel() / V);
        const at::Tensor *off = a.tensor(), *tokens = a.tensor(), *mask = a.tensor(), *ht = a.tensor(), *ho = a.tensor();
        const at::Tensor *rep = a.tensor(), *pres = a.tensor(), *freq = a.tensor();
        const at::Tensor *bt = a.tensor(), *bv = a.tensor(), *bo = a.tensor(), *allowed = a.tensor();
        at_least(off, (int64_t)S + 1, "node_offsets");
        at_least(tokens, R, "node_tokens");
        rows_of(mask, R, ((int64_t)T + 31) / 32, "mask");
        at_least(ho, (int64_t)S + 1, "hist_offsets");
        at_least(bo, (int64_t)S + 1, "bias_offsets");
        rows_of(allowed, R, ((int64_t)V + 31) / 32, "allowed");
        for (const at::Tensor* t : {rep, pres, freq}) at_least(t, S, "a penalty");
        if (bt) at_least(bv, bt->numel(), "bias_values");
        if (!z.is_cuda()) value_error("tensor must be on the CUDA device");
        rows_of(&z, R, V, "logits");
        if (z.numel() != (int64_t)R * V) value_error("logits must be rows of V");
        const c10::cuda::CUDAGuard guard(z.device());
        const at::Tensor out = output(a.tensor(), {R, V}, z.scalar_type(), z);
        one_device(z, {off, tokens, mask, ht, ho, rep, pres, freq, bt, bv, bo, allowed, &out});
        const Tail t(a, z);
        const at::ScalarType type = z.scalar_type();
        check(f_logits(address(&z, type), address(&out, type), dtype_code(z), R, V, S, T, i32(off), i32(tokens),
                       reinterpret_cast<const uint32_t*>(i32(mask)), i32(ht), i32(ho), ht ? dim(ht->numel()) : 0, f32(rep), f32(pres),
                       f32(freq), i32(bt), f32(bv), i32(bo), bt ? dim(bt->numel()) : 0, reinterpret_cast<const uint32_t*>(i32(allowed)),
                       t.ws, t.bytes, t.stream),
              "logits_process");
        return THPVariable_Wrap(out);
    });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, nullptr},
    {"kv_slot_map", (PyCFunction)(void (*)(void))py_slot_map, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, nullptr},
    {"tree_mask", (PyCFunction)(void (*)(void))py_tree_mask, METH_FASTCALL, nullptr},
    {"tree_attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, nullptr},
    {"logits_process", (PyCFunction)(void (*)(void))py_logits, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "The calls around the verify over the C ABI.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
