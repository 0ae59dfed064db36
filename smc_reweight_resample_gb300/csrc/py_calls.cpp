// py_calls.cpp -- argument marshalling of the calls around the verify, as a CPython module over the C ABI of
// libsmcsd.so: the tensors' checks, the missing outputs and the call itself in one step, because a small call's
// time is its issue (on the Grace CPU the same marshalling through ctypes takes 15 to 25 us, here about 4).
// The module holds no code of the operators: `bind` is given the addresses of the library's entry points, and the
// functions here return what the entry points write. Wrong types raise TypeError, wrong shapes and devices
// ValueError, and a status other than SMCSD_OK calls the error function that `bind` was given.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/TensorOptions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

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
decltype(&kv_pagetable_remap) f_remap;
decltype(&beam_select) f_beam;
decltype(&state_reorder) f_reorder;
decltype(&kv_fork) f_fork;
decltype(&kv_free) f_free;
decltype(&kv_compact) f_compact;
decltype(&kv_copy_pages) f_copy;
decltype(&distill_loss) f_distill;
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
    void skip() { ++i_; }
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

// A new tensor, without the dispatcher where it lies on the GPU (a third of a small call's time is its outputs).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    if (!like.is_cuda()) return at::empty(shape, like.options().dtype(type));
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// New tensors of one call in one allocation, where together they are small: of a small call's 4 to 6 us each allocation is half of one.
class Together {
  public:
    // for `n` tensors of `words` 4-byte elements in all
    Together(const at::Tensor& like, int n, int64_t words) : like_(like), room_(4 * words + n * kAlign) {}
    at::Tensor take(at::IntArrayRef shape, at::ScalarType type) {
        if (room_ > kMost || !like_.is_cuda()) return fresh(shape, type, like_);
        if (!all_.defined()) all_ = fresh({room_}, at::kByte, like_);
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all_.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                c10::scalarTypeToTypeMeta(type));
        const int64_t each = (int64_t)c10::elementSize(type);
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        t.unsafeGetTensorImpl()->set_storage_offset(used_ / each);
        used_ += (t.numel() * each + kAlign - 1) / kAlign * kAlign;
        if (used_ > room_) value_error("outputs larger than their memory");
        return t;
    }

  private:
    static constexpr int64_t kAlign = 256, kMost = 64 << 10;
    const at::Tensor& like_;
    int64_t room_, used_ = 0;
    at::Tensor all_;
};

// An output: the given tensor, or a new one.
at::Tensor output(const at::Tensor* t, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, Together* with = nullptr) {
    if (!t) return with ? with->take(shape, type) : fresh(shape, type, like);
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
        Args a(args, n, 14);
        f_slot_map = reinterpret_cast<decltype(f_slot_map)>((uintptr_t)a.integer());
        f_append = reinterpret_cast<decltype(f_append)>((uintptr_t)a.integer());
        f_tree_mask = reinterpret_cast<decltype(f_tree_mask)>((uintptr_t)a.integer());
        f_attention = reinterpret_cast<decltype(f_attention)>((uintptr_t)a.integer());
        f_logits = reinterpret_cast<decltype(f_logits)>((uintptr_t)a.integer());
        f_remap = reinterpret_cast<decltype(f_remap)>((uintptr_t)a.integer());
        f_beam = reinterpret_cast<decltype(f_beam)>((uintptr_t)a.integer());
        f_reorder = reinterpret_cast<decltype(f_reorder)>((uintptr_t)a.integer());
        f_fork = reinterpret_cast<decltype(f_fork)>((uintptr_t)a.integer());
        f_free = reinterpret_cast<decltype(f_free)>((uintptr_t)a.integer());
        f_compact = reinterpret_cast<decltype(f_compact)>((uintptr_t)a.integer());
        f_copy = reinterpret_cast<decltype(f_copy)>((uintptr_t)a.integer());
        f_distill = reinterpret_cast<decltype(f_distill)>((uintptr_t)a.integer());
        Py_XDECREF(f_error);
        f_error = Py_NewRef(args[13]);
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

// Rows of at least V elements, each contiguous: elements from one row to the next.
int64_t matrix_stride(const at::Tensor& t, int64_t V, const char* what) {
    if (t.dim() != 2 || t.size(1) < V || (t.size(1) > 1 && t.stride(1) != 1)) value_error(std::string(what) + " must be rows of V");
    // rows that share memory, or a step that is never taken
    if (t.size(0) > 1 && t.stride(0) < V) value_error(std::string(what) + " must be rows of V");
    return t.size(0) > 1 ? t.stride(0) : V;
}

// The tensors of a list or tuple.
std::vector<const at::Tensor*> tensors_of(PyObject* o, size_t most, const char* what) {
    if (!PyList_Check(o) && !PyTuple_Check(o)) type_error(std::string(what) + " must be a list of tensors");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(o);
    if (n < 1 || (size_t)n > most) value_error(std::string(what) + " must be 1 to " + std::to_string(most) + " tensors");
    std::vector<const at::Tensor*> got;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* t = PySequence_Fast_GET_ITEM(o, i);
        if (!THPVariable_Check(t)) type_error("expected a tensor");
        got.push_back(&THPVariable_Unpack(t));
    }
    return got;
}
constexpr size_t kMostStates = 64, kMostCaches = 256;

// beam_select(logits, G, N, V, M, temperature, scores, finished, pad, eos, tokens, ancestors, out_scores, out_finished, ws, bytes)
PyObject* py_beam(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 16);
        const at::Tensor& z = a.some();
        const int G = a.size(), N = a.size(), V = a.size(), M = a.size();
        const double temperature = a.real();
        const at::Tensor *scores = a.tensor(), *finished = a.tensor();
        const int pad = a.size(), eos = a.size();
        if (G <= 0 || N <= 0 || V <= 0 || M <= 0) value_error("sizes must be positive");
        const int64_t stride = matrix_stride(z, V, "logits"), rows = (int64_t)G * N;
        if (z.size(0) != rows) value_error("logits must have G * N rows");
        at_least(scores, rows, "scores");
        at_least(finished, rows, "finished");
        const int dtype = dtype_code(z);
        if (!z.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(z.device());
        const int64_t out = (int64_t)G * M;
        Together made(z, 4, 4 * out);
        const at::Tensor tokens = output(a.tensor(), {out}, at::kInt, z, &made), ancestors = output(a.tensor(), {out}, at::kInt, z, &made);
        const at::Tensor out_scores = output(a.tensor(), {out}, at::kFloat, z, &made), over = output(a.tensor(), {out}, at::kInt, z, &made);
        one_device(z, {scores, finished, &tokens, &ancestors, &out_scores, &over});
        const Tail t(a, z);
        check(f_beam(z.data_ptr(), stride, dtype, G, N, V, M, (float)temperature, f32(scores), i32(finished), pad, eos, i32(&tokens),
                     i32(&ancestors), f32(&out_scores), i32(&over), t.ws, t.bytes, t.stream),
              "beam_select");
        return tuple({tokens, ancestors, out_scores, over});
    });
}

// state_reorder(states, ancestors, G, N, M, out, ws, bytes)
PyObject* py_reorder(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n < 1) type_error("wrong number of arguments");
        Args a(args + 1, n - 1, 7);
        const std::vector<const at::Tensor*> src = tensors_of(args[0], kMostStates, "states");
        const at::Tensor& ancestors = a.some();
        const int G = a.size(), N = a.size(), M = a.size();
        if (G <= 0 || N <= 0 || M <= 0) value_error("sizes must be positive");
        const int64_t rows = (int64_t)G * N, rows_out = (int64_t)G * M;
        at_least(&ancestors, rows_out, "ancestors");
        if (!ancestors.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(ancestors.device());
        std::vector<const at::Tensor*> given;
        if (!a.none()) given = tensors_of(args[5], kMostStates, "out"), a.skip();
        if (!given.empty() && given.size() != src.size()) value_error("out must have a tensor for each state");
        std::vector<at::Tensor> dst;
        int64_t words = 0;
        for (const at::Tensor* t : src) words += ((int64_t)t->nbytes() / rows * rows_out + 3) / 4;
        Together made(ancestors, (int)src.size(), words);
        const void* from[kMostStates];
        void* to[kMostStates];
        long long bytes[kMostStates];
        for (size_t i = 0; i < src.size(); ++i) {
            const at::Tensor& t = *src[i];
            if (!t.is_cuda() || t.device() != ancestors.device()) value_error("tensors must be on one device");
            if (t.dim() < 1 || t.size(0) != rows || t.numel() == 0) value_error("states must have G * N rows");
            if (!t.is_contiguous()) value_error("tensor must be contiguous");
            std::vector<int64_t> shape = t.sizes().vec();
            shape[0] = rows_out;
            if (given.empty()) {
                dst.push_back(made.take(shape, t.scalar_type()));
            } else {
                const at::Tensor& o = *given[i];
                if (o.device() != t.device()) value_error("tensors must be on one device");
                if (o.scalar_type() != t.scalar_type()) type_error("out must have the states' types");
                if (!o.sizes().equals(shape)) value_error("out must have the states' shapes, with G * M rows");
                if (!o.is_contiguous()) value_error("tensor must be contiguous");
                dst.push_back(o);
            }
            from[i] = t.data_ptr();
            to[i] = dst.back().data_ptr();
            bytes[i] = (long long)(t.numel() / rows) * t.element_size();
        }
        const Tail t(a, ancestors);
        check(f_reorder(from, to, bytes, (int)src.size(), i32(&ancestors), G, N, M, t.ws, t.bytes, t.stream), "state_reorder");
        PyObject* list = PyList_New((Py_ssize_t)dst.size());
        if (!list) throw Raised{};
        for (size_t i = 0; i < dst.size(); ++i) {
            PyObject* o = THPVariable_Wrap(dst[i]);
            if (!o) {
                Py_DECREF(list);
                throw Raised{};
            }
            PyList_SET_ITEM(list, (Py_ssize_t)i, o);
        }
        return list;
    });
}

// kv_pagetable_remap(ancestors, resampled, G, N, table_in, pages_per_seq, num_pages, table_out, refcount, with_refcount, ws, bytes)
PyObject* py_remap(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 12);
        const at::Tensor& ancestors = a.some();
        const at::Tensor* resampled = a.tensor();
        const int G = a.size(), N = a.size();
        const at::Tensor& table = a.some();
        const int pages_per_seq = a.size(), num_pages = a.size();
        const at::Tensor *table_in_out = a.tensor(), *refcount = a.tensor();
        const bool with_refcount = a.integer() != 0;
        for (const at::Tensor* t : {&ancestors, resampled, &table, table_in_out, refcount})
            if (t && t->scalar_type() != at::kInt) type_error(std::string("tensor must be Int, not ") + c10::toString(t->scalar_type()));
        if (G > 0 && N > 0 && pages_per_seq > 0) {  // others are refused by the call
            const int64_t rows = (int64_t)G * N;
            at_least(&ancestors, rows, "ancestors");
            at_least(resampled, G, "resampled");
            for (const at::Tensor* t : {&table, table_in_out}) {
                if (t && (__int128)rows * pages_per_seq > t->numel()) value_error("a table is too small");
                if (rows > 1) rows_of(t, rows, pages_per_seq, "a table");  // of one row the rest is not looked at
            }
        }
        at_least(refcount, num_pages, "refcount");
        if (!table.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(table.device());
        Together made(table, 2, table.numel() + (with_refcount && num_pages > 0 ? num_pages : 0));
        const at::Tensor table_out = table_in_out ? *table_in_out : made.take(table.sizes(), at::kInt);
        at::Tensor ref;
        if (refcount)
            ref = *refcount;
        else if (with_refcount)
            ref = made.take({num_pages}, at::kInt);
        one_device(table, {&ancestors, resampled, &table_out, ref.defined() ? &ref : nullptr});
        const Tail t(a, table);
        check(f_remap(i32(&ancestors), i32(resampled), G, N, i32(&table), i32(&table_out), pages_per_seq, ref.defined() ? i32(&ref) : nullptr,
                      num_pages, t.ws, t.bytes, t.stream),
              "kv_pagetable_remap");
        return tuple({table_out, ref});
    });
}

// kv_fork(table_in, refcount_in, parents, page_size, lengths, table_out, refcount_out, ws, bytes)
PyObject* py_fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 9);
        const at::Tensor &table = a.some(), &ref = a.some(), &parents = a.some();
        const int page = a.size();
        const at::Tensor* lengths = a.tensor();
        if (table.dim() != 2) value_error("table_in must be [S, pages_per_seq]");
        const int S = dim(table.size(0)), pages = dim(ref.numel());
        at_least(&parents, S, "parents");
        at_least(lengths, S, "lengths");
        if (!table.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(table.device());
        Together made(table, 2, table.numel() + pages);
        const at::Tensor table_out = output(a.tensor(), table.sizes(), at::kInt, table, &made);
        const at::Tensor ref_out = output(a.tensor(), {pages}, at::kInt, table, &made);
        one_device(table, {&ref, &parents, lengths, &table_out, &ref_out});
        const Tail t(a, table);
        check(f_fork(i32(&parents), i32(lengths), S, i32(&table), i32(&table_out), dim(table.size(1)), page, i32(&ref), i32(&ref_out), pages,
                     t.ws, t.bytes, t.stream),
              "kv_fork");
        return tuple({table_out, ref_out});
    });
}

// kv_free(table_in, refcount_in, lengths, page_size, table_out, refcount_out, ws, bytes)
PyObject* py_free(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 8);
        const at::Tensor &table = a.some(), &ref = a.some(), &lengths = a.some();
        const int page = a.size();
        if (table.dim() != 2) value_error("table_in must be [S, pages_per_seq]");
        const int S = dim(table.size(0)), pages = dim(ref.numel());
        at_least(&lengths, S, "lengths");
        if (!table.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(table.device());
        Together made(table, 2, table.numel() + pages);
        const at::Tensor table_out = output(a.tensor(), table.sizes(), at::kInt, table, &made);
        const at::Tensor ref_out = output(a.tensor(), {pages}, at::kInt, table, &made);
        one_device(table, {&ref, &lengths, &table_out, &ref_out});
        const Tail t(a, table);
        check(f_free(i32(&lengths), S, i32(&table), i32(&table_out), dim(table.size(1)), page, i32(&ref), i32(&ref_out), pages, t.ws, t.bytes,
                     t.stream),
              "kv_free");
        return tuple({table_out, ref_out});
    });
}

// kv_compact(table_in, refcount_in, table_out, refcount_out, src, dst, counts, ws, bytes)
PyObject* py_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 9);
        const at::Tensor &table = a.some(), &ref = a.some();
        if (table.dim() != 2) value_error("table_in must be [S, pages_per_seq]");
        const int S = dim(table.size(0)), pages = dim(ref.numel());
        if (!table.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(table.device());
        Together made(table, 5, table.numel() + 2 * (int64_t)pages + 2);
        const at::Tensor table_out = output(a.tensor(), table.sizes(), at::kInt, table, &made);
        const at::Tensor ref_out = output(a.tensor(), {pages}, at::kInt, table, &made);
        const at::Tensor src = output(a.tensor(), {pages / 2}, at::kInt, table, &made), dst = output(a.tensor(), {pages / 2}, at::kInt, table, &made);
        const at::Tensor counts = output(a.tensor(), {2}, at::kInt, table, &made);
        one_device(table, {&ref, &table_out, &ref_out, &src, &dst, &counts});
        const Tail t(a, table);
        check(f_compact(S, i32(&table), i32(&table_out), dim(table.size(1)), i32(&ref), i32(&ref_out), pages, i32(&src), i32(&dst),
                        i32(&counts), t.ws, t.bytes, t.stream),
              "kv_compact");
        return tuple({table_out, ref_out, src, dst, counts});
    });
}

// kv_copy_pages(caches, src, dst, count, ws, bytes)
PyObject* py_copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n < 1) type_error("wrong number of arguments");
        Args a(args + 1, n - 1, 5);
        const std::vector<const at::Tensor*> caches = tensors_of(args[0], kMostCaches, "caches");
        const at::Tensor &src = a.some(), &dst = a.some();
        const at::Tensor* count = a.tensor();
        const int moves = dim(src.numel());
        if (dst.numel() != moves) value_error("src and dst must be alike");
        at_least(count, 1, "count");
        const at::Tensor& like = *caches[0];
        if (!like.is_cuda()) value_error("tensor must be on the CUDA device");
        if (like.dim() < 1 || like.numel() == 0) value_error("caches must be [num_pages, ...]");
        const c10::cuda::CUDAGuard guard(like.device());
        void* at_[kMostCaches];
        for (size_t i = 0; i < caches.size(); ++i) {
            const at::Tensor& c = *caches[i];
            if (c.scalar_type() != like.scalar_type()) type_error("caches must have one type");
            if (!c.sizes().equals(like.sizes())) value_error("caches must be alike");
            if (!c.is_contiguous()) value_error("tensor must be contiguous");
            one_device(like, {&c});
            at_[i] = c.data_ptr();
        }
        one_device(like, {&src, &dst, count});
        const Tail t(a, like);
        if (moves == 0) Py_RETURN_NONE;
        check(f_copy(at_, (int)caches.size(), (long long)(like.numel() / like.size(0)) * like.element_size(), dim(like.size(0)), i32(&src),
                     i32(&dst), moves, i32(count), t.ws, t.bytes, t.stream),
              "kv_copy_pages");
        Py_RETURN_NONE;
    });
}

// distill_loss(logits, top_tokens, top_values, V, temperature, rest, weight, loss, dlogits, grad, with_loss, ws, bytes)
PyObject* py_distill(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n, 13);
        const at::Tensor &z = a.some(), &tokens = a.some(), &values = a.some();
        const int V = a.size();
        const double temperature = a.real();
        const bool rest = a.integer() != 0;
        const at::Tensor* weight = a.tensor();
        if (V <= 0) value_error("V must be positive");
        const int64_t stride = matrix_stride(z, V, "logits");
        const int R = dim(z.size(0)), dtype = dtype_code(z);
        if (tokens.dim() != 2 || tokens.size(0) != R || !tokens.sizes().equals(values.sizes()))
            value_error("top_tokens and top_values must be [R, K]");
        at_least(weight, R, "weight");
        if (!z.is_cuda()) value_error("tensor must be on the CUDA device");
        const c10::cuda::CUDAGuard guard(z.device());
        const at::Tensor *loss_in = a.tensor(), *grad_in = a.tensor();
        at::Tensor loss, grad;
        const bool want_grad = a.integer() || grad_in;
        if (a.integer() || loss_in) loss = output(loss_in, {R}, at::kFloat, z);
        int64_t grad_stride = 0;
        if (want_grad) {
            grad = grad_in ? *grad_in : fresh({R, V}, z.scalar_type(), z);
            grad_stride = matrix_stride(grad, V, "dlogits");
            if (grad.size(0) != R) value_error("dlogits must have the logits' rows");
            if (grad.scalar_type() != z.scalar_type()) type_error("dlogits must have the logits' type");
            if (R == 1 && grad.data_ptr() == z.data_ptr()) grad_stride = stride;
        }
        one_device(z, {&tokens, &values, weight, loss.defined() ? &loss : nullptr, grad.defined() ? &grad : nullptr});
        const Tail t(a, z);
        check(f_distill(z.data_ptr(), stride, dtype, R, V, i32(&tokens), f32(&values), dim(tokens.size(1)), (float)temperature, rest,
                        f32(weight), loss.defined() ? f32(&loss) : nullptr, grad.defined() ? grad.data_ptr() : nullptr, grad_stride, t.ws,
                        t.bytes, t.stream),
              "distill_loss");
        return tuple({loss, grad});
    });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, nullptr},
    {"kv_slot_map", (PyCFunction)(void (*)(void))py_slot_map, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, nullptr},
    {"tree_mask", (PyCFunction)(void (*)(void))py_tree_mask, METH_FASTCALL, nullptr},
    {"tree_attention", (PyCFunction)(void (*)(void))py_attention, METH_FASTCALL, nullptr},
    {"logits_process", (PyCFunction)(void (*)(void))py_logits, METH_FASTCALL, nullptr},
    {"kv_pagetable_remap", (PyCFunction)(void (*)(void))py_remap, METH_FASTCALL, nullptr},
    {"beam_select", (PyCFunction)(void (*)(void))py_beam, METH_FASTCALL, nullptr},
    {"state_reorder", (PyCFunction)(void (*)(void))py_reorder, METH_FASTCALL, nullptr},
    {"kv_fork", (PyCFunction)(void (*)(void))py_fork, METH_FASTCALL, nullptr},
    {"kv_free", (PyCFunction)(void (*)(void))py_free, METH_FASTCALL, nullptr},
    {"kv_compact", (PyCFunction)(void (*)(void))py_compact, METH_FASTCALL, nullptr},
    {"kv_copy_pages", (PyCFunction)(void (*)(void))py_copy, METH_FASTCALL, nullptr},
    {"distill_loss", (PyCFunction)(void (*)(void))py_distill, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", "The calls around the verify over the C ABI.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
