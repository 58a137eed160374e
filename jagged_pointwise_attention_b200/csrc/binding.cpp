// binding.cpp -- Python calls of the serving entry points (include/hstu.h).
//
// A serving step makes several of these calls for a few microseconds of GPU
// work each, so their own cost counts: through ctypes, with the checks in
// Python, a call took 13 to 25 us of host time. Here tensors are unpacked,
// checked and allocated in C++, and the call goes straight to the library. The
// library's functions come as addresses from the one loaded libhstu.so
// (bind()), so nothing is linked twice. No C++ exception leaves a function:
// each becomes a Python one.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "hstu.h"

namespace {

struct Refusal {                // becomes a Python exception of this type
    PyObject* type;
    std::string what;
};

[[noreturn]] void value_error(std::string s) { throw Refusal{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void type_error(std::string s) { throw Refusal{PyExc_TypeError, std::move(s)}; }
struct PythonError {};          // a Python exception is set already

struct Api {
    decltype(&hstu_cache_plan) plan;
    decltype(&hstu_cache_append) append;
    decltype(&hstu_attn_cached_workspace_bytes) attn_bytes;
    decltype(&hstu_attn_cached_fwd) attn;
    decltype(&hstu_quant_groups_w4) quant;
    decltype(&hstu_linear_w4_fwd) linear;
} api;
PyObject* check_fn = nullptr;   // check(name, status) raises

void check(const char* name, hstu_status_t st) {
    if (st == HSTU_OK) return;
    PyObject* r = PyObject_CallFunction(check_fn, "si", name, static_cast<int>(st));
    Py_XDECREF(r);
    if (r == nullptr) throw PythonError{};
    throw Refusal{PyExc_RuntimeError, std::string(name) + " failed"};
}

// Arguments of one call: tensors must be on the current device.
class Args {
  public:
    Args(PyObject* const* v, Py_ssize_t n, Py_ssize_t want) : v_(v) {
        if (n != want) type_error("wrong number of arguments");
    }

    const at::Tensor* maybe(int i, const char* what) {
        if (v_[i] == Py_None) return nullptr;
        if (!THPVariable_Check(v_[i])) type_error(std::string(what) + " must be a tensor");
        const at::Tensor& t = THPVariable_Unpack(v_[i]);
        if (!t.is_cuda()) value_error("all tensors must be on the current CUDA device");
        if (dev_ < 0) dev_ = c10::cuda::current_device();
        if (t.get_device() != dev_) value_error("all tensors must be on the current CUDA device");
        return &t;
    }
    const at::Tensor& tensor(int i, const char* what) {
        const at::Tensor* t = maybe(i, what);
        if (t == nullptr) type_error(std::string(what) + " must be a tensor");
        return *t;
    }
    int64_t integer(int i) {
        const long long x = PyLong_AsLongLong(v_[i]);
        if (x == -1 && PyErr_Occurred()) throw PythonError{};
        return x;
    }
    int32_t int32(int i, const char* what) {
        const int64_t x = integer(i);
        if (x != static_cast<int32_t>(x)) value_error(std::string(what) + " is out of range");
        return static_cast<int32_t>(x);
    }
    // the raw stream: the current one for None. Comes after the tensors and before
    // empty().
    void* stream(int i) {
        const c10::cuda::CUDAStream now =
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_));
        raw_ = now.stream();
        if (v_[i] == Py_None) return raw_;
        cudaStream_t given = reinterpret_cast<cudaStream_t>(integer(i));
        if (given == cudaStreamLegacy) given = nullptr;     // the default stream by another name
        other_ = given != raw_;
        raw_ = given;
        return raw_;
    }
    // Memory of the call's own stream: a block of the current stream's may still be
    // in use there by work that is queued, whoever let go of it.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) {
        c10::cuda::OptionalCUDAStreamGuard guard;
        if (other_)
            guard.reset_stream(
                c10::cuda::getStreamFromExternal(raw_, static_cast<c10::DeviceIndex>(dev_)));
        return at::detail::empty_cuda(shape, dtype, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev_)),
                                      std::nullopt);
    }
    // A result that the caller's current stream will read: the allocator must not
    // hand it out again, once it is let go of, before that use.
    void result(const at::Tensor& t) {
        if (!other_ || !t.defined() || t.numel() == 0) return;
        c10::cuda::CUDACachingAllocator::recordStream(
            t.storage().data_ptr(),
            c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_)));
    }

  private:
    PyObject* const* v_;
    int dev_ = -1;
    bool other_ = false;         // a stream was given that is not the current one
    cudaStream_t raw_ = nullptr;
};

std::string shape_text(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

void want_type(const at::Tensor& t, at::ScalarType dtype, const char* what) {
    if (t.scalar_type() != dtype)
        type_error(std::string(what) + " must be " + c10::toString(dtype) + ", got " +
                   c10::toString(t.scalar_type()));
}

void want_flat(const at::Tensor& t, at::ScalarType dtype, const char* what, int64_t n) {
    want_type(t, dtype, what);
    if (t.dim() != 1 || t.size(0) != n)
        value_error(std::string(what) + " must have shape [" + std::to_string(n) + "], got " +
                    shape_text(t.sizes()));
    if (!t.is_contiguous()) value_error(std::string(what) + " must be contiguous");
}

int64_t batch(const at::Tensor& off) {
    want_type(off, at::kLong, "new_offsets");
    if (off.dim() != 1 || off.size(0) < 1 || !off.is_contiguous())
        value_error("new_offsets must be a contiguous [B + 1]");
    if (off.size(0) - 1 > INT32_MAX) value_error("new_offsets is too long");
    return off.size(0) - 1;
}

hstu_dtype_t dtype_of(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kBFloat16) return HSTU_DTYPE_BF16;
    if (t.scalar_type() == at::kFloat) return HSTU_DTYPE_F32;
    type_error(std::string(what) + " must be bfloat16 or float32, got " +
               c10::toString(t.scalar_type()));
}

// token stride of a [T, H, d] view; a single token's means nothing
int64_t rows_of(const at::Tensor& t, const char* what, int64_t T, int64_t H, int64_t d) {
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != d)
        value_error(std::string(what) + " must be " + shape_text({T, H, d}) + ", got " +
                    shape_text(t.sizes()));
    if (T == 0) return H * d;
    if ((d > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != d))
        value_error(std::string(what) + ": heads and features must be contiguous inside a token");
    return T > 1 ? t.stride(0) : H * d;
}

struct Cache {
    int64_t page, tok;          // strides
};

Cache cache_of(const at::Tensor& t, const char* what) {
    if (t.dim() != 4) value_error(std::string(what) + " must be [num_pages, page_size, H, d]");
    const int64_t H = t.size(2), d = t.size(3);
    if ((d > 1 && t.stride(3) != 1) || (H > 1 && t.stride(2) != d))
        value_error(std::string(what) + ": heads and features must be contiguous inside a token");
    const int64_t tok = t.size(1) > 1 ? t.stride(1) : H * d;
    return {t.size(0) > 1 ? t.stride(0) : t.size(1) * tok, tok};
}

int64_t ts_page(const at::Tensor* t, int64_t pages, int64_t page) {
    if (t == nullptr) return 0;
    want_type(*t, at::kLong, "ts_cache");
    if (t->dim() != 2 || t->size(0) != pages || t->size(1) != page || (page > 1 && t->stride(1) != 1))
        value_error("ts_cache must be [num_pages, page_size] with contiguous pages");
    return pages > 1 ? t->stride(0) : page;
}

int64_t table_of(const at::Tensor& t, int64_t B) {
    want_type(t, at::kInt, "block_table");
    if (t.dim() != 2 || t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1) || t.size(1) > INT32_MAX)
        value_error("block_table must be [B, max_pages] with contiguous rows");
    return B > 1 ? t.stride(0) : t.size(1);
}

int32_t small(int64_t x, const char* what) {
    if (x > INT32_MAX) value_error(std::string(what) + " is too large");
    return static_cast<int32_t>(x);
}

template <typename T>
T* data(const at::Tensor* t) {
    return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}

PyObject* py_tensor(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// ------------------------------------------------------------------ calls

PyObject* cache_plan(PyObject* const* v, Py_ssize_t n) {
    Args a(v, n, 10);
    const at::Tensor &ctx = a.tensor(0, "ctx_lens"), &off = a.tensor(1, "new_offsets"),
                     &free = a.tensor(2, "free_pages"), &start = a.tensor(3, "free_start"),
                     &table = a.tensor(4, "block_table");
    const int64_t B = batch(off), total = a.integer(6);
    want_flat(ctx, at::kInt, "ctx_lens", B);
    want_flat(free, at::kInt, "free_pages", free.numel());
    want_flat(start, at::kInt, "free_start", 1);
    const int64_t stride = table_of(table, B);
    if (total < 0) value_error("total_new is negative");
    const at::Tensor *slots = a.maybe(7, "slots"), *end = a.maybe(8, "free_end");
    void* s = a.stream(9);
    at::Tensor own_slots, own_end;
    if (slots) want_flat(*slots, at::kLong, "slots", total);
    else slots = &(own_slots = a.empty({total}, at::kLong));
    if (end) {
        want_flat(*end, at::kInt, "free_end", 1);
        if (end->data_ptr() == start.data_ptr()) value_error("free_end must not be free_start");
    } else {
        end = &(own_end = a.empty({1}, at::kInt));
    }
    check("hstu_cache_plan",
          api.plan(data<int32_t>(&ctx), data<int64_t>(&off), static_cast<int32_t>(B), total,
                   a.int32(5, "page_size"), data<int32_t>(&free), small(free.numel(), "free_pages"),
                   data<int32_t>(&start), data<int32_t>(&table), stride,
                   static_cast<int32_t>(table.size(1)), data<int64_t>(slots), data<int32_t>(end), s));
    a.result(own_slots);
    a.result(own_end);
    PyObject *x = py_tensor(*slots), *y = py_tensor(*end);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

PyObject* cache_append(PyObject* const* v, Py_ssize_t n) {
    Args a(v, n, 8);
    const at::Tensor &k = a.tensor(0, "k"), &val = a.tensor(1, "v"), &slots = a.tensor(3, "slots"),
                     &kc = a.tensor(4, "k_cache"), &vc = a.tensor(5, "v_cache");
    const at::Tensor *ts = a.maybe(2, "timestamps"), *tsc = a.maybe(6, "ts_cache");
    if (k.dim() != 3 || val.dim() != 3) value_error("k and v must be [T, H, d]");
    const int64_t T = k.size(0), H = k.size(1), dqk = k.size(2), dv = val.size(2);
    const hstu_dtype_t dt = dtype_of(k, "k");
    if (val.scalar_type() != k.scalar_type() || kc.scalar_type() != k.scalar_type() ||
        vc.scalar_type() != k.scalar_type())
        type_error("k, v and the caches must share their dtype");
    const Cache ck = cache_of(kc, "k_cache"), cv = cache_of(vc, "v_cache");
    const int64_t pages = kc.size(0), page = kc.size(1);
    if (kc.size(2) != H || kc.size(3) != dqk || vc.size(0) != pages || vc.size(1) != page ||
        vc.size(2) != H || vc.size(3) != dv)
        value_error("k, v, k_cache and v_cache do not fit together");
    want_flat(slots, at::kLong, "slots", T);
    if (ts) want_flat(*ts, at::kLong, "timestamps", T);
    if ((ts == nullptr) != (tsc == nullptr)) value_error("timestamps and ts_cache come together");
    const int64_t ks = rows_of(k, "k", T, H, dqk), vs = rows_of(val, "v", T, H, dv);
    void* s = a.stream(7);
    check("hstu_cache_append",
          api.append(dt, k.data_ptr(), ks, val.data_ptr(), vs, data<int64_t>(ts),
                     data<int64_t>(&slots), T, small(H, "H"), small(dqk, "d_qk"), small(dv, "d_v"),
                     kc.data_ptr(), ck.page, ck.tok, vc.data_ptr(), cv.page, cv.tok,
                     data<int64_t>(tsc), ts_page(tsc, pages, page), small(pages, "num_pages"),
                     small(page, "page_size"), s));
    Py_RETURN_NONE;
}

PyObject* attn_cached(PyObject* const* v, Py_ssize_t n) {
    Args a(v, n, 16);
    const at::Tensor &q = a.tensor(0, "q"), &kc = a.tensor(1, "k_cache"), &vc = a.tensor(2, "v_cache"),
                     &table = a.tensor(4, "block_table"), &ctx = a.tensor(5, "ctx_lens"),
                     &off = a.tensor(6, "new_offsets");
    const at::Tensor *tsc = a.maybe(3, "ts_cache"), *ts = a.maybe(7, "timestamps"),
                     *par = a.maybe(8, "parents"), *pos = a.maybe(9, "pos_bias"),
                     *tb = a.maybe(10, "time_bias"), *out = a.maybe(13, "out"),
                     *ws = a.maybe(14, "workspace");
    if (q.dim() != 3) value_error("q must be [T, H, d_qk]");
    const int64_t T = q.size(0), H = q.size(1), dqk = q.size(2), B = batch(off);
    const hstu_dtype_t dt = dtype_of(q, "q");
    if (kc.scalar_type() != q.scalar_type() || vc.scalar_type() != q.scalar_type())
        type_error("q and the caches must share their dtype");
    const Cache ck = cache_of(kc, "k_cache"), cv = cache_of(vc, "v_cache");
    const int64_t pages = kc.size(0), page = kc.size(1), dv = vc.size(3);
    if (kc.size(2) != H || kc.size(3) != dqk || vc.size(0) != pages || vc.size(1) != page ||
        vc.size(2) != H)
        value_error("q, k_cache and v_cache do not fit together");
    want_flat(ctx, at::kInt, "ctx_lens", B);
    if (ts) want_flat(*ts, at::kLong, "timestamps", T);
    if (par) want_flat(*par, at::kInt, "parents", T);
    for (const at::Tensor* t : {pos, tb}) {
        if (t == nullptr) continue;
        want_type(*t, at::kFloat, "bias tables");
        if (t->dim() != 2 || t->size(0) != H || !t->is_contiguous())
            value_error("bias tables must be contiguous [H, entries]");
    }
    const int64_t stride = table_of(table, B), qs = rows_of(q, "q", T, H, dqk);
    const int32_t max_seqlen = a.int32(11, "max_seqlen"), max_new = a.int32(12, "max_new");
    void* s = a.stream(15);
    at::Tensor own_out, own_ws;
    if (out) {
        if (out->scalar_type() != q.scalar_type()) type_error("out must have q's dtype");
    } else {
        out = &(own_out = a.empty({T, H, dv}, q.scalar_type()));
    }
    const int64_t os = rows_of(*out, "out", T, H, dv);
    if (ws == nullptr) {
        const size_t need = api.attn_bytes(dt, max_new, small(dv, "d_v"));
        ws = &(own_ws = a.empty({static_cast<int64_t>(need < 16 ? 16 : need)}, at::kByte));
    } else if (!ws->is_contiguous()) {
        value_error("workspace must be contiguous");
    }
    check("hstu_attn_cached_fwd",
          api.attn(dt, q.data_ptr(), qs, kc.data_ptr(), ck.page, ck.tok, vc.data_ptr(), cv.page,
                   cv.tok, data<int64_t>(tsc), ts_page(tsc, pages, page), small(pages, "num_pages"),
                   small(page, "page_size"), data<int32_t>(&table), stride,
                   static_cast<int32_t>(table.size(1)), data<int32_t>(&ctx), data<int64_t>(&off),
                   static_cast<int32_t>(B), T, max_new, small(H, "H"), small(dqk, "d_qk"),
                   small(dv, "d_v"), data<int64_t>(ts), data<int32_t>(par), data<float>(pos),
                   pos ? small(pos->size(1), "num_pos") : 0, data<float>(tb),
                   tb ? small(tb->size(1), "num_time_buckets") : 0, max_seqlen, out->data_ptr(), os,
                   ws->data_ptr(), static_cast<size_t>(ws->nbytes()), s));
    a.result(own_out);
    return py_tensor(*out);
}

// a [rows, cols] matrix with unit column stride; its row stride
int64_t matrix(const at::Tensor& t, at::ScalarType dtype, const char* what, int64_t rows, int64_t cols) {
    want_type(t, dtype, what);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols ||
        (cols > 1 && rows > 0 && t.stride(1) != 1))
        value_error(std::string(what) + " must be " + shape_text({rows, cols}) +
                    " with unit column stride, got " + shape_text(t.sizes()));
    return rows > 1 ? t.stride(0) : cols;
}

PyObject* quant_w4(PyObject* const* v, Py_ssize_t n) {
    Args a(v, n, 3);
    const at::Tensor& W = a.tensor(0, "W");
    if (W.dim() != 2) value_error("W must be [N, K]");
    const int64_t N = W.size(0), K = W.size(1);
    const int32_t G = a.int32(1, "group");
    const int64_t ld = matrix(W, at::kBFloat16, "W", N, K);
    void* s = a.stream(2);
    at::Tensor codes = a.empty({N, K / 2}, at::kByte);
    at::Tensor scales = a.empty({N, G > 0 ? K / G : 0}, at::kBFloat16);
    check("hstu_quant_groups_w4", api.quant(W.data_ptr(), ld, N, small(K, "K"), G, codes.data_ptr(),
                                            K / 2, scales.data_ptr(), scales.size(1), s));
    a.result(codes);
    a.result(scales);
    PyObject *x = py_tensor(codes), *y = py_tensor(scales);
    PyObject* r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

PyObject* linear_w4(PyObject* const* v, Py_ssize_t n) {
    Args a(v, n, 8);
    const at::Tensor &x = a.tensor(0, "x"), &codes = a.tensor(1, "codes"), &scales = a.tensor(2, "scales");
    const at::Tensor *bias = a.maybe(3, "bias"), *res = a.maybe(5, "residual"), *out = a.maybe(6, "out");
    const int32_t epi = a.int32(4, "epilogue");
    if (x.dim() != 2 || codes.dim() != 2 || scales.dim() != 2)
        value_error("x, codes and scales must be matrices");
    const int64_t M = x.size(0), K = x.size(1), N = codes.size(0), ng = scales.size(1);
    if (ng < 1 || K % ng) value_error("scales must be [N, K / group]");
    const int64_t ldx = matrix(x, at::kBFloat16, "x", M, K);
    if (K % 2) value_error("K must be even");
    const int64_t ldc = matrix(codes, at::kByte, "codes", N, K / 2);
    const int64_t lds = matrix(scales, at::kBFloat16, "scales", N, ng);
    if (bias) want_flat(*bias, at::kFloat, "bias", N);
    if (epi == HSTU_EPI_RESIDUAL && res == nullptr) value_error("the residual epilogue needs residual");
    const int64_t ldr = epi == HSTU_EPI_RESIDUAL ? matrix(*res, at::kBFloat16, "residual", M, N) : 0;
    void* s = a.stream(7);
    at::Tensor own;
    if (out == nullptr) out = &(own = a.empty({M, N}, at::kBFloat16));
    const int64_t ldy = matrix(*out, at::kBFloat16, "out", M, N);
    check("hstu_linear_w4_fwd",
          api.linear(x.data_ptr(), ldx, M, small(K, "K"), codes.data_ptr(), ldc, scales.data_ptr(),
                     lds, static_cast<int32_t>(K / ng), small(N, "N"), data<float>(bias),
                     static_cast<hstu_epilogue_t>(epi),
                     epi == HSTU_EPI_RESIDUAL ? res->data_ptr() : nullptr, ldr, out->data_ptr(), ldy,
                     s));
    a.result(own);
    return py_tensor(*out);
}

// ------------------------------------------------------------------ the module

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* v, Py_ssize_t n) {
    try {
        if (check_fn == nullptr) throw Refusal{PyExc_RuntimeError, "bind() comes first"};
        return F(v, n);
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.what.c_str());
    } catch (const PythonError&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* m = PyImport_ImportModule("torch");
        PyObject* t = m ? PyObject_GetAttrString(m, "OutOfMemoryError") : nullptr;
        PyErr_SetString(t ? t : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(t);
        Py_XDECREF(m);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// bind(check, addresses of the library's functions)
PyObject* bind(PyObject*, PyObject* args) {
    PyObject* f;
    unsigned long long p[6];
    if (!PyArg_ParseTuple(args, "OKKKKKK", &f, &p[0], &p[1], &p[2], &p[3], &p[4], &p[5])) return nullptr;
    api.plan = reinterpret_cast<decltype(api.plan)>(p[0]);
    api.append = reinterpret_cast<decltype(api.append)>(p[1]);
    api.attn_bytes = reinterpret_cast<decltype(api.attn_bytes)>(p[2]);
    api.attn = reinterpret_cast<decltype(api.attn)>(p[3]);
    api.quant = reinterpret_cast<decltype(api.quant)>(p[4]);
    api.linear = reinterpret_cast<decltype(api.linear)>(p[5]);
    Py_INCREF(f);
    Py_XDECREF(check_fn);
    check_fn = f;
    Py_RETURN_NONE;
}

#define FAST(name) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(cache_plan), FAST(cache_append), FAST(attn_cached), FAST(quant_w4),
                         FAST(linear_w4), {"bind", bind, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
// The build reads the tag back from the file, to see whether it still fits.
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", HSTU_BINDING_TAG, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
