// binding.cpp -- the host path of the serving calls, from torch tensors to the C ABI.
//
// A decode step makes four of these calls and their kernels take a few microseconds each, so with
// descriptions built and buffers allocated from Python the GPU waits for the host.  Here each call
// checks what the C ABI cannot see (devices, shapes and strides behind bare pointers), allocates
// missing outputs and scratch, and calls the library's entry point, whose address the Python side
// hands over (so a debug or trace build of the library is used where one is chosen).  Nothing is
// computed.  A call returns its outputs, or the library's status as an int when that is not FA_OK.
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa_b200.h"

namespace {

// Raised as the Python exception of its type by `guarded`.
struct Refused {
    PyObject* type;
    std::string what;
};

struct Entry {
    decltype(&fa_rotary) rotary;
    decltype(&fa_cache_append) append;
    decltype(&fa_cache_read) read;
    decltype(&fa_decode) decode;
    decltype(&fa_decode_workspace_bytes) decode_bytes;
} g_entry;

void require(bool ok, const char* what) {
    if (!ok) throw Refused{PyExc_ValueError, what};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, {}};
    return v;
}

int32_t int32(PyObject* o, const char* name) {
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{PyExc_ValueError, std::string(name) + " does not fit in 32 bits"};
    return (int32_t)v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, {}};
    return v;
}

int cuda_index(const at::Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

fa_tensor_t describe(const at::Tensor& t) {
    require(t.dim() == 4, "expected a (B, H, S, D) tensor");
    fa_tensor_t d;
    d.data = t.data_ptr();
    d.dtype = t.scalar_type() == at::kBFloat16 ? FA_DTYPE_BF16 : t.scalar_type() == at::kHalf ? FA_DTYPE_F16 : -1;
    d.B = t.size(0), d.H = t.size(1), d.S = t.size(2), d.D = t.size(3);
    for (int i = 0; i < 4; ++i) d.stride[i] = t.stride(i);
    return d;
}

// The address of a contiguous int32 tensor of n values on the device; None gives NULL where allowed.
const int32_t* int32_rows(PyObject* o, const char* name, int device, int64_t n, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || cuda_index(t) != device || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        throw Refused{PyExc_ValueError, std::string(name) + " must be a contiguous int32 tensor of " + std::to_string(n) +
                                            " values on the cache's device"};
    return t.data_ptr<int32_t>();
}

struct Table {
    const int32_t* data;
    int64_t stride, width;
};
Table page_table(PyObject* o, int device, int64_t B) {
    const at::Tensor& t = tensor(o, "page_table");
    require(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == B && cuda_index(t) == device &&
                (t.size(1) <= 1 || t.stride(1) == 1),
            "page_table must be an int32 tensor (B, n) with contiguous rows on the cache's device");
    return {t.data_ptr<int32_t>(), B > 1 ? t.stride(0) : t.size(1), t.size(1)};
}

// The device and the stream of a call: the caller's (an address) or the device's current one.  Both
// are current while it lives, so what is allocated belongs to that stream: memory freed when the
// call returns goes to no other stream's work while the kernels may still be running.
struct Place {
    Place(int device, PyObject* stream) : on(static_cast<c10::DeviceIndex>(device)) {
        if (stream == Py_None) {
            at = c10::cuda::getCurrentCUDAStream(on.current_device().index()).stream();
            return;
        }
        at = static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
        if (!at && PyErr_Occurred()) throw Refused{nullptr, {}};
        const auto index = on.current_device().index();
        using_stream.reset_stream(at ? c10::cuda::getStreamFromExternal(at, index) : c10::cuda::getDefaultCUDAStream(index));
    }
    c10::cuda::CUDAGuard on;
    c10::cuda::OptionalCUDAStreamGuard using_stream;
    cudaStream_t at = nullptr;
};

const fa_kv_cache_t* cache_at(PyObject* o) {
    const auto* c = static_cast<const fa_kv_cache_t*>(PyLong_AsVoidPtr(o));
    if (!c) throw Refused{PyExc_ValueError, "no cache"};
    return c;
}

PyObject* status_or(fa_status_t s, const at::Tensor& a, const at::Tensor* b) {
    if (s != FA_OK) return PyLong_FromLong(s);
    PyObject* t = PyTuple_New(2);
    if (!t) throw Refused{nullptr, {}};
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    if (b) PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(*b));
    else PyTuple_SET_ITEM(t, 1, Py_NewRef(Py_None));
    return t;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& call) {
    try {
        if (n != want) throw Refused{PyExc_TypeError, "wrong number of arguments"};
        at::AutoDispatchBelowADInplaceOrView below;      // allocations only: nothing to differentiate
        return call();
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.what.c_str());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (q, k or None, positions or None, first, frequencies, layout, factor, inverse, q_out or None,
//  k_out or None, stream or None)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Tensor& q = tensor(a[0], "q");
        const bool has_k = a[1] != Py_None;
        const at::Tensor k = has_k ? tensor(a[1], "k") : at::Tensor();
        const int device = cuda_index(q);
        require(device >= 0 && (!has_k || cuda_index(k) == device), "q and k must be CUDA tensors of one device");
        const at::Tensor& f = tensor(a[4], "frequencies");
        require(f.scalar_type() == at::kDouble && cuda_index(f) == device && f.dim() == 1 && f.is_contiguous(),
                "frequencies must be a contiguous 1-D float64 tensor on q's device");
        fa_tensor_t dq = describe(q), dk = {}, dqo, dko = {};
        const int32_t* pos = nullptr;
        int64_t pos_stride = 0;
        if (a[2] != Py_None) {
            const at::Tensor& p = tensor(a[2], "positions");
            const bool rows = p.dim() == 2 && p.size(0) == dq.B && p.size(1) == dq.S;
            require(p.scalar_type() == at::kInt && cuda_index(p) == device && (rows || (p.dim() == 1 && p.size(0) == dq.S)) &&
                        (dq.S <= 1 || p.stride(-1) == 1),
                    "positions must be an int or an int32 tensor (B, S) or (S,) with contiguous rows on q's device");
            pos = p.data_ptr<int32_t>();
            pos_stride = rows && dq.B > 1 ? p.stride(0) : 0;
        }
        const Place place(device, a[10]);
        const at::Tensor q_out = a[8] == Py_None ? at::empty_like(q) : tensor(a[8], "q_out");
        require(cuda_index(q_out) == device, "q_out must be on q's device");
        dqo = describe(q_out);
        at::Tensor k_out;
        if (has_k) {
            k_out = a[9] == Py_None ? at::empty_like(k) : tensor(a[9], "k_out");
            require(cuda_index(k_out) == device, "k_out must be on q's device");
            dk = describe(k);
            dko = describe(k_out);
        } else {
            require(a[9] == Py_None, "k_out without k");
        }
        const fa_status_t s = g_entry.rotary(&dq, has_k ? &dk : nullptr, pos, pos_stride, integer(a[3]), f.data_ptr<double>(),
                                             (int32_t)std::min<int64_t>(2 * f.numel(), INT32_MAX), int32(a[5], "layout"),
                                             (float)number(a[6]), int32(a[7], "inverse"), &dqo, has_k ? &dko : nullptr, place.at);
        return status_or(s, q_out, has_k ? &k_out : nullptr);
    });
}

// (cache address, device, k, v, page_table, start, count or None, stream or None)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject* {
        const fa_kv_cache_t* c = cache_at(a[0]);
        const int device = int32(a[1], "device");
        const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        require(cuda_index(k) == device && cuda_index(v) == device, "k and v must be on the cache's device");
        const fa_tensor_t dk = describe(k), dv = describe(v);
        const Table t = page_table(a[4], device, dk.B);
        const int32_t* start = int32_rows(a[5], "start", device, dk.B);
        const int32_t* count = int32_rows(a[6], "count", device, dk.B, true);
        const Place place(device, a[7]);
        const fa_status_t s = g_entry.append(&dk, &dv, c, t.data, t.stride, t.width, start, count, place.at);
        if (s != FA_OK) return PyLong_FromLong(s);
        Py_RETURN_NONE;
    });
}

// (cache address, device, page_table, kv_lens, S, start or None, bf16, k_out or None, v_out or None,
//  stream or None)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const fa_kv_cache_t* c = cache_at(a[0]);
        const int device = int32(a[1], "device");
        const at::Tensor& table = tensor(a[2], "page_table");
        require(table.dim() == 2, "page_table must be an int32 tensor (B, n) with contiguous rows on the cache's device");
        const int64_t B = table.size(0), S = integer(a[4]);
        require(S >= 0, "S must not be negative");
        const Table t = page_table(a[2], device, B);
        const int32_t* lens = int32_rows(a[3], "kv_lens", device, B);
        const int32_t* start = int32_rows(a[5], "start", device, B, true);
        const Place place(device, a[9]);
        at::Tensor out[2];
        fa_tensor_t d[2];
        for (int i = 0; i < 2; ++i) {
            PyObject* given = a[7 + i];
            out[i] = given == Py_None ? at::empty({B, c->H, S, c->D}, table.options().dtype(integer(a[6]) ? at::kBFloat16 : at::kHalf))
                                      : tensor(given, "k_out and v_out");
            d[i] = describe(out[i]);
            require(cuda_index(out[i]) == device && d[i].B == B && d[i].H == c->H && d[i].S == S && d[i].D == c->D,
                    "k_out and v_out must be (B, H, S, D) tensors on the cache's device");
        }
        const fa_status_t s = g_entry.read(c, t.data, t.stride, t.width, start, lens, &d[0], &d[1], place.at);
        return status_or(s, out[0], &out[1]);
    });
}

// (cache address, device, q, page_table, kv_lens, window, score_mod, params address or None, scale,
//  out or None, lse or None, return_lse, workspace or None, stream or None)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        const fa_kv_cache_t* c = cache_at(a[0]);
        const int device = int32(a[1], "device");
        const at::Tensor& q = tensor(a[2], "q");
        require(cuda_index(q) == device, "q must be on the cache's device");
        fa_tensor_t dq = describe(q);
        const Table t = page_table(a[3], device, dq.B);
        const int32_t* lens = int32_rows(a[4], "kv_lens", device, dq.B);
        const Place place(device, a[13]);
        const at::Tensor out = a[9] == Py_None ? at::empty_like(q) : tensor(a[9], "out");
        require(cuda_index(out) == device, "out must be on the cache's device");
        fa_tensor_t dout = describe(out);
        at::Tensor lse;
        if (a[10] != Py_None) {
            lse = tensor(a[10], "lse");
            require(lse.scalar_type() == at::kFloat && cuda_index(lse) == device && lse.dim() == 3 && lse.size(0) == dq.B &&
                        lse.size(1) == dq.H && lse.size(2) == 1 && lse.is_contiguous(),
                    "lse must be a contiguous float32 tensor (B, HQ, 1) on the cache's device");
        } else if (integer(a[11])) {
            lse = at::empty({dq.B, dq.H, 1}, q.options().dtype(at::kFloat));
        }
        at::Tensor ws;
        if (a[12] != Py_None) {
            ws = tensor(a[12], "workspace");
            // Its bytes have to be its own: a strided or broadcast tensor counts more than its memory holds.
            require(cuda_index(ws) == device && ws.is_contiguous(), "workspace must be a contiguous tensor on the cache's device");
        } else {
            ws = at::empty({(int64_t)g_entry.decode_bytes(dq.B, dq.H, c->H, dq.D)}, q.options().dtype(at::kByte));
        }
        const fa_status_t s = g_entry.decode(
            &dq, c, t.data, t.stride, t.width, lens, int32(a[5], "window"), (uint32_t)int32(a[6], "score_mod"),
            a[7] == Py_None ? nullptr : static_cast<const fa_score_params_t*>(PyLong_AsVoidPtr(a[7])), (float)number(a[8]),
            &dout, lse.defined() ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), (size_t)ws.nbytes(), place.at);
        return status_or(s, out, lse.defined() ? &lse : nullptr);
    });
}

// (addresses of fa_rotary, fa_cache_append, fa_cache_read, fa_decode, fa_decode_workspace_bytes)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject* {
        g_entry.rotary = reinterpret_cast<decltype(g_entry.rotary)>(PyLong_AsVoidPtr(a[0]));
        g_entry.append = reinterpret_cast<decltype(g_entry.append)>(PyLong_AsVoidPtr(a[1]));
        g_entry.read = reinterpret_cast<decltype(g_entry.read)>(PyLong_AsVoidPtr(a[2]));
        g_entry.decode = reinterpret_cast<decltype(g_entry.decode)>(PyLong_AsVoidPtr(a[3]));
        g_entry.decode_bytes = reinterpret_cast<decltype(g_entry.decode_bytes)>(PyLong_AsVoidPtr(a[4]));
        Py_RETURN_NONE;
    });
}

#define FA_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FA_METHOD(bind), FA_METHOD(rotary), FA_METHOD(append), FA_METHOD(read), FA_METHOD(decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fa_b200_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fa_b200_torch(void) { return PyModule_Create(&g_module); }
