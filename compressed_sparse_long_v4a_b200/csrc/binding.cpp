// binding.cpp -- argument marshalling of the serving calls (rotary positions, attention over a shared prefix,
// attention weights, eviction) as a CPython module over the C ABI.
//
// A decode step makes several of these calls with a dozen tensors each, on kernels of a few microseconds:
// reading dtypes, shapes, strides and pointers through the interpreter took 14 to 25 us per call, here
// it is below one.  The functions take what the Python wrappers of the same names document, positionally,
// raise ValueError or TypeError for tensors that do not fit together, and return the C ABI's status.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "v4a.h"

namespace {

struct Raised {};                                       // a Python error is set
struct ValueError : std::runtime_error { using std::runtime_error::runtime_error; };
struct TypeError : std::runtime_error { using std::runtime_error::runtime_error; };

using T = const at::Tensor*;

T tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a tensor or None");
    return &THPVariable_Unpack(o);
}
T required(PyObject* o, const char* name) {
    T t = tensor(o, name);
    if (!t) throw TypeError(std::string(name) + " must be a tensor");
    return t;
}
long long integer(PyObject* o) {
    long long v;
    if (PyLong_Check(o)) {
        v = PyLong_AsLongLong(o);
    } else {
        PyObject* n = PyNumber_Long(o);
        if (!n) throw Raised();
        v = PyLong_AsLongLong(n);
        Py_DECREF(n);
    }
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
int small(PyObject* o, const char* name) {
    const long long v = integer(o);
    if (v < INT_MIN || v > INT_MAX) throw ValueError(std::string(name) + " is out of range");
    return (int)v;
}
int size_of(int64_t v, const char* name) {
    if (v > INT_MAX) throw ValueError(std::string(name) + " is out of range");
    return (int)v;
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}
void* ptr(T t) { return t ? t->data_ptr() : nullptr; }

v4a_dtype float_dtype(T t) {
    if (t->scalar_type() == at::kFloat) return V4A_F32;
    if (t->scalar_type() == at::kBFloat16) return V4A_BF16;
    throw TypeError(std::string("unsupported dtype ") + at::toString(t->scalar_type()));
}
void contiguous(T t, const char* name) {
    if (t && !t->is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
}
std::string text(at::IntArrayRef s) {
    std::ostringstream o;
    o << s;
    return o.str();
}
// a contiguous tensor of this dtype and shape (null passes)
void typed(T t, const char* name, at::ScalarType dtype, std::initializer_list<int64_t> shape) {
    if (!t) return;
    const at::IntArrayRef want(shape.begin(), shape.size());
    if (t->scalar_type() != dtype || t->sizes() != want)
        throw ValueError(std::string(name) + " must be " + at::toString(dtype) + " " + text(want) + ", got " +
                         at::toString(t->scalar_type()) + " " + text(t->sizes()));
    contiguous(t, name);
}
void status_word(T t) {
    if (t && (t->scalar_type() != at::kInt || t->numel() < 1)) throw ValueError("dev_status must be int32 with one element");
}

// the one CUDA device of a call's tensors
struct Device {
    int index = -1;
    void add(T t, const char* name) {
        if (!t) return;
        if (!t->is_cuda()) throw ValueError("libv4a takes CUDA tensors");
        const int i = t->device().index();
        if (index < 0) {
            index = i;
        } else if (i != index) {
            throw ValueError(std::string(name) + " is on cuda:" + std::to_string(i) + ", the other tensors on cuda:" + std::to_string(index));
        }
    }
};

// makes the device current for the call and finds its stream: the device's current one, or the one given
struct Place {
    c10::cuda::CUDAGuard guard;
    void* stream;
    bool other = false;  // not the current stream
    Place(const Device& d, PyObject* given) : guard((c10::DeviceIndex)d.index) {
        void* current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)d.index).stream();
        stream = current;
        if (given == Py_None) return;
        PyObject* p = PyObject_GetAttrString(given, "cuda_stream");
        if (!p) PyErr_Clear();
        long long v = integer(p ? p : given);
        Py_XDECREF(p);
        if (v == 1) v = 0;  // cudaStreamLegacy, the default stream, which torch knows as 0
        stream = reinterpret_cast<void*>(v);
        other = stream != current;
    }
};

bool capturing(void* stream) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &s) != cudaSuccess) {
        (void)cudaGetLastError();  // the default stream while another one is captured: the call itself will say so
        return false;
    }
    return s != cudaStreamCaptureStatusNone;
}

// wraps a function of (args, n): checks the count, turns C++ exceptions into Python's
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)f());
    } catch (const Raised&) {
    } catch (const ValueError& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const TypeError& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* rope(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> int {
        PyObject* seq = PySequence_Fast(arg[0], "pairs must be a sequence of (x, out)");
        if (!seq) throw Raised();
        struct Hold { PyObject* o; ~Hold() { Py_DECREF(o); } } hold{seq};
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
        if (count == 0) return V4A_OK;
        v4a_rope_io io[8];
        v4a_rope_params par;
        par.rope_dims = small(arg[1], "rope_dims");
        T positions = tensor(arg[2], "positions");
        const bool last = arg[5] == Py_None;
        const int offset = last ? 0 : small(arg[5], "rope_offset");
        Device dev;
        int64_t B = 0, tokens = 0;
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* pair = PySequence_Fast(PySequence_Fast_GET_ITEM(seq, i), "pairs must be a sequence of (x, out)");
            if (!pair) throw Raised();
            Hold hold_pair{pair};
            if (PySequence_Fast_GET_SIZE(pair) != 2) throw ValueError("pairs must be a sequence of (x, out)");
            T x = required(PySequence_Fast_GET_ITEM(pair, 0), "x"), out = required(PySequence_Fast_GET_ITEM(pair, 1), "out");
            const int64_t dim = x->dim();
            if ((dim != 3 && dim != 4) || x->sizes() != out->sizes() || x->scalar_type() != out->scalar_type())
                throw ValueError("x and out must be [batch][n_tok][heads][d] or [batch][n_tok][d], of one shape and dtype");
            if (i == 0) {
                B = x->size(0);
                tokens = x->size(1);
            } else if (B != x->size(0) || tokens != x->size(1)) {
                throw ValueError("the streams of a call have the same batch and tokens");
            }
            const int d = size_of(x->size(dim - 1), "d");
            if (d > 1 && (x->stride(dim - 1) != 1 || out->stride(dim - 1) != 1)) throw ValueError("x and out must have dense rows");
            const v4a_dtype dt = float_dtype(x);
            dev.add(x, "x");
            dev.add(out, "out");
            if (i >= 8) continue;  // refused by the call
            const bool four = dim == 4;
            io[i] = {x->data_ptr(), out->data_ptr(), four ? size_of(x->size(2), "heads") : 1, d, last ? d - par.rope_dims : offset, dt,
                     x->stride(0), x->stride(1), four ? x->stride(2) : 0, out->stride(0), out->stride(1), four ? out->stride(2) : 0};
        }
        if (positions) {
            if (positions->scalar_type() != at::kLong || positions->dim() != 2 || positions->size(0) != B || positions->size(1) != tokens)
                throw ValueError("positions must be int64 [batch][n_tok]");
            if (tokens > 1 && positions->stride(1) != 1) throw ValueError("positions must have dense rows");
            dev.add(positions, "positions");
        }
        par.base = number(arg[6]);
        par.half = truth(arg[7]);
        par.inverse = truth(arg[8]);
        par.factor = number(arg[9]);
        par.orig_ctx = integer(arg[10]);
        par.beta_fast = number(arg[11]);
        par.beta_slow = number(arg[12]);
        par.out_scale = number(arg[13]);
        const Place at(dev, arg[14]);
        return v4a_rope(io, (int)std::min<Py_ssize_t>(count, 9), size_of(B, "batch"), tokens,
                        positions ? static_cast<const int64_t*>(positions->data_ptr()) : nullptr, positions ? positions->stride(0) : 0,
                        integer(arg[3]), integer(arg[4]), &par, at.stream);
    });
}

struct Query {
    int64_t B, n_q, H, d;
};
Query query(T q) {
    contiguous(q, "q");
    if (q->dim() != 4) throw ValueError("q must be [batch][n_q][heads][d]");
    return {q->size(0), q->size(1), q->size(2), q->size(3)};
}

v4a_shared_cache cache(const Query& s, T q, T prefix, long long n_prefix, T own, T ring, T own_count, T own_entry, T ctx_lens) {
    const auto dt = q->scalar_type();
    if (own && own->dim() != 3) throw ValueError("own must be [batch][own_rows][d]");
    if (prefix && prefix->dim() != 2) throw ValueError("prefix must be [n_prefix][d]");
    if (ring && ring->dim() != 3) throw ValueError("ring must be [batch][ring_rows][d]");
    const int64_t rows = own ? own->size(1) : 0, ring_rows = ring ? ring->size(1) : 0;
    typed(own, "own", dt, {s.B, rows, s.d});
    typed(own_count, "own_count", at::kInt, {s.B});
    typed(own_entry, "own_entry", at::kInt, {s.B, rows});
    typed(ctx_lens, "ctx_lens", at::kLong, {s.B});
    if (prefix) typed(prefix, "prefix", dt, {prefix->size(0), s.d});
    typed(ring, "ring", dt, {s.B, ring_rows, s.d});
    return {ptr(prefix), n_prefix, ptr(own), size_of(rows, "own_rows"), static_cast<const int32_t*>(ptr(own_count)),
            static_cast<const int32_t*>(ptr(own_entry)), ptr(ring), size_of(ring_rows, "ring_rows"),
            static_cast<const int64_t*>(ptr(ctx_lens))};
}

v4a_shape shape(const Query& s, PyObject* m, int window, PyObject* ctx_len) {
    return {size_of(s.B, "batch"), size_of(s.n_q, "n_q"), size_of(s.H, "heads"), size_of(s.d, "d"), small(m, "m"), 0, window, integer(ctx_len)};
}

PyObject* hca_attend_shared(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    return guarded(n, 18, [&]() -> int {
        T q = required(arg[0], "q"), prefix = tensor(arg[1], "prefix"), own = tensor(arg[2], "own"), ring = tensor(arg[3], "ring"),
          out = required(arg[4], "out"), ctx_lens = tensor(arg[8], "ctx_lens"), own_count = tensor(arg[9], "own_count"),
          own_entry = tensor(arg[10], "own_entry"), lse = tensor(arg[11], "lse"), workspace = tensor(arg[12], "workspace"),
          dev_status = tensor(arg[13], "dev_status"), sink = tensor(arg[14], "sink");
        const Query s = query(q);
        Device dev;
        dev.add(q, "q");
        dev.add(prefix, "prefix");
        dev.add(own, "own");
        dev.add(ring, "ring");
        dev.add(out, "out");
        dev.add(ctx_lens, "ctx_lens");
        dev.add(own_count, "own_count");
        dev.add(own_entry, "own_entry");
        dev.add(lse, "lse");
        dev.add(workspace, "workspace");
        dev.add(dev_status, "dev_status");
        dev.add(sink, "sink");
        const long long n_prefix = prefix && prefix->dim() > 0 ? prefix->size(0) : 0;
        const v4a_shared_cache c = cache(s, q, prefix, n_prefix, own, ring, own_count, own_entry, ctx_lens);
        typed(out, "out", out->scalar_type(), {s.B, s.n_q, s.H, s.d});
        typed(lse, "lse", at::kFloat, {s.B, s.n_q, s.H});
        typed(sink, "sink", at::kFloat, {s.H});
        status_word(dev_status);
        contiguous(workspace, "workspace");
        const v4a_shape sh = shape(s, arg[5], small(arg[6], "window"), arg[7]);
        const v4a_dtype dt = float_dtype(q), out_dt = float_dtype(out);
        const v4a_attend_ext ext = {static_cast<const float*>(ptr(sink)), small(arg[15], "rope_dims"), (float)number(arg[16])};
        const Place at(dev, arg[17]);
        at::Tensor made;
        if (!workspace) {
            if (at.other && capturing(at.stream))  // a graph would keep using memory that goes back to the allocator
                throw ValueError("workspace is required where a stream that is not the current one is captured");
            const size_t bytes = v4a_shared_workspace_size(&sh, n_prefix, c.own_rows, dt);
            // From the pool of the stream that will use it: a block of another stream's may still be in use there, by
            // kernels queued before its last owner let go of it, and goes back there while this stream uses it.
            c10::cuda::OptionalCUDAStreamGuard used_on;
            if (at.other)
                used_on.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(at.stream), (c10::DeviceIndex)dev.index));
            made = at::empty({(int64_t)std::max<size_t>(bytes, 256)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev.index));
            workspace = &made;
        }
        return v4a_hca_attend_shared(q->data_ptr(), &c, out->data_ptr(), out_dt, static_cast<float*>(ptr(lse)), dt, workspace->data_ptr(),
                                     workspace->nbytes(), static_cast<int*>(ptr(dev_status)), sink || ext.rope_dims ? &ext : nullptr, &sh,
                                     at.stream);
    });
}

PyObject* attend_weights(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> int {
        T q = required(arg[0], "q"), own = tensor(arg[1], "own"), lse = tensor(arg[2], "lse"), weights = tensor(arg[3], "weights"),
          out = tensor(arg[4], "out"), ctx_lens = tensor(arg[8], "ctx_lens"), own_count = tensor(arg[9], "own_count"),
          own_entry = tensor(arg[10], "own_entry"), dev_status = tensor(arg[12], "dev_status");
        const Query s = query(q);
        Device dev;
        dev.add(q, "q");
        dev.add(own, "own");
        dev.add(lse, "lse");
        dev.add(weights, "weights");
        dev.add(out, "out");
        dev.add(ctx_lens, "ctx_lens");
        dev.add(own_count, "own_count");
        dev.add(own_entry, "own_entry");
        dev.add(dev_status, "dev_status");
        const v4a_shared_cache c = cache(s, q, nullptr, integer(arg[7]), own, nullptr, own_count, own_entry, ctx_lens);
        typed(lse, "lse", at::kFloat, {s.B, s.n_q, s.H});
        typed(weights, "weights", at::kFloat, {s.B, c.own_rows});
        typed(out, "out", at::kFloat, {s.B, c.own_rows});
        status_word(dev_status);
        const v4a_shape sh = shape(s, arg[5], 0, arg[6]);
        const v4a_dtype dt = float_dtype(q);
        const float decay = (float)number(arg[11]);
        const Place at(dev, arg[13]);
        return v4a_attend_weights(q->data_ptr(), &c, static_cast<const float*>(ptr(lse)), static_cast<const float*>(ptr(weights)),
                                  static_cast<float*>(ptr(out)), decay, dt, static_cast<int*>(ptr(dev_status)), &sh, at.stream);
    });
}

PyObject* evict(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> int {
        T own = required(arg[0], "own"), weights = required(arg[1], "weights"), own_out = required(arg[2], "own_out"),
          weights_out = required(arg[3], "weights_out"), kept = required(arg[4], "kept"), count_out = required(arg[5], "count_out"),
          own_count = tensor(arg[9], "own_count"), own_entry = tensor(arg[10], "own_entry"), entry_out = tensor(arg[11], "entry_out"),
          dev_status = tensor(arg[13], "dev_status");
        if (own->dim() != 3 || own_out->dim() != 3) throw ValueError("own and own_out must be [batch][rows][d]");
        Device dev;
        dev.add(own, "own");
        dev.add(weights, "weights");
        dev.add(own_out, "own_out");
        dev.add(weights_out, "weights_out");
        dev.add(kept, "kept");
        dev.add(count_out, "count_out");
        dev.add(own_count, "own_count");
        dev.add(own_entry, "own_entry");
        dev.add(entry_out, "entry_out");
        dev.add(dev_status, "dev_status");
        const int64_t B = own->size(0), rows = own->size(1), d = own->size(2), out_rows = own_out->size(1);
        const int budget = small(arg[6], "budget");
        contiguous(own, "own");
        typed(weights, "weights", at::kFloat, {B, rows});
        typed(own_count, "own_count", at::kInt, {B});
        typed(own_entry, "own_entry", at::kInt, {B, rows});
        typed(own_out, "own_out", own->scalar_type(), {B, out_rows, d});
        typed(weights_out, "weights_out", at::kFloat, {B, out_rows});
        typed(entry_out, "entry_out", at::kInt, {B, out_rows});
        typed(kept, "kept", at::kInt, {B, budget});
        typed(count_out, "count_out", at::kInt, {B});
        status_word(dev_status);
        const v4a_evict_io io = {own->data_ptr(), static_cast<const float*>(weights->data_ptr()), static_cast<const int32_t*>(ptr(own_count)),
                                 static_cast<const int32_t*>(ptr(own_entry)), size_of(rows, "rows"), size_of(d, "d"), float_dtype(own),
                                 own_out->data_ptr(), static_cast<float*>(weights_out->data_ptr()), static_cast<int32_t*>(ptr(entry_out)),
                                 static_cast<int32_t*>(kept->data_ptr()), static_cast<int32_t*>(count_out->data_ptr()),
                                 size_of(out_rows, "rows of own_out"), small(arg[12], "first_entry")};
        const Place at(dev, arg[14]);
        return v4a_evict(&io, size_of(B, "batch"), budget, small(arg[7], "keep_first"), small(arg[8], "keep_recent"),
                         static_cast<int*>(ptr(dev_status)), at.stream);
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope), FAST(hca_attend_shared), FAST(attend_weights), FAST(evict), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", V4A_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
