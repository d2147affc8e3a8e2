// py_bdfp8.cpp -- the Python side of bdfp8_append and bdfp8_decode: tensor checks
// and marshalling for bdfp8.py.
//
// A serving loop calls these once per layer and token, and at small batches a
// call's host time is what it costs: checking eight to fourteen tensors in Python
// and passing two dozen arguments through ctypes took 18 (decode) and 23 us
// (append) a call, several times the kernels' own time.  Here a tensor is a few
// loads.  Nothing is computed or kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/bdfp8.h"

namespace {

PyObject* g_error = nullptr;   // BDFP4Error

// A failed check; what() is the message.
struct Refused {
    std::string what;
};

std::string describe(const at::Tensor& t) {
    std::string s = c10::toString(t.scalar_type());
    s += " [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    s += "] strides [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
    return s + "] on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw Refused{std::string(what) + ": want a tensor"};
    return THPVariable_Unpack(o);
}

// Data of a contiguous tensor of this device, type and shape.
void* like(PyObject* o, const at::Device& dev, at::ScalarType type, std::initializer_list<int64_t> shape, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (t.device() != dev || t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_contiguous()) {
        std::string s = std::string(what) + ": want contiguous " + c10::toString(type) + " [";
        for (int64_t n : shape) s += (s.back() == '[' ? "" : ", ") + std::to_string(n);
        throw Refused{s + "] on " + dev.str() + ", got " + describe(t)};
    }
    return t.data_ptr();
}

// bf16 rows [T][H][d] whose heads are contiguous: data and the stride of a token.
void* rows(PyObject* o, const at::Device& dev, int64_t T, int64_t H, int64_t d, int64_t* stride, const char* what) {
    const at::Tensor& t = tensor(o, what);
    if (t.device() != dev || t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != T || t.size(1) != H ||
        t.size(2) != d || t.stride(2) != 1 || (H > 1 && t.stride(1) != d))
        throw Refused{std::string(what) + ": want bf16 [" + std::to_string(T) + ", " + std::to_string(H) + ", " +
                      std::to_string(d) + "] with contiguous heads on " + dev.str() + ", got " + describe(t)};
    *stride = T > 1 ? t.stride(0) : H * d;
    return t.data_ptr();
}

int64_t whole(PyObject* o, const char* what) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{std::string(what) + ": want an integer"};
    }
    return v;
}

int small(PyObject* o, const char* what) {
    const int64_t v = whole(o, what);
    if (v != (int)v) throw Refused{std::string(what) + ": " + std::to_string(v) + " is out of range"};
    return (int)v;
}

int extent(int64_t n, const char* what) {
    if (n != (int)n) throw Refused{std::string(what) + ": " + std::to_string(n) + " is out of range"};
    return (int)n;
}

int32_t* status(PyObject* o, const at::Device& dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "dev_status");
    if (t.device() != dev || t.scalar_type() != at::kInt || t.numel() != 1)
        throw Refused{"dev_status: want one int32 on " + dev.str() + ", got " + describe(t)};
    return (int32_t*)t.data_ptr();
}

struct Pages {
    void *k, *v;
    float* scales;
    int64_t num_pages;
    int H, d;
    bdfp8_fmt fmt;
};

// args: k_pages, v_pages, kv_scales, num_pages, H_kv, d, fmt
Pages pages(PyObject* const* a, const at::Device& dev) {
    Pages p;
    p.num_pages = whole(a[3], "num_pages");
    p.H = small(a[4], "H_kv");
    p.d = small(a[5], "d");
    p.fmt = (bdfp8_fmt)small(a[6], "fmt");
    p.k = like(a[0], dev, at::kByte, {p.num_pages, p.H, 64 * (int64_t)p.d}, "k_pages");
    p.v = like(a[1], dev, at::kByte, {p.num_pages, p.H, 64 * (int64_t)p.d}, "v_pages");
    p.scales = (float*)like(a[2], dev, at::kFloat, {p.num_pages, p.H, 2, 4}, "kv_scales");
    return p;
}

const at::Tensor& table(PyObject* o) {
    const at::Tensor& t = tensor(o, "block_table");
    if (t.dim() != 2) throw Refused{"block_table: want int32 [B, pages], got " + describe(t)};
    return t;
}

// The call itself, with the tensors' device current and on its current stream unless one is given.
template <class Call>
PyObject* on_device(const at::Device& dev, PyObject* stream, const Call& call) {
    if (!dev.is_cuda()) throw Refused{"tensors must be on a CUDA device, got " + dev.str()};
    void* st = stream == Py_None ? (void*)c10::cuda::getCurrentCUDAStream(dev.index()).stream() : PyLong_AsVoidPtr(stream);
    if (!st && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{"stream: want a CUDA stream"};
    }
    const c10::cuda::CUDAGuard guard(dev);
    PyThreadState* const held = PyEval_SaveThread();   // a launch may wait for the queue
    const int rc = call(st);
    PyEval_RestoreThread(held);
    return PyLong_FromLong(rc);
}

template <class Body>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, const Body& body) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "want %zd arguments, got %zd", want, nargs);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused& e) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// k, v, cu_tokens, seq_lens, block_table, cos_sin, <7 of the cache>, k_open, v_open, q, q_out, positions, pairing,
// dev_status, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 21, [&] {
        const at::Tensor& k = tensor(a[0], "k");
        const at::Device dev = k.device();
        const Pages p = pages(a + 6, dev);
        const at::Tensor& bt = table(a[4]);
        const int64_t T = k.dim() ? k.size(0) : 0, B = bt.size(0);
        int64_t ks, vs, qs = 0;
        void* kp = rows(a[0], dev, T, p.H, p.d, &ks, "k");
        void* vp = rows(a[1], dev, T, p.H, p.d, &vs, "v");
        void *qp = nullptr, *op = nullptr;
        int64_t Hq = p.H;
        if (a[15] != Py_None) {
            const at::Tensor& q = tensor(a[15], "q");
            Hq = q.dim() == 3 ? q.size(1) : 0;
            qp = rows(a[15], dev, T, Hq, p.d, &qs, "q");
            op = like(a[16], dev, at::kBFloat16, {T, Hq, p.d}, "q_out");
        } else if (a[16] != Py_None) {
            throw Refused{"q_out without q"};
        }
        int64_t max_pos = 0, rot = 0;
        const float* cs = nullptr;
        if (a[5] != Py_None) {
            const at::Tensor& t = tensor(a[5], "cos_sin");
            if (t.dim() != 2) throw Refused{"cos_sin: want fp32 [max_pos, rot_dim], got " + describe(t)};
            max_pos = t.size(0);
            rot = t.size(1);
            cs = (const float*)like(a[5], dev, at::kFloat, {max_pos, rot}, "cos_sin");
        }
        const int32_t* cu = (const int32_t*)like(a[2], dev, at::kInt, {B + 1}, "cu_tokens");
        const int32_t* sl = (const int32_t*)like(a[3], dev, at::kInt, {B}, "seq_lens");
        const int32_t* tb = (const int32_t*)like(a[4], dev, at::kInt, {B, bt.size(1)}, "block_table");
        float* ko = (float*)like(a[13], dev, at::kFloat, {B, 16, p.H, p.d}, "k_open");
        void* vo = like(a[14], dev, at::kBFloat16, {B, 16, p.H, p.d}, "v_open");
        const int32_t* ps = a[17] == Py_None ? nullptr : (const int32_t*)like(a[17], dev, at::kInt, {T}, "positions");
        const int pairing = small(a[18], "pairing"), iB = extent(B, "B"), iT = extent(T, "T"), iH = extent(Hq, "H_q"),
                  ir = extent(rot, "rot_dim"), im = extent(max_pos, "max_pos"), mp = extent(bt.size(1), "pages");
        int32_t* st = status(a[19], dev);
        return on_device(dev, a[20], [&](void* stream) {
            return bdfp8_append(kp, ks, vp, vs, qp, qs, op, cu, sl, ps, cs, ir, im, pairing, ko, vo, tb, iB, iT, iH, p.H, p.d,
                                mp, p.num_pages, p.fmt, p.k, p.v, p.scales, st, stream);
        });
    });
}

// q, <7 of the cache>, block_table, seq_lens, sm_scale, chunk_tiles, workspace, out, window, sinks, dev_status, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 18, [&] {
        const at::Tensor& q = tensor(a[0], "q");
        const at::Device dev = q.device();
        const Pages p = pages(a + 1, dev);
        if (q.dim() != 4 || q.size(3) != p.d)
            throw Refused{"q: want bf16 [B, T_q, H_q, " + std::to_string(p.d) + "], got " + describe(q)};
        const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2);
        const at::Tensor& bt = table(a[8]);
        const void* qp = like(a[0], dev, at::kBFloat16, {B, T, Hq, p.d}, "q");
        const int32_t* tb = (const int32_t*)like(a[8], dev, at::kInt, {B, bt.size(1)}, "block_table");
        const int32_t* sl = (const int32_t*)like(a[9], dev, at::kInt, {B}, "seq_lens");
        void* out = like(a[13], dev, at::kBFloat16, {B, T, Hq, p.d}, "out");
        void* ws = nullptr;
        size_t wb = 0;
        if (a[12] != Py_None) {
            const at::Tensor& w = tensor(a[12], "workspace");
            if (w.device() != dev || !w.is_contiguous()) throw Refused{"workspace: want contiguous memory on " + dev.str()};
            ws = w.data_ptr();
            wb = w.nbytes();
        }
        const double scale = PyFloat_AsDouble(a[10]);
        if (scale == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Refused{"sm_scale: want a number"};
        }
        const int chunk = small(a[11], "chunk_tiles"), window = small(a[14], "window"), sinks = small(a[15], "sinks"),
                  iB = extent(B, "B"), iT = extent(T, "T_q"), iH = extent(Hq, "H_q"), mp = extent(bt.size(1), "pages");
        int32_t* st = status(a[16], dev);
        return on_device(dev, a[17], [&](void* stream) {
            return bdfp8_decode(qp, p.k, p.v, p.scales, tb, sl, iB, iT, iH, p.H, p.d, mp, p.num_pages, p.fmt, window, sinks,
                                (float)scale, chunk, ws, wb, out, st, stream);
        });
    });
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_XINCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bdfp8_py", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bdfp8_py(void) { return PyModule_Create(&kModule); }
