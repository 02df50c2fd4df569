// marshal.cpp -- the binding's tensor checks and calls as compiled code.
//
// A small call is bound by the host: checking an argument from Python costs
// about 0.45 us, a ctypes call 0.5 to 1.3 us, the launch itself 2.5 us.  Here
// a tensor's check takes some 10 ns.  What an entry point takes is described
// once by abi.py (names, dtypes, shapes as expressions of the descriptor's
// fields); this module compares and calls, and abi.py words the errors.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <memory>
#include <utility>
#include <vector>

namespace {

// value = (a < 0 ? 1 : fields[a]) * (b < 0 ? 1 : fields[b]) / div + add, or
// only `add` where a < 0.
struct Dim {
    int a, b, div, add;
};
enum Kind { kRows = 0, kF32 = 1, kI32 = 2, kU8 = 3, kWorkspace = 4 };
struct Arg {
    int kind;
    bool optional;
    std::vector<Dim> shape;
};
struct Spec {
    void *fn;
    int fields, dtype_at;  // ints of the descriptor, and the one that is the rows' dtype
    std::vector<Arg> args;
};
constexpr const char *kName = "beam_spec";
constexpr int kMaxArgs = 20;

void free_spec(PyObject *capsule) {
    delete static_cast<Spec *>(PyCapsule_GetPointer(capsule, kName));
}

// spec(fn, fields, dtype_at, [(kind, optional, [(a, b, div, add), ...]), ...])
PyObject *make_spec(PyObject *, PyObject *args) try {
    unsigned long long fn;
    int fields, dtype_at;
    PyObject *list;
    if (!PyArg_ParseTuple(args, "KiiO!", &fn, &fields, &dtype_at, &PyList_Type, &list)) return nullptr;
    auto spec = std::make_unique<Spec>();
    spec->fn = reinterpret_cast<void *>(fn);
    spec->fields = fields;
    spec->dtype_at = dtype_at;
    Py_ssize_t slots = 2;  // descriptor and stream
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); ++i) {
        Arg arg;
        int optional;
        PyObject *dims;
        if (!PyArg_ParseTuple(PyList_GET_ITEM(list, i), "ipO!", &arg.kind, &optional, &PyList_Type, &dims))
            return nullptr;
        arg.optional = optional != 0;
        for (Py_ssize_t j = 0; j < PyList_GET_SIZE(dims); ++j) {
            Dim d;
            if (!PyArg_ParseTuple(PyList_GET_ITEM(dims, j), "iiii", &d.a, &d.b, &d.div, &d.add)) return nullptr;
            if (d.a >= fields || d.b >= fields || d.div < 1) {
                PyErr_SetString(PyExc_ValueError, "a shape outside the descriptor");
                return nullptr;
            }
            arg.shape.push_back(d);
        }
        slots += arg.kind == kWorkspace ? 2 : 1;
        spec->args.push_back(std::move(arg));
    }
    if (slots > kMaxArgs || dtype_at >= fields) {
        PyErr_SetString(PyExc_ValueError, "too many arguments");
        return nullptr;
    }
    PyObject *capsule = PyCapsule_New(spec.get(), kName, free_spec);
    if (capsule) spec.release();
    return capsule;
} catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
}

using P = void *;
// Every argument is a pointer or an integer: one register class, so the count
// alone makes the call's type.
template <size_t... I>
int call_n(void *fn, P *v, std::index_sequence<I...>) {
    return reinterpret_cast<int (*)(decltype(static_cast<void>(I), P())...)>(fn)(v[I]...);
}
int call(void *fn, P *v, int n) {
    switch (n) {
#define CASE(N) \
    case N: \
        return call_n(fn, v, std::make_index_sequence<N>());
        CASE(3) CASE(4) CASE(5) CASE(6) CASE(7) CASE(8) CASE(9) CASE(10) CASE(11) CASE(12)
        CASE(13) CASE(14) CASE(15) CASE(16) CASE(17) CASE(18) CASE(19) CASE(20)
#undef CASE
    }
    return 1;
}

at::ScalarType scalar_of(int kind) {
    return kind == kF32 ? at::kFloat : kind == kI32 ? at::kInt : at::kByte;
}

// The address of a contiguous CUDA tensor of this type and shape; false if it
// is another one.  *device: that of the first, which all others have to share.
bool address(PyObject *obj, at::ScalarType type, const long long *shape, size_t dims, int *device, P *out) {
    if (!THPVariable_Check(obj)) return false;
    const at::Tensor &t = THPVariable_Unpack(obj);
    // (a lazily negated view holds the other sign in memory)
    if (t.layout() != at::kStrided || t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous() || t.is_neg())
        return false;
    if (shape) {
        const auto sizes = t.sizes();
        if (sizes.size() != dims) return false;
        for (size_t i = 0; i < dims; ++i)
            if (sizes[i] != shape[i]) return false;
    }
    const int dev = t.get_device();
    if (*device < 0) {
        if (dev != c10::cuda::current_device()) return false;
        *device = dev;
    } else if (dev != *device) {
        return false;
    }
    *out = t.data_ptr();
    return true;
}

// The raw handle of a stream given as None (the current one), int or object.
bool stream_of(PyObject *stream, int device, P *out) {
    if (stream == Py_None) {
        *out = c10::cuda::getCurrentCUDAStream(device).stream();
        return true;
    }
    PyObject *raw = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
    if (!raw) return false;
    *out = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    return !PyErr_Occurred();
}

struct Buffer {  // given back on every way out, a torch error's too
    Py_buffer view;
    ~Buffer() { PyBuffer_Release(&view); }
};

// run(spec, descriptor, stream, tensors...): the entry point's status, or
// -(i + 1) where tensor i is not what the descriptor asks for.
PyObject *run(PyObject *, PyObject *const *argv, Py_ssize_t argc) {
    if (argc < 3) {
        PyErr_SetString(PyExc_TypeError, "spec, descriptor and stream are wanted");
        return nullptr;
    }
    const Spec *spec = static_cast<Spec *>(PyCapsule_GetPointer(argv[0], kName));
    if (!spec) return nullptr;
    if (size_t(argc - 3) != spec->args.size()) {
        PyErr_SetString(PyExc_TypeError, "another number of tensors");
        return nullptr;
    }
    Buffer held = {};
    Py_buffer &view = held.view;
    if (PyObject_GetBuffer(argv[1], &view, PyBUF_SIMPLE)) return nullptr;
    const int *f = static_cast<const int *>(view.buf);
    int status = 0, device = -1, n = 0;
    P v[kMaxArgs];
    if (view.len < Py_ssize_t(spec->fields * sizeof(int))) status = -1;
    v[n++] = view.buf;
    for (size_t i = 0; i < spec->args.size() && status == 0; ++i) {
        const Arg &a = spec->args[i];
        PyObject *obj = argv[3 + i];
        if (obj == Py_None && a.optional) {
            v[n++] = nullptr;
            continue;
        }
        long long shape[4];
        for (size_t j = 0; j < a.shape.size() && j < 4; ++j) {
            const Dim &d = a.shape[j];
            long long s = d.a < 0 ? 0 : f[d.a];
            if (d.b >= 0) s *= f[d.b];
            shape[j] = s / d.div + d.add;
        }
        const at::ScalarType type = a.kind == kRows ? (f[spec->dtype_at] == 0 ? at::kBFloat16 : at::kFloat)
                                    : a.kind == kWorkspace ? at::kByte : scalar_of(a.kind);
        if (!address(obj, type, a.kind == kWorkspace ? nullptr : shape, a.shape.size(), &device, &v[n])) {
            status = -int(i) - 1;
            break;
        }
        ++n;
        if (a.kind == kWorkspace)
            v[n++] = reinterpret_cast<P>(THPVariable_Unpack(obj).numel());
    }
    if (status == 0) {
        if (!stream_of(argv[2], device, &v[n++])) return nullptr;
        Py_BEGIN_ALLOW_THREADS;  // a full launch queue may make it wait
        status = call(spec->fn, v, n);
        Py_END_ALLOW_THREADS;
    }
    return PyLong_FromLong(status);
}

// rows(fn, quantize, values, codes, scales, n_rows, tiled, stream): the 4-bit
// row conversions, whose sizes are the values' own; status, or -1.
PyObject *rows(PyObject *, PyObject *const *argv, Py_ssize_t argc) {
    if (argc != 8) {
        PyErr_SetString(PyExc_TypeError, "eight arguments are wanted");
        return nullptr;
    }
    void *fn = PyLong_AsVoidPtr(argv[0]);
    const bool quantize = PyObject_IsTrue(argv[1]) == 1, tiled = PyObject_IsTrue(argv[6]) == 1;
    if (PyErr_Occurred()) return nullptr;
    int device = -1;
    P x, codes, scales, n_rows = nullptr, stream;
    if (!THPVariable_Check(argv[2])) return PyLong_FromLong(-1);
    const at::Tensor &t = THPVariable_Unpack(argv[2]);
    const auto type = t.scalar_type();
    if (t.dim() != 2 || (type != at::kBFloat16 && type != at::kFloat) || t.size(1) % 32 != 0 ||
        t.size(1) > 0x7fffffff)
        return PyLong_FromLong(-1);
    const long long r = t.size(0), c = t.size(1);
    const long long cs[2] = {r, c / 2}, ss[2] = {r, c / 32}, one[1] = {1};
    if (!address(argv[2], type, nullptr, 0, &device, &x) ||
        !address(argv[3], at::kByte, cs, 2, &device, &codes) ||
        !address(argv[4], at::kByte, ss, 2, &device, &scales) ||
        (argv[5] != Py_None && !address(argv[5], at::kInt, one, 1, &device, &n_rows)))
        return PyLong_FromLong(-1);
    if (!stream_of(argv[7], device, &stream)) return nullptr;
    const int dtype = type == at::kBFloat16 ? 0 : 1;
    int status;
    Py_BEGIN_ALLOW_THREADS;
    if (quantize)
        status = reinterpret_cast<int (*)(int, long long, int, P, P, P, P, int, P)>(fn)(
            dtype, r, int(c), x, n_rows, codes, scales, int(tiled), stream);
    else
        status = reinterpret_cast<int (*)(int, long long, int, P, P, int, P, P)>(fn)(
            dtype, r, int(c), codes, scales, int(tiled), x, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// A C++ exception (a torch error inside a check) must not leave a C entry.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *argv, Py_ssize_t argc) {
    try {
        return F(self, argv, argc);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"spec", make_spec, METH_VARARGS, nullptr},
    {"run", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<run>)), METH_FASTCALL, nullptr},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<rows>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
