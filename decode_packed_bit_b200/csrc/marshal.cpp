// marshal.cpp -- what the Python binding of the decode-side calls does per
// operand and per call, compiled: these calls take 2 to 10 us on the GPU, and
// checking an operand from Python took 0.55 us, handing over 20 arguments
// through ctypes 2.7.  The module checks a tensor and gives its address, and
// calls an entry point that takes its arguments as a block of 64-bit words.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>

namespace {

constexpr int kMaxWords = 128;

PyObject *refuse(PyObject *t, PyObject *dtype, PyObject *shape, PyObject *what, const char *form, long long dev)
{
    PyObject *d = PyObject_GetAttrString(t, "dtype"), *s = PyObject_GetAttrString(t, "shape");
    PyObject *st = PyObject_CallMethod(t, "stride", nullptr), *at = PyObject_GetAttrString(t, "device");
    if (d && s && st && at) {
        PyObject *dims = PySequence_Tuple(s);
        if (dims)
            PyErr_Format(PyExc_ValueError, "%S: expected a %S tensor of shape %S %s on cuda:%lld, got %S %S with strides %S on %S", what,
                         dtype, shape, form, dev, d, dims, st, at);
        Py_XDECREF(dims);
    }
    Py_XDECREF(d);
    Py_XDECREF(s);
    Py_XDECREF(st);
    Py_XDECREF(at);
    return nullptr;
}

// (t, dtype or a tuple of them, shape, what, device): whether t is a tensor of this type and shape there.
bool fits(PyObject *const *args, Py_ssize_t n, const at::Tensor *&t, long long &dev, bool &error)
{
    error = true;
    if (n != 5 || !THPVariable_Check(args[0]) || !PyTuple_Check(args[2])) {
        PyErr_SetString(PyExc_TypeError, "expected (tensor, dtype, shape tuple, name, device)");
        return false;
    }
    dev = PyLong_AsLongLong(args[4]);
    if (dev == -1 && PyErr_Occurred()) return false;
    t = &THPVariable_Unpack(args[0]);
    const Py_ssize_t dims = PyTuple_GET_SIZE(args[2]);
    PyObject *type = reinterpret_cast<PyObject *>(torch::getTHPDtype(t->scalar_type()));
    bool typed = type == args[1];
    if (PyTuple_Check(args[1]))  // any of these
        for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(args[1]); ++i) typed |= type == PyTuple_GET_ITEM(args[1], i);
    bool ok = typed && t->layout() == at::kStrided && t->is_cuda() && t->get_device() == dev && t->dim() == dims;
    for (Py_ssize_t i = 0; ok && i < dims; ++i) {
        const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(args[2], i));
        if (v == -1 && PyErr_Occurred()) return false;
        ok = t->size(i) == v;
    }
    error = false;
    return ok;
}

PyObject *dense(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS  // a tensor without storage throws
    const at::Tensor *t;
    long long dev;
    bool error;
    const bool ok = fits(args, n, t, dev, error);
    if (error) return nullptr;
    if (!ok || !t->is_contiguous()) return refuse(args[0], args[1], args[2], args[3], "(contiguous)", dev);
    return PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t->data_ptr()));
    END_HANDLE_TH_ERRORS
}

// A [rows][heads][dim] tensor whose rows are dense and may lie apart: address and row stride.
PyObject *rows(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS  // a tensor without storage throws
    const at::Tensor *t;
    long long dev;
    bool error;
    const bool ok = fits(args, n, t, dev, error);
    if (error) return nullptr;
    long long stride = 0;
    bool good = ok && t->dim() == 3;
    if (good && t->is_contiguous())
        stride = t->size(1) * t->size(2);
    else if (good && t->stride(2) == 1 && (t->stride(1) == t->size(2) || t->size(1) <= 1))
        stride = t->stride(0);
    else
        good = false;
    if (!good) return refuse(args[0], args[1], args[2], args[3], "(dense rows)", dev);
    PyObject *out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, PyLong_FromUnsignedLongLong(reinterpret_cast<uintptr_t>(t->data_ptr())));
    PyTuple_SET_ITEM(out, 1, PyLong_FromLongLong(stride));
    return out;
    END_HANDLE_TH_ERRORS
}

// (t, device): address and bytes of a workspace, (0, 0) for None.
PyObject *scratch(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS  // a tensor without storage throws
    if (n != 2 || (args[0] != Py_None && !THPVariable_Check(args[0]))) {
        PyErr_SetString(PyExc_TypeError, "workspace: expected a tensor or None");
        return nullptr;
    }
    const long long dev = PyLong_AsLongLong(args[1]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    unsigned long long at = 0, bytes = 0;
    if (args[0] != Py_None) {
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous()) {
            PyErr_Format(PyExc_ValueError, "workspace: expected a contiguous tensor on cuda:%lld", dev);
            return nullptr;
        }
        at = reinterpret_cast<uintptr_t>(t.data_ptr());
        bytes = t.nbytes();
    }
    PyObject *out = PyTuple_New(2);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, PyLong_FromUnsignedLongLong(at));
    PyTuple_SET_ITEM(out, 1, PyLong_FromUnsignedLongLong(bytes));
    return out;
    END_HANDLE_TH_ERRORS
}

// (address of a function that takes a block, words...): integers, floats (as a double's bits), None (0).
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n < 1 || n > kMaxWords) {
        PyErr_SetString(PyExc_TypeError, "expected a function's address and at most 127 words");
        return nullptr;
    }
    int64_t block[kMaxWords] = {};
    const unsigned long long f = PyLong_AsUnsignedLongLong(args[0]);
    if (PyErr_Occurred()) return nullptr;
    for (Py_ssize_t i = 1; i < n; ++i) {
        if (PyLong_Check(args[i])) {
            block[i - 1] = PyLong_AsLongLong(args[i]);
        } else if (args[i] == Py_None) {
            block[i - 1] = 0;
        } else if (PyFloat_Check(args[i])) {
            const double d = PyFloat_AS_DOUBLE(args[i]);
            std::memcpy(&block[i - 1], &d, sizeof(d));
        } else {
            PyErr_Format(PyExc_TypeError, "word %zd: expected an int, a float or None, got %R", i, args[i]);
        }
        if (PyErr_Occurred()) return nullptr;
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<int (*)(const int64_t *)>(static_cast<uintptr_t>(f))(block);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

PyMethodDef methods[] = {
    {"dense", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dense)), METH_FASTCALL,
     "dense(t, dtype, shape, what, device) -> the address of a contiguous CUDA tensor, or ValueError"},
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL,
     "rows(t, dtype, shape, what, device) -> (address, row stride) of a tensor with dense rows, or ValueError"},
    {"scratch", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scratch)), METH_FASTCALL,
     "scratch(t, device) -> (address, bytes) of a workspace, or ValueError"},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "call(function address, *words) -> the status of the function, called with the words as its block"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Operand checks and calls of the decode-side entry points.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
