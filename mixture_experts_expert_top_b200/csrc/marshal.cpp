// marshal.cpp -- the binding's tensor checks in one call (Python module
// _marshal): type, size, contiguity and device of every tensor of an entry
// point, and their addresses. Marshalling only, as the rest of the binding: in
// Python the checks take 0.3 us per tensor, longer in sum than the launch of a
// kernel that serves one token.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

namespace {

// Address of argument p, a new reference; nullptr, without a Python error, if it
// is a tensor that does not fit. As Tensor.data_ptr() does, a tensor that still
// shares its storage lazily with another is given its own first: the kernels
// write through these addresses.
PyObject *address(PyObject *p, long dev, PyObject *elements, PyObject *code) {
    if (p == Py_None || PyLong_CheckExact(p)) {
        Py_INCREF(p);
        return p;
    }
    if (!THPVariable_Check(p)) return nullptr;
    const long long n = PyLong_AsLongLong(elements);
    const long type = PyLong_AsLong(code);
    if ((n == -1 || type == -1) && PyErr_Occurred()) return nullptr;
    try {
        const at::Tensor &t = THPVariable_Unpack(p);
        if (t.layout() == c10::kStrided && static_cast<long>(t.scalar_type()) == type && t.is_cuda() &&
            t.get_device() == dev && t.numel() >= n && t.is_contiguous())
            return PyLong_FromVoidPtr(t.mutable_data_ptr());
    } catch (const std::exception &e) {                          // no C++ exception crosses into the interpreter
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// addresses(dev, t0, n0, type0, t1, n1, type1, ...): a tuple of the tensors'
// addresses. None and ints pass as they are. None in the place of the tuple if
// a tensor has another element type (a c10::ScalarType code), fewer than n
// elements, gaps, or is not on CUDA device dev: the caller says what is wrong.
PyObject *addresses(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs < 1 || (nargs - 1) % 3) {
        PyErr_SetString(PyExc_TypeError, "addresses(dev, tensor, elements, type, ...)");
        return nullptr;
    }
    const long dev = PyLong_AsLong(args[0]);
    if (dev == -1 && PyErr_Occurred()) return nullptr;
    PyObject *out = PyTuple_New((nargs - 1) / 3);
    if (!out) return nullptr;
    for (Py_ssize_t i = 1; i < nargs; i += 3) {
        PyObject *a = address(args[i], dev, args[i + 1], args[i + 2]);
        if (!a) {
            Py_DECREF(out);
            if (PyErr_Occurred()) return nullptr;
            Py_RETURN_NONE;
        }
        PyTuple_SET_ITEM(out, (i - 1) / 3, a);
    }
    return out;
}

PyMethodDef kMethods[] = {{"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(addresses)), METH_FASTCALL,
                           "Checked addresses of tensors, or None."},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
