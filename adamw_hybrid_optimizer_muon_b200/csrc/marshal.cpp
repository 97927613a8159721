// Addresses and element counts of a list of torch tensors, as the arrays that
// the C entry points take: through Python's methods a tensor costs 60 ns a
// value, here about 2.
//
// A Python extension module, built against the installed torch and loaded with
// that torch and that Python alone (the versions are in the file's name); the
// binding goes through the methods where it is not there. Both functions raise
// TypeError when an item is not a plain tensor (the binding then does it the
// long way, with that way's errors).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <exception>

#include <torch/csrc/autograd/python_variable.h>

namespace {

template <typename F>
PyObject* each(PyObject* list, F value) {
    PyObject* seq = PySequence_Fast(list, "a sequence of tensors");
    if (!seq) return nullptr;
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    PyObject* out = PyByteArray_FromStringAndSize(nullptr, 8 * n);
    bool ok = out != nullptr;
    int64_t* v = ok ? reinterpret_cast<int64_t*>(PyByteArray_AS_STRING(out)) : nullptr;
    try {
        for (Py_ssize_t i = 0; ok && i < n; ++i) {
            PyObject* t = PySequence_Fast_GET_ITEM(seq, i);
            if ((ok = THPVariable_Check(t))) v[i] = value(THPVariable_Unpack(t));
        }
    } catch (const std::exception&) {
        ok = false;
    }
    Py_DECREF(seq);
    if (ok) return out;
    Py_XDECREF(out);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "not a plain tensor");
    return nullptr;
}

PyObject* pointers(PyObject*, PyObject* list) {
    return each(list, [](const at::Tensor& t) { return (int64_t)reinterpret_cast<intptr_t>(t.data_ptr()); });
}

PyObject* numels(PyObject*, PyObject* list) {
    return each(list, [](const at::Tensor& t) { return (int64_t)t.numel(); });
}

PyMethodDef methods[] = {
    {"pointers", pointers, METH_O, "data_ptr() of every tensor of a sequence, 8 bytes each, as a bytearray"},
    {"numels", numels, METH_O, "numel() of every tensor of a sequence, 8 bytes each, as a bytearray"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
