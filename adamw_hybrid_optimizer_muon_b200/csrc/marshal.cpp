// Addresses and element counts of a list of torch tensors, as the arrays that
// the C entry points take: through Python's methods a tensor costs 60 ns a
// value, here about 2.
//
// A Python extension module, built against the installed torch and loaded with
// that torch and that Python alone (the versions are in the file's name); the
// binding goes through the methods where it is not there. The functions that
// make arrays raise TypeError when an item is not a plain tensor (the binding
// then does it the long way, with that way's errors).
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

// Whether a list's tensors are at the addresses, and have the counts, of two arrays that were made of it earlier.
PyObject* unchanged(PyObject*, PyObject* args) {
    PyObject *list, *ptrs, *counts;
    if (!PyArg_ParseTuple(args, "O!O!O!", &PyList_Type, &list, &PyByteArray_Type, &ptrs, &PyByteArray_Type, &counts))
        return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(list);
    if (PyByteArray_GET_SIZE(ptrs) != 8 * n || PyByteArray_GET_SIZE(counts) != 8 * n) Py_RETURN_FALSE;
    const int64_t* p = reinterpret_cast<const int64_t*>(PyByteArray_AS_STRING(ptrs));
    const int64_t* c = reinterpret_cast<const int64_t*>(PyByteArray_AS_STRING(counts));
    bool same = true;
    try {
        for (Py_ssize_t i = 0; same && i < n; ++i) {
            PyObject* item = PyList_GET_ITEM(list, i);
            if (!(same = THPVariable_Check(item))) break;
            const at::Tensor& t = THPVariable_Unpack(item);
            same = (int64_t) reinterpret_cast<intptr_t>(t.const_data_ptr()) == p[i] && (int64_t)t.numel() == c[i];
        }
    } catch (const std::exception&) {
        same = false;
    }
    if (same) Py_RETURN_TRUE;
    Py_RETURN_FALSE;
}

PyMethodDef methods[] = {
    {"pointers", pointers, METH_O, "data_ptr() of every tensor of a sequence, 8 bytes each, as a bytearray"},
    {"numels", numels, METH_O, "numel() of every tensor of a sequence, 8 bytes each, as a bytearray"},
    {"unchanged", unchanged, METH_VARARGS, "whether (list, pointers, numels) still belong together"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
