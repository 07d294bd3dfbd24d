// Checks of torch tensors for the binding of include/attention.h: the device
// pointer of a tensor of the expected type, shape and strides.  A call of
// qk_rope_forward checks seven tensors; in Python that took 2.4 of the 7.2 us
// that the call costs the host.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// The i-th entry of a tuple of ints, -1 if it is none.
int64_t entry(PyObject* tuple, Py_ssize_t i) {
    const int64_t v = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (v == -1 && PyErr_Occurred()) PyErr_Clear();
    return v;
}

// tensor(t, what, dtype, shape, strides): strides None stands for a dense
// tensor; dimensions of length 1 may have any stride.  t None gives None.
PyObject* check(PyObject* const* args, Py_ssize_t n) {
    if (n != 5 || !PyUnicode_Check(args[1]) || !THPDtype_Check(args[2]) || !PyTuple_Check(args[3]) ||
        !(args[4] == Py_None || PyTuple_Check(args[4]))) {
        PyErr_SetString(PyExc_TypeError, "tensor(t, what, dtype, shape, strides)");
        return nullptr;
    }
    if (args[0] == Py_None) Py_RETURN_NONE;
    const char* what = PyUnicode_AsUTF8(args[1]);
    if (!what) return nullptr;
    if (!THPVariable_Check(args[0]))
        return PyErr_Format(PyExc_TypeError, "%s: a GPU tensor expected, got %R", what, (PyObject*)Py_TYPE(args[0]));
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    if (t.scalar_type() != reinterpret_cast<THPDtype*>(args[2])->scalar_type || !t.is_cuda())
        return PyErr_Format(PyExc_TypeError, "%s: a GPU tensor of %R expected, got one of %s on %s", what, args[2],
                            c10::toString(t.scalar_type()), t.device().str().c_str());
    if (t.layout() != at::kStrided) return PyErr_Format(PyExc_TypeError, "%s: a strided tensor expected", what);
    const at::IntArrayRef sizes = t.sizes(), strides = t.strides();
    bool fits = (Py_ssize_t)sizes.size() == PyTuple_GET_SIZE(args[3]);
    for (size_t i = 0; fits && i < sizes.size(); ++i) fits = sizes[i] == entry(args[3], (Py_ssize_t)i);
    if (!fits) {
        PyObject* have = PyObject_GetAttrString(args[0], "shape");
        if (have) PyErr_Format(PyExc_ValueError, "%s: shape %S, expected %S", what, have, args[3]);
        Py_XDECREF(have);
        return nullptr;
    }
    if (args[4] == Py_None) {
        if (!t.is_contiguous()) return PyErr_Format(PyExc_ValueError, "%s: tensor must be contiguous", what);
    } else {
        fits = (Py_ssize_t)strides.size() == PyTuple_GET_SIZE(args[4]);
        for (size_t i = 0; fits && i < strides.size(); ++i)
            fits = sizes[i] <= 1 || strides[i] == entry(args[4], (Py_ssize_t)i);
        if (!fits) {
            PyObject* have = PyObject_CallMethod(args[0], "stride", nullptr);
            if (have) PyErr_Format(PyExc_ValueError, "%s: strides %S, the descriptor has %S", what, have, args[4]);
            Py_XDECREF(have);
            return nullptr;
        }
    }
    void* p = t.data_ptr();
    if (!p && t.numel() > 0) return PyErr_Format(PyExc_TypeError, "%s: a tensor without memory", what);
    return PyLong_FromVoidPtr(p);
}

// torch throws where a tensor has no plain sizes, strides or memory (symbolic
// sizes, a tensor under vmap); from a C entry that would end the process.
PyObject* tensor(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        return check(args, n);
    } catch (python_error& e) {
        e.restore();
        return nullptr;
    } catch (const c10::Error& e) {
        return PyErr_Format(PyExc_TypeError, "%S: %s", args[1], e.what_without_backtrace());
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_RuntimeError, "%S: %s", args[1], e.what());
    }
}

PyMethodDef methods[] = {{"tensor", (PyCFunction)(void (*)())tensor, METH_FASTCALL,
                          "tensor(t, what, dtype, shape, strides) -> device pointer"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
