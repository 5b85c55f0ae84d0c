// binding.cpp -- the argument checks of a decoding call in one native call.
//
// A step of a small batch takes 10 to 20 us on the GPU and has up to 16 tensor
// arguments; reading type, shape, device, layout and address of one from Python
// takes 0.45 us.  pointers() does it for all of them at once (host time of a call:
// commit 15.3 -> 8.2 us, tree step 17.7 -> 11.2, slot map 9.7 -> 7.1).  It knows the
// usual case only: what it does not accept, the caller looks at again in Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// Is t a dense CUDA tensor of this type and shape (None: any)?
bool fits(const at::Tensor &t, PyObject *dtype, PyObject *shape) {
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous() || t.numel() == 0) return false;
    if (!THPDtype_Check(dtype) || reinterpret_cast<THPDtype *>(dtype)->scalar_type != t.scalar_type()) return false;
    if (shape == Py_None) return true;
    if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
    for (int64_t i = 0; i < t.dim(); ++i)
        if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != t.size(i)) return false;   // -1 on an error fits no size
    return true;
}

// pointers(plan, ws, *tensors): plan is a tuple of (name, dtype, shape or None,
// may be None), one for each tensor.  Returns their addresses (None for a
// tensor that may be and is None), then the workspace's address, bytes and
// device index; or None when an argument is not as the plan says.
PyObject *pointers(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 2 || !PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != n - 2) {
        PyErr_SetString(PyExc_TypeError, "pointers(plan, ws, *tensors): one tensor for each entry of the plan");
        return nullptr;
    }
    if (!THPVariable_CheckExact(args[1])) Py_RETURN_NONE;
    const at::Tensor &ws = THPVariable_Unpack(args[1]);
    if (!ws.defined() || !ws.is_cuda() || ws.layout() != at::kStrided || !ws.is_contiguous() || ws.numel() == 0 ||
        ws.scalar_type() != at::kByte)
        Py_RETURN_NONE;
    const Py_ssize_t m = n - 2;
    PyObject *out = PyTuple_New(m + 3);
    if (!out) return nullptr;
    bool ok = true;
    for (Py_ssize_t i = 0; ok && i < m; ++i) {
        PyObject *spec = PyTuple_GET_ITEM(args[0], i), *o = args[2 + i], *p = nullptr;
        ok = PyTuple_Check(spec) && PyTuple_GET_SIZE(spec) == 4;
        if (!ok) break;
        if (o == Py_None && PyTuple_GET_ITEM(spec, 3) == Py_True) {
            p = Py_None;
            Py_INCREF(p);
        } else if (THPVariable_CheckExact(o)) {
            const at::Tensor &t = THPVariable_Unpack(o);
            if (fits(t, PyTuple_GET_ITEM(spec, 1), PyTuple_GET_ITEM(spec, 2)) && t.get_device() == ws.get_device())
                p = PyLong_FromVoidPtr(t.data_ptr());
        }
        ok = p != nullptr;
        if (ok) PyTuple_SET_ITEM(out, i, p);
    }
    if (ok) {
        PyObject *tail[3] = {PyLong_FromVoidPtr(ws.data_ptr()), PyLong_FromLongLong(ws.numel()), PyLong_FromLong(ws.get_device())};
        for (int i = 0; i < 3; ++i) {
            ok = ok && tail[i];
            if (tail[i]) PyTuple_SET_ITEM(out, m + i, tail[i]);
        }
    }
    if (ok) return out;
    Py_DECREF(out);
    PyErr_Clear();
    Py_RETURN_NONE;
}

// No C++ exception leaves the module (data_ptr() and the like may throw).
PyObject *pointers_guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    try {
        return pointers(self, args, n);
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyMethodDef methods[] = {{"pointers", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(pointers_guarded)), METH_FASTCALL,
                          "Addresses of tensors that are as their plan says, else None."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch and the Python of the headers above (at::Tensor's layout is
// compiled in), which the caller compares with those that run.
PyMODINIT_FUNC PyInit__binding() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", RAT_BUILT_FOR) < 0) {
        Py_DECREF(m);
        m = nullptr;
    }
    return m;
}
