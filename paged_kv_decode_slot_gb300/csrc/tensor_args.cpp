// tensor_args.cpp - the binding's check of one tensor argument, as a Python extension: a step makes several calls of ten
// arguments each, some for a few microseconds of GPU work, and five attribute look-ups a tensor in Python take longer than
// the launch.  It holds no computation and launches nothing; binding.py's own _arg does the same where it is not built.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject *g_refuse = nullptr;  // binding._refuse(t, dtype, shape, name, dev): raises, or accepts pinned host memory

// arg(t, dtype, shape, name, dev) -> the address of a contiguous tensor of this type and shape on CUDA device dev
PyObject *arg(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "arg(t, dtype, shape, name, dev)");
        return nullptr;
    }
    if (THPVariable_Check(a[0]) && THPDtype_Check(a[1]) && PyTuple_Check(a[2])) {
        const at::Tensor &t = THPVariable_Unpack(a[0]);
        const long dev = PyLong_AsLong(a[4]);
        if (dev == -1 && PyErr_Occurred()) return nullptr;
        const auto sizes = t.sizes();
        bool same = t.scalar_type() == reinterpret_cast<THPDtype *>(a[1])->scalar_type && t.is_cuda() &&
                    t.get_device() == dev && PyTuple_GET_SIZE(a[2]) == (Py_ssize_t)sizes.size() && t.is_contiguous();
        for (size_t i = 0; same && i < sizes.size(); ++i) {
            const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(a[2], i));
            if (s == -1 && PyErr_Occurred()) return nullptr;
            same = s == sizes[i];
        }
        if (same) return PyLong_FromVoidPtr(t.data_ptr());
    }
    if (!g_refuse) {
        PyErr_SetString(PyExc_RuntimeError, "set_refuse was not called");
        return nullptr;
    }
    return PyObject_Vectorcall(g_refuse, a, 5, nullptr);
}

// maybe(t, ...): None for None
PyObject *maybe(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n == 5 && a[0] == Py_None) Py_RETURN_NONE;
    return arg(self, a, n);
}

PyObject *set_refuse(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(g_refuse, f);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"arg", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(arg)), METH_FASTCALL, nullptr},
    {"maybe", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(maybe)), METH_FASTCALL, nullptr},
    {"set_refuse", set_refuse, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_args() { return PyModule_Create(&module); }
