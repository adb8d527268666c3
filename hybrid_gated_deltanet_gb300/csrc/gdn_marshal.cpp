// gdn_marshal.cpp -- a call's tensors, checked natively: ptr(tensor, name, dtype, shape, device) is the tensor's
// address if it is a dense tensor of that dtype, shape and device.  If it is not, explain() of the same arguments
// raises the error (it is written in Python, where the messages are).  A call made once per layer and step has up to
// 14 tensors, and 0.5 us for each of them in Python was more than the launch (the host's part of a verify of one tree:
// 12.5 us, now 8.3; of an append 7.8, now 5.5).
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* g_explain = nullptr;

// never throws: what has no plain sizes or storage (a subclass without them) does not fit
bool fits(PyObject* const* args, const void** address) {
    if (!THPVariable_Check(args[0]) || !THPDtype_Check(args[2]) || !PyTuple_Check(args[3])) return false;
    const long device = PyLong_AsLong(args[4]);
    if (device == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    try {
        const at::Tensor& t = THPVariable_Unpack(args[0]);
        if (t.get_device() != device || t.scalar_type() != reinterpret_cast<THPDtype*>(args[2])->scalar_type ||
            !t.is_contiguous())
            return false;
        const auto sizes = t.sizes();
        if ((Py_ssize_t)sizes.size() != PyTuple_GET_SIZE(args[3])) return false;
        for (size_t i = 0; i < sizes.size(); ++i) {
            const long long want = PyLong_AsLongLong(PyTuple_GET_ITEM(args[3], (Py_ssize_t)i));
            if (want == -1 && PyErr_Occurred()) {
                PyErr_Clear();
                return false;
            }
            if (sizes[i] != want) return false;
        }
        *address = t.mutable_data_ptr();  // (an empty tensor may have none)
        return true;
    } catch (...) {
        return false;
    }
}

PyObject* ptr(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "ptr takes a tensor, its name, dtype, shape and device");
        return nullptr;
    }
    const void* p = nullptr;
    if (fits(args, &p)) return PyLong_FromVoidPtr(const_cast<void*>(p));
    if (!g_explain) {
        PyErr_SetString(PyExc_RuntimeError, "explain is not set");
        return nullptr;
    }
    return PyObject_Vectorcall(g_explain, args, (size_t)n, nullptr);
}

PyObject* explain(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XDECREF(g_explain);
    g_explain = f;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL, nullptr},
                         {"explain", explain, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
