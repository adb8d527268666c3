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

// rows(tensor, name, dtype, n, head_dim, device) -> (address, elements between tokens, heads) of [n, heads, head_dim] whose
// heads are dense and whose tokens may lie inside wider rows; explain_rows() of the same arguments where it is not that
bool row_fits(PyObject* const* args, const void** address, long long* ld, long long* heads) {
    if (!THPVariable_Check(args[0]) || !THPDtype_Check(args[2])) return false;
    const long long n = PyLong_AsLongLong(args[3]), dim = PyLong_AsLongLong(args[4]), device = PyLong_AsLongLong(args[5]);
    if ((n == -1 || dim == -1 || device == -1) && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    try {
        const at::Tensor& t = THPVariable_Unpack(args[0]);
        if (t.get_device() != device || t.scalar_type() != reinterpret_cast<THPDtype*>(args[2])->scalar_type || t.dim() != 3)
            return false;
        const auto sizes = t.sizes(), strides = t.strides();
        *heads = sizes[1];
        *ld = n <= 1 || *heads == 0 ? *heads * dim : strides[0];  // (a stride that is never taken)
        if (sizes[0] != n || sizes[2] != dim || strides[2] != 1 || (*heads > 1 && strides[1] != dim) || *ld < *heads * dim)
            return false;
        *address = t.mutable_data_ptr();
        return true;
    } catch (...) {
        return false;
    }
}

PyObject* g_explain_rows = nullptr;

PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "rows takes a tensor, its name, dtype, tokens, head_dim and device");
        return nullptr;
    }
    const void* p = nullptr;
    long long ld = 0, heads = 0;
    if (row_fits(args, &p, &ld, &heads)) return Py_BuildValue("NLL", PyLong_FromVoidPtr(const_cast<void*>(p)), ld, heads);
    if (!g_explain_rows) {
        PyErr_SetString(PyExc_RuntimeError, "explain_rows is not set");
        return nullptr;
    }
    return PyObject_Vectorcall(g_explain_rows, args, (size_t)n, nullptr);
}

PyObject* explain_rows(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XDECREF(g_explain_rows);
    g_explain_rows = f;
    Py_RETURN_NONE;
}

PyObject* explain(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XDECREF(g_explain);
    g_explain = f;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(ptr)), METH_FASTCALL, nullptr},
                         {"explain", explain, METH_O, nullptr},
                         {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rows)), METH_FASTCALL, nullptr},
                         {"explain_rows", explain_rows, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
