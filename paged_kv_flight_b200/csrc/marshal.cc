// marshal.cc -- the Python binding's argument checks and calls without the
// interpreter's share (module paged_kv_flight_b200._marshal; pkv.py does the
// same in Python where it is not built, and raises the errors in any case).
//
// The calls of a small step are bound by the host: with the checks in Python
// and the call through ctypes pkv_slot_map took 10.4 us, of which the kernel's
// launch is 2 to 3.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

// pointer(x, kind, size, ...): the device address of a contiguous CUDA tensor
// of the kind's element type and these sizes (-1: any; none given: any shape),
// or None: then the caller looks closer.
// kind 0: int32, 1: bf16, 2: a pool (bf16, uint8 or E4M3 codes), 3: float32; plus
// 4 (g + 1) where only tensors on cuda:g will do.
PyObject* pointer_of(PyObject* const* args, Py_ssize_t n)
{
    if (n < 2) {
        PyErr_SetString(PyExc_TypeError, "pointer(x, kind, sizes...)");
        return nullptr;
    }
    if (!THPVariable_CheckExact(args[0])) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(args[0]);
    const long code = PyLong_AsLong(args[1]), kind = code & 3, device = (code >> 2) - 1;
    if (code == -1 && PyErr_Occurred()) return nullptr;
    const at::ScalarType s = t.scalar_type();
    const bool type = kind == 0   ? s == at::kInt
                      : kind == 1 ? s == at::kBFloat16
                      : kind == 2 ? s == at::kBFloat16 || s == at::kByte || s == at::kFloat8_e4m3fn
                                  : kind == 3 && s == at::kFloat;
    if (!type || !t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) Py_RETURN_NONE;
    if (device >= 0 && t.get_device() != device) Py_RETURN_NONE;
    if (n > 2) {
        if (t.dim() != n - 2) Py_RETURN_NONE;
        for (Py_ssize_t i = 2; i < n; ++i) {
            const long long want = PyLong_AsLongLong(args[i]);
            if (want == -1 && PyErr_Occurred()) return nullptr;
            if (want != -1 && want != t.size(i - 2)) Py_RETURN_NONE;
        }
    }
    return PyLong_FromUnsignedLongLong(reinterpret_cast<unsigned long long>(t.data_ptr()));
}

// Tensors without storage (inside torch.func's transforms) throw when asked for
// their address: an exception must not pass through the interpreter.
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    try {
        return pointer_of(args, n);
    } catch (const std::exception&) {
        Py_RETURN_NONE;
    }
}

// call(address, a, ...): the C function at the address with up to 20 integers
// or pointers (None: NULL).  Each takes a whole register or stack slot, whatever
// its width (System V x86-64), of which the function reads what it declares.
constexpr int kMaxArgs = 20;
using Word = unsigned long long;
using Function = int (*)(Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word, Word,
                         Word, Word, Word, Word);

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n < 1 || n > kMaxArgs + 1) {
        PyErr_SetString(PyExc_TypeError, "call(address, up to 20 integers)");
        return nullptr;
    }
    Word a[kMaxArgs + 1] = {};
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (args[i] == Py_None) continue;
        a[i] = PyLong_AsUnsignedLongLongMask(args[i]);
        if (a[i] == ~Word(0) && PyErr_Occurred()) return nullptr;
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = reinterpret_cast<Function>(a[0])(a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12],
                                              a[13], a[14], a[15], a[16], a[17], a[18], a[19], a[20]);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

PyMethodDef methods[] = {
    {"pointer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pointer)), METH_FASTCALL, nullptr},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this was built against (build.py compares it before it keeps the file,
// pkv.py before it uses the module).
#ifndef PKV_STAMP
#error "PKV_STAMP: the versions of torch and Python, from build.py"
#endif

PyMODINIT_FUNC PyInit__marshal()
{
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", PKV_STAMP) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
