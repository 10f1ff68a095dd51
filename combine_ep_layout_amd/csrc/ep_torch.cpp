// CPython helper of the binding: checks a list of tensors and collects their
// addresses in one pass.  An optimiser step takes hundreds of tensors in four
// or more lists; asking each for its type, device, layout, length and address
// from Python took 0.35 ms for 300 tensors, ten times the step itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// What was wrong, as gather() returns it.
enum Wrong { kNone, kLength, kTensor, kType, kDevice, kContiguous, kNumel };

// gather(tensors, dtype, device_index, sizes, count, per, out, stride) -> (what was wrong, which tensor)
//   sizes: address of int64 [count]; with per == 0 it receives the tensors'
//   lengths, else tensor i must hold ceil(sizes[i] / per) values.
//   out: address of the first tensor's place, stride bytes between places.
PyObject* gather(PyObject*, PyObject* args) {
    PyObject *list, *dtype;
    int device;
    Py_ssize_t count;
    unsigned long long sizes_at, out_at, stride;
    long long per;
    if (!PyArg_ParseTuple(args, "OOiKnLKK", &list, &dtype, &device, &sizes_at, &count, &per, &out_at, &stride)) return nullptr;
    if (!THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "dtype");
        return nullptr;
    }
    const at::ScalarType type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    int64_t* const sizes = reinterpret_cast<int64_t*>(sizes_at);
    PyObject* const seq = PySequence_Fast(list, "a list of tensors");
    if (!seq) return nullptr;
    int wrong = kNone;
    Py_ssize_t i = 0;
    if (PySequence_Fast_GET_SIZE(seq) != count) wrong = kLength;
    PyObject** const items = PySequence_Fast_ITEMS(seq);
    try {
        for (; wrong == kNone && i < count; ++i) {
            if (!THPVariable_Check(items[i])) wrong = kTensor;
            else {
                const at::Tensor& t = THPVariable_Unpack(items[i]);
                if (t.layout() != at::kStrided) wrong = kTensor;
                else if (t.scalar_type() != type) wrong = kType;
                else if (!t.is_cuda() || t.get_device() != device) wrong = kDevice;
                else if (!t.is_contiguous()) wrong = kContiguous;
                else {
                    if (per == 0) sizes[i] = t.numel();
                    else if (t.numel() != (sizes[i] + per - 1) / per) wrong = kNumel;
                    *reinterpret_cast<uint64_t*>(out_at + static_cast<unsigned long long>(i) * stride) =
                        reinterpret_cast<uint64_t>(t.numel() ? t.data_ptr() : nullptr);
                }
            }
            if (wrong != kNone) break;
        }
    } catch (const std::exception& e) {         // a tensor without memory of its own
        Py_DECREF(seq);
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_DECREF(seq);
    return Py_BuildValue("in", wrong, i);
}

PyMethodDef methods[] = {{"gather", gather, METH_VARARGS, "Checks tensors and collects their addresses."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ep_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ep_torch() { return PyModule_Create(&module); }
