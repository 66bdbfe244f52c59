// q8_lists.cpp -- a CPython module that turns a list of gradients into the
// q8_grad array that q8_grad_norm and q8_clip_grads take, with the checks that
// the binding owes them.  A list of 580 gradients and outputs takes 420 us in
// Python, a call of a method for each tensor and property, and 16 us here.
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "q8train.h"

namespace {

struct Refused {
    const char* what;
};

// A tensor's q8_dtype; checks that it is one that the library can take.
int32_t kind_of(const at::Tensor& t, const char* type_error, const char* layout_error, const char* device_error, int64_t* device)
{
    if (t.layout() != at::kStrided) throw Refused{layout_error};
    const at::ScalarType type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) throw Refused{type_error};
    if (!t.is_contiguous()) throw Refused{layout_error};
    if (!t.is_cuda() || (*device >= 0 && t.get_device() != *device)) throw Refused{device_error};
    *device = t.get_device();
    return type == at::kFloat ? Q8_F32 : Q8_BF16;
}

const at::Tensor& tensor_of(PyObject* o, const char* error)
{
    if (!THPVariable_Check(o)) throw Refused{error};
    return THPVariable_Unpack(o);
}

// pack(gradients, outputs or None) -> (bytes of the q8_grad array, device index or -1)
PyObject* pack(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 2) {
        PyErr_SetString(PyExc_TypeError, "pack takes two lists");
        return nullptr;
    }
    const bool in_place = args[1] == Py_None;
    PyObject* grads = PySequence_Fast(args[0], "gradients must be a sequence");
    PyObject* outs = !grads ? nullptr : in_place ? (Py_INCREF(Py_None), Py_None) : PySequence_Fast(args[1], "out must be a sequence");
    PyObject* bytes = nullptr;
    PyObject* result = nullptr;
    if (grads && outs) {
        try {
            const Py_ssize_t n = PySequence_Fast_GET_SIZE(grads);
            if (!in_place && PySequence_Fast_GET_SIZE(outs) != n)
                throw Refused{"out must hold a tensor of each gradient's number of elements"};
            bytes = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(q8_grad)));
            if (bytes) {
                auto* entry = reinterpret_cast<q8_grad*>(PyBytes_AS_STRING(bytes));
                int64_t device = -1;
                for (Py_ssize_t i = 0; i < n; ++i, ++entry) {
                    const at::Tensor& g = tensor_of(PySequence_Fast_GET_ITEM(grads, i), "gradients must be tensors");
                    entry->grad_dtype = kind_of(g, "gradients must be bfloat16 or float32", "gradients must be contiguous",
                                                "gradients must be CUDA tensors of one device", &device);
                    entry->numel = g.numel();
                    entry->grad = g.const_data_ptr();
                    if (in_place) {
                        entry->out = g.data_ptr();
                        entry->out_dtype = entry->grad_dtype;
                    } else {
                        const at::Tensor& o = tensor_of(PySequence_Fast_GET_ITEM(outs, i), "out must be tensors");
                        entry->out_dtype = kind_of(o, "out must be bfloat16 or float32", "out must be contiguous",
                                                   "out must be CUDA tensors of the gradients' device", &device);
                        if (o.numel() != entry->numel) throw Refused{"out must hold a tensor of each gradient's number of elements"};
                        entry->out = o.data_ptr();
                    }
                }
                result = Py_BuildValue("OL", bytes, static_cast<long long>(device));
            }
        } catch (const Refused& r) {
            PyErr_SetString(PyExc_ValueError, r.what);
        } catch (const std::exception& e) {
            PyErr_SetString(PyExc_RuntimeError, e.what());
        }
    }
    Py_XDECREF(bytes);
    Py_XDECREF(outs);
    Py_XDECREF(grads);
    return result;
}

PyMethodDef methods[] = {{"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pack)), METH_FASTCALL,
                          "pack(gradients, outputs or None) -> (q8_grad array as bytes, device index or -1)"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "q8_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_q8_lists() { return PyModule_Create(&module); }
