// host_tensors.cpp -- tensors that claim to live on a CUDA device, over host
// memory, for the tests of the Python binding's checks without a GPU.
#include <Python.h>

#include <ATen/ops/from_blob.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

// (address, shape, type: "f32" | "bf16" | "i32" | "i64", device index) -> tensor
PyObject *cuda_tensor(PyObject *, PyObject *args)
{
    HANDLE_TH_ERRORS
    unsigned long long address;
    PyObject *shape;
    const char *type;
    int device;
    if (!PyArg_ParseTuple(args, "KO!si", &address, &PyTuple_Type, &shape, &type, &device))
        return nullptr;
    std::vector<int64_t> sizes;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i)
        sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)));
    const std::string t = type;
    const at::ScalarType s = t == "f32" ? at::kFloat : t == "bf16" ? at::kBFloat16
                             : t == "i32" ? at::kInt : at::kLong;
    const at::Device d(at::kCUDA, c10::DeviceIndex(device));
    return THPVariable_Wrap(at::for_blob(reinterpret_cast<void *>(address), sizes)
                                .options(at::TensorOptions().dtype(s).device(d))
                                .target_device(d)
                                .make_tensor());
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"cuda_tensor", cuda_tensor, METH_VARARGS, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "host_tensors", nullptr, -1, methods};

} // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit_host_tensors(void)
{
    return PyModule_Create(&module);
}
