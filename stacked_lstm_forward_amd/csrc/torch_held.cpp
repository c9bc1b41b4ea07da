// What torch's tensors are, read in one call for a list of them: a problem over
// hundreds of tensors asks before every launch whether each is still what it was
// made for.  From Python that is four attributes a tensor, 50 ns each (602 tensors:
// 190 us, longer than their kernels); here all four take 8 ns.
//
// Loaded with the GIL held (ctypes.PyDLL), built against the installed torch.
#include <Python.h>
#include <stdint.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

namespace {

struct Held {
  int64_t address, count;
  int32_t type, contiguous;
};

Held of(PyObject* o) {
  const at::Tensor& t = THPVariable_Unpack(o);
  return {(int64_t)(uintptr_t)t.data_ptr(), t.numel(), (int32_t)t.scalar_type(), (int32_t)t.is_contiguous()};
}

}  // namespace

extern "C" {

const char* lstm_held_torch() { return TORCH_VERSION; }

// Writes what each tensor of the tuple is; 0 if one cannot be read (or is none).
int lstm_held_read(PyObject* tensors, void* held) {
  try {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tensors); ++i) {
      PyObject* o = PyTuple_GET_ITEM(tensors, i);
      if (!THPVariable_Check(o)) return 0;
      ((Held*)held)[i] = of(o);
    }
    return 1;
  } catch (...) {
    return 0;
  }
}

// Whether each tensor of the tuple still is what lstm_held_read found.
int lstm_held_same(PyObject* tensors, const void* held) {
  try {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(tensors); ++i) {
      const Held now = of(PyTuple_GET_ITEM(tensors, i)), &was = ((const Held*)held)[i];
      if (now.address != was.address || now.count != was.count || now.type != was.type ||
          now.contiguous != was.contiguous)
        return 0;
    }
    return 1;
  } catch (...) {
    return 0;
  }
}

}  // extern "C"
