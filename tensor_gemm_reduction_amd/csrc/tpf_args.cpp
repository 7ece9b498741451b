// Checks of a call's tensors, their addresses, and its output tensors, for the
// Python binding.
//
// A decode step's kernels run for a few microseconds; looking at each of a
// call's tensors from Python takes about half of one, here 20 ns, and making a
// tensor there takes about 1.5, here a third of that (a 4-bit product over 8
// shards, 16 tokens: 31 us a call before, 22 after, 3 of them in each unbind of
// the caller's).
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/Context.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>

#include <exception>
#include <vector>

namespace {

// One group: (sequence of tensors, dtype, shape).  Appends the tensors'
// addresses to `out`; false when one is not a contiguous tensor of that dtype
// and shape on GPU `device`.
bool addresses(PyObject* seq, PyObject* dtype, PyObject* shape, long device, PyObject** out) {
  if (!THPDtype_Check(dtype) || !PyTuple_Check(shape)) return false;
  const auto type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
  int64_t want[8];
  if (dims > 8) return false;
  for (Py_ssize_t i = 0; i < dims; ++i) {
    want[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (want[i] == -1 && PyErr_Occurred()) return false;
  }
  PyObject* fast = PySequence_Fast(seq, "expected a sequence of tensors");
  if (!fast) return false;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
  PyObject* bytes = PyBytes_FromStringAndSize(nullptr, n * (Py_ssize_t)sizeof(void*));
  bool ok = bytes != nullptr;
  void** to = ok ? reinterpret_cast<void**>(PyBytes_AS_STRING(bytes)) : nullptr;
  try {
    for (Py_ssize_t i = 0; ok && i < n; ++i) {
      PyObject* item = PySequence_Fast_GET_ITEM(fast, i);
      ok = THPVariable_Check(item);
      if (!ok) break;
      const at::Tensor& t = THPVariable_Unpack(item);
      ok = t.defined() && t.is_cuda() && t.get_device() == device && t.scalar_type() == type && t.dim() == dims &&
           t.is_contiguous();
      for (Py_ssize_t d = 0; ok && d < dims; ++d) ok = t.size(d) == want[d];
      if (ok) to[i] = t.data_ptr();
    }
  } catch (...) {   // a tensor without storage, say: not an operand
    ok = false;
  }
  Py_DECREF(fast);
  if (!ok) {
    Py_XDECREF(bytes);
    return false;
  }
  *out = bytes;
  return true;
}

// operands(device, seq, dtype, shape, seq, dtype, shape, ...): the addresses of
// each group's tensors as bytes, in a tuple, or None when a check fails (the
// caller then names what is wrong).
PyObject* operands(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 1 || n % 3 != 1) {
    PyErr_SetString(PyExc_TypeError, "operands(device, tensors, dtype, shape, ...)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[0]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  PyObject* result = PyTuple_New(n / 3);
  if (!result) return nullptr;
  for (Py_ssize_t g = 0; g < n / 3; ++g) {
    PyObject* bytes = nullptr;
    if (!addresses(args[1 + 3 * g], args[2 + 3 * g], args[3 + 3 * g], device, &bytes)) {
      Py_DECREF(result);
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    PyTuple_SET_ITEM(result, g, bytes);
  }
  return result;
}

// A tuple of whole numbers.
bool sizes_of(PyObject* shape, std::vector<int64_t>& dims) {
  if (!PyTuple_Check(shape)) {
    PyErr_SetString(PyExc_TypeError, "expected a tuple of sizes");
    return false;
  }
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(shape); ++i) {
    dims.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)));
    if (dims.back() == -1 && PyErr_Occurred()) return false;
  }
  return true;
}

// Whether new tensors have to come through torch's dispatcher: something
// watches or replaces its calls, or fills new memory.
bool watched() {
  return c10::impl::dispatch_mode_enabled() ||
         (at::globalContext().deterministicAlgorithms() && at::globalContext().deterministicFillUninitializedMemory());
}

at::Tensor new_tensor(PyObject* dtype, const std::vector<int64_t>& dims, long device) {
  const at::Device where(at::kCUDA, (at::DeviceIndex)device);
  const auto type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (watched()) return at::empty(dims, at::TensorOptions().dtype(type).device(where));
  return at::Tensor(at::detail::empty_cuda(dims, type, where, std::nullopt));
}

// Tensor k of those laid one after the other in `all` ([p, ...]): its memory,
// but no view of it, with a version of its own.
at::Tensor part_of(const at::Tensor& all, long k, const std::vector<int64_t>& dims) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  impl->set_storage_offset(k * (all.numel() / all.size(0)));
  impl->set_sizes_contiguous(dims);
  return at::Tensor(std::move(impl));
}

// Shards below this size share an allocation: a pack of eight small shards takes
// 17 us of host time, 27 with an allocation each.  torch's allocator takes small
// allocations from common blocks of 2 MiB anyway; a larger shard has its own, so
// that keeping it holds no other's memory.
constexpr int64_t kSharedBytes = 1 << 20;

// empty(device, dtype, shape, dtype, shape, ...): new tensors on the GPU, in a
// tuple; None for a shape of None.
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 1 || n % 2 != 1) {
    PyErr_SetString(PyExc_TypeError, "empty(device, dtype, shape, ...)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[0]);
  if (device == -1 && PyErr_Occurred()) return nullptr;
  PyObject* result = PyTuple_New(n / 2);
  if (!result) return nullptr;
  try {
    for (Py_ssize_t g = 0; g < n / 2; ++g) {
      PyObject *dtype = args[1 + 2 * g], *shape = args[2 + 2 * g], *o = nullptr;
      std::vector<int64_t> dims;
      if (shape == Py_None) {
        Py_INCREF(Py_None);
        o = Py_None;
      } else if (!THPDtype_Check(dtype)) {
        PyErr_SetString(PyExc_TypeError, "empty: expected a dtype");
      } else if (sizes_of(shape, dims)) {
        o = THPVariable_Wrap(new_tensor(dtype, dims, device));
      }
      if (!o) {
        Py_DECREF(result);
        return nullptr;
      }
      PyTuple_SET_ITEM(result, g, o);
    }
  } catch (...) {   // out of memory above all: raised as torch raises it
    Py_DECREF(result);
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
  return result;
}

// shards(device, p, dtype, shape, ...): for each group p new tensors of that
// shape and their addresses as bytes: (tensors, bytes, tensors, bytes, ...).
PyObject* shards(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 2 || n % 2 != 0) {
    PyErr_SetString(PyExc_TypeError, "shards(device, p, dtype, shape, ...)");
    return nullptr;
  }
  const long device = PyLong_AsLong(args[0]), p = PyLong_AsLong(args[1]);
  if (PyErr_Occurred()) return nullptr;
  PyObject* result = PyTuple_New(n - 2);
  if (!result) return nullptr;
  try {
    for (Py_ssize_t g = 2; g < n; g += 2) {
      std::vector<int64_t> dims;
      if (!THPDtype_Check(args[g]) || !sizes_of(args[g + 1], dims)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "shards: expected a dtype");
        Py_DECREF(result);
        return nullptr;
      }
      int64_t size = (int64_t)c10::elementSize(reinterpret_cast<THPDtype*>(args[g])->scalar_type);
      for (const int64_t d : dims) size *= d;
      at::Tensor all;
      if (p > 1 && size < kSharedBytes && !watched()) {
        std::vector<int64_t> together{p};
        together.insert(together.end(), dims.begin(), dims.end());
        all = new_tensor(args[g], together, device);
      }
      PyObject* bytes = PyBytes_FromStringAndSize(nullptr, p * (Py_ssize_t)sizeof(void*));
      PyObject* tensors = PyTuple_New(p);
      PyTuple_SET_ITEM(result, g - 2, tensors);   // held by `result` from here on
      PyTuple_SET_ITEM(result, g - 1, bytes);
      if (!bytes || !tensors) {
        Py_DECREF(result);
        return nullptr;
      }
      void** to = reinterpret_cast<void**>(PyBytes_AS_STRING(bytes));
      for (long k = 0; k < p; ++k) {
        at::Tensor t = all.defined() ? part_of(all, k, dims) : new_tensor(args[g], dims, device);
        to[k] = t.data_ptr();
        PyObject* o = THPVariable_Wrap(std::move(t));
        if (!o) {
          Py_DECREF(result);
          return nullptr;
        }
        PyTuple_SET_ITEM(tensors, k, o);
      }
    }
  } catch (...) {
    Py_DECREF(result);
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
  return result;
}

PyMethodDef methods[] = {
    {"operands", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(operands)), METH_FASTCALL,
     "operands(device, tensors, dtype, shape, ...): addresses of each group's tensors, or None"},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empty)), METH_FASTCALL,
     "empty(device, dtype, shape, ...): new tensors on the GPU"},
    {"shards", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(shards)), METH_FASTCALL,
     "shards(device, p, dtype, shape, ...): p new tensors of each shape, and their addresses"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__args() { return PyModule_Create(&module); }
