// What the binding asks of many tensors, in one call from Python: the addresses
// and sizes of a list, those of a call's arguments, new tensors, and their versions.
//
// An optimizer's step over hundreds of small tensors is over on the GPU before
// an interpreter has asked each of them for its address, its size, its type,
// its device and its layout (400 tensors: about 140 us); here that is a few
// nanoseconds a tensor.  What does not pass is left to the caller to explain.
#define PY_SSIZE_T_CLEAN
#include <ATen/Functions.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>
#include <torch/csrc/utils/pybind.h>

#include <cstdint>
#include <cstring>
#include <utility>
#include <vector>

namespace {

// addresses(list, device, sizes, per, gaps) -> (addresses, sizes, dtype), or None.
// All items have to be contiguous CUDA tensors of one type on that device and,
// where sizes is not None, item i holds ceil(sizes[i] / per) numbers; with gaps
// an item may be None (address and size 0).  Both results are bytes: 64-bit words
// in the list's order.  The type is None where there is no tensor.
PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 5 || !PyList_CheckExact(args[0])) {
    PyErr_SetString(PyExc_TypeError, "addresses(list, device, sizes, per, gaps)");
    return nullptr;
  }
  const bool gaps = args[4] == Py_True;
  const Py_ssize_t n = PyList_GET_SIZE(args[0]);
  const long device = PyLong_AsLong(args[1]), per = PyLong_AsLong(args[3]);
  if (PyErr_Occurred()) return nullptr;
  const char* want = nullptr;
  if (args[2] != Py_None) {
    if (!PyBytes_Check(args[2]) || PyBytes_GET_SIZE(args[2]) != n * 8 || per < 1) Py_RETURN_NONE;
    want = PyBytes_AS_STRING(args[2]);
  }
  PyObject* where = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* sizes = PyBytes_FromStringAndSize(nullptr, n * 8);
  PyObject* dtype = Py_None;
  bool good = where && sizes;
  try {
    c10::ScalarType type = c10::ScalarType::Undefined;
    bool any = false;
    for (Py_ssize_t i = 0; good && i < n; ++i) {
      PyObject* item = PyList_GET_ITEM(args[0], i);
      if (gaps && item == Py_None) {
        std::memset(PyBytes_AS_STRING(where) + 8 * i, 0, 8);
        std::memset(PyBytes_AS_STRING(sizes) + 8 * i, 0, 8);
        continue;
      }
      if (!THPVariable_Check(item)) {
        good = false;
        break;
      }
      const at::Tensor& t = THPVariable_Unpack(item);
      if (!any) type = t.scalar_type();
      any = true;
      good = t.layout() == c10::kStrided && t.is_cuda() && t.get_device() == device && t.scalar_type() == type &&
             t.is_contiguous();
      if (!good) break;
      const int64_t count = t.numel();
      if (want) {
        int64_t w;
        std::memcpy(&w, want + 8 * i, 8);
        if (count != (w + per - 1) / per) {
          good = false;
          break;
        }
      }
      const uint64_t address = reinterpret_cast<uint64_t>(t.data_ptr());
      std::memcpy(PyBytes_AS_STRING(where) + 8 * i, &address, 8);
      std::memcpy(PyBytes_AS_STRING(sizes) + 8 * i, &count, 8);
    }
    if (good && any) dtype = reinterpret_cast<PyObject*>(torch::getTHPDtype(type));
  } catch (...) {  // a tensor without memory of its own, for one
    good = false;
  }
  PyObject* r = good ? PyTuple_Pack(3, where, sizes, dtype) : nullptr;
  Py_XDECREF(where);
  Py_XDECREF(sizes);
  if (r || PyErr_Occurred()) return r;
  Py_RETURN_NONE;
}

// changed(list or None, ...): the versions of the lists' tensors rise by one, as
// after an in-place change by torch (those made in inference mode have none; None
// may stand in a tensor's place).
PyObject* changed(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  for (Py_ssize_t a = 0; a < nargs; ++a) {
    if (args[a] == Py_None) continue;
    TORCH_CHECK_TYPE(PyList_CheckExact(args[a]), "changed(list or None, ...)");
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(args[a]); ++i) {
      PyObject* item = PyList_GET_ITEM(args[a], i);
      if (item == Py_None) continue;
      TORCH_CHECK_TYPE(THPVariable_Check(item), "changed: a list of tensors");
      const at::Tensor& t = THPVariable_Unpack(item);
      if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
  }
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// empties(device, dtype, shape, dtype, shape, ...) -> a list of new tensors.
PyObject* empties(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(nargs % 2 == 1, "empties(device, dtype, shape, ...)");
  const long device = PyLong_AsLong(args[0]);
  if (PyErr_Occurred()) return nullptr;
  THPObjectPtr out(PyList_New(nargs / 2));
  if (!out) return nullptr;
  for (Py_ssize_t i = 1; i < nargs; i += 2) {
    TORCH_CHECK_TYPE(THPDtype_Check(args[i]) && PyTuple_Check(args[i + 1]), "empties(device, dtype, shape, ...)");
    std::vector<int64_t> shape(static_cast<size_t>(PyTuple_GET_SIZE(args[i + 1])));
    for (size_t d = 0; d < shape.size(); ++d)
      shape[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[i + 1], static_cast<Py_ssize_t>(d)));
    if (PyErr_Occurred()) return nullptr;
    const auto options = at::TensorOptions()
                             .dtype(reinterpret_cast<THPDtype*>(args[i])->scalar_type)
                             .device(c10::kCUDA, static_cast<c10::DeviceIndex>(device));
    at::Tensor t;
    {
      pybind11::gil_scoped_release unlocked;
      t = at::empty(shape, options);
    }
    PyList_SET_ITEM(out.get(), i / 2, THPVariable_Wrap(std::move(t)));
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

// match(pattern, device, tensor, ...) -> (address, ..., size, ...), or None.
// The pattern has a word a tensor: its type, `?` where None may take its place
// (address None), `:` and a letter a dimension.  Types: f binary32, b bfloat16,
// F either, i int32, c one byte of any type, . any.  The same letter is the same
// size everywhere; the sizes follow the addresses in the order of their letters'
// first places.  `#` for the dimensions: any, and the tensor's bytes as a size.
// All are contiguous CUDA tensors on the device.
PyObject* match(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(nargs >= 2 && PyUnicode_Check(args[0]), "match(pattern, device, tensor, ...)");
  const char* at = PyUnicode_AsUTF8(args[0]);
  const long device = PyLong_AsLong(args[1]);
  if (!at || PyErr_Occurred()) return nullptr;
  constexpr Py_ssize_t kMost = 16;
  const Py_ssize_t n = nargs - 2;
  TORCH_CHECK_TYPE(n <= kMost, "at most 16 tensors");
  uint64_t address[kMost];
  bool given[kMost];
  char letters[2 * kMost];
  int64_t sizes[2 * kMost];
  int count = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    while (*at == ' ') ++at;
    const char type = *at;
    TORCH_CHECK_TYPE(type, "a pattern for fewer tensors");
    const bool optional = *++at == '?';
    if (optional) ++at;
    TORCH_CHECK_TYPE(*at == ':', "a pattern's word is type:dimensions");
    ++at;
    given[i] = args[i + 2] != Py_None;
    if (!given[i]) {
      if (!optional) Py_RETURN_NONE;
      while (*at && *at != ' ') ++at;
      continue;
    }
    if (!THPVariable_Check(args[i + 2])) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(args[i + 2]);
    if (t.layout() != c10::kStrided || !t.is_cuda() || t.get_device() != device || !t.is_contiguous()) Py_RETURN_NONE;
    const c10::ScalarType st = t.scalar_type();
    const bool f32 = st == c10::ScalarType::Float, bf16 = st == c10::ScalarType::BFloat16;
    const bool right = type == 'f' ? f32
                       : type == 'b' ? bf16
                       : type == 'F' ? f32 || bf16
                       : type == 'i' ? st == c10::ScalarType::Int
                       : type == 'c' ? t.element_size() == 1
                                     : type == '.';
    if (!right) Py_RETURN_NONE;
    if (*at == '#') {
      TORCH_CHECK_TYPE(count < 2 * kMost, "too many sizes");
      letters[count] = '\0';  // no letter's
      sizes[count++] = t.numel() * static_cast<int64_t>(t.element_size());
      ++at;
    } else {
      int64_t d = 0;
      for (; *at && *at != ' '; ++at, ++d) {
        if (d >= t.dim()) Py_RETURN_NONE;
        int j = 0;
        while (j < count && letters[j] != *at) ++j;
        if (j == count) {
          TORCH_CHECK_TYPE(count < 2 * kMost, "too many sizes");
          letters[count] = *at;
          sizes[count++] = t.size(d);
        } else if (sizes[j] != t.size(d)) {
          Py_RETURN_NONE;
        }
      }
      if (d != t.dim()) Py_RETURN_NONE;
    }
    address[i] = reinterpret_cast<uint64_t>(t.data_ptr());
  }
  THPObjectPtr out(PyTuple_New(n + count));
  if (!out) return nullptr;
  for (Py_ssize_t i = 0; i < n + count; ++i) {
    PyObject* v;
    if (i >= n) {
      v = PyLong_FromLongLong(sizes[i - n]);
    } else if (given[i]) {
      v = PyLong_FromUnsignedLongLong(address[i]);
    } else {
      Py_INCREF(Py_None);
      v = Py_None;
    }
    if (!v) return nullptr;
    PyTuple_SET_ITEM(out.get(), i, v);
  }
  return out.release();
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(addresses)), METH_FASTCALL,
     "Addresses, sizes and type of a list of contiguous CUDA tensors, or None."},
    {"match", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(match)), METH_FASTCALL,
     "Addresses and sizes of a call's tensors that fit a pattern, or None."},
    {"empties", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(empties)), METH_FASTCALL,
     "New CUDA tensors of given types and shapes."},
    {"changed", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(changed)), METH_FASTCALL,
     "Raises the versions of lists of tensors."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_lists", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_lists() { return PyModule_Create(&module); }
