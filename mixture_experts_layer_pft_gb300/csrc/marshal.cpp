// Argument marshalling of the Python binding: checks tensors and takes their addresses.
//
// A call of the C ABI takes some 2 us; the same checks of ten tensors in Python took 6 more, and those of an optimizer
// step over 57 tensors 150.  Nothing here touches a GPU.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

namespace {

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

bool refuse(PyObject* kind, const std::string& text) {
  PyErr_SetString(kind, text.c_str());
  return false;
}

const at::Tensor* tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

bool on_device(const at::Tensor& t, const char* name) {
  if (t.layout() != at::kStrided) return refuse(PyExc_ValueError, std::string(name) + ": tensor must be strided");
  if (!t.is_cuda()) return refuse(PyExc_ValueError, std::string(name) + ": tensor must be on a CUDA device");
  if (!t.is_contiguous()) return refuse(PyExc_ValueError, std::string(name) + ": tensor must be contiguous");
  return true;
}

// pointer(t, name, dtype, shape): t's address after checks; None for None.
PyObject* pointer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 || !THPDtype_Check(args[2]) || !PyTuple_Check(args[3])) {
    PyErr_SetString(PyExc_TypeError, "pointer(tensor, name, dtype, shape)");
    return nullptr;
  }
  if (args[0] == Py_None) Py_RETURN_NONE;
  const char* name = PyUnicode_AsUTF8(args[1]);
  if (name == nullptr) return nullptr;
  const at::Tensor* t = tensor_of(args[0], name);
  if (t == nullptr) return nullptr;
  const THPDtype* want = reinterpret_cast<THPDtype*>(args[2]);
  bool same = t->scalar_type() == want->scalar_type && t->dim() == PyTuple_GET_SIZE(args[3]);
  for (int64_t i = 0; same && i < t->dim(); ++i) {
    const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(args[3], i));
    if (v == -1 && PyErr_Occurred()) return nullptr;
    same = t->size(i) == v;
  }
  if (!same) {
    PyObject* shape = PyObject_Repr(args[3]);
    const char* text = shape != nullptr ? PyUnicode_AsUTF8(shape) : nullptr;
    if (text != nullptr)
      refuse(PyExc_ValueError, std::string(name) + " must be torch." + want->name + " " + text + ", got " +
                                   at::toString(t->scalar_type()) + " " + shape_of(*t));
    Py_XDECREF(shape);
    return nullptr;
  }
  if (!on_device(*t, name)) return nullptr;
  return PyLong_FromVoidPtr(t->data_ptr());
}

struct Items {  // a list or tuple, held while it is read
  PyObject* seq = nullptr;
  Py_ssize_t n = 0;
  bool open(PyObject* o, const char* name) {
    seq = PySequence_Fast(o, name);
    if (seq == nullptr) return false;
    n = PySequence_Fast_GET_SIZE(seq);
    return true;
  }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
  ~Items() { Py_XDECREF(seq); }
};

template <typename T>
PyObject* bytes_of(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()), static_cast<Py_ssize_t>(v.size() * sizeof(T)));
}

// One list of an optimizer step: the addresses of tensors of the types and sizes given, 0 for None.
PyObject* addresses(PyObject* list, const char* name, const std::vector<at::ScalarType>& types, const std::vector<int64_t>& sizes) {
  if (list == Py_None) Py_RETURN_NONE;
  Items items;
  if (!items.open(list, name)) return nullptr;
  const Py_ssize_t n = static_cast<Py_ssize_t>(sizes.size());
  if (items.n != n) {
    refuse(PyExc_ValueError, std::string(name) + ": " + std::to_string(items.n) + " tensors for " + std::to_string(n) + " parameters");
    return nullptr;
  }
  std::vector<uint64_t> out(n, 0);
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (items[i] == Py_None) continue;
    const at::Tensor* t = tensor_of(items[i], name);
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != types[i] || t->numel() != sizes[i]) {
      refuse(PyExc_ValueError, std::string(name) + "[" + std::to_string(i) + "] must have " + std::to_string(sizes[i]) + " values of " +
                                   at::toString(types[i]) + ", got " + std::to_string(t->numel()) + " of " + at::toString(t->scalar_type()));
      return nullptr;
    }
    if (!on_device(*t, name)) return nullptr;
    out[i] = reinterpret_cast<uint64_t>(t->data_ptr());
  }
  return bytes_of(out);
}

// optimizer(params, grads, masters, m, v, m_scale, v_scale): the arrays of moe_adamw_step as bytes, in that order, then the
// sizes (int64) and types (int32, moe_dtype).
PyObject* optimizer(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "optimizer(params, grads, masters, m, v, m_scale, v_scale)");
    return nullptr;
  }
  Items params;
  if (!params.open(args[0], "params must be a list")) return nullptr;
  const bool q8 = args[5] != Py_None;
  if (q8 != (args[6] != Py_None)) {
    PyErr_SetString(PyExc_ValueError, "m_scale and v_scale go together");
    return nullptr;
  }
  std::vector<at::ScalarType> types(params.n);
  std::vector<int64_t> sizes(params.n), blocks(params.n);
  std::vector<int32_t> codes(params.n);
  for (Py_ssize_t i = 0; i < params.n; ++i) {
    const at::Tensor* t = tensor_of(params[i], "params");
    if (t == nullptr) return nullptr;
    types[i] = t->scalar_type();
    sizes[i] = t->numel();
    blocks[i] = (sizes[i] + 255) / 256;
    if (types[i] != at::kFloat && types[i] != at::kBFloat16) {
      refuse(PyExc_TypeError, std::string("unsupported dtype ") + at::toString(types[i]));
      return nullptr;
    }
    codes[i] = types[i] == at::kBFloat16 ? 1 : 0;
  }
  const std::vector<at::ScalarType> f32(params.n, at::kFloat), e4m3(params.n, at::kFloat8_e4m3fn), e5m2(params.n, at::kFloat8_e5m2);
  const char* names[7] = {"params", "grads", "masters", "m", "v", "m_scale", "v_scale"};
  const std::vector<at::ScalarType>* want[7] = {&types, &types, &f32, q8 ? &e4m3 : &f32, q8 ? &e5m2 : &f32, &f32, &f32};
  PyObject* out = PyTuple_New(9);
  if (out == nullptr) return nullptr;
  for (int k = 0; k < 7; ++k) {
    PyObject* b = addresses(args[k], names[k], *want[k], k < 5 ? sizes : blocks);
    if (b == nullptr) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, k, b);
  }
  PyTuple_SET_ITEM(out, 7, bytes_of(sizes));
  PyTuple_SET_ITEM(out, 8, bytes_of(codes));
  return out;
}

// torch reports by exception what a tensor cannot answer (a nested one its sizes, one without memory its address): none may
// pass through the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyMethodDef methods[] = {
    {"pointer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<pointer>)), METH_FASTCALL, "address of a checked tensor"},
    {"optimizer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<optimizer>)), METH_FASTCALL, "arrays of an optimizer step"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "argument marshalling of the binding", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
