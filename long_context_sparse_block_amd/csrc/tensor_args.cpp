// Tensor arguments of the Python wrappers (module _tensor_args): the pointer of a
// dense tensor, the pointer and strides of a [tokens, heads, head_dim] one, a page
// pool's, a workspace.  Looked up attribute by attribute from Python, each costs
// three to four times as much, and a call of a few microseconds checks half a
// dozen.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* dtype_of(const at::Tensor& t) { return reinterpret_cast<PyObject*>(torch::getTHPDtype(t.scalar_type())); }

// ValueError "<name><what>", or the longer forms below; always nullptr
PyObject* refuse(PyObject* name, const char* what) {
  PyErr_Format(PyExc_ValueError, "%U%s", name, what);
  return nullptr;
}

PyObject* refuse_shape(PyObject* name, const at::Tensor& t, PyObject* want) {
  PyObject* got = PyTuple_New(t.dim());
  if (got == nullptr) return nullptr;
  for (int64_t i = 0; i < t.dim(); ++i) PyTuple_SET_ITEM(got, i, PyLong_FromLongLong(t.size(i)));
  PyObject* plain = PyTuple_Check(want) ? PySequence_Tuple(want) : (Py_INCREF(want), want);   // (of a torch.Size)
  if (plain != nullptr) PyErr_Format(PyExc_ValueError, "%U: shape %R, expected %S", name, got, plain);
  Py_XDECREF(plain);
  Py_DECREF(got);
  return nullptr;
}

bool same_shape(const at::Tensor& t, PyObject* want) {
  if (!PyTuple_Check(want) || PyTuple_GET_SIZE(want) != t.dim()) return false;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(want, i)) != t.size(i)) return false;
  return !PyErr_Occurred();
}

// The tensor on GPU `dev`, or nullptr with the error set
const at::Tensor* gpu_tensor(PyObject* x, PyObject* name, PyObject* dev) {
  if (x == Py_None) return refuse(name, " is required"), nullptr;
  if (!THPVariable_Check(x)) return refuse(name, " must be a tensor"), nullptr;
  const at::Tensor& t = THPVariable_Unpack(x);
  if (!t.is_cuda()) return refuse(name, " must be a GPU tensor"), nullptr;
  const long want = PyLong_AsLong(dev);
  if (want == -1 && PyErr_Occurred()) return nullptr;
  if (t.get_device() != want) {
    PyErr_Format(PyExc_ValueError, "%U is on cuda:%d, expected cuda:%ld", name, (int)t.get_device(), want);
    return nullptr;
  }
  return &t;
}

// dense(tensor, dtype, shape, name, dev) -> pointer
PyObject* dense(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !PyUnicode_Check(a[3])) {
    PyErr_SetString(PyExc_TypeError, "dense(tensor, dtype, shape, name, dev)");
    return nullptr;
  }
  const at::Tensor* t = gpu_tensor(a[0], a[3], a[4]);
  if (t == nullptr) return nullptr;
  if (dtype_of(*t) != a[1]) {
    PyErr_Format(PyExc_ValueError, "%U: dtype %S, expected %S", a[3], dtype_of(*t), a[1]);
    return nullptr;
  }
  if (!same_shape(*t, a[2])) return PyErr_Occurred() ? nullptr : refuse_shape(a[3], *t, a[2]);
  if (!t->is_contiguous()) return refuse(a[3], " must be contiguous");
  return PyLong_FromVoidPtr(t->data_ptr());
}

// rows(tensor, dtypes, name, dev, shape or None) -> pointer, token stride, head stride
PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if ((n != 4 && n != 5) || !PyUnicode_Check(a[2])) {
    PyErr_SetString(PyExc_TypeError, "rows(tensor, dtypes, name, dev, shape=None)");
    return nullptr;
  }
  const at::Tensor* t = gpu_tensor(a[0], a[2], a[3]);
  if (t == nullptr) return nullptr;
  const int known = PySequence_Contains(a[1], dtype_of(*t));
  if (known < 0) return nullptr;
  if (known == 0) {
    PyObject* want = PySequence_Tuple(a[1]);
    if (want == nullptr) return nullptr;
    PyErr_Format(PyExc_ValueError, "%U: dtype %S, expected one of %R", a[2], dtype_of(*t), want);
    Py_DECREF(want);
    return nullptr;
  }
  const bool fixed = n == 5 && a[4] != Py_None;
  if (fixed ? !same_shape(*t, a[4]) : t->dim() != 3) {
    if (PyErr_Occurred()) return nullptr;
    PyObject* want = fixed ? (Py_INCREF(a[4]), a[4]) : PyUnicode_FromString("[tokens, heads, head_dim]");
    if (want != nullptr) refuse_shape(a[2], *t, want);
    Py_XDECREF(want);
    return nullptr;
  }
  if (t->dim() != 3) return refuse(a[2], ": expected [tokens, heads, head_dim]");
  if (t->stride(2) != 1 && t->size(2) > 1) return refuse(a[2], ": the last dimension must be dense");
  // the strides of dimensions of one element mean nothing
  const long long st = t->size(0) > 1 ? t->stride(0) : 0, sh = t->size(1) > 1 ? t->stride(1) : 0;
  void* const at = t->data_ptr();
  return Py_BuildValue("(NLL)", PyLong_FromVoidPtr(at), st, sh);
}

// pool(pages, heads, head_dim, name, dev) -> pointer, code type (misa_kdtype), pages, rows a page
PyObject* pool(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !PyUnicode_Check(a[3])) {
    PyErr_SetString(PyExc_TypeError, "pool(pages, heads, head_dim, name, dev)");
    return nullptr;
  }
  const at::Tensor* t = gpu_tensor(a[0], a[3], a[4]);
  if (t == nullptr) return nullptr;
  const long long heads = PyLong_AsLongLong(a[1]), dim = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  const auto type = t->scalar_type();
  const bool codes = type == at::kByte || type == at::kFloat8_e4m3fn;
  if (!codes && type != at::kBFloat16) {
    PyErr_Format(PyExc_ValueError, "%U: dtype %S (expected bfloat16 or float8_e4m3fn/uint8 codes)", a[3], dtype_of(*t));
    return nullptr;
  }
  const int64_t nd = t->dim();
  const bool fits = (nd == 4 && t->size(2) == heads && t->size(3) == dim) || (nd == 3 && heads == 1 && t->size(2) == dim);
  if (!fits) {
    PyObject* want = PyUnicode_FromFormat("(n_pages, page_keys, %lld, %lld)", heads, dim);
    if (want != nullptr) refuse_shape(a[3], *t, want);
    Py_XDECREF(want);
    return nullptr;
  }
  if (!t->is_contiguous()) return refuse(a[3], " must be contiguous");
  const long long n_pages = t->size(0), page_keys = t->size(1);
  void* const at = t->data_ptr();
  return Py_BuildValue("(NiLL)", PyLong_FromVoidPtr(at), codes ? 1 : 0, n_pages, page_keys);
}

// scratch(bytes, like) -> uint8 tensor on like's device, pointer
PyObject* scratch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !THPVariable_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "scratch(bytes, like)");
    return nullptr;
  }
  const long long bytes = PyLong_AsLongLong(a[0]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor t = at::empty({bytes}, at::TensorOptions().device(THPVariable_Unpack(a[1]).device()).dtype(at::kByte));
  void* const at = t.data_ptr();
  return Py_BuildValue("(NN)", THPVariable_Wrap(t), PyLong_FromVoidPtr(at));
}

// Torch throws where a tensor has no pointer, sizes or strides of its own (under
// vmap, while tracing), and where memory runs out: its Python errors, nothing
// past this border.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>)); }

PyMethodDef methods[] = {
    {"pool", entry<pool>(), METH_FASTCALL,
     "pool(pages, heads, head_dim, name, dev): pointer, code type, n_pages, page_keys of a page pool"},
    {"scratch", entry<scratch>(), METH_FASTCALL,
     "scratch(bytes, like): a workspace on like's device, and its pointer"},
    {"dense", entry<dense>(), METH_FASTCALL,
     "dense(tensor, dtype, shape, name, dev): pointer of a dense tensor of this type and shape on GPU dev"},
    {"rows", entry<rows>(), METH_FASTCALL,
     "rows(tensor, dtypes, name, dev, shape=None): pointer, token and head strides of a [tokens, heads, head_dim] tensor"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
