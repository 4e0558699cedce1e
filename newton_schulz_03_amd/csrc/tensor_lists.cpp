// Reads lists of torch tensors for the binding: what each call checks of its
// tensors, and the arrays of sizes and pointers it hands to the C ABI.  Read
// attribute by attribute from Python, 223 tensors took 50 us, as long as the
// kernel that norms them; here they take about 7.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include <torch/csrc/autograd/python_variable.h>

#include <vector>

namespace {

// What holds for every tensor of a list, as bits.
enum : long {
  kSameDevice = 1,   // the first one's HIP device
  kContiguous = 2,
  kSameDtype = 4,    // the first one's
  kMatrices = 8,     // two dimensions
  kAll = 15,
};

int32_t dtype_code(const at::Tensor& t) {  // MUON_BF16, MUON_FP32, or -1
  return t.scalar_type() == at::kBFloat16 ? 0 : t.scalar_type() == at::kFloat ? 1 : -1;
}

int device_of(const at::Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }

// A borrowed list or tuple's items, or null with an exception set.
PyObject* items(PyObject* arg, Py_ssize_t* n) {
  if (!PyList_Check(arg) && !PyTuple_Check(arg)) {
    PyErr_SetString(PyExc_TypeError, "a list or tuple of tensors is needed");
    return nullptr;
  }
  *n = PySequence_Fast_GET_SIZE(arg);
  return arg;
}

const at::Tensor* tensor_at(PyObject* list, Py_ssize_t i) {
  PyObject* o = PySequence_Fast_GET_ITEM(list, i);
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "item %zd is no tensor", i);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

template <typename T>
PyObject* as_bytes(const std::vector<T>& v) {
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(v.data()),
                                   static_cast<Py_ssize_t>(v.size() * sizeof(T)));
}

// scan(tensors) -> (device, flags, dtype codes, element counts, pointers, rows, columns)
// device: of the first tensor, -1 if that is no HIP device; the arrays as bytes
// (int32, then int64); rows and columns of two-dimensional tensors, else 0.
PyObject* scan(PyObject*, PyObject* arg) {
  Py_ssize_t n;
  PyObject* list = items(arg, &n);
  if (list == nullptr) return nullptr;
  try {
    std::vector<int32_t> codes(n);
    std::vector<int64_t> numels(n), ptrs(n), rows(n), cols(n);
    long flags = kAll;
    int device = -1;
    at::ScalarType first = at::kFloat;
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t = tensor_at(list, i);
      if (t == nullptr) return nullptr;
      if (i == 0) {
        device = device_of(*t);
        first = t->scalar_type();
      }
      if (device < 0 || device_of(*t) != device) flags &= ~kSameDevice;
      if (!t->is_contiguous()) flags &= ~kContiguous;
      if (t->scalar_type() != first) flags &= ~kSameDtype;
      if (t->dim() == 2) {
        rows[i] = t->size(0);
        cols[i] = t->size(1);
      } else {
        flags &= ~kMatrices;
      }
      codes[i] = dtype_code(*t);
      numels[i] = t->numel();
      ptrs[i] = static_cast<int64_t>(reinterpret_cast<intptr_t>(t->const_data_ptr()));
    }
    return Py_BuildValue("ilNNNNN", device, flags, as_bytes(codes), as_bytes(numels),
                         as_bytes(ptrs), as_bytes(rows), as_bytes(cols));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// same_shapes(a, b): whether two equally long lists of tensors have equal shapes.
PyObject* same_shapes(PyObject*, PyObject* args) {
  PyObject *a, *b;
  if (!PyArg_ParseTuple(args, "OO", &a, &b)) return nullptr;
  Py_ssize_t n, m;
  if (items(a, &n) == nullptr || items(b, &m) == nullptr) return nullptr;
  if (n != m) Py_RETURN_FALSE;
  try {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor *x = tensor_at(a, i), *y = tensor_at(b, i);
      if (x == nullptr || y == nullptr) return nullptr;
      if (x->sizes() != y->sizes()) Py_RETURN_FALSE;
    }
    Py_RETURN_TRUE;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// scan_f8(operands, block) -> (device, bad, kind, rows, padded K, values, scales)
// of (values, scales) pairs.  bad: the first operand that is none, or -1; kind:
// what is wrong with it: 1 the dtypes, 2 device, contiguity or dimensions, 3 the
// shapes.
PyObject* scan_f8(PyObject*, PyObject* args) {
  PyObject* arg;
  long block;
  if (!PyArg_ParseTuple(args, "Ol", &arg, &block)) return nullptr;
  Py_ssize_t n;
  PyObject* list = items(arg, &n);
  if (list == nullptr) return nullptr;
  try {
    std::vector<int64_t> rows(n), kps(n), qs(n), ss(n);
    int device = -1, kind = 0;
    Py_ssize_t bad = -1;
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* pair = PySequence_Fast_GET_ITEM(list, i);
      Py_ssize_t two;
      if (items(pair, &two) == nullptr) return nullptr;
      if (two != 2) {
        PyErr_Format(PyExc_TypeError, "operand %zd is no pair of values and scales", i);
        return nullptr;
      }
      const at::Tensor *q = tensor_at(pair, 0), *s = tensor_at(pair, 1);
      if (q == nullptr || s == nullptr) return nullptr;
      if (i == 0) device = device_of(*q);
      int wrong = 0;
      if (q->scalar_type() != at::kFloat8_e4m3fn || s->scalar_type() != at::kByte)
        wrong = 1;
      else if (device < 0 || device_of(*q) != device || device_of(*s) != device ||
               !q->is_contiguous() || !s->is_contiguous() || q->dim() != 2 || s->dim() != 2)
        wrong = 2;
      else if (q->size(1) % block != 0 || s->size(0) != q->size(1) / block ||
               s->size(1) != (q->size(0) + 15) / 16 * 16)
        wrong = 3;
      if (wrong != 0 && bad < 0) {
        bad = i;
        kind = wrong;
      }
      if (wrong == 0) {
        rows[i] = q->size(0);
        kps[i] = q->size(1);
        qs[i] = static_cast<int64_t>(reinterpret_cast<intptr_t>(q->const_data_ptr()));
        ss[i] = static_cast<int64_t>(reinterpret_cast<intptr_t>(s->const_data_ptr()));
      }
    }
    return Py_BuildValue("iniNNNN", device, bad, kind, as_bytes(rows), as_bytes(kps), as_bytes(qs),
                         as_bytes(ss));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"scan", scan, METH_O, "scan(tensors): device, flags, dtype codes, sizes, pointers"},
    {"same_shapes", same_shapes, METH_VARARGS, "same_shapes(a, b)"},
    {"scan_f8", scan_f8, METH_VARARGS, "scan_f8(operands, block)"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_lists", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_lists() {
  PyObject* m = PyModule_Create(&module);
  if (m == nullptr) return nullptr;
  if (PyModule_AddIntConstant(m, "SAME_DEVICE", kSameDevice) != 0 ||
      PyModule_AddIntConstant(m, "CONTIGUOUS", kContiguous) != 0 ||
      PyModule_AddIntConstant(m, "SAME_DTYPE", kSameDtype) != 0 ||
      PyModule_AddIntConstant(m, "MATRICES", kMatrices) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
