// Reads lists of torch tensors for the binding: what each call checks of its
// tensors, and the arrays of sizes and pointers it hands to the C ABI.  Read
// attribute by attribute from Python, 223 tensors took 50 us, as long as the
// kernel that norms them; here they take about 7.  Also makes lists of outputs in
// one allocation: the operands of 32 matrices and of their transposes took 285 us
// one torch.empty at a time, and take 22.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include <ATen/ops/empty.h>
#include <c10/core/TensorImpl.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

namespace {

// What holds for every tensor of a list, as bits (the binding has the same four).
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

int hip_index(const at::Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }

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

// A tensor's address.  For one that the call writes, a tensor that shares its
// data copy-on-write is given memory of its own first, as Tensor.data_ptr() does;
// one that is only read keeps sharing.
int64_t address(const at::Tensor& t, bool written) {
  const void* p = written ? t.mutable_data_ptr() : t.const_data_ptr();
  return static_cast<int64_t>(reinterpret_cast<intptr_t>(p));
}

// scan(tensors, written) -> (device, flags, dtype codes, element counts, pointers, rows, columns)
// device: of the first tensor, -1 if that is no HIP device; the arrays as bytes
// (int32, then int64); rows and columns of two-dimensional tensors, else 0.
// The written lists of a call go first: to give one tensor its own memory moves
// every tensor of the same storage, whose address, taken before, is then another's.
PyObject* scan(PyObject*, PyObject* args) {
  PyObject* arg;
  int written;
  if (!PyArg_ParseTuple(args, "Op", &arg, &written)) return nullptr;
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
        device = hip_index(*t);
        first = t->scalar_type();
      }
      if (device < 0 || hip_index(*t) != device) flags &= ~kSameDevice;
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
      ptrs[i] = address(*t, written != 0);
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

// scan_f8(operands, block, written) -> (device, bad, kind, rows, padded K, values,
// scales) of (values, scales) pairs.  bad: the first operand that is none, or -1;
// kind: what is wrong with it: 1 the dtypes, 2 device, contiguity or dimensions, 3
// the shapes.  written: as in scan.
PyObject* scan_f8(PyObject*, PyObject* args) {
  PyObject* arg;
  long block;
  int written;
  if (!PyArg_ParseTuple(args, "Olp", &arg, &block, &written)) return nullptr;
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
      if (i == 0) device = hip_index(*q);
      int wrong = 0;
      if (q->scalar_type() != at::kFloat8_e4m3fn || s->scalar_type() != at::kByte)
        wrong = 1;
      else if (device < 0 || hip_index(*q) != device || hip_index(*s) != device ||
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
        qs[i] = address(*q, written != 0);
        ss[i] = address(*s, written != 0);
      }
    }
    return Py_BuildValue("iniNNNN", device, bad, kind, as_bytes(rows), as_bytes(kps), as_bytes(qs),
                         as_bytes(ss));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// Room for tensors on one HIP device: one allocation, cut into contiguous
// pieces at multiples of 256 bytes.
class Room {
 public:
  // Counts a piece; returns its offset.
  int64_t add(int64_t rows, int64_t cols, int64_t size) {
    const int64_t at = bytes_;
    bytes_ += (rows * cols * size + 255) / 256 * 256;
    return at;
  }
  void allocate(int device) {
    whole_ = at::empty({bytes_}, at::TensorOptions().dtype(at::kByte).device(
                                     at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device))));
  }
  PyObject* piece(int64_t at, c10::IntArrayRef sizes, at::ScalarType type) const {
    auto impl = c10::make_intrusive<c10::TensorImpl>(
        c10::Storage(whole_.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
        c10::scalarTypeToTypeMeta(type));
    impl->set_sizes_contiguous(sizes);
    impl->set_storage_offset((whole_.storage_offset() + at) / static_cast<int64_t>(c10::elementSize(type)));
    return THPVariable_Wrap(at::Tensor(std::move(impl)));
  }

 private:
  int64_t bytes_ = 0;
  at::Tensor whole_;
};

// Two equally long byte strings of int64, or false with an exception set.
bool shapes(PyObject* r, PyObject* c, const int64_t** rows, const int64_t** cols, Py_ssize_t* n) {
  if (!PyBytes_Check(r) || !PyBytes_Check(c) || PyBytes_GET_SIZE(r) != PyBytes_GET_SIZE(c)) {
    PyErr_SetString(PyExc_TypeError, "rows and columns are equally long bytes");
    return false;
  }
  *rows = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(r));
  *cols = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(c));
  *n = PyBytes_GET_SIZE(r) / static_cast<Py_ssize_t>(sizeof(int64_t));
  return true;
}

// room(rows, columns, dtype code, device) -> list of tensors
PyObject* room(PyObject*, PyObject* args) {
  PyObject *r, *c;
  int code, device;
  if (!PyArg_ParseTuple(args, "OOii", &r, &c, &code, &device)) return nullptr;
  const int64_t *rows, *cols;
  Py_ssize_t n;
  if (!shapes(r, c, &rows, &cols, &n)) return nullptr;
  PyObject* list = nullptr;
  try {
    const at::ScalarType type = code == 0 ? at::kBFloat16 : at::kFloat;
    Room all;
    std::vector<int64_t> at(n);
    for (Py_ssize_t i = 0; i < n; ++i) at[i] = all.add(rows[i], cols[i], code == 0 ? 2 : 4);
    all.allocate(device);
    list = PyList_New(n);
    for (Py_ssize_t i = 0; list != nullptr && i < n; ++i) {
      PyObject* t = all.piece(at[i], {rows[i], cols[i]}, type);
      if (t == nullptr) {
        Py_CLEAR(list);
        break;
      }
      PyList_SET_ITEM(list, i, t);
    }
    return list;
  } catch (const std::exception& e) {
    Py_XDECREF(list);
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// room_f8(rows, columns, block, device, kind) -> list of kind(values, scales)
PyObject* room_f8(PyObject*, PyObject* args) {
  PyObject *r, *c, *kind;
  long block;
  int device;
  if (!PyArg_ParseTuple(args, "OOliO", &r, &c, &block, &device, &kind)) return nullptr;
  const int64_t *rows, *cols;
  Py_ssize_t n;
  if (!shapes(r, c, &rows, &cols, &n)) return nullptr;
  PyObject* list = nullptr;
  try {
    Room all;
    std::vector<int64_t> q(n), s(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const int64_t kb = (cols[i] + block - 1) / block;
      q[i] = all.add(rows[i], kb * block, 1);
      s[i] = all.add(kb, (rows[i] + 15) / 16 * 16, 1);
    }
    all.allocate(device);
    list = PyList_New(n);
    for (Py_ssize_t i = 0; list != nullptr && i < n; ++i) {
      const int64_t kb = (cols[i] + block - 1) / block;
      PyObject* a = all.piece(q[i], {rows[i], kb * block}, at::kFloat8_e4m3fn);
      PyObject* b = a == nullptr ? nullptr
                                 : all.piece(s[i], {kb, (rows[i] + 15) / 16 * 16}, at::kByte);
      PyObject* op = b == nullptr ? nullptr : PyObject_CallFunctionObjArgs(kind, a, b, nullptr);
      Py_XDECREF(a);
      Py_XDECREF(b);
      if (op == nullptr) {
        Py_CLEAR(list);
        break;
      }
      PyList_SET_ITEM(list, i, op);
    }
    return list;
  } catch (const std::exception& e) {
    Py_XDECREF(list);
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// room_norm(bytes, device) -> (workspace of so many bytes, two float32).  Two
// allocations: a caller keeps the result, step after step, and must not keep the
// workspace (17 KB and more) with it.
PyObject* room_norm(PyObject*, PyObject* args) {
  long long bytes;
  int device;
  if (!PyArg_ParseTuple(args, "Li", &bytes, &device)) return nullptr;
  try {
    const at::TensorOptions on = at::TensorOptions().device(
        at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
    return Py_BuildValue("NN", THPVariable_Wrap(at::empty({bytes}, on.dtype(at::kByte))),
                         THPVariable_Wrap(at::empty({2}, on.dtype(at::kFloat))));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef methods[] = {
    {"room_norm", room_norm, METH_VARARGS, "room_norm(bytes, device)"},
    {"room", room, METH_VARARGS, "room(rows, columns, dtype code, device)"},
    {"room_f8", room_f8, METH_VARARGS, "room_f8(rows, columns, block, device, kind)"},
    {"scan", scan, METH_VARARGS, "scan(tensors, written): device, flags, dtype codes, sizes, pointers"},
    {"same_shapes", same_shapes, METH_VARARGS, "same_shapes(a, b)"},
    {"scan_f8", scan_f8, METH_VARARGS, "scan_f8(operands, block, written)"},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "tensor_lists", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tensor_lists() {
  return PyModule_Create(&module);
}
