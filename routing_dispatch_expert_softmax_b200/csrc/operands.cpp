// The tensor checks of the binding's calls, natively.  A small call's time is the
// host's: the checks of one tensor take 0.4 us through torch's Python attributes, most
// of the 9 us of a call with nine of them, and about a tenth of that here.
//
//   Operands(where)  the tensors of one call; .where, .index (the CUDA device that
//                    its tensors lie on, or None before the first)
//     .ptr(t, dtype, shape, name, optional=False)  the address of t, a contiguous CUDA
//                    tensor of that dtype and shape (None: any) on the call's device;
//                    None for an optional t that is None.  Anything else goes to
//                    ._refuse(t, dtype, shape, name), which a subclass has to raise in.
//   addresses(a, b)  the data pointers of the lists' tensors (b may be None), as bytes
//   layouts(a, b)  their element counts, dtypes, devices and whether they are contiguous,
//                    as bytes to be compared with others
//   TORCH            the whole version of torch that this was built against (the header
//                    has its first three numbers only)
// Another Python than it was built for gets an ImportError.
#include <Python.h>

#include <structmember.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <cstring>
#include <exception>

namespace {

struct Operands {
  PyObject_HEAD
  PyObject* where;
  int device;  // the device's index + 1; 0: none yet
};

int operands_init(Operands* self, PyObject* args, PyObject* kw) {
  PyObject* where = nullptr;
  if (kw && PyDict_GET_SIZE(kw)) {
    PyErr_SetString(PyExc_TypeError, "Operands takes no keyword arguments");
    return -1;
  }
  if (!PyArg_ParseTuple(args, "O:Operands", &where)) return -1;
  Py_INCREF(where);
  Py_XSETREF(self->where, where);
  self->device = 0;
  return 0;
}

void operands_dealloc(Operands* self) {
  PyTypeObject* type = Py_TYPE(self);
  Py_XDECREF(self->where);
  type->tp_free(reinterpret_cast<PyObject*>(self));
}

// Whether t is a contiguous tensor of this dtype and shape (a tuple, or None for any).
bool fits(const at::Tensor& t, PyObject* dtype, PyObject* shape) {
  if (!THPDtype_Check(dtype) || t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type)
    return false;
  if (!t.is_cuda() || !t.is_contiguous()) return false;
  if (shape == Py_None) return true;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
  for (int64_t i = 0; i < t.dim(); ++i) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (n != t.size(i)) {
      PyErr_Clear();
      return false;
    }
  }
  return true;
}

PyObject* operands_ptr(Operands* self, PyObject* const* args, Py_ssize_t n) {
  if (n != 4 && n != 5) {
    PyErr_SetString(PyExc_TypeError, "ptr(t, dtype, shape, name, optional=False)");
    return nullptr;
  }
  PyObject* t = args[0];
  if (t == Py_None && n == 5) {
    const int optional = PyObject_IsTrue(args[4]);
    if (optional < 0) return nullptr;
    if (optional) Py_RETURN_NONE;
  }
  try {
    if (THPVariable_Check(t)) {
      const at::Tensor& v = THPVariable_Unpack(t);
      if (fits(v, args[1], args[2])) {
        const int device = static_cast<int>(v.get_device()) + 1;
        if (device > 0 && (self->device == 0 || self->device == device)) {
          self->device = device;
          return PyLong_FromVoidPtr(v.data_ptr());
        }
      }
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  PyObject* refuse = PyObject_GetAttrString(reinterpret_cast<PyObject*>(self), "_refuse");
  if (!refuse) return nullptr;
  PyObject* r = PyObject_CallFunctionObjArgs(refuse, args[0], args[1], args[2], args[3], nullptr);
  Py_DECREF(refuse);
  if (!r) return nullptr;
  Py_DECREF(r);
  PyErr_SetString(PyExc_RuntimeError, "an operand was refused without a reason");
  return nullptr;
}

PyObject* get_index(Operands* self, void*) {
  if (self->device == 0) Py_RETURN_NONE;
  return PyLong_FromLong(self->device - 1);
}

int set_index(Operands* self, PyObject* value, void*) {
  const long i = value ? PyLong_AsLong(value) : -1;
  if (i == -1 && PyErr_Occurred()) return -1;
  if (i < 0 || i >= 1024) {
    PyErr_SetString(PyExc_ValueError, "index of a CUDA device expected");
    return -1;
  }
  self->device = static_cast<int>(i) + 1;
  return 0;
}

PyMethodDef operands_methods[] = {
    {"ptr", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(operands_ptr)), METH_FASTCALL,
     "The address of a checked tensor."},
    {nullptr, nullptr, 0, nullptr}};
PyMemberDef operands_members[] = {
    {"where", T_OBJECT_EX, offsetof(Operands, where), READONLY, "the call's name"},
    {nullptr, 0, 0, 0, nullptr}};
PyGetSetDef operands_getset[] = {
    {"index", reinterpret_cast<getter>(get_index), reinterpret_cast<setter>(set_index),
     "the tensors' CUDA device, or None", nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};
PyTypeObject operands_type = {PyVarObject_HEAD_INIT(nullptr, 0)};

// The bytes that fn makes of each of the lists' tensors, a list's after the other's.
template <class T, class F>
PyObject* each_tensor(PyObject* const* args, Py_ssize_t n, const char* usage, F&& fn) {
  if (n != 2 || !PyList_Check(args[0]) || (args[1] != Py_None && !PyList_Check(args[1]))) {
    PyErr_SetString(PyExc_TypeError, usage);
    return nullptr;
  }
  const Py_ssize_t na = PyList_GET_SIZE(args[0]);
  const Py_ssize_t nb = args[1] == Py_None ? 0 : PyList_GET_SIZE(args[1]);
  PyObject* out = PyBytes_FromStringAndSize(nullptr, (na + nb) * sizeof(T));
  if (!out) return nullptr;
  char* to = PyBytes_AS_STRING(out);
  try {
    for (Py_ssize_t i = 0; i < na + nb; ++i) {
      PyObject* t = i < na ? PyList_GET_ITEM(args[0], i) : PyList_GET_ITEM(args[1], i - na);
      if (!THPVariable_Check(t)) {
        Py_DECREF(out);
        PyErr_Format(PyExc_TypeError, "entry %zd is not a torch.Tensor", i < na ? i : i - na);
        return nullptr;
      }
      const T v = fn(THPVariable_Unpack(t));
      std::memcpy(to + i * sizeof(T), &v, sizeof(T));
    }
  } catch (const std::exception& e) {
    Py_DECREF(out);
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  return out;
}

PyObject* addresses(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return each_tensor<void*>(args, n, "addresses(list, list or None)",
                            [](const at::Tensor& t) { return t.data_ptr(); });
}

struct Layout {
  int64_t elements;
  int32_t dtype;
  int16_t device, contiguous;
};

PyObject* layouts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return each_tensor<Layout>(args, n, "layouts(list, list or None)", [](const at::Tensor& t) {
    return Layout{t.numel(), static_cast<int32_t>(t.scalar_type()),
                  static_cast<int16_t>(t.is_cuda() ? t.get_device() : -1),
                  static_cast<int16_t>(t.is_contiguous())};
  });
}

PyMethodDef module_methods[] = {
    {"addresses", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(addresses)), METH_FASTCALL,
     "The data pointers of the lists' tensors, as bytes."},
    {"layouts", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(layouts)), METH_FASTCALL,
     "The lists' tensors' element counts, dtypes, devices and contiguity, as bytes."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_operands", "Operand checks of the binding.", -1,
                          module_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operands() {
  // objects' layouts belong to a minor version: look before any is made
  int major = 0, minor = 0;
  if (std::sscanf(Py_GetVersion(), "%d.%d", &major, &minor) != 2 || major != PY_MAJOR_VERSION ||
      minor != PY_MINOR_VERSION) {
    PyErr_Format(PyExc_ImportError, "built for Python %d.%d", PY_MAJOR_VERSION, PY_MINOR_VERSION);
    return nullptr;
  }
  operands_type.tp_name = "_operands.Operands";
  operands_type.tp_basicsize = sizeof(Operands);
  operands_type.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_BASETYPE;
  operands_type.tp_new = PyType_GenericNew;
  operands_type.tp_init = reinterpret_cast<initproc>(operands_init);
  operands_type.tp_dealloc = reinterpret_cast<destructor>(operands_dealloc);
  operands_type.tp_methods = operands_methods;
  operands_type.tp_members = operands_members;
  operands_type.tp_getset = operands_getset;
  if (PyType_Ready(&operands_type) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module_def);
  if (!m) return nullptr;
  Py_INCREF(&operands_type);
  if (PyModule_AddObject(m, "Operands", reinterpret_cast<PyObject*>(&operands_type)) < 0 ||
      PyModule_AddStringConstant(m, "TORCH", MOE_BUILT_FOR_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
