// CPython helper of the binding: device pointers of torch tensors whose device, type, shape and
// contiguity it checks.
//
// A drafted step makes half a dozen calls of a few microseconds each, with up to fifteen
// tensors. Asking each tensor through its Python methods costs about 0.4 us, more in all than
// the launches; reading the tensor objects directly costs a few nanoseconds.
#include <exception>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject* g_refuse = nullptr;  // refuse(tensor, name, dtype, dev, shape) raises what is wrong

// Raises through `refuse`, which knows how to say it.
void refuse(PyObject* t, PyObject* name, PyObject* dtype, PyObject* dev, PyObject* shape) {
  if (g_refuse != nullptr) {
    PyObject* r = PyObject_CallFunctionObjArgs(g_refuse, t, name, dtype, dev, shape, nullptr);
    Py_XDECREF(r);
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a tensor does not fit the call");
}

// Tensors of some kinds throw where their memory or sizes are asked for (batched by a transform,
// nested, sparse): f's exceptions become Python's, none may reach the interpreter's C frames.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (python_error& e) {
    e.restore();
  } catch (const c10::Error& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a tensor could not be read");
  return nullptr;
}

// A shape's entry that is no integer leaves a Python error behind.
bool same_shape(const at::Tensor& t, PyObject* shape) {
  if (shape == Py_None) return true;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != t.dim()) return false;
  for (Py_ssize_t i = 0; i < t.dim(); ++i)
    if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != t.size(i)) return false;
  return true;
}

// The tensor behind a Python object on CUDA device `dev` with type `dtype`, or null.
const at::Tensor* tensor_on(PyObject* o, PyObject* dtype, long dev) {
  if (!THPVariable_Check(o) || !THPDtype_Check(dtype)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != dev ||
      t.scalar_type() != reinterpret_cast<THPDtype*>(dtype)->scalar_type)
    return nullptr;
  return &t;
}

// ptrs(dev, tensor, name, dtype, shape, tensor, name, dtype, shape, ...) -> pointers.
// A tensor may be None (its pointer is None), a shape None (any).
PyObject* ptrs(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n < 1 || (n - 1) % 4 != 0) {
    PyErr_SetString(PyExc_TypeError, "ptrs(dev, tensor, name, dtype, shape, ...)");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[0]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  const Py_ssize_t count = (n - 1) / 4;
  PyObject* out = PyTuple_New(count);
  if (out == nullptr) return nullptr;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject* const* a = args + 1 + 4 * i;
    PyObject* p = nullptr;
    if (a[0] == Py_None) {
      p = Py_NewRef(Py_None);
    } else {
      p = guarded([&]() -> PyObject* {
        const at::Tensor* t = tensor_on(a[0], a[2], dev);
        if (t != nullptr && t->is_contiguous() && same_shape(*t, a[3]))
          return PyLong_FromVoidPtr(t->data_ptr());
        if (!PyErr_Occurred()) refuse(a[0], a[1], a[2], args[0], a[3]);
        return nullptr;
      });
      if (p == nullptr) {
        Py_DECREF(out);
        return nullptr;
      }
    }
    PyTuple_SET_ITEM(out, i, p);
  }
  return out;
}

// rows(dev, tensor, name, dtype, shape) -> (pointer, stride of the first dimension) of rows
// [T, heads, d] that may be strided along T.
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "rows(dev, tensor, name, dtype, shape)");
    return nullptr;
  }
  const long dev = PyLong_AsLong(args[0]);
  if (dev == -1 && PyErr_Occurred()) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor* t = tensor_on(args[1], args[3], dev);
    if (t == nullptr || t->dim() != 3 || !same_shape(*t, args[4]) ||
        (t->stride(2) != 1 && t->size(2) > 1) || (t->stride(1) != t->size(2) && t->size(1) > 1)) {
      if (!PyErr_Occurred()) refuse(args[1], args[2], args[3], args[0], args[4]);
      return nullptr;
    }
    // a single row has no stride of its own
    const int64_t stride = t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
    return Py_BuildValue("NL", PyLong_FromVoidPtr(t->data_ptr()), (long long)stride);
  });
}

PyObject* on_refusal(PyObject*, PyObject* f) {
  Py_XSETREF(g_refuse, Py_NewRef(f));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"ptrs", (PyCFunction)(void (*)(void))ptrs, METH_FASTCALL,
     "ptrs(dev, tensor, name, dtype, shape, ...) -> tuple of device pointers"},
    {"rows", (PyCFunction)(void (*)(void))rows, METH_FASTCALL,
     "rows(dev, tensor, name, dtype, shape) -> (device pointer, row stride)"},
    {"on_refusal", on_refusal, METH_O, "sets the function that says what does not fit"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void) { return PyModule_Create(&module); }
