// Python's way into the entry points whose callers count microseconds: checks a call's
// tensors and makes the call (module _py_call). A small call is bound by the host: in
// Python each tensor costs five attribute calls, here a few loads.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <tuple>
#include <type_traits>

#include "moe.h"

namespace {

constexpr int kMaxTensors = 16;

// What a call passes beside the descriptor: pointers in the order of the arguments (the
// stream last), a float, a size.
struct Args {
  void* p[kMaxTensors + 1];
  int next = 0;
  double value = 0;
  size_t tail = 0;
};
template <class T>
T take(Args& a) {
  if constexpr (std::is_pointer_v<T>) return static_cast<T>(a.p[a.next++]);
  else if constexpr (std::is_floating_point_v<T>) return static_cast<T>(a.value);
  else return static_cast<T>(a.tail);
}
template <class... A>
moe_status_t make(moe_status_t (*f)(const moe_layer_desc_t*, A...), const moe_layer_desc_t* d, Args& a) {
  std::tuple<A...> args{take<A>(a)...};  // (braces: in order)
  return std::apply([&](A... x) { return f(d, x...); }, args);
}
using Entry = moe_status_t (*)(const moe_layer_desc_t*, Args&);
template <auto F>
moe_status_t entry(const moe_layer_desc_t* d, Args& a) {
  return make(F, d, a);
}
struct Named {
  const char* name;
  Entry call;
};
#define ENTRY(f) {#f, entry<&f>}
constexpr Named kEntries[] = {
    ENTRY(moe_fp8_quantize_weights), ENTRY(moe_permute_fp8), ENTRY(moe_expert_ffn_fwd_fp8),
    ENTRY(moe_combine_bwd_fp8), ENTRY(moe_expert_ffn_bwd_dgrad_fp8), ENTRY(moe_fp4_quantize_weights),
    ENTRY(moe_permute_fp4), ENTRY(moe_expert_ffn_fwd_fp4), ENTRY(moe_rms_norm), ENTRY(moe_rms_norm_bwd)};

struct Spec {
  Entry call;
  int n;
  at::ScalarType type[kMaxTensors];
  bool optional[kMaxTensors];
};
constexpr const char* kSpecName = "moe_call_spec";
void free_spec(PyObject* c) { delete static_cast<Spec*>(PyCapsule_GetPointer(c, kSpecName)); }

// spec(name, ((dtype, may be None), ...)) -> capsule
PyObject* make_spec(PyObject*, PyObject* args) {
  const char* name;
  PyObject* types;
  if (!PyArg_ParseTuple(args, "sO!", &name, &PyTuple_Type, &types)) return nullptr;
  Spec s = {};
  for (const Named& e : kEntries)
    if (!strcmp(e.name, name)) s.call = e.call;
  s.n = (int)PyTuple_GET_SIZE(types);
  if (!s.call || s.n > kMaxTensors) {
    PyErr_Format(PyExc_ValueError, "%s is not a call of this module", name);
    return nullptr;
  }
  for (int i = 0; i < s.n; ++i) {
    PyObject* dtype;
    int optional;
    if (!PyArg_ParseTuple(PyTuple_GET_ITEM(types, i), "Op", &dtype, &optional)) return nullptr;
    if (!THPDtype_Check(dtype)) {
      PyErr_SetString(PyExc_TypeError, "not a dtype");
      return nullptr;
    }
    s.type[i] = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    s.optional[i] = optional;
  }
  return PyCapsule_New(new Spec(s), kSpecName, free_spec);
}

// call(spec, descriptor's address, device, stream, sizes, value, tail, tensors) -> status,
// or None where a tensor is refused: of another type or device, not contiguous, with fewer
// elements than its size, or None where there has to be one.
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8 || !PyTuple_Check(a[4]) || !PyTuple_Check(a[7])) {
    PyErr_SetString(PyExc_TypeError, "call(spec, desc, device, stream, sizes, value, tail, tensors)");
    return nullptr;
  }
  const Spec* s = static_cast<const Spec*>(PyCapsule_GetPointer(a[0], kSpecName));
  if (!s) return nullptr;
  const auto* d = static_cast<const moe_layer_desc_t*>(PyLong_AsVoidPtr(a[1]));
  const long device = PyLong_AsLong(a[2]);
  Args args;
  args.p[s->n] = PyLong_AsVoidPtr(a[3]);
  args.value = PyFloat_AsDouble(a[5]);
  args.tail = PyLong_AsSize_t(a[6]);
  if (PyErr_Occurred()) return nullptr;
  if (PyTuple_GET_SIZE(a[4]) != s->n || PyTuple_GET_SIZE(a[7]) != s->n) {
    PyErr_SetString(PyExc_TypeError, "another number of tensors");
    return nullptr;
  }
  for (int i = 0; i < s->n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(a[7], i);
    if (o == Py_None) {
      if (!s->optional[i]) Py_RETURN_NONE;
      args.p[i] = nullptr;
      continue;
    }
    if (!THPVariable_Check(o)) Py_RETURN_NONE;
    const at::Tensor& t = THPVariable_Unpack(o);
    const long long size = PyLong_AsLongLong(PyTuple_GET_ITEM(a[4], i));
    if (size == -1 && PyErr_Occurred()) return nullptr;
    if (t.layout() != at::kStrided || t.scalar_type() != s->type[i] || !t.is_cuda() ||
        t.get_device() != device || t.numel() < size || !t.is_contiguous())
      Py_RETURN_NONE;
    args.p[i] = t.data_ptr();
  }
  moe_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = s->call(d, args);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// C++ exceptions (of a tensor without storage, say) end here
PyObject* guarded_call(PyObject* m, PyObject* const* a, Py_ssize_t n) {
  try {
    return call(m, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyMethodDef kMethods[] = {
    {"spec", make_spec, METH_VARARGS, nullptr},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(guarded_call)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_py_call", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__py_call(void) {
  PyObject* m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
