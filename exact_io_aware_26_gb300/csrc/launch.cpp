// launch.cpp -- the short way from Python to a C entry point: repeats a call whose
// arguments have the sizes, strides, types and devices of an earlier one.
//
// A single-token step makes calls whose kernels take a few microseconds; argument
// checks, parameter structs and ctypes marshalling in Python take several times that.
// They depend on the arguments' shapes alone, so the binding (ops.py) does them once per
// combination and registers the outcome here as a plan: the entry point's address, where
// each of its arguments comes from, and the results to allocate.  run() looks the plan up
// by the tensors' sizes, strides, types and device and the call's scalars, allocates the
// results on the current stream and calls the entry point.  Nothing of a tensor's
// contents, address or identity is kept.
//
// An allocation costs 1.4 us, as much as a launch; so results of up to 1 MB share one (a
// result that is kept keeps at most a few MB of the others), and a workspace is a bare
// block that goes back when the call returns, for work that comes later on the stream.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <memory>
#include <unordered_map>
#include <vector>

namespace {

// Where an argument or a result comes from.
enum Kind : long { kInput = 0, kOutput = 1, kConstant = 2, kStream = 3 };
struct Source {
  long kind;
  long long value;  // index of a tensor, or the constant
};
struct Output {
  std::vector<int64_t> sizes;
  at::ScalarType type;
  size_t bytes = 0;
  size_t offset = 0;    // in the shared block
  bool result = false;  // or a workspace
  bool shared = false;
};
constexpr size_t kShared = 1 << 20, kAlign = 512;

c10::Storage block(size_t bytes) {
  c10::Allocator* from = c10::cuda::CUDACachingAllocator::get();
  return c10::Storage(c10::Storage::use_byte_size_t(), bytes, from->allocate(bytes), from, /*resizable=*/true);
}

at::Tensor tensor_in(const c10::Storage& storage, const Output& o) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::Storage(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(o.type));
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(static_cast<int64_t>(o.offset / c10::elementSize(o.type)));
  impl->set_sizes_contiguous(o.sizes);
  return t;
}
struct Plan {
  Plan() = default;
  Plan(const Plan&) = delete;
  Plan& operator=(const Plan&) = delete;
  ~Plan() {
    Py_XDECREF(scalars);
    Py_XDECREF(keep);
  }
  std::vector<int64_t> signature;
  PyObject* scalars = nullptr;
  PyObject* keep = nullptr;  // what the constants point to
  uintptr_t entry;
  int device;
  std::vector<Source> args, results;
  std::vector<Output> outputs;
  size_t shared = 0;  // bytes of the block of the small results
};

constexpr size_t kMaxPlans = 4096, kMaxArgs = 16, kMaxOutputs = 6;
std::unordered_map<uint64_t, std::vector<std::shared_ptr<Plan>>>* g_plans;
size_t g_count = 0;

void forget() {
  std::unordered_map<uint64_t, std::vector<std::shared_ptr<Plan>>> old;
  old.swap(*g_plans);
  g_count = 0;
}

// The signature of a tuple of tensors and Nones: type, device, sizes and strides of each.
bool sign(long op, PyObject* tensors, std::vector<int64_t>& out) {
  out.clear();
  out.push_back(op);
  const Py_ssize_t n = PyTuple_GET_SIZE(tensors);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = PyTuple_GET_ITEM(tensors, i);
    if (o == Py_None) {
      out.push_back(-1);
      continue;
    }
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "expected a tensor, not %s", Py_TYPE(o)->tp_name);
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) {
      PyErr_SetString(PyExc_TypeError, "expected a strided tensor");
      return false;
    }
    out.push_back(static_cast<int64_t>(t.scalar_type()));
    out.push_back(t.is_cuda() ? t.device().index() : -1);
    const auto sizes = t.sizes(), strides = t.strides();
    out.push_back(static_cast<int64_t>(sizes.size()));
    out.insert(out.end(), sizes.begin(), sizes.end());
    out.insert(out.end(), strides.begin(), strides.end());
  }
  return true;
}

uint64_t hash_of(const std::vector<int64_t>& v, PyObject* scalars, bool& ok) {
  const Py_hash_t s = PyObject_Hash(scalars);
  ok = s != -1;
  uint64_t h = 1469598103934665603ull ^ static_cast<uint64_t>(s);
  for (const int64_t x : v) h = (h ^ static_cast<uint64_t>(x)) * 1099511628211ull;
  return h;
}

// The plan for these arguments; nullptr where there is none (or an error is set).  Held by
// its caller: what a call runs into may register others.
std::shared_ptr<Plan> find(const std::vector<int64_t>& sig, PyObject* scalars, uint64_t h) {
  const auto it = g_plans->find(h);
  if (it == g_plans->end()) return nullptr;
  for (const auto& p : it->second)
    if (p->signature == sig) {
      const int same = PyObject_RichCompareBool(p->scalars, scalars, Py_EQ);
      if (same < 0) return nullptr;
      if (same) return p;
    }
  return nullptr;
}

int call(uintptr_t f, const uintptr_t* a, size_t n) {
  using P = uintptr_t;
  switch (n) {
    case 7: return reinterpret_cast<int (*)(P, P, P, P, P, P, P)>(f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
    case 10:
      return reinterpret_cast<int (*)(P, P, P, P, P, P, P, P, P, P)>(f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7],
                                                                       a[8], a[9]);
    case 12:
      return reinterpret_cast<int (*)(P, P, P, P, P, P, P, P, P, P, P, P)>(f)(a[0], a[1], a[2], a[3], a[4], a[5], a[6],
                                                                             a[7], a[8], a[9], a[10], a[11]);
    case 16:
      return reinterpret_cast<int (*)(P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P)>(f)(
          a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11], a[12], a[13], a[14], a[15]);
    default: return -1;  // register_plan admits no other count
  }
}

// run(op, tensors, scalars): the results, as a tuple; an int, the status, where the entry
// point refused; None where no plan is registered.
PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 3 || !PyLong_Check(args[0]) || !PyTuple_Check(args[1]) || !PyTuple_Check(args[2])) {
    PyErr_SetString(PyExc_TypeError, "run(op, tensors, scalars)");
    return nullptr;
  }
  HANDLE_TH_ERRORS
  static thread_local std::vector<int64_t> sig;
  if (!sign(PyLong_AsLong(args[0]), args[1], sig)) return nullptr;
  bool ok;
  const uint64_t h = hash_of(sig, args[2], ok);
  if (!ok) return nullptr;
  const std::shared_ptr<Plan> p = find(sig, args[2], h);
  if (!p) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
  const int here = c10::cuda::current_device();
  if (here != p->device) {
    PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, the current device is cuda:%d", p->device, here);
    return nullptr;
  }
  at::Tensor out[kMaxOutputs];
  c10::DataPtr scratch[kMaxOutputs];
  c10::Storage shared;
  if (p->shared > 0) shared = block(p->shared);
  for (size_t i = 0; i < p->outputs.size(); ++i) {
    const Output& o = p->outputs[i];
    if (o.result)
      out[i] = tensor_in(o.shared ? shared : block(o.bytes), o);
    else
      scratch[i] = c10::cuda::CUDACachingAllocator::get()->allocate(o.bytes);
  }
  uintptr_t a[kMaxArgs];
  for (size_t i = 0; i < p->args.size(); ++i) {
    const Source& s = p->args[i];
    if (s.kind == kInput) {
      PyObject* o = PyTuple_GET_ITEM(args[1], s.value);
      a[i] = o == Py_None ? 0 : reinterpret_cast<uintptr_t>(THPVariable_Unpack(o).data_ptr());
    } else if (s.kind == kOutput) {
      a[i] = reinterpret_cast<uintptr_t>(p->outputs[s.value].result ? out[s.value].data_ptr() : scratch[s.value].get());
    } else if (s.kind == kStream) {
      a[i] = reinterpret_cast<uintptr_t>(c10::cuda::getCurrentCUDAStream(p->device).stream());
    } else {
      a[i] = static_cast<uintptr_t>(s.value);
    }
  }
  const int status = call(p->entry, a, p->args.size());
  if (status != 0) return PyLong_FromLong(status);
  PyObject* results = PyTuple_New(static_cast<Py_ssize_t>(p->results.size()));
  if (!results) return nullptr;
  for (size_t i = 0; i < p->results.size(); ++i) {
    const Source& s = p->results[i];
    PyObject* o;
    if (s.kind == kInput) {
      o = PyTuple_GET_ITEM(args[1], s.value);
      Py_INCREF(o);
    } else {
      o = THPVariable_Wrap(out[s.value]);
    }
    if (!o) {
      Py_DECREF(results);
      return nullptr;
    }
    PyTuple_SET_ITEM(results, static_cast<Py_ssize_t>(i), o);
  }
  return results;
  END_HANDLE_TH_ERRORS  // out of memory is torch.OutOfMemoryError
}

bool sources(PyObject* list, std::vector<Source>& out, Py_ssize_t tensors, size_t outputs) {
  const Py_ssize_t n = PySequence_Size(list);
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* item = PySequence_GetItem(list, i);
    Source s{};
    const bool ok = item && PyArg_ParseTuple(item, "lL", &s.kind, &s.value);
    Py_XDECREF(item);
    if (!ok) return false;
    if (s.kind < kInput || s.kind > kStream || (s.kind == kInput && (s.value < 0 || s.value >= tensors)) ||
        (s.kind == kOutput && (s.value < 0 || s.value >= static_cast<long long>(outputs)))) {
      PyErr_SetString(PyExc_ValueError, "a source is out of range");
      return false;
    }
    out.push_back(s);
  }
  return n >= 0;
}

// register(op, tensors, scalars, entry, device, args, outputs, results, keep)
PyObject* register_plan(PyObject*, PyObject* args) {
  long op;
  PyObject *tensors, *scalars, *arg_list, *out_list, *res_list, *keep;
  unsigned long long entry;
  int device;
  if (!PyArg_ParseTuple(args, "lO!O!KiOOOO", &op, &PyTuple_Type, &tensors, &PyTuple_Type, &scalars, &entry, &device,
                        &arg_list, &out_list, &res_list, &keep))
    return nullptr;
  try {
    auto p = std::make_shared<Plan>();
    p->entry = static_cast<uintptr_t>(entry);
    p->device = device;
    if (!sign(op, tensors, p->signature)) return nullptr;
    bool ok;
    const uint64_t h = hash_of(p->signature, scalars, ok);
    if (!ok) return nullptr;
    const Py_ssize_t n_out = PySequence_Size(out_list);
    for (Py_ssize_t i = 0; i < n_out; ++i) {
      PyObject* item = PySequence_GetItem(out_list, i);
      PyObject *sizes, *type;
      Output o;
      bool good = item && PyArg_ParseTuple(item, "O!O", &PyTuple_Type, &sizes, &type) && THPDtype_Check(type);
      if (good) {
        o.type = reinterpret_cast<THPDtype*>(type)->scalar_type;
        for (Py_ssize_t k = 0; k < PyTuple_GET_SIZE(sizes); ++k) o.sizes.push_back(PyLong_AsLongLong(PyTuple_GET_ITEM(sizes, k)));
        good = !PyErr_Occurred();
      }
      Py_XDECREF(item);
      if (!good) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "an output is (sizes, dtype)");
        return nullptr;
      }
      p->outputs.push_back(std::move(o));
    }
    if (!sources(arg_list, p->args, PyTuple_GET_SIZE(tensors), p->outputs.size()) ||
        !sources(res_list, p->results, PyTuple_GET_SIZE(tensors), p->outputs.size()))
      return nullptr;
    for (const Source& r : p->results)
      if (r.kind == kOutput) p->outputs[r.value].result = true;
    for (Output& o : p->outputs) {
      o.bytes = c10::elementSize(o.type);
      for (const int64_t k : o.sizes) o.bytes *= static_cast<size_t>(k);
      o.shared = o.result && o.bytes > 0 && o.bytes <= kShared;
      if (!o.shared) continue;
      o.offset = p->shared;
      p->shared += (o.bytes + kAlign - 1) / kAlign * kAlign;
    }
    const size_t n = p->args.size();
    if (!(n == 7 || n == 10 || n == 12 || n == 16) || p->outputs.size() > kMaxOutputs) {
      PyErr_SetString(PyExc_ValueError, "no such count of arguments or outputs");
      return nullptr;
    }
    if (g_count >= kMaxPlans) forget();
    Py_INCREF(scalars);
    Py_INCREF(keep);
    p->scalars = scalars;
    p->keep = keep;
    (*g_plans)[h].push_back(std::move(p));
    ++g_count;
    Py_RETURN_NONE;
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* clear(PyObject*, PyObject*) {
  forget();
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"run", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(run)), METH_FASTCALL, nullptr},
    {"register", register_plan, METH_VARARGS, nullptr},
    {"clear", clear, METH_NOARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_launch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__launch() {
  g_plans = new std::unordered_map<uint64_t, std::vector<std::shared_ptr<Plan>>>;
  return PyModule_Create(&g_module);
}
