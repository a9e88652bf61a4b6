// pkv_binding.cpp -- the Python side of the calls that a speculative decoding
// step makes once per layer (paged_kv_cache_mapping_gb300/speculative.py).
//
// It only marshals: tensors into pkv_tensor descriptors, the tensors' device
// made current, its current stream, and the C ABI's status back.  Those kernels
// take two to four microseconds, and eight descriptors filled from Python took
// eight; here they take a few hundred nanoseconds.  The library's functions are
// handed over by address (bind), so that this module and ctypes use the one
// libpkv.so that the package loads.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pkv.h"

namespace {

PyObject* g_error;  // PkvError

decltype(&pkv_rope_append) f_rope_append;
decltype(&pkv_tree_mask) f_tree_mask;
decltype(&pkv_tree_attention) f_tree_attention;
decltype(&pkv_tree_commit) f_tree_commit;

bool refuse(int status, const std::string& what) {
  if (g_error == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, what.c_str());
  } else if (PyObject* e = PyObject_CallFunction(g_error, "is", status, what.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return false;
}

// Descriptors of a call's tensors, all on one CUDA device.
struct Tensors {
  pkv_tensor t[8];
  int n = 0;
  int dev = -1;
  const char* first = "";

  bool add(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
      return false;
    }
    const at::Tensor& x = THPVariable_Unpack(o);
    if (!x.is_cuda()) return refuse(PKV_ERR_INVALID_ARGUMENT, std::string(name) + " must be a CUDA tensor (there is no CPU path)");
    const int d = x.device().index();
    if (n > 0 && d != dev)
      return refuse(PKV_ERR_INVALID_ARGUMENT, std::string(name) + " is on cuda:" + std::to_string(d) + ", " + first +
                                                  " on cuda:" + std::to_string(dev));
    if (x.dim() > 4) return refuse(PKV_ERR_INVALID_ARGUMENT, std::string(name) + " has more than 4 dimensions");
    pkv_tensor& p = t[n];
    switch (x.scalar_type()) {
      case at::kFloat: p.dtype = PKV_F32; break;
      case at::kBFloat16: p.dtype = PKV_BF16; break;
      case at::kFloat8_e4m3fn: p.dtype = PKV_FP8_E4M3; break;
      case at::kInt: p.dtype = PKV_I32; break;
      case at::kLong: p.dtype = PKV_I64; break;
      default: return refuse(PKV_ERR_UNSUPPORTED, std::string(name) + ": unsupported dtype " + c10::toString(x.scalar_type()));
    }
    p.data = x.data_ptr();
    p.ndim = static_cast<int32_t>(x.dim());
    for (int i = 0; i < p.ndim; ++i) {
      p.shape[i] = x.size(i);
      p.stride[i] = x.stride(i);
    }
    if (n++ == 0) {
      dev = d;
      first = name;
    }
    return true;
  }
};

struct WithoutLock {
  PyThreadState* const state = PyEval_SaveThread();
  ~WithoutLock() { PyEval_RestoreThread(state); }
};

// Runs f(stream) with the device current, without the interpreter lock.
template <typename F>
PyObject* run(int dev, F f) {
  pkv_status rc;
  {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    cudaStream_t st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    const WithoutLock unlocked;
    rc = f(st);
  }
  return PyLong_FromLong(rc);
}

// A method as Python calls it.  PyTorch throws, for a tensor without storage
// (sparse, or under vmap) already when its address is asked for, and no C++
// exception may leave through the interpreter's frames: it becomes a Python one.
template <PyObject* (*kBody)(PyObject* const*, Py_ssize_t)>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return kBody(a, n);
  } catch (python_error& e) {
    e.restore();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// A reference that is given up when it goes out of scope.
struct Held {
  PyObject* o;
  explicit Held(PyObject* p) : o(p) {}
  Held(const Held&) = delete;
  Held& operator=(const Held&) = delete;
  ~Held() { Py_XDECREF(o); }
};

bool want(Py_ssize_t n, Py_ssize_t expected) {
  if (n != expected) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
  return n == expected;
}

bool real(PyObject* o, float& x) {
  x = static_cast<float>(PyFloat_AsDouble(o));
  return PyErr_Occurred() == nullptr;
}

// bind(PkvError, rope_append, tree_mask, tree_attention, tree_commit): addresses as integers
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 5)) return nullptr;
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  f_rope_append = reinterpret_cast<decltype(f_rope_append)>(p[0]);
  f_tree_mask = reinterpret_cast<decltype(f_tree_mask)>(p[1]);
  f_tree_attention = reinterpret_cast<decltype(f_tree_attention)>(p[2]);
  f_tree_commit = reinterpret_cast<decltype(f_tree_commit)>(p[3]);
  Py_RETURN_NONE;
}

// rope_append(q, k, v, positions, slot_mapping, rope, q_out, k_cache, v_cache, k_scale, v_scale)
PyObject* rope_append(PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 11)) return nullptr;
  Tensors t;
  float ks, vs;
  if (!t.add(a[0], "q") || !t.add(a[1], "k") || !t.add(a[2], "v") || !t.add(a[3], "positions") ||
      !t.add(a[4], "slot_mapping") || !t.add(a[6], "q_out") || !t.add(a[7], "k_cache") || !t.add(a[8], "v_cache") ||
      !real(a[9], ks) || !real(a[10], vs))
    return nullptr;
  struct Buffer : Py_buffer {
    ~Buffer() { PyBuffer_Release(this); }
  } b;
  b.obj = nullptr;  // nothing to release until it is filled
  if (PyObject_GetBuffer(a[5], &b, PyBUF_SIMPLE) != 0) return nullptr;
  if (b.len != sizeof(pkv_rope)) {
    PyErr_SetString(PyExc_TypeError, "rope must come from pkv_rope_init");
    return nullptr;
  }
  return run(t.dev, [&](cudaStream_t st) {
    return f_rope_append(&t.t[0], &t.t[1], &t.t[2], &t.t[3], &t.t[4], static_cast<const pkv_rope*>(b.buf), &t.t[5], &t.t[6],
                         &t.t[7], ks, vs, st);
  });
}

// tree_mask(parents, cu_seqlens_q, seq_lens, max_q_len, tree_mask or None, positions or None) -> (status, tree_mask,
// positions); what is None is allocated
PyObject* tree_mask(PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 6)) return nullptr;
  Tensors t;
  if (!t.add(a[0], "parents") || !t.add(a[1], "cu_seqlens_q") || !t.add(a[2], "seq_lens")) return nullptr;
  const long long max_q = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor& parents = THPVariable_Unpack(a[0]);
  const Held mask(a[4] == Py_None ? THPVariable_Wrap(at::empty({parents.dim() == 1 ? parents.size(0) : 0, max_q > 32 ? (max_q - 1) / 32 + 1 : 1},
                                                               parents.options()))
                                  : Py_NewRef(a[4]));
  if (mask.o == nullptr) return nullptr;
  const Held positions(a[5] == Py_None ? THPVariable_Wrap(at::empty(parents.sizes(), parents.options())) : Py_NewRef(a[5]));
  if (positions.o == nullptr || !t.add(mask.o, "tree_mask") || !t.add(positions.o, "positions")) return nullptr;
  const Held rc(run(t.dev, [&](cudaStream_t st) { return f_tree_mask(&t.t[0], &t.t[1], &t.t[2], &t.t[3], &t.t[4], st); }));
  return rc.o != nullptr ? Py_BuildValue("(OOO)", rc.o, mask.o, positions.o) : nullptr;
}

// tree_attention(q, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, tree_mask, scale, k_scale, v_scale, max_q_len,
//                out, workspace)
PyObject* tree_attention(PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 13)) return nullptr;
  Tensors t;
  float scale, ks, vs;
  if (!t.add(a[0], "q") || !t.add(a[1], "cu_seqlens_q") || !t.add(a[2], "seq_lens") || !t.add(a[3], "block_tables") ||
      !t.add(a[4], "k_cache") || !t.add(a[5], "v_cache") || !t.add(a[6], "tree_mask") || !t.add(a[11], "out") ||
      !real(a[7], scale) || !real(a[8], ks) || !real(a[9], vs))
    return nullptr;
  const long long max_q = PyLong_AsLongLong(a[10]);
  if (PyErr_Occurred()) return nullptr;
  if (max_q > INT32_MAX) {
    refuse(PKV_ERR_INVALID_ARGUMENT, "max_q_len beyond int32");
    return nullptr;
  }
  if (!THPVariable_Check(a[12])) {
    PyErr_SetString(PyExc_TypeError, "workspace must be a torch.Tensor");
    return nullptr;
  }
  const at::Tensor& ws = THPVariable_Unpack(a[12]);
  if (!ws.is_cuda() || ws.device().index() != t.dev || !ws.is_contiguous()) {
    refuse(PKV_ERR_INVALID_ARGUMENT, "workspace must be contiguous, on cuda:" + std::to_string(t.dev));
    return nullptr;
  }
  return run(t.dev, [&](cudaStream_t st) {
    return f_tree_attention(&t.t[0], &t.t[1], &t.t[2], &t.t[3], &t.t[4], &t.t[5], &t.t[6], scale, ks, vs,
                            static_cast<int32_t>(max_q < 0 ? 0 : max_q), &t.t[7], ws.data_ptr(), ws.nbytes(), st);
  });
}

// tree_commit(accepted, accepted_lens, cu_seqlens_q, seq_lens, block_tables, k_cache, v_cache, new_seq_lens)
PyObject* tree_commit(PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 8)) return nullptr;
  Tensors t;
  if (!t.add(a[0], "accepted") || !t.add(a[1], "accepted_lens") || !t.add(a[2], "cu_seqlens_q") || !t.add(a[3], "seq_lens") ||
      !t.add(a[4], "block_tables") || !t.add(a[5], "k_cache") || !t.add(a[6], "v_cache") || !t.add(a[7], "new_seq_lens"))
    return nullptr;
  return run(t.dev, [&](cudaStream_t st) {
    return f_tree_commit(&t.t[0], &t.t[1], &t.t[2], &t.t[3], &t.t[4], &t.t[5], &t.t[6], &t.t[7], st);
  });
}

#define PKV_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(method<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PKV_METHOD(bind),           PKV_METHOD(rope_append), PKV_METHOD(tree_mask),
                         PKV_METHOD(tree_attention), PKV_METHOD(tree_commit), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
