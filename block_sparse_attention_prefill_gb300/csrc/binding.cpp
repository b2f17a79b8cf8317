// The tree calls as a decode step makes them: plain tensors on the current
// device, outputs to be made, on the current stream.  Checked, allocated and
// called here they take 4-7 us of the host's time; through ctypes, where each
// look at a tensor is a call of the interpreter's, 10-33 us.
//
// Every function returns its outputs, or the library's error code, or None for
// arguments that are not of that form or not sound: tree.py then looks at them
// one by one, with its messages, and makes the call itself.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include "msa.h"

namespace {

// libmsa's functions, by address
struct Calls {
  decltype(&msa_rope_write) rope_write, rope_write_nvfp4;
  decltype(&msa_tree_mask) tree_mask;
  decltype(&msa_tree_accept) tree_accept, tree_accept_nvfp4;
  decltype(&msa_logprobs) logprobs;
  decltype(&msa_tree_attention) tree_attention;
  decltype(&msa_prefix_attention_workspace_bytes) attention_bytes;
} calls;

// A tensor proper (no subclass), or nullptr.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

int type_of(at::ScalarType t) {
  return t == at::kFloat ? MSA_DTYPE_F32 : t == at::kBFloat16 ? MSA_DTYPE_BF16
         : t == at::kHalf ? MSA_DTYPE_F16 : -1;
}

// The current device, which all tensors of a call have to be on (none where the
// first of them is on no GPU: there may be no GPU to ask).
struct Place {
  int dev;
  explicit Place(const at::Tensor* first) : dev(first && first->is_cuda() ? c10::cuda::current_device() : -2) {}
  bool has(const at::Tensor& t) const { return t.is_cuda() && t.get_device() == dev; }
  bool i32(const at::Tensor* t, int64_t dims) const {
    return t && t->scalar_type() == at::kInt && t->dim() == dims && t->is_contiguous() && has(*t);
  }
  // A new tensor on the current device, with storage of its own: what a caller does
  // with one output (resize_, out=) cannot reach another.
  static at::Tensor empty(at::IntArrayRef size, at::ScalarType type) {
    return at::Tensor(at::detail::empty_generic(size, c10::cuda::CUDACachingAllocator::get(),
                                                c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

// A page pool [num_pages, Hkv, ...] of a format.
bool is_pool(const at::Tensor& t, bool fp4, const Place& at_) {
  return (t.scalar_type() == at::kByte || (t.scalar_type() == at::kFloat8_e4m3fn && !fp4)) && t.dim() == 4 &&
         t.size(2) == (fp4 ? 2 : MSA_PAGE_SIZE) && t.size(3) == (fp4 ? MSA_NVFP4_SLOT_BYTES : 2 * MSA_HEAD_DIM) &&
         t.is_contiguous() && at_.has(t);
}

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

PyObject* outputs(std::initializer_list<at::Tensor> list) {
  PyObject* r = PyTuple_New((Py_ssize_t)list.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : list) {
    PyObject* o = nullptr;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
      if (!o) {
        Py_DECREF(r);
        return nullptr;
      }
    } else {
      o = Py_NewRef(Py_None);
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

bool number(PyObject* o, double* x) {  // (a tensor, which could be read too, is none)
  if (!PyFloat_Check(o) && !PyLong_CheckExact(o)) return false;
  *x = PyFloat_AsDouble(o);
  if (*x == -1.0 && PyErr_Occurred()) return PyErr_Clear(), false;
  return true;
}
bool whole(PyObject* o, int64_t lo, int64_t hi, int64_t* x) {
  if (!PyLong_CheckExact(o)) return false;
  *x = PyLong_AsLongLong(o);
  if (*x == -1 && PyErr_Occurred()) return PyErr_Clear(), false;
  return *x >= lo && *x <= hi;
}

// C++ exceptions become the interpreter's.
template <typename F>
PyObject* guarded(F body) {
  try {
    return body();
  } catch (const c10::OutOfMemoryError&) {
    Py_RETURN_NONE;  // tree.py's own allocation raises it as PyTorch does
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The interpreter's lock given up while the library launches: a launch waits where
// the device's queue is full, and other threads must not wait with it.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() noexcept(false) { PyEval_RestoreThread(state_); }  // (ends the thread where the interpreter has ended)
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};
template <typename F, typename... A>
int launch(F* f, A... a) {
  const Unlocked now;
  return f(a...);
}

// (address of the msa_rope_t, its axes, its weights' device or -1, fp4, q, k, v,
// kv, q_scale, k_scale, v_scale, block_table, cu_seqlens_q, cu_seqlens_k,
// positions)
PyObject* rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 15) Py_RETURN_NONE;
    const msa_rope_t* rope = static_cast<const msa_rope_t*>(PyLong_AsVoidPtr(a[0]));
    int64_t axes, weights;
    if (!rope || !whole(a[1], 1, MSA_ROPE_MAX_AXES, &axes) || !whole(a[2], -1, 1 << 20, &weights)) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    const bool fp4 = a[3] == Py_True, bf16 = a[8] == Py_None;
    const at::Tensor *q = tensor(a[4]), *k = tensor(a[5]), *v = tensor(a[6]), *kv = tensor(a[7]);
    const at::Tensor *table = tensor(a[11]), *cu_q = tensor(a[12]), *cu_k = tensor(a[13]);
    const at::Tensor* pos = a[14] == Py_None ? nullptr : tensor(a[14]);
    const Place here(kv);
    if (!q || !k || !v || !kv || (a[14] != Py_None && !pos) || !is_pool(*kv, fp4, here) ||
        (weights >= 0 && weights != here.dev) || !here.i32(table, 2) || !here.i32(cu_q, 1) || !here.i32(cu_k, 1))
      Py_RETURN_NONE;
    const int64_t T = k->dim() == 3 ? k->size(0) : -1, Hkv = kv->size(1), B = table->size(0);
    const int type = type_of(k->scalar_type());
    auto rows = [&](const at::Tensor& x, int64_t heads) {
      return x.dim() == 3 && x.size(0) == T && (heads < 0 || x.size(1) == heads) && x.size(2) == MSA_HEAD_DIM &&
             x.stride(2) == 1 && x.scalar_type() == k->scalar_type() && here.has(x);
    };
    if (T < 0 || type < 0 || !rows(*k, Hkv) || !rows(*v, Hkv) || !rows(*q, -1) || cu_q->size(0) != B + 1 ||
        cu_k->size(0) != B + 1)
      Py_RETURN_NONE;
    if (pos && !((here.i32(pos, 2) && pos->size(0) >= axes && pos->size(1) == T) ||
                 (axes == 1 && here.i32(pos, 1) && pos->size(0) == T)))
      Py_RETURN_NONE;
    double q_scale = 1.0, k_scale, v_scale;
    if ((!bf16 && !number(a[8], &q_scale)) || !number(a[9], &k_scale) || !number(a[10], &v_scale)) Py_RETURN_NONE;
    const at::Tensor out = here.empty({T, q->size(1), MSA_HEAD_DIM}, bf16 ? at::kBFloat16 : at::kFloat8_e4m3fn);
    const int rc = launch(
        fp4 ? calls.rope_write_nvfp4 : calls.rope_write, rope, data<int32_t>(pos), q->data_ptr(), q->stride(0), q->stride(1), k->data_ptr(), k->stride(0),
        k->stride(1), v->data_ptr(), v->stride(0), v->stride(1), type, out.data_ptr(), bf16, (float)q_scale,
        data<uint8_t>(kv), kv->size(0), (float)k_scale, (float)v_scale, data<int32_t>(table), table->size(1),
        data<int32_t>(cu_q), data<int32_t>(cu_k), B, T, q->size(1), Hkv, nullptr, here.stream());
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// (parents, cu_seqlens_q, cu_seqlens_k, max_seqlen_q)
PyObject* tree_mask(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t most;
    if (n != 4 || !whole(a[3], 0, MSA_TREE_MAX_TOKENS, &most)) Py_RETURN_NONE;
    const at::Tensor *parents = tensor(a[0]), *cu_q = tensor(a[1]), *cu_k = tensor(a[2]);
    const Place here(parents);
    if (!here.i32(parents, 1) || !here.i32(cu_q, 1) || !here.i32(cu_k, 1) || cu_q->size(0) < 1 ||
        cu_k->size(0) != cu_q->size(0))
      Py_RETURN_NONE;
    const int64_t T = parents->size(0);
    const int64_t words = (most + 31) / 32;
    const at::Tensor mask = here.empty({T, words}, at::kInt), positions = here.empty({T}, at::kInt);
    const int rc = launch(calls.tree_mask, data<int32_t>(parents), data<int32_t>(cu_q), data<int32_t>(cu_k),
                          cu_q->size(0) - 1, T, most, data<uint32_t>(mask), data<int32_t>(positions), nullptr,
                          here.stream());
    return rc ? PyLong_FromLong(rc) : outputs({mask, positions});
  });
}

// (q, kv, q_scale, k_scale, v_scale, softmax_scale, block_table, cu_seqlens_q,
// cu_seqlens_k, mask, prefix_pages, max_seqlen_q, max_seqlen_k, want_lse)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 14 || !PyBool_Check(a[13])) Py_RETURN_NONE;
    const at::Tensor *q = tensor(a[0]), *kv = tensor(a[1]), *table = tensor(a[6]), *cu_q = tensor(a[7]);
    const at::Tensor *cu_k = tensor(a[8]), *mask = tensor(a[9]);
    double scale[4];
    int64_t prefix, max_q, max_k;
    for (int i = 0; i < 4; ++i)
      if (!number(a[2 + i], scale + i)) Py_RETURN_NONE;
    if (!whole(a[10], 0, INT64_MAX, &prefix) || !whole(a[11], 0, MSA_TREE_MAX_TOKENS, &max_q) ||
        !whole(a[12], 0, INT64_MAX, &max_k))
      Py_RETURN_NONE;
    const Place here(kv);
    if (!kv || !is_pool(*kv, false, here) || !q || !here.has(*q) || q->dim() != 3 ||
        q->size(2) != MSA_HEAD_DIM || !q->is_contiguous() ||
        (q->scalar_type() != at::kByte && q->scalar_type() != at::kFloat8_e4m3fn) || !here.i32(table, 2) ||
        !here.i32(cu_q, 1) || !here.i32(cu_k, 1) || !here.i32(mask, 2))
      Py_RETURN_NONE;
    const int64_t T = q->size(0), Hq = q->size(1), Hkv = kv->size(1), B = table->size(0);
    if (cu_q->size(0) != B + 1 || cu_k->size(0) != B + 1 || mask->size(0) != T || mask->size(1) * 32 < max_q)
      Py_RETURN_NONE;
    size_t bytes = 0;
    int rc = calls.attention_bytes(B, T, Hq, Hkv, prefix, max_q, max_k, &bytes);
    if (rc) return PyLong_FromLong(rc);
    const at::Tensor workspace = here.empty({(int64_t)bytes}, at::kByte);
    const at::Tensor out = here.empty({T, Hq, MSA_HEAD_DIM}, at::kBFloat16);
    at::Tensor lse;
    if (a[13] == Py_True) lse = here.empty({T, Hq}, at::kFloat);
    rc = launch(calls.tree_attention, data<uint8_t>(q), data<uint8_t>(kv), kv->size(0), (float)scale[0],
                (float)scale[1], (float)scale[2], (float)scale[3], data<int32_t>(table), table->size(1),
                data<int32_t>(cu_q), data<int32_t>(cu_k), data<uint32_t>(mask), mask->size(1), B, T, Hq, Hkv, prefix,
                max_q, max_k, workspace.data_ptr(), bytes, data<uint16_t>(out),
                lse.defined() ? data<float>(lse) : nullptr, nullptr, here.stream());
    return rc ? PyLong_FromLong(rc) : outputs({out, lse});
  });
}

// (fp4, draft_tokens, parents, chosen, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
// kv: a list or tuple of pools, a pool, a tensor [layers, ...] of them or None,
// block_table)
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t most;
    if (n != 9 || !whole(a[6], 0, MSA_TREE_MAX_TOKENS, &most)) Py_RETURN_NONE;
    const bool fp4 = a[0] == Py_True;
    const at::Tensor *drafts = tensor(a[1]), *parents = tensor(a[2]), *chosen = tensor(a[3]);
    const at::Tensor *cu_q = tensor(a[4]), *cu_k = tensor(a[5]);
    const Place here(drafts);
    if (!here.i32(drafts, 1) || !here.i32(parents, 1) || !here.i32(chosen, 1) || !here.i32(cu_q, 1) ||
        !here.i32(cu_k, 1) || cu_q->size(0) < 1 || cu_k->size(0) != cu_q->size(0))
      Py_RETURN_NONE;
    const int64_t T = drafts->size(0), B = cu_q->size(0) - 1;
    if (parents->size(0) != T || chosen->size(0) != T) Py_RETURN_NONE;
    uint8_t* pools[MSA_TREE_MAX_LAYERS];
    int64_t layers = 0, pages = 0, heads = 0;
    auto add = [&](const at::Tensor* t) {
      if (!t || layers == MSA_TREE_MAX_LAYERS || !is_pool(*t, fp4, here)) return false;
      if (layers == 0) pages = t->size(0), heads = t->size(1);
      pools[layers++] = data<uint8_t>(t);
      return t->size(0) == pages && t->size(1) == heads;
    };
    THPObjectPtr held;  // (another thread may change a list during the launch)
    if (PyList_CheckExact(a[7]) || PyTuple_CheckExact(a[7])) {
      held = PySequence_Tuple(a[7]);
      if (!held) return nullptr;
      for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(held.get()); ++i)
        if (!add(tensor(PyTuple_GET_ITEM(held.get(), i)))) Py_RETURN_NONE;
    } else if (const at::Tensor* t = a[7] == Py_None ? nullptr : tensor(a[7])) {
      if (t->dim() != 5) {
        if (!add(t)) Py_RETURN_NONE;
      } else {
        for (int64_t i = 0; i < t->size(0); ++i) {
          const at::Tensor one = t->select(0, i);
          if (!add(&one)) Py_RETURN_NONE;
        }
      }
    } else if (a[7] != Py_None) {
      Py_RETURN_NONE;
    }
    const at::Tensor* table = layers ? tensor(a[8]) : nullptr;
    if (layers && (!here.i32(table, 2) || table->size(0) != B)) Py_RETURN_NONE;
    const at::Tensor tokens = here.empty({B, most}, at::kInt), accepted = here.empty({B}, at::kInt),
                     path = here.empty({B, most}, at::kInt);
    const int rc = launch(
        fp4 ? calls.tree_accept_nvfp4 : calls.tree_accept, data<int32_t>(drafts), data<int32_t>(parents), data<int32_t>(chosen), data<int32_t>(cu_q),
        data<int32_t>(cu_k), B, T, most, pools, layers, pages, heads, data<int32_t>(table),
        table ? table->size(1) : 0, data<int32_t>(tokens), data<int32_t>(accepted), data<int32_t>(path), nullptr,
        here.stream());
    return rc ? PyLong_FromLong(rc) : outputs({tokens, accepted, path});
  });
}

// (logits, tokens, top)
PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t top;
    if (n != 3 || !whole(a[2], 0, MSA_LOGPROBS_MAX_TOP, &top)) Py_RETURN_NONE;
    const at::Tensor* logits = tensor(a[0]);
    const at::Tensor* tokens = a[1] == Py_None ? nullptr : tensor(a[1]);
    const Place here(logits);
    const int type = logits ? type_of(logits->scalar_type()) : -1;
    if (type < 0 || logits->dim() != 2 || !here.has(*logits) || (logits->stride(1) != 1 && logits->size(1) != 1) ||
        (a[1] != Py_None && (!here.i32(tokens, 1) || tokens->size(0) != logits->size(0))))
      Py_RETURN_NONE;
    const int64_t T = logits->size(0);
    at::Tensor logprob, rank;
    if (tokens) logprob = here.empty({T}, at::kFloat), rank = here.empty({T}, at::kInt);
    const at::Tensor entropy = here.empty({T}, at::kFloat), best = here.empty({T, top}, at::kInt),
                     value = here.empty({T, top}, at::kFloat);
    const int rc = launch(calls.logprobs, logits->data_ptr(), logits->stride(0), type, data<int32_t>(tokens), T,
                          logits->size(1), top, tokens ? data<float>(logprob) : nullptr,
                          tokens ? data<int32_t>(rank) : nullptr, data<float>(entropy), data<int32_t>(best),
                          data<float>(value), here.stream());
    return rc ? PyLong_FromLong(rc) : outputs({logprob, rank, entropy, best, value});
  });
}

// The functions' addresses, in the order of Calls.
PyObject* connect(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[8];
  if (n != 8) return PyErr_Format(PyExc_TypeError, "8 addresses are wanted, got %zd", n);
  for (int i = 0; i < 8; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "address %d is NULL", i);
  }
  calls.rope_write = reinterpret_cast<decltype(calls.rope_write)>(at[0]);
  calls.rope_write_nvfp4 = reinterpret_cast<decltype(calls.rope_write_nvfp4)>(at[1]);
  calls.tree_mask = reinterpret_cast<decltype(calls.tree_mask)>(at[2]);
  calls.tree_accept = reinterpret_cast<decltype(calls.tree_accept)>(at[3]);
  calls.tree_accept_nvfp4 = reinterpret_cast<decltype(calls.tree_accept_nvfp4)>(at[4]);
  calls.logprobs = reinterpret_cast<decltype(calls.logprobs)>(at[5]);
  calls.tree_attention = reinterpret_cast<decltype(calls.tree_attention)>(at[6]);
  calls.attention_bytes = reinterpret_cast<decltype(calls.attention_bytes)>(at[7]);
  Py_RETURN_NONE;
}

#define MSA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MSA_METHOD(connect),     MSA_METHOD(rope_write), MSA_METHOD(tree_mask),
                         MSA_METHOD(tree_accept), MSA_METHOD(logprobs),   MSA_METHOD(tree_attention),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "msa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_msa_binding(void) { return PyModule_Create(&module); }
