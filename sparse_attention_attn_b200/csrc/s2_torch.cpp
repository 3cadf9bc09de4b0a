// Short way from torch tensors to the C calls of the norm and decoding
// operators, as a CPython extension (_s2torch.so).  Their smallest calls take a
// few microseconds on the GPU, less than the Python checks and ctypes take on
// the host; this does the usual case -- every operand as the call wants it, new
// outputs, the operands' device current -- in one step.  Anything else, and
// any status but OK, returns None: the Python function then takes its own path,
// whose checks name what is wrong.  No arithmetic happens here.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>

#include "s2attn.h"

namespace {

// The C calls, by address: libs2attn.so is loaded (and its build selected) by the ctypes binding.
struct Calls {
  decltype(&s2attn_qknorm_rope_fwd) norm_fwd = nullptr;
  decltype(&s2attn_qknorm_rope_bwd) norm_bwd = nullptr;
  decltype(&s2attn_qknorm_rope_bwd_workspace_bytes) norm_ws = nullptr;
  decltype(&s2attn_cache_append) append = nullptr;
  decltype(&s2attn_cache_plan) plan = nullptr;
  decltype(&s2attn_cache_attn) attn = nullptr;
  decltype(&s2attn_cache_attn_workspace_bytes) attn_ws = nullptr;
} calls;

// The tensor of a plain torch.Tensor or Parameter, else null (subclasses take the Python path).  A tensor
// inside torch.vmap or torch.func.grad is of the plain type too, but has no memory of its own: null.
const at::Tensor* plain(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.has_storage() ? &t : nullptr;
}

bool fits(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape, c10::Device dev) {
  return t != nullptr && t->scalar_type() == type && t->layout() == at::kStrided && t->device() == dev &&
         t->sizes() == shape && t->is_contiguous();
}

// A CUDA tensor of `dims` dimensions on the current device, all sizes in int range.
bool leads(const at::Tensor* t, int64_t dims) {
  if (t == nullptr || !t->is_cuda() || t->dim() != dims || t->get_device() != c10::cuda::current_device()) return false;
  for (const int64_t s : t->sizes())
    if (s > INT_MAX) return false;
  return true;
}

bool small(int64_t v) { return v >= 0 && v <= INT_MAX; }

void* stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

// A float argument; false where it is none.
bool number(PyObject* o, double* v) {
  *v = PyFloat_AsDouble(o);
  if (*v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// Two norm weights [D] of one type; -1: not so, else whether they are fp32.
int weights(const at::Tensor* wq, const at::Tensor* wk, int64_t D, c10::Device dev) {
  if (wq == nullptr) return -1;
  const at::ScalarType t = wq->scalar_type();
  if (t != at::kFloat && t != at::kBFloat16) return -1;
  return fits(wq, t, {D}, dev) && fits(wk, t, {D}, dev) ? t == at::kFloat : -1;
}

// f() without the interpreter lock, which is taken back however f ends: an exception reaches the handlers
// of HANDLE_TH_ERRORS, which use Python.
template <typename F>
int released(F f) {
  struct Release {
    PyThreadState* state = PyEval_SaveThread();
    ~Release() { PyEval_RestoreThread(state); }
  } release;
  return f();
}

template <typename T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* ptr(const at::Tensor* t) {
  return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}

// A new contiguous tensor, straight from the allocator: through the dispatcher each
// costs some 0.2 us more, and a narrowed view 0.8 us (a plan of 64 requests 5.1 us
// a call, 8.6 with them).
at::Tensor fresh_tensor(at::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}

// `n` values of a one-dimensional tensor from `from` on: a tensor on the same memory.
at::Tensor piece(const at::Tensor& t, int64_t from, int64_t n) {
  at::Tensor p = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
  p.unsafeGetTensorImpl()->set_storage_offset(from);
  p.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return p;
}

// Whether the operand, where there is one, has memory: the address 0 (of a tensor inside functionalize)
// would read as the operand's absence.
bool there(const at::Tensor* t) { return t == nullptr || t->const_data_ptr() != nullptr; }

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (out == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}

// (q, k, w_q, w_k, table, eps) -> (q_out, k_out)
PyObject* qknorm_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6 || calls.norm_fwd == nullptr) Py_RETURN_NONE;
  const at::Tensor *q = plain(args[0]), *k = plain(args[1]), *wq = plain(args[2]), *wk = plain(args[3]);
  double eps;
  if (!leads(q, 4) || k == nullptr || k->dim() != 4 || !number(args[5], &eps)) Py_RETURN_NONE;
  const c10::Device dev = q->device();
  const int64_t B = q->size(0), N = q->size(1), H = q->size(2), D = q->size(3), Hkv = k->size(2);
  const int w32 = weights(wq, wk, D, dev);
  if (!small(Hkv) || w32 < 0 || !fits(q, at::kBFloat16, {B, N, H, D}, dev) ||
      !fits(k, at::kBFloat16, {B, N, Hkv, D}, dev) || !fits(plain(args[4]), at::kFloat, {N, D / 2, 2}, dev))
    Py_RETURN_NONE;
  at::Tensor yq = fresh_tensor(q->sizes(), at::kBFloat16, dev), yk = fresh_tensor(k->sizes(), at::kBFloat16, dev);
  const float* table = ptr<float>(plain(args[4]));
  void* s = stream_of(*q);
  const int st = released([&] {
    return calls.norm_fwd(ptr(*q), ptr(*k), ptr(*wq), ptr(*wk), table, ptr(yq), ptr(yk), B, N, H, Hkv, D, w32, eps, s);
  });
  if (st != S2ATTN_OK) Py_RETURN_NONE;
  return tuple_of({yq, yk});
  END_HANDLE_TH_ERRORS
}

// (q, k, w_q, w_k, dq_out, dk_out, table, eps) -> (dq, dk, dw_q, dw_k)
PyObject* qknorm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8 || calls.norm_bwd == nullptr) Py_RETURN_NONE;
  const at::Tensor *q = plain(args[0]), *k = plain(args[1]), *wq = plain(args[2]), *wk = plain(args[3]);
  const at::Tensor *gq = plain(args[4]), *gk = plain(args[5]), *table = plain(args[6]);
  double eps;
  if (!leads(q, 4) || k == nullptr || k->dim() != 4 || !number(args[7], &eps)) Py_RETURN_NONE;
  const c10::Device dev = q->device();
  const int64_t B = q->size(0), N = q->size(1), H = q->size(2), D = q->size(3), Hkv = k->size(2);
  const int w32 = weights(wq, wk, D, dev);
  if (!small(Hkv) || w32 < 0 || !fits(q, at::kBFloat16, {B, N, H, D}, dev) ||
      !fits(k, at::kBFloat16, {B, N, Hkv, D}, dev) || !fits(gq, at::kBFloat16, {B, N, H, D}, dev) ||
      !fits(gk, at::kBFloat16, {B, N, Hkv, D}, dev) || !fits(table, at::kFloat, {N, D / 2, 2}, dev))
    Py_RETURN_NONE;
  const size_t ws = calls.norm_ws(static_cast<int>(D));
  if (ws == 0) Py_RETURN_NONE;
  at::Tensor dq = fresh_tensor(q->sizes(), at::kBFloat16, dev), dk = fresh_tensor(k->sizes(), at::kBFloat16, dev);
  at::Tensor dwq = fresh_tensor({D}, wq->scalar_type(), dev), dwk = fresh_tensor({D}, wq->scalar_type(), dev);
  at::Tensor work = fresh_tensor({static_cast<int64_t>(ws)}, at::kByte, dev);
  void* s = stream_of(*q);
  const int st = released([&] {
    return calls.norm_bwd(ptr(*q), ptr(*k), ptr(*wq), ptr(*wk), ptr<float>(*table), ptr(*gq), ptr(*gk), ptr(dq), ptr(dk),
                          ptr(dwq), ptr(dwk), B, N, H, Hkv, D, w32, eps, ptr(work), ws, s);
  });
  if (st != S2ATTN_OK) Py_RETURN_NONE;
  return tuple_of({dq, dk, dwq, dwk});
  END_HANDLE_TH_ERRORS
}

// (q, k, v, table, positions, slots, k_cache, v_cache, w_q, w_k, eps, q_out) -> q_out; w_q, w_k, q_out may be None
PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12 || calls.append == nullptr) Py_RETURN_NONE;
  const at::Tensor *q = plain(args[0]), *k = plain(args[1]), *v = plain(args[2]), *table = plain(args[3]);
  const at::Tensor *pos = plain(args[4]), *slots = plain(args[5]), *kc = plain(args[6]), *vc = plain(args[7]);
  const bool norm = args[8] != Py_None, fresh = args[11] == Py_None;
  double eps;
  if (!leads(q, 3) || k == nullptr || k->dim() != 3 || table == nullptr || table->dim() != 3 || kc == nullptr ||
      kc->dim() != 4 || norm != (args[9] != Py_None) || !number(args[10], &eps))
    Py_RETURN_NONE;
  const c10::Device dev = q->device();
  const int64_t T = q->size(0), H = q->size(1), D = q->size(2), Hkv = k->size(1), rows = table->size(0);
  const int64_t nb = kc->size(0), bs = kc->size(1);
  const at::Tensor *tq = norm ? plain(args[8]) : nullptr, *tk = norm ? plain(args[9]) : nullptr;
  const int w32 = norm ? weights(tq, tk, D, dev) : 0;
  if (!small(Hkv) || !small(rows) || !small(nb) || !small(bs) || w32 < 0 || !fits(q, at::kBFloat16, {T, H, D}, dev) ||
      !fits(k, at::kBFloat16, {T, Hkv, D}, dev) || !fits(v, at::kBFloat16, {T, Hkv, D}, dev) ||
      !fits(table, at::kFloat, {rows, D / 2, 2}, dev) || !fits(pos, at::kInt, {T}, dev) ||
      !fits(slots, at::kInt, {T}, dev) || !fits(kc, at::kBFloat16, {nb, bs, Hkv, D}, dev) ||
      !fits(vc, at::kBFloat16, {nb, bs, Hkv, D}, dev) ||
      (!fresh && !fits(plain(args[11]), at::kBFloat16, {T, H, D}, dev)) || !there(tq) || !there(tk))
    Py_RETURN_NONE;
  at::Tensor out = fresh ? fresh_tensor(q->sizes(), at::kBFloat16, dev) : *plain(args[11]);
  const void *wq = ptr(tq), *wk = ptr(tk);
  void* s = stream_of(*q);
  const int st = released([&] {
    return calls.append(ptr(*q), ptr(*k), ptr(*v), wq, wk, ptr<float>(*table), ptr<int>(*pos), ptr<int>(*slots), ptr(out),
                        ptr(*kc), ptr(*vc), T, H, Hkv, D, rows, nb * bs, w32, eps, s);
  });
  if (st != S2ATTN_OK) Py_RETURN_NONE;
  if (!fresh) {
    Py_INCREF(args[11]);
    return args[11];
  }
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (ctx_lens, new_lens, block_tables, free_blocks, block_size, num_tokens, parents) ->
// (cu_seqlens, positions, slots, mask or None, counts); parents may be None
PyObject* cache_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7 || calls.plan == nullptr) Py_RETURN_NONE;
  const at::Tensor *ctx = plain(args[0]), *add = plain(args[1]), *tab = plain(args[2]), *free_ = plain(args[3]);
  const bool tree = args[6] != Py_None;
  const at::Tensor* par = tree ? plain(args[6]) : nullptr;
  int64_t bs, T;
  if (!leads(ctx, 1) || tab == nullptr || tab->dim() != 2 || free_ == nullptr || free_->dim() != 1 ||
      !whole(args[4], &bs) || !whole(args[5], &T) || !small(bs) || !small(T) || T == 0)
    Py_RETURN_NONE;
  const c10::Device dev = ctx->device();
  const int64_t R = ctx->size(0), width = tab->size(1), nf = free_->size(0);
  if (!small(width) || !small(nf) || !fits(ctx, at::kInt, {R}, dev) || !fits(add, at::kInt, {R}, dev) ||
      !fits(tab, at::kInt, {R, width}, dev) || !fits(free_, at::kInt, {nf}, dev) ||
      (tree && !fits(par, at::kInt, {T}, dev)) || !there(par))
    Py_RETURN_NONE;
  at::Tensor buf = fresh_tensor({2 * T + R + 5}, at::kInt, dev), mask;  // one allocation for the int32 outputs
  if (tree) mask = fresh_tensor({T}, at::kLong, dev);
  int* p = ptr<int>(buf);
  void* s = stream_of(*ctx);
  const int st = released([&] {
    return calls.plan(ptr<int>(*ctx), ptr<int>(*add), ptr<int>(*tab), ptr<int>(*free_), ptr<int>(par), p + 2 * T, p, p + T,
                      tree ? ptr<int64_t>(mask) : nullptr, p + 2 * T + R + 1, R, width, nf, bs, T, s);
  });
  if (st != S2ATTN_OK) Py_RETURN_NONE;
  PyObject* out = PyTuple_New(5);
  if (out == nullptr) return nullptr;
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(piece(buf, 2 * T, R + 1)));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(piece(buf, 0, T)));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(piece(buf, T, T)));
  if (tree) {
    PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(mask));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, 3, Py_None);
  }
  PyTuple_SET_ITEM(out, 4, THPVariable_Wrap(piece(buf, 2 * T + R + 1, 4)));
  return out;
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, block_tables, ctx_lens, cu_seqlens, mask) -> (o, lse); mask may be None
PyObject* cache_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7 || calls.attn == nullptr) Py_RETURN_NONE;
  const at::Tensor *q = plain(args[0]), *kc = plain(args[1]), *vc = plain(args[2]), *tab = plain(args[3]);
  const bool masked = args[6] != Py_None;
  const at::Tensor* mask = masked ? plain(args[6]) : nullptr;
  if (!leads(q, 3) || kc == nullptr || kc->dim() != 4 || tab == nullptr || tab->dim() != 2) Py_RETURN_NONE;
  const c10::Device dev = q->device();
  const int64_t T = q->size(0), H = q->size(1), D = q->size(2), nb = kc->size(0), bs = kc->size(1), Hkv = kc->size(2);
  const int64_t R = tab->size(0), width = tab->size(1);
  if (!small(nb) || !small(bs) || !small(Hkv) || !small(R) || !small(width) ||
      !fits(q, at::kBFloat16, {T, H, D}, dev) || !fits(kc, at::kBFloat16, {nb, bs, Hkv, D}, dev) ||
      !fits(vc, at::kBFloat16, {nb, bs, Hkv, D}, dev) || !fits(tab, at::kInt, {R, width}, dev) ||
      !fits(plain(args[4]), at::kInt, {R}, dev) || !fits(plain(args[5]), at::kInt, {R + 1}, dev) ||
      (masked && !fits(mask, at::kLong, {T}, dev)) || !there(mask))
    Py_RETURN_NONE;
  const size_t ws = calls.attn_ws(static_cast<int>(D));
  if (ws == 0) Py_RETURN_NONE;
  at::Tensor o = fresh_tensor(q->sizes(), at::kBFloat16, dev), lse = fresh_tensor({H, T}, at::kFloat, dev);
  at::Tensor work = fresh_tensor({static_cast<int64_t>(ws)}, at::kByte, dev);
  const int *ctx = ptr<int>(plain(args[4])), *cu = ptr<int>(plain(args[5]));
  void* s = stream_of(*q);
  const int st = released([&] {
    return calls.attn(ptr(*q), ptr(*kc), ptr(*vc), ptr<int>(*tab), ctx, cu, ptr<int64_t>(mask), ptr(o), ptr<float>(lse), T,
                      R, H, Hkv, D, nb, bs, width, ptr(work), ws, s);
  });
  if (st != S2ATTN_OK) Py_RETURN_NONE;
  return tuple_of({o, lse});
  END_HANDLE_TH_ERRORS
}

// The addresses of the seven C calls, in the order of struct Calls.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  calls.norm_fwd = reinterpret_cast<decltype(calls.norm_fwd)>(p[0]);
  calls.norm_bwd = reinterpret_cast<decltype(calls.norm_bwd)>(p[1]);
  calls.norm_ws = reinterpret_cast<decltype(calls.norm_ws)>(p[2]);
  calls.append = reinterpret_cast<decltype(calls.append)>(p[3]);
  calls.plan = reinterpret_cast<decltype(calls.plan)>(p[4]);
  calls.attn = reinterpret_cast<decltype(calls.attn)>(p[5]);
  calls.attn_ws = reinterpret_cast<decltype(calls.attn_ws)>(p[6]);
  Py_RETURN_NONE;
}

#define S2_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {S2_METHOD(bind),       S2_METHOD(qknorm_fwd),      S2_METHOD(qknorm_bwd), S2_METHOD(cache_append),
                         S2_METHOD(cache_plan), S2_METHOD(cache_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_s2torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this was compiled against (the loader compares it with the library and the torch it finds).
#ifndef S2ATTN_HEADER_HASH
#define S2ATTN_HEADER_HASH "unknown"
#endif
#ifndef S2TORCH_VERSION
#define S2TORCH_VERSION "unknown"
#endif

PyMODINIT_FUNC PyInit__s2torch() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && (PyModule_AddStringConstant(m, "header_hash", S2ATTN_HEADER_HASH) != 0 ||
                       PyModule_AddStringConstant(m, "torch_version", S2TORCH_VERSION) != 0)) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
