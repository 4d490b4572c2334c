// attention_calls.cpp - the quick way from Python to the attention calls of the C ABI.
//
// Checking a dozen tensors in Python takes 15 us, three times as long as the kernels of a
// small decode step. These functions take the usual call - tensors of one CUDA device that is
// the current one, the right types, layouts that need no copy - read the tensors directly and
// call the library, in about 5 us. Anything else, mistakes among it, is not handled here: they
// return None, and the binding in attention.py goes the long way, with its copies and
// its messages. They raise nothing and keep nothing between calls.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "svdq.h"

namespace {

decltype(&svdq_qk_norm_rope) g_norm_rope = nullptr;
decltype(&svdq_kv_append) g_append = nullptr;
decltype(&svdq_attention_prompt) g_prompt = nullptr;
decltype(&svdq_attention_prompt_workspace_size) g_prompt_size = nullptr;
decltype(&svdq_attention_decode) g_decode = nullptr;
decltype(&svdq_attention_decode_workspace_size) g_decode_size = nullptr;

// What one call needs: the device all tensors must live on, and whether all was as expected.
struct Call {
  int device;
  bool good = true;
  Call() : device(c10::cuda::current_device()) {}

  const at::Tensor* tensor(PyObject* o) {   // nullptr for None
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      good = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.get_device() != device || t.layout() != at::kStrided) good = false;
    return &t;
  }
  const at::Tensor* needed(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t) good = false;
    return t;
  }
  // A contiguous vector of n elements, or nothing.
  const void* vector(const at::Tensor* t, at::ScalarType type, int64_t n) {
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) good = false;
    return good ? t->const_data_ptr() : nullptr;
  }
  svdq_stream_t stream() const { return reinterpret_cast<svdq_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream()); }
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The strides of all axes but the last as the library takes them; those of axes of one
// element as a dense tensor has them.
template <int kAxes>
bool outer_strides(const at::Tensor& t, int64_t (&s)[kAxes]) {
  const int64_t dim = t.size(kAxes), size = t.element_size();
  if (t.stride(kAxes) != 1 && dim > 1) return false;
  int64_t dense = (dim + 7) / 8 * 8;
  for (int i = kAxes - 1; i >= 0; --i) {
    s[i] = t.size(i) <= 1 ? dense : t.stride(i);
    if (s[i] * size % 16 != 0 || s[i] < dim) return false;
    dense = std::max(dense, s[i] * t.size(i));
  }
  return aligned16(t.const_data_ptr());
}

// A [tokens, heads, dim] tensor of the given type; tokens and dim below 0: any.
svdq_heads heads(Call& c, const at::Tensor* t, at::ScalarType type, int64_t tokens, int64_t dim) {
  svdq_heads h{nullptr, 0, 0, 0};
  int64_t s[2];
  if (!c.good || !t) return h;
  if (t->scalar_type() != type || t->dim() != 3 || t->size(0) < 1 || t->size(1) < 1 || t->size(1) > INT32_MAX ||
      t->size(2) < 1 || (tokens >= 0 && t->size(0) != tokens) || (dim >= 0 && t->size(2) != dim) ||
      !outer_strides<2>(*t, s)) {
    c.good = false;
    return h;
  }
  h.data = const_cast<void*>(t->const_data_ptr());
  h.token_ld = s[0], h.head_ld = s[1], h.heads = static_cast<int32_t>(t->size(1));
  return h;
}

// The output for x: the given tensor, or a dense new one in *made.
svdq_heads output(Call& c, const at::Tensor* x, const at::Tensor* given, at::Tensor* made) {
  svdq_heads h{nullptr, 0, 0, 0};
  if (!c.good || !x) return h;
  if (given) {
    h = heads(c, given, x->scalar_type(), x->size(0), x->size(2));
    if (h.heads != x->size(1)) c.good = false;
    return h;
  }
  *made = at::empty(x->sizes(), x->options());
  h.data = made->data_ptr();
  h.head_ld = x->size(2), h.token_ld = x->size(1) * x->size(2), h.heads = static_cast<int32_t>(x->size(1));
  return h;
}

svdq_rope rotation(Call& c, PyObject* turns, PyObject* interleaved, PyObject* amplitude, const at::Tensor* positions,
                   int64_t tokens, int64_t dim, const int64_t** at) {
  svdq_rope r{nullptr, 0, 0, 1.0f};
  *at = nullptr;
  const at::Tensor* t = c.tensor(turns);
  if (!c.good || !t) return r;
  const int64_t n = t->numel();
  r.turns = static_cast<const double*>(c.vector(t, at::kDouble, n));
  if (n < 1 || 2 * n > dim || !positions) c.good = false;
  *at = static_cast<const int64_t*>(c.vector(positions, at::kLong, tokens));
  const int truth = PyObject_IsTrue(interleaved);
  const double a = PyFloat_AsDouble(amplitude);
  if (truth < 0 || (a == -1.0 && PyErr_Occurred())) {
    PyErr_Clear();
    c.good = false;
  }
  r.rot_dim = static_cast<int32_t>(2 * n), r.interleaved = truth, r.amplitude = static_cast<float>(a);
  return r;
}

// A norm weight; both of a call have one type.
const void* weight(Call& c, const at::Tensor* w, int64_t dim, const at::Tensor* other, svdq_dtype* type) {
  if (!c.good || !w) return nullptr;
  if (other && other->scalar_type() != w->scalar_type()) c.good = false;
  if (w->scalar_type() != at::kBFloat16 && w->scalar_type() != at::kFloat) c.good = false;
  *type = w->scalar_type() == at::kBFloat16 ? SVDQ_BF16 : SVDQ_F32;
  const void* p = c.vector(w, w->scalar_type(), dim);
  if (!aligned16(p)) c.good = false;
  return p;
}

bool number(PyObject* o, float* x) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *x = static_cast<float>(d);
  return true;
}

// 1 / sqrt(head_dim), rounded once, as the long way has it (in fp32 throughout it is a step off for
// heads of 24, 72, 96 and 112).
float default_scale(int64_t dim) { return static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim))); }

svdq_kv_cache cache(Call& c, const at::Tensor* k, const at::Tensor* v) {
  svdq_kv_cache r{};
  int64_t ks[3], vs[3];
  if (!c.good) return r;
  if (k->dim() != 4 || k->scalar_type() != at::kBFloat16 || v->scalar_type() != at::kBFloat16 ||
      v->sizes() != k->sizes() || k->numel() == 0 || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX ||
      k->size(3) > INT32_MAX || !outer_strides<3>(*k, ks) || !outer_strides<3>(*v, vs) || ks[0] != vs[0] ||
      ks[1] != vs[1] || ks[2] != vs[2]) {
    c.good = false;
    return r;
  }
  r.k = const_cast<void*>(k->const_data_ptr()), r.v = const_cast<void*>(v->const_data_ptr());
  r.pages = k->size(0), r.page_size = static_cast<int32_t>(k->size(1)), r.heads = static_cast<int32_t>(k->size(2));
  r.head_dim = static_cast<int32_t>(k->size(3));
  r.page_ld = ks[0], r.slot_ld = ks[1], r.head_ld = ks[2];
  return r;
}

// The Python object of an output: the one that was given, or that of the new tensor.
PyObject* result(PyObject* given, at::Tensor& made) {
  if (given != Py_None) return Py_NewRef(given);
  return THPVariable_Wrap(std::move(made));
}

// Runs `body`, which returns a new reference or nullptr for "not handled".
template <typename Body>
PyObject* guarded(Body&& body) {
  PyObject* r = nullptr;
  try {
    at::AutoDispatchBelowADInplaceOrView below;   // nothing here is differentiated
    r = body();
  } catch (...) {   // an allocation that failed, say: the long way says so
    r = nullptr;
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// q, k, positions, turns, interleaved, amplitude, q_weight, k_weight, eps, q_out, k_out
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11 || !g_norm_rope) return nullptr;
    Call c;
    const at::Tensor *q = c.needed(a[0]), *k = c.needed(a[1]), *positions = c.tensor(a[2]);
    const at::Tensor *qw = c.tensor(a[6]), *kw = c.tensor(a[7]), *qo = c.tensor(a[9]), *ko = c.tensor(a[10]);
    if (!c.good) return nullptr;
    const at::ScalarType type = q->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return nullptr;
    const svdq_heads qh = heads(c, q, type, -1, -1);
    if (!c.good) return nullptr;
    const int64_t tokens = q->size(0), dim = q->size(2);
    const svdq_heads kh = heads(c, k, type, tokens, dim);
    const int64_t* at = nullptr;
    const svdq_rope rope = rotation(c, a[3], a[4], a[5], positions, tokens, dim, &at);
    svdq_dtype wt = SVDQ_BF16;
    const void* qwp = weight(c, qw, dim, kw, &wt);
    const void* kwp = weight(c, kw, dim, qw, &wt);
    float eps = 0.0f;
    if (!c.good || dim > INT32_MAX || !number(a[8], &eps)) return nullptr;
    at::Tensor made_q, made_k;
    const svdq_heads qoh = output(c, q, qo, &made_q), koh = output(c, k, ko, &made_k);
    if (!c.good || g_norm_rope(qh, kh, type == at::kBFloat16 ? SVDQ_BF16 : SVDQ_F32, tokens, static_cast<int32_t>(dim),
                               at, rope, qwp, kwp, wt, eps, qoh, koh, c.stream()) != SVDQ_OK)
      return nullptr;
    PyObject *r0 = result(a[9], made_q), *r1 = result(a[10], made_k);
    PyObject* both = r0 && r1 ? PyTuple_Pack(2, r0, r1) : nullptr;
    Py_XDECREF(r0);
    Py_XDECREF(r1);
    return both;
  });
}

// k_cache, v_cache, k, v, slots, positions, turns, interleaved, amplitude, k_weight, eps, q, q_weight, q_out, k_out.
// With a q only.
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 15 || !g_append) return nullptr;
    Call c;
    const at::Tensor *kc = c.needed(a[0]), *vc = c.needed(a[1]), *k = c.needed(a[2]), *v = c.needed(a[3]);
    const at::Tensor *slots = c.needed(a[4]), *positions = c.tensor(a[5]), *kw = c.tensor(a[9]), *q = c.needed(a[11]);
    const at::Tensor *qw = c.tensor(a[12]), *qo = c.tensor(a[13]), *ko = c.tensor(a[14]);
    if (!c.good) return nullptr;
    const svdq_kv_cache store = cache(c, kc, vc);
    const int64_t dim = store.head_dim;
    const svdq_heads kh = heads(c, k, at::kBFloat16, -1, dim);
    if (!c.good) return nullptr;
    const int64_t tokens = k->size(0);
    const svdq_heads vh = heads(c, v, at::kBFloat16, tokens, dim), qh = heads(c, q, at::kBFloat16, tokens, dim);
    const int64_t* at = nullptr;
    const svdq_rope rope = rotation(c, a[6], a[7], a[8], positions, tokens, dim, &at);
    const int64_t* slot = static_cast<const int64_t*>(c.vector(slots, at::kLong, tokens));
    svdq_dtype wt = SVDQ_BF16;
    const void* qwp = weight(c, qw, dim, kw, &wt);
    const void* kwp = weight(c, kw, dim, qw, &wt);
    float eps = 0.0f;
    if (!c.good || kh.heads != store.heads || vh.heads != store.heads || !number(a[10], &eps)) return nullptr;
    at::Tensor made;
    const svdq_heads qoh = output(c, q, qo, &made);
    svdq_heads koh{nullptr, 0, 0, 0};
    if (ko) koh = output(c, k, ko, nullptr);
    if (!c.good ||
        g_append(&store, kh, vh, slot, tokens, at, rope, kwp, wt, eps, qh, qwp, qoh, koh, c.stream()) != SVDQ_OK)
      return nullptr;
    return result(a[13], made);
  });
}

// q, k, v, cu_q, cu_k, causal, scale (None: 1 / sqrt(dim)), out. Without a workspace of the caller's.
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8 || !g_prompt) return nullptr;
    Call c;
    const at::Tensor *q = c.needed(a[0]), *k = c.needed(a[1]), *v = c.needed(a[2]);
    const at::Tensor *cu_q = c.tensor(a[3]), *cu_k = c.tensor(a[4]), *out = c.tensor(a[7]);
    const svdq_heads qh = heads(c, q, at::kBFloat16, -1, -1);
    if (!c.good) return nullptr;
    const int64_t dim = q->size(2);
    const svdq_heads kh = heads(c, k, at::kBFloat16, -1, dim);
    if (!c.good) return nullptr;
    const svdq_heads vh = heads(c, v, at::kBFloat16, k->size(0), dim);
    int64_t batch = 1;
    if (cu_q) batch = cu_q->numel() - 1;
    if ((cu_k && cu_q && cu_k->numel() != cu_q->numel()) || (cu_k && !cu_q && cu_k->numel() != 2)) c.good = false;
    const void* cq = c.vector(cu_q, at::kInt, batch + 1);
    const void* ck = c.vector(cu_k, at::kInt, batch + 1);
    const int causal = PyObject_IsTrue(a[5]);
    float scale = default_scale(dim);
    if (!c.good || causal < 0 || batch < 1 || batch > INT32_MAX || dim > INT32_MAX || kh.heads != vh.heads ||
        (a[6] != Py_None && !number(a[6], &scale)))
      return nullptr;
    at::Tensor made, scratch;
    const svdq_heads oh = output(c, q, out, &made);
    size_t bytes = 0;
    if (!c.good || g_prompt_size(qh.heads, kh.heads, static_cast<int32_t>(dim), static_cast<int32_t>(batch), q->size(0),
                                 k->size(0), &bytes) != SVDQ_OK)
      return nullptr;
    if (bytes) scratch = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
    if (g_prompt(qh, kh, vh, static_cast<const int32_t*>(cq), static_cast<const int32_t*>(ck),
                 static_cast<int32_t>(batch), q->size(0), k->size(0), static_cast<int32_t>(dim), causal, scale, oh,
                 bytes ? scratch.data_ptr() : nullptr, bytes, c.stream()) != SVDQ_OK)
      return nullptr;
    return result(a[7], made);
  });
}

// q, k_cache, v_cache, page_table, kv_len, scale (None: 1 / sqrt(dim)), out. Without a workspace of the caller's.
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7 || !g_decode) return nullptr;
    Call c;
    const at::Tensor *q = c.needed(a[0]), *kc = c.needed(a[1]), *vc = c.needed(a[2]), *table = c.needed(a[3]);
    const at::Tensor *lens = c.needed(a[4]), *out = c.tensor(a[6]);
    if (!c.good) return nullptr;
    const svdq_kv_cache store = cache(c, kc, vc);
    const svdq_heads qh = heads(c, q, at::kBFloat16, -1, store.head_dim);
    if (!c.good) return nullptr;
    const int64_t batch = q->size(0);
    const void* len = c.vector(lens, at::kInt, batch);
    float scale = default_scale(store.head_dim);
    if (!c.good || batch > INT32_MAX || table->scalar_type() != at::kInt || table->dim() != 2 || table->size(0) != batch ||
        !table->is_contiguous() || (a[5] != Py_None && !number(a[5], &scale)))
      return nullptr;
    size_t bytes = 0;
    at::Tensor made;
    const svdq_heads oh = output(c, q, out, &made);
    if (!c.good ||
        g_decode_size(static_cast<int32_t>(batch), qh.heads, store.heads, store.head_dim, &bytes) != SVDQ_OK)
      return nullptr;
    const at::Tensor scratch = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
    if (g_decode(qh, &store, static_cast<const int32_t*>(table->const_data_ptr()), table->size(1),
                 static_cast<const int32_t*>(len), static_cast<int32_t>(batch), scale, oh, scratch.data_ptr(), bytes,
                 c.stream()) != SVDQ_OK)
      return nullptr;
    return result(a[6], made);
  });
}

// The addresses of the six functions of the loaded library, in the order above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_prompt = reinterpret_cast<decltype(g_prompt)>(p[2]);
  g_prompt_size = reinterpret_cast<decltype(g_prompt_size)>(p[3]);
  g_decode = reinterpret_cast<decltype(g_decode)>(p[4]);
  g_decode_size = reinterpret_cast<decltype(g_decode_size)>(p[5]);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm_rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prompt)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", "Quick calls of the attention operators.", -1, g_methods,
                        nullptr,               nullptr,  nullptr,                                   nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&g_module); }
