// Python entry points of the serving operators (mpk.PagedBatch,
// mpk.DraftVerifier): torch tensors are checked and handed to the C calls.
//
// A serving loop makes two of these calls a layer and a decoding step's are a
// few microseconds of GPU time each, so that argument checks in Python and
// ctypes' conversions (8 us an append, 9 us a verification on the Grace host)
// took longer than the kernels.  Here they take well under one.
//
// Every function returns 0, the C call's status, or a text that says which
// argument is refused; the Python side raises.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "mpk.h"

namespace {

// A refusal on its way out.
struct Refused {
  std::string what;
};
// A Python exception is set.
struct Raised {};

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    throw Refused{std::string(name) + " must be a torch tensor"};
  return THPVariable_Unpack(o);
}
bool here(const at::Tensor& t, at::ScalarType type, int device) {
  return t.defined() && t.scalar_type() == type &&
         t.layout() == at::kStrided && t.is_cuda() &&
         t.device().index() == device;
}
std::string on(int device) { return " on cuda:" + std::to_string(device); }

// Device pointer of a contiguous vector of at least n values; None: null.
template <typename T>
T* vec(PyObject* o, int64_t n, at::ScalarType type, int device,
       const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!here(t, type, device) || t.numel() < n || !t.is_contiguous())
    throw Refused{std::string(name) + " must be a contiguous " +
                  c10::toString(type) + " tensor of " + std::to_string(n) +
                  " values" + on(device)};
  return static_cast<T*>(t.data_ptr());
}
float* floats(PyObject* o, int64_t n, int device, const char* name) {
  return vec<float>(o, n, at::kFloat, device, name);
}
int32_t* ints(PyObject* o, int64_t n, int device, const char* name) {
  return vec<int32_t>(o, n, at::kInt, device, name);
}

struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
};
// [n, width] or [n, heads, head_dim] bf16 rows whose values lie side by side
Rows rows(PyObject* o, int64_t n, int64_t width, int64_t head_dim, int device,
          const char* name) {
  const at::Tensor& t = tensor(o, name);
  bool ok = here(t, at::kBFloat16, device);
  if (ok) {
    const auto sh = t.sizes(), st = t.strides();
    if (t.dim() == 2)
      ok = sh[0] >= n && sh[1] == width && st[1] == 1;
    else
      ok = t.dim() == 3 && sh[0] >= n && sh[2] == head_dim &&
           sh[1] * sh[2] == width && st[2] == 1 &&
           (sh[1] == 1 || st[1] == sh[2]);
  }
  if (!ok)
    throw Refused{std::string(name) + " must be bfloat16 [" +
                  std::to_string(n) + ", " + std::to_string(width) + "]" +
                  on(device) + " with contiguous rows"};
  return Rows{t.data_ptr(), n > 1 ? t.stride(0) : width};
}
// [n, vocab] fp32
const float* matrix(PyObject* o, int64_t n, int64_t vocab, int device,
                    const char* name, int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  if (!here(t, at::kFloat, device) || t.dim() != 2 || t.size(0) < n ||
      t.size(1) != vocab || (vocab > 1 && t.stride(1) != 1))
    throw Refused{std::string(name) + " must be float32 [" +
                  std::to_string(n) + ", " + std::to_string(vocab) + "]" +
                  on(device) + " with contiguous rows"};
  *stride = n > 1 ? t.stride(0) : vocab;
  return static_cast<const float*>(t.data_ptr());
}
// None: torch's current stream; a stream object or an address
void* stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  if (PyLong_Check(o)) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
  }
  PyObject* a = PyObject_GetAttrString(o, "cuda_stream");
  if (!a) throw Raised{};
  void* p = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}
int64_t whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}
double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}
template <typename T>
T* address(PyObject* o) {
  return o == Py_None ? nullptr : reinterpret_cast<T*>(whole(o));
}

// The call, on the tensors' own device and without the interpreter's lock.
template <typename F>
PyObject* call(int device, F f) {
  const c10::cuda::CUDAGuard guard(device);
  mpk_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
      return nullptr;
    }
    return f();
  } catch (const Refused& r) {
    return PyUnicode_FromString(r.what.c_str());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// What a mpk.PagedBatch holds; the structures are its own.
struct Paged {
  const mpk_attn_shape* shape;
  const mpk_token_batch* tok;
  const mpk_kv_cache* kv;
  const mpk_prefix_groups* groups;
  uint32_t* status;
  int64_t layers;
  int device;
};
// What a mpk.DraftVerifier holds.
struct Judge {
  int64_t batch, n_tokens, vocab, max_out;
  uint32_t* status;
  void* ws;
  size_t ws_bytes;
  int device;
};

template <typename T>
PyObject* keep(const T& x, const char* name) {
  T* p = new T(x);
  PyObject* c = PyCapsule_New(p, name, [](PyObject* o) {
    delete static_cast<T*>(PyCapsule_GetPointer(o, PyCapsule_GetName(o)));
  });
  if (!c) delete p;
  return c;
}
template <typename T>
const T& kept(PyObject* c, const char* name) {
  const void* p = PyCapsule_GetPointer(c, name);
  if (!p) throw Raised{};
  return *static_cast<const T*>(p);
}

// paged(shape, tok, kv, groups, status, layers, device)
PyObject* paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    return keep(Paged{address<mpk_attn_shape>(a[0]),
                      address<mpk_token_batch>(a[1]),
                      address<mpk_kv_cache>(a[2]),
                      address<mpk_prefix_groups>(a[3]),
                      address<uint32_t>(a[4]), whole(a[5]),
                      (int)whole(a[6])},
                "paged");
  });
}

int layer_of(const Paged& p, PyObject* o) {
  const int64_t layer = whole(o);
  if (layer < 0 || layer >= p.layers)
    throw Refused{"layer " + std::to_string(layer) + " of " +
                  std::to_string(p.layers)};
  return (int)layer;
}

// append(paged, layer, q, k, v, rope, q_out, q_norm, k_norm, eps, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const Paged& p = kept<Paged>(a[0], "paged");
    const mpk_attn_shape& s = *p.shape;
    const int layer = layer_of(p, a[1]);
    const int64_t rw = p.tok->n_tokens, d = s.head_dim;
    const Rows k = rows(a[3], rw, s.n_kv_heads * d, d, p.device, "k");
    const Rows v = rows(a[4], rw, s.n_kv_heads * d, d, p.device, "v");
    Rows q, out;
    if (a[6] != Py_None) {
      if (a[2] == Py_None) throw Refused{"q_out without q"};
      q = rows(a[2], rw, s.n_q_heads * d, d, p.device, "q");
      out = rows(a[6], rw, s.n_q_heads * d, d, p.device, "q_out");
    }
    const void* qn = vec<void>(a[7], d, at::kBFloat16, p.device, "q_norm");
    const void* kn = vec<void>(a[8], d, at::kBFloat16, p.device, "k_norm");
    const float eps = (float)real(a[9]);
    const mpk_rope* rope = address<mpk_rope>(a[5]);
    void* stream = stream_of(a[10], p.device);
    return call(p.device, [&] {
      return mpk_kv_append(p.shape, p.tok, p.kv, layer, q.p, q.stride, k.p,
                           k.stride, v.p, v.stride, qn, kn, eps, rope, out.p,
                           out.stride, p.status, stream);
    });
  });
}

// attend(paged, layer, q, out, lse, scale, workspace, its bytes, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const Paged& p = kept<Paged>(a[0], "paged");
    const mpk_attn_shape& s = *p.shape;
    const int layer = layer_of(p, a[1]);
    const int64_t rw = p.tok->n_tokens, d = s.head_dim;
    const Rows q = rows(a[2], rw, s.n_q_heads * d, d, p.device, "q");
    const Rows out = rows(a[3], rw, s.n_q_heads * d, d, p.device, "out");
    float* lse = floats(a[4], rw * s.n_q_heads, p.device, "lse");
    const float scale = (float)real(a[5]);
    void* ws = address<void>(a[6]);
    const size_t bytes = (size_t)whole(a[7]);
    void* stream = stream_of(a[8], p.device);
    return call(p.device, [&] {
      return mpk_prefix_attention(p.shape, p.tok, p.groups, p.kv, layer, q.p,
                                  q.stride, scale, out.p, out.stride, lse, ws,
                                  bytes, p.status, stream);
    });
  });
}

// judge(batch, n_tokens, vocab, max_out, status, workspace, its bytes, device)
PyObject* judge(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    return keep(Judge{whole(a[0]), whole(a[1]), whole(a[2]), whole(a[3]),
                      address<uint32_t>(a[4]), address<void>(a[5]),
                      (size_t)whole(a[6]), (int)whole(a[7])},
                "judge");
  });
}

// verify(judge, tokens, logits, uniform, noise, n_accepted, out_tokens,
//        q_start, draft, draft_is_logits, temperature, logprobs, next_tokens,
//        seq_lens, seq_lens_out, stream)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    const Judge& j = kept<Judge>(a[0], "judge");
    const int64_t B = j.batch, T = j.n_tokens;
    const int dev = j.device;
    mpk_token_batch tok{};
    tok.batch = (int)B;
    tok.n_tokens = (int)T;
    if (a[7] == Py_None) {
      if (T % B)
        throw Refused{
            "n_tokens must be a multiple of the batch without q_start"};
      tok.tokens_per_seq = (int)(T / B);
    } else {
      tok.q_start = ints(a[7], B + 1, dev, "q_start");
    }
    mpk_verify_args v{};
    v.vocab = (int)j.vocab;
    v.max_out = (int)j.max_out;
    v.tokens = ints(a[1], T, dev, "tokens");
    v.logits = matrix(a[2], T, j.vocab, dev, "logits", &v.logits_stride);
    if (a[8] != Py_None) {
      v.draft = matrix(a[8], T, j.vocab, dev, "draft", &v.draft_stride);
      v.draft_is_logits = PyObject_IsTrue(a[9]);
      if (v.draft_is_logits < 0) throw Raised{};
    }
    v.temperature = floats(a[10], B, dev, "temperature");
    v.uniform = floats(a[3], T, dev, "uniform");
    v.noise = matrix(a[4], B, j.vocab, dev, "noise", &v.noise_stride);
    v.n_accepted = ints(a[5], B, dev, "n_accepted");
    v.out_tokens = ints(a[6], B * j.max_out, dev, "out_tokens");
    v.logprobs = floats(a[11], B * j.max_out, dev, "logprobs");
    v.next_tokens = ints(a[12], B, dev, "next_tokens");
    v.seq_lens = ints(a[13], B, dev, "seq_lens");
    v.seq_lens_out = ints(a[14], B, dev, "seq_lens_out");
    void* stream = stream_of(a[15], dev);
    return call(dev, [&] {
      return mpk_verify_drafts(&tok, &v, j.ws, j.ws_bytes, j.status, stream);
    });
  });
}

#define FAST(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), \
   METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(paged),  FAST(append), FAST(attend),
                         FAST(judge),  FAST(verify), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
