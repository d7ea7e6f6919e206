// Marshalling of torch tensors for the operators around the layer: checks,
// outputs and workspaces, and the call of the C entry point, in one compiled step.
// The smallest calls run for a few microseconds on the GPU; the same steps in
// Python took 20 to 40 microseconds a call.  Everything that is computed is behind
// the C entry points, whose addresses the Python side hands over (bind), so there
// is one copy of the library in the process.
//
// A call makes its tensors' device current, and its stream too when one is given:
// what it allocates belongs to that stream.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <optional>
#include <sstream>
#include <string>

#include "../../include/gsa.h"

namespace {

struct Refused {
  std::string what;
};
template <typename... A>
[[noreturn]] void refuse(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{s.str()};
}

// set by bind()
PyObject* g_error = nullptr;
struct {
  decltype(&gsa_qk_norm_rope) norm_rope;
  decltype(&gsa_qk_norm_rope_backward) norm_rope_backward;
  decltype(&gsa_qk_norm_rope_workspace_bytes) norm_rope_bytes;
  decltype(&gsa_cache_append) append;
  decltype(&gsa_cache_attention) attention;
  decltype(&gsa_cache_attention_workspace_bytes) attention_bytes;
  decltype(&gsa_strerror) strerror;
} g_lib;

constexpr int64_t DIM = 64;

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return &THPVariable_Unpack(o);
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be a number");
  }
  return v;
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, " must be an integer");
  }
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, " is out of range: ", v);
  return static_cast<int>(v);
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(name, " must be true or false");
  }
  return v == 1;
}

int gsa_type(at::ScalarType t) {
  return t == at::kBFloat16 ? GSA_BF16 : t == at::kFloat ? GSA_FP32 : -1;
}
void expect(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device dev) {
  if (t.scalar_type() != type || t.device() != dev)
    refuse(name, " must be a ", type, " tensor on ", dev, ", got ", t.scalar_type(), " on ", t.device());
}
at::Tensor make(at::IntArrayRef size, at::ScalarType type, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(size, type, dev, std::nullopt));
}

// A contiguous tensor of `size` at `offset` elements of an allocation.
at::Tensor part_of(const at::Tensor& whole, int64_t offset, at::IntArrayRef size) {
  auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
  impl->set_sizes_contiguous(size);
  impl->set_storage_offset(offset);
  return at::Tensor(std::move(impl));
}
// Outputs [outer, tokens, heads, 64] (head_major: heads first) for those of `want`, by their heads.  Small ones
// share one allocation: each takes 0.9 us, as much as a fifth of a small call; large ones are each their own,
// so that one can be freed while another is kept.
constexpr int64_t SHARED_BYTES = 1 << 18;
void make_outputs(at::Tensor (&res)[3], const bool (&want)[3], const int64_t (&heads)[3], int64_t outer, int64_t tokens,
                  bool head_major, at::ScalarType type, c10::Device dev) {
  int64_t all = 0, count = 0;
  for (int i = 0; i < 3; ++i)
    if (want[i]) {
      all += heads[i];
      ++count;
    }
  const bool fits = outer * tokens <= SHARED_BYTES / DIM &&
                    outer * tokens * all * DIM * static_cast<int64_t>(at::elementSize(type)) <= SHARED_BYTES;
  at::Tensor whole;
  if (count > 1 && fits) whole = make({outer * tokens * all * DIM}, type, dev);
  int64_t at = 0;
  for (int i = 0; i < 3; ++i) {
    if (!want[i]) continue;
    const std::array<int64_t, 4> size = head_major ? std::array<int64_t, 4>{heads[i], outer, tokens, DIM}
                                                   : std::array<int64_t, 4>{outer, tokens, heads[i], DIM};
    res[i] = whole.defined() ? part_of(whole, at, size) : make(size, type, dev);
    at += outer * tokens * heads[i] * DIM;
  }
}

// the tensors' device, and the stream if one is given, for the time of the call
struct On {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* stream;
  On(c10::Device dev, PyObject* given) : device(dev) {
    if (given != Py_None) {
      const int64_t raw = integer(given, "stream");
      // 1 and 2 name default streams by their kind, which the allocator's bookkeeping does not know
      if (raw == 1 || raw == 2) refuse("stream must be 0 or the handle of a stream, got ", raw);
      auto* h = reinterpret_cast<cudaStream_t>(raw);
      guard.emplace(c10::cuda::getStreamFromExternal(h, dev.index()));
      stream = h;
    } else {
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
  }
};

// [outer, tokens, heads, 64], or [heads, outer, tokens, 64]
struct Shape {
  int64_t outer = -1, tokens = -1;
};
gsa_rows rows4(const at::Tensor& t, const char* name, at::ScalarType type, c10::Device dev, bool head_major, Shape& s,
               int64_t heads) {
  expect(t, name, type, dev);
  if (t.dim() != 4 || t.size(3) != DIM) refuse(name, " must have four dimensions, the last of 64, got ", t.sizes());
  const auto n = t.sizes(), st = t.strides();
  const int o = head_major ? 1 : 0, k = head_major ? 2 : 1, h = head_major ? 0 : 2;
  if (s.outer < 0) {
    s.outer = n[o];
    s.tokens = n[k];
  }
  if (n[o] != s.outer || n[k] != s.tokens || (heads >= 0 && n[h] != heads))
    refuse(name, " must have ", s.outer, " x ", s.tokens, " tokens", heads >= 0 ? " and as many heads as its input" : "",
           ", got ", n);
  if (st[3] != 1) refuse(name, ": the 64 channels must be contiguous");
  if (n[h] > INT32_MAX) refuse(name, " has too many heads");
  return gsa_rows{t.data_ptr(), static_cast<int>(n[h]), st[o], st[k], st[h]};
}

const void* affine(const at::Tensor* t, const char* name, at::ScalarType type, c10::Device dev) {
  if (!t) return nullptr;
  expect(*t, name, type, dev);
  if (t->dim() != 1 || t->size(0) != DIM || !t->is_contiguous()) refuse(name, " must be contiguous with shape (64,)");
  return t->data_ptr();
}

struct Positions {
  const int32_t* p = nullptr;
  int64_t so = 0;
  int axes = 0;
};
Positions positions(const at::Tensor* t, const Shape& s, c10::Device dev) {
  Positions r;
  if (!t) return r;
  expect(*t, "positions", at::kInt, dev);
  const int64_t d = t->dim();
  if (d != 2 && d != 3) refuse("positions must be [tokens, axes] or [outer, tokens, axes], got ", t->sizes());
  const auto n = t->sizes(), st = t->strides();
  const int64_t axes = n[d - 1];
  if (n[d - 2] != s.tokens || (d == 3 && n[0] != s.outer) || (axes != 1 && axes != 2))
    refuse("positions must be [", s.tokens, ", axes] or [", s.outer, ", ", s.tokens, ", axes] with 1 or 2 axes, got ", n);
  if ((axes > 1 && st[d - 1] != 1) || (s.tokens > 1 && st[d - 2] != axes))
    refuse("positions: the tokens' coordinates must be contiguous");
  r.p = static_cast<const int32_t*>(t->data_ptr());
  r.so = d == 3 ? st[0] : 0;
  r.axes = static_cast<int>(axes);
  return r;
}

// tensor i of `out`: None, or a sequence of three tensors or Nones.  A sequence may make its items
// as they are asked for (a tensor of three does), so the item is held until its tensor is.
at::Tensor item(PyObject* out, Py_ssize_t i, const char* name) {
  if (out == Py_None) return at::Tensor();
  struct Held {
    PyObject* o;
    ~Held() { Py_XDECREF(o); }
  } held{PySequence_Check(out) && PySequence_Size(out) == 3 ? PySequence_GetItem(out, i) : nullptr};
  if (!held.o) {
    PyErr_Clear();
    refuse("out must be three tensors or Nones");
  }
  const at::Tensor* t = tensor(held.o, name);
  return t ? *t : at::Tensor();
}

// A tensor of the caller's that a call has written (through its pointer): autograd and every other holder of a saved
// tensor learn of it by the version.  Tensors made in inference mode have none.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// No call records a gradient.  Where autograd would (grad mode, and an argument that requires one), a result that the
// call makes says so when a gradient is asked of it; the caller's own memory cannot, and is not written.
bool requires_grad(const at::Tensor* t) { return t && t->requires_grad(); }
// a weight or bias that a call with this norm reads
const at::Tensor* used(int norm, const at::Tensor* t) { return norm == GSA_NORM_NONE ? nullptr : t; }
template <typename... T>
bool recorded(const T*... t) {
  return at::GradMode::is_enabled() && (requires_grad(t) || ...);
}
constexpr const char* UNRECORDED = "call it under torch.no_grad() or with detached tensors";
void no_history(const char* op, const char* what) {
  refuse(op, " records no gradient and would write ", what, " with values that require one: ", UNRECORDED);
}
// the results `res` depend on `t`
template <typename... T>
void no_gradient(const char* op, const char* instead, std::initializer_list<at::Tensor> res, const T*... t) {
  torch::autograd::edge_list edges;
  for (const at::Tensor* x : {t...})
    if (requires_grad(x)) edges.push_back(torch::autograd::impl::gradient_edge(*x));
  auto node = std::make_shared<torch::autograd::Error>(
      std::string(op) + " records no gradient: " + instead + UNRECORDED, std::move(edges));
  for (const at::Tensor& r : res)
    if (r.defined()) torch::autograd::set_history(r, node);
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
void check(int rc, const char* what) {
  if (rc != GSA_OK) refuse(what, " failed: ", g_lib.strerror(rc), " (status ", rc, ")");
}

template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    if (!g_error) refuse("the library is not bound");
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("expected ", want, " arguments, got ", n);
}

// q, k, v, norm, eps, q_weight, q_bias, k_weight, k_bias, positions, rope_base, head_major, out, stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 14);
    static const char* names[3] = {"q", "k", "v"};
    static const char* outs[3] = {"q output", "k output", "v output"};
    const at::Tensor* in[3];
    const at::Tensor* first = nullptr;
    for (int i = 2; i >= 0; --i)
      if ((in[i] = tensor(a[i], names[i]))) first = in[i];
    if (!first) refuse("nothing to do: q, k and v are None");
    if (!first->is_cuda()) refuse("q, k, v must be CUDA tensors");
    const auto type = first->scalar_type();
    const auto dev = first->device();
    if (gsa_type(type) < 0) refuse("q, k, v must be bfloat16 or float32, got ", type);
    On on(dev, a[13]);
    const bool head_major = truth(a[11], "head_major");
    Shape s;
    gsa_rows ri[3], ro[3];
    const gsa_rows *pi[3] = {}, *po[3] = {};
    at::Tensor res[3];
    bool want[3] = {};
    int64_t heads[3] = {};
    for (int i = 0; i < 3; ++i) {
      if (!in[i]) continue;
      ri[i] = rows4(*in[i], names[i], type, dev, false, s, -1);
      heads[i] = ri[i].heads;
      res[i] = item(a[12], i, outs[i]);
      want[i] = !res[i].defined();
    }
    const int norm = small(a[3], "norm");
    const at::Tensor* w[3] = {tensor(a[5], "q_weight"), tensor(a[7], "k_weight"), nullptr};
    const at::Tensor* b[3] = {tensor(a[6], "q_bias"), tensor(a[8], "k_bias"), nullptr};
    for (int i = 0; i < 3; ++i)
      if (in[i] && !want[i] && recorded(in[i], used(norm, w[i]), used(norm, b[i]), &res[i])) no_history("qk_norm_rope", outs[i]);
    make_outputs(res, want, heads, s.outer, s.tokens, head_major, type, dev);
    for (int i = 0; i < 3; ++i) {
      if (!in[i]) continue;
      ro[i] = rows4(res[i], outs[i], type, dev, head_major, s, heads[i]);
      pi[i] = &ri[i];
      po[i] = &ro[i];
    }
    const Positions p = positions(tensor(a[9], "positions"), s, dev);
    const gsa_norm_rope op{gsa_type(type), norm, static_cast<float>(number(a[4], "eps")), p.axes,
                           number(a[10], "rope_base")};
    check(g_lib.norm_rope(&op, s.outer, s.tokens, pi[0], pi[1], pi[2], po[0], po[1], po[2],
                          affine(w[0], "q_weight", type, dev), affine(b[0], "q_bias", type, dev),
                          affine(w[1], "k_weight", type, dev), affine(b[1], "k_bias", type, dev), p.p, p.so, on.stream),
          "gsa_qk_norm_rope");
    for (int i = 0; i < 3; ++i) {
      if (!in[i]) continue;
      if (!want[i]) written(res[i]);
      else if (recorded(in[i], used(norm, w[i]), used(norm, b[i])))
        no_gradient("qk_norm_rope", "its gradients are those of qk_norm_rope_backward; ", {res[i]}, in[i], used(norm, w[i]),
                    used(norm, b[i]));
    }
    PyObject* t = PyTuple_New(3);
    for (int i = 0; i < 3; ++i) PyTuple_SET_ITEM(t, i, wrap(res[i]));
    return t;
  });
}

// q, k, dq, dk, dv, norm, eps, q_weight, q_bias, k_weight, k_bias, positions, rope_base, head_major, out, stream
PyObject* norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 16);
    static const char* names[3] = {"dq", "dk", "dv"};
    static const char* outs[3] = {"dq output", "dk output", "dv output"};
    static const char* xnames[2] = {"q", "k"};
    const at::Tensor* g[3];
    const at::Tensor* first = nullptr;
    for (int i = 2; i >= 0; --i)
      if ((g[i] = tensor(a[2 + i], names[i]))) first = g[i];
    if (!first) refuse("nothing to do: dq, dk and dv are None");
    if (!first->is_cuda()) refuse("dq, dk, dv must be CUDA tensors");
    const auto gtype = first->scalar_type();
    const auto dev = first->device();
    const at::Tensor* x[2];
    at::ScalarType type = gtype;
    for (int i = 1; i >= 0; --i)
      if ((x[i] = g[i] ? tensor(a[i], xnames[i]) : nullptr)) type = x[i]->scalar_type();
    if (gsa_type(gtype) < 0 || gsa_type(type) < 0)
      refuse("inputs and gradients must be bfloat16 or float32, got ", type, " and ", gtype);
    const int norm = small(a[5], "norm");
    const bool normed = norm != GSA_NORM_NONE;
    On on(dev, a[15]);
    const bool head_major = truth(a[13], "head_major");
    Shape s;
    gsa_rows rx[2], rg[3], rd[3];
    const gsa_rows *px[2] = {}, *pg[3] = {}, *pd[3] = {};
    at::Tensor res[3], all_sums, sums[4];
    bool want[3] = {};
    int64_t heads[3] = {};
    float* ps[4] = {};
    for (int i = 0; i < 3; ++i) {
      if (!g[i]) continue;
      rg[i] = rows4(*g[i], names[i], gtype, dev, head_major, s, -1);
      heads[i] = rg[i].heads;
      pg[i] = &rg[i];
      if (i < 2 && normed) {
        if (!x[i]) refuse(names[i], " needs its input ", xnames[i]);
        rx[i] = rows4(*x[i], xnames[i], type, dev, false, s, heads[i]);
        px[i] = &rx[i];
        for (int b = 0; b < 2; ++b) {              // a bias has a gradient when it is given
          if (b == 1 && a[8 + 2 * i] == Py_None) continue;
          if (!all_sums.defined()) all_sums = make({4 * DIM}, at::kFloat, dev);
          sums[2 * i + b] = part_of(all_sums, (2 * i + b) * DIM, {DIM});
          ps[2 * i + b] = sums[2 * i + b].data_ptr<float>();
        }
      }
      res[i] = item(a[14], i, outs[i]);
      want[i] = !res[i].defined();
    }
    make_outputs(res, want, heads, s.outer, s.tokens, false, gtype, dev);
    for (int i = 0; i < 3; ++i) {
      if (!g[i]) continue;
      rd[i] = rows4(res[i], outs[i], gtype, dev, false, s, heads[i]);
      pd[i] = &rd[i];
    }
    const Positions p = positions(tensor(a[11], "positions"), s, dev);
    const gsa_norm_rope op{gsa_type(type), norm, static_cast<float>(number(a[6], "eps")), p.axes,
                           number(a[12], "rope_base")};
    at::Tensor ws;
    size_t bytes = 0;
    if (normed) {
      bytes = g_lib.norm_rope_bytes();
      ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    }
    check(g_lib.norm_rope_backward(&op, gsa_type(gtype), s.outer, s.tokens, px[0], px[1], pg[0], pg[1], pg[2], pd[0],
                                   pd[1], pd[2], affine(tensor(a[7], "q_weight"), "q_weight", type, dev),
                                   affine(tensor(a[9], "k_weight"), "k_weight", type, dev), p.p, p.so, ps[0], ps[1],
                                   ps[2], ps[3], normed ? ws.data_ptr() : nullptr, bytes, on.stream),
          "gsa_qk_norm_rope_backward");
    for (int i = 0; i < 3; ++i)
      if (g[i] && !want[i]) written(res[i]);
    static const char* keys[7] = {"dq", "dk", "dv", "dq_weight", "dq_bias", "dk_weight", "dk_bias"};
    PyObject* d = PyDict_New();
    for (int i = 0; i < 7; ++i) {
      PyObject* v = wrap(i < 3 ? res[i] : sums[i - 3]);
      PyDict_SetItemString(d, keys[i], v);
      Py_DECREF(v);
    }
    return d;
  });
}

// a cache's pools and a block table
gsa_kv_cache cache_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table) {
  expect(table, "block_table", at::kInt, k.device());
  if (table.dim() != 2 || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("block_table must be [batch, max_pages] with contiguous rows, got ", table.sizes());
  if (table.size(0) > INT32_MAX || table.size(1) > INT32_MAX || k.size(0) > INT32_MAX) refuse("block_table is too large");
  return gsa_kv_cache{k.data_ptr(), v.data_ptr(), gsa_type(k.scalar_type()), static_cast<int>(k.size(0)),
                      static_cast<int>(k.size(2)), static_cast<int>(k.size(1)),
                      static_cast<const int32_t*>(table.data_ptr()), static_cast<int>(table.size(0)),
                      static_cast<int>(table.size(1)), table.stride(0)};
}
const int32_t* ints(const at::Tensor* t, const char* name, int64_t n, c10::Device dev) {
  if (!t) refuse(name, " must be a tensor");
  expect(*t, name, at::kInt, dev);
  if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous()) refuse(name, " must be contiguous int32 [", n, "]");
  return static_cast<const int32_t*>(t->data_ptr());
}
gsa_rows rows3(const at::Tensor* t, const char* name, at::ScalarType type, c10::Device dev, const at::Tensor* like) {
  if (!t) refuse(name, " must be a tensor");
  expect(*t, name, type, dev);
  if (t->dim() != 3 || t->size(2) != DIM || (like && t->sizes() != like->sizes()))
    refuse(name, " must be [tokens, heads, 64]", like ? " as the others" : "", ", got ", t->sizes());
  if (t->stride(2) != 1) refuse(name, ": the 64 channels must be contiguous");
  if (t->size(1) > INT32_MAX) refuse(name, " has too many heads");
  return gsa_rows{t->data_ptr(), static_cast<int>(t->size(1)), 0, t->stride(0), t->stride(1)};
}
const at::Tensor& given(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(name, " must be a tensor");
  return *t;
}

// k_pages, v_pages, k, v, block_table, start, cu_tokens, norm, eps, k_weight, k_bias, positions, rope_axes, rope_base, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 15);
    const at::Tensor &kp = given(a[0], "k_pages"), &vp = given(a[1], "v_pages");
    const auto type = kp.scalar_type();
    const auto dev = kp.device();
    On on(dev, a[14]);
    const gsa_kv_cache c = cache_of(kp, vp, given(a[4], "block_table"));
    const at::Tensor& k = given(a[2], "k");
    const at::Tensor *v = tensor(a[3], "v"), *w = tensor(a[9], "k_weight"), *b = tensor(a[10], "k_bias");
    const gsa_rows rk = rows3(&k, "k", type, dev, nullptr), rv = rows3(v, "v", type, dev, &k);
    const int norm = small(a[7], "norm");
    if (recorded(&k, v, used(norm, w), used(norm, b), &kp, &vp)) no_history("KVCache.append", "the cache");
    Shape s;
    s.outer = 1;
    s.tokens = k.size(0);
    const Positions p = positions(tensor(a[11], "positions"), s, dev);
    const int axes = small(a[12], "rope_axes");
    if (p.p && p.axes != axes) refuse("positions have ", p.axes, " axes, rope_axes is ", axes);
    const gsa_norm_rope op{gsa_type(type), norm, static_cast<float>(number(a[8], "eps")), axes,
                           number(a[13], "rope_base")};
    check(g_lib.append(&c, &op, s.tokens, &rk, &rv, ints(tensor(a[6], "cu_tokens"), "cu_tokens", c.batch + 1ll, dev),
                       ints(tensor(a[5], "start"), "start", c.batch, dev),
                       affine(w, "k_weight", type, dev), affine(b, "k_bias", type, dev), p.p, on.stream),
          "gsa_cache_append");
    written(kp);
    written(vp);
    Py_RETURN_NONE;
  });
}

// k_pages, v_pages, q, block_table, lengths, cu_tokens, max_new, max_len, causal, softmax_scale, return_lse, out, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 13);
    const at::Tensor &kp = given(a[0], "k_pages"), &vp = given(a[1], "v_pages");
    const auto type = kp.scalar_type();
    const auto dev = kp.device();
    On on(dev, a[12]);
    const gsa_kv_cache c = cache_of(kp, vp, given(a[3], "block_table"));
    const at::Tensor& q = given(a[2], "q");
    const gsa_rows rq = rows3(&q, "q", type, dev, nullptr);
    const int64_t tokens = q.size(0);
    const int max_new = small(a[6], "max_new");
    const int64_t max_len = a[7] == Py_None ? static_cast<int64_t>(c.max_pages) * c.page_size : integer(a[7], "max_len");
    at::Tensor out, lse, ws;
    const at::Tensor* to = tensor(a[11], "out");
    if (to && recorded(&q, &kp, &vp, to)) no_history("KVCache.attention", "out");
    out = to ? *to : make({tokens, q.size(1), DIM}, type, dev);
    const gsa_rows ro = rows3(&out, "out", type, dev, &q);
    if (truth(a[10], "return_lse")) lse = make({q.size(1), tokens}, at::kFloat, dev);
    const double given_scale = number(a[9], "softmax_scale");
    const float scale = static_cast<float>(given_scale);
    if (given_scale != 0.0 && scale == 0.f) refuse("softmax_scale is 0 in 32 bits, which stands for 1 / 8: ", given_scale);
    const size_t bytes = g_lib.attention_bytes(&c, tokens, rq.heads, max_new, max_len);
    if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, dev);
    check(g_lib.attention(&c, tokens, &rq, &ro, ints(tensor(a[5], "cu_tokens"), "cu_tokens", c.batch + 1ll, dev),
                          ints(tensor(a[4], "lengths"), "lengths", c.batch, dev), max_new, max_len,
                          truth(a[8], "causal"), scale,
                          lse.defined() ? lse.data_ptr<float>() : nullptr, bytes ? ws.data_ptr() : nullptr, bytes,
                          on.stream),
          "gsa_cache_attention");
    if (to) written(out);
    else if (recorded(&q, &kp, &vp)) no_gradient("KVCache.attention", "", {out, lse}, &q, &kp, &vp);
    if (!lse.defined()) return wrap(out);
    PyObject* t = PyTuple_New(2);
    PyTuple_SET_ITEM(t, 0, wrap(out));
    PyTuple_SET_ITEM(t, 1, wrap(lse));
    return t;
  });
}

// error class, then the addresses of the entry points in the order of g_lib
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes the error class and seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a null address");
      return nullptr;
    }
  }
  g_lib.norm_rope = reinterpret_cast<decltype(g_lib.norm_rope)>(p[0]);
  g_lib.norm_rope_backward = reinterpret_cast<decltype(g_lib.norm_rope_backward)>(p[1]);
  g_lib.norm_rope_bytes = reinterpret_cast<decltype(g_lib.norm_rope_bytes)>(p[2]);
  g_lib.append = reinterpret_cast<decltype(g_lib.append)>(p[3]);
  g_lib.attention = reinterpret_cast<decltype(g_lib.attention)>(p[4]);
  g_lib.attention_bytes = reinterpret_cast<decltype(g_lib.attention_bytes)>(p[5]);
  g_lib.strerror = reinterpret_cast<decltype(g_lib.strerror)>(p[6]);
  Py_XDECREF(g_error);
  g_error = a[0];
  Py_INCREF(g_error);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {{"bind", FAST(bind)},
                         {"norm_rope", FAST(norm_rope)},
                         {"norm_rope_backward", FAST(norm_rope_backward)},
                         {"append", FAST(append)},
                         {"attention", FAST(attention)},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
