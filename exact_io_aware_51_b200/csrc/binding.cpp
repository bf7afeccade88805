// Python calls of the operators around the attention: argument checks, output
// tensors and the call of the C ABI, in C++ (the CPython module `_binding`).
//
// The GPU takes 2 to 6 us for one token of a batch; the same checks and
// allocations spelled out in Python took 9 to 17 us a call, which is what a decode
// loop then waits for.  Nothing is computed here: every function checks its
// tensors as the header asks, allocates outputs and scratch from PyTorch on the
// current stream (so a temporary's memory is only handed out again behind the
// kernels that use it), and calls one entry point of the library that the package
// has loaded (their addresses come through init()).
#include <Python.h>

#include <array>
#include <climits>
#include <cmath>
#include <memory>
#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

using at::Tensor;

struct Api {
  decltype(&fa_qk_norm_rope) norm_rope;
  decltype(&fa_qk_norm_rope_bwd) norm_rope_bwd;
  decltype(&fa_qk_norm_rope_workspace_size) norm_rope_ws;
  decltype(&fa_cache_append) append;
  decltype(&fa_cache_read) read;
  decltype(&fa_decode_paged_fp8) decode;
  decltype(&fa_decode_fp8_workspace_size) decode_ws;
};
Api api = {};
PyObject* error_class = nullptr;  // FAError

// A status of the library on its way to Python
struct Status : std::runtime_error {
  Status(int rc_, const char* name_) : std::runtime_error(std::string(name_) + ": status " + std::to_string(rc_)), rc(rc_), name(name_) {}
  int rc;
  const char* name;
};

void check_status(int rc, const char* name) {
  if (rc != FA_OK) throw Status(rc, name);
}

int as_int(int64_t v, const char* what) {
  TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, what, " is out of range");
  return static_cast<int>(v);
}

const void* ptr(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* mut(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The device that a call runs on, made current for its duration, and its current stream.
struct Here {
  explicit Here(const Tensor& t) : guard(t.device()), handle(c10::cuda::getCurrentCUDAStream(t.get_device()).stream()) {}
  c10::cuda::CUDAGuard guard;
  void* handle;
};

// The C call itself runs without the interpreter's lock where this thread holds it
// (autograd's threads do not): a full launch queue would make it wait.  The lock is taken back on
// every way out: asking a tensor without storage (under vmap, say) for its pointer throws.
template <typename F>
int call_unlocked(F&& f) {
  struct Unlocked {
    PyThreadState* s = PyGILState_Check() ? PyEval_SaveThread() : nullptr;
    ~Unlocked() {
      if (s) PyEval_RestoreThread(s);
    }
  } unlocked;
  return f();
}

// (batch, position, head) strides of a [B, N, heads, d] tensor whose features are contiguous
struct Strides {
  std::array<long long, 3> s{};
  bool dense = true;
  const long long* get() const { return dense ? nullptr : s.data(); }
  Strides(const Tensor& t, const char* name) {
    if (t.is_contiguous() || t.numel() == 0) return;
    dense = false;
    TORCH_CHECK_VALUE(t.stride(3) == 1, name, ": the features of a head must be contiguous");
    const int64_t unit = 16 / t.element_size();
    for (int i = 0; i < 3; ++i) {
      s[i] = t.size(i) == 1 ? 0 : t.stride(i);
      TORCH_CHECK_VALUE(s[i] % unit == 0, name, ": strides must be multiples of 16 bytes");
    }
  }
};

void check_out(const Tensor& t, at::IntArrayRef shape, at::ScalarType type, const Tensor& like, const char* name) {
  TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == type && t.device() == like.device() && t.is_contiguous(),
                    name, " must be a contiguous ", type, " tensor of shape ", shape, " on ", like.device());
}

// A caller's tensor that a call writes: autograd has to know, so that a graph that saved it for its
// backward refuses to run, as after any in-place operation
void will_write(const Tensor& t, const char* name) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(!(at::GradMode::is_enabled() && t.requires_grad()), name,
                    " is written in place and must not be one that requires a gradient");
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// a dense tensor on like's device, without the dispatcher's 0.5 us
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}

Tensor out_or_new(const Tensor& given, at::IntArrayRef shape, at::ScalarType type, const Tensor& like, const char* name) {
  if (!given.defined()) return fresh(shape, type, like);
  check_out(given, shape, type, like, name);
  will_write(given, name);
  return given;
}

void check_cuda(const Tensor& t) {
  TORCH_CHECK_VALUE(t.is_cuda(), "tensors must live on a CUDA device (there is no CPU path)");
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, "unsupported dtype ", t.scalar_type(), "; use bfloat16 or float32");
  return FA_FP32;
}

// ---------------------------------------------------------------------------
// Norm and rotation
// ---------------------------------------------------------------------------
struct Rope {
  Tensor q, k, cos, sin, wq, wk, positions;
  double eps;
  bool interleaved;
  int B, N, H, Hkv, d, rows, dtype, wdtype;

  void check() {
    TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4, "expected q [B, N, H, d] and k [B, N, Hkv, d]");
    TORCH_CHECK_VALUE(k.size(0) == q.size(0) && k.size(1) == q.size(1) && k.size(3) == q.size(3),
                      "q and k must agree in batch, positions and head dim");
    dtype = wdtype = dtype_code(q);
    TORCH_CHECK_TYPE(k.scalar_type() == q.scalar_type(), "q and k must have one dtype");
    TORCH_CHECK_TYPE(cos.scalar_type() == at::kFloat && sin.scalar_type() == at::kFloat, "cos and sin must be float32");
    TORCH_CHECK_VALUE(cos.dim() == 2 && cos.size(1) * 2 == q.size(3) && sin.sizes() == cos.sizes(),
                      "cos and sin must be [positions, d / 2] tables");
    TORCH_CHECK_VALUE(cos.is_contiguous() && sin.is_contiguous(), "cos and sin must be contiguous");
    TORCH_CHECK_VALUE(wq.defined() == wk.defined(), "give both gains or none");
    bool same = k.device() == q.device() && cos.device() == q.device() && sin.device() == q.device();
    if (wq.defined()) {
      wdtype = dtype_code(wq);
      TORCH_CHECK_TYPE(wk.scalar_type() == wq.scalar_type(), "q_weight and k_weight must have one dtype");
      TORCH_CHECK_VALUE(wq.dim() == 1 && wk.dim() == 1 && wq.size(0) == q.size(3) && wk.size(0) == q.size(3),
                        "q_weight and k_weight must be [d]");
      TORCH_CHECK_VALUE(wq.is_contiguous() && wk.is_contiguous(), "q_weight and k_weight must be contiguous");
      same = same && wq.device() == q.device() && wk.device() == q.device();
    }
    if (positions.defined()) {
      TORCH_CHECK_TYPE(positions.scalar_type() == at::kInt, "positions must be int32");
      TORCH_CHECK_VALUE(positions.dim() == 2 && positions.size(0) == q.size(0) && positions.size(1) == q.size(1) &&
                            positions.is_contiguous(),
                        "positions must be a contiguous [B, N] tensor");
      same = same && positions.device() == q.device();
    } else {
      TORCH_CHECK_VALUE(q.size(1) <= cos.size(0) || q.size(0) == 0, "the tables have fewer rows than there are positions");
    }
    TORCH_CHECK_VALUE(same, "all tensors must share one device");
    check_cuda(q);
    B = as_int(q.size(0), "the batch");
    N = as_int(q.size(1), "the positions");
    H = as_int(q.size(2), "the heads");
    Hkv = as_int(k.size(2), "the heads");
    d = as_int(q.size(3), "the head dim");
    rows = as_int(cos.size(0), "the tables");
  }

  std::pair<Tensor, Tensor> forward(const Tensor& q_out, const Tensor& k_out) const {
    Here here(q);
    const Strides qs(q, "q"), ks(k, "k");
    Tensor qo = out_or_new(q_out, q.sizes(), q.scalar_type(), q, "q_out");
    Tensor ko = out_or_new(k_out, k.sizes(), q.scalar_type(), q, "k_out");
    check_status(call_unlocked([&] {
                   return api.norm_rope(ptr(q), ptr(k), ptr(wq), ptr(wk), cos.const_data_ptr<float>(),
                                        sin.const_data_ptr<float>(), static_cast<const int*>(ptr(positions)), mut(qo),
                                        mut(ko), B, N, H, Hkv, d, qs.get(), ks.get(), rows, static_cast<float>(eps),
                                        interleaved, dtype, wdtype, here.handle);
                 }),
                 "fa_qk_norm_rope");
    return {qo, ko};
  }

  // (dq, dk, dq_weight, dk_weight); the last two undefined without gains
  std::array<Tensor, 4> backward(const Tensor& gq, const Tensor& gk, const Tensor& workspace) const {
    Here here(q);
    const Strides qs(q, "q"), ks(k, "k"), gqs(gq, "dq_out"), gks(gk, "dk_out");
    Tensor dq = fresh(q.sizes(), q.scalar_type(), q), dk = fresh(k.sizes(), q.scalar_type(), q), dwq, dwk, ws = workspace;
    size_t bytes = 0;
    if (wq.defined()) {
      will_write(ws, "workspace");
      dwq = fresh(wq.sizes(), wq.scalar_type(), q);
      dwk = fresh(wk.sizes(), wk.scalar_type(), q);
      if (!ws.defined()) ws = fresh({static_cast<int64_t>(api.norm_rope_ws(d))}, at::kByte, q);
      bytes = ws.nbytes();
    }
    check_status(call_unlocked([&] {
                   return api.norm_rope_bwd(ptr(q), ptr(k), ptr(wq), ptr(wk), cos.const_data_ptr<float>(),
                                            sin.const_data_ptr<float>(), static_cast<const int*>(ptr(positions)), ptr(gq),
                                            ptr(gk), mut(dq), mut(dk), mut(dwq), mut(dwk), B, N, H, Hkv, d, qs.get(),
                                            ks.get(), gqs.get(), gks.get(), rows, static_cast<float>(eps), interleaved,
                                            dtype, wdtype, mut(ws), bytes, here.handle);
                 }),
                 "fa_qk_norm_rope_bwd");
    return {dq, dk, dwq, dwk};
  }
};

// An incoming gradient as the kernels read it: features contiguous, 16-byte strides and base
Tensor readable(const Tensor& g) {
  const int64_t unit = 16 / g.element_size();
  const bool base = reinterpret_cast<uintptr_t>(g.const_data_ptr()) % 16 == 0;
  if (base && (g.is_contiguous() || (g.stride(3) == 1 && g.stride(0) % unit == 0 && g.stride(1) % unit == 0 && g.stride(2) % unit == 0)))
    return g;
  return g.clone(at::MemoryFormat::Contiguous);
}

class RopeFunction : public torch::autograd::Function<RopeFunction> {
 public:
  using Maybe = std::optional<Tensor>;  // apply() takes no undefined tensor
  static Maybe given(const Tensor& t) { return t.defined() ? Maybe(t) : std::nullopt; }
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k,
                                                const Maybe& wq, const Maybe& wk, const Tensor& cos, const Tensor& sin,
                                                const Maybe& positions, double eps, bool interleaved) {
    Rope r{q, k, cos, sin, wq.value_or(Tensor()), wk.value_or(Tensor()), positions.value_or(Tensor()), eps, interleaved};
    r.check();
    ctx->save_for_backward({q, k, r.wq, r.wk, cos, sin, r.positions});
    ctx->saved_data["eps"] = eps;
    ctx->saved_data["interleaved"] = interleaved;
    auto out = r.forward({}, {});
    return {out.first, out.second};
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list g) {
    const auto s = ctx->get_saved_variables();
    Rope r{s[0], s[1], s[4], s[5], s[2], s[3], s[6], ctx->saved_data["eps"].toDouble(), ctx->saved_data["interleaved"].toBool()};
    std::array<Tensor, 4> grads;
    {
      at::NoGradGuard no_grad;
      r.check();
      grads = r.backward(readable(g[0]), readable(g[1]), {});
    }
    torch::autograd::variable_list out(9);
    for (int i = 0; i < 4; ++i) out[i] = grads[i];
    if (at::GradMode::is_enabled()) {  // asked for with create_graph: a second derivative has to fail, not to be left out
      torch::autograd::variable_list some;
      for (auto& t : grads)
        if (t.defined()) some.push_back(t.detach().set_requires_grad(true));
      auto error = std::make_shared<torch::autograd::DelayedError>("qk_norm_rope is differentiable once", some.size());
      some = (*error)(std::move(some));
      size_t j = 0;
      for (int i = 0; i < 4; ++i)
        if (grads[i].defined()) out[i] = some[j++];
    }
    return out;
  }
};

// ---------------------------------------------------------------------------
// Paged cache
// ---------------------------------------------------------------------------
struct Cache {
  Tensor k, v, scale, table, lengths;
  const char* what;  // of the lengths
  bool fp8;
  int pages, page_size, Hkv, d, B, max_pages;

  void check() {
    TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes(), "k_cache and v_cache must be [num_pages, page_size, Hkv, d]");
    const auto type = k.scalar_type();
    fp8 = type == at::kFloat8_e4m3fn || type == at::kByte;
    TORCH_CHECK_TYPE((fp8 || type == at::kBFloat16) && v.scalar_type() == type,
                     "k_cache and v_cache must both be bfloat16, or float8_e4m3fn (or its uint8 codes)");
    bool dense = k.is_contiguous() && v.is_contiguous() && table.is_contiguous() && lengths.is_contiguous();
    bool same = v.device() == k.device() && table.device() == k.device() && lengths.device() == k.device();
    if (fp8) {
      TORCH_CHECK_VALUE(scale.defined(), "an 8-bit cache needs kv_scale [num_pages, Hkv, 2, page_size]");
      TORCH_CHECK_TYPE(scale.scalar_type() == at::kByte || scale.scalar_type() == at::kFloat8_e8m0fnu,
                       "kv_scale must be uint8 (or float8_e8m0fnu)");
      TORCH_CHECK_VALUE(scale.dim() == 4 && scale.size(0) == k.size(0) && scale.size(1) == k.size(2) &&
                            scale.size(2) == 2 && scale.size(3) == k.size(1),
                        "kv_scale must be [num_pages, Hkv, 2, page_size]");
      dense = dense && scale.is_contiguous();
      same = same && scale.device() == k.device();
    } else {
      TORCH_CHECK_VALUE(!scale.defined(), "a bfloat16 cache takes no kv_scale");
    }
    TORCH_CHECK_TYPE(table.scalar_type() == at::kInt && lengths.scalar_type() == at::kInt, "block_table and ", what,
                     " must be int32");
    TORCH_CHECK_VALUE(table.dim() == 2 && lengths.dim() == 1 && lengths.size(0) == table.size(0),
                      "block_table must be [B, max_pages] and ", what, " [B]");
    TORCH_CHECK_VALUE(dense, "cache tensors must be contiguous");
    TORCH_CHECK_VALUE(same, "all tensors must share one device");
    check_cuda(k);
    pages = as_int(k.size(0), "the pool");
    page_size = as_int(k.size(1), "the page size");
    Hkv = as_int(k.size(2), "the heads");
    d = as_int(k.size(3), "the head dim");
    B = as_int(table.size(0), "the batch");
    max_pages = as_int(table.size(1), "the block table");
  }
  const int* table_ptr() const { return static_cast<const int*>(ptr(table)); }
  const int* lengths_ptr() const { return static_cast<const int*>(ptr(lengths)); }
};

void cache_append(const Tensor& k, const Tensor& v, Cache c, const Tensor& count) {
  c.check();
  TORCH_CHECK_VALUE(k.dim() == 4 && v.sizes() == k.sizes() && k.size(0) == c.B && k.size(2) == c.Hkv && k.size(3) == c.d,
                    "k and v must be [B, N, Hkv, d] for the cache's Hkv and d and block_table's B");
  TORCH_CHECK_TYPE(k.scalar_type() == at::kBFloat16 && v.scalar_type() == at::kBFloat16, "k and v must be bfloat16");
  TORCH_CHECK_VALUE(k.device() == c.k.device() && v.device() == c.k.device(), "all tensors must share one device");
  if (count.defined()) {
    TORCH_CHECK_TYPE(count.scalar_type() == at::kInt, "count must be int32");
    TORCH_CHECK_VALUE(count.sizes() == c.lengths.sizes() && count.is_contiguous() && count.device() == c.k.device(),
                      "count must be a contiguous [B] tensor on the cache's device");
  }
  const Strides ks(k, "k"), vs(v, "v");
  const int N = as_int(k.size(1), "the positions");
  will_write(c.k, "k_cache");
  will_write(c.v, "v_cache");
  will_write(c.scale, "kv_scale");
  Here here(c.k);
  check_status(call_unlocked([&] {
                 return api.append(ptr(k), ptr(v), mut(c.k), mut(c.v), mut(c.scale), c.table_ptr(), c.lengths_ptr(),
                                   static_cast<const int*>(ptr(count)), c.B, N, c.Hkv, c.d, ks.get(), vs.get(),
                                   c.page_size, c.pages, c.max_pages, c.fp8, here.handle);
               }),
               "fa_cache_append");
}

std::pair<Tensor, Tensor> cache_read(Cache c, int64_t length, const Tensor& k_out, const Tensor& v_out) {
  c.check();
  TORCH_CHECK_VALUE(length >= 0, "length must be >= 0");
  const int N = as_int(length, "length");
  Here here(c.k);
  const std::array<int64_t, 4> shape{c.B, N, c.Hkv, c.d};
  Tensor k = out_or_new(k_out, shape, at::kBFloat16, c.k, "k_out"), v = out_or_new(v_out, shape, at::kBFloat16, c.k, "v_out");
  check_status(call_unlocked([&] {
                 return api.read(ptr(c.k), ptr(c.v), ptr(c.scale), c.table_ptr(), c.lengths_ptr(), mut(k), mut(v), c.B, N,
                                 c.Hkv, c.d, c.page_size, c.pages, c.max_pages, c.fp8, here.handle);
               }),
               "fa_cache_read");
  return {k, v};
}

std::pair<Tensor, Tensor> decode(const Tensor& q, Cache c, double scale, int window, const Tensor& out, const Tensor& lse,
                                 const Tensor& workspace) {
  TORCH_CHECK_TYPE(c.k.scalar_type() == at::kFloat8_e4m3fn || c.k.scalar_type() == at::kByte,
                   "decode_paged_fp8 takes an 8-bit cache (decode_paged: bfloat16)");
  c.check();
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(0) == c.B && q.size(2) == c.d,
                    "q must be [B, H, d] for block_table's B and the cache's d");
  TORCH_CHECK_TYPE(q.scalar_type() == at::kBFloat16, "q must be bfloat16");
  TORCH_CHECK_VALUE(q.device() == c.k.device() && q.is_contiguous(), "q must be contiguous, on the cache's device");
  TORCH_CHECK_VALUE(!workspace.defined() || (workspace.device() == q.device() && workspace.is_contiguous()),
                    "workspace must be contiguous, on the device of q");
  const int H = as_int(q.size(1), "the heads");
  Here here(q);
  Tensor o = out_or_new(out, q.sizes(), at::kBFloat16, q, "out"), ws = workspace;
  Tensor l = out_or_new(lse, {c.B, H}, at::kFloat, q, "lse");
  will_write(ws, "workspace");
  if (!ws.defined()) {
    const size_t need = api.decode_ws(c.B, H, c.Hkv, c.d, c.page_size, c.max_pages, window);
    if (need) ws = fresh({static_cast<int64_t>(need)}, at::kByte, q);
  }
  const size_t bytes = ws.defined() ? ws.nbytes() : 0;
  check_status(call_unlocked([&] {
                 return api.decode(ptr(q), ptr(c.k), ptr(c.v), ptr(c.scale), c.table_ptr(), c.lengths_ptr(), mut(o),
                                   static_cast<float*>(mut(l)), c.B, H, c.Hkv, c.d, c.page_size, c.pages, c.max_pages,
                                   static_cast<float>(scale), window, mut(ws), bytes, here.handle);
               }),
               "fa_decode_paged_fp8");
  return {o, l};
}

// ---------------------------------------------------------------------------
// The Python side: positional arguments, None for what is not given
// ---------------------------------------------------------------------------
Tensor tensor(PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), "expected a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o) { return o == Py_None ? Tensor() : tensor(o); }
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}

PyObject* pack(const Tensor* t, Py_ssize_t n) {
  PyObject* r = PyTuple_New(n);
  if (!r) throw python_error();
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* o = t[i].defined() ? THPVariable_Wrap(t[i]) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw python_error();
    }
    PyTuple_SET_ITEM(r, i, o);
  }
  return r;
}
PyObject* pack(const std::pair<Tensor, Tensor>& p) {
  const Tensor t[2] = {p.first, p.second};
  return pack(t, 2);
}

// Runs f(args); a library status becomes the package's FAError, the others Python's own
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(given == wanted, "expected ", wanted, " arguments, got ", given);
  TORCH_CHECK(error_class != nullptr, "the binding is not initialised");
  try {
    return f();
  } catch (const Status& e) {
    PyObject* x = PyObject_CallFunction(error_class, "is", e.rc, e.name);
    if (x) {
      PyErr_SetObject(error_class, x);
      Py_DECREF(x);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

Rope rope_of(PyObject* const* a) {  // q, k, cos, sin, q_weight, k_weight, positions, eps, interleaved
  return Rope{tensor(a[0]), tensor(a[1]), tensor(a[2]), tensor(a[3]), maybe(a[4]),
              maybe(a[5]),  maybe(a[6]),  number(a[7]), truth(a[8])};
}

PyObject* py_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {  // rope_of, with autograd
  return guarded(n, 9, [&] {
    Rope r = rope_of(a);
    // tangents need no requires_grad; they live on a level that is asked for first (six lookups take 0.2 us)
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && torch::autograd::ForwardADLevel::try_get_by_idx(0)) {
      for (const Tensor* t : {&r.q, &r.k, &r.wq, &r.wk, &r.cos, &r.sin})
        TORCH_CHECK_NOT_IMPLEMENTED(!t->defined() || !t->_fw_grad(/*level=*/0).defined(),
                                    "qk_norm_rope has no forward-mode derivative");
    }
    auto wants = [](const Tensor& t) { return t.defined() && t.requires_grad(); };
    if (at::GradMode::is_enabled() && (wants(r.q) || wants(r.k) || wants(r.wq) || wants(r.wk))) {
      const auto out = RopeFunction::apply(r.q, r.k, RopeFunction::given(r.wq), RopeFunction::given(r.wk), r.cos, r.sin,
                                           RopeFunction::given(r.positions), r.eps, r.interleaved);
      return pack(out.data(), 2);
    }
    r.check();
    return pack(r.forward({}, {}));
  });
}

PyObject* py_norm_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {  // rope_of, q_out, k_out
  return guarded(n, 11, [&] {
    Rope r = rope_of(a);
    r.check();
    return pack(r.forward(maybe(a[9]), maybe(a[10])));
  });
}

PyObject* py_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {  // rope_of, dq_out, dk_out, workspace
  return guarded(n, 12, [&] {
    Rope r = rope_of(a);
    r.check();
    const Tensor gq = tensor(a[9]), gk = tensor(a[10]), ws = maybe(a[11]);
    auto like = [](const Tensor& g, const Tensor& x, const char* name) {
      TORCH_CHECK_VALUE(g.sizes() == x.sizes() && g.scalar_type() == x.scalar_type() && g.device() == x.device(), name,
                        " must have the shape, dtype and device of its output");
    };
    like(gq, r.q, "dq_out");
    like(gk, r.k, "dk_out");
    TORCH_CHECK_VALUE(!ws.defined() || (ws.device() == r.q.device() && ws.is_contiguous()),
                      "workspace must be contiguous, on the device of q");
    const auto g = r.backward(gq, gk, ws);
    return pack(g.data(), 4);
  });
}

Cache cache_of(PyObject* const* a, const char* what) {  // k_cache, v_cache, kv_scale, block_table, lengths
  return Cache{tensor(a[0]), tensor(a[1]), maybe(a[2]), tensor(a[3]), tensor(a[4]), what};
}

PyObject* py_cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {  // k, v, cache_of, count
  return guarded(n, 8, [&]() -> PyObject* {
    cache_append(tensor(a[0]), tensor(a[1]), cache_of(a + 2, "start"), maybe(a[7]));
    Py_RETURN_NONE;
  });
}

PyObject* py_cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {  // cache_of, length, k_out, v_out
  return guarded(n, 8, [&] { return pack(cache_read(cache_of(a, "seqlens"), integer(a[5]), maybe(a[6]), maybe(a[7]))); });
}

PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {  // q, cache_of, scale, window, out, lse, workspace
  return guarded(n, 11, [&] {
    const Tensor q = tensor(a[0]);
    Cache c = cache_of(a + 1, "seqlens");
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(q.dim() > 0 ? q.size(-1) : 1)) : number(a[6]);
    return pack(decode(q, c, scale, as_int(integer(a[7]), "window_left"), maybe(a[8]), maybe(a[9]), maybe(a[10])));
  });
}

// init(FAError, addresses of the seven entry points in the order of Api)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_TYPE(n == 8, "expected 8 arguments, got ", n);
  void* p[7];
  for (int i = 0; i < 7; ++i) p[i] = reinterpret_cast<void*>(static_cast<uintptr_t>(integer(a[1 + i])));
  api.norm_rope = reinterpret_cast<decltype(api.norm_rope)>(p[0]);
  api.norm_rope_bwd = reinterpret_cast<decltype(api.norm_rope_bwd)>(p[1]);
  api.norm_rope_ws = reinterpret_cast<decltype(api.norm_rope_ws)>(p[2]);
  api.append = reinterpret_cast<decltype(api.append)>(p[3]);
  api.read = reinterpret_cast<decltype(api.read)>(p[4]);
  api.decode = reinterpret_cast<decltype(api.decode)>(p[5]);
  api.decode_ws = reinterpret_cast<decltype(api.decode_ws)>(p[6]);
  Py_INCREF(a[0]);
  error_class = a[0];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

using FastCall = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, FastCall f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("init", py_init),
                         method("norm_rope", py_norm_rope),
                         method("norm_rope_fwd", py_norm_rope_fwd),
                         method("norm_rope_bwd", py_norm_rope_bwd),
                         method("cache_append", py_cache_append),
                         method("cache_read", py_cache_read),
                         method("decode_paged_fp8", py_decode),
                         {nullptr, nullptr, 0, nullptr}};
// build.py looks for the tag in the file, so that another PyTorch's binding is neither kept nor loaded
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding",
                      "Calls of the operators around the attention (see binding.cpp).\n" FA_BINDING_TAG, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
