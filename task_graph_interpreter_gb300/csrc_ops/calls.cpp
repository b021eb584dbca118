// The tensor-level calls of the paged-cache operators and of draft
// verification, as a CPython module: checks of the tensors, fresh outputs and
// scratch, the current stream, and the C ABI call, without a Python-level
// access per property.  A decode step makes two such calls per layer, and in
// Python the checks took longer than the small kernels: norms of one token
// 10.4 us per call with Python checks and ctypes.
//
// Functions of libmk are handed over by address (bind), so that this module
// and the ctypes binding use the one library that the binding loaded.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <mutex>
#include <stdexcept>
#include <string>
#include <tuple>

#include "mk.h"

namespace {

decltype(&mk_paged_plan) paged_plan = nullptr;
decltype(&mk_qk_norm_rope) qk_norm_rope = nullptr;
decltype(&mk_paged_attention) paged_attention = nullptr;
decltype(&mk_paged_attention_workspace) paged_attention_workspace = nullptr;
decltype(&mk_verify_drafts) verify_drafts = nullptr;
decltype(&mk_last_error) last_error = nullptr;
PyObject* mk_error = nullptr;  // the binding's exception class

struct PythonError {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& msg) { throw std::invalid_argument(msg); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}
int small_integer(PyObject* o, const char* name) {
  const long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return (int)v;
}
int small_size(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return (int)v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

// The CUDA device of an operator's first tensor.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return (int)t.get_device();
}
// The operators have no derivatives: a gradient or a forward-mode tangent that would silently be missing is refused.
// (torch.no_grad() does not end forward mode; its levels are one at most.)
void no_gradient(const at::Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, and this operator has none (call it under torch.no_grad())");
  if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
    refuse(std::string(name) + " carries a forward-mode tangent, and this operator has none (unpack the dual tensor)");
}
bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

int32_t* int32s(const at::Tensor& t, const char* name, int64_t n, int dev) {
  if (t.scalar_type() != at::kInt || !on(t, dev) || !t.is_contiguous() || t.numel() < n)
    refuse(std::string(name) + " must be a contiguous int32 tensor of at least " + std::to_string(n) +
           " elements on cuda:" + std::to_string(dev));
  return static_cast<int32_t*>(t.data_ptr());
}
int32_t* int32s_or_null(PyObject* o, const char* name, int64_t n, int dev) {
  const at::Tensor* t = tensor_or_none(o, name);
  return t ? int32s(*t, name, n, dev) : nullptr;
}
// block tables of at least B requests; pages per request
int32_t* block_table(const at::Tensor& t, int64_t B, int dev, int* max_pages) {
  if (t.dim() != 2 || t.size(0) < B)
    refuse("table must be contiguous int32 [" + std::to_string(B) + " or more requests, pages]");
  int32_t* p = int32s(t, "table", 0, dev);
  *max_pages = small_size(t.size(1), "table's width");
  return p;
}
struct Pools {
  void *k, *v;
  int num_pages, Hkv, page, D;
};
Pools pools(const at::Tensor& k, const at::Tensor& v, int dev) {
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 ||
      !k.is_contiguous() || !v.is_contiguous() || !on(k, dev) || !on(v, dev))
    refuse("kpool and vpool must be contiguous bf16 [num_pages, Hkv, page_size, D] on cuda:" + std::to_string(dev));
  no_gradient(k, "kpool");
  no_gradient(v, "vpool");
  return {k.data_ptr(), v.data_ptr(), small_size(k.size(0), "num_pages"), small_size(k.size(1), "Hkv"),
          small_size(k.size(2), "page_size"), small_size(k.size(3), "D")};
}
// elements between the rows of bf16 [N, Hq, D], which may lie apart
int64_t row_stride(const at::Tensor& t, const char* name, int64_t N, int64_t Hq, int64_t D, int dev) {
  if (t.scalar_type() != at::kBFloat16 || !on(t, dev) || t.dim() != 3 || t.size(0) != N || t.size(1) != Hq ||
      t.size(2) != D)
    refuse(std::string(name) + " must be bf16 [" + std::to_string(N) + ", " + std::to_string(Hq) + ", " +
           std::to_string(D) + "] on cuda:" + std::to_string(dev));
  no_gradient(t, name);
  if (t.is_contiguous() || N == 0) return Hq * D;
  if ((D > 1 && t.stride(2) != 1) || (Hq > 1 && t.stride(1) != D))
    refuse(std::string("each row of ") + name + " must be contiguous");
  return N > 1 ? t.stride(0) : Hq * D;
}
void* gain(PyObject* o, const char* name, int64_t D, int dev) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) return nullptr;
  if (t->scalar_type() != at::kBFloat16 || t->numel() != D || !t->is_contiguous() || !on(*t, dev))
    refuse(std::string(name) + " must be bf16 [" + std::to_string(D) + "] on cuda:" + std::to_string(dev));
  no_gradient(*t, name);
  return t->data_ptr();
}
// elements between the rows of f32 [B, rows, V]
int64_t probability_stride(const at::Tensor& t, const char* name, int64_t B, int64_t rows, int64_t V, int dev) {
  if (t.scalar_type() != at::kFloat || !on(t, dev) || t.dim() != 3 || t.size(0) != B || t.size(1) != rows ||
      t.size(2) != V)
    refuse(std::string(name) + " must be f32 [" + std::to_string(B) + ", " + std::to_string(rows) + ", " +
           std::to_string(V) + "] on cuda:" + std::to_string(dev));
  no_gradient(t, name);
  if (t.is_contiguous()) return V;
  if ((V > 1 && t.stride(2) != 1) || (B > 1 && rows > 1 && t.stride(0) != rows * t.stride(1)))
    refuse(std::string(name) + " must have evenly spaced contiguous rows");
  return rows > 1 ? t.stride(1) : B > 1 ? t.stride(0) : V;
}
at::Tensor fresh(at::IntArrayRef size, at::ScalarType type, int dev) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev)));
}

void check(int rc, const char* fn) {
  if (rc == MK_OK) return;
  PyObject* e = PyObject_CallFunction(mk_error, "sis", fn, rc, last_error());
  if (e) {
    PyErr_SetObject(mk_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

// Run `body`; C++ exceptions become Python ones.
template <typename F>
PyObject* guarded(const char* fn, Py_ssize_t want, Py_ssize_t n, F body) {
  if (n != want || !paged_plan) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, and bind() first", fn, want);
    return nullptr;
  }
  try {
    return body();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// The call itself, without the interpreter's lock (a full launch queue makes it wait).
template <typename F>
int unlocked(F call) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call();
  Py_END_ALLOW_THREADS
  return rc;
}

// plan(ctx_len, new_len, table, held, held_out, free_pages, free_count, count_out, page_size, cu, positions, slots,
//      max_tokens, status) -> (cu, positions, slots)
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("plan", 14, n, [&]() -> PyObject* {
    const at::Tensor& ctx = tensor(a[0], "ctx_len");
    const int dev = device_of(ctx, "ctx_len");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const int B = small_size(ctx.numel(), "the number of requests");
    int max_pages = 0;
    int32_t* table = block_table(tensor(a[2], "table"), B, dev, &max_pages);
    int32_t* held = int32s(tensor(a[3], "held"), "held", B, dev);
    int32_t* held_out = int32s_or_null(a[4], "held_out", B, dev);
    const at::Tensor& free_pages = tensor(a[5], "free_pages");
    int32_t* count = int32s(tensor(a[6], "free_count"), "free_count", 1, dev);
    int32_t* count_out = int32s_or_null(a[7], "count_out", 1, dev);
    const int page = small_integer(a[8], "page_size");
    const at::Tensor *pos = tensor_or_none(a[10], "positions"), *slots = tensor_or_none(a[11], "slots");
    if ((!pos || !slots) && a[12] == Py_None) refuse("give positions and slots, or max_tokens");
    const int64_t tokens = pos ? pos->numel() : slots ? slots->numel() : small_integer(a[12], "max_tokens");
    if (tokens < 0) refuse("max_tokens must be positive");
    const at::Tensor cu_t = a[9] != Py_None ? tensor(a[9], "cu") : fresh({B + 1}, at::kInt, dev);
    const at::Tensor pos_t = pos ? *pos : fresh({tokens}, at::kInt, dev);
    const at::Tensor slots_t = slots ? *slots : fresh({tokens}, at::kInt, dev);
    int32_t* cu = int32s(cu_t, "cu", B + 1, dev);
    int32_t* p = int32s(pos_t, "positions", tokens, dev);
    int32_t* s = int32s(slots_t, "slots", tokens, dev);
    int32_t* status = int32s_or_null(a[13], "status", 1, dev);
    const int32_t *c = int32s(ctx, "ctx_len", B, dev), *len = int32s(tensor(a[1], "new_len"), "new_len", B, dev);
    int32_t* f = int32s(free_pages, "free_pages", 1, dev);
    const int pages = small_size(free_pages.numel(), "free_pages");
    const int most = small_size(tokens, "max_tokens");
    void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    check(unlocked([&] {
            return paged_plan(stream, B, page, max_pages, pages, most, c, len, table, held, held_out ? held_out : held,
                              f, count, count_out ? count_out : count, cu, p, s, status);
          }),
          "mk_paged_plan");
    return Py_BuildValue("(NNN)", THPVariable_Wrap(cu_t), THPVariable_Wrap(pos_t), THPVariable_Wrap(slots_t));
  });
}

// qk_norm_rope(qkv, Hq, Hkv, D, positions, slots, kpool, vpool, q_gamma, k_gamma, eps, rope_theta, out, status) -> out
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope", 14, n, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "qkv");
    const int dev = device_of(x, "qkv");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const int Hq = small_integer(a[1], "Hq"), Hkv = small_integer(a[2], "Hkv"), D = small_integer(a[3], "D");
    const int64_t width = ((int64_t)Hq + 2 * (int64_t)Hkv) * D;
    const bool f32 = x.scalar_type() == at::kFloat;
    if ((!f32 && x.scalar_type() != at::kBFloat16) || x.dim() != 2 || x.size(1) != width ||
        (width > 1 && x.stride(1) != 1))
      refuse("qkv must be f32 or bf16 [N, " + std::to_string(width) + "] with contiguous rows");
    no_gradient(x, "qkv");
    const int N = small_size(x.size(0), "N");
    const Pools pl = pools(tensor(a[6], "kpool"), tensor(a[7], "vpool"), dev);
    if (pl.Hkv != Hkv || pl.D != D)
      refuse("the pools have " + std::to_string(pl.Hkv) + " heads of " + std::to_string(pl.D) + ", the call " +
             std::to_string(Hkv) + " of " + std::to_string(D));
    void *gq = gain(a[8], "q_gamma", D, dev), *gk = gain(a[9], "k_gamma", D, dev);
    const float eps = (float)number(a[10]);
    const double theta = number(a[11]);
    const at::Tensor* given = tensor_or_none(a[12], "out");
    const at::Tensor out = given ? *given : fresh({N, Hq, D}, at::kBFloat16, dev);
    const int64_t ld = row_stride(out, "out", N, Hq, D, dev);
    const int32_t* pos = int32s(tensor(a[4], "positions"), "positions", N, dev);
    const int32_t* slots = int32s(tensor(a[5], "slots"), "slots", N, dev);
    int32_t* status = int32s_or_null(a[13], "status", 1, dev);
    if (N > 0) {
      void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      const int64_t ld_x = N > 1 ? x.stride(0) : width;
      check(unlocked([&] {
              return qk_norm_rope(stream, N, Hq, Hkv, D, x.data_ptr(), f32 ? MK_F32 : MK_BF16, ld_x, gq, gk, eps, theta,
                                  pos, slots, out.data_ptr(), ld, pl.k, pl.v, pl.num_pages, pl.page, status);
            }),
            "mk_qk_norm_rope");
    }
    return THPVariable_Wrap(out);
  });
}

// Workspace bytes, asked of the library once per device and shape.  The lock is never held where Python code can
// run (the exception of a refused shape is Python code): another thread may be waiting for it with the interpreter's
// lock.
size_t workspace_size(int dev, int max_new, int Hq, int Hkv, int D) {
  static std::mutex mu;
  static std::map<std::tuple<int, int, int, int, int>, size_t> known;
  const auto key = std::make_tuple(dev, max_new, Hq, Hkv, D);
  {
    const std::lock_guard<std::mutex> lock(mu);
    const auto it = known.find(key);
    if (it != known.end()) return it->second;
  }
  size_t bytes = 0;
  check(paged_attention_workspace(max_new, Hq, Hkv, D, &bytes), "mk_paged_attention_workspace");
  const std::lock_guard<std::mutex> lock(mu);
  known.emplace(key, bytes);
  return bytes;
}

// Scratch of one call from PyTorch's allocator, ordered by the stream as a tensor's memory is.
struct Scratch {
  void* p = nullptr;
  ~Scratch() {
    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
};

// attention(q, kpool, vpool, table, cu, ctx_len, max_new, scale, out, workspace, status) -> out
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("attention", 11, n, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const int dev = device_of(q, "q");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    const Pools pl = pools(tensor(a[1], "kpool"), tensor(a[2], "vpool"), dev);
    if (q.dim() != 3) refuse("q must be bf16 [N, Hq, D]");
    const int N = small_size(q.size(0), "N"), Hq = small_size(q.size(1), "Hq");
    const int64_t ld_q = row_stride(q, "q", N, Hq, pl.D, dev);
    const at::Tensor* given = tensor_or_none(a[8], "out");
    const at::Tensor out = given ? *given : fresh({N, Hq, pl.D}, at::kBFloat16, dev);
    const int64_t ld_out = row_stride(out, "out", N, Hq, pl.D, dev);
    const at::Tensor& ctx = tensor(a[5], "ctx_len");
    const int B = small_size(ctx.numel(), "the number of requests");
    int max_pages = 0;
    int32_t* table = block_table(tensor(a[3], "table"), B, dev, &max_pages);
    const int32_t *cu = int32s(tensor(a[4], "cu"), "cu", B + 1, dev), *c = int32s(ctx, "ctx_len", B, dev);
    const int max_new = small_integer(a[6], "max_new");
    const float scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)pl.D)) : (float)number(a[7]);
    int32_t* status = int32s_or_null(a[10], "status", 1, dev);
    if (N > 0 && B > 0) {
      const at::Tensor* ws = tensor_or_none(a[9], "workspace");
      Scratch scratch;
      void* work;
      size_t size;
      if (ws) {
        if (!ws->is_contiguous() || !on(*ws, dev)) refuse("workspace must be contiguous on cuda:" + std::to_string(dev));
        work = ws->data_ptr();
        size = ws->nbytes();
      } else {
        size = workspace_size(dev, max_new, Hq, pl.Hkv, pl.D);
        work = scratch.p = c10::cuda::CUDACachingAllocator::raw_alloc(size);
      }
      void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      check(unlocked([&] {
              return paged_attention(stream, B, N, max_new, Hq, pl.Hkv, pl.D, q.data_ptr(), ld_q, pl.k, pl.v,
                                     pl.num_pages, pl.page, table, max_pages, cu, c, scale, out.data_ptr(), ld_out, work,
                                     size, status);
            }),
            "mk_paged_attention");
    }
    return THPVariable_Wrap(out);
  });
}

// verify(p, drafts, u, q, draft_len, tokens, accepted, status) -> (tokens, accepted)
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("verify", 8, n, [&]() -> PyObject* {
    const at::Tensor& p = tensor(a[0], "p");
    const int dev = device_of(p, "p");
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    if (p.dim() != 3 || p.size(1) < 1) refuse("p must be f32 [B, K + 1, V]");
    const int B = small_size(p.size(0), "B"), K = small_size(p.size(1) - 1, "K"), V = small_size(p.size(2), "V");
    const int64_t ld_p = probability_stride(p, "p", B, K + 1, V, dev);
    const at::Tensor* q = K > 0 ? tensor_or_none(a[3], "q") : nullptr;
    const int64_t ld_q = q ? probability_stride(*q, "q", B, K, V, dev) : V;
    const at::Tensor &drafts = tensor(a[1], "drafts"), &u = tensor(a[2], "u");
    if (u.scalar_type() != at::kFloat || !on(u, dev) || u.numel() != (int64_t)B * (K + 1) || !u.is_contiguous())
      refuse("u must be contiguous f32 [" + std::to_string(B) + ", " + std::to_string(K + 1) + "] on cuda:" +
             std::to_string(dev));
    no_gradient(u, "u");
    if (drafts.numel() != (int64_t)B * K)
      refuse("drafts must be int32 [" + std::to_string(B) + ", " + std::to_string(K) + "]");
    const int32_t* d = int32s(drafts, "drafts", (int64_t)B * K, dev);
    const int32_t* len = int32s_or_null(a[4], "draft_len", B, dev);
    const at::Tensor tokens = a[5] != Py_None ? tensor(a[5], "tokens") : fresh({B, K + 1}, at::kInt, dev);
    const at::Tensor accepted = a[6] != Py_None ? tensor(a[6], "accepted") : fresh({B}, at::kInt, dev);
    int32_t* tk = int32s(tokens, "tokens", (int64_t)B * (K + 1), dev);
    int32_t* ac = int32s(accepted, "accepted", B, dev);
    int32_t* status = int32s_or_null(a[7], "status", 1, dev);
    if (B > 0) {
      void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      const float *pp = static_cast<const float*>(p.data_ptr()), *uu = static_cast<const float*>(u.data_ptr());
      const float* qq = q ? static_cast<const float*>(q->data_ptr()) : nullptr;
      check(unlocked([&] { return verify_drafts(stream, B, K, V, pp, ld_p, qq, ld_q, d, len, uu, tk, ac, status); }),
            "mk_verify_drafts");
    }
    return Py_BuildValue("(NN)", THPVariable_Wrap(tokens), THPVariable_Wrap(accepted));
  });
}

// bind(MkError, addresses of mk_paged_plan, mk_qk_norm_rope, mk_paged_attention, mk_paged_attention_workspace,
//      mk_verify_drafts, mk_last_error)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes 7 arguments");
    return nullptr;
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  Py_XDECREF(mk_error);
  mk_error = a[0];
  qk_norm_rope = reinterpret_cast<decltype(qk_norm_rope)>(f[1]);
  paged_attention = reinterpret_cast<decltype(paged_attention)>(f[2]);
  paged_attention_workspace = reinterpret_cast<decltype(paged_attention_workspace)>(f[3]);
  verify_drafts = reinterpret_cast<decltype(verify_drafts)>(f[4]);
  last_error = reinterpret_cast<decltype(last_error)>(f[5]);
  paged_plan = reinterpret_cast<decltype(paged_plan)>(f[0]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {{"bind", fast(py_bind), METH_FASTCALL, nullptr},
                         {"plan", fast(py_plan), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", fast(py_norm), METH_FASTCALL, nullptr},
                         {"attention", fast(py_attention), METH_FASTCALL, nullptr},
                         {"verify", fast(py_verify), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
