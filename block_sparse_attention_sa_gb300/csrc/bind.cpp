// bind.cpp -- the paged-cache calls from Python. One of these calls serves one
// token, so its own cost counts: checking and marshalling a dozen tensors takes
// 10 us in Python, 1 us here, next to 4 us to enqueue the kernels. The module
// only reads tensors (device, type, shape, strides, address), fills
// sa_cache_params and calls the C ABI through the addresses it is given; what
// the ABI itself can check it leaves to it.
#include <Python.h>

#include <cstdint>
#include <stdexcept>
#include <string>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sa.h"

namespace {

decltype(&sa_cache_append) g_append = nullptr;
decltype(&sa_route_pages) g_route = nullptr;
decltype(&sa_attn_decode) g_decode = nullptr;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

// The calls' arguments in order; `device` is that of every tensor.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;
  int64_t device = -1;

  PyObject* next() {
    if (left-- <= 0) refuse("too few arguments");
    return *at++;
  }
  int64_t integer(const char* name) {
    const int64_t v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) refuse(std::string(name) + " must be an integer");
    return v;
  }
  int32_t int32(const char* name) {
    const int64_t v = integer(name);
    if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
    return static_cast<int32_t>(v);
  }
  float real(const char* name) {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) refuse(std::string(name) + " must be a number");
    return static_cast<float>(v);
  }
  // None for null
  const at::Tensor* tensor(const char* name) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.get_device() != device || !t.is_cuda())
      refuse(std::string(name) + " must be on cuda:" + std::to_string(device) +
             " (the first tensor's device)");
    return &t;
  }
  const at::Tensor& given(const char* name) {
    const at::Tensor* t = tensor(name);
    if (!t) refuse(std::string(name) + " must be a tensor");
    return *t;
  }
  // A contiguous tensor of n elements (any number: n < 0), or null for None.
  void* vector(const char* name, at::ScalarType type, int64_t n) {
    const at::Tensor* t = tensor(name);
    if (!t) return nullptr;
    if (t->scalar_type() != type || !t->is_contiguous() || (n >= 0 && t->numel() != n))
      refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor" +
             (n >= 0 ? " with " + std::to_string(n) + " elements" : std::string()));
    return t->data_ptr();
  }
};

constexpr at::ScalarType kF32 = at::kFloat, kI32 = at::kInt;

// bf16 [B, S, heads, D] with d contiguous: its address; its strides into `to`.
void* tokens(const at::Tensor& t, const char* name, int64_t B, int64_t S, int64_t heads, int64_t D,
             int64_t to[3]) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || t.size(0) != B || t.size(1) != S ||
      t.size(2) != heads || t.size(3) != D || t.stride(3) != 1)
    refuse(std::string(name) + " must be bf16 [" + std::to_string(B) + ", " + std::to_string(S) + ", " +
           std::to_string(heads) + ", " + std::to_string(D) + "] with a contiguous last dimension");
  for (int i = 0; i < 3; ++i) to[i] = t.stride(i);
  return t.data_ptr();
}

int32_t narrow(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

const int32_t* table(Args& a, sa_cache_params* p) {
  const at::Tensor& t = a.given("page_table");
  if (t.scalar_type() != kI32 || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    refuse("page_table must be int32 [B, max_pages], its rows contiguous");
  p->B = narrow(t.size(0), "B");
  p->max_pages = narrow(t.size(1), "max_pages");
  p->table_stride = t.stride(0);
  return static_cast<const int32_t*>(t.data_ptr());
}

void pool(Args& a, sa_cache_params* p, void** kc, void** vc) {
  const at::Tensor& k = a.given("k_cache");
  const at::Tensor& v = a.given("v_cache");
  const at::ScalarType type = k.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat8_e4m3fn && type != at::kByte)
    refuse("k_cache, v_cache must be bfloat16, float8_e4m3fn or uint8 (e4m3)");
  if (k.dim() != 4 || k.size(2) != 64 || v.sizes() != k.sizes() || v.scalar_type() != type ||
      k.stride(3) != 1 || v.stride(3) != 1)
    refuse("k_cache, v_cache must be alike, [n_pages, H_kv, 64, D] with a contiguous last dimension");
  p->cache_format = type == at::kBFloat16 ? SA_CACHE_BF16 : SA_CACHE_FP8;
  p->n_pages = narrow(k.size(0), "n_pages");
  p->H_kv = narrow(k.size(1), "H_kv");
  p->D = narrow(k.size(3), "D");
  for (int i = 0; i < 3; ++i) {
    p->kc_stride[i] = k.stride(i);
    p->vc_stride[i] = v.stride(i);
  }
  *kc = k.data_ptr();
  *vc = v.data_ptr();
}

// An entry: arguments in, the call's status out; nothing thrown leaves it.
template <class F>
PyObject* entry(PyObject* const* args, Py_ssize_t n, F body) {
  try {
    Args a{args, n};
    a.device = a.integer("device");
    const sa_status s = body(a);
    if (a.left != 0) refuse("too many arguments");
    return PyLong_FromLong(s);
  } catch (const std::exception& e) {
    PyErr_Clear();
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    const at::Tensor& k = a.given("k");
    const at::Tensor& v = a.given("v");
    void *kc, *vc;
    pool(a, &p, &kc, &vc);
    const int32_t* pages = table(a, &p);
    const int64_t B = p.B, Hkv = p.H_kv, D = p.D, S = k.dim() == 4 ? k.size(1) : -1;
    p.S = narrow(S, "S");
    void* kp = tokens(k, "k", B, S, Hkv, D, p.k_stride);
    void* vp = tokens(v, "v", B, S, Hkv, D, p.v_stride);
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, B));
    const at::Tensor* q = a.tensor("q");
    const at::Tensor* q_out = a.tensor("q_out");
    if ((q == nullptr) != (q_out == nullptr)) refuse("q and q_out go together");
    void *qp = nullptr, *qo = nullptr;
    p.H = p.H_kv;
    if (q) {
      const int64_t H = q->dim() == 4 ? q->size(2) : -1;
      p.H = narrow(H, "H");
      qp = tokens(*q, "q", B, S, H, D, p.q_stride);
      qo = tokens(*q_out, "q_out", B, S, H, D, p.o_stride);
    }
    const auto* fresh = static_cast<const int32_t*>(a.vector("new_lens", kI32, B));
    p.qk_norm = a.int32("qk_norm");
    const auto* gq = static_cast<const float*>(a.vector("gamma_q", kF32, D));
    const auto* gk = static_cast<const float*>(a.vector("gamma_k", kF32, D));
    p.eps = a.real("eps");
    const at::Tensor* cos = a.tensor("cos");
    const at::Tensor* sin = a.tensor("sin");
    const float* angles[2] = {};
    if (cos || sin) {
      if (!cos || !sin || cos->dim() != 2 || cos->size(0) < 1 || cos->size(1) != D / 2 || sin->sizes() != cos->sizes() ||
          cos->scalar_type() != kF32 || sin->scalar_type() != kF32 || !cos->is_contiguous() ||
          !sin->is_contiguous())
        refuse("cos and sin go together, both contiguous fp32 [rows, D/2] with rows >= 1");
      p.rope_rows = narrow(cos->size(0), "rope_rows");
      angles[0] = static_cast<const float*>(cos->data_ptr());
      angles[1] = static_cast<const float*>(sin->data_ptr());
    }
    p.rope_layout = a.int32("rope");
    const auto* ks = static_cast<const float*>(a.vector("k_scale", kF32, Hkv));
    const auto* vs = static_cast<const float*>(a.vector("v_scale", kF32, Hkv));
    auto* k_sum = static_cast<float*>(a.vector("k_sum", kF32, p.n_pages * Hkv * D));
    auto* lens_out = static_cast<int32_t*>(a.vector("lens_out", kI32, B));
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_append(&p, kp, vp, qp, qo, gq, gk, angles[0], angles[1], kc, vc, ks, vs, k_sum, pages,
                    lens, fresh, lens_out, status, stream);
  });
}

PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    const at::Tensor& q = a.given("q");
    const at::Tensor& k_sum = a.given("k_sum");
    if (q.dim() != 4 || k_sum.dim() != 3 || k_sum.scalar_type() != kF32 || !k_sum.is_contiguous())
      refuse("q must be [B, 1, H, D], k_sum contiguous fp32 [n_pages, H_kv, D]");
    p.n_pages = narrow(k_sum.size(0), "n_pages");
    p.H_kv = narrow(k_sum.size(1), "H_kv");
    p.D = narrow(k_sum.size(2), "D");
    const int32_t* pages = table(a, &p);
    p.S = narrow(q.size(1), "S");
    p.H = narrow(q.size(2), "H");
    void* qp = tokens(q, "q", p.B, p.S, p.H, p.D, p.q_stride);
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, p.B));
    p.prefix_len = a.int32("prefix_len");
    p.page_budget = a.int32("budget");
    auto* row_ptr = static_cast<int32_t*>(
        a.vector("row_ptr", kI32, static_cast<int64_t>(p.B) * p.H_kv + 1));
    const at::Tensor& cols = a.given("col_idx");
    if (cols.scalar_type() != kI32 || !cols.is_contiguous()) refuse("col_idx must be contiguous int32");
    const at::Tensor& ws = a.given("workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_route(&p, qp, static_cast<const float*>(k_sum.data_ptr()), pages, lens, row_ptr,
                   static_cast<int32_t*>(cols.data_ptr()), cols.numel(), ws.data_ptr(), ws.nbytes(),
                   status, stream);
  });
}

PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    const at::Tensor& q = a.given("q");
    void *kc, *vc;
    pool(a, &p, &kc, &vc);
    const int32_t* pages = table(a, &p);
    if (q.dim() != 4) refuse("q must be [B, 1, H, D]");
    p.S = narrow(q.size(1), "S");
    p.H = narrow(q.size(2), "H");
    void* qp = tokens(q, "q", p.B, p.S, p.H, p.D, p.q_stride);
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, p.B));
    p.softmax_scale = a.real("scale");
    const auto* row_ptr = static_cast<const int32_t*>(
        a.vector("row_ptr", kI32, static_cast<int64_t>(p.B) * p.H_kv + 1));
    const at::Tensor* cols = a.tensor("col_idx");
    if ((row_ptr == nullptr) != (cols == nullptr)) refuse("row_ptr and col_idx go together");
    if (cols && (cols->scalar_type() != kI32 || !cols->is_contiguous()))
      refuse("col_idx must be contiguous int32");
    const auto* ks = static_cast<const float*>(a.vector("k_scale", kF32, p.H_kv));
    const auto* vs = static_cast<const float*>(a.vector("v_scale", kF32, p.H_kv));
    void* op = tokens(a.given("o"), "o", p.B, p.S, p.H, p.D, p.o_stride);
    auto* lse = static_cast<float*>(a.vector("lse", kF32, static_cast<int64_t>(p.B) * p.H));
    const at::Tensor& ws = a.given("workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_decode(&p, qp, kc, vc, ks, vs, pages, lens, row_ptr,
                    cols ? static_cast<const int32_t*>(cols->data_ptr()) : nullptr,
                    cols ? cols->numel() : 0, op, lse, ws.data_ptr(), ws.nbytes(), status, stream);
  });
}

// The addresses of sa_cache_append, sa_route_pages and sa_attn_decode.
PyObject* attach(PyObject*, PyObject* args) {
  unsigned long long f[3];
  if (!PyArg_ParseTuple(args, "KKK", &f[0], &f[1], &f[2])) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_route = reinterpret_cast<decltype(g_route)>(f[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[2]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"attach", attach, METH_VARARGS, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(route)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sa_bind", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sa_bind() { return PyModule_Create(&module); }
