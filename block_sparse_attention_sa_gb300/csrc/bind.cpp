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
decltype(&sa_cache_append_axes) g_append_axes = nullptr;
decltype(&sa_attn_tree) g_tree = nullptr;
decltype(&sa_cache_accept) g_accept = nullptr;
decltype(&sa_cache_copy) g_copy = nullptr;
decltype(&sa_pages_fork) g_fork = nullptr;
decltype(&sa_pages_resize) g_resize = nullptr;
decltype(&sa_pages_compact) g_compact = nullptr;

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

// int32 [B, n] with its rows contiguous
void check_rows(const at::Tensor& t, const char* name, const char* n) {
  if (t.scalar_type() != kI32 || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1))
    refuse(std::string(name) + " must be int32 [B, " + n + "], its rows contiguous");
}

const int32_t* table(Args& a, sa_cache_params* p) {
  const at::Tensor& t = a.given("page_table");
  check_rows(t, "page_table", "max_pages");
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

// positions (int32 [B, S, n_axes], or None) and the axes of the pairs (D / 2 bytes, or
// None: no axes): whether there are axes.
bool rope_axes(Args& a, int64_t B, int64_t S, int64_t D, sa_rope_axes* x) {
  const at::Tensor* pos = a.tensor("positions");
  PyObject* of = a.next();
  x->n_axes = a.int32("n_axes");
  if (of == Py_None) {
    if (pos) refuse("positions go with axes");
    return false;
  }
  if (!PyBytes_Check(of) || PyBytes_GET_SIZE(of) != D / 2)
    refuse("axes must name an axis for each of the D/2 pairs");
  for (int64_t i = 0; i < D / 2 && i < 64; ++i)
    x->axis_of[i] = static_cast<uint8_t>(PyBytes_AS_STRING(of)[i]);
  if (!pos) return true;
  if (pos->scalar_type() != kI32 || pos->dim() != 3 || pos->size(0) != B || pos->size(1) != S ||
      pos->size(2) != x->n_axes || (pos->stride(2) != 1 && pos->size(2) != 1))
    refuse("positions must be int32 [" + std::to_string(B) + ", " + std::to_string(S) + ", " +
           std::to_string(x->n_axes) + "], the axes contiguous");
  x->positions = static_cast<const int32_t*>(pos->data_ptr());
  x->pos_stride[0] = pos->stride(0);
  x->pos_stride[1] = pos->stride(1);
  return true;
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

template <class T>
T* required(T* p, const char* name) {
  if (!p) refuse(std::string(name) + " must be a tensor");
  return p;
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
    sa_rope_axes axes{};
    const bool by_axes = rope_axes(a, B, S, D, &axes);
    if (by_axes && !angles[0]) refuse("positions and axes go with cos and sin");
    axes.rows = p.rope_rows;
    const auto* ks = static_cast<const float*>(a.vector("k_scale", kF32, Hkv));
    const auto* vs = static_cast<const float*>(a.vector("v_scale", kF32, Hkv));
    auto* k_sum = static_cast<float*>(a.vector("k_sum", kF32, p.n_pages * Hkv * D));
    auto* lens_out = static_cast<int32_t*>(a.vector("lens_out", kI32, B));
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    if (by_axes)
      return g_append_axes(&p, kp, vp, qp, qo, gq, gk, angles[0], angles[1], &axes, kc, vc, ks, vs,
                           k_sum, pages, lens, fresh, lens_out, status, stream);
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

PyObject* tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    const at::Tensor& q = a.given("q");
    void *kc, *vc;
    pool(a, &p, &kc, &vc);
    const int32_t* pages = table(a, &p);
    if (q.dim() != 4) refuse("q must be [B, S, H, D]");
    p.S = narrow(q.size(1), "S");
    p.H = narrow(q.size(2), "H");
    void* qp = tokens(q, "q", p.B, p.S, p.H, p.D, p.q_stride);
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, p.B));
    p.softmax_scale = a.real("scale");
    const at::Tensor* up = a.tensor("parents");
    int64_t up_stride = 0;
    if (up) {
      const int64_t d = up->dim();
      if (up->scalar_type() != kI32 || (d != 1 && d != 2) || up->size(d - 1) != p.S ||
          (d == 2 && up->size(0) != p.B) || (up->stride(d - 1) != 1 && p.S != 1))
        refuse("parents must be int32 [B, S] or [S], the tokens contiguous");
      if (d == 2) up_stride = up->stride(0);
    }
    const auto* fresh = static_cast<const int32_t*>(a.vector("new_lens", kI32, p.B));
    const auto* row_ptr = static_cast<const int32_t*>(
        a.vector("row_ptr", kI32, static_cast<int64_t>(p.B) * p.H_kv + 1));
    const at::Tensor* cols = a.tensor("col_idx");
    if ((row_ptr == nullptr) != (cols == nullptr)) refuse("row_ptr and col_idx go together");
    if (cols && (cols->scalar_type() != kI32 || !cols->is_contiguous()))
      refuse("col_idx must be contiguous int32");
    const auto* ks = static_cast<const float*>(a.vector("k_scale", kF32, p.H_kv));
    const auto* vs = static_cast<const float*>(a.vector("v_scale", kF32, p.H_kv));
    void* op = tokens(a.given("o"), "o", p.B, p.S, p.H, p.D, p.o_stride);
    auto* lse = static_cast<float*>(a.vector("lse", kF32, static_cast<int64_t>(p.B) * p.H * p.S));
    const at::Tensor& ws = a.given("workspace");
    if (!ws.is_contiguous()) refuse("workspace must be contiguous");
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_tree(&p, qp, kc, vc, ks, vs, pages, lens, fresh,
                  up ? static_cast<const int32_t*>(up->data_ptr()) : nullptr, up_stride, row_ptr,
                  cols ? static_cast<const int32_t*>(cols->data_ptr()) : nullptr,
                  cols ? cols->numel() : 0, op, lse, ws.data_ptr(), ws.nbytes(), status, stream);
  });
}

PyObject* accept(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    void *kc, *vc;
    pool(a, &p, &kc, &vc);
    p.H = p.H_kv;
    const int32_t* pages = table(a, &p);
    const auto* lens = required(static_cast<const int32_t*>(a.vector("seq_lens", kI32, p.B)), "seq_lens");
    const at::Tensor& path = a.given("path");
    check_rows(path, "path", "S");
    if (path.size(0) != p.B) refuse("path must have a row for each sequence");
    p.S = narrow(path.size(1), "S");
    const auto* path_lens = required(static_cast<const int32_t*>(a.vector("path_lens", kI32, p.B)), "path_lens");
    auto* k_sum = static_cast<float*>(
        a.vector("k_sum", kF32, static_cast<int64_t>(p.n_pages) * p.H_kv * p.D));
    const auto* ks = static_cast<const float*>(a.vector("k_scale", kF32, p.H_kv));
    auto* lens_out = static_cast<int32_t*>(a.vector("lens_out", kI32, p.B));
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_accept(&p, kc, vc, ks, k_sum, pages, lens, static_cast<const int32_t*>(path.data_ptr()),
                    path.stride(0), path_lens, lens_out, status, stream);
  });
}

// moves: contiguous int32 [n, 2]; n
int32_t* moves_of(Args& a, int64_t* n) {
  const at::Tensor& m = a.given("moves");
  if (m.scalar_type() != kI32 || m.dim() != 2 || m.size(1) != 2 || !m.is_contiguous())
    refuse("moves must be contiguous int32 [n, 2]");
  *n = m.size(0);
  return static_cast<int32_t*>(m.data_ptr());
}

PyObject* copy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    sa_cache_params p{};
    p.page = 64;
    p.B = p.S = p.max_pages = 1;
    void *kc, *vc;
    pool(a, &p, &kc, &vc);
    p.H = p.H_kv;
    int64_t cap;
    const int32_t* moves = moves_of(a, &cap);
    const auto* count = static_cast<const int32_t*>(a.vector("n_moves", kI32, 1));
    auto* k_sum = static_cast<float*>(
        a.vector("k_sum", kF32, static_cast<int64_t>(p.n_pages) * p.H_kv * p.D));
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_copy(&p, kc, vc, k_sum, moves, cap, count, status, stream);
  });
}

// What the calls on pages share: the pool's size and a table.
struct PageTable {
  int32_t* at;
  int32_t rows, max_pages;
  int64_t stride;
};

PageTable page_table(const at::Tensor& t, const char* name) {
  check_rows(t, name, "max_pages");
  return {static_cast<int32_t*>(t.data_ptr()), narrow(t.size(0), name), narrow(t.size(1), name),
          t.stride(0)};
}

int32_t* counts(Args& a, const char* name, int32_t* n_pages) {
  const at::Tensor& t = a.given(name);
  if (t.scalar_type() != kI32 || t.dim() != 1 || !t.is_contiguous())
    refuse(std::string(name) + " must be contiguous int32 [n_pages]");
  if (*n_pages >= 0 && t.numel() != *n_pages) refuse(std::string(name) + " must be as long as refs");
  *n_pages = narrow(t.numel(), name);
  return static_cast<int32_t*>(t.data_ptr());
}

const at::Tensor& scratch(Args& a) {
  const at::Tensor& ws = a.given("workspace");
  if (!ws.is_contiguous()) refuse("workspace must be contiguous");
  return ws;
}

PyObject* fork(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    const PageTable old = page_table(a.given("page_table"), "page_table");
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, old.rows));
    int32_t n_pages = -1;
    const int32_t* refs = counts(a, "refs", &n_pages);
    const at::Tensor& src = a.given("src");
    if (src.scalar_type() != kI32 || src.dim() != 1 || !src.is_contiguous())
      refuse("src must be contiguous int32 [N]");
    const PageTable out = page_table(a.given("table_out"), "table_out");
    if (out.rows != src.numel() || out.max_pages != old.max_pages)
      refuse("table_out must be [N, max_pages]");
    auto* lens_out = static_cast<int32_t*>(a.vector("lens_out", kI32, out.rows));
    int32_t* refs_out = counts(a, "refs_out", &n_pages);
    int64_t cap;
    int32_t* moves = moves_of(a, &cap);
    if (cap < out.rows) refuse("moves must have room for N pairs");
    auto* n_moves = required(static_cast<int32_t*>(a.vector("n_moves", kI32, 1)), "n_moves");
    const at::Tensor& ws = scratch(a);
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_fork(n_pages, old.max_pages, old.rows, out.rows, old.at, old.stride, lens, refs,
                  static_cast<const int32_t*>(src.data_ptr()), out.at, out.stride, lens_out,
                  refs_out, moves, n_moves, ws.data_ptr(), ws.nbytes(), status, stream);
  });
}

PyObject* resize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    const PageTable t = page_table(a.given("page_table"), "page_table");
    int32_t n_pages = -1;
    int32_t* refs = counts(a, "refs", &n_pages);
    const auto* lens = static_cast<const int32_t*>(a.vector("seq_lens", kI32, t.rows));
    const int32_t more = a.int32("more");
    const auto* more_lens = static_cast<const int32_t*>(a.vector("more_lens", kI32, t.rows));
    const at::Tensor& ws = scratch(a);
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_resize(n_pages, t.max_pages, t.rows, t.at, t.stride, refs, lens, more_lens, more,
                    ws.data_ptr(), ws.nbytes(), status, stream);
  });
}

PyObject* compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return entry(args, n, [](Args& a) {
    int32_t n_pages = -1;
    const int32_t* refs = counts(a, "refs", &n_pages);
    PageTable t{nullptr, 0, 1, 1}, out = t;
    const at::Tensor* table = a.tensor("page_table");
    const at::Tensor* table_out = a.tensor("table_out");
    if ((table == nullptr) != (table_out == nullptr)) refuse("page_table and table_out go together");
    if (table) {
      t = page_table(*table, "page_table");
      out = page_table(*table_out, "table_out");
      if (out.rows != t.rows || out.max_pages != t.max_pages)
        refuse("table_out must be as large as page_table");
    }
    int32_t* refs_out = counts(a, "refs_out", &n_pages);
    int64_t cap;
    int32_t* moves = moves_of(a, &cap);
    if (cap < 1 || cap < n_pages / 2) refuse("moves must have room for n_pages / 2 pairs (at least one)");
    auto* n_moves = required(static_cast<int32_t*>(a.vector("n_moves", kI32, 1)), "n_moves");
    auto* n_used = required(static_cast<int32_t*>(a.vector("n_used", kI32, 1)), "n_used");
    const at::Tensor& ws = scratch(a);
    auto* status = static_cast<int32_t*>(a.vector("dev_status", kI32, -1));
    void* stream = reinterpret_cast<void*>(a.integer("stream"));
    return g_compact(n_pages, t.max_pages, t.rows, t.at, t.stride, refs, out.at, out.stride,
                     refs_out, moves, n_moves, n_used, ws.data_ptr(), ws.nbytes(), status, stream);
  });
}

// The addresses of the calls, in the order of the pointers above.
PyObject* attach(PyObject*, PyObject* args) {
  unsigned long long f[10];
  if (!PyArg_ParseTuple(args, "KKKKKKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7],
                        &f[8], &f[9]))
    return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_route = reinterpret_cast<decltype(g_route)>(f[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[2]);
  g_append_axes = reinterpret_cast<decltype(g_append_axes)>(f[3]);
  g_tree = reinterpret_cast<decltype(g_tree)>(f[4]);
  g_accept = reinterpret_cast<decltype(g_accept)>(f[5]);
  g_copy = reinterpret_cast<decltype(g_copy)>(f[6]);
  g_fork = reinterpret_cast<decltype(g_fork)>(f[7]);
  g_resize = reinterpret_cast<decltype(g_resize)>(f[8]);
  g_compact = reinterpret_cast<decltype(g_compact)>(f[9]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"attach", attach, METH_VARARGS, nullptr},
    method<append>("append"), method<route>("route"), method<decode>("decode"),
    method<tree>("tree"), method<accept>("accept"), method<copy>("copy"), method<fork>("fork"),
    method<resize>("resize"), method<compact>("compact"),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sa_bind", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sa_bind() { return PyModule_Create(&module); }
