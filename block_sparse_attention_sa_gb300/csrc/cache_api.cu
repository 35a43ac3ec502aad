// cache_api.cu -- the extern "C" boundary of the paged cache: argument checks
// and launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "cache_internal.cuh"

namespace sa {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sa_status check_cache(const sa_cache_params* p) {
  if (!p) return SA_ERR_INVALID_ARG;
  if (p->B < 1 || p->S < 1 || p->H < 1 || p->H_kv < 1 || p->D < 1) return SA_ERR_INVALID_ARG;
  if (p->H % p->H_kv != 0 || p->page != kBlock) return SA_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->max_pages < 1 || p->max_pages >= (1 << 25)) return SA_ERR_INVALID_ARG;
  if (p->cache_format != SA_CACHE_BF16 && p->cache_format != SA_CACHE_FP8) return SA_ERR_INVALID_ARG;
  if (p->rope_layout != SA_ROPE_INTERLEAVED && p->rope_layout != SA_ROPE_HALF)
    return SA_ERR_INVALID_ARG;
  if (p->prefix_len < 0 || p->page_budget < 0 || p->rope_rows < 0) return SA_ERR_INVALID_ARG;
  if (p->qk_norm != 0 && p->qk_norm != 1) return SA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return SA_ERR_INVALID_ARG;
  if (!(p->softmax_scale >= 0.f) || !std::isfinite(p->softmax_scale)) return SA_ERR_INVALID_ARG;
  if (p->B > 1 && p->table_stride < p->max_pages) return SA_ERR_INVALID_ARG;
  if (p->D != 64 && p->D != 128) return SA_ERR_UNSUPPORTED;
  if (p->B > 65535 || p->H > 65535) return SA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->B) * p->H > INT32_MAX) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

// Strides are positive multiples of `mult` elements; that of an axis with one
// entry is never used.
bool strides_fit(const int64_t s[3], const int64_t extent[3], int64_t mult) {
  for (int i = 0; i < 3; ++i)
    if (extent[i] > 1 && (s[i] <= 0 || s[i] % mult != 0)) return false;
  return true;
}

sa_status check_tokens(const sa_cache_params* p, const void* x, const int64_t s[3], int heads) {
  const int64_t extent[3] = {p->B, p->S, heads};
  return aligned(x, 16) && strides_fit(s, extent, 8) ? SA_OK : SA_ERR_INVALID_ARG;
}

// Whether two arrays of n lengths (b may be null) share an entry.
bool lens_overlap(const int32_t* a, const int32_t* b, int n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return b && (x > y ? x - y : y - x) < static_cast<uintptr_t>(n) * sizeof(int32_t);
}

// The pool, its scales and the page table.
sa_status check_pool(const sa_cache_params* p, const void* kc, const void* vc, const float* ks,
                     const float* vs, const int32_t* table, const int32_t* lens) {
  if (!kc || !vc || !table || !lens) return SA_ERR_INVALID_ARG;
  if (!aligned(kc, 16) || !aligned(vc, 16)) return SA_ERR_INVALID_ARG;
  const int64_t extent[3] = {p->n_pages, p->H_kv, kBlock};
  const int64_t mult = p->cache_format == SA_CACHE_FP8 ? 16 : 8;
  if (!strides_fit(p->kc_stride, extent, mult) || !strides_fit(p->vc_stride, extent, mult))
    return SA_ERR_INVALID_ARG;
  if (p->cache_format == SA_CACHE_BF16 && (ks || vs)) return SA_ERR_INVALID_ARG;
  return SA_OK;
}

PageMap page_map(const sa_cache_params* p, const int32_t* table, const int32_t* lens) {
  PageMap m{};
  m.table = table;
  m.seq_lens = lens;
  m.table_stride = p->B > 1 ? p->table_stride : 0;
  m.n_pages = p->n_pages;
  m.max_pages = p->max_pages;
  return m;
}

void copy3(int64_t to[3], const int64_t from[3]) {
  for (int i = 0; i < 3; ++i) to[i] = from[i];
}

int64_t most_pages(const sa_cache_params* p) {
  const int64_t forced = (static_cast<int64_t>(p->prefix_len) + kBlock - 1) / kBlock + 1;
  return std::min<int64_t>(p->max_pages, std::max<int64_t>(p->page_budget, forced));
}

sa_status check_route_pages(const sa_cache_params* p) {
  const sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  if (p->S != 1) return SA_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(p->B) * p->H_kv;
  if (p->max_pages > (1 << 20) || rows * p->max_pages > INT32_MAX || rows * most_pages(p) > INT32_MAX)
    return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

// [n_pages, Hkv, 64, D] -> 4-D map (D, token, head, page); the box is one
// head's page, at most 128 bytes of each token, swizzled over as many bytes.
sa_status encode_cache(CUtensorMap* m, const void* base, const sa_cache_params* p,
                       const int64_t st[3]) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return SA_ERR_CUDA;
  const bool f8 = p->cache_format == SA_CACHE_FP8;
  const cuuint64_t elt = f8 ? 1 : 2, D = static_cast<cuuint64_t>(p->D);
  // the stride of an axis with one entry is never used, but must be encodable
  auto bytes = [&](int i, int64_t extent) { return extent > 1 ? static_cast<cuuint64_t>(st[i]) * elt : D * elt; };
  const cuuint64_t dims[4] = {D, kBlock, static_cast<cuuint64_t>(p->H_kv),
                              static_cast<cuuint64_t>(p->n_pages)};
  const cuuint64_t strides[3] = {bytes(2, kBlock), bytes(1, p->H_kv), bytes(0, p->n_pages)};
  const bool wide = D * elt >= 128;
  const cuuint32_t box[4] = {wide ? static_cast<cuuint32_t>(128 / elt) : 64u, kBlock, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE,
                        wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SA_OK : SA_ERR_INVALID_ARG;
}

// A pool of n_pages and a table of `rows` sequences, `stride` entries apart.
sa_status check_pages(int64_t n_pages, int64_t max_pages, int64_t rows, int64_t stride) {
  if (n_pages < 1 || max_pages < 1 || rows < 1) return SA_ERR_INVALID_ARG;
  if (rows > 1 && stride < max_pages) return SA_ERR_INVALID_ARG;
  if (n_pages >= (1 << 25) || max_pages >= (1 << 25) || rows > 16384) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

sa_status check_pages_ws(int n_pages, int rows, const void* ws, size_t bytes) {
  if (!ws || !aligned(ws, 256)) return SA_ERR_INVALID_ARG;
  return bytes < pages_ws_bytes(n_pages, rows) ? SA_ERR_CAPACITY : SA_OK;
}

int64_t table_entries(int64_t max_pages, int64_t rows, int64_t stride) {
  return (rows - 1) * stride + max_pages;
}

bool overlap(const int32_t* a, int64_t n, const int32_t* b, int64_t m) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(m) * 4 && y < x + static_cast<uintptr_t>(n) * 4;
}

sa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

}  // namespace
}  // namespace sa

using namespace sa;

extern "C" {

void sa_cache_params_init(sa_cache_params* p, int32_t B, int32_t H, int32_t H_kv, int32_t D,
                          int32_t n_pages, int32_t max_pages) {
  if (!p) return;
  std::memset(p, 0, sizeof(*p));
  p->B = B;
  p->S = 1;
  p->H = H;
  p->H_kv = H_kv;
  p->D = D;
  p->page = kBlock;
  p->n_pages = n_pages;
  p->max_pages = max_pages;
  p->eps = 1e-6f;
  p->table_stride = max_pages;
  const int64_t d = D;
  const int64_t qs[3] = {H * d, H * d, d}, ks[3] = {H_kv * d, H_kv * d, d};
  const int64_t cs[3] = {H_kv * kBlock * d, kBlock * d, d};
  copy3(p->q_stride, qs);
  copy3(p->o_stride, qs);
  copy3(p->k_stride, ks);
  copy3(p->v_stride, ks);
  copy3(p->kc_stride, cs);
  copy3(p->vc_stride, cs);
}

static sa_status append(const sa_cache_params* p, const void* k, const void* v, const void* q,
                        void* q_out, const float* gamma_q, const float* gamma_k,
                        const float* rope_cos, const float* rope_sin, const sa_rope_axes* axes,
                        void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                        float* k_sum, const int32_t* page_table, const int32_t* seq_lens,
                        const int32_t* new_lens, int32_t* lens_out, int32_t* dev_status,
                        void* stream) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  if (axes && ((s = check_axes(axes, p->B, p->S, p->D)) != SA_OK)) return s;
  if (axes && (!rope_cos || !rope_sin)) return SA_ERR_INVALID_ARG;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return SA_ERR_INVALID_ARG;
  if ((s = check_pool(p, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)) != SA_OK)
    return s;
  if ((s = check_tokens(p, k, p->k_stride, p->H_kv)) != SA_OK) return s;
  if ((s = check_tokens(p, v, p->v_stride, p->H_kv)) != SA_OK) return s;
  if (q) {
    if ((s = check_tokens(p, q, p->q_stride, p->H)) != SA_OK) return s;
    if ((s = check_tokens(p, q_out, p->o_stride, p->H)) != SA_OK) return s;
  }
  if (!p->qk_norm && (gamma_q || gamma_k)) return SA_ERR_INVALID_ARG;
  if (!aligned(gamma_q, 16) || !aligned(gamma_k, 16) || !aligned(rope_cos, 16) ||
      !aligned(rope_sin, 16) || !aligned(k_sum, 16))
    return SA_ERR_INVALID_ARG;
  if ((rope_cos == nullptr) != (rope_sin == nullptr)) return SA_ERR_INVALID_ARG;
  // written by some CTAs while others still read those
  if (lens_out && (lens_overlap(lens_out, seq_lens, p->B) || lens_overlap(lens_out, new_lens, p->B)))
    return SA_ERR_INVALID_ARG;
  if (q && q == q_out)
    for (int i = 0; i < 3; ++i)
      if (p->q_stride[i] != p->o_stride[i]) return SA_ERR_INVALID_ARG;
  // blocks of the launch, counted in 32 bits
  const int64_t rows = static_cast<int64_t>(p->B) * (p->S / kBlock + 2) * p->H_kv +
                       static_cast<int64_t>(p->B) * p->S;
  if (rows > INT32_MAX) return SA_ERR_UNSUPPORTED;
  AppendArgs a{};
  a.pm = page_map(p, page_table, seq_lens);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  copy3(a.qs, p->q_stride);
  copy3(a.ks, p->k_stride);
  copy3(a.vs, p->v_stride);
  copy3(a.os, p->o_stride);
  a.gamma_q = gamma_q;
  a.gamma_k = gamma_k;
  a.cos = rope_cos;
  a.sin = rope_sin;
  a.kc = k_cache;
  a.vc = v_cache;
  copy3(a.kcs, p->kc_stride);
  copy3(a.vcs, p->vc_stride);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.k_sum = k_sum;
  a.new_lens = new_lens;
  a.lens_out = lens_out;
  a.dev_status = dev_status;
  a.B = p->B;
  a.S = p->S;
  a.H = p->H;
  a.Hkv = p->H_kv;
  a.rope_rows = p->rope_rows;
  a.eps = p->eps;
  a.norm = p->qk_norm;
  if (axes) a.axes = *axes;
  return from_cuda(launch_append(a, p->D, p->cache_format == SA_CACHE_FP8,
                                 p->rope_layout == SA_ROPE_HALF,
                                 static_cast<cudaStream_t>(stream)));
}

sa_status sa_cache_append(const sa_cache_params* p, const void* k, const void* v, const void* q,
                          void* q_out, const float* gamma_q, const float* gamma_k,
                          const float* rope_cos, const float* rope_sin, void* k_cache,
                          void* v_cache, const float* k_scale, const float* v_scale, float* k_sum,
                          const int32_t* page_table, const int32_t* seq_lens,
                          const int32_t* new_lens, int32_t* lens_out, int32_t* dev_status,
                          void* stream) {
  return append(p, k, v, q, q_out, gamma_q, gamma_k, rope_cos, rope_sin, nullptr, k_cache, v_cache,
                k_scale, v_scale, k_sum, page_table, seq_lens, new_lens, lens_out, dev_status,
                stream);
}

sa_status sa_cache_append_axes(const sa_cache_params* p, const void* k, const void* v,
                               const void* q, void* q_out, const float* gamma_q,
                               const float* gamma_k, const float* rope_cos,
                               const float* rope_sin, const sa_rope_axes* axes, void* k_cache,
                               void* v_cache, const float* k_scale, const float* v_scale,
                               float* k_sum, const int32_t* page_table, const int32_t* seq_lens,
                               const int32_t* new_lens, int32_t* lens_out, int32_t* dev_status,
                               void* stream) {
  if (!axes) return SA_ERR_INVALID_ARG;
  return append(p, k, v, q, q_out, gamma_q, gamma_k, rope_cos, rope_sin, axes, k_cache, v_cache,
                k_scale, v_scale, k_sum, page_table, seq_lens, new_lens, lens_out, dev_status,
                stream);
}

int64_t sa_route_pages_max_nnz(const sa_cache_params* p) {
  if (check_route_pages(p) != SA_OK) return 0;
  return static_cast<int64_t>(p->B) * p->H_kv * most_pages(p);
}

size_t sa_route_pages_workspace_bytes(const sa_cache_params* p) {
  if (check_route_pages(p) != SA_OK) return 0;
  return route_pages_ws_bytes(static_cast<int64_t>(p->B) * p->H_kv, p->max_pages);
}

sa_status sa_route_pages(const sa_cache_params* p, const void* q, const float* k_sum,
                         const int32_t* page_table, const int32_t* seq_lens, int32_t* row_ptr,
                         int32_t* col_idx, int64_t col_cap, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream) {
  sa_status s = check_route_pages(p);
  if (s != SA_OK) return s;
  if (!q || !k_sum || !page_table || !seq_lens || !row_ptr || !col_idx || !workspace)
    return SA_ERR_INVALID_ARG;
  if (col_cap < 0 || !aligned(k_sum, 16) || !aligned(workspace, 256)) return SA_ERR_INVALID_ARG;
  if ((s = check_tokens(p, q, p->q_stride, p->H)) != SA_OK) return s;
  if (ws_bytes < sa_route_pages_workspace_bytes(p)) return SA_ERR_CAPACITY;
  RoutePagesArgs a{};
  a.pm = page_map(p, page_table, seq_lens);
  a.q = static_cast<const uint16_t*>(q);
  a.k_sum = k_sum;
  copy3(a.qs, p->q_stride);
  a.row_ptr = row_ptr;
  a.col_idx = col_idx;
  a.col_cap = col_cap;
  a.ws = static_cast<char*>(workspace);
  a.dev_status = dev_status;
  a.B = p->B;
  a.H = p->H;
  a.Hkv = p->H_kv;
  a.D = p->D;
  a.prefix = p->prefix_len;
  a.budget = p->page_budget;
  return from_cuda(launch_route_pages(a, static_cast<cudaStream_t>(stream)));
}

size_t sa_attn_decode_workspace_bytes(const sa_cache_params* p) {
  if (check_cache(p) != SA_OK || p->S != 1) return 0;
  return decode_ws_bytes(p->H / p->H_kv, p->D);
}

size_t sa_attn_tree_workspace_bytes(const sa_cache_params* p) {
  if (check_cache(p) != SA_OK || p->S > SA_TREE_MAX) return 0;
  return tree_ws_bytes(p->S * (p->H / p->H_kv), p->D);
}

// Attention over the cache: of one new token, or (tree) of a few.
static sa_status attend(const sa_cache_params* p, const void* q, const void* k_cache,
                        const void* v_cache, const float* k_scale, const float* v_scale,
                        const int32_t* page_table, const int32_t* seq_lens,
                        const int32_t* new_lens, const int32_t* parents, int64_t parent_stride,
                        const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap, void* o,
                        float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                        void* stream, bool tree) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  if (p->S > (tree ? SA_TREE_MAX : 1)) return SA_ERR_UNSUPPORTED;
  // the pages of all units are counted in 31 bits; with a tree a row of the route may
  // list the two that hold new tokens besides
  const int rows = p->S * (p->H / p->H_kv);
  if (static_cast<int64_t>(p->B) * p->H_kv * decode_row_tiles(rows) >
      INT32_MAX / (static_cast<int64_t>(p->max_pages) + (tree ? 2 : 0)))
    return SA_ERR_UNSUPPORTED;
  if (col_cap < 0) return SA_ERR_INVALID_ARG;
  if (!q || !o || !workspace || (row_ptr == nullptr) != (col_idx == nullptr))
    return SA_ERR_INVALID_ARG;
  if (parents && p->B > 1 && (parent_stride < 0 || (parent_stride > 0 && parent_stride < p->S)))
    return SA_ERR_INVALID_ARG;
  if ((s = check_pool(p, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)) != SA_OK)
    return s;
  if ((s = check_tokens(p, q, p->q_stride, p->H)) != SA_OK) return s;
  if ((s = check_tokens(p, o, p->o_stride, p->H)) != SA_OK) return s;
  if (!aligned(workspace, 256)) return SA_ERR_INVALID_ARG;
  if (ws_bytes < (tree ? tree_ws_bytes(rows, p->D) : decode_ws_bytes(rows, p->D))) return SA_ERR_CAPACITY;
  if (o == q) return SA_ERR_INVALID_ARG;       // read by CTAs that others' outputs would meet
  DecodeArgs a{};
  a.pm = page_map(p, page_table, seq_lens);
  a.q = static_cast<const uint16_t*>(q);
  a.kc = k_cache;
  a.vc = v_cache;
  copy3(a.qs, p->q_stride);
  copy3(a.os, p->o_stride);
  copy3(a.kcs, p->kc_stride);
  copy3(a.vcs, p->vc_stride);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.row_ptr = row_ptr;
  a.col_idx = col_idx;
  a.col_cap = col_cap;
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.dev_status = dev_status;
  a.B = p->B;
  a.S = p->S;
  a.H = p->H;
  a.Hkv = p->H_kv;
  a.D = p->D;
  a.new_lens = new_lens;
  a.parents = parents;
  a.parent_stride = p->B > 1 ? parent_stride : 0;
  const double scale = p->softmax_scale > 0.f ? static_cast<double>(p->softmax_scale)
                                              : 1.0 / std::sqrt(static_cast<double>(p->D));
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  a.ws = static_cast<char*>(workspace);
  CUtensorMap kmap, vmap;
  if ((s = encode_cache(&kmap, k_cache, p, p->kc_stride)) != SA_OK) return s;
  if ((s = encode_cache(&vmap, v_cache, p, p->vc_stride)) != SA_OK) return s;
  const bool fp8 = p->cache_format == SA_CACHE_FP8;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return from_cuda(tree ? launch_tree(a, kmap, vmap, fp8, st) : launch_decode(a, kmap, vmap, fp8, st));
}

sa_status sa_attn_decode(const sa_cache_params* p, const void* q, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale,
                         const int32_t* page_table, const int32_t* seq_lens,
                         const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap,
                         void* o, float* lse, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream) {
  return attend(p, q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, nullptr, nullptr,
                0, row_ptr, col_idx, col_cap, o, lse, workspace, ws_bytes, dev_status, stream,
                false);
}

sa_status sa_attn_tree(const sa_cache_params* p, const void* q, const void* k_cache,
                       const void* v_cache, const float* k_scale, const float* v_scale,
                       const int32_t* page_table, const int32_t* seq_lens,
                       const int32_t* new_lens, const int32_t* parents, int64_t parent_stride,
                       const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap, void* o,
                       float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status,
                       void* stream) {
  return attend(p, q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, new_lens, parents,
                parent_stride, row_ptr, col_idx, col_cap, o, lse, workspace, ws_bytes, dev_status,
                stream, true);
}

sa_status sa_cache_accept(const sa_cache_params* p, void* k_cache, void* v_cache,
                          const float* k_scale, float* k_sum, const int32_t* page_table,
                          const int32_t* seq_lens, const int32_t* path, int64_t path_stride,
                          const int32_t* path_lens, int32_t* lens_out, int32_t* dev_status,
                          void* stream) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  if (p->S > SA_TREE_MAX) return SA_ERR_UNSUPPORTED;
  if ((s = check_pool(p, k_cache, v_cache, k_scale, nullptr, page_table, seq_lens)) != SA_OK)
    return s;
  if (!path || !path_lens || !aligned(k_sum, 16)) return SA_ERR_INVALID_ARG;
  if (p->B > 1 && path_stride < p->S) return SA_ERR_INVALID_ARG;
  // written by some CTAs while others still read those
  if (lens_out && (lens_overlap(lens_out, seq_lens, p->B) || lens_overlap(lens_out, path_lens, p->B)))
    return SA_ERR_INVALID_ARG;
  AcceptArgs a{};
  a.pm = page_map(p, page_table, seq_lens);
  a.kc = static_cast<char*>(k_cache);
  a.vc = static_cast<char*>(v_cache);
  const int64_t elt = p->cache_format == SA_CACHE_FP8 ? 1 : 2;
  for (int i = 0; i < 3; ++i) {
    a.kcs[i] = p->kc_stride[i] * elt;
    a.vcs[i] = p->vc_stride[i] * elt;
  }
  a.k_scale = k_scale;
  a.k_sum = k_sum;
  a.path = path;
  a.path_stride = p->B > 1 ? path_stride : 0;
  a.path_lens = path_lens;
  a.lens_out = lens_out;
  a.dev_status = dev_status;
  a.B = p->B;
  a.S = p->S;
  a.Hkv = p->H_kv;
  return from_cuda(launch_accept(a, p->D, elt == 1, static_cast<cudaStream_t>(stream)));
}

sa_status sa_cache_copy(const sa_cache_params* p, void* k_cache, void* v_cache, float* k_sum,
                        const int32_t* moves, int64_t move_cap, const int32_t* n_moves,
                        int32_t* dev_status, void* stream) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  // no table or lengths here: the moves stand in for them in the check of the pool
  if ((s = check_pool(p, k_cache, v_cache, nullptr, nullptr, moves, moves)) != SA_OK) return s;
  if (move_cap < 1 || !aligned(k_sum, 16)) return SA_ERR_INVALID_ARG;
  if (move_cap > INT32_MAX) return SA_ERR_UNSUPPORTED;
  CopyArgs a{};
  a.kc = static_cast<char*>(k_cache);
  a.vc = static_cast<char*>(v_cache);
  const int64_t elt = p->cache_format == SA_CACHE_FP8 ? 1 : 2;
  for (int i = 0; i < 3; ++i) {
    a.kcs[i] = p->kc_stride[i] * elt;
    a.vcs[i] = p->vc_stride[i] * elt;
  }
  a.k_sum = k_sum;
  a.moves = moves;
  a.n_moves = n_moves;
  a.move_cap = move_cap;
  a.dev_status = dev_status;
  a.n_pages = p->n_pages;
  a.Hkv = p->H_kv;
  a.D = p->D;
  a.row_bytes = static_cast<int>(p->D * elt);
  return from_cuda(launch_copy(a, static_cast<cudaStream_t>(stream)));
}

size_t sa_pages_workspace_bytes(int32_t n_pages, int32_t rows) {
  return check_pages(n_pages, 1, rows, 1) == SA_OK ? pages_ws_bytes(n_pages, rows) : 0;
}

sa_status sa_pages_fork(int32_t n_pages, int32_t max_pages, int32_t B, int32_t N,
                        const int32_t* page_table, int64_t table_stride,
                        const int32_t* seq_lens, const int32_t* refs, const int32_t* src,
                        int32_t* table_out, int64_t out_stride, int32_t* lens_out,
                        int32_t* refs_out, int32_t* moves, int32_t* n_moves, void* workspace,
                        size_t ws_bytes, int32_t* dev_status, void* stream) {
  sa_status s = check_pages(n_pages, max_pages, B, table_stride);
  if (s != SA_OK || (s = check_pages(n_pages, max_pages, N, out_stride)) != SA_OK) return s;
  if (!page_table || !seq_lens || !refs || !src || !table_out || !lens_out || !refs_out || !moves ||
      !n_moves)
    return SA_ERR_INVALID_ARG;
  if ((s = check_pages_ws(n_pages, std::max(B, N), workspace, ws_bytes)) != SA_OK) return s;
  const int64_t in = table_entries(max_pages, B, table_stride), out = table_entries(max_pages, N, out_stride);
  if (overlap(table_out, out, page_table, in) || overlap(lens_out, N, seq_lens, B) ||
      (refs_out != refs && overlap(refs_out, n_pages, refs, n_pages)))
    return SA_ERR_INVALID_ARG;
  PagesArgs a{};
  a.table = page_table;
  a.stride = table_stride;
  a.table_out = table_out;
  a.out_stride = out_stride;
  a.lens = seq_lens;
  a.refs = refs;
  a.refs_out = refs_out;
  a.src = src;
  a.lens_out = lens_out;
  a.moves = moves;
  a.n_moves = n_moves;
  a.ws = static_cast<int32_t*>(workspace);
  a.dev_status = dev_status;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.B = B;
  a.N = N;
  return from_cuda(launch_pages_fork(a, static_cast<cudaStream_t>(stream)));
}

sa_status sa_pages_resize(int32_t n_pages, int32_t max_pages, int32_t B, int32_t* page_table,
                          int64_t table_stride, int32_t* refs, const int32_t* seq_lens,
                          const int32_t* more_lens, int32_t more, void* workspace,
                          size_t ws_bytes, int32_t* dev_status, void* stream) {
  sa_status s = check_pages(n_pages, max_pages, B, table_stride);
  if (s != SA_OK) return s;
  if (!page_table || !seq_lens || !refs) return SA_ERR_INVALID_ARG;
  if ((s = check_pages_ws(n_pages, B, workspace, ws_bytes)) != SA_OK) return s;
  PagesArgs a{};
  a.table = a.table_out = page_table;
  a.stride = a.out_stride = table_stride;
  a.lens = seq_lens;
  a.more_lens = more_lens;
  a.more = more;
  a.refs = a.refs_out = refs;
  a.ws = static_cast<int32_t*>(workspace);
  a.dev_status = dev_status;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.B = B;
  return from_cuda(launch_pages_resize(a, static_cast<cudaStream_t>(stream)));
}

sa_status sa_pages_compact(int32_t n_pages, int32_t max_pages, int32_t B,
                           const int32_t* page_table, int64_t table_stride, const int32_t* refs,
                           int32_t* table_out, int64_t out_stride, int32_t* refs_out,
                           int32_t* moves, int32_t* n_moves, int32_t* n_used, void* workspace,
                           size_t ws_bytes, int32_t* dev_status, void* stream) {
  sa_status s = B == 0 ? check_pages(n_pages, 1, 1, 1) : check_pages(n_pages, max_pages, B, table_stride);
  if (s != SA_OK) return s;
  if (B > 0 && (s = check_pages(n_pages, max_pages, B, out_stride)) != SA_OK) return s;
  if ((B > 0) != (page_table != nullptr) || (B > 0) != (table_out != nullptr)) return SA_ERR_INVALID_ARG;
  if (!refs || !refs_out || !moves || !n_moves || !n_used) return SA_ERR_INVALID_ARG;
  if ((s = check_pages_ws(n_pages, std::max(B, 1), workspace, ws_bytes)) != SA_OK) return s;
  if (B > 0 && !(table_out == page_table && (B == 1 || out_stride == table_stride)) &&
      overlap(table_out, table_entries(max_pages, B, out_stride), page_table,
              table_entries(max_pages, B, table_stride)))
    return SA_ERR_INVALID_ARG;
  if (refs_out != refs && overlap(refs_out, n_pages, refs, n_pages)) return SA_ERR_INVALID_ARG;
  PagesArgs a{};
  a.table = page_table;
  a.stride = table_stride;
  a.table_out = table_out;
  a.out_stride = out_stride;
  a.refs = refs;
  a.refs_out = refs_out;
  a.moves = moves;
  a.n_moves = n_moves;
  a.n_used = n_used;
  a.ws = static_cast<int32_t*>(workspace);
  a.dev_status = dev_status;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.B = B;
  return from_cuda(launch_pages_compact(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
