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

sa_status sa_cache_append(const sa_cache_params* p, const void* k, const void* v, const void* q,
                          void* q_out, const float* gamma_q, const float* gamma_k,
                          const float* rope_cos, const float* rope_sin, void* k_cache,
                          void* v_cache, const float* k_scale, const float* v_scale, float* k_sum,
                          const int32_t* page_table, const int32_t* seq_lens,
                          const int32_t* new_lens, int32_t* lens_out, int32_t* dev_status,
                          void* stream) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
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
  return from_cuda(launch_append(a, p->D, p->cache_format == SA_CACHE_FP8,
                                 p->rope_layout == SA_ROPE_HALF,
                                 static_cast<cudaStream_t>(stream)));
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
  return decode_ws_bytes(p->H, p->H_kv, p->D);
}

sa_status sa_attn_decode(const sa_cache_params* p, const void* q, const void* k_cache,
                         const void* v_cache, const float* k_scale, const float* v_scale,
                         const int32_t* page_table, const int32_t* seq_lens,
                         const int32_t* row_ptr, const int32_t* col_idx, int64_t col_cap,
                         void* o, float* lse, void* workspace, size_t ws_bytes,
                         int32_t* dev_status, void* stream) {
  sa_status s = check_cache(p);
  if (s != SA_OK) return s;
  if (p->S != 1) return SA_ERR_UNSUPPORTED;
  // the pages of all units are counted in 31 bits
  if (static_cast<int64_t>(p->B) * p->H_kv * decode_row_tiles(p->H, p->H_kv) >
      INT32_MAX / static_cast<int64_t>(p->max_pages))
    return SA_ERR_UNSUPPORTED;
  if (col_cap < 0) return SA_ERR_INVALID_ARG;
  if (!q || !o || !workspace || (row_ptr == nullptr) != (col_idx == nullptr))
    return SA_ERR_INVALID_ARG;
  if ((s = check_pool(p, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)) != SA_OK)
    return s;
  if ((s = check_tokens(p, q, p->q_stride, p->H)) != SA_OK) return s;
  if ((s = check_tokens(p, o, p->o_stride, p->H)) != SA_OK) return s;
  if (!aligned(workspace, 256)) return SA_ERR_INVALID_ARG;
  if (ws_bytes < sa_attn_decode_workspace_bytes(p)) return SA_ERR_CAPACITY;
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
  a.H = p->H;
  a.Hkv = p->H_kv;
  a.D = p->D;
  const double scale = p->softmax_scale > 0.f ? static_cast<double>(p->softmax_scale)
                                              : 1.0 / std::sqrt(static_cast<double>(p->D));
  a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
  a.ws = static_cast<char*>(workspace);
  CUtensorMap kmap, vmap;
  if ((s = encode_cache(&kmap, k_cache, p, p->kc_stride)) != SA_OK) return s;
  if ((s = encode_cache(&vmap, v_cache, p, p->vc_stride)) != SA_OK) return s;
  return from_cuda(launch_decode(a, kmap, vmap, p->cache_format == SA_CACHE_FP8,
                                 static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
