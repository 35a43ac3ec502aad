// cache_internal.cuh -- shared between the paged-cache host code and kernels.
#pragma once

#include "sa_internal.cuh"

namespace sa {

// Where the tokens of a sequence live (sa_cache_params).
struct PageMap {
  const int32_t* table;      // [B][table_stride]
  const int32_t* seq_lens;   // [B]
  int64_t table_stride;
  int n_pages, max_pages;
};

struct AppendArgs {
  PageMap pm;
  const uint16_t* k;         // bf16 bits, [B, S, Hkv, D]
  const uint16_t* v;
  const uint16_t* q;         // [B, S, H, D] or nullptr
  uint16_t* q_out;
  int64_t qs[3], ks[3], vs[3], os[3];
  const float* gamma_q;      // [D] or nullptr (ones)
  const float* gamma_k;
  const float* cos;          // [rope_rows][D/2] or nullptr (then sin too)
  const float* sin;
  void* kc;                  // bf16 bits or e4m3 codes
  void* vc;
  int64_t kcs[3], vcs[3];    // element strides of page, head, token
  const float* k_scale;      // [Hkv] or nullptr (ones)
  const float* v_scale;
  float* k_sum;              // [n_pages][Hkv][D] or nullptr
  const int32_t* new_lens;   // [B] or nullptr (S each)
  int32_t* lens_out;         // [B] or nullptr
  int32_t* dev_status;
  int B, S, H, Hkv, rope_rows;
  float eps;
  int norm;
};

struct DecodeArgs {
  PageMap pm;
  const uint16_t* q;         // bf16 bits, [B, 1, H, D]
  const void* kc;
  const void* vc;
  int64_t qs[3], os[3], kcs[3], vcs[3];
  const float* k_scale;
  const float* v_scale;
  const int32_t* row_ptr;    // nullptr: every page
  const int32_t* col_idx;
  int64_t col_cap;
  uint16_t* o;
  float* lse;
  int32_t* dev_status;
  int B, H, Hkv, D;
  float scale_log2;          // softmax_scale * log2(e)
  char* ws;
};

struct RoutePagesArgs {
  PageMap pm;
  const uint16_t* q;
  const float* k_sum;
  int64_t qs[3];
  int32_t* row_ptr;
  int32_t* col_idx;
  int64_t col_cap;
  char* ws;
  int32_t* dev_status;
  int B, H, Hkv, D, prefix, budget;
};

cudaError_t launch_append(const AppendArgs& a, int D, bool fp8, bool half, cudaStream_t st);
size_t decode_ws_bytes(int H, int Hkv, int D);
cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          bool fp8, cudaStream_t st);
size_t route_pages_ws_bytes(int64_t rows, int max_pages);
cudaError_t launch_route_pages(const RoutePagesArgs& a, cudaStream_t st);

#ifdef __CUDACC__
// A length inside what the page table can hold.
__device__ __forceinline__ int clamp_len(int n, const PageMap& pm, bool* bad) {
  const int most = pm.max_pages * kBlock;
  *bad = n < 0 || n > most;
  return n < 0 ? 0 : (n > most ? most : n);
}
#endif

}  // namespace sa
