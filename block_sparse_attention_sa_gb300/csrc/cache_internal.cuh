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
int decode_row_tiles(int H, int Hkv);   // CTAs' worth of query heads on a key-value head
cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          bool fp8, cudaStream_t st);
size_t route_pages_ws_bytes(int64_t rows, int max_pages);
cudaError_t launch_route_pages(const RoutePagesArgs& a, cudaStream_t st);

#ifdef __CUDACC__
// A call's second kernel is launched while its first still runs and waits for
// its end, so that launch and set-up overlap. Not so from call to call: blocks
// of a next call that sit waiting on an SM take the place of a run of this one
// (e4m3 decoding of 3 x 112,640 tokens: 115 us so, 150 us with every launch close).
__device__ __forceinline__ void let_next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_first() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Loads of what an earlier kernel may have written. Never through the read-only
// path: such a load might be moved ahead of the wait.
template <class T>
__device__ __forceinline__ T get(const T* p) {
  return *p;
}

template <class... P, class... A>
cudaError_t launch_close(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// A length inside what the page table can hold.
__device__ __forceinline__ int clamp_len(int n, const PageMap& pm, bool* bad) {
  const int most = pm.max_pages * kBlock;
  *bad = n < 0 || n > most;
  return n < 0 ? 0 : (n > most ? most : n);
}

// The run of C an item of a list of T items lies in: the first T % C runs hold
// one item more than the others.
__device__ __forceinline__ int run_of(unsigned T, unsigned C, unsigned item) {
  const unsigned base = T / C, rem = T - base * C, big = rem * (base + 1);
  return item < big ? item / (base + 1) : rem + (item - big) / base;
}

struct Run {
  int T, lo, hi;           // items of the list, and this CTA's among them
  int group, off;          // where a run that is not empty begins: item `off` of a group,
  int count, size;         // and what count gave for that group
};

// The list is that of `groups` groups in order, each count(i, size) * per_group
// items (the host has checked that 31 bits hold them all); `size` is the caller's,
// given back for the first group, so that nothing is read twice on the way to the
// first item (a load takes 500 cycles and more here). Every CTA of the grid
// finds its run of it by a scan of the counts: up to 32 groups by each warp for
// itself, more by the CTA. All NT threads call it and get the same; it ends with
// every thread past a barrier.
template <int NT, class Count>
__device__ __forceinline__ Run plan_run(int groups, int per_group, Count count) {
  __shared__ int warp_sum[NT / 32], start[4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool few = groups <= 32;
  const int per_thread = few ? 1 : (groups + NT - 1) / NT, first = few ? lane : tid * per_thread;
  const int g0 = min(first, groups), g1 = min(g0 + per_thread, groups);
  int mine = 0, size = 0;
  for (int i = g0; i < g1; ++i) mine += count(i, &size);
  int incl = mine;
  if (groups > 1) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
  }
  int before = 0, total = 0;
  if (few) {
    total = __shfl_sync(0xffffffffu, incl, groups - 1);
  } else {
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
  }
  Run r;
  r.T = total * per_group;
  const unsigned C = gridDim.x, c = blockIdx.x;
  const unsigned base = static_cast<unsigned>(r.T) / C, rem = r.T - base * C;
  r.lo = base * c + min(c, rem);
  r.hi = r.lo + base + (c < rem ? 1 : 0);
  int at = (before + incl - mine) * per_group;
  const bool here = r.lo < r.hi && r.lo >= at && r.lo < at + mine * per_group;
  if (few) {                                 // a lane, a group
    r.group = max(__ffs(__ballot_sync(0xffffffffu, here)) - 1, 0);
    r.off = max(r.lo - __shfl_sync(0xffffffffu, at, r.group), 0);
    r.count = __shfl_sync(0xffffffffu, mine, r.group);
    r.size = __shfl_sync(0xffffffffu, size, r.group);
    __syncthreads();
    return r;
  }
  if (here) {
    int i = g0, n;
    while (r.lo >= at + (n = count(i, &size)) * per_group) {
      at += n * per_group;
      ++i;
    }
    start[0] = i;
    start[1] = r.lo - at;
    start[2] = n;
    start[3] = size;
  }
  __syncthreads();
  const bool any = r.lo < r.hi;
  r.group = any ? start[0] : 0;
  r.off = any ? start[1] : 0;
  r.count = any ? start[2] : 0;
  r.size = any ? start[3] : 0;
  return r;
}
#endif

}  // namespace sa
