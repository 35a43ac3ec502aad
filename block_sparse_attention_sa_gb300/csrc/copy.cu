// copy.cu -- what the pages of a cache hold: whole pages to others (sa_cache_copy), and
// the tokens of an accepted path together in their sequence's last pages
// (sa_cache_accept). Bytes as they are, 16 at a time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

// ---------------------------------------------------------------- copy --
// Bound by the memory. A CTA takes 16 KB of one page's keys or values at a time, four
// pieces of 16 bytes a thread on their way at once; with eight CTAs an SM as many bytes
// are in flight as the memory needs.
constexpr int kCopyThreads = 256;
constexpr int kPieces = 4;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a, int log_pieces, int slices) {
  const int64_t n = a.n_moves ? min(static_cast<int64_t>(max(get(a.n_moves), 0)), a.move_cap) : a.move_cap;
  const int total = a.Hkv * kBlock << log_pieces;          // pieces of a page
  int status = 0;
  for (int64_t it = blockIdx.x; it < n * 2 * slices; it += gridDim.x) {
    const int64_t i = it / (2 * slices);
    const int part = static_cast<int>(it - i * 2 * slices), which = part >= slices;
    const int slice = part - which * slices;
    const int from = get(a.moves + 2 * i), to = get(a.moves + 2 * i + 1);
    if (from < 0 || from >= a.n_pages || to < 0 || to >= a.n_pages) {
      status |= SA_DEV_BAD_CACHE;
      continue;
    }
    char* cache = which ? a.vc : a.kc;
    const int64_t* s = which ? a.vcs : a.kcs;
    uint4 w[kPieces];
    int64_t at[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int c = (slice * kPieces + u) * kCopyThreads + threadIdx.x;
      const int row = c >> log_pieces, head = row / kBlock;
      at[u] = c < total ? head * s[1] + row % kBlock * s[2] + (c & ((1 << log_pieces) - 1)) * 16 : -1;
      if (at[u] >= 0) w[u] = __ldcs(reinterpret_cast<const uint4*>(cache + from * s[0] + at[u]));
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      if (at[u] >= 0) __stcs(reinterpret_cast<uint4*>(cache + to * s[0] + at[u]), w[u]);
    if (a.k_sum && part == 0) {
      const int64_t per = static_cast<int64_t>(a.Hkv) * a.D;
      for (int e = threadIdx.x * 4; e < per; e += 4 * kCopyThreads)
        *reinterpret_cast<float4*>(a.k_sum + to * per + e) = *reinterpret_cast<const float4*>(a.k_sum + from * per + e);
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// -------------------------------------------------------------- accept --
// A CTA takes the keys, or the values, of one head of one sequence: all pieces of the
// path's tokens are read before the first is written, so that old and new places may
// overlap. Bound by its chain of dependent loads: lengths and path, page, keys, sums.
constexpr int kAcceptThreads = 256;

template <bool kFp8>
__device__ __forceinline__ void add_values(uint4 w, float* sum) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kFp8) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[i] >> (16 * y)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        sum[4 * i + 2 * y] += f.x;
        sum[4 * i + 2 * y + 1] += f.y;
      }
    } else {
      sum[2 * i] += __uint_as_float(u[i] << 16);
      sum[2 * i + 1] += __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(AcceptArgs a) {
  constexpr int kBytes = kFp8 ? D : 2 * D, kP = kBytes / 16;   // 16-byte pieces of a token
  constexpr int kRows = kAcceptThreads / kP;                   // tokens at a time
  constexpr int kPasses = SA_TREE_MAX / kRows, kElts = kFp8 ? 16 : 8;
  __shared__ int sm_page[2][SA_TREE_MAX], sm_from[SA_TREE_MAX];
  __shared__ uint32_t sm_good[2];
  __shared__ float sm_sum[kRows][D];
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
  const bool keys = blockIdx.y == 0;
  int status = 0;
  bool bad;
  const int base = clamp_len(get(a.pm.seq_lens + b), a.pm, &bad);
  if (bad) status |= SA_DEV_BAD_CACHE;
  const int m = min(max(get(a.path_lens + b), 0), a.S);
  const int32_t* table = a.pm.table + b * a.pm.table_stride;
  if (tid < SA_TREE_MAX) {
    const int32_t* path = a.path + b * a.path_stride;
    const int at = tid < m ? get(path + tid) : -1, prev = tid > 0 && tid < m ? get(path + tid - 1) : -1;
    const bool good = tid < m && at > prev && at < SA_TREE_MAX && at < a.pm.max_pages * kBlock - base;
    sm_from[tid] = at;
    if (good) {
      // where it lies and where it goes
      const int from = get(table + (base + at) / kBlock), to = get(table + (base + tid) / kBlock);
      const bool there = from >= 0 && from < a.pm.n_pages && to >= 0 && to < a.pm.n_pages;
      if (!there) status |= SA_DEV_BAD_CACHE;
      sm_page[0][tid] = there && at != tid ? from : -1;
      sm_page[1][tid] = to;
    }
    const uint32_t all = __ballot_sync(0xffffffffu, good);
    if (tid % 32 == 0) sm_good[tid / 32] = all;
  }
  __syncthreads();
  const uint64_t good = static_cast<uint64_t>(sm_good[1]) << 32 | sm_good[0];
  const int count = good == ~0ull ? SA_TREE_MAX : __ffsll(~good) - 1;     // as far as the path holds
  if (count < m) status |= SA_DEV_BAD_TREE;
  const int piece = tid % kP, grp = tid / kP;
  char* cache = (keys ? a.kc : a.vc) + h * (keys ? a.kcs[1] : a.vcs[1]) + piece * 16;
  const int64_t s_page = keys ? a.kcs[0] : a.vcs[0], s_tok = keys ? a.kcs[2] : a.vcs[2];
  uint4 w[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int i = u * kRows + grp;
    if (i < count && sm_page[0][i] >= 0)
      w[u] = *reinterpret_cast<const uint4*>(cache + sm_page[0][i] * s_page + (base + sm_from[i]) % kBlock * s_tok);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int i = u * kRows + grp;
    if (i < count && sm_page[0][i] >= 0)
      *reinterpret_cast<uint4*>(cache + sm_page[1][i] * s_page + (base + i) % kBlock * s_tok) = w[u];
  }
  const int end = base + count;
  if (keys && a.k_sum) {
    const float scale = kFp8 && a.k_scale ? get(a.k_scale + h) : 1.f;
    for (int j = base / kBlock; j * kBlock < end; ++j) {
      __syncthreads();                       // the keys are stored; the last page's sums are read
      const int page = get(table + j), live = min(kBlock, end - j * kBlock);
      if (page < 0 || page >= a.pm.n_pages) {
        status |= SA_DEV_BAD_CACHE;
        continue;
      }
      float sum[kElts] = {};
#pragma unroll
      for (int u = 0; u < kBlock / kRows; ++u) {
        const int t = u * kRows + grp;
        if (t < live)
          add_values<kFp8>(*reinterpret_cast<const uint4*>(cache + page * s_page + t * s_tok), sum);
      }
#pragma unroll
      for (int i = 0; i < kElts; ++i) sm_sum[grp][piece * kElts + i] = sum[i];
      __syncthreads();
      if (tid < D) {
        float all = 0.f;
#pragma unroll 8
        for (int g = 0; g < kRows; ++g) all += sm_sum[g][tid];
        a.k_sum[(static_cast<int64_t>(page) * a.Hkv + h) * D + tid] = all * scale;
      }
    }
  }
  if (a.lens_out && h == 0 && keys && tid == 0) a.lens_out[b] = end;
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

template <int D, bool kFp8>
cudaError_t launch(const AcceptArgs& a, cudaStream_t st) {
  accept_kernel<D, kFp8><<<dim3(static_cast<unsigned>(a.B * a.Hkv), 2), kAcceptThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, int D, bool fp8, cudaStream_t st) {
  if (D == 64) return fp8 ? launch<64, true>(a, st) : launch<64, false>(a, st);
  return fp8 ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

cudaError_t launch_copy(const CopyArgs& a, cudaStream_t st) {
  const int pieces = a.row_bytes / 16, log_pieces = pieces == 4 ? 2 : (pieces == 8 ? 3 : 4);
  const int slices = (a.Hkv * kBlock * pieces + kCopyThreads * kPieces - 1) / (kCopyThreads * kPieces);
  const int64_t items = a.move_cap * 2 * slices;
  const int grid = static_cast<int>(items < 152 * 8 ? items : 152 * 8);
  copy_kernel<<<grid, kCopyThreads, 0, st>>>(a, log_pieces, slices);
  return cudaGetLastError();
}

}  // namespace sa
