// copy.cu -- what the pages of a cache hold: whole pages to others (sa_cache_copy), and
// the tokens of an accepted path together in their sequence's last pages
// (sa_cache_accept). Bytes as they are, 16 at a time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

// ---------------------------------------------------------------- copy --
// Bound by the memory: 1,396 pages of 8 heads of 128 in bf16, 366 MB read and as much
// written in 118 us, 6.2 TB/s. A CTA takes 16 KB of one page's keys or values at a time, four pieces
// of 16 bytes a thread on their way at once; with eight CTAs an SM as many bytes are in
// flight as the memory needs.
constexpr int kCopyThreads = 256;
constexpr int kPieces = 4;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyArgs a, int log_pieces, int slices) {
  wait_for_first();                  // launched while what names the pages still runs
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
// overlap. What counts is the chain of dependent loads: lengths and path, pages, then at
// once the tokens and, for the sums, the keys that lie before them in their page. The sums
// come from the registers; only tokens of two pages can be among them. 128 sequences of 64
// new tokens, 8 heads of 128 in e4m3: 6.8 us in a graph (10.3 us with the sums read back
// from the page behind the stores and 256 threads a CTA, in two waves).
constexpr int kAcceptThreads = 128;

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
  // where a token lies and where it goes, as page * 64 + slot; -1: nowhere
  __shared__ int64_t sm_from[SA_TREE_MAX], sm_to[SA_TREE_MAX];
  __shared__ uint32_t sm_good[2];
  __shared__ float sm_sum[2][kAcceptThreads / 32][D];
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, tid = threadIdx.x;
  const bool keys = blockIdx.y == 0, sums = keys && a.k_sum != nullptr;
  int status = 0;
  // the path is on its way with the lengths
  const int32_t* path = a.path + b * a.path_stride;
  const int at = tid < a.S ? get(path + tid) : -1, prev = tid > 0 && tid < a.S ? get(path + tid - 1) : -1;
  bool bad;
  const int base = clamp_len(get(a.pm.seq_lens + b), a.pm, &bad);
  if (bad) status |= SA_DEV_BAD_CACHE;
  const int m = min(max(get(a.path_lens + b), 0), a.S);
  const int32_t* table = a.pm.table + b * a.pm.table_stride;
  const int place0 = base / kBlock, before = base % kBlock;
  const bool has0 = place0 < a.pm.max_pages;
  const int page0 = sums && has0 ? get(table + place0) : -1;
  const int page1 = sums && place0 + 1 < a.pm.max_pages ? get(table + place0 + 1) : -1;
  if (tid < SA_TREE_MAX) {
    const bool good = tid < m && at > prev && at < SA_TREE_MAX && at < a.pm.max_pages * kBlock - base;
    if (good) {
      const int from = get(table + (base + at) / kBlock), to = get(table + (base + tid) / kBlock);
      const bool has_from = from >= 0 && from < a.pm.n_pages, has_to = to >= 0 && to < a.pm.n_pages;
      if (!has_from || !has_to) status |= SA_DEV_BAD_CACHE;
      sm_to[tid] = has_to ? static_cast<int64_t>(to) * kBlock + (base + tid) % kBlock : -1;
      // without a source the place keeps what it holds
      sm_from[tid] = has_from ? static_cast<int64_t>(from) * kBlock + (base + at) % kBlock : sm_to[tid];
    }
    const uint32_t all = __ballot_sync(0xffffffffu, good);
    if (tid % 32 == 0) sm_good[tid / 32] = all;
  }
  __syncthreads();
  const uint64_t good = static_cast<uint64_t>(sm_good[1]) << 32 | sm_good[0];
  const int count = good == ~0ull ? SA_TREE_MAX : __ffsll(~good) - 1;     // as far as the path holds
  if (count < m) status |= SA_DEV_BAD_TREE;
  const int end = base + count;
  const int piece = tid % kP, grp = tid / kP;
  char* cache = (keys ? a.kc : a.vc) + h * (keys ? a.kcs[1] : a.vcs[1]) + piece * 16;
  const int64_t s_page = keys ? a.kcs[0] : a.vcs[0], s_tok = keys ? a.kcs[2] : a.vcs[2];
  auto address = [&](int64_t place) { return reinterpret_cast<uint4*>(cache + place / kBlock * s_page + place % kBlock * s_tok); };
  // pages whose sums are renewed
  const bool sum0 = sums && (before > 0 || count > 0) && has0, sum1 = sums && end > (place0 + 1) * kBlock;
  const bool there0 = sum0 && page0 >= 0 && page0 < a.pm.n_pages, there1 = sum1 && page1 >= 0 && page1 < a.pm.n_pages;
  if ((sum0 && !there0) || (sum1 && !there1)) status |= SA_DEV_BAD_CACHE;
  uint4 w[kPasses], old[kPasses];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int i = u * kRows + grp;
    w[u] = old[u] = make_uint4(0u, 0u, 0u, 0u);
    if (i < count && sm_to[i] >= 0 && (sums || sm_from[i] != sm_to[i])) w[u] = *address(sm_from[i]);
    if (there0 && i < before) old[u] = *address(static_cast<int64_t>(page0) * kBlock + i);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int i = u * kRows + grp;
    if (i < count && sm_to[i] >= 0 && sm_from[i] != sm_to[i]) *address(sm_to[i]) = w[u];
  }
  if (a.lens_out && h == 0 && keys && tid == 0) a.lens_out[b] = end;
  if (there0 || there1) {
    float s[2][kElts] = {};
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      add_values<kFp8>(old[u], s[0]);
      if (before + u * kRows + grp < kBlock)       // tokens that do not count are zeros
        add_values<kFp8>(w[u], s[0]);
      else
        add_values<kFp8>(w[u], s[1]);
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (x == 1 && !there1) break;
#pragma unroll
      for (int i = 0; i < kElts; ++i) {
#pragma unroll
        for (int off = kP; off < 32; off <<= 1) s[x][i] += __shfl_xor_sync(0xffffffffu, s[x][i], off);
        if (tid % 32 < kP) sm_sum[x][tid / 32][piece * kElts + i] = s[x][i];
      }
    }
    __syncthreads();
    const float scale = kFp8 && a.k_scale ? get(a.k_scale + h) : 1.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (!(x == 0 ? there0 : there1) || tid >= D) continue;
      float all = 0.f;
#pragma unroll
      for (int g = 0; g < kAcceptThreads / 32; ++g) all += sm_sum[x][g][tid];
      a.k_sum[(static_cast<int64_t>(x == 0 ? page0 : page1) * a.Hkv + h) * D + tid] = all * scale;
    }
  }
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
  return launch_close(copy_kernel, dim3(grid), kCopyThreads, 0, st, a, log_pieces, slices);
}

}  // namespace sa
