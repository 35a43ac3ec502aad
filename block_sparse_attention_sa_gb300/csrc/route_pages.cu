// route_pages.cu -- the pages one new token attends: per (sequence, key-value
// head) the forced pages and those of largest pooled score within a budget.
#include "cache_internal.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;

// Entries of every row of a sequence of n tokens, and how many are forced.
__device__ __forceinline__ void row_counts(int n, int prefix, int budget, int* nb, int* sink,
                                           int* keep) {
  *nb = (n + kBlock - 1) / kBlock;
  *sink = (min(prefix, n) + kBlock - 1) / kBlock;
  const int forced = *nb == 0 ? 0 : (*sink == *nb ? *nb : *sink + 1);
  *keep = max(forced, min(*nb, budget));
}

__device__ int block_sum(int v, int* buf) {
  __syncthreads();
  buf[threadIdx.x] = v;
  __syncthreads();
  for (int off = kThreads / 2; off; off >>= 1) {
    if (static_cast<int>(threadIdx.x) < off) buf[threadIdx.x] += buf[threadIdx.x + off];
    __syncthreads();
  }
  return buf[0];
}

// grid (B * Hkv): fp64 scores, then the rank of every free page by counting.
__global__ void __launch_bounds__(kThreads) route_pages_kernel(RoutePagesArgs a) {
  __shared__ int buf[kThreads];
  const int row = blockIdx.x, b = row / a.Hkv, g = row % a.Hkv, G = a.H / a.Hkv;
  double* score = reinterpret_cast<double*>(a.ws) + static_cast<int64_t>(row) * a.pm.max_pages;
  bool bad;
  int nb, sink, keep, status = 0, before = 0;
  for (int i = threadIdx.x; i < b; i += kThreads) {
    row_counts(clamp_len(a.pm.seq_lens[i], a.pm, &bad), a.prefix, a.budget, &nb, &sink, &keep);
    before += keep;
  }
  const int start_b = block_sum(before, buf) * a.Hkv;
  const int n = clamp_len(a.pm.seq_lens[b], a.pm, &bad);
  if (bad) status |= SA_DEV_BAD_CACHE;
  row_counts(n, a.prefix, a.budget, &nb, &sink, &keep);
  const int start = start_b + g * keep;
  if (threadIdx.x == 0) {
    a.row_ptr[row] = start;
    if (row == a.B * a.Hkv - 1) a.row_ptr[row + 1] = start + keep;
    if (start + keep > a.col_cap) status |= SA_DEV_CAPACITY;
  }
  for (int j = threadIdx.x; j < nb; j += kThreads) {
    const int page = a.pm.table[b * a.pm.table_stride + j];
    double best = -INFINITY;
    if (page < 0 || page >= a.pm.n_pages) {
      status |= SA_DEV_BAD_CACHE;
    } else {
      const float* ks = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + g) * a.D;
      for (int h = 0; h < G; ++h) {
        const uint16_t* q = a.q + b * a.qs[0] + (g * G + h) * a.qs[2];
        double s = 0.0;
        for (int d = 0; d < a.D; ++d)
          s = fma(static_cast<double>(__uint_as_float(static_cast<uint32_t>(q[d]) << 16)),
                  static_cast<double>(ks[d]), s);
        best = fmax(best, s);
      }
    }
    score[j] = best;
  }
  __syncthreads();
  const int want = keep - (sink < nb ? sink + 1 : nb);
  int at = start;
  for (int j0 = 0; j0 < nb; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    bool take = j < nb && (j < sink || j == nb - 1);
    if (j < nb && !take) {
      int rank = 0;
      for (int i = sink; i < nb - 1; ++i) rank += score[i] > score[j] || (score[i] == score[j] && i < j);
      take = rank < want;
    }
    buf[threadIdx.x] = take;
    __syncthreads();
    int pos = at, total = 0;
    for (int i = 0; i < kThreads; ++i) {
      if (i < static_cast<int>(threadIdx.x)) pos += buf[i];
      total += buf[i];
    }
    if (take && pos < a.col_cap) a.col_idx[pos] = j;
    at += total;
    __syncthreads();
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace

size_t route_pages_ws_bytes(int64_t rows, int max_pages) {
  return static_cast<size_t>(rows) * max_pages * sizeof(double);
}

cudaError_t launch_route_pages(const RoutePagesArgs& a, cudaStream_t st) {
  route_pages_kernel<<<a.B * a.Hkv, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
