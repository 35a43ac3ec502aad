// pages.cu -- page tables and reference counts of a pool: forking, resizing and
// compacting. Only numbers move here; copy.cu moves what the pages hold.
//
// Each call is one launch of one cluster of eight CTAs, which meets at the cluster's
// barrier between its steps (0.5 us each, where another kernel costs 2 us). The work is
// a few integers a page: what counts is how few dependent steps there are. Pages that
// are free are found by ballot, a warp for a run of pages; a warp's place in the order
// comes from the counts of all 256 warps, which each warp leaves in every CTA's shared
// memory before the barrier. So ids come out in ascending order, the same every time,
// without a list of free pages that would have to be kept in step with refs.
//
// Bound by the chain of dependent steps. In a graph, four sequences of 777 tokens (256 of
// up to 2,048): fork 6.2 us (7.6), resize 3.3 (4.3); compact 4.1 us for a pool of 128
// pages, 7.2 for one of 6,144. Fork, resize and the copy called one by one on an idle GPU:
// 12 us (22), 20.5 (31) with every launch behind the end of the one before.
#include "cache_internal.cuh"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kMostRows = 16384;    // sequences of a table (check_pages)
constexpr int kCtas = 8;            // the largest cluster that every part runs
constexpr int kThreads = 1024;
constexpr int kWarps = kCtas * kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ int cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// Every thread of the cluster meets, and what each wrote is seen by all.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The cluster's CTAs are placed together, but need not have begun together, and the shared
// memory of one may be touched only once it runs. So each says first of all that it does, and
// sums_of waits for all to have said so: behind the loads and the counting, where they long have.
__device__ __forceinline__ void cluster_begun() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_begun() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What other CTAs of this launch have written: from L2, past this SM's L1.
__device__ __forceinline__ int fresh(const int32_t* p) { return __ldcg(p); }

struct Counts {
  int2 of[kWarps];                  // two counts of every warp of the cluster
};

// The sums of two counts over the warps before this one (first) and over all (second).
// Meets the cluster once, behind cluster_begun().
struct Sums {
  int2 before, all;
};
__device__ __forceinline__ Sums sums_of(Counts& c, int warp, int lane, int x, int y) {
  cluster_wait_begun();
  if (lane < kCtas) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(&c.of[warp])), "r"(lane));
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(x), "r"(y) : "memory");
  }
  cluster_sync();
  int2 before{0, 0}, all{0, 0};
#pragma unroll
  for (int i = 0; i < kWarps / 32; ++i) {
    const int w = i * 32 + lane;
    const int2 v = c.of[w];
    all.x += v.x;
    all.y += v.y;
    before.x += w < warp ? v.x : 0;
    before.y += w < warp ? v.y : 0;
  }
  Sums s;
  s.before.x = __reduce_add_sync(kFull, before.x);
  s.before.y = __reduce_add_sync(kFull, before.y);
  s.all.x = __reduce_add_sync(kFull, all.x);
  s.all.y = __reduce_add_sync(kFull, all.y);
  return s;
}

// A warp's run of n items, in whole groups of 32.
struct Part {
  int lo, hi;
};
__device__ __forceinline__ Part part_of(int n, int warp) {
  const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int64_t lo = static_cast<int64_t>(per) * warp;
  return {static_cast<int>(min(lo, static_cast<int64_t>(n))),
          static_cast<int>(min(lo + per, static_cast<int64_t>(n)))};
}

// A warp's run of n rows, which it walks one by one.
__device__ __forceinline__ Part rows_of(int n, int warp) {
  const int per = (n + kWarps - 1) / kWarps;
  return {min(per * warp, n), min(per * warp + per, n)};
}

__device__ __forceinline__ int below(unsigned mask, int lane) { return __popc(mask & ((1u << lane) - 1)); }

// The free pages of a warp's part: how many.
__device__ __forceinline__ int count_free(const PagesArgs& a, Part p, int lane) {
  int n = 0;
#pragma unroll 4
  for (int i = p.lo; i < p.hi; i += 32) {
    const bool is = i + lane < p.hi && a.refs[i + lane] <= 0;
    n += __popc(__ballot_sync(kFull, is));
  }
  return n;
}

// And their ids into list, from place `at` on, as far as `most`.
__device__ __forceinline__ void list_free(const PagesArgs& a, Part p, int lane, int at, int most, int32_t* list) {
#pragma unroll 4
  for (int i = p.lo; i < p.hi; i += 32) {
    if (at >= most) break;
    const bool is = i + lane < p.hi && a.refs[i + lane] <= 0;
    const unsigned m = __ballot_sync(kFull, is);
    const int k = at + below(m, lane);
    if (is && k < most) list[k] = i + lane;
    at += __popc(m);
  }
}

// An entry of the table, -1 if it names no page.
__device__ __forceinline__ int page_at(const PagesArgs& a, int e, int* status) {
  if (e >= 0 && e < a.n_pages) return e;
  if (e != -1) *status |= SA_DEV_BAD_CACHE;
  return -1;
}

__device__ __forceinline__ int length_of(const PagesArgs& a, int b, int* status) {
  const int n = a.lens[b], most = a.max_pages * kBlock;      // max_pages < 2^25
  if (n >= 0 && n <= most) return n;
  *status |= SA_DEV_BAD_CACHE;
  return n < 0 ? 0 : most;
}

__device__ __forceinline__ int source_of(const PagesArgs& a, int i, int* status) {
  const int s = a.src[i];
  if (s >= 0 && s < a.B) return s;
  if (s != -1) *status |= SA_DEV_BAD_TREE;
  return -1;
}

__device__ __forceinline__ void report(const PagesArgs& a, int status) {
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// ---------------------------------------------------------------- fork --

// Every CTA counts for itself, in shared memory, who continues whom: two meetings of the
// cluster less than with counts in global memory (8.2 us a call, four beams).
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) pages_fork_kernel(PagesArgs a) {
  cluster_begun();
  let_next_launch();
  wait_for_first();
  __shared__ Counts counts;
  extern __shared__ int32_t of_old[];   // [B] the first that continues it, [B] how many do
  int32_t *first = of_old, *takers = first + a.B;
  const int t = cta_rank() * kThreads + threadIdx.x, warp = t >> 5, lane = t & 31;
  int32_t *copy = a.ws, *list = copy + a.N;   // which copy a new sequence gets; the copies' pages
  int status = 0;
  for (int b = threadIdx.x; b < a.B; b += kThreads) {
    first[b] = a.N;
    takers[b] = 0;
  }
  if (a.refs_out != a.refs)
    for (int p = t; p < a.n_pages; p += kCtas * kThreads) a.refs_out[p] = a.refs[p];
  const Part rows = part_of(a.N, warp), pages = part_of(a.n_pages, warp);
  const int free_pages = count_free(a, pages, lane);
  __syncthreads();
  for (int i = threadIdx.x; i < a.N; i += kThreads) {
    const int s = source_of(a, i, &status);
    if (s < 0) continue;
    atomicMin(first + s, i);
    atomicAdd(takers + s, 1);
  }
  __syncthreads();
  // the new sequences that need a copy, in order, and the free pages
  auto needs_copy = [&](int i) {
    if (i >= rows.hi) return false;
    const int s = source_of(a, i, &status);
    if (s < 0 || first[s] == i) return false;
    const int n = length_of(a, s, &status);
    return n % kBlock > 0 && page_at(a, a.table[s * a.stride + n / kBlock], &status) >= 0;
  };
  int need = 0;
  for (int i = rows.lo; i < rows.hi; i += 32) need += __popc(__ballot_sync(kFull, needs_copy(i + lane)));
  const Sums sum = sums_of(counts, warp, lane, need, free_pages);
  list_free(a, pages, lane, sum.before.y, min(sum.all.x, sum.all.y), list);
  int k = sum.before.x;
  for (int i = rows.lo; i < rows.hi; i += 32) {
    const bool is = needs_copy(i + lane);
    const unsigned m = __ballot_sync(kFull, is);
    if (i + lane < rows.hi) copy[i + lane] = is ? k + below(m, lane) : -1;
    k += __popc(m);
  }
  if (t == 0) a.n_moves[0] = min(sum.all.x, sum.all.y);
  cluster_sync();
  // new rows
  for (int i = warp; i < a.N; i += kWarps) {
    const int c = fresh(copy + i), s = source_of(a, i, &status);
    const int n = s < 0 ? 0 : length_of(a, s, &status), whole = n / kBlock;
    const bool again = s >= 0 && first[s] != i;
    int page = -1, end = n;
    if (c >= 0) {
      if (c < sum.all.y) {
        page = fresh(list + c);
        if (lane == 0) {
          a.moves[2 * c] = a.table[s * a.stride + whole];
          a.moves[2 * c + 1] = page;
          a.refs_out[page] = 1;
        }
      } else {                       // no page is free: the full ones only
        end = whole * kBlock;
        status |= SA_DEV_CAPACITY;
      }
    }
    if (lane == 0) a.lens_out[i] = end;
#pragma unroll 4
    for (int j = lane; j < a.max_pages; j += 32) {
      int e = s < 0 ? -1 : page_at(a, a.table[s * a.stride + j], &status);
      if (again && j >= whole) e = j == whole ? page : -1;
      a.table_out[i * a.out_stride + j] = e;
    }
  }
  // the old rows' places, less those that were taken over
  for (int b = warp; b < a.B; b += kWarps) {
    const int n = takers[b];
    if (n == 1) continue;
    const int whole = length_of(a, b, &status) / kBlock;
#pragma unroll 4
    for (int j = lane; j < a.max_pages; j += 32) {
      const int e = page_at(a, a.table[b * a.stride + j], &status);
      const int more = n == 0 ? -1 : (j < whole ? n - 1 : 0);
      if (e >= 0 && more != 0) atomicAdd(a.refs_out + e, more);
    }
  }
  report(a, status);
}

// -------------------------------------------------------------- resize --

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) pages_resize_kernel(PagesArgs a) {
  cluster_begun();
  let_next_launch();
  wait_for_first();
  __shared__ Counts counts;
  const int t = cta_rank() * kThreads + threadIdx.x, warp = t >> 5, lane = t & 31;
  int status = 0;
  // the pages sequence b shall hold
  auto wanted = [&](int b) {
    const int64_t n = static_cast<int64_t>(a.lens[b]) + (a.more_lens ? a.more_lens[b] : a.more);
    if (n < 0) {
      status |= SA_DEV_BAD_CACHE;
      return 0;
    }
    const int64_t w = (n + kBlock - 1) / kBlock;
    if (w > a.max_pages) status |= SA_DEV_CAPACITY;
    return static_cast<int>(min(w, static_cast<int64_t>(a.max_pages)));
  };
  const Part rows = rows_of(a.B, warp), pages = part_of(a.n_pages, warp);
  int need = 0;
  for (int b = rows.lo; b < rows.hi; ++b) {
    const int want = wanted(b);
#pragma unroll 4
    for (int j = 0; j < want; j += 32) {
      const bool is = j + lane < want && page_at(a, a.table[b * a.stride + j + lane], &status) < 0;
      need += __popc(__ballot_sync(kFull, is));
    }
  }
  const Sums sum = sums_of(counts, warp, lane, need, count_free(a, pages, lane));
  list_free(a, pages, lane, sum.before.y, min(sum.all.x, sum.all.y), a.ws);
  cluster_sync();
  int k = sum.before.x;
  for (int b = rows.lo; b < rows.hi; ++b) {
    const int want = wanted(b);
    int32_t* row = a.table_out + b * a.out_stride;
#pragma unroll 4
    for (int j = 0; j < a.max_pages; j += 32) {
      const int at = j + lane, e = at < a.max_pages ? row[at] : -1;
      const bool has = e >= 0 && e < a.n_pages, missing = at < want && !has;
      const unsigned m = __ballot_sync(kFull, missing);
      if (missing) {
        const int c = k + below(m, lane), page = c < sum.all.y ? fresh(a.ws + c) : -1;
        if (page >= 0)
          a.refs_out[page] = 1;
        else
          status |= SA_DEV_CAPACITY;
        if (page != e) row[at] = page;
      } else if (at >= want && at < a.max_pages && e != -1) {
        if (has)
          atomicSub(a.refs_out + e, 1);
        else
          status |= SA_DEV_BAD_CACHE;
        row[at] = -1;
      }
      k += __popc(m);
    }
  }
  report(a, status);
}

// ------------------------------------------------------------- compact --

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) pages_compact_kernel(PagesArgs a) {
  cluster_begun();
  let_next_launch();
  wait_for_first();
  __shared__ Counts counts;
  const int t = cta_rank() * kThreads + threadIdx.x, warp = t >> 5, lane = t & 31;
  // a page's id afterwards (of one from n_used on, which is found by its place among those:
  // -1 - that, from the end); the free pages before n_used, ascending; the pages from n_used
  // on, descending; how many those are
  int32_t *now = a.ws, *hole = now + a.n_pages, *late = hole + a.n_pages, *n_late = late + a.n_pages;
  int status = 0;
  const Part pages = part_of(a.n_pages, warp);
  int n = 0;
#pragma unroll 4
  for (int i = pages.lo; i < pages.hi; i += 32) {
    const bool is = i + lane < pages.hi && a.refs[i + lane] > 0;
    n += __popc(__ballot_sync(kFull, is));
  }
  const Sums sum = sums_of(counts, warp, lane, n, 0);
  const int used = sum.all.x;
  int before = sum.before.x;          // pages in use before the warp's next 32
#pragma unroll 4
  for (int i = pages.lo; i < pages.hi; i += 32) {
    const int p = i + lane;
    const bool in = p < pages.hi;
    const int r = in ? a.refs[p] : 0;
    const unsigned m = __ballot_sync(kFull, r > 0);
    const int rank = before + below(m, lane);
    if (in) {
      const bool moves = p >= used && r > 0;
      now[p] = moves ? -1 - (used - 1 - rank) : p;
      if (p < used && r <= 0) hole[p - rank] = p;
      if (moves) late[used - 1 - rank] = p;
      if (p == used) n_late[0] = used - rank;
      if (a.refs_out != a.refs) a.refs_out[p] = r;
    }
    before += __popc(m);
  }
  if (used == a.n_pages && t == 0) n_late[0] = 0;
  cluster_sync();
  const int moved = fresh(n_late);
  for (int k = t; k < moved; k += kCtas * kThreads) {
    const int from = fresh(late + moved - 1 - k), to = fresh(hole + k);
    a.moves[2 * k] = from;
    a.moves[2 * k + 1] = to;
    a.refs_out[to] = a.refs[from];
    a.refs_out[from] = 0;
  }
  if (t == 0) {
    a.n_moves[0] = moved;
    a.n_used[0] = used;
  }
  for (int b = warp; b < a.B; b += kWarps)
#pragma unroll 4
    for (int j = lane; j < a.max_pages; j += 32) {
      const int e = page_at(a, a.table[b * a.stride + j], &status);
      int to = e < 0 ? -1 : fresh(now + e);
      if (e >= 0 && to < 0) to = fresh(hole + moved + to);       // hole[moved - 1 - place]
      a.table_out[b * a.out_stride + j] = to;
    }
  report(a, status);
}

// Launched while the kernel before still runs where that allows it (these do, and
// sa_cache_copy's): the steps of a fork come one behind the other, 8 of 152 SMs busy.
cudaError_t launch(void (*kernel)(PagesArgs), const PagesArgs& a, size_t smem, cudaStream_t st) {
  return launch_close(kernel, dim3(kCtas), kThreads, smem, st, a);
}

}  // namespace

size_t pages_ws_bytes(int n_pages, int rows) {
  // fork: a copy's number for each row and a list as long; resize: a list of pages;
  // compact: three
  return (2 * static_cast<size_t>(rows) + 3 * static_cast<size_t>(n_pages) + 64) * sizeof(int32_t);
}

cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t st) {
  // for the most rows, whatever this call has: the limit is the kernel's, for all threads of
  // the host, and a smaller one could come between another's and its launch
  constexpr int kMostSmem = 2 * kMostRows * sizeof(int32_t);
  static_assert(kMostSmem + sizeof(Counts) <= 227 * 1024, "counts do not fit shared memory");
  const size_t smem = 2 * static_cast<size_t>(a.B) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(pages_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
  }
  return launch(pages_fork_kernel, a, smem, st);
}
cudaError_t launch_pages_resize(const PagesArgs& a, cudaStream_t st) { return launch(pages_resize_kernel, a, 0, st); }
cudaError_t launch_pages_compact(const PagesArgs& a, cudaStream_t st) { return launch(pages_compact_kernel, a, 0, st); }

}  // namespace sa
