// route_pages.cu -- the pages one new token attends: per (sequence, key-value
// head) the forced pages and those of largest pooled score within a budget.
//   s_j = max over the head group of q_h . k_sum_j
//
// score_kernel reads every key sum once (4 D bytes a page and head, 1/64 of what
// the page's keys and values take in bf16) and is bound by that. Eight pages and
// up to 16 query heads are one tile of mma.m16n8k16: the fp32 sums go in as two
// bf16 terms, so the products are right to 2^-18, and the tensor cores leave the
// loads alone. Tiles are cut into equal runs, one per CTA, whatever the lengths.
//
// select_kernel, one CTA per row, finds the score that the budget ends at by
// bisection. An order statistic moves by no more than the values do, so a page
// whose score is more than twice the error bound above or below that score is
// decided; the few in between (usually the last page alone) are computed again
// in fp64 and ranked. Rows with scores that are not finite are ranked in fp64
// whole.
//
// Error of a score against fp64, over sum_d |q_d k_d| <= |q| |k|: 2^-18 from the
// two terms, and 2 D / 16 tensor-core steps that each add 16 products to the sum
// with less than 2^-22 of it lost: below 2^-17.9 + 2^-18. kErr doubles that.
#include <cuda_bf16.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 8;               // pages of a score tile
constexpr int kScoreCtas = 2 * 152;    // two CTAs on each SM
constexpr float kErr = 1.f / 32768.f;  // 2^-15
constexpr int kItems = 8;              // pages a thread of select_kernel holds at once
constexpr int kSpan = kThreads * kItems;
constexpr int kNear = 256;             // undecided pages ranked in shared memory
constexpr unsigned kFull = 0xffffffffu;

// Workspace: scores, per tile the largest error bound, fp64 scores of pages
// that are ranked exactly where they are more than kNear.
struct Layout {
  size_t score, err, exact, total;
};

__host__ __device__ inline Layout layout(int64_t rows, int max_pages) {
  const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t n = static_cast<size_t>(rows) * max_pages;
  const size_t tiles = static_cast<size_t>(rows) * ((max_pages + kTile - 1) / kTile);
  Layout l{};
  l.err = up(n * sizeof(float));
  l.exact = l.err + up(tiles * sizeof(float));
  l.total = l.exact + up(n * sizeof(double));
  return l;
}

// Pages of a sequence of n tokens, how many of them are sink pages, and how
// many every row of it keeps.
__device__ __forceinline__ void row_counts(int n, int prefix, int budget, int* nb, int* sink,
                                           int* keep) {
  *nb = (n + kBlock - 1) / kBlock;
  *sink = (min(prefix, n) + kBlock - 1) / kBlock;
  const int forced = *sink == *nb ? *nb : *sink + 1;
  *keep = max(forced, min(*nb, budget));
}

__device__ __forceinline__ float bits_f32(uint32_t b) { return __uint_as_float(b << 16); }

// A squared norm, infinite where the products it bounds might overflow or are
// no numbers.
__device__ __forceinline__ float capped(float n2) { return n2 < 1e38f ? n2 : INFINITY; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
               "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 query heads from h0 on as A fragments (heads beyond the group zero) and
// their largest squared norm, in every lane. The 16 dims of a step are taken in
// the order the key sums' 16-byte loads give: lane quad c holds 4c .. 4c + 3.
template <int D>
__device__ __forceinline__ float load_heads(const RoutePagesArgs& a, int b, int g, int G, int h0,
                                            int lane, uint32_t qa[D / 16][4]) {
  const int r = lane >> 2, c = lane & 3;
  float norm = 0.f;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const bool there = h0 + r + 8 * x < G;
    const uint16_t* q = a.q + b * a.qs[0] + (g * G + (there ? h0 + r + 8 * x : 0)) * a.qs[2];
    float n2 = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint2 w = there ? __ldg(reinterpret_cast<const uint2*>(q + 16 * k + 4 * c))
                            : make_uint2(0u, 0u);
      qa[k][x] = w.x;
      qa[k][2 + x] = w.y;
      const float f[4] = {bits_f32(w.x), __uint_as_float(w.x & 0xffff0000u), bits_f32(w.y),
                          __uint_as_float(w.y & 0xffff0000u)};
#pragma unroll
      for (int i = 0; i < 4; ++i) n2 = fmaf(f[i], f[i], n2);
    }
    n2 += __shfl_xor_sync(kFull, n2, 1);
    n2 += __shfl_xor_sync(kFull, n2, 2);
    norm = fmaxf(norm, capped(n2));
  }
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1) norm = fmaxf(norm, __shfl_xor_sync(kFull, norm, off));
  return norm;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(RoutePagesArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.H / a.Hkv;
  const Layout L = layout(static_cast<int64_t>(a.B) * a.Hkv, a.pm.max_pages);
  float* score = reinterpret_cast<float*>(a.ws);
  float* err = reinterpret_cast<float*>(a.ws + L.err);
  const int row_tiles = (a.pm.max_pages + kTile - 1) / kTile;
  int status = 0;
  auto pages = [&](int b) {
    bool bad;
    const int n = clamp_len(__ldg(a.pm.seq_lens + b), a.pm, &bad);
    if (bad) status |= SA_DEV_BAD_CACHE;
    return (n + kBlock - 1) / kBlock;
  };
  auto tiles = [&](int b) { return static_cast<int64_t>((pages(b) + kTile - 1) / kTile); };
  const Run run = plan_run<kThreads>(a.B, a.Hkv, tiles);
  // the CTA's run, a consecutive part of it for each warp
  const int64_t n_cta = run.hi - run.lo;
  int64_t left = n_cta * (warp + 1) / kWarps - n_cta * warp / kWarps;
  if (left > 0) {
    int b = run.group;
    int64_t off = run.off + n_cta * warp / kWarps;
    uint32_t qa[D / 16][4];
    float q2 = 0.f;
    int have = -1;                           // the row whose queries are loaded
    while (left > 0 && b < a.B) {
      const int nb = pages(b), cnt = (nb + kTile - 1) / kTile;
      if (off >= static_cast<int64_t>(cnt) * a.Hkv) {
        off -= static_cast<int64_t>(cnt) * a.Hkv;
        ++b;
        continue;
      }
      const int g = static_cast<int>(off / cnt);
      int tile = static_cast<int>(off % cnt);
      const int take = static_cast<int>(min(left, static_cast<int64_t>(cnt - tile)));
      const int64_t row = static_cast<int64_t>(b) * a.Hkv + g;
      auto page_at = [&](int t) {            // lane: page lane / 4 of tile t
        const int j = t * kTile + (lane >> 2);
        if (j >= nb) return -1;
        const int page = __ldg(a.pm.table + b * a.pm.table_stride + j);
        if (page >= 0 && page < a.pm.n_pages) return page;
        status |= SA_DEV_BAD_CACHE;
        return -1;
      };
      int page = page_at(tile);
      for (int i = 0; i < take; ++i, ++tile) {
        float4 w[D / 16];
        const float* src = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + g) * D + 4 * (lane & 3);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          w[k] = page >= 0 ? __ldg(reinterpret_cast<const float4*>(src + 16 * k))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        const bool known = page >= 0;
        if (i + 1 < take) page = page_at(tile + 1);
        if (have != row && G <= 16) {
          q2 = load_heads<D>(a, b, g, G, 0, lane, qa);
          have = static_cast<int>(row);
        }
        // lane's scores: pages 2 (lane % 4) + {0, 1}, heads lane / 4 and + 8
        float best[2] = {-INFINITY, -INFINITY};
        for (int h0 = 0; h0 < G; h0 += 16) {
          if (G > 16) {
            const float n2 = load_heads<D>(a, b, g, G, h0, lane, qa);
            q2 = h0 == 0 ? n2 : fmaxf(q2, n2);
          }
          float c[4] = {};
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t hi0 = pack_bf16(w[k].x, w[k].y), hi1 = pack_bf16(w[k].z, w[k].w);
            const uint32_t lo0 = pack_bf16(w[k].x - bits_f32(hi0), w[k].y - __uint_as_float(hi0 & 0xffff0000u));
            const uint32_t lo1 = pack_bf16(w[k].z - bits_f32(hi1), w[k].w - __uint_as_float(hi1 & 0xffff0000u));
            mma(c, qa[k], hi0, hi1);
            mma(c, qa[k], lo0, lo1);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)        // fmaxf passes over NaN
            if (h0 + (lane >> 2) + 8 * (x >> 1) < G) best[x & 1] = fmaxf(best[x & 1], c[x]);
        }
        float k2 = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          k2 = fmaf(w[k].x, w[k].x, k2);
          k2 = fmaf(w[k].y, w[k].y, k2);
          k2 = fmaf(w[k].z, w[k].z, k2);
          k2 = fmaf(w[k].w, w[k].w, k2);
        }
        k2 += __shfl_xor_sync(kFull, k2, 1);
        k2 = capped(k2 + __shfl_xor_sync(kFull, k2, 2));
#pragma unroll
        for (int off4 = 4; off4 <= 16; off4 <<= 1) {
          best[0] = fmaxf(best[0], __shfl_xor_sync(kFull, best[0], off4));
          best[1] = fmaxf(best[1], __shfl_xor_sync(kFull, best[1], off4));
          k2 = fmaxf(k2, __shfl_xor_sync(kFull, k2, off4));
        }
        const unsigned ok = __ballot_sync(kFull, known);
        if (lane < 4) {
          float* to = score + row * a.pm.max_pages + tile * kTile + 2 * lane;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (tile * kTile + 2 * lane + x < nb)
              to[x] = (ok >> (4 * (2 * lane + x))) & 1u ? best[x] : -INFINITY;
        }
        if (lane == 0) err[row * row_tiles + tile] = kErr * sqrtf(q2) * sqrtf(k2);
      }
      off += take;
      left -= take;
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// Sum (or largest) of one value per thread, in every thread. `buf` holds two
// sets of kWarps entries that alternate by `turn`, so one barrier does.
__device__ __forceinline__ int block_sum(int v, int* buf, int turn) {
  v = __reduce_add_sync(kFull, v);
  int* set = buf + (turn & 1) * kWarps;
  if ((threadIdx.x & 31) == 0) set[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += set[w];
  return s;
}

// fp64 score of one page by a whole warp; NaN heads are passed over.
__device__ double exact_score(const RoutePagesArgs& a, int b, int g, int j, int lane) {
  const int page = __ldg(a.pm.table + b * a.pm.table_stride + j), G = a.H / a.Hkv;
  if (page < 0 || page >= a.pm.n_pages) return -INFINITY;
  const float* k = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + g) * a.D;
  double best = -INFINITY;
  for (int h = 0; h < G; ++h) {
    const uint16_t* q = a.q + b * a.qs[0] + static_cast<int64_t>(g * G + h) * a.qs[2];
    double s = 0.0;
    for (int d = lane; d < a.D; d += 32)
      s = fma(static_cast<double>(bits_f32(__ldg(q + d))), static_cast<double>(__ldg(k + d)), s);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
    best = fmax(best, s);
  }
  return best + 0.0;                         // -0 and +0 are equal
}

// Order-preserving integer of a double that is not NaN.
__device__ __forceinline__ uint64_t order64(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | (1ull << 63);
}

// grid (B * Hkv): one row.
__global__ void __launch_bounds__(kThreads) select_kernel(RoutePagesArgs a) {
  __shared__ int sums[2 * kWarps];
  __shared__ float ext[3][kWarps];
  __shared__ int near_j[kNear];
  __shared__ double near_s[kNear];
  __shared__ int near_n;
  __shared__ int warp_n[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv;
  const int row = blockIdx.x, b = row / a.Hkv, g = row % a.Hkv;
  int turn = 0, status = 0;
  bool bad;
  // the row's place in the list: counts follow from the lengths alone
  int nb, sink, keep, before = 0;
  for (int i = tid; i < b; i += kThreads) {
    row_counts(clamp_len(__ldg(a.pm.seq_lens + i), a.pm, &bad), a.prefix, a.budget, &nb, &sink, &keep);
    before += keep;
  }
  before = block_sum(before, sums, turn++);
  row_counts(clamp_len(__ldg(a.pm.seq_lens + b), a.pm, &bad), a.prefix, a.budget, &nb, &sink, &keep);
  const int start = before * a.Hkv + g * keep;
  if (tid == 0) {
    near_n = 0;
    a.row_ptr[row] = start;
    if (row == rows - 1) a.row_ptr[rows] = start + keep;
    if (start + keep > a.col_cap) status |= SA_DEV_CAPACITY;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const Layout L = layout(rows, a.pm.max_pages);
  const float* score = reinterpret_cast<const float*>(a.ws) + static_cast<int64_t>(row) * a.pm.max_pages;
  const int row_tiles = (a.pm.max_pages + kTile - 1) / kTile;
  const float* err = reinterpret_cast<const float*>(a.ws + L.err) + static_cast<int64_t>(row) * row_tiles;
  double* exact = reinterpret_cast<double*>(a.ws + L.exact) + static_cast<int64_t>(row) * a.pm.max_pages;
  const int f0 = min(sink, nb), f1 = max(f0, nb - 1);      // the pages that compete
  const int want = keep - (sink < nb ? sink + 1 : nb);
  // thread's pages of a span: span + 256 warp + 32 i + lane, so that a warp's
  // ballots are in the order of the pages
  float v[kItems];
  auto load = [&](int span) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int j = span + warp * 32 * kItems + 32 * i + lane;
      v[i] = j < f1 ? score[j] : -INFINITY;
    }
  };
  // A page scores above `above`: in; below `below`: out; else by its exact
  // score, largest first, against `edge` with `ties` of the equal ones in.
  float above = INFINITY, below = INFINITY;
  const bool all = want >= f1 - f0;
  int need = 0;                              // of the undecided ones
  bool by_list = false, by_exact = false;
  uint64_t edge = 0;
  int ties = 0;
  if (want > 0 && !all) {
    // extremes of the scores, and the error bound
    float lo = INFINITY, hi = -INFINITY, d = 0.f;
    for (int span = f0; span < f1; span += kSpan) {
      load(span);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        if (span + warp * 32 * kItems + 32 * i + lane >= f1) continue;
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
      }
    }
    for (int t = f0 / kTile + tid; t < (f1 + kTile - 1) / kTile; t += kThreads) d = fmaxf(d, err[t]);
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(kFull, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, off));
      d = fmaxf(d, __shfl_xor_sync(kFull, d, off));
    }
    if (lane == 0) {
      ext[0][warp] = lo;
      ext[1][warp] = hi;
      ext[2][warp] = d;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      lo = fminf(lo, ext[0][w]);
      hi = fmaxf(hi, ext[1][w]);
      d = fmaxf(d, ext[2][w]);
    }
    const bool finite = lo > -1e38f && hi < 1e38f && d < 1e30f;
    if (finite) {
      // the want-th largest score lies in [lo, hi]: at least want are >= lo,
      // fewer than want are > hi
      const bool held = f1 - f0 <= kSpan;    // v holds every page already
      while (hi - lo > d) {
        const float mid = 0.5f * lo + 0.5f * hi;
        if (!(mid > lo && mid < hi)) break;
        int n = 0;
        for (int span = f0; span < f1; span += kSpan) {
          if (!held) load(span);
#pragma unroll
          for (int i = 0; i < kItems; ++i) n += v[i] >= mid;
        }
        if (block_sum(n, sums, turn++) >= want) lo = mid;
        else hi = mid;
      }
      above = hi + 2.f * d;
      below = lo - 2.f * d;
    } else {
      below = -INFINITY;                     // none is decided
    }
    int in = 0, mine = 0;
    for (int span = f0; span < f1; span += kSpan) {
      load(span);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int j = span + warp * 32 * kItems + 32 * i + lane;
        if (j >= f1) continue;
        const bool yes = v[i] > above;
        in += yes;
        if (!yes && v[i] >= below) {
          ++mine;
          const int at = atomicAdd(&near_n, 1);
          if (at < kNear) near_j[at] = j;
        }
      }
    }
    in = block_sum(in, sums, turn++);
    const int n_near = block_sum(mine, sums, turn++);
    need = want - in;
    if (need < n_near) {
      if (n_near <= kNear) {
        by_list = true;
        for (int i = warp; i < n_near; i += kWarps) {
          const double s = exact_score(a, b, g, near_j[i], lane);
          if (lane == 0) near_s[i] = s;
        }
        __syncthreads();
        // a thread ranks one page; the pages that are out leave the list
        bool out = false;
        if (tid < n_near) {
          int rank = 0;
          for (int i = 0; i < n_near; ++i)
            rank += near_s[i] > near_s[tid] || (near_s[i] == near_s[tid] && near_j[i] < near_j[tid]);
          out = rank >= need;
        }
        __syncthreads();
        if (out) near_j[tid] = -1;
        __syncthreads();
        near_n = n_near;
      } else {
        by_exact = true;
        for (int span = f0; span < f1; span += 32 * kWarps) {
          // a warp's 32 pages, one after another
          const int j0 = span + warp * 32;
          for (int i = 0; i < 32 && j0 + i < f1; ++i) {
            const float s = score[j0 + i];
            if (s > above || !(s >= below)) continue;
            const double e = exact_score(a, b, g, j0 + i, lane);
            if (lane == 0) exact[j0 + i] = e;
          }
        }
        __syncthreads();
        // the need-th largest: the largest edge that `need` of them reach
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t mid = edge | (1ull << bit);
          int n = 0;
          for (int j = f0 + tid; j < f1; j += kThreads) {
            const float s = score[j];
            if (s <= above && s >= below) n += order64(exact[j]) >= mid;
          }
          if (block_sum(n, sums, turn++) >= need) edge = mid;
        }
        int over = 0;
        for (int j = f0 + tid; j < f1; j += kThreads) {
          const float s = score[j];
          if (s <= above && s >= below) over += order64(exact[j]) > edge;
        }
        ties = need - block_sum(over, sums, turn++);
      }
    }                                        // else every undecided page is in
  }

  // the list: sink pages, the chosen ones in order, the newest page
  for (int j = tid; j < f0; j += kThreads)
    if (start + j < a.col_cap) a.col_idx[start + j] = j;
  if (tid == 0 && f0 < nb && start + keep - 1 < a.col_cap) a.col_idx[start + keep - 1] = nb - 1;
  int at = start + f0, tied = 0;
  if (want > 0) {
    for (int span = f0; span < f1; span += kSpan) {
      load(span);
      unsigned take[kItems], equal[kItems];
      int n_take = 0, n_equal = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int j = span + warp * 32 * kItems + 32 * i + lane;
        bool t = false, q = false;
        if (j < f1) {
          if (all || v[i] > above) {
            t = true;
          } else if (v[i] >= below) {
            if (by_list) {
              for (int x = 0; x < near_n; ++x) t |= near_j[x] == j;
            } else if (by_exact) {
              const uint64_t e = order64(exact[j]);
              t = e > edge;
              q = e == edge;
            } else {
              t = true;
            }
          }
        }
        take[i] = __ballot_sync(kFull, t);
        equal[i] = __ballot_sync(kFull, q);
        n_take += __popc(take[i]);
        n_equal += __popc(equal[i]);
      }
      if (by_exact) {
        // of the equal ones the first `ties` are in
        if (lane == 0) warp_n[0][warp] = n_equal;
        __syncthreads();
        int rank = tied, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) rank += warp_n[0][w];
          total += warp_n[0][w];
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const bool q = (equal[i] >> lane) & 1u;
          const bool t = q && rank + __popc(equal[i] & ((1u << lane) - 1u)) < ties;
          const unsigned more = __ballot_sync(kFull, t);
          take[i] |= more;
          n_take += __popc(more);
          rank += __popc(equal[i]);
        }
        tied += total;
      }
      if (lane == 0) warp_n[1][warp] = n_take;
      __syncthreads();
      int to = at, total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) to += warp_n[1][w];
        total += warp_n[1][w];
      }
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int j = span + warp * 32 * kItems + 32 * i + lane;
        const int p = to + __popc(take[i] & ((1u << lane) - 1u));
        if (((take[i] >> lane) & 1u) && p < a.col_cap) a.col_idx[p] = j;
        to += __popc(take[i]);
      }
      at += total;
      __syncthreads();                       // warp_n is written again
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace

size_t route_pages_ws_bytes(int64_t rows, int max_pages) { return layout(rows, max_pages).total; }

cudaError_t launch_route_pages(const RoutePagesArgs& a, cudaStream_t st) {
  if (a.D == 64)
    score_kernel<64><<<kScoreCtas, kThreads, 0, st>>>(a);
  else
    score_kernel<128><<<kScoreCtas, kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // launched while the scores are made; it waits for them
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B * a.Hkv));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel, a);
}

}  // namespace sa
