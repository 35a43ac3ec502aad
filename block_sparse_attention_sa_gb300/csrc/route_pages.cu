// route_pages.cu -- the pages one new token attends: per (sequence, key-value
// head) the forced pages and those of largest pooled score within a budget.
//   s_j = max over the head group of q_h . k_sum_j
//
// score_kernel reads every key sum once (4 D bytes a page and head, 1/64 of what
// the page's keys and values take in bf16). Sixteen pages and eight query heads
// are one tile of mma.m16n8k16, the heads as its columns; the fp32 sums go in as
// two bf16 terms, so the products are right to 2^-17. Sums come into shared
// memory by bulk copies, two tiles ahead of each warp; tiles are cut into equal
// runs, one per CTA, whatever the lengths. Measured on GB300: 144 MB (32
// sequences of up to 112,640 tokens, 32/8 heads of 128) in 30 us, 63% of the
// DRAM rate, issue slots 42% busy with the splitting; 38 us with select_kernel.
//
// select_kernel, one CTA per row, narrows down the score that the budget ends at
// by histograms of 256 bins until a few dozen pages are left, and ranks those. An
// order statistic moves by no more than the values do, so a page whose score is
// more than twice the error bound above or below that score is decided; the few
// in between (usually the last page alone) are computed again in paired fp32, and
// those of them that this leaves within its own error of the edge in fp64.
// Rows with scores that are not finite or so small that fp32 loses their ends,
// and rows with very many undecided pages, are ranked in fp64. Latency bounds it:
// 11.6 us for 8 rows of 598 pages with both kernels.
//
// Error of a score against fp64, over sum_d |q_d k_d| <= |q|_1 max |k|: 2^-17
// from the two terms; and D / 16 tensor-core steps for each (the second 2^-8 of the
// first), which add 16 products and the running sum, each cut to 24 bits of the
// largest, a unit in the last place each: 17 2^-23 a step, 2^-15.9 at D = 128.
// Together below kErr = 2^-15.34. The second term loses its end where |k| is below
// 2^-110 or so (bf16 has nothing below 2^-133), so max |k| counts as 2^-100 at
// least, and |q|_1, unless it is 0, as 2^-40, so that the product is 0 for a row of
// zeros only.
#include <cuda_bf16.h>

#include "cache_internal.cuh"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 16;              // pages of a score tile
constexpr int kScoreWarps = 4;
static_assert((kScoreWarps & (kScoreWarps - 1)) == 0, "heads, a power of two, divide them");
constexpr int kScoreCtas = 3 * 152;    // three CTAs on each SM
constexpr int kAhead = 2;              // tiles a warp has in flight
constexpr float kErr = 0x1.94p-16f;
static_assert(kErr >= 0x1p-17 + 128 / 16 * 17 * 0x1p-23 * (1 + 0x1p-8) + 0x1p-24,
              "two terms, the steps of both, and their sum");
constexpr float kLeastK = 0x1p-100f, kLeastQ = 0x1p-40f;
// Below these the ends of products are lost in fp32: the error bound of a row,
// and |q|_1 max |k| of a page that is scored again.
constexpr float kLeastErr = 0x1p-90f, kLeastSize = 0x1p-60f;
constexpr int kItems = 8;              // pages a thread of select_kernel holds at once
constexpr int kSpan = kThreads * kItems;
constexpr int kNear = kThreads;        // undecided pages ranked in shared memory
constexpr int kFew = 48;               // pages that are ranked rather than counted once more
constexpr double kPairedErr = 0x1p-37;   // of a paired score, over the row's largest |q|_1 max |k|
constexpr unsigned kFull = 0xffffffffu;

// Workspace: per page its score and |q|_1 max |k| (what bounds the score's
// error; a score that is no number or infinite speaks for itself), and fp64
// scores where more than kNear pages are ranked exactly.
struct Layout {
  size_t score, err, exact, total;
};

__host__ __device__ inline Layout layout(int64_t rows, int max_pages) {
  const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t n = static_cast<size_t>(rows) * max_pages;
  Layout l{};
  l.err = up(n * sizeof(float));
  l.exact = l.err + up(n * sizeof(float));
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

// A sum of magnitudes, infinite where it is no number.
__device__ __forceinline__ float capped(float n) { return n < 1e38f ? n : INFINITY; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void mma(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
               "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// 8 query heads from h0 on as B fragments (heads beyond the group zero) and the
// largest of their sums of magnitudes, in every lane. The 16 dims of a step are
// taken in the order the key sums' 16-byte loads give: lane quad c holds 4c .. 4c + 3.
template <int D>
__device__ __forceinline__ float load_heads(const RoutePagesArgs& a, int b, int g, int G, int h0,
                                            int lane, uint2 qb[D / 16]) {
  const int h = h0 + (lane >> 2), c = lane & 3;
  const bool there = h < G;
  const uint16_t* q = a.q + b * a.qs[0] + (g * G + (there ? h : 0)) * a.qs[2];
  float n1 = 0.f;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    qb[k] = there ? get(reinterpret_cast<const uint2*>(q + 16 * k + 4 * c)) : make_uint2(0u, 0u);
    const float f[4] = {bits_f32(qb[k].x), __uint_as_float(qb[k].x & 0xffff0000u), bits_f32(qb[k].y),
                        __uint_as_float(qb[k].y & 0xffff0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) n1 += fabsf(f[i]);
  }
  n1 += __shfl_xor_sync(kFull, n1, 1);
  n1 = capped(n1 + __shfl_xor_sync(kFull, n1, 2));
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1) n1 = fmaxf(n1, __shfl_xor_sync(kFull, n1, off));
  return n1 > 0.f ? fmaxf(n1, kLeastQ) : 0.f;
}

// A place in the list of items: item `at` of `cnt` of head block `gb` of
// sequence b. An item is one tile for each warp of a CTA: `heads` warps take
// neighbouring heads of the same pages, which lie side by side in memory, the
// others the next tiles.
struct Cursor {
  int b, gb, at, cnt, nb;
};

// kOne: at most eight query heads share a key-value head, so their fragments
// stay in registers along a row.
template <int D, bool kOne>
__global__ void __launch_bounds__(32 * kScoreWarps, 3) score_kernel(RoutePagesArgs a, int heads) {
  constexpr int kSteps = D / 16;
  // Every warp has the next tiles on their way into its part of shared memory,
  // [warp][stage][page]: one bulk copy a page, rows 64 bytes further apart than
  // they are long, so that the two rows a quarter of a warp reads meet no bank twice.
  constexpr int kRow = D / 4 + 4;            // in 16-byte pieces
  extern __shared__ __align__(16) float4 ring[];
  __shared__ __align__(8) uint64_t full[kScoreWarps][kAhead];
  __shared__ volatile int abort_flag;
  let_next_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.H / a.Hkv;
  const Layout L = layout(static_cast<int64_t>(a.B) * a.Hkv, a.pm.max_pages);
  float* score = reinterpret_cast<float*>(a.ws);
  float* err = reinterpret_cast<float*>(a.ws + L.err);
  const int wide = kScoreWarps / heads * kTile;   // pages of an item
  const int blocks = a.Hkv / heads, wg = warp % heads, wt = warp / heads;
  float4* mine = ring + warp * kAhead * kTile * kRow;
  int status = 0;
  if (threadIdx.x == 0) {
    for (int w = 0; w < kScoreWarps; ++w)
      for (int s = 0; s < kAhead; ++s) mbar_init(smem_u32(&full[w][s]), 1);
    fence_barrier_init();
    abort_flag = 0;
  }
  auto pages = [&](int b) {
    bool bad;
    const int n = clamp_len(get(a.pm.seq_lens + b), a.pm, &bad);
    if (bad) status |= SA_DEV_BAD_CACHE;
    return (n + kBlock - 1) / kBlock;
  };
  const Run run = plan_run<32 * kScoreWarps>(
      a.B, blocks, [&](int b, int* nb) { return ((*nb = pages(b)) + wide - 1) / wide; });
  const int n_items = run.hi - run.lo;
  if (n_items > 0) {
    auto enter = [&](Cursor& c) {            // what follows from c.b
      c.nb = c.b < a.B ? pages(c.b) : 0;
      c.cnt = (c.nb + wide - 1) / wide;
    };
    auto step = [&](Cursor& c) {             // to the next item
      if (++c.at < c.cnt) return;
      c.at = 0;
      if (++c.gb < blocks) return;
      c.gb = 0;
      do {
        ++c.b;
        enter(c);
      } while (c.cnt == 0 && c.b < a.B);
    };
    Cursor now{run.group, 0, run.off, run.count, run.size};
    if (now.at >= now.cnt) {
      now.gb = run.off / now.cnt;
      now.at = run.off - now.gb * now.cnt;
    }
    auto first_page = [&](const Cursor& c) { return c.at * wide + wt * kTile; };
    auto page_at = [&](const Cursor& c) {    // lane: page lane % 16 of the warp's tile
      const int j = first_page(c) + (lane & 15);
      return j < c.nb ? get(a.pm.table + c.b * a.pm.table_stride + j) : -2;
    };
    // the tile's sums on their way; which of its pages are there, by bit
    auto fetch = [&](const Cursor& c, int page, int st) {
      const bool there = page >= 0 && page < a.pm.n_pages;
      if (!there && page != -2) status |= SA_DEV_BAD_CACHE;
      const unsigned bits = __ballot_sync(kFull, there) & 0xffffu;
      const uint32_t bar = smem_u32(&full[warp][st]);
      __syncwarp();                          // every lane has read what lay there
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(bits) * D * 4);
      __syncwarp();
      if (there && lane < kTile)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                     ::"r"(smem_u32(mine + (st * kTile + lane) * kRow)),
                       "l"(a.k_sum + (static_cast<int64_t>(page) * a.Hkv + c.gb * heads + wg) * D),
                       "r"(D * 4), "r"(bar) : "memory");
      return bits;
    };
    Cursor ahead = now;                      // the item to fetch next
    int left = n_items;                      // items not yet fetched
    int page[kAhead + 1];                    // looked up an item before it is fetched
    unsigned known[kAhead] = {};
    {
      Cursor c = now;
#pragma unroll
      for (int st = 0; st <= kAhead; ++st) {
        page[st] = -2;
        if (st < n_items) {
          page[st] = page_at(c);
          step(c);
        }
      }
    }
#pragma unroll
    for (int st = 0; st < kAhead; ++st) {
      if (left > 0) {
        known[st] = fetch(ahead, page[st], st);
        step(ahead);
        --left;
      }
    }
    int next = page[kAhead];
    uint2 qb[kSteps];
    float q1 = 0.f;
    int64_t have = -1;                       // the row whose queries are loaded
    int st = 0;
    uint32_t phase = 0;
    for (int i = 0; i < n_items; ++i, step(now)) {
      const int g = now.gb * heads + wg, j0 = first_page(now);
      const int b = min(now.b, a.B - 1);     // should the lengths change under the call
      const int64_t row = static_cast<int64_t>(b) * a.Hkv + g;
      if (kOne && have != row) {
        q1 = load_heads<D>(a, b, g, G, 0, lane, qb);
        have = row;
      }
      if (!mbar_wait_warp(smem_u32(&full[warp][st]), phase, AbortSignal{&abort_flag, nullptr})) {
        // give up, but not before the copies still in flight have come in
        if (lane == 0) {
          status |= SA_DEV_TIMEOUT;
          abort_flag = 1;
          const volatile int never = 0;
          for (int s = 0; s < kAhead; ++s)
            if (i + s < n_items)
              mbar_wait(smem_u32(&full[warp][(st + s) % kAhead]), phase ^ (st + s >= kAhead ? 1u : 0u),
                        AbortSignal{&never, nullptr});
        }
        break;
      }
      const float4* w = mine + (st * kTile + (lane >> 2)) * kRow + (lane & 3);
      // lane's scores: pages lane / 4 and + 8, over its heads
      float best[2] = {-INFINITY, -INFINITY}, top[2];
      for (int h0 = 0; h0 < (kOne ? 1 : G); h0 += 8) {
        if (!kOne) q1 = fmaxf(h0 == 0 ? 0.f : q1, load_heads<D>(a, b, g, G, h0, lane, qb));
        float c[4] = {}, d[4] = {};
        top[0] = top[1] = kLeastK;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint4 hi, lo;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float4 v = w[8 * x * kRow + 4 * k];
            top[x] = fmaxf(fmaxf(fmaxf(top[x], fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
            const uint32_t h01 = pack_bf16(v.x, v.y), h23 = pack_bf16(v.z, v.w);
            const uint32_t l01 = pack_bf16(v.x - bits_f32(h01), v.y - __uint_as_float(h01 & 0xffff0000u));
            const uint32_t l23 = pack_bf16(v.z - bits_f32(h23), v.w - __uint_as_float(h23 & 0xffff0000u));
            (x ? hi.y : hi.x) = h01;
            (x ? hi.w : hi.z) = h23;
            (x ? lo.y : lo.x) = l01;
            (x ? lo.w : lo.z) = l23;
          }
          mma(c, hi, qb[k].x, qb[k].y);
          mma(d, lo, qb[k].x, qb[k].y);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)          // fmaxf passes over NaN
          if (h0 + 2 * (lane & 3) + (x & 1) < G) best[x >> 1] = fmaxf(best[x >> 1], c[x] + d[x]);
      }
      const unsigned there = kAhead == 2 ? (st ? known[1] : known[0]) : known[0];
      // this stage's pieces have been read: the next tile's take their place
      if (left > 0) {
        const unsigned bits = fetch(ahead, next, st);
        if (st) known[1] = bits;
        else known[0] = bits;
        step(ahead);
        if (--left > 0) next = page_at(ahead);
      }
      if (++st == kAhead) {
        st = 0;
        phase ^= 1u;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        best[x] = fmaxf(best[x], __shfl_xor_sync(kFull, best[x], 1));
        best[x] = fmaxf(best[x], __shfl_xor_sync(kFull, best[x], 2));
        top[x] = fmaxf(top[x], __shfl_xor_sync(kFull, top[x], 1));
        top[x] = fmaxf(top[x], __shfl_xor_sync(kFull, top[x], 2));
      }
      if ((lane & 3) < 2) {                  // one lane a page
        const int j = (lane >> 2) + 8 * (lane & 1);
        if (j0 + j < now.nb) {
          const int64_t at = row * a.pm.max_pages + j0 + j;
          score[at] = (there >> j) & 1u ? (lane & 1 ? best[1] : best[0]) : -INFINITY;
          err[at] = (there >> j) & 1u ? q1 * (lane & 1 ? top[1] : top[0]) : 0.f;
        }
      }
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
  const int page = get(a.pm.table + b * a.pm.table_stride + j), G = a.H / a.Hkv;
  if (page < 0 || page >= a.pm.n_pages) return -INFINITY;
  const float* k = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + g) * a.D;
  double best = -INFINITY;
  for (int h = 0; h < G; ++h) {
    const uint16_t* q = a.q + b * a.qs[0] + static_cast<int64_t>(g * G + h) * a.qs[2];
    double s = 0.0;
    for (int d = lane; d < a.D; d += 32)
      s = fma(static_cast<double>(bits_f32(get(q + d))), static_cast<double>(get(k + d)), s);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
    best = fmax(best, s);
  }
  return best + 0.0;                         // -0 and +0 are equal
}

// Score of one page by a whole warp as a sum of two floats, each product and
// sum kept with its rounding error. A lane's D / 4 steps keep errors of at most
// 2^-24 (size + |p|) each, size = |q|_1 max |k|, so what is kept stays below 2^-18 size
// (D = 128) and its own roundings add up to 2^-37 size at most: kPairedErr. Eight heads
// at a time, four lanes each. (In fp64, which runs at 1/64 of fp32's rate here,
// three pages took 14,700 cycles, more than all else in the kernel.) For finite
// scores only.
template <int D>
__device__ double paired_score(const RoutePagesArgs& a, int b, int g, int j, int lane) {
  const int page = get(a.pm.table + b * a.pm.table_stride + j), G = a.H / a.Hkv, c = lane & 3;
  const float* k = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + g) * D + 4 * c;
  float4 kv[D / 16];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) kv[s] = get(reinterpret_cast<const float4*>(k + 16 * s));
  float top = -INFINITY, low = 0.f;
  for (int h0 = 0; h0 < G; h0 += 8) {
    const int h = h0 + (lane >> 2);
    const uint16_t* q = a.q + b * a.qs[0] + static_cast<int64_t>(g * G + min(h, G - 1)) * a.qs[2] + 4 * c;
    float sum = 0.f, rest = 0.f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint2 w = get(reinterpret_cast<const uint2*>(q + 16 * s));
      const float qv[4] = {bits_f32(w.x), __uint_as_float(w.x & 0xffff0000u), bits_f32(w.y),
                           __uint_as_float(w.y & 0xffff0000u)};
      const float x[4] = {kv[s].x, kv[s].y, kv[s].z, kv[s].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = qv[i] * x[i], e = fmaf(qv[i], x[i], -p);
        const float t = sum + p, bb = t - sum;
        rest += ((sum - (t - bb)) + (p - bb)) + e;
        sum = t;
      }
    }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      const float p = __shfl_xor_sync(kFull, sum, off), t = sum + p, bb = t - sum;
      rest += __shfl_xor_sync(kFull, rest, off);
      rest += (sum - (t - bb)) + (p - bb);
      sum = t;
    }
    const float hi = sum + rest, lo = rest - (hi - sum);
    if (h < G && (hi > top || (hi == top && lo > low))) {
      top = hi;
      low = lo;
    }
  }
#pragma unroll
  for (int off = 4; off <= 16; off <<= 1) {
    const float hi = __shfl_xor_sync(kFull, top, off), lo = __shfl_xor_sync(kFull, low, off);
    if (hi > top || (hi == top && lo > low)) {
      top = hi;
      low = lo;
    }
  }
  return static_cast<double>(top) + static_cast<double>(low) + 0.0;   // -0 and +0 are equal
}

// Order-preserving integers: of a float, of a double that is not NaN.
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | (1u << 31);
}
__device__ __forceinline__ float unorder32(uint32_t u) {
  return __uint_as_float(u >> 31 ? u ^ (1u << 31) : ~u);
}
__device__ __forceinline__ uint64_t order64(double x) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | (1ull << 63);
}

constexpr int kBins = 256, kPasses = 4;

// grid (B * Hkv): one row. Three CTAs an SM: with the 128 registers that the
// compiler takes for two, 12.3 us for 11 (8 rows of 598 pages, the error bound at 2^-16).
template <int D>
__global__ void __launch_bounds__(kThreads, 3) select_kernel(RoutePagesArgs a) {
  __shared__ int sums[2 * kWarps];
  __shared__ uint4 ext[kWarps];
  __shared__ __align__(16) int hist[kPasses][kBins];
  __shared__ int near_j[kNear], open_at[kNear], near_n, open_n;
  __shared__ float near_v[kNear];
  __shared__ double open_s[kNear];
  __shared__ bool is_close[kNear];
  __shared__ unsigned chosen[kSpan / 32];    // of a span's undecided pages, by bit
  __shared__ int warp_n[2][kWarps], list_n[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv;
  const int row = blockIdx.x, b = row / a.Hkv, g = row % a.Hkv;
  int turn = 0, status = 0;
  bool bad;
  // the row's place in the list: counts follow from the lengths alone
  int nb, sink, keep, before = 0;
  for (int i = tid; i < b; i += kThreads) {
    row_counts(clamp_len(get(a.pm.seq_lens + i), a.pm, &bad), a.prefix, a.budget, &nb, &sink, &keep);
    before += keep;
  }
  if (tid == 0) near_n = open_n = 0;
  if (tid < kSpan / 32) chosen[tid] = 0u;
  for (int i = tid; i < kPasses * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  before = block_sum(before, sums, turn++);
  row_counts(clamp_len(get(a.pm.seq_lens + b), a.pm, &bad), a.prefix, a.budget, &nb, &sink, &keep);
  const int start = before * a.Hkv + g * keep;
  if (tid == 0) {
    a.row_ptr[row] = start;
    if (row == rows - 1) a.row_ptr[rows] = start + keep;
    if (start + keep > a.col_cap) status |= SA_DEV_CAPACITY;
  }
  wait_for_first();

  const Layout L = layout(rows, a.pm.max_pages);
  const int64_t row_at = static_cast<int64_t>(row) * a.pm.max_pages;
  const float* score = reinterpret_cast<const float*>(a.ws) + row_at;
  const float* err = reinterpret_cast<const float*>(a.ws + L.err) + row_at;
  double* exact = reinterpret_cast<double*>(a.ws + L.exact) + row_at;
  const int f0 = min(sink, nb), f1 = max(f0, nb - 1);      // the pages that compete
  const int want = keep - (sink < nb ? sink + 1 : nb);
  const bool held = f1 - f0 <= kSpan;
  bool all = want >= f1 - f0;                // the competing pages below `last` are in
  int last = f1;
  // thread's pages of a span: span + 256 warp + 32 i + lane, so that a warp's
  // ballots are in the order of the pages; one span is read once and held
  const int mine = warp * 32 * kItems + lane;
  float v[kItems];
  auto load = [&](int span) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int j = span + mine + 32 * i;
      v[i] = j < f1 ? get(score + j) : -INFINITY;
    }
  };
  // A page scores above `above`: in; below `below`: out; else by its exact
  // score, largest first, against `edge` with `ties` of the equal ones in.
  float above = INFINITY, below = INFINITY;
  int need = 0;                              // of the undecided ones
  bool by_list = false, by_exact = false;
  uint64_t edge = 0;
  int ties = 0;
  if (want > 0 && !all) {
    // extremes of the scores, and the error bound
    uint32_t k_lo = ~0u, k_hi = 0u, k_d = 0u;
    for (int span = f0; span < f1; span += kSpan) {
      float d[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) d[i] = span + mine + 32 * i < f1 ? get(err + span + mine + 32 * i) : 0.f;
      load(span);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        if (span + mine + 32 * i >= f1) continue;
        const uint32_t u = order32(v[i]);
        k_lo = min(k_lo, u);
        k_hi = max(k_hi, u);
        k_d = max(k_d, __float_as_uint(d[i]));       // not negative: ordered as they are
      }
    }
    k_lo = __reduce_min_sync(kFull, k_lo);
    k_hi = __reduce_max_sync(kFull, k_hi);
    k_d = __reduce_max_sync(kFull, k_d);
    if (lane == 0) ext[warp] = make_uint4(k_lo, k_hi, k_d, 0u);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint4 x = ext[w];
      k_lo = min(k_lo, x.x);
      k_hi = max(k_hi, x.y);
      k_d = max(k_d, x.z);
    }
    float lo = unorder32(k_lo), hi = unorder32(k_hi);
    const float d = kErr * __uint_as_float(k_d);
    if (lo > -1e38f && hi < 1e38f && d < 1e30f && (k_d == 0u || d > kLeastErr)) {
      // The want-th largest score lies in [lo, hi]. Each pass counts the pages
      // in 256 bins of that range, from the top, and goes on in the bin the
      // count passes `want` in, widened by what its edges may be rounded by.
      int in_bin = f1 - f0;
      for (int pass = 0; pass < kPasses && in_bin > kFew && hi - lo > d; ++pass) {
        const float scale = kBins / (hi - lo), width = (hi - lo) / kBins;
        for (int span = f0; span < f1; span += kSpan) {
          if (!held) load(span);
#pragma unroll
          for (int i = 0; i < kItems; ++i)
            if (span + mine + 32 * i < f1) {
              const float x = fminf(fmaxf((v[i] - lo) * scale, 0.f), kBins - 1.f);
              atomicAdd(&hist[pass][kBins - 1 - static_cast<int>(x)], 1);
            }
        }
        __syncthreads();
        const int4 h0 = reinterpret_cast<const int4*>(hist[pass])[2 * lane];
        const int4 h1 = reinterpret_cast<const int4*>(hist[pass])[2 * lane + 1];
        const int h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
        int total = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) total += h[i];
        int upto = total;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int x = __shfl_up_sync(kFull, upto, off);
          if (lane >= off) upto += x;
        }
        int bin = 8 * lane, n = upto - total;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (n < want) in_bin = h[i];
          n += h[i];
          bin += n < want;
        }
        // the first lane whose bins reach `want` holds the bin
        const unsigned reached = __ballot_sync(kFull, upto >= want);
        bin = kBins - 1 - __shfl_sync(kFull, bin, __ffs(reached) - 1);
        in_bin = __shfl_sync(kFull, in_bin, __ffs(reached) - 1);
        const float slack = 0.01f * width + 0x1p-22f * fmaxf(fabsf(lo), fabsf(hi));
        const float new_lo = lo + bin * width - slack, new_hi = lo + (bin + 1) * width + slack;
        if (bin > 0) lo = fmaxf(lo, new_lo);
        if (bin < kBins - 1) hi = fminf(hi, new_hi);
      }
      above = hi + 2.f * d;
      below = lo - 2.f * d;
      if (k_d == 0u) {                       // queries of zeros, as a padded row has them
        above = below = INFINITY;
        all = true;
        last = f0 + want;
      }
    } else {
      below = -INFINITY;                     // none is decided
    }
    int in = 0, n_near = 0;
    for (int span = f0; span < f1; span += kSpan) {
      if (!held) load(span);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int j = span + mine + 32 * i;
        if (j >= f1) continue;
        const bool yes = v[i] > above;
        in += yes;
        if (!yes && v[i] >= below) {
          ++n_near;
          const int at = atomicAdd(&near_n, 1);
          if (at < kNear) {
            near_j[at] = j;
            near_v[at] = v[i];
          }
        }
      }
    }
    // two counts at once: neither passes 2^20
    const int in_warp = __reduce_add_sync(kFull, in), near_warp = __reduce_add_sync(kFull, n_near);
    if (lane == 0) {
      warp_n[0][warp] = in_warp;
      warp_n[1][warp] = near_warp;
    }
    __syncthreads();
    in = n_near = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      in += warp_n[0][w];
      n_near += warp_n[1][w];
    }
    need = want - in;
    if (need < n_near) {
      const bool finite = below > -INFINITY;
      if (n_near <= kNear) {
        // A page is in if fewer than `need` others may score as much, out if
        // `need` do score more; what is left open is decided by exact scores.
        by_list = true;
        const int j = tid < n_near ? near_j[tid] : -1;
        bool yes = false, open = j >= 0;
        int slot = 0;
        if (finite && open) {
          const float mine_v = near_v[tid];
          int more = 0, reach = 0;
          for (int i = 0; i < n_near; ++i) {
            more += near_v[i] > mine_v + 2.f * d;
            reach += near_v[i] >= mine_v - 2.f * d;
          }
          yes = reach <= need;
          open = !yes && more < need;
        }
        if (open) {
          slot = atomicAdd(&open_n, 1);
          open_at[slot] = j;
        }
        const int rest = need - block_sum(yes, sums, turn++), n_open = open_n;
        if (rest > 0 && rest < n_open) {
          for (int i = warp; i < n_open; i += kWarps) {
            const int page = open_at[i];
            const float size = get(err + page);
            double s = finite ? paired_score<D>(a, b, g, page, lane) : 0.0;
            if (!finite || (size > 0.f && size < kLeastSize)) s = exact_score(a, b, g, page, lane);
            if (lane == 0) open_s[i] = s;
          }
          __syncthreads();
          // the same once more, with what a paired score may be off by (compared as
          // integers: fp64 is slow here); the exact scores have the last word
          bool close = open;
          if (open) {
            if (finite) {
              const double mine_s = open_s[slot], margin = 2.0 * kPairedErr * __uint_as_float(k_d);
              const uint64_t hi_u = order64(mine_s + margin), lo_u = order64(mine_s - margin);
              int more = 0, reach = 0;
              for (int i = 0; i < n_open; ++i) {
                const uint64_t u = order64(open_s[i]);
                more += u > hi_u;
                reach += u >= lo_u;
              }
              yes = reach <= rest;
              close = !yes && more < rest;
            }
            is_close[slot] = close;
          }
          if (__syncthreads_or(close)) {
            const int rest_close = rest - __syncthreads_count(open && yes);
            if (finite) {
              for (int i = warp; i < n_open; i += kWarps) {
                if (!is_close[i]) continue;
                const double s = exact_score(a, b, g, open_at[i], lane);
                if (lane == 0) open_s[i] = s;
              }
              __syncthreads();
            }
            if (close) {
              const uint64_t mine_u = order64(open_s[slot]);
              int before = 0;
              for (int i = 0; i < n_open; ++i) {
                const uint64_t u = order64(open_s[i]);
                before += is_close[i] && (u > mine_u || (u == mine_u && open_at[i] < j));
              }
              yes = before < rest_close;
            }
          }
        } else {
          yes |= open && rest > 0;
        }
        if (yes && j - f0 < kSpan) atomicOr(&chosen[(j - f0) >> 5], 1u << ((j - f0) & 31));
        if (!yes) near_j[tid] = -1;
        __syncthreads();
      } else {
        by_exact = true;
        // a warp's 32 pages, one after another
        for (int j0 = f0 + 32 * warp; j0 < f1; j0 += 32 * kWarps) {
          for (int j = j0; j < min(j0 + 32, f1); ++j) {
            const float s = score[j];
            if (s > above || !(s >= below)) continue;
            const double e = exact_score(a, b, g, j, lane);
            if (lane == 0) exact[j] = e;
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
  for (int span = f0, turns = 0; want > 0 && span < last; span += kSpan, ++turns) {
    if (!held) load(span);
    unsigned take[kItems];
    int n_take = 0;
    if (!by_exact) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const bool t = all || v[i] > above || (!by_list && v[i] >= below);
        take[i] = __ballot_sync(kFull, t && span + mine + 32 * i < last);
        if (by_list) take[i] |= chosen[warp * kItems + i];
        n_take += __popc(take[i]);
      }
    } else {
      // of the undecided ones those above the edge, and the first `ties` at it
      unsigned equal[kItems];
      int n_equal = 0;
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int j = span + mine + 32 * i;
        bool t = j < f1 && v[i] > above, q = false;
        if (j < f1 && !t && v[i] >= below) {
          const uint64_t e = order64(exact[j]);
          t = e > edge;
          q = e == edge;
        }
        take[i] = __ballot_sync(kFull, t);
        equal[i] = __ballot_sync(kFull, q);
        n_take += __popc(take[i]);
        n_equal += __popc(equal[i]);
      }
      __syncthreads();                       // warp_n has been read
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
    int* count = list_n[turns & 1];          // read for the last time two barriers ago
    if (lane == 0) count[warp] = n_take;
    __syncthreads();
    int to = at, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) to += count[w];
      total += count[w];
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int p = to + __popc(take[i] & ((1u << lane) - 1u));
      if (((take[i] >> lane) & 1u) && p < a.col_cap) a.col_idx[p] = span + mine + 32 * i;
      to += __popc(take[i]);
    }
    at += total;
    if (by_list && span + kSpan < f1) {      // the next span's
      if (tid < kSpan / 32) chosen[tid] = 0u;
      __syncthreads();
      const int j = tid < near_n ? near_j[tid] - (span + kSpan) : -1;
      if (j >= 0 && j < kSpan) atomicOr(&chosen[j >> 5], 1u << (j & 31));
      __syncthreads();
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace

size_t route_pages_ws_bytes(int64_t rows, int max_pages) { return layout(rows, max_pages).total; }

cudaError_t launch_route_pages(const RoutePagesArgs& a, cudaStream_t st) {
  const size_t smem = static_cast<size_t>(kScoreWarps) * kAhead * kTile * (a.D / 4 + 4) * sizeof(float4);
  const bool one = a.H / a.Hkv <= 8;
  const auto score = a.D == 64 ? (one ? score_kernel<64, true> : score_kernel<64, false>)
                               : (one ? score_kernel<128, true> : score_kernel<128, false>);
  cudaError_t e = cudaFuncSetAttribute(score, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // the heads side by side that the warps of a CTA divide between them
  int heads = 1;
  while (heads < kScoreWarps && a.Hkv % (2 * heads) == 0) heads *= 2;
  score<<<kScoreCtas, 32 * kScoreWarps, smem, st>>>(a, heads);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_close(a.D == 64 ? select_kernel<64> : select_kernel<128>,
                      dim3(static_cast<unsigned>(a.B * a.Hkv)), kThreads, 0, st, a);
}

}  // namespace sa
