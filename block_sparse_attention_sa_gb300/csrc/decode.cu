// decode.cu -- attention of one new token per sequence over the paged cache.
//   l_u = scale q.k_u,  a = softmax(l),  o = sum a_u v_u,  lse = log sum exp l
//
// One pass over the cached keys and values with the running maximum and sum of
// the softmax. Every byte of the cache is used for the G = H / H_kv query heads
// that share a key-value head and for nothing else, 2 G (bf16) or 4 G (e4m3)
// flops a byte, so up to a few dozen heads the kernel is bound by the memory and
// what matters is that loads never pause:
//
// - The pages of all (sequence, key-value head) units are one list, cut into
//   equal runs, one per CTA, so that any mix of lengths keeps every SM loading
//   until the end. A CTA finds its run from the lengths (or the route's row
//   spans) itself: no host plan, nothing to keep between calls.
// - A producer warp looks the pages up, 32 at a time, and feeds a ring of pages
//   by TMA, swizzled so that ldmatrix meets no bank twice. Consumer warps take
//   32 or 64 keys of a page at a time: S = Q K^T on the tensor cores with the
//   query heads as the 16 rows of mma.m16n8k16 (16, 32 or 64 of them in a CTA),
//   the softmax in registers, P V with P as the A operand straight from those
//   registers. With up to 16 heads tcgen05 has nothing to gain: the product
//   waits for DRAM, and its accumulators would go through tensor memory. For many
//   heads on one key-value head it (with the keys as the rows, the heads as the
//   columns) has not been tried.
// - A unit that lies in one run is finished there. One that is cut leaves fp32
//   partial results (maximum, sum, unnormalised o) in the workspace, which
//   join_kernel adds in the order of the runs: no atomics, the same bits every
//   time. join_kernel is launched while the first kernel runs and waits for it.
//
// P keeps what fp32 has of it, but for the last two or three bits, as a sum of
// terms that an operand holds: three of bf16, 8 bits each, or with an e4m3 cache
// two of fp16, 11 bits each, scaled by 2^15 so that what is lost of a weight below
// 2^-18 of the largest is 2^-40 of that. (As two terms and one, an output in a
// thousand and in a hundred fell on the other side of its rounding to bf16 than
// with weights in fp32; now no more than between two orders of fp32 sums.) Where at
// most eight query heads share a key-value head the rows r + 8 of a tile are free
// and hold the terms that rows r leave: e4m3, 3 x 112,640 tokens of 56/8 heads, 111
// us so, 121.6 us with a product for each term (one term: 112); 64 x up to 8,192 in
// bf16, 213 us either way. More heads pay for a product a term: 56/1 of 64 in bf16
// 49 us (two terms: 43), 56/1 of 128 in e4m3 69 us (one: 58).
//
// Measured on GB300 (copy rate 6.79 TB/s), 56/8 heads of 128: 64 sequences of up
// to 8,192 tokens 213 us for 1.37 GB, 6.4 TB/s; 3 x 112,640 tokens in e4m3 111 us,
// 6.2 TB/s; 24 x 38,247 tokens routed to 96 pages 103 us, 5.9 TB/s. 56 heads of 64 on
// one key-value head, 16 x up to 38,247 tokens: 49 us for 100 MB, 2.0 TB/s: the
// latency of each warp's chain bounds it, with two consumer warps a scheduler. Of 6.0
// warp cycles an instruction a warp waits 1.6 for its own last result, 1.1 for global
// and 0.4 for shared memory, 0.5 for the tensor pipe, which is busy 51% of the time.
// 777 tokens, 32/8 heads: 8.9 us, 3 of them launches, the rest the chain lengths,
// table, page, product, partial, join; of the first kernel's 4.6 us the page takes 0.5,
// its products 1, its partial 0.9, the way to the page the rest.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_internal.cuh"
#include "ptx.cuh"

namespace sa {
namespace {

constexpr int kSms = 152;
// Runs, of which the workspace holds two partials each, with RG groups of 16 rows.
constexpr int max_runs(int RG) { return (RG < 4 ? 3 : 2) * kSms; }
constexpr int kMaxRuns = max_runs(1);
constexpr float kFp16Shift = 15.f;     // P is held as 2^15 p in fp16 terms

// A CTA holds RG groups of 16 rows of query heads (kTwin: 8, each in two rows of a
// tile). 4 / RG warps divide a page's keys for each group, so a CTA has four consumer
// warps (eight with one CTA an SM, 56 heads of 64 on one key-value head, P in two terms:
// 48.5 us for 43.8; two CTAs of eight 47.3 for 43.1).
template <int D, bool kFp8, int RG, bool kTwin>
struct Shape {
  static constexpr int kRows = 16 * RG;
  static constexpr int kX = kTwin ? 1 : 2;  // rows of a lane, r and r + 8, that are heads
  // products with a page's values for one of P: its terms, two in one where rows are free
  static constexpr int kTerms = kTwin ? (kFp8 ? 1 : 2) : (kFp8 ? 2 : 3);
  static constexpr int kKeyWarps = 4 / RG;
  static constexpr int kWarps = kKeyWarps * RG;         // consumer warps
  static constexpr int kSlices = RG == 4 ? 4 : 2;   // 16-key slices a warp takes at once (one at
                                               // a time: 213 us for 210, 64 sequences in bf16)
  static constexpr int kParts = 4 / kSlices;            // warps that share a page
  static constexpr int kPhases = kKeyWarps / kParts;    // pages being worked on
  static constexpr int kThreads = 32 * (kWarps + 1);
  // CTAs on an SM: three where the registers allow it and two pages fit the
  // ring (e4m3, 3 x 112,640 tokens of 56/8 heads: 110 us with three, 112 with two;
  // 16 sequences of up to 38,247 tokens, 32/1 heads of 64 in bf16: 33.3 and 34.8),
  // else two (12/1 heads of 128 in e4m3, where three spill: 32.7 and 31.5)
  static constexpr int kCtas = (kTwin && kFp8) || (RG < 4 && D == 64) ? 3 : 2;
  static constexpr int kRuns = kSms * kCtas;
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;    // one token of one head
  static constexpr int kPage = kBlock * kRowBytes;
  static constexpr int kBox = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kStage = 2 * kPage;
  static constexpr int kRing = (kCtas == 3 ? 48 : (RG == 1 ? 96 : 64)) * 1024;
  static constexpr int kStages = kRing / kStage < 16 ? kRing / kStage : 16;
  static constexpr int kChunk = 32;                     // columns joined at a time
  static constexpr int kPad = kChunk + 8;               // row stride of the join buffer
  static constexpr int kJoin = kWarps * 16 * kPad * 4;
  static constexpr int kQueries = RG * (D / 16) * 32 * 16;
  static constexpr int kSmem = kStages * kStage + kJoin + kQueries + 1024;
};

// A unit: 16 RG query heads (tile rt of those) of one sequence that share a
// key-value head. dest: -1 if the run holds it whole, else which of the run's
// partials its piece is.
struct __align__(16) Unit {
  int b, g, rt, dest;
};

struct __align__(16) PageMeta {
  Unit unit;
  int live;     // tokens of the page that count
  int flags;    // 1: first page of a unit's piece, 2: last
};

// A unit that is cut, for join_kernel, and its first and last run.
struct __align__(16) Cut {
  int unit, first, last, pad;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool kFp16>
__device__ __forceinline__ void mma(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  if (kFp16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two pairs of fp16 values, lower bytes first; exact.
__device__ __forceinline__ uint2 e4m3x4_half4(uint32_t x) {
  uint2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(r.x), "=r"(r.y) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The upper 16 bits of two floats: the values cut to bf16.
__device__ __forceinline__ uint32_t top_bf16(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

__device__ __forceinline__ float lo_f32(uint32_t bf2) { return __uint_as_float(bf2 << 16); }
__device__ __forceinline__ float hi_f32(uint32_t bf2) { return __uint_as_float(bf2 & 0xffff0000u); }

// Two weights as sums of terms that an A fragment holds: three of bf16 (2^-22 of the
// weight is lost), the last times `third`, or two of fp16 (2^-22, and below 2^-14 the last
// 2^-25). bf16 terms are cut, not rounded, and 2^-24 of the weight is added twice to what
// is left, so that all are positive: an infinite value stays one (e4m3 has none).
template <bool kFp8>
__device__ __forceinline__ void split(float p0, float p1, float third, uint32_t* t) {
  if (kFp8) {
    t[0] = pack_half(p0, p1);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&t[0]));
    t[1] = pack_half(p0 - h.x, p1 - h.y);
  } else {
    t[0] = top_bf16(p0, p1);
    const float r0 = fmaf(p0, 0x1p-24f, p0 - lo_f32(t[0]));
    const float r1 = fmaf(p1, 0x1p-24f, p1 - hi_f32(t[0]));
    t[1] = top_bf16(r0, r1);
    t[2] = pack_bf16(third * fmaf(p0, 0x1p-24f, r0 - lo_f32(t[1])),
                     third * fmaf(p1, 0x1p-24f, r1 - hi_f32(t[1])));
  }
}

// A page as TMA lays it out: boxes of at most 128 bytes a token, their 16-byte
// pieces XORed with the row (rows 0 .. 7, or every second one in 64-byte boxes).
// piece_row is where piece `half` (0, 1) of a row lies; next_piece steps from
// there to piece 2 k + half: one XOR, as nothing below the row is added.
template <int kBox>
__device__ __forceinline__ uint32_t piece_row(int row, int half) {
  if (kBox == 64) return row * 64 + ((half ^ ((row >> 1) & 3)) << 4);
  return row * 128 + ((half ^ (row & 7)) << 4);
}

template <int kBox>
__device__ __forceinline__ uint32_t next_piece(uint32_t at, int k) {
  constexpr int kPairs = kBox / 32;          // pieces of a box row, in pairs
  return (at ^ ((k % kPairs) << 5)) + k / kPairs * (kBlock * kBox);
}

// Pages of group `i` of the list: a sequence (every page) and its length, or a
// row of the route and where that begins.
__device__ __forceinline__ int group_pages(const DecodeArgs& a, int i, int* from, int* status) {
  if (a.row_ptr) {
    const int beg = get(a.row_ptr + i), end = get(a.row_ptr + i + 1);
    *from = beg;
    if (beg < 0 || end < beg || end > a.col_cap || end - beg > a.pm.max_pages) {
      *status |= SA_DEV_BAD_ROUTE;
      return 0;
    }
    return end - beg;
  }
  bool bad;
  const int n = clamp_len(get(a.pm.seq_lens + i), a.pm, &bad);
  if (bad) *status |= SA_DEV_BAD_CACHE;
  *from = n;
  return (n + kBlock - 1) / kBlock;
}

// Whether join_kernel finds the units that are cut in a list, by the run that a
// unit starts in. Where the units are no more than the runs and a warp reads the
// groups' sizes at once, it works them out by itself (777 tokens: 8.9 us, listed
// 9.6; 24 x 96 pages, 192 rows: 104.8 us, listed 102.3).
__host__ __device__ inline bool cuts_listed(const DecodeArgs& a, int RT, int runs) {
  return a.B * a.Hkv * RT > runs || (a.row_ptr ? a.B * a.Hkv : a.B) > 32;
}

template <int D, bool kFp8, int RG, bool kTwin>
__global__ void __launch_bounds__(Shape<D, kFp8, RG, kTwin>::kThreads, Shape<D, kFp8, RG, kTwin>::kCtas)
decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              DecodeArgs a, int RT, float* partial, Cut* cuts) {
  using S = Shape<D, kFp8, RG, kTwin>;
  constexpr int kX = S::kX;
  constexpr int NS = S::kStages, W = S::kWarps, NT = S::kThreads;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[NS], empty[NS], joined;
  __shared__ PageMeta meta[NS];
  __shared__ float sm_m[W][16], sm_l[W][16];
  __shared__ Unit sm_unit[W];                // each warp's copy of its unit
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* join = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)) + NS * S::kStage);
  uint4* sm_q = reinterpret_cast<uint4*>(reinterpret_cast<char*>(join) + S::kJoin);
  const int G = a.H / a.Hkv, C = gridDim.x, c = blockIdx.x;
  const bool routed = a.row_ptr != nullptr;
  const int n_groups = routed ? a.B * a.Hkv : a.B;
  const int per_group = routed ? RT : a.Hkv * RT;        // units of a group
  const bool listed = cuts_listed(a, RT, C);
  const AbortSignal abort{&abort_flag, nullptr};
  int status = 0;

  let_next_launch();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), W);
    }
    mbar_init(smem_u32(&joined), W);
    fence_barrier_init();
    abort_flag = 0;
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }

  // this CTA's run of the page list
  const Run run = plan_run<NT>(
      n_groups, per_group,
      [&](int i, int* from) { return group_pages(a, i, from, &status); });
  // groups without a page: nothing to attend
  for (int i = c + C * warp; i < n_groups; i += C * (NT / 32)) {
    int from;
    if (group_pages(a, i, &from, &status) != 0) continue;
    const int b = routed ? i / a.Hkv : i;
    const int h0 = routed ? (i % a.Hkv) * G : 0, nh = routed ? G : a.H;
    for (int e = lane; e < nh * (D / 8); e += 32)
      *reinterpret_cast<uint4*>(a.o + b * a.os[0] + (h0 + e / (D / 8)) * a.os[2] + e % (D / 8) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int h = lane; h < nh; h += 32) a.lse[static_cast<int64_t>(b) * a.H + h0 + h] = -INFINITY;
  }

  if (warp == W) {
    // ---------------------------------------------------------- producer --
    int left = run.hi - run.lo, group = run.group;
    int off = run.off;                          // pages into the group's units
    int cnt = run.count, from = run.size;       // as group_pages gives them
    int s = 0, in_ring = 0;                     // next stage; stages ever used, up to NS
    uint32_t ph = 0;
    Cut cut{-1, 0, 0, 0};
    bool ok = true;
    while (left > 0 && ok) {
      if (group >= n_groups) break;             // the lengths changed under the call
      if (off >= cnt * per_group) {
        off = 0;
        if (++group < n_groups) cnt = group_pages(a, group, &from, &status);
        continue;
      }
      // (divisions, 100 cycles and more each, only where there is something to divide)
      const int sub = off < cnt ? 0 : off / cnt, p0 = off - sub * cnt, take = min(left, cnt - p0);
      const int tile = RT == 1 ? sub : sub / RT;
      const int b = routed ? group / a.Hkv : group, g = routed ? group - b * a.Hkv : tile;
      const int rt = routed ? sub : sub - tile * RT;
      bool bad = false;
      const int n = routed ? clamp_len(get(a.pm.seq_lens + b), a.pm, &bad) : from;
      if (bad) status |= SA_DEV_BAD_CACHE;
      const int nb = (n + kBlock - 1) / kBlock;
      const int dest = take == cnt ? -1 : (p0 == 0 ? 1 : 0);
      for (int q0 = 0; q0 < take && ok; q0 += 32) {
        // 32 pages are looked up at once, then fed one by one
        const int q = q0 + lane;
        int page = -1, live = 0;
        if (q < take) {
          int j = p0 + q;
          if (routed) {
            const int at = from + j;
            const bool there = from >= 0 && at < a.col_cap;
            const int prev = there && j > 0 ? get(a.col_idx + at - 1) : -1;
            j = there ? get(a.col_idx + at) : -1;
            if (j < 0 || j >= nb || j <= prev) {
              status |= SA_DEV_BAD_ROUTE;
              j = -1;
            }
          }
          if (j >= 0) {
            page = get(a.pm.table + b * a.pm.table_stride + j);
            live = min(kBlock, n - j * kBlock);
            if (page < 0 || page >= a.pm.n_pages) {
              status |= SA_DEV_BAD_CACHE;
              live = 0;
            }
          }
        }
        const int m = min(32, take - q0);
        for (int x = 0; x < m; ++x) {
          const int pg = __shfl_sync(0xffffffffu, page, x);
          const int lv = __shfl_sync(0xffffffffu, live, x);
          if (!mbar_wait_warp(smem_u32(&empty[s]), ph ^ 1u, abort)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            meta[s] = PageMeta{Unit{b, g, rt, dest}, lv,
                               (q0 + x == 0 ? 1 : 0) | (q0 + x == take - 1 ? 2 : 0)};
            const uint32_t bar = smem_u32(&full[s]);
            if (lv > 0) {
              mbar_arrive_expect_tx(bar, S::kStage);
              const uint32_t dst = ring + s * S::kStage;
              constexpr int kElts = kFp8 ? S::kBox : S::kBox / 2;    // elements of a box row
#pragma unroll
              for (int i = 0; i < D / kElts; ++i) {
                tma_load_4d(dst + i * kBlock * S::kBox, &kmap, bar, i * kElts, 0, g, pg);
                tma_load_4d(dst + S::kPage + i * kBlock * S::kBox, &vmap, bar, i * kElts, 0, g, pg);
              }
            } else {
              mbar_arrive(bar);
            }
          }
          __syncwarp();
          if (++s == NS) {
            s = 0;
            ph ^= 1u;
          }
          if (in_ring < NS) ++in_ring;
        }
      }
      if (dest == 1)
        cut = Cut{(b * a.Hkv + g) * RT + rt, c, run_of(run.T, C, run.hi - left + cnt - 1), 0};
      off += take;
      left -= take;
    }
    if (lane == 0) {
      if (listed) cuts[c] = cut;
      if (!ok) {
        abort_flag = 1;
        status |= SA_DEV_TIMEOUT;
      }
      // no copy may be in flight when the CTA ends
      const volatile int never = 0;
      for (int i = 0; i < in_ring; ++i) {
        // from the newest stage back: those below `s` have its phase
        const int at = s > i ? s - 1 - i : s - 1 - i + NS;
        mbar_wait(smem_u32(&full[at]), s > i ? ph : ph ^ 1u, AbortSignal{&never, nullptr});
      }
    }
  } else {
    // --------------------------------------------------------- consumers --
    const int rg = warp / S::kKeyWarps, kw = warp % S::kKeyWarps;
    const int r = lane >> 2, cq = lane & 3;
    const int n_pages = run.hi - run.lo;
    uint4* q_frag = sm_q + rg * (D / 16) * 32 + lane;       // A fragment k at [32 k]
    float o[D / 8][4];
    // rows r and r + 8 of the warp's 16: largest q.k, sum, and what takes q.k to a
    // logit (base 2)
    float m[2], l[2], f[2];
    uint32_t join_phase = 0;
    bool ok = true;
    // all consumer warps meet; false if one of them gave up
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&joined));
      const bool done = mbar_wait_warp(smem_u32(&joined), join_phase, abort);
      join_phase ^= 1u;
      return done;
    };
    // A unit's queries as A fragments, rows beyond the group's heads zero: kept
    // in shared memory, every warp of a row group writing some of them.
    auto load_queries = [&](int b, int g, int rt) {
      uint32_t qa[D / 16][4];
      const float base = a.scale_log2 * (kFp8 && a.k_scale ? get(a.k_scale + g) : 1.f);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = rt * S::kRows + rg * 16 + r + 8 * x;
        const bool there = x < kX && row < G;
        const uint16_t* q = a.q + b * a.qs[0] + (g * G + (there ? row : 0)) * a.qs[2];
        f[x] = base;
        if (!kFp8) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            qa[k][x] = there ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * cq) : 0u;
            qa[k][2 + x] = there ? *reinterpret_cast<const uint32_t*>(q + 16 * k + 2 * cq + 8) : 0u;
          }
        } else {
          // in fp16, a row scaled by a power of two so that its largest
          // element is in [2^14, 2^15): bits are lost only below 2^-39 of it
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint2 w = there ? *reinterpret_cast<const uint2*>(q + 16 * k + 4 * cq)
                                  : make_uint2(0u, 0u);
            qa[k][x] = w.x;
            qa[k][2 + x] = w.y;
            top = fmaxf(top, fmaxf(fmaxf(fabsf(lo_f32(w.x)), fabsf(hi_f32(w.x))),
                                   fmaxf(fabsf(lo_f32(w.y)), fabsf(hi_f32(w.y)))));
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = top > 0.f && top < INFINITY ? 14 - ilogbf(top) : 0;
          // 2^e in two steps: that of a subnormal row is beyond one float
          const float up1 = ldexpf(1.f, e / 2), up2 = ldexpf(1.f, e - e / 2);
          f[x] = base * ldexpf(1.f, -(e / 2)) * ldexpf(1.f, -(e - e / 2));
          if (f[x] == 0.f) f[x] = 0x1p-149f;   // a masked -inf times 0 would be no number
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t w = qa[k][2 * y + x];
              qa[k][2 * y + x] = pack_half(lo_f32(w) * up1 * up2, hi_f32(w) * up1 * up2);
            }
        }
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        if (k % S::kKeyWarps == kw) q_frag[32 * k] = make_uint4(qa[k][0], qa[k][1], qa[k][2], qa[k][3]);
    };
    // those of the first unit need not wait for its first page
    if (n_pages > 0) {
      const int sub = run.off < run.count ? 0 : run.off / run.count;
      const int b = routed ? run.group / a.Hkv : run.group;
      load_queries(b, routed ? run.group - b * a.Hkv : sub / RT, routed ? sub : sub % RT);
      ok = meet();
    }
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_pages && ok; ++i) {
      if (!mbar_wait_warp(smem_u32(&full[s]), ph, abort)) {
        ok = false;
        break;
      }
      const int flags = meta[s].flags, page_live = meta[s].live;
      const bool mine = i % S::kPhases == kw / S::kParts;
      if (flags & 1) {
        const Unit unit = meta[s].unit;
        if (lane == 0) sm_unit[warp] = unit;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        if (i > 0) {
          load_queries(unit.b, unit.g, unit.rt);
          if (!meet()) {
            ok = false;
            break;
          }
        }
      }
      constexpr int SL = S::kSlices, kTerms = S::kTerms;
      // the warp's first key of the page, and how many from it on count
      const int k0 = 16 * SL * (kw % S::kParts), live = page_live - k0;
      if (mine && live > 0) {
        const uint32_t kp = ring + s * S::kStage, vp = kp + S::kPage;
        // The fragments of a batch of steps are loaded before the first of them
        // is used, and the first of V before the softmax.
        constexpr int kSteps = D / (kFp8 ? 32 : 16), kQ = kFp8 ? 2 : 1;
        constexpr int KB = SL == 4 || kFp8 ? 1 : 4 / SL, VB = kFp8 ? 2 : 4;   // steps of a batch
        float sc[2 * SL][4] = {};
        const uint32_t k_at = kp + piece_row<S::kBox>(k0 + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
        for (int k = 0; k < kSteps; k += KB) {
          uint4 qf[KB * kQ];
          uint32_t kb[KB][SL][4];
#pragma unroll
          for (int u = 0; u < KB; ++u) {
#pragma unroll
            for (int y = 0; y < SL; ++y)
              ldsm4(kb[u][y], next_piece<S::kBox>(k_at, k + u) + 16 * y * S::kBox);
#pragma unroll
            for (int x = 0; x < kQ; ++x) qf[kQ * u + x] = q_frag[32 * (kQ * (k + u) + x)];
          }
#pragma unroll
          for (int u = 0; u < KB; ++u)
#pragma unroll
            for (int y = 0; y < SL; ++y) {
              if (!kFp8) {
                mma<false>(sc[2 * y], qf[u], kb[u][y][0], kb[u][y][1]);
                mma<false>(sc[2 * y + 1], qf[u], kb[u][y][2], kb[u][y][3]);
              } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint2 k0h = e4m3x4_half4(kb[u][y][x]), k1h = e4m3x4_half4(kb[u][y][2 + x]);
                  mma<true>(sc[2 * y], qf[2 * u + x], k0h.x, k0h.y);
                  mma<true>(sc[2 * y + 1], qf[2 * u + x], k1h.x, k1h.y);
                }
              }
            }
        }
        const uint32_t v_at = vp + piece_row<S::kBox>(k0 + (lane & 15), lane >> 4);
        uint32_t vb[VB][4];
#pragma unroll
        for (int u = 0; u < VB; ++u) ldsm4_t(vb[u], next_piece<S::kBox>(v_at, u));
        // lane's scores: rows r (0, 1) and r + 8 (2, 3), keys 8 t + 2 cq + {0, 1}
        const bool part = live < 16 * SL;
        if (part) {
#pragma unroll
          for (int t = 0; t < 2 * SL; ++t)
#pragma unroll
            for (int x = 0; x < 2 * kX; ++x)
              if (8 * t + 2 * cq + (x & 1) >= live) sc[t][x] = -INFINITY;
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 2 * SL; ++t)
#pragma unroll
          for (int x = 0; x < 2 * kX; ++x) top[x >> 1] = fmaxf(top[x >> 1], sc[t][x]);
        bool grew = false;
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
          top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
          grew |= top[x] > m[x];
        }
        if (__any_sync(0xffffffffu, grew)) {
          float corr[2];
#pragma unroll
          for (int x = 0; x < kX; ++x) {
            const float now = fmaxf(m[x], top[x]);
            corr[x] = now == -INFINITY ? 1.f : ex2((m[x] - now) * f[x]);
            m[x] = now;
            l[x] *= corr[x];
          }
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][0] *= corr[0];
            o[j][1] *= corr[0];
            o[j][2] *= corr[kX - 1];
            o[j][3] *= corr[kX - 1];
          }
        }
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          // m is subtracted before the scaling: the largest key has weight 1
          // however coarse fp32 is at its logit's size
          const float mx = m[x] == -INFINITY ? 0.f : m[x];
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < 2 * SL; ++t) {
            sc[t][2 * x] = ex2(kFp8 ? fmaf(sc[t][2 * x] - mx, f[x], kFp16Shift) : (sc[t][2 * x] - mx) * f[x]);
            sc[t][2 * x + 1] = ex2(kFp8 ? fmaf(sc[t][2 * x + 1] - mx, f[x], kFp16Shift) : (sc[t][2 * x + 1] - mx) * f[x]);
            sum += sc[t][2 * x] + sc[t][2 * x + 1];
          }
          l[x] += sum;
        }
        // V: a key that does not count has weight 0, and whatever lies there
        // (NaN) must not meet it
#pragma unroll
        for (int y = 0; y < SL; ++y) {
          uint32_t keep[2] = {~0u, ~0u};
          if (part) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int k = 16 * y + 8 * t + 2 * cq;
              keep[t] = (k < live ? 0xffffu : 0u) | (k + 1 < live ? 0xffff0000u : 0u);
            }
          }
          // P as A fragments: registers 0 and 2 are row r, 1 and 3 row r + 8
          uint32_t pw[kTerms][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (x % 2 >= kX) continue;
            const float p0 = sc[2 * y + (x >> 1)][2 * (x & 1)], p1 = sc[2 * y + (x >> 1)][2 * (x & 1) + 1];
            uint32_t t[3];
            split<kFp8>(p0, p1, kTwin ? 0.5f : 1.f, t);
            pw[0][x] = t[0];
            if (!kTwin) {
              for (int z = 1; z < kTerms; ++z) pw[z][x] = t[z];
            } else {
              pw[0][x + 1] = t[1];
              if (!kFp8) pw[kTerms - 1][x] = pw[kTerms - 1][x + 1] = t[2];
            }
          }
          uint4 pt[kTerms];
#pragma unroll
          for (int z = 0; z < kTerms; ++z) pt[z] = make_uint4(pw[z][0], pw[z][1], pw[z][2], pw[z][3]);
#pragma unroll
          for (int j = 0; j < kSteps; j += VB) {
            if (y > 0 || j > 0)
#pragma unroll
              for (int u = 0; u < VB; ++u)
                ldsm4_t(vb[u], next_piece<S::kBox>(v_at, j + u) + 16 * y * S::kBox);
            if (part)
#pragma unroll
              for (int u = 0; u < VB; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) vb[u][x] &= keep[x & 1];
            if (!kFp8) {
#pragma unroll
              for (int z = 0; z < kTerms; ++z)
#pragma unroll
                for (int u = 0; u < VB; ++u) {
                  mma<false>(o[2 * (j + u)], pt[z], vb[u][0], vb[u][1]);
                  mma<false>(o[2 * (j + u) + 1], pt[z], vb[u][2], vb[u][3]);
                }
            } else {
              // a transposed 16-bit element is two neighbouring dims: the even
              // ones make one column tile, the odd ones the next
#pragma unroll
              for (int u = 0; u < VB; ++u) {
                uint2 w[2][2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  w[x][0] = e4m3x4_half4(__byte_perm(vb[u][2 * x], 0, 0x3120));
                  w[x][1] = e4m3x4_half4(__byte_perm(vb[u][2 * x + 1], 0, 0x3120));
                }
#pragma unroll
                for (int z = 0; z < kTerms; ++z)
#pragma unroll
                  for (int x = 0; x < 2; ++x) {
                    mma<true>(o[4 * (j + u) + 2 * x], pt[z], w[x][0].x, w[x][1].x);
                    mma<true>(o[4 * (j + u) + 2 * x + 1], pt[z], w[x][0].y, w[x][1].y);
                  }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
      if (++s == NS) {
        s = 0;
        ph ^= 1u;
      }

      if (flags & 2) {
        const Unit unit = sm_unit[warp];
        const int dest = unit.dest, rt = unit.rt, b = unit.b, g = unit.g;
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
          l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
          m[x] *= f[x];
        }
        // the piece ends: the key warps' results are added
#pragma unroll
        for (int x = 0; x < kX; ++x)
          if (cq == 0) {
            sm_m[warp][r + 8 * x] = m[x];
            sm_l[warp][r + 8 * x] = l[x];
          }
        if (!meet()) {
          ok = false;
          break;
        }
        float w[2];
#pragma unroll
        for (int x = 0; x < kX; ++x) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < S::kKeyWarps; ++k)
            top = fmaxf(top, sm_m[rg * S::kKeyWarps + k][r + 8 * x]);
          w[x] = m[x] == -INFINITY ? 0.f : ex2(m[x] - top);
        }
        // scaled in place: as products inside the loop below they would be kept
        // beside the sums, 64 more registers and spills in the loop over pages
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          if (kTwin) {                         // the rows of one head's terms
            o[j][0] += o[j][2];
            o[j][1] += o[j][3];
          }
          o[j][0] *= w[0];
          o[j][1] *= w[0];
          o[j][2] *= w[kX - 1];
          o[j][3] *= w[kX - 1];
        }
        float* part = partial + static_cast<int64_t>(2 * c + max(dest, 0)) * S::kRows * (D + 2);
        // through the join buffer 32 columns at a time, or, behind a run's last
        // page, through the ring all at once: no page will be loaded any more
        const bool at_once = i == n_pages - 1;
        float* buf = at_once ? reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw))) : join;
        const int cols = at_once ? D : S::kChunk, pad = cols + 8;
        constexpr int kLogD = D == 64 ? 6 : 7;
        const int quads = at_once ? kLogD - 2 : 3;       // of a row, as a power of two
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += cols) {
          float* row0 = buf + (warp * 16 + r) * pad - c0;
          float* row1 = row0 + 8 * pad;
#pragma unroll
          for (int j = 0; j < D / 8; j += 2) {
            if (8 * j < c0 || 8 * j >= c0 + cols) continue;
            // columns of a tile: consecutive, or (e4m3) every second dim of 16
            if (kFp8) {
              const int col = 8 * j + 4 * cq;
              *reinterpret_cast<float4*>(row0 + col) = make_float4(o[j][0], o[j + 1][0], o[j][1], o[j + 1][1]);
              *reinterpret_cast<float4*>(row1 + col) = make_float4(o[j][2], o[j + 1][2], o[j][3], o[j + 1][3]);
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int col = 8 * (j + y) + 2 * cq;
                *reinterpret_cast<float2*>(row0 + col) = make_float2(o[j + y][0], o[j + y][1]);
                *reinterpret_cast<float2*>(row1 + col) = make_float2(o[j + y][2], o[j + y][3]);
              }
            }
          }
          if (!meet()) {
            ok = false;
            break;
          }
          for (int e = warp * 32 + lane; e < S::kRows << quads; e += 32 * W) {
            const int row = e >> quads, col = (e & ((1 << quads) - 1)) * 4, grp = row >> 4, rr = row & 15;
            const int head = rt * S::kRows + row;
            if (head >= G) continue;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, tot = 0.f;
#pragma unroll
            for (int k = 0; k < S::kKeyWarps; ++k) {
              const int wp = grp * S::kKeyWarps + k;
              const float4 v = *reinterpret_cast<const float4*>(buf + (wp * 16 + rr) * pad + col);
              sum.x += v.x;
              sum.y += v.y;
              sum.z += v.z;
              sum.w += v.w;
              top = fmaxf(top, sm_m[wp][rr]);
            }
#pragma unroll
            for (int k = 0; k < S::kKeyWarps; ++k) {
              const int wp = grp * S::kKeyWarps + k;
              // without a maximum the sum is 0, or NaN if only NaN was there
              tot += sm_m[wp][rr] == -INFINITY ? sm_l[wp][rr] : sm_l[wp][rr] * ex2(sm_m[wp][rr] - top);
            }
            const int col_g = c0 + col;
            if (dest < 0) {
              const float inv = tot == 0.f ? 0.f : (a.v_scale ? get(a.v_scale + g) : 1.f) / tot;
              const int h = g * G + head;
              *reinterpret_cast<uint2*>(a.o + b * a.os[0] + h * a.os[2] + col_g) = make_uint2(
                  pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
              if (col_g == 0 && a.lse)
                a.lse[static_cast<int64_t>(b) * a.H + h] =
                    tot == 0.f ? -INFINITY
                               : (top + log2f(kFp8 ? tot * 0x1p-15f : tot)) * 0.69314718055994530942f;
            } else {
              *reinterpret_cast<float4*>(part + row * D + col_g) = sum;
              if (col_g == 0)
                *reinterpret_cast<float2*>(part + S::kRows * D + 2 * row) = make_float2(top, tot);
            }
          }
          // the buffer is written again only after every warp has read it
          if (!at_once && !meet()) {
            ok = false;
            break;
          }
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) {
      abort_flag = 1;
      status |= SA_DEV_TIMEOUT;
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

// grid (units, or runs if listed; heads of a unit), 256 threads: adds the partials of one
// unit that is cut for one query head, eight warps taking every eighth piece.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_kernel(DecodeArgs a, int RT, int rows, int runs, float unit, const float* partial,
            const Cut* cuts) {
  __shared__ float sm_o[kJoinWarps][D];
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, units = a.B * a.Hkv * RT;
  // Every CTA passes the wait, whatever it has to do: were this grid to end ahead
  // of the first, the call's outputs would be taken for finished.
  Cut cut{static_cast<int>(blockIdx.x), 0, -1, 0};
  if (cuts_listed(a, RT, runs)) {
    wait_for_first();
    const int4 whole = *reinterpret_cast<const int4*>(cuts + blockIdx.x);   // in one load
    cut = Cut{whole.x, whole.y, whole.z, 0};
    if (cut.unit < 0 || cut.unit >= units) return;
  } else {
    // a unit's place in the list of pages follows from the lengths, which are
    // there before the first kernel is done
    const bool routed = a.row_ptr != nullptr;
    const int n_groups = routed ? a.B * a.Hkv : a.B, per_group = units / n_groups;
    const int group = cut.unit / per_group;
    int status = 0, before = 0, total = 0, cnt = 0;
    if (lane < n_groups) {
      int from;
      total = group_pages(a, lane, &from, &status);
      if (lane < group) before = total;
      if (lane == group) cnt = total;
    }
    total = __reduce_add_sync(0xffffffffu, total) * per_group;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    before = __reduce_add_sync(0xffffffffu, before) * per_group + (cut.unit - group * per_group) * cnt;
    if (cnt > 0) {
      cut.first = run_of(total, runs, before);
      cut.last = run_of(total, runs, before + cnt - 1);
    }
    wait_for_first();
  }
  if (cut.first < 0 || cut.last <= cut.first || cut.last >= runs) return;
  const int G = a.H / a.Hkv, rt = cut.unit % RT, bg = cut.unit / RT;
  const int b = bg / a.Hkv, g = bg % a.Hkv, row = blockIdx.y, head = rt * rows + row;
  if (head >= G) return;
  constexpr int V = D / 32;
  const int64_t stride = static_cast<int64_t>(rows) * (D + 2);
  // the first piece is the second partial of its run (the run ends in it), the
  // others the first of theirs
  auto piece = [&](int i) {
    return partial + stride * (2 * static_cast<int64_t>(cut.first + i) + (i == 0 ? 1 : 0));
  };
  const int n = cut.last - cut.first + 1;
  float o[V] = {}, m = -INFINITY, l = 0.f;
  // four pieces on their way at once
  for (int i0 = warp; i0 < n; i0 += 4 * kJoinWarps) {
    float2 ml[4];
    float v[4][V];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* p = piece(min(i0 + u * kJoinWarps, n - 1));
      ml[u] = *reinterpret_cast<const float2*>(p + rows * D + 2 * row);
#pragma unroll
      for (int x = 0; x < V; ++x) v[u][x] = p[row * D + lane + 32 * x];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i0 + u * kJoinWarps >= n) break;
      const float pm = ml[u].x, pl = ml[u].y;
      if (pm == -INFINITY) {                 // nothing counted there (a sum of 0, or NaN)
        l += pl;
        continue;
      }
      const float now = fmaxf(m, pm), c0 = m == -INFINITY ? 0.f : ex2(m - now), c1 = ex2(pm - now);
      l = (m == -INFINITY ? l : l * c0) + pl * c1;
      m = now;
#pragma unroll
      for (int x = 0; x < V; ++x) o[x] = o[x] * c0 + v[u][x] * c1;
    }
  }
#pragma unroll
  for (int x = 0; x < V; ++x) sm_o[warp][lane + 32 * x] = o[x];
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float top = -INFINITY, tot = 0.f, sum = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sm_m[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (sm_m[w] == -INFINITY) {
      tot += sm_l[w];
      continue;
    }
    const float c = ex2(sm_m[w] - top);
    tot += sm_l[w] * c;
    sum += sm_o[w][threadIdx.x] * c;
  }
  const float inv = tot == 0.f ? 0.f : (a.v_scale ? a.v_scale[g] : 1.f) / tot;
  const int h = g * G + head;
  a.o[b * a.os[0] + h * a.os[2] + threadIdx.x] = __bfloat16_as_ushort(__float2bfloat16_rn(sum * inv));
  if (threadIdx.x == 0 && a.lse)
    a.lse[static_cast<int64_t>(b) * a.H + h] =
        tot == 0.f ? -INFINITY : (top + log2f(tot * unit)) * 0.69314718055994530942f;
}

// Row groups a CTA holds for G query heads per key-value head: as few as hold them
// (16 sequences of up to 38,247 tokens, heads of 128 in bf16: 16 heads in 16 rows 41.7
// us, in 32 rows 47.3; 17 heads in 32 rows 47.8, in 64 rows 73.9), 64 rows at most.
int row_groups(int G) { return G <= 16 ? 1 : (G <= 32 ? 2 : 4); }

size_t cuts_bytes() { return (sizeof(Cut) * kMaxRuns + 255) & ~static_cast<size_t>(255); }

template <int D, bool kFp8, int RG, bool kTwin>
cudaError_t launch(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   cudaStream_t st) {
  using S = Shape<D, kFp8, RG, kTwin>;
  static_assert(S::kRuns <= max_runs(RG), "the workspace holds the partials of every run");
  static_assert(S::kWarps * 16 * (D + 8) * 4 <= S::kStages * S::kStage, "the ring holds a unit's sums");
  // with 2 KB for the static arrays and the 1 KB that every CTA costs beside
  static_assert(S::kCtas * (S::kSmem + 3 * 1024) <= 228 * 1024, "the ring does not fit shared memory");
  const int G = a.H / a.Hkv, RT = (G + S::kRows - 1) / S::kRows;
  Cut* cuts = reinterpret_cast<Cut*>(a.ws);
  float* partial = reinterpret_cast<float*>(a.ws + cuts_bytes());
  cudaError_t e = cudaFuncSetAttribute(decode_kernel<D, kFp8, RG, kTwin>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = static_cast<int64_t>(a.B) * a.Hkv * RT;
  decode_kernel<D, kFp8, RG, kTwin><<<S::kRuns, S::kThreads, S::kSmem, st>>>(kmap, vmap, a, RT, partial, cuts);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_close(join_kernel<D>,
                      dim3(static_cast<unsigned>(cuts_listed(a, RT, S::kRuns) ? S::kRuns : units),
                           static_cast<unsigned>(G < S::kRows ? G : S::kRows)),
                      32 * kJoinWarps, 0, st, a, RT, S::kRows, S::kRuns, kFp8 ? 0x1p-15f : 1.f,
                      partial, cuts);
}

template <int D, bool kFp8>
cudaError_t launch_d(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     cudaStream_t st) {
  switch (row_groups(a.H / a.Hkv)) {
    case 1: return a.H / a.Hkv <= 8 ? launch<D, kFp8, 1, true>(a, kmap, vmap, st)
                                    : launch<D, kFp8, 1, false>(a, kmap, vmap, st);
    case 2: return launch<D, kFp8, 2, false>(a, kmap, vmap, st);
    default: return launch<D, kFp8, 4, false>(a, kmap, vmap, st);
  }
}

}  // namespace

int decode_row_tiles(int H, int Hkv) {
  const int G = H / Hkv, rows = 16 * row_groups(G);
  return (G + rows - 1) / rows;
}

size_t decode_ws_bytes(int H, int Hkv, int D) {
  // two partials of every run
  const int groups = row_groups(H / Hkv);
  const size_t rows = static_cast<size_t>(max_runs(groups)) * 16 * groups;
  return cuts_bytes() + 2 * rows * (D + 2) * sizeof(float);
}

cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          bool fp8, cudaStream_t st) {
  if (a.D == 64)
    return fp8 ? launch_d<64, true>(a, kmap, vmap, st) : launch_d<64, false>(a, kmap, vmap, st);
  return fp8 ? launch_d<128, true>(a, kmap, vmap, st) : launch_d<128, false>(a, kmap, vmap, st);
}

}  // namespace sa
