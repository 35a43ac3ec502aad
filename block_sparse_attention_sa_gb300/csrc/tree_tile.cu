// tree_tile.cu -- attention of a tree of new tokens over the paged cache where more than
// 16 rows (pairs of a new token and a query head) share a key-value head: tcgen05.
//   l_u = scale q.k_u,  a = softmax(l),  o = sum a_u v_u,  lse = log sum exp l
//
// Tiles. A CTA holds 128 rows (tcgen05 M = 128) and walks a run of pages, two (128 keys)
// a step. The list of all (sequence, key-value head) units' steps is cut into equal runs,
// as decode_kernel.cuh cuts its pages; grid (runs, row tiles), so that the tiles of one
// unit walk the same pages side by side and all but the first find them in L2. A unit
// that is cut leaves partial results, which tile_join_kernel adds in order.
//
// Pipeline, as in attn.cu: TMEM holds three S buffers and one O accumulator. S(j) = Q K(j)^T
// goes to buffer j % 3; the softmax turns it into P over the same columns; O += P V(j).
// K is K-major as the page lies (rows of d), and so is V as an MN-major operand (rows of
// keys): no transpose, no repacking. S runs up to two steps ahead of P.
// P as two terms of 16 bits, high and low, each 64 columns: both fit the buffer that S
// leaves. Bf16 terms are cut, not rounded, and 2^-24 of the weight is added to what is
// left, so that both are positive and an infinite value stays one; weights to 2^-16.
// Over a cache in e4m3 the terms are fp16 of 2^5 p (weights to 2^-21 of themselves or
// 2^-30 of the largest), against codes turned into fp16, exact, by a warpgroup of its own
// on their way from TMA's stages to the MMA's.
//
// Softmax. Two warpgroups take the steps in turn, one thread a row. The running maximum
// passes from step to step through shared memory and moves only when a step's exceeds it
// by more than 2^14 (e4m3: 2^10).
//
// Steps that hold new tokens, the last page or a page that is not there are masked bit by
// bit (the ancestors of a row's token, shifted to the page); their warpgroup also takes
// out of V in shared memory, before it hands over P, the rows that do not count and what
// is no finite number among the new tokens' values: a weight of 0 would not silence
// those. Rows that see such a value get it added in the epilogue.
//
// Bounds. 32 sequences of 16 new tokens behind 8,192, 56/8 heads of 128 in bf16, 112 rows a
// unit: 195 us for 1.08 GB, 5.5 TB/s, the memory. 64 new tokens behind 3 x 112,640, 448
// rows: 580 to 597 us in bf16, 1,040 to 1,070 TFLOP/s: the tensor pipe (82% busy), which
// does half as much again for the second term of P; a step's products take 1,536 cycles, a
// step 1,700 to 1,800, at the clock that the power leaves (1.5 to 1.8 GHz). In e4m3 640 to
// 650 us with pauses between the calls, 687 to 695 back to back at the power limit, pipe 60%
// busy: there is room for two steps' keys and values in 16 bits, and the way of each from its
// codes' arrival to the product (wait, read, convert, write, told) is 2,000 cycles.
// With one warp for all products bf16 took 705 us, with 32 keys of the softmax unrolled to
// 128 774 us: a step's code then does not fit the instruction cache. 777 tokens, 64 new
// ones: 17.5 us, the chain lengths, page, queries, scores, weights, output, partial, join.
//
// Warps: 0-3 softmax of even steps, 4-7 of odd ones, 8 pages and loads of K, 9
// and 10 the products, 11 the queries (rows gathered by token and head, for e4m3 scaled by a
// power of two; the first by warps 0-7) and loads of V, 12-15 conversion (e4m3). Every wait is bounded
// (SA_DEV_TIMEOUT).
#include "decode_kernel.cuh"

namespace sa {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int kSBuf = 3;
constexpr int kInfo = 16;            // steps whose pages are remembered
constexpr int kProducer = 8, kScore = 9, kMma = 10, kValue = 11, kConvert = 12;
constexpr int kColO = 384;           // S[b] at columns [128 b, 128 b + 128)
constexpr float kTileShift = 5.f;    // e4m3: P is held as 2^5 p

// A unit's piece of a run, for the roles; steps < 0: no more.
struct Head {
  int b, g, dest, steps, pages, base, fresh, special;
};

// The pages of a step: their ids, how many tokens of each count, and the new token in the
// first slot (-64: none before the second page's end).
struct StepInfo {
  int page[2], live[2], first[2];
  int masked;
};

template <int D, bool kFp8>
struct Tile {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  // The running maximum moves when it is exceeded by this power of two (each move rescales
  // O): fp16 holds 2^5 2^10, bf16 any.
  static constexpr float kRaise = kFp8 ? 10.f : 14.f;
  static constexpr int kRegion = BM * 128;              // 128 bytes of each of 128 rows
  static constexpr int kQBytes = BM * D * 2;
  static constexpr int kTile = BN * D * 2;              // K or V of a step, 16 bits an element
  // Stages of K and of V (steps; D = 64 has room for more), and of what is still in e4m3.
  static constexpr int kK = D == 64 ? 3 : 2, kV = D == 64 || !kFp8 ? 3 : 2;
  static constexpr int kRow = D * (kFp8 ? 1 : 2);       // a token of the cache
  static constexpr int kPageBytes = kBlock * kRow;
  static constexpr int kRaw = kFp8 ? 3 : 0;             // pages of codes of K and as many of V
  static constexpr int oQ = 0, oK = oQ + kQBytes, oV = oK + kK * kTile, oRaw = oV + kV * kTile;
  static constexpr int oBar = oRaw + 2 * kRaw * kPageBytes;
  // barriers
  static constexpr int bHeadFull = 0, bHeadEmpty = 2, bQFull = 4, bQEmpty = 5, bQRaw = 6, bKFull = 7;
  static constexpr int bKEmpty = bKFull + kK, bVFull = bKEmpty + kK, bVEmpty = bVFull + kV;
  static constexpr int bSFull = bVEmpty + kV, bPFull = bSFull + kSBuf, bPvDone = bPFull + kSBuf;
  static constexpr int bTileDone = bPvDone + 2, bOFree = bTileDone + 1, bPvIssued = bOFree + 1;
  static constexpr int bFin = bPvIssued + kSBuf, bInfo = bFin + 2, bRawFull = bInfo + kInfo;
  static constexpr int bRawEmpty = bRawFull + 2 * kRaw, bQFirst = bRawEmpty + 2 * kRaw, kBars = bQFirst + 1;
  static constexpr int oMisc = oBar + kBars * 8;        // tmem base, abort flag, odd values [2]
  static constexpr int oHead = oMisc + 16;
  static constexpr int oInfo = oHead + 2 * static_cast<int>(sizeof(Head));
  static constexpr int oSeen = (oInfo + kInfo * static_cast<int>(sizeof(StepInfo)) + 7) & ~7;   // [2][64]
  static constexpr int oFactor = oSeen + 2 * 64 * 8;    // [2][128]
  static constexpr int oXch = oFactor + 2 * BM * 4;     // [2][2][128] of (m, l, stop)
  static constexpr int oHand = oXch + 2 * 2 * BM * 12;  // [2][128]
  static constexpr int kBytes = oHand + 2 * BM * 8 + 1024;
  static_assert(kBytes <= 227 * 1024, "the tile does not fit shared memory");
  static_assert(oMisc % 8 == 0 && oHand % 8 == 0 && oXch % 4 == 0, "alignment");
};

struct TileCut {
  int unit, first, last, pad;
};

// The MN-major operand of 16 keys of a page of V in the 128-byte swizzle: rows of 128
// bytes (64 d), 8-row atoms of 1,024 bytes along the keys, the next 64 d 8 KB on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(8192 >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
         static_cast<uint64_t>(2) << 61;
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint4 w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}

// 16 bytes to shared memory, zeros without a source.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ bool elected() {
  uint32_t pred = 0;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(pred));
  return pred != 0;
}

// Both pages (-1: none) of a step's K or V in bf16 into a tile, by one lane: all rows of a
// slice of 64 d follow each other in K, a page's slices in V.
template <int D, bool kValues>
__device__ __forceinline__ void load_tile(const CUtensorMap* map, uint32_t f, uint32_t dst, int pa, int pb, int g) {
  constexpr uint32_t kSlice = kValues ? kBlock * 128 : BM * 128, kNext = kValues ? kBlock * D * 2 : kBlock * 128;
  if (elected()) {
    const int bytes = ((pa >= 0) + (pb >= 0)) * (kBlock * D * 2);
    if (bytes > 0)
      mbar_arrive_expect_tx(f, bytes);
    else
      mbar_arrive(f);
    if (pa >= 0) {
      tma_load_4d(dst, map, f, 0, 0, g, pa);
      if (D == 128) tma_load_4d(dst + kSlice, map, f, 64, 0, g, pa);
    }
    if (pb >= 0) {
      tma_load_4d(dst + kNext, map, f, 0, 0, g, pb);
      if (D == 128) tma_load_4d(dst + kNext + kSlice, map, f, 64, 0, g, pb);
    }
  }
  __syncwarp();
}

// a b + c with subnormal numbers as they are: the factor of a row of small queries may be
// one, and a masked logit of -inf times 0 would be NaN.
__device__ __forceinline__ uint64_t fma2_subnormal(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// p = 2^((s - m) f) for 32 logits as two terms, pairs of keys in a word (e4m3: of 2^5 p);
// returns the sum of the p. Subtracting before scaling, the largest key has weight 1
// however coarse fp32 is at its logit's size.
template <bool kFp8>
__device__ __forceinline__ float weigh32(const uint32_t* v, float m, float f, uint32_t* hi, uint32_t* lo) {
  const uint64_t nm = f2_pack(-m, -m), ff = f2_pack(f, f);
  const uint64_t add = kFp8 ? f2_pack(kTileShift, kTileShift) : 0ull;
  const uint64_t minus = f2_pack(-1.f, -1.f), more = f2_pack(1.f + 0x1p-23f, 1.f + 0x1p-23f);
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int u = 0; u < 32; u += 2) {
    const uint64_t d = f2_add(f2_pack(__uint_as_float(v[u]), __uint_as_float(v[u + 1])), nm);
    float y0, y1;
    f2_unpack(fma2_subnormal(d, ff, add), y0, y1);
    const float p0 = fast_exp2(y0), p1 = fast_exp2(y1);
    const uint64_t p = f2_pack(p0, p1);
    acc[(u >> 1) & 1] = f2_add(acc[(u >> 1) & 1], p);
    float r0, r1;
    if (kFp8) {
      const uint32_t h = pack_half(p0, p1);
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
      hi[u >> 1] = h;
      f2_unpack(f2_fma(f2_pack(b.x, b.y), minus, p), r0, r1);
      lo[u >> 1] = pack_half(r0, r1);
    } else {
      hi[u >> 1] = top_bf16(p0, p1);
      // less what the high term holds, and 2^-23 of the weight more
      const float n0 = __uint_as_float((__float_as_uint(p0) & 0xffff0000u) | 0x80000000u);
      const float n1 = __uint_as_float((__float_as_uint(p1) & 0xffff0000u) | 0x80000000u);
      f2_unpack(f2_fma(p, more, f2_pack(n0, n1)), r0, r1);
      lo[u >> 1] = pack_bf16(r0, r1);
    }
  }
  float a, b;
  f2_unpack(f2_add(acc[0], acc[1]), a, b);
  return a + b;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// O += P V of 64 keys, one term of P: 16 keys are 8 of its columns (32 keys each 32 columns
// of the buffer: the high term's 16, the low one's) and 2 KB of V.
__device__ __forceinline__ void pv_elect(uint32_t o_tmem, uint32_t p_tmem, uint64_t v0, uint64_t v1, uint64_t v2,
                                         uint64_t v3, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b32 a1, a2, a3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "setp.eq.b32 t, %7, %7;\n\t"
      "add.u32 a1, %1, 8;\n\t"
      "add.u32 a2, %1, 32;\n\t"
      "add.u32 a3, %1, 40;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %6, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %3, %6, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], %4, %6, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], %5, %6, t;\n\t}"
      ::"r"(o_tmem), "r"(p_tmem), "l"(v0), "l"(v1), "l"(v2), "l"(v3), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ float max32(const uint32_t* v) {
  float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; i += 4)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      m[c] = fmax3(m[c], __uint_as_float(v[i + 2 * c]), __uint_as_float(v[i + 2 * c + 1]));
  return fmaxf(m[0], m[1]);
}

__device__ __forceinline__ void keep32(uint32_t* v, uint32_t bits) {
#pragma unroll
  for (int u = 0; u < 32; ++u)
    if (!(bits >> u & 1)) v[u] = __float_as_uint(-INFINITY);
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(Tile<D, kFp8>::kThreads, 1)
tree_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const DecodeArgs a, float* partial, TileCut* cuts) {
  using L = Tile<D, kFp8>;
  constexpr unsigned full = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.H / a.Hkv, rt = blockIdx.y, run_id = blockIdx.x, runs = gridDim.x;
  const bool routed = a.row_ptr != nullptr;
  const int n_groups = routed ? a.B * a.Hkv : a.B, per_group = routed ? 1 : a.Hkv;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::oMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* odd_seen = reinterpret_cast<volatile int*>(misc + 2);
  const AbortSignal abort{abort_flag, nullptr};
  const volatile int never_flag = 0;
  const AbortSignal drain{&never_flag, nullptr};
  volatile Head* heads = reinterpret_cast<volatile Head*>(smem + L::oHead);
  volatile StepInfo* infos = reinterpret_cast<volatile StepInfo*>(smem + L::oInfo);
  volatile uint64_t* seen_sets = reinterpret_cast<volatile uint64_t*>(smem + L::oSeen);
  volatile float* factors = reinterpret_cast<volatile float*>(smem + L::oFactor);
  auto bar = [&](int i) { return sbase + L::oBar + 8u * static_cast<uint32_t>(i); };
  auto fail = [&]() {
    *abort_flag = 1;
    if (a.dev_status) atomicOr(a.dev_status, SA_DEV_TIMEOUT);
  };
  int status = 0;
  let_next_launch();
  for (int i = tid; i < L::kBars; i += L::kThreads) {      // one by one they take 1,000 cycles
    uint32_t n = 1;
    if (i >= L::bHeadEmpty && i < L::bHeadEmpty + 2) n = 2 + 8 + 1;     // products, softmax, queries and V
    if (i >= L::bPFull && i < L::bPFull + kSBuf) n = 128;
    if (i == L::bOFree) n = 256;
    if (kFp8 && i == L::bQFull) n = 4;     // converting warps
    if (kFp8 && ((i >= L::bKFull && i < L::bKEmpty) || (i >= L::bVFull && i < L::bVEmpty) || (i >= L::bRawEmpty && i < L::bQFirst)))
      n = 2;                               // converting warps
    if (i == L::bQFirst) n = 8;            // softmax warps
    mbar_init(bar(i), n);
    fence_barrier_init();
  }
  if (tid == 0) {
    *abort_flag = 0;
    odd_seen[0] = odd_seen[1] = 0;
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (tid < 256) reinterpret_cast<uint64_t*>(smem + L::oHand)[tid] = 0xffffffff00000000ull;
  if (warp == kMma) {
    tmem_alloc(sbase + L::oMisc, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  // this CTA's run of the list of steps of the sequences that have rows in this tile
  const Run run = plan_run<L::kThreads>(n_groups, per_group, [&](int i, int* from) {
    const int pages = group_pages<true>(a, i, from, &status);
    int base, none;
    const int fresh = new_tokens(a, routed ? i / a.Hkv : i, &base, &none);
    return static_cast<int64_t>(fresh) * G > rt * BM ? (pages + 1) / 2 : 0;
  });
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int total_steps = run.hi - run.lo;

  // K's or V's pages (-1: none) of the next step into its ring: tiles of bf16, or pages of
  // codes that have yet to be turned into fp16. Addresses and pages are in registers: read
  // from shared memory box by box they took 1,500 cycles a tile, and the kernel's pace.
  auto load_step = [&](bool values, int& st, int& ph, int& filled, int pa, int pb, int g) -> bool {
    if constexpr (!kFp8) {
      if (!mbar_wait_warp(bar((values ? L::bVEmpty : L::bKEmpty) + st), ph, abort)) return false;
      if (values)
        load_tile<D, true>(&vmap, bar(L::bVFull + st), sbase + L::oV + st * L::kTile, pa, pb, g);
      else
        load_tile<D, false>(&kmap, bar(L::bKFull + st), sbase + L::oK + st * L::kTile, pa, pb, g);
      ++filled;
      if (++st == (values ? L::kV : L::kK)) {
        st = 0;
        ph ^= 1;
      }
    } else {
      for (int kh = 0; kh < 2; ++kh) {
        const int at = (values ? L::kRaw : 0) + st, page = kh ? pb : pa;
        if (!mbar_wait_warp(bar(L::bRawEmpty + at), ph, abort)) return false;
        if (elected()) {
          const uint32_t f = bar(L::bRawFull + at);
          if (page >= 0) {
            mbar_arrive_expect_tx(f, L::kPageBytes);
            tma_load_4d(sbase + L::oRaw + at * L::kPageBytes, values ? &vmap : &kmap, f, 0, 0, g, page);
          } else {
            mbar_arrive(f);
          }
        }
        __syncwarp();
        ++filled;
        if (++st == L::kRaw) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    return true;
  };
  // no copy may be in flight when the CTA ends
  auto drain_loads = [&](bool values, int filled) {
    const int n = kFp8 ? L::kRaw : (values ? L::kV : L::kK);
    const int f = kFp8 ? L::bRawFull + (values ? L::kRaw : 0) : (values ? L::bVFull : L::bKFull);
    for (int s = 0; s < n && s < filled; ++s)       // the fills of stage s before its last one
      mbar_wait(bar(f + s), (filled - 1 - s) / n & 1, drain);
  };

  // A piece's queries, all rows on their way at once, straight to where the MMA reads them,
  // by `threads` threads of which this is the t-th: those of the first piece by the softmax
  // warps, which have nothing else to do (64 new tokens behind 777: 17.5 us, by one warp
  // 18.3), later ones by the warp that loads V, while the piece before is still at work.
  auto load_queries = [&](int x, int t, int threads) {
    constexpr int kLanes = D / 8;                     // threads of a row
    const int once = threads / kLanes, sub = t % kLanes, r0 = t / kLanes;
    const int b = heads[x].b, g = heads[x].g, rows = heads[x].fresh * G;
    const int first = rt * BM + r0, d_tok = once / G, d_head = once - d_tok * G;
    const int64_t step = d_tok * a.qs[1] + d_head * a.qs[2], wrap = a.qs[1] - G * a.qs[2];
    int head = first % G, left = rows - first;        // rows from this one on
    const uint16_t* src = a.q + b * a.qs[0] + first / G * a.qs[1] + (g * G + head) * a.qs[2] + 8 * sub;
    uint32_t dst = sbase + L::oQ + (sub >> 3) * L::kRegion + r0 * 128;
#pragma unroll 4
    for (int r = r0; r < BM; r += once) {
      copy_16(dst + (((sub & 7) ^ (r & 7)) << 4), left > 0 ? src : a.q, left > 0);
      if (!kFp8 && sub == 0) factors[x * BM + r] = a.scale_log2;
      src += step;
      head += d_head;
      if (head >= G) {
        head -= G;
        src += wrap;
      }
      dst += once * 128;
      left -= once;
    }
  };
  // e4m3: QFull is told by the converting warps, for every piece
  auto queries_there = [&](int it) {
    if (kFp8) return mbar_wait_warp(bar(L::bQFull), it & 1, abort);
    return it == 0 ? mbar_wait_warp(bar(L::bQFirst), 0, abort) : mbar_wait_warp(bar(L::bQFull), (it - 1) & 1, abort);
  };
  auto load_ancestors = [&](int x) {
    uint64_t set[2];
    ancestors(a, heads[x].b, heads[x].fresh, lane, set, &status);
    seen_sets[x * 64 + lane] = set[0];
    seen_sets[x * 64 + 32 + lane] = set[1];
  };
  auto finish_queries = [&](int i) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };

  if (warp == kProducer) {
    // ---------------------------------------------------------- producer --
    int left = total_steps, group = run.group, off = run.off, cnt = run.count;
    int it = 0, gstep = 0;
    int k_st = 0, k_ph = 1, filled = 0;   // the next stage of K (e4m3: page of codes)
    TileCut cut{-1, 0, 0, 0};
    bool ok = true;
    while (left > 0 && ok && group < n_groups) {
      int from;
      const int pages = group_pages<true>(a, group, &from, &status);
      if (off >= cnt * per_group) {
        off = 0;
        if (++group < n_groups) {
          int base, none;
          const int fresh = new_tokens(a, routed ? group / a.Hkv : group, &base, &none);
          cnt = static_cast<int64_t>(fresh) * G > rt * BM
                    ? (group_pages<true>(a, group, &from, &status) + 1) / 2 : 0;
        }
        continue;
      }
      const int sub = off < cnt ? 0 : off / cnt, s0 = off - sub * cnt, take = min(left, cnt - s0);
      const int b = routed ? group / a.Hkv : group, g = routed ? group - b * a.Hkv : sub;
      int base;
      const int fresh = new_tokens(a, b, &base, &status);
      const int n = base + fresh, nb = (n + kBlock - 1) / kBlock, own = base / kBlock;
      const int entries = pages - (nb - own);
      const int dest = take == cnt ? -1 : (s0 == 0 ? 1 : 0);
      const int p0 = 2 * s0, n_pages = min(2 * take, pages - p0);
      const int x = it & 1;
      if (it >= 2 && !mbar_wait_warp(bar(L::bHeadEmpty + x), ((it >> 1) - 1) & 1, abort)) {
        if (lane == 0) fail();
        break;
      }
      if (lane == 0) {
        volatile Head* h = heads + x;
        h->b = b;
        h->g = g;
        h->dest = dest;
        h->steps = take;
        h->pages = n_pages;
        h->base = base;
        h->fresh = fresh;
        h->special = routed ? p0 + n_pages > entries : p0 + n_pages > own;
        odd_seen[x] = 0;
        mbar_arrive(bar(L::bHeadFull + x));
      }
      __syncwarp();
      if (dest == 1)
        cut = TileCut{b * a.Hkv + g, run_id, run_of(run.T, runs, run.hi - left + cnt - 1), 0};
      // Loads of a step's two pages. (Addresses and pages in registers: this warp's own
      // pace, with its pages read from shared memory 1,500 cycles a tile, was the kernel's.)
      int pg = 0, lv = 0, fs = 0;         // 32 pages that were looked up, a lane each
      for (int j = 0; j < take && ok; ++j) {
        int ka, kb;
        {
          const int q = 2 * j % 32;
          if (q == 0) {                   // the next 32 pages are looked up
            const int at = 2 * j + lane;
            pg = -1;
            lv = 0;
            fs = -kBlock;
            if (at < n_pages) {
              int p = p0 + at;
              if (routed && p >= entries) {
                p += own - entries;
              } else if (routed) {
                const int c = from + p;
                const bool there = from >= 0 && c < a.col_cap;
                const int prev = there && p > 0 ? get(a.col_idx + c - 1) : -1;
                p = there ? get(a.col_idx + c) : -1;
                if (p < 0 || p >= nb || p <= prev) {
                  status |= SA_DEV_BAD_ROUTE;
                  p = -1;
                }
                if (p >= own) p = -1;
              }
              if (p >= 0) {
                pg = get(a.pm.table + b * a.pm.table_stride + p);
                lv = min(kBlock, n - p * kBlock);
                fs = max(p * kBlock - base, -kBlock);
                if (pg < 0 || pg >= a.pm.n_pages) {
                  status |= SA_DEV_BAD_CACHE;
                  lv = 0;
                }
              }
              if (lv <= 0) pg = -1;
            }
          }
          ka = __shfl_sync(full, pg, q);
          kb = __shfl_sync(full, pg, q + 1);
          const int lv0 = __shfl_sync(full, lv, q), lv1 = __shfl_sync(full, lv, q + 1);
          const int fs0 = __shfl_sync(full, fs, q), fs1 = __shfl_sync(full, fs, q + 1);
          if (lane == 0) {
            volatile StepInfo* in = infos + (gstep + j) % kInfo;
            in->page[0] = ka;
            in->page[1] = kb;
            in->live[0] = lv0;
            in->live[1] = lv1;
            in->first[0] = fs0;
            in->first[1] = fs1;
            in->masked = lv0 < kBlock || fs0 > -kBlock || (2 * j + 1 < n_pages && (lv1 < kBlock || fs1 > -kBlock));
            mbar_arrive(bar(L::bInfo + (gstep + j) % kInfo));
          }
          __syncwarp();
        }
        ok = load_step(false, k_st, k_ph, filled, ka, kb, g);
      }
      if (!ok) {
        if (lane == 0) fail();
        break;
      }
      gstep += take;
      off += take;
      left -= take;
      ++it;
    }
    // no more units
    const int x = it & 1;
    if (it >= 2 && !mbar_wait_warp(bar(L::bHeadEmpty + x), ((it >> 1) - 1) & 1, abort)) {
      if (lane == 0) fail();
    } else if (lane == 0) {
      heads[x].steps = -1;
      mbar_arrive(bar(L::bHeadFull + x));
    }
    if (lane == 0) {
      cuts[static_cast<int64_t>(rt) * runs + run_id] = cut;
      drain_loads(false, filled);
    }
  } else if (warp == kScore) {
    // ------------------------------------------------------------ Q K^T --
    // Two warps feed the tensor pipe, one the scores, one the outputs. It takes products a
    // few ahead of the one it works on, and a warp's waits, commits and 50 cycles a product
    // (of 64) add up to 2,200 cycles a step of 1,536. S of step g takes the buffer of step
    // g - 3 once that one's PV is issued; the fences order the two warps' products.
    constexpr uint32_t kIdQK128 = idesc_f16(BM, 128, kFp8 ? 0 : 1), kIdQK64 = idesc_f16(BM, 64, kFp8 ? 0 : 1);
    constexpr int kKS = D / 16;
    uint64_t qd[kKS];
#pragma unroll
    for (int k = 0; k < kKS; ++k)
      qd[k] = sdesc_kmajor_sw128(sbase + L::oQ + (k >> 2) * L::kRegion + (k & 3) * 32);
    const uint64_t kd = sdesc_kmajor_sw128(sbase + L::oK);
    int g = 0, sb = 0, sb_ph = 1, st = 0, ph = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int x = it & 1;
      ok = mbar_wait_warp(bar(L::bHeadFull + x), (it >> 1) & 1, abort);
      if (!ok) break;
      const int n = heads[x].steps, n_pages = heads[x].pages;
      if (n < 0) break;
      ok = queries_there(it);
      for (int j = 0; j < n && ok; ++j) {
        ok = mbar_wait_warp(bar(L::bKFull + st), ph, abort) &&
             (g < kSBuf || mbar_wait_warp(bar(L::bPvIssued + sb), sb_ph, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = 2 * j + 1 < n_pages ? kIdQK128 : kIdQK64;
        const uint64_t kb = kd + static_cast<uint64_t>(st * (L::kTile >> 4));
#pragma unroll
        for (int h = 0; h < kKS / 4; ++h) {
          const uint64_t k0 = kb + static_cast<uint64_t>((h * L::kRegion) >> 4);
          umma_ss_x4_elect(tmem + sb * 128, qd[4 * h], qd[4 * h + 1], qd[4 * h + 2], qd[4 * h + 3], k0, k0 + 2,
                           k0 + 4, k0 + 6, idesc, h > 0);
        }
        umma_commit_elect(bar(L::bSFull + sb));
        umma_commit_elect(bar(L::bKEmpty + st));
        if (j == n - 1) umma_commit_elect(bar(L::bQEmpty));
        ++g;
        if (++st == L::kK) {
          st = 0;
          ph ^= 1;
        }
        if (++sb == kSBuf) {
          sb = 0;
          sb_ph ^= 1;
        }
      }
      if (ok && elected()) mbar_arrive(bar(L::bHeadEmpty + x));
    }
    if (!ok && lane == 0) fail();
    umma_commit_elect(bar(L::bFin));
    mbar_wait_warp(bar(L::bFin), 0, drain);
  } else if (warp == kMma) {
    // --------------------------------------------------------------- P V --
    constexpr uint32_t kIdPV = idesc_f16(BM, D, kFp8 ? 0 : 1) | (1u << 16);      // B is MN-major
    const uint64_t vd = sdesc_mn_sw128(sbase + L::oV);
    const uint32_t o_tmem = tmem + kColO;
    int g = 0, sb = 0, sb_ph = 0, st = 0, ph = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int x = it & 1;
      ok = mbar_wait_warp(bar(L::bHeadFull + x), (it >> 1) & 1, abort);
      if (!ok) break;
      const int n = heads[x].steps, n_pages = heads[x].pages;
      if (n < 0) break;
      // the last piece's epilogue has read O
      ok = it == 0 || mbar_wait_warp(bar(L::bOFree), (it - 1) & 1, abort);
      for (int j = 0; j < n && ok; ++j) {
        bool unused = false;
        ok = mbar_wait2_warp(bar(L::bPFull + sb), sb_ph, bar(L::bVFull + st), ph, false, 0u, 0u, &unused, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t pa = tmem + sb * 128;
        const uint64_t v0 = vd + static_cast<uint64_t>(st * (L::kTile >> 4));
        // 16 keys are 2 KB of rows
        pv_elect(o_tmem, pa, v0, v0 + 128, v0 + 256, v0 + 384, kIdPV, j > 0);
        pv_elect(o_tmem, pa + 16, v0, v0 + 128, v0 + 256, v0 + 384, kIdPV, 1u);
        if (2 * j + 1 < n_pages) {
          const uint64_t v1 = v0 + (kBlock * D * 2 >> 4);
          pv_elect(o_tmem, pa + 64, v1, v1 + 128, v1 + 256, v1 + 384, kIdPV, 1u);
          pv_elect(o_tmem, pa + 80, v1, v1 + 128, v1 + 256, v1 + 384, kIdPV, 1u);
        }
        umma_commit_elect(bar(L::bVEmpty + st));
        umma_commit_elect(bar(L::bPvDone + (g & 1)));
        // behind the commits: S(g + 3) is there only after PV(g) has been told done
        tc_fence_before();
        if (elected()) mbar_arrive(bar(L::bPvIssued + sb));
        ++g;
        if (++st == L::kV) {
          st = 0;
          ph ^= 1;
        }
        if (++sb == kSBuf) {
          sb = 0;
          sb_ph ^= 1;
        }
      }
      if (!ok) break;
      umma_commit_elect(bar(L::bTileDone));
      if (elected()) mbar_arrive(bar(L::bHeadEmpty + x));
    }
    if (!ok && lane == 0) fail();
    umma_commit_elect(bar(L::bFin + 1));
    mbar_wait_warp(bar(L::bFin + 1), 0, drain);
  } else if (warp == kValue) {
    // ---------------------------------------- queries, then loads of V --
    int st = 0, ph = 1, gv = 0, filled = 0;
    bool ok = true;
    for (int it = 0; ok; ++it) {
      const int x = it & 1;
      ok = mbar_wait_warp(bar(L::bHeadFull + x), (it >> 1) & 1, abort);
      if (!ok) break;
      const int n = heads[x].steps, g = heads[x].g;
      if (n < 0) break;
      ok = it == 0 || mbar_wait_warp(bar(L::bQEmpty), (it - 1) & 1, abort);
      if (!ok) break;
      if (it > 0) {
        load_queries(x, lane, 32);
        if (heads[x].special) load_ancestors(x);
        finish_queries(kFp8 ? L::bQRaw : L::bQFull);
      }
      for (int j = 0; j < n && ok; ++j, ++gv) {
        const volatile StepInfo* in = infos + gv % kInfo;
        ok = mbar_wait_warp(bar(L::bInfo + gv % kInfo), (gv / kInfo) & 1, abort);
        if (ok) ok = load_step(true, st, ph, filled, in->page[0], in->page[1], g);
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar(L::bHeadEmpty + x));
    }
    if (!ok && lane == 0) fail();
    if (lane == 0) drain_loads(true, filled);
  } else if (kFp8 && warp >= kConvert) {
    // -------------------------------------------------------- conversion --
    // Two warps turn K into fp16, two V: a thread two rows (tokens) of each. As read, so
    // written, without bank conflicts, as the rows' pieces are swizzled alike. A page's codes
    // are read before the wait for the tile's place (when that was tried, 3 x 64 new tokens
    // behind 112,640 took 676 us so; waiting first 713; both pages' codes at once 756; all four
    // warps for K, then V 810).
    // Their stage is given back only behind the stores, which need the loads' results: an
    // arrival may pass loads that are still under way.
    const bool values = warp >= kConvert + 2;
    const int row = tid & 63, raw0 = values ? L::kRaw : 0;
    constexpr int NR = kFp8 ? L::kRaw : 1;
    bool ok = true;
    int it = 0, last = 0;                       // the next piece, and where the last one ends
    for (int g = 0; g < total_steps && ok; ++g) {
      if (g == last) {
        // a piece begins: its queries
        const int x = it & 1;
        ok = mbar_wait_warp(bar(L::bHeadFull + x), (it >> 1) & 1, abort);
        if (!ok || heads[x].steps < 0) break;
        last += heads[x].steps;
        const float scale = a.scale_log2 * (a.k_scale ? get(a.k_scale + heads[x].g) : 1.f);
        ok = it == 0 ? mbar_wait_warp(bar(L::bQFirst), 0, abort) : mbar_wait_warp(bar(L::bQRaw), (it - 1) & 1, abort);
        if (!ok) break;
        constexpr int kLanes = D / 8, kRowsOnce = 32 / kLanes;
        const int sub = lane % kLanes, r0 = (warp - kConvert) * 32 + lane / kLanes;
        // in fp16, a row scaled by a power of two so that its largest element is in
        // [2^14, 2^15): bits are lost only below 2^-39 of it
#pragma unroll 1
        for (int i = 0; i < 32; i += 4 * kRowsOnce) {      // four at once
          uint4 w[4];
          float top[4];
          auto at = [&](int u) {
            const int r = r0 + i + u * kRowsOnce;
            return sbase + L::oQ + (sub >> 3) * L::kRegion + r * 128 + (((sub & 7) ^ (r & 7)) << 4);
          };
#pragma unroll
          for (int u = 0; u < 4; ++u) w[u] = load_shared(at(u));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* e = &w[u].x;
            top[u] = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) top[u] = fmaxf(top[u], fmaxf(fabsf(lo_f32(e[y])), fabsf(hi_f32(e[y]))));
          }
#pragma unroll
          for (int s = kLanes / 2; s >= 1; s >>= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) top[u] = fmaxf(top[u], __shfl_xor_sync(full, top[u], s));
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            // its exponent; beyond 2^127 a row next to the least floats is scaled by that
            const int ex = top[u] < INFINITY ? min(141 - static_cast<int>(__float_as_uint(top[u]) >> 23), 127) : 0;
            const float up = power_of_two(ex);
            float f = scale * power_of_two(-(ex / 2)) * power_of_two(-(ex - ex / 2));
            if (f == 0.f) f = 0x1p-149f;
            if (sub == 0) factors[x * BM + r0 + i + u * kRowsOnce] = f;
            uint32_t* e = &w[u].x;
#pragma unroll
            for (int y = 0; y < 4; ++y) e[y] = pack_half(lo_f32(e[y]) * up, hi_f32(e[y]) * up);
            store_shared(at(u), w[u]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bQFull));
        ++it;
      }
      const int st = values ? g % L::kV : g % L::kK, round = values ? g / L::kV : g / L::kK;
#pragma unroll 1
      for (int kh = 0; kh < 2 && ok; ++kh) {
        const int c = 2 * g + kh, rs = raw0 + c % NR;
        ok = mbar_wait_warp(bar(L::bRawFull + rs), (c / NR) & 1, abort);
        const uint32_t src = sbase + L::oRaw + rs * L::kPageBytes;
        const uint32_t dst = sbase + (values ? L::oV + st * L::kTile + kh * (kBlock * D * 2)
                                             : L::oK + st * L::kTile + kh * 8192) + row * 128;
        const uint32_t slice = values ? 8192 : L::kRegion;
        constexpr int kPieces = D / 16;           // of a row of codes
        uint4 w[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
          w[p] = load_shared(src + (D == 64 ? row * 64 + ((p ^ ((row >> 1) & 3)) << 4) : row * 128 + ((p ^ (row & 7)) << 4)));
        if (kh == 0 && ok) ok = mbar_wait_warp(bar((values ? L::bVEmpty : L::bKEmpty) + st), (round & 1) ^ 1, abort);
        if (!ok) break;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const uint2 h0 = e4m3x4_half4(w[p].x), h1 = e4m3x4_half4(w[p].y), h2 = e4m3x4_half4(w[p].z), h3 = e4m3x4_half4(w[p].w);
          const uint32_t c0 = (p & 3) * 2, to = dst + (p >> 2) * slice;
          store_shared(to + ((c0 ^ (row & 7)) << 4), make_uint4(h0.x, h0.y, h1.x, h1.y));
          store_shared(to + (((c0 + 1) ^ (row & 7)) << 4), make_uint4(h2.x, h2.y, h3.x, h3.y));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bRawEmpty + rs));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar((values ? L::bVFull : L::bKFull) + st));
    }
    if (!ok && lane == 0) fail();
  } else {
    // ----------------------------------------------------------- softmax --
    const int sm = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t pair_bar = 1 + quarter;
    float* xm = reinterpret_cast<float*>(smem + L::oXch);
    float* xl = xm + 4 * BM;
    int* xs = reinterpret_cast<int*>(xl + 4 * BM);
    volatile uint64_t* hand = reinterpret_cast<volatile uint64_t*>(smem + L::oHand);
    volatile uint64_t* hand_mine = hand + sm * BM + r;
    const volatile uint64_t* hand_theirs = hand + (sm ^ 1) * BM + r;
    int xc = 0;
    auto pair_xchg = [&](float m, float l, bool stop, float& m_o, float& l_o) -> bool {
      const int sl = xc & 1;
      ++xc;
      const int mine = (sl * 2 + sm) * BM + r, theirs = (sl * 2 + (sm ^ 1)) * BM + r;
      xm[mine] = m;
      xl[mine] = l;
      xs[mine] = stop ? 1 : 0;
      named_bar_sync(pair_bar, 64);
      m_o = xm[theirs];
      l_o = xl[theirs];
      return stop || xs[theirs] != 0;
    };
    auto wait_handoff = [&](int g_prev, uint64_t& hv) -> bool {
      hv = *hand_theirs;
      if (__all_sync(full, static_cast<int>(hv >> 32) >= g_prev)) return true;
      unsigned long long t0 = 0;
      if (lane == 0) t0 = globaltimer();
      for (uint32_t i = 1;; ++i) {
        hv = *hand_theirs;
        if (__all_sync(full, static_cast<int>(hv >> 32) >= g_prev)) return true;
        if ((i & 63u) == 0u) {
          int give_up = 0;
          if (lane == 0) give_up = abort.raised() || (globaltimer() - t0 > kWaitTimeoutNs);
          if (__shfl_sync(full, give_up, 0)) return false;
        }
      }
    };
    int gs = 0;
    for (int it = 0;; ++it) {
      const int x = it & 1;
      bool stop = !mbar_wait_warp(bar(L::bHeadFull + x), (it >> 1) & 1, abort);
      if (stop && lane == 0) fail();
      float u0, u1;
      if (pair_xchg(0.f, 0.f, stop, u0, u1)) break;
      const int n = heads[x].steps;
      if (n < 0) break;
      const int b = heads[x].b, g = heads[x].g, dest = heads[x].dest, n_pages = heads[x].pages;
      const int n_rows = heads[x].fresh * G, row = rt * BM + r;
      const bool special = heads[x].special != 0;
      if (it == 0) {
        load_queries(x, tid, 256);
        if (warp == 0 && special) load_ancestors(x);
        finish_queries(L::bQFirst);
      }
      stop = !queries_there(it);                        // and the rows' factors
      if (stop && lane == 0) fail();
      const float f = factors[x * BM + r];
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = (gs ^ sm) & 1; j < n && !stop; j += 2) {
        const int gg = gs + j, sb = gg % kSBuf;
        const uint32_t s_col = sb * 128;
        const bool two = 2 * j + 1 < n_pages;
        volatile StepInfo* in = infos + gg % kInfo;
        if (!mbar_wait_warp(bar(L::bInfo + gg % kInfo), (gg / kInfo) & 1, abort)) {
          stop = true;
          break;
        }
        const bool masked = in->masked != 0;
        if (!mbar_wait_warp(bar(L::bSFull + sb), (gg / kSBuf) & 1, abort)) {
          stop = true;
          break;
        }
        if (masked) {
          // V's rows that do not count, and among the new tokens what is no finite number
          // (a barrier tells a phase from the next only: the stage's last use, of step gg - 2
          // or before, has to be over, and for that one, as S(gg) is there, step gg - 4's is)
          const int st = gg % L::kV;
          if ((gg >= 2 && !mbar_wait_warp(bar(L::bPvDone + (gg & 1)), ((gg - 2) >> 1) & 1, abort)) ||
              !mbar_wait_warp(bar(L::bVFull + st), (gg / L::kV) & 1, abort)) {
            stop = true;
            break;
          }
          const int kh = r >> 6, key = r & 63;
          if (kh == 0 || two) {
            const int lv = in->live[kh], fs = in->first[kh];
            const uint32_t v = sbase + L::oV + st * L::kTile + kh * (kBlock * D * 2) + key * 128;
            if (key >= lv) {
#pragma unroll 4
              for (int p = 0; p < D / 8; ++p)
                store_shared(v + (p >> 3) * 8192 + (((p & 7) ^ (key & 7)) << 4), make_uint4(0u, 0u, 0u, 0u));
            } else if (fs + key >= 0) {
              constexpr uint32_t kOdd = kFp8 ? 0x7c00u : 0x7f80u;
              bool odd = false;
#pragma unroll 4
              for (int p = 0; p < D / 8; ++p) {
                const uint32_t at = v + (p >> 3) * 8192 + (((p & 7) ^ (key & 7)) << 4);
                uint4 w = load_shared(at);
                uint32_t* e = &w.x;
                bool here = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  if ((e[i] & kOdd) == kOdd) {
                    e[i] &= 0xffff0000u;
                    here = true;
                  }
                  if ((e[i] >> 16 & kOdd) == kOdd) {
                    e[i] &= 0xffffu;
                    here = true;
                  }
                }
                if (here) store_shared(at, w);
                odd |= here;
              }
              if (odd) odd_seen[x] = 1;
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_after();
        // the step's maximum, 64 keys at a time (masked: by bits, and written back so)
        const uint32_t s_addr = lane_base + s_col;
        const int groups = two ? 4 : 2;
        float bmax = -INFINITY;
        if (!masked) {
#pragma unroll 1
          for (int c = 0; c < groups; c += 2) {
            uint32_t sr[64];
            float mx0, mx1;
            tmem_ld32_max(s_addr + 32 * c, sr, mx0);
            tmem_ld32_max(s_addr + 32 * c + 32, sr + 32, mx1);
            tmem_wait_ld();
            reg_fence64(sr);
            reg_fence_f(mx0);
            reg_fence_f(mx1);
            bmax = fmax3(bmax, mx0, mx1);
          }
        } else {
          const uint64_t set = special ? seen_sets[x * 64 + min(row / G, 63)] : 0ull;
#pragma unroll 1
          for (int c = 0; c < groups; ++c) {
            const int lv = in->live[c >> 1], fs = in->first[c >> 1];
            uint64_t keep = lv >= kBlock ? ~0ull : (1ull << lv) - 1;
            if (fs > -kBlock) keep &= slots_seen(set, fs);
            uint32_t sr[32];
            tmem_ld32(s_addr + 32 * c, sr);
            tmem_wait_ld();
            reg_fence32(sr);
            keep32(sr, static_cast<uint32_t>(keep >> (32 * (c & 1))));
            bmax = fmaxf(bmax, max32(sr));
            tmem_st32(s_addr + 32 * c, sr);
          }
          tmem_wait_st();
        }
        float m_prev = -INFINITY;
        if (j > 0) {
          uint64_t hv;
          if (!wait_handoff(gg - 1, hv)) {
            stop = true;
            break;
          }
          m_prev = __uint_as_float(static_cast<uint32_t>(hv));
        }
        float m_new = m_prev;
        if (m_prev == -INFINITY || (bmax - m_prev) * f > L::kRaise) m_new = fmaxf(bmax, m_prev);
        *hand_mine = (static_cast<uint64_t>(static_cast<uint32_t>(gg)) << 32) | __float_as_uint(m_new);
        const bool raised = m_new != m_prev && m_prev != -INFINITY;
        if (__any_sync(full, raised)) {
          if (!mbar_wait_warp(bar(L::bPvDone + ((gg - 1) & 1)), ((gg - 1) >> 1) & 1, abort)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const float alpha = raised ? fast_exp2((m_prev - m_new) * f) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(lane_base + kColO + 32 * cc, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
            tmem_st32(lane_base + kColO + 32 * cc, o);
          }
        }
        // P over S, 32 keys at a time: a loop of few instructions, as a step's worth of them
        // unrolled would leave the other warps waiting for theirs
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        float rs = 0.f;
#pragma unroll 1
        for (int c = 0; c < groups; ++c) {
          uint32_t sr[32], hi[16], lo[16];
          tmem_ld32(s_addr + 32 * c, sr);
          tmem_wait_ld();
          reg_fence32(sr);
          rs += weigh32<kFp8>(sr, m_use, f, hi, lo);
          tmem_st16(s_addr + 32 * c, hi);
          tmem_st16(s_addr + 32 * c + 16, lo);
        }
        if (m_run != -INFINITY && m_run != m_new) l_run *= fast_exp2((m_run - m_new) * f);
        l_run += rs;
        m_run = m_new;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(L::bPFull + sb));
      }
      if (stop && lane == 0) fail();
      gs += n;
      // -------------------------------------------------------- epilogue --
      if (!stop) {
        stop = !mbar_wait_warp(bar(L::bTileDone), it & 1, abort);
        if (stop && lane == 0) fail();
      }
      float m_oth, l_oth;
      if (pair_xchg(m_run, l_run, stop, m_oth, l_oth)) break;
      tc_fence_after();
      const float m_tot = fmaxf(m_run, m_oth);
      // a set without a maximum has a sum of 0, or NaN if only NaN was there
      const float l_tot = (m_run == -INFINITY || m_run == m_tot ? l_run : l_run * fast_exp2((m_run - m_tot) * f)) +
                          (m_oth == -INFINITY || m_oth == m_tot ? l_oth : l_oth * fast_exp2((m_oth - m_tot) * f));
      const bool row_ok = row < n_rows;
      const int tok = row / G, h = g * G + row - tok * G, c0 = sm * (D / 2);
      const float inv = l_tot == 0.f ? 0.f : (kFp8 && a.v_scale ? get(a.v_scale + g) : 1.f) / l_tot;
      const uint64_t odd_of = special && row_ok && odd_seen[x] ? seen_sets[x * 64 + tok] : 0ull;
      float* part = partial + ((static_cast<int64_t>(rt) * runs + run_id) * 2 + max(dest, 0)) * (BM * (D + 2));
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t ov[32];
        tmem_ld32(lane_base + kColO + c0 + 32 * cc, ov);
        tmem_wait_ld();
        reg_fence32(ov);
        if (!row_ok) continue;
        // values that were taken out and that this row sees
        for (uint64_t left = odd_of; left; left &= left - 1) {
          const int t = heads[x].base + __ffsll(left) - 1;
          const int page = get(a.pm.table + b * a.pm.table_stride + t / kBlock);
          if (page < 0 || page >= a.pm.n_pages) continue;
          const int64_t at = page * a.vcs[0] + g * a.vcs[1] + t % kBlock * a.vcs[2] + c0 + 32 * cc;
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            float v;
            if (kFp8) {
              const uint8_t code = static_cast<const uint8_t*>(a.vc)[at + u];
              v = (code & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : 0.f;
            } else {
              const uint16_t w = static_cast<const uint16_t*>(a.vc)[at + u];
              v = (w & 0x7f80u) == 0x7f80u ? __uint_as_float(static_cast<uint32_t>(w) << 16) : 0.f;
            }
            ov[u] = __float_as_uint(__uint_as_float(ov[u]) + v);
          }
        }
        if (dest < 0) {
          uint16_t* out = a.o + b * a.os[0] + tok * a.os[1] + h * a.os[2] + c0 + 32 * cc;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float y[8];
            // a row without weight may face an O that was never written
#pragma unroll
            for (int u = 0; u < 8; ++u) y[u] = l_tot == 0.f ? 0.f : __uint_as_float(ov[8 * v + u]) * inv;
            *reinterpret_cast<uint4*>(out + 8 * v) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                                pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
          }
        } else {
          // four columns of all rows follow each other: lanes are rows
          float4* out = reinterpret_cast<float4*>(part) + (c0 / 4 + 8 * cc) * BM + r;
#pragma unroll
          for (int v = 0; v < 8; ++v)
            out[v * BM] =
                l_tot == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                             : make_float4(__uint_as_float(ov[4 * v]), __uint_as_float(ov[4 * v + 1]),
                                           __uint_as_float(ov[4 * v + 2]), __uint_as_float(ov[4 * v + 3]));
        }
      }
      tc_fence_before();
      mbar_arrive(bar(L::bOFree));
      if (row_ok && sm == 0) {
        const float m2 = m_tot * f;
        if (dest >= 0)
          *reinterpret_cast<float2*>(part + BM * D + 2 * r) = make_float2(m_tot == -INFINITY ? -INFINITY : m2, l_tot);
        else if (a.lse)
          a.lse[(static_cast<int64_t>(b) * a.H + h) * a.S + tok] =
              l_tot == 0.f ? -INFINITY
                           : (m2 + log2f(kFp8 ? l_tot * 0x1p-5f : l_tot)) * 0.69314718055994530942f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bHeadEmpty + x));
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

// grid (row tiles * runs, D / 8), 256 threads: adds the partials of the unit that is cut
// behind a run's end, in the order of the runs; a thread has four columns of a row.
template <int D>
__global__ void __launch_bounds__(256)
tile_join_kernel(DecodeArgs a, int runs, float unit, const float* partial, const TileCut* cuts) {
  wait_for_first();
  const int4 whole = *reinterpret_cast<const int4*>(cuts + blockIdx.x);
  const int rt = blockIdx.x / runs, bg = whole.x, first = whole.y, last = whole.z;
  if (bg < 0 || bg >= a.B * a.Hkv || first < 0 || last <= first || last >= runs) return;
  const int r = threadIdx.x % BM, c4 = blockIdx.y * 2 + threadIdx.x / BM, row = rt * BM + r;
  const int G = a.H / a.Hkv, b = bg / a.Hkv, g = bg - b * a.Hkv;
  int base, none = 0;
  if (row >= new_tokens(a, b, &base, &none) * G) return;
  float o[4] = {}, m = -INFINITY, l = 0.f;
  auto piece = [&](int i) {
    return partial + ((static_cast<int64_t>(rt) * runs + i) * 2 + (i == first ? 1 : 0)) * (BM * (D + 2));
  };
  constexpr int kOnce = 4;
  for (int i0 = first; i0 <= last; i0 += kOnce) {
    float2 ml[kOnce];
    float4 v[kOnce];
#pragma unroll
    for (int u = 0; u < kOnce; ++u) {
      const float* p = piece(min(i0 + u, last));
      ml[u] = *reinterpret_cast<const float2*>(p + BM * D + 2 * r);
      v[u] = reinterpret_cast<const float4*>(p)[c4 * BM + r];
    }
#pragma unroll
    for (int u = 0; u < kOnce; ++u) {
      if (i0 + u > last) break;
      if (ml[u].x == -INFINITY) {            // nothing counted there (a sum of 0, or NaN)
        l += ml[u].y;
        continue;
      }
      const float now = fmaxf(m, ml[u].x), c0 = m == -INFINITY ? 0.f : ex2(m - now), c1 = ex2(ml[u].x - now);
      l = (m == -INFINITY ? l : l * c0) + ml[u].y * c1;
      m = now;
      o[0] = o[0] * c0 + v[u].x * c1;
      o[1] = o[1] * c0 + v[u].y * c1;
      o[2] = o[2] * c0 + v[u].z * c1;
      o[3] = o[3] * c0 + v[u].w * c1;
    }
  }
  const int tok = row / G, h = g * G + row - tok * G;
  const float inv = l == 0.f ? 0.f : (a.v_scale ? a.v_scale[g] : 1.f) / l;
  *reinterpret_cast<uint2*>(a.o + b * a.os[0] + tok * a.os[1] + h * a.os[2] + 4 * c4) =
      make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  if (c4 == 0 && a.lse)
    a.lse[(static_cast<int64_t>(b) * a.H + h) * a.S + tok] =
        l == 0.f ? -INFINITY : (m + log2f(l * unit)) * 0.69314718055994530942f;
}

int tile_runs(int rows) {
  const int RT = (rows + BM - 1) / BM;
  return RT < kSms ? kSms / RT : 1;
}

template <int D, bool kFp8>
cudaError_t launch_tile(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t st) {
  using L = Tile<D, kFp8>;
  const int rows = a.S * (a.H / a.Hkv), RT = (rows + BM - 1) / BM, runs = tile_runs(rows);
  TileCut* cuts = reinterpret_cast<TileCut*>(a.ws);
  float* partial = reinterpret_cast<float*>(a.ws + ((static_cast<size_t>(RT) * runs * sizeof(TileCut) + 255) & ~static_cast<size_t>(255)));
  const auto kernel = tree_tile_kernel<D, kFp8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<dim3(static_cast<unsigned>(runs), static_cast<unsigned>(RT)), L::kThreads, L::kBytes, st>>>(kmap, vmap, a, partial, cuts);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_close(tile_join_kernel<D>, dim3(static_cast<unsigned>(RT * runs), D / 8), 256, 0, st, a, runs,
                      kFp8 ? 0x1p-5f : 1.f, partial, cuts);
}

}  // namespace

size_t tree_tile_ws_bytes(int rows, int D) {
  const size_t n = static_cast<size_t>((rows + BM - 1) / BM) * tile_runs(rows);
  return ((n * sizeof(TileCut) + 255) & ~static_cast<size_t>(255)) + n * 2 * BM * (D + 2) * sizeof(float);
}

cudaError_t launch_tree_tile(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, bool fp8,
                             cudaStream_t st) {
  if (a.D == 64) return fp8 ? launch_tile<64, true>(a, kmap, vmap, st) : launch_tile<64, false>(a, kmap, vmap, st);
  return fp8 ? launch_tile<128, true>(a, kmap, vmap, st) : launch_tile<128, false>(a, kmap, vmap, st);
}

}  // namespace sa
