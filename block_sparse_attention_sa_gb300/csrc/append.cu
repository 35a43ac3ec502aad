// append.cu -- new tokens into a paged key-value cache: QK-norm + rotation of
// k (and of q, which goes out in bf16), the store of k and v as bf16 or e4m3,
// and the per-page key sums the page router reads.
//   y = x / sqrt(mean(x^2) + eps) * gamma,  (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c)
//
// Every byte is read and written once, so the kernel is bound by the memory, or
// for one token by its chain of dependent loads (length, page, angle). D / 8
// lanes hold a head vector, eight elements each: with the halves of a vector as
// pairs, four from each half, so that both rotations turn pairs a lane holds.
//
// One launch, two kinds of CTAs. Key-value CTAs own whole pages of one head: a
// page's tokens of this call are summed in a fixed order by the lanes that
// store them, so its k_sum needs no atomics and is the same every time. Query
// CTAs own a few tokens: a token's angles are loaded once for all heads. At most
// 72 registers a thread, so that seven CTAs of 128 threads share an SM, which costs 40
// bytes of spills: loads in flight come from many warps, not from deep ones (38,247
// tokens, 56/8 heads: 282 us with four CTAs and four tokens in flight a lane group,
// 227 us with six CTAs without spills, 217 us with seven, 227 us with eight).
//
// Measured on GB300 (copy rate 6.79 TB/s): 38,247 tokens, 56/8 heads of 128,
// bf16, 1.43 GB in 217 us, 6.6 TB/s. 5 x up to 2,047 tokens, 16/16 heads of 64,
// e4m3, 62 MB in 16.7 us, 3.7 TB/s: instructions bound it, 61% of the issue slots
// while its CTAs run. One token 3.5 us, 128 tokens 4.1 us: launch and the chain of loads.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

constexpr int kGroups = 8;         // lane groups of a CTA, D / 8 lanes each
constexpr int kQueryHeads = 8;     // heads a lane group has in flight
constexpr int kTokens = 2;         // tokens a lane group has in flight

struct Vec {                       // a lane's eight elements
  float x[8];
};

// Where a lane's elements lie: [8 l, 8 l + 8), or [4 l, 4 l + 4) of each half.
template <int D, bool kHalf>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int l) {
  if (!kHalf) return *reinterpret_cast<const uint4*>(p + 8 * l);
  const uint2 a = *reinterpret_cast<const uint2*>(p + 4 * l);
  const uint2 b = *reinterpret_cast<const uint2*>(p + D / 2 + 4 * l);
  return make_uint4(a.x, a.y, b.x, b.y);
}

template <int D, bool kHalf>
__device__ __forceinline__ void store8(uint16_t* p, int l, uint4 w) {
  if (!kHalf) {
    *reinterpret_cast<uint4*>(p + 8 * l) = w;
  } else {
    *reinterpret_cast<uint2*>(p + 4 * l) = make_uint2(w.x, w.y);
    *reinterpret_cast<uint2*>(p + D / 2 + 4 * l) = make_uint2(w.z, w.w);
  }
}

template <int D, bool kHalf>
__device__ __forceinline__ void load8f(const float* p, int l, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p + (kHalf ? 4 * l : 8 * l));
  const float4 b = *reinterpret_cast<const float4*>(p + (kHalf ? D / 2 + 4 * l : 8 * l + 4));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <int D, bool kHalf>
__device__ __forceinline__ void store8f(float* p, int l, const float* x) {
  *reinterpret_cast<float4*>(p + (kHalf ? 4 * l : 8 * l)) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + (kHalf ? D / 2 + 4 * l : 8 * l + 4)) =
      make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ Vec unpack(uint4 w) {
  Vec v;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v.x[2 * i] = __uint_as_float(u[i] << 16);
    v.x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
  return v;
}

__device__ __forceinline__ uint4 pack(const Vec& v) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A head's scale and its reciprocal, rounded to nearest.
struct Scale {
  float s, inv;
};

__device__ __forceinline__ Scale scale_of(const float* scale, int h) {
  const float s = scale ? get(scale + h) : 1.f;
  return {s, 1.f / s};
}

// The e4m3 codes nearest to the fp32 quotients of values and a scale (ties to even),
// saturating. The product with the reciprocal may be two units in the last place off
// the quotient and so on the other side of the middle between two codes; its
// remainder, exact in one fused step, puts that right (Markstein 1990). Beyond the
// largest code, where it could overflow, no bit of the quotient matters.
__device__ __forceinline__ uint2 pack_e4m3(const Vec& v, const Scale& c) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = v.x[i] * c.inv;
    if (fabsf(q[i]) < 512.f) q[i] = fmaf(fmaf(-q[i], c.s, v.x[i]), c.inv, q[i]);
  }
  uint32_t u[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    u[i] = lo | (hi << 16);
  }
  return make_uint2(u[0], u[1]);
}

template <int D, bool kHalf>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int l, uint2 w) {
  if (!kHalf) {
    *reinterpret_cast<uint2*>(p + 8 * l) = w;
  } else {
    *reinterpret_cast<uint32_t*>(p + 4 * l) = w.x;
    *reinterpret_cast<uint32_t*>(p + D / 2 + 4 * l) = w.y;
  }
}

// The angles of a lane's four pairs at one position.
struct Angle {
  float4 c, s;
};

template <int D>
__device__ __forceinline__ Angle angle_at(const AppendArgs& a, int t, int l) {
  Angle g{make_float4(1.f, 1.f, 1.f, 1.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  if (a.cos) {
    const int64_t at = static_cast<int64_t>(t) * (D / 2) + 4 * l;
    g.c = get(reinterpret_cast<const float4*>(a.cos + at));
    g.s = get(reinterpret_cast<const float4*>(a.sin + at));
  }
  return g;
}

// Norm and rotation of a vector held by D / 8 lanes of a converged warp.
template <int D, bool kHalf>
__device__ __forceinline__ void turn(Vec& v, const AppendArgs& a, const float* gamma, const Angle& g) {
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v.x[i], v.x[i], ss);
#pragma unroll
    for (int off = D / 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[i] = v.x[i] * r * gamma[i];
  }
  if (a.cos) {
    const float c[4] = {g.c.x, g.c.y, g.c.z, g.c.w}, s[4] = {g.s.x, g.s.y, g.s.z, g.s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& p = v.x[kHalf ? i : 2 * i];
      float& q = v.x[kHalf ? 4 + i : 2 * i + 1];
      const float p0 = p, q0 = q;
      p = fmaf(p0, c[i], -q0 * s[i]);
      q = fmaf(p0, s[i], q0 * c[i]);
    }
  }
}

// How many of the new tokens of sequence b have a place: in its page table, and
// in the rotation tables where there are some.
__device__ __forceinline__ int tokens_of(const AppendArgs& a, int b, int* base, int* status) {
  bool bad;
  *base = clamp_len(get(a.pm.seq_lens + b), a.pm, &bad);
  int n = a.new_lens ? min(max(get(a.new_lens + b), 0), a.S) : a.S;
  int room = a.pm.max_pages * kBlock - *base;
  if (a.cos) room = min(room, max(0, a.rope_rows - *base));
  if (bad) *status |= SA_DEV_BAD_CACHE;
  if (n > room) {
    n = room;
    *status |= SA_DEV_CAPACITY;
  }
  return n;
}

// The page of position t, or -1 with the reason in *status.
__device__ __forceinline__ int page_of(const AppendArgs& a, int b, int t, int* status) {
  const int page = get(a.pm.table + b * a.pm.table_stride + static_cast<unsigned>(t) / kBlock);
  if (page >= 0 && page < a.pm.n_pages) return page;
  *status |= SA_DEV_BAD_CACHE;
  return -1;
}

// A key-value unit: the tokens of this call in page place `pu` (counted from
// the first one touched) of sequence b, one head; kShare lane groups take
// every kShare-th token. Returns with the lanes' sums of what they stored.
template <int D, bool kFp8, bool kHalf, int kShare>
__device__ __forceinline__ void key_value_unit(const AppendArgs& a, int b, int pu, int h, int grp,
                                               int l, bool there, int* page, int* slot0,
                                               float* sum, int* status) {
  // with one new token its address needs no length: the loads go first
  const uint16_t* k = a.k + b * a.ks[0] + h * a.ks[2];
  const uint16_t* v = a.v + b * a.vs[0] + h * a.vs[2];
  uint4 kw[kTokens], vw[kTokens];
  const bool early = kShare == 1 && a.S == 1 && there;
  if (early) {
    kw[0] = load8<D, kHalf>(k, l);
    vw[0] = load8<D, false>(v, l);
  }
  float gk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gk[i] = 1.f;
  if (a.gamma_k) load8f<D, kHalf>(a.gamma_k, l, gk);
  Scale ck{}, cv{};
  if (kFp8) {
    ck = scale_of(a.k_scale, h);
    cv = scale_of(a.v_scale, h);
  }
  int base = 0;
  const int n = there ? tokens_of(a, b, &base, status) : 0;
  // tokens [s0, s1) of the page
  const int64_t edge = (static_cast<int64_t>(base / kBlock) + pu) * kBlock - base;
  const int s0 = edge > 0 ? static_cast<int>(min(edge, static_cast<int64_t>(n))) : 0;
  const int s1 = static_cast<int>(min(edge + kBlock, static_cast<int64_t>(n)));
  // the page is not waited for before the first store
  *page = s0 < s1 ? page_of(a, b, base + s0, status) : -1;
  *slot0 = static_cast<unsigned>(base + s0) % kBlock;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  // token s0 + grp and every kShare-th one after it: what is left of them, and
  // where the next one is read and stored
  int left = (s1 - s0 - grp + kShare - 1) / kShare;
  int t = base + s0 + grp;
  k += (s0 + grp) * a.ks[1];
  v += (s0 + grp) * a.vs[1];
  const int64_t k_step = kShare * a.ks[1], v_step = kShare * a.vs[1];
  const int elt = kFp8 ? 1 : 2;
  char* kc = static_cast<char*>(a.kc) +
             (*page * a.kcs[0] + h * a.kcs[1] + (*slot0 + grp) * a.kcs[2]) * elt;
  char* vc = static_cast<char*>(a.vc) +
             (*page * a.vcs[0] + h * a.vcs[1] + (*slot0 + grp) * a.vcs[2]) * elt;
  const int64_t kc_step = kShare * a.kcs[2] * elt, vc_step = kShare * a.vcs[2] * elt;
  // every lane of the warp makes the same number of rounds: turn() shuffles
  int rounds = (max(left, 0) + kTokens - 1) / kTokens;
  rounds = __reduce_max_sync(0xffffffffu, rounds);
  for (int r = 0; r < rounds; ++r) {
    Angle g[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      if (u >= left) continue;
      if (!early) {
        kw[u] = load8<D, kHalf>(k, l);
        vw[u] = load8<D, false>(v, l);
      }
      g[u] = angle_at<D>(a, t + u * kShare, l);
      k += k_step;
      v += v_step;
    }
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const bool on = u < left;
      Vec y = unpack(on ? kw[u] : make_uint4(0u, 0u, 0u, 0u));
      turn<D, kHalf>(y, a, gk, g[u]);
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += y.x[i];
      if (*page < 0) continue;
      if (kFp8) {
        store8_e4m3<D, kHalf>(reinterpret_cast<uint8_t*>(kc), l, pack_e4m3(y, ck));
        store8_e4m3<D, false>(reinterpret_cast<uint8_t*>(vc), l, pack_e4m3(unpack(vw[u]), cv));
      } else {
        store8<D, kHalf>(reinterpret_cast<uint16_t*>(kc), l, pack(y));
        store8<D, false>(reinterpret_cast<uint16_t*>(vc), l, vw[u]);
      }
      kc += kc_step;
      vc += vc_step;
    }
    left -= kTokens;
    t += kTokens * kShare;
  }
}

// kWhole: a CTA takes one key-value unit, else each of its lane groups one.
template <int D, bool kFp8, bool kHalf, bool kWhole>
__global__ void __launch_bounds__(D, (kWhole ? 7 : 4) * 128 / D) append_kernel(AppendArgs a, int units, int page_units,
                                                          int kv_ctas, int per_log2) {
  constexpr int L = D / 8;
  const int grp = threadIdx.x / L, l = threadIdx.x % L;
  int status = 0;
  if (static_cast<int>(blockIdx.x) < kv_ctas) {
    // ------------------------------------------------------ keys, values --
    const unsigned u = kWhole ? blockIdx.x : blockIdx.x * kGroups + grp;
    const bool there = u < static_cast<unsigned>(units);
    const unsigned bp = u / static_cast<unsigned>(a.Hkv);
    const int h = u - bp * a.Hkv, b = there ? bp / static_cast<unsigned>(page_units) : 0;
    const int pu = there ? bp - b * static_cast<unsigned>(page_units) : 0;
    int page, slot0;
    float sum[8];
    key_value_unit<D, kFp8, kHalf, kWhole ? kGroups : 1>(a, b, pu, h, kWhole ? grp : 0, l, there,
                                                         &page, &slot0, sum, &status);
    if (there && a.lens_out && pu == 0 && h == 0 && l == 0 && (!kWhole || grp == 0)) {
      int base;
      const int n = tokens_of(a, b, &base, &status);
      a.lens_out[b] = base + n;
    }
    if (kWhole && a.k_sum) {
      // the lane groups' sums: across a warp, then the warps' in their order
      __shared__ float part[D / 32][D];
#pragma unroll
      for (int off = L; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
      if (threadIdx.x % 32 < L) store8f<D, false>(part[threadIdx.x / 32], l, sum);   // in the lane's own order
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int w = 1; w < D / 32; ++w)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += part[w][8 * l + i];
      }
    }
    if (a.k_sum && page >= 0 && (!kWhole || grp == 0)) {
      float* out = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + h) * D;
      if (slot0 > 0) {
        float old[8];
        load8f<D, kHalf>(out, l, old);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += old[i];
      }
      store8f<D, kHalf>(out, l, sum);
    }
  } else {
    // ----------------------------------------------------------- queries --
    // `per` lane groups share a token, every per-th head each
    const int per = 1 << per_log2;
    const unsigned token = (blockIdx.x - kv_ctas) * (kGroups >> per_log2) + (grp >> per_log2);
    const bool there = token < static_cast<unsigned>(a.B) * a.S;
    const int b = there ? token / static_cast<unsigned>(a.S) : 0, s = token - b * a.S;
    const int hg = grp & (per - 1);
    const uint16_t* q = a.q + b * a.qs[0] + s * a.qs[1];
    uint16_t* out = a.q_out + b * a.os[0] + s * a.os[1];
    uint4 w[kQueryHeads];
    auto load = [&](int h0, bool on) {
#pragma unroll
      for (int u = 0; u < kQueryHeads; ++u) {
        const int h = h0 + u * per + hg;
        w[u] = on && h < a.H ? load8<D, kHalf>(q + h * a.qs[2], l) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    // a token that may not count is not read before that is known
    const bool early = a.new_lens == nullptr;
    if (early) load(0, there);
    float gq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) gq[i] = 1.f;
    if (a.gamma_q) load8f<D, kHalf>(a.gamma_q, l, gq);
    int base = 0, none = 0;             // the key-value CTAs report what is wrong
    bool on = there && s < tokens_of(a, b, &base, &none);
    const int t = base + (on ? s : 0);
    if (!__any_sync(0xffffffffu, on)) return;
    // the queries and their angles are on their way while the page is looked up
    if (!early) load(0, on);
    Angle g = {};
    if (on) g = angle_at<D>(a, t, l);
    on = on && page_of(a, b, t, &none) >= 0;
    for (int h0 = 0; h0 < a.H; h0 += kQueryHeads * per) {
      if (h0 > 0) load(h0, on);
#pragma unroll
      for (int u = 0; u < kQueryHeads; ++u) {
        if (h0 + u * per >= a.H) break;
        const int h = h0 + u * per + hg;
        Vec y = unpack(w[u]);
        turn<D, kHalf>(y, a, gq, g);
        if (on && h < a.H) store8<D, kHalf>(out + h * a.os[2], l, pack(y));
      }
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

template <int D, bool kFp8, bool kHalf>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
  // the pages S tokens can touch, wherever the first of them lies
  const int64_t page_units = (static_cast<int64_t>(a.S) + kBlock - 2) / kBlock + 1;
  const int64_t units = a.B * page_units * a.Hkv;
  const bool whole = a.S > kTokens;
  const int64_t kv = whole ? units : (units + kGroups - 1) / kGroups;
  // lane groups per token: so many that each has all its heads in flight at once
  // and a token's angles are loaded by few (a group for each head instead, as far
  // as they go: the same for 1 to 4,096 tokens)
  const int64_t tokens = static_cast<int64_t>(a.B) * a.S;
  const int want = (a.H + kQueryHeads - 1) / kQueryHeads;
  int per_log2 = 0;
  while ((1 << per_log2) < want && (2 << per_log2) <= kGroups) ++per_log2;
  const int64_t at_once = kGroups >> per_log2;
  const int64_t grid = kv + (a.q ? (tokens + at_once - 1) / at_once : 0);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  const auto kernel = whole ? append_kernel<D, kFp8, kHalf, true> : append_kernel<D, kFp8, kHalf, false>;
  kernel<<<static_cast<unsigned>(grid), D, 0, st>>>(
      a, static_cast<int>(units), static_cast<int>(page_units), static_cast<int>(kv), per_log2);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, bool fp8, bool half, cudaStream_t st) {
  if (fp8) return half ? launch<D, true, true>(a, st) : launch<D, true, false>(a, st);
  return half ? launch<D, false, true>(a, st) : launch<D, false, false>(a, st);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int D, bool fp8, bool half, cudaStream_t st) {
  return D == 64 ? launch_d<64>(a, fp8, half, st) : launch_d<128>(a, fp8, half, st);
}

}  // namespace sa
