// decode.cu -- attention of one new token per sequence over the paged cache.
//   l_u = scale q.k_u,  a = softmax(l),  o = sum a_u v_u,  lse = log sum exp l
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

template <bool kFp8>
__device__ __forceinline__ float load(const void* p, int64_t at) {
  if (kFp8) {
    __nv_fp8_e4m3 x;
    x.__x = static_cast<const uint8_t*>(p)[at];
    return static_cast<float>(x);
  }
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[at]) << 16);
}

// grid (B, H), one warp: one pass over the row's pages with the running
// maximum and sum of the softmax, lane l holding dims l, l + 32, ...
template <bool kFp8>
__global__ void __launch_bounds__(32) decode_kernel(DecodeArgs a) {
  const int b = blockIdx.x, h = blockIdx.y, g = h / (a.H / a.Hkv), lane = threadIdx.x;
  const int nd = a.D / 32;
  bool bad;
  const int n = clamp_len(a.pm.seq_lens[b], a.pm, &bad), nb = (n + kBlock - 1) / kBlock;
  int status = bad ? SA_DEV_BAD_CACHE : 0;
  int beg = 0, end = nb;
  if (a.row_ptr) {
    const int r = b * a.Hkv + g;
    beg = a.row_ptr[r];
    end = a.row_ptr[r + 1];
    if (beg < 0 || end < beg || end > a.col_cap || end - beg > a.pm.max_pages) {
      status |= SA_DEV_BAD_ROUTE;
      beg = end = 0;
    }
  }
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  const float ks = a.k_scale ? a.k_scale[g] : 1.f, vs = a.v_scale ? a.v_scale[g] : 1.f;
  for (int i = 0; i < nd; ++i)
    q[i] = load<false>(a.q, b * a.qs[0] + h * a.qs[2] + lane + 32 * i);
  float m = -INFINITY, l = 0.f;
  for (int e = beg; e < end; ++e) {
    const int j = a.row_ptr ? a.col_idx[e] : e;
    if (j < 0 || j >= nb || (a.row_ptr && e > beg && j <= a.col_idx[e - 1])) {
      status |= SA_DEV_BAD_ROUTE;
      continue;
    }
    const int page = a.pm.table[b * a.pm.table_stride + j];
    if (page < 0 || page >= a.pm.n_pages) {
      status |= SA_DEV_BAD_CACHE;
      continue;
    }
    const int live = min(kBlock, n - j * kBlock);
    for (int s = 0; s < live; ++s) {
      float x = 0.f;
      const int64_t kat = page * a.kcs[0] + g * a.kcs[1] + s * a.kcs[2] + lane;
      const int64_t vat = page * a.vcs[0] + g * a.vcs[1] + s * a.vcs[2] + lane;
      for (int i = 0; i < nd; ++i) x = fmaf(q[i], load<kFp8>(a.kc, kat + 32 * i), x);
      for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      x *= a.scale_log2 * ks;
      const float mn = fmaxf(m, x), c = mn == -INFINITY ? 1.f : exp2f(m - mn);
      const float p = mn == -INFINITY ? 0.f : exp2f(x - mn);
      m = mn;
      l = l * c + p;
      for (int i = 0; i < nd; ++i) o[i] = fmaf(p, load<kFp8>(a.vc, vat + 32 * i), o[i] * c);
    }
  }
  const float inv = l > 0.f ? vs / l : (l == 0.f ? 0.f : l);
  for (int i = 0; i < nd; ++i)
    a.o[b * a.os[0] + h * a.os[2] + lane + 32 * i] =
        __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  if (lane == 0 && a.lse)
    a.lse[b * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
  if (status && lane == 0 && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, bool fp8, cudaStream_t st) {
  const dim3 grid(a.B, a.H);
  if (fp8)
    decode_kernel<true><<<grid, 32, 0, st>>>(a);
  else
    decode_kernel<false><<<grid, 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
