// append.cu -- new tokens into a paged key-value cache: QK-norm + rotation of
// k (and of q, which goes out in bf16), the store of k and v as bf16 or e4m3,
// and the per-page key sums the page router reads.
//   y = x / sqrt(mean(x^2) + eps) * gamma,  (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c)
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_internal.cuh"

namespace sa {
namespace {

__device__ __forceinline__ float bits_f32(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// One thread per (token, head vector): reads it twice (norm, then values).
template <int D, bool kFp8, bool kHalf>
__device__ void turn(const AppendArgs& a, const uint16_t* x, const float* gamma, int t, float* y) {
  for (int d = 0; d < D; ++d) y[d] = bits_f32(x[d]);
  if (a.norm) {
    float ss = 0.f;
    for (int d = 0; d < D; ++d) ss = fmaf(y[d], y[d], ss);
    const float r = rsqrtf(ss / D + a.eps);
    for (int d = 0; d < D; ++d) y[d] = y[d] * r * (gamma ? gamma[d] : 1.f);
  }
  if (a.cos) {
    for (int i = 0; i < D / 2; ++i) {
      const int ia = kHalf ? i : 2 * i, ib = kHalf ? i + D / 2 : 2 * i + 1;
      const float c = a.cos[static_cast<int64_t>(t) * (D / 2) + i];
      const float s = a.sin[static_cast<int64_t>(t) * (D / 2) + i];
      const float ya = y[ia], yb = y[ib];
      y[ia] = fmaf(ya, c, -yb * s);
      y[ib] = fmaf(ya, s, yb * c);
    }
  }
}

template <bool kFp8>
__device__ void store(void* cache, int64_t at, float y, float inv_scale) {
  if (kFp8)
    static_cast<uint8_t*>(cache)[at] = __nv_cvt_float_to_fp8(y * inv_scale, __NV_SATFINITE, __NV_E4M3);
  else
    static_cast<uint16_t*>(cache)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

// grid (B, Hkv + H): one thread per token of head blockIdx.y; a key-value
// head's k_sum is summed token by token by thread 0.
template <int D, bool kFp8, bool kHalf>
__global__ void append_kernel(AppendArgs a) {
  const int b = blockIdx.x, S = a.S;
  bool bad;
  const int base = clamp_len(a.pm.seq_lens[b], a.pm, &bad);
  int n = a.new_lens ? min(max(a.new_lens[b], 0), S) : S;
  const int most = a.pm.max_pages * kBlock;
  int status = bad ? SA_DEV_BAD_CACHE : 0;
  if (n > most - base) {
    n = most - base;
    status |= SA_DEV_CAPACITY;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0 && a.lens_out) a.lens_out[b] = base + n;
  const bool is_q = static_cast<int>(blockIdx.y) >= a.Hkv;
  const int h = is_q ? blockIdx.y - a.Hkv : blockIdx.y;
  float y[D];
  const bool sums = !is_q && a.k_sum;
  for (int s = threadIdx.x; s < n; s += blockDim.x) {
    const int t = base + s;
    const int page = a.pm.table[b * a.pm.table_stride + t / kBlock];
    if (page < 0 || page >= a.pm.n_pages) {
      status |= SA_DEV_BAD_CACHE;
      continue;
    }
    if (a.cos && t >= a.rope_rows) {
      status |= SA_DEV_CAPACITY;
      continue;
    }
    if (is_q) {
      turn<D, kFp8, kHalf>(a, a.q + b * a.qs[0] + s * a.qs[1] + h * a.qs[2], a.gamma_q, t, y);
      for (int d = 0; d < D; ++d)
        store<false>(a.q_out, b * a.os[0] + s * a.os[1] + h * a.os[2] + d, y[d], 1.f);
      continue;
    }
    turn<D, kFp8, kHalf>(a, a.k + b * a.ks[0] + s * a.ks[1] + h * a.ks[2], a.gamma_k, t, y);
    const float ik = a.k_scale ? 1.f / a.k_scale[h] : 1.f, iv = a.v_scale ? 1.f / a.v_scale[h] : 1.f;
    const int slot = t % kBlock;
    for (int d = 0; d < D; ++d) {
      store<kFp8>(a.kc, page * a.kcs[0] + h * a.kcs[1] + slot * a.kcs[2] + d, y[d], ik);
      store<kFp8>(a.vc, page * a.vcs[0] + h * a.vcs[1] + slot * a.vcs[2] + d,
                  bits_f32(a.v[b * a.vs[0] + s * a.vs[1] + h * a.vs[2] + d]), iv);
    }
    // the first token of a page in this call sums the page's tokens
    if (sums && (s == 0 || slot == 0)) {
      float* out = a.k_sum + (static_cast<int64_t>(page) * a.Hkv + h) * D;
      const int end = min(n, s + kBlock - slot);
      float z[D];
      for (int d = 0; d < D; ++d) z[d] = slot == 0 ? 0.f : out[d];
      for (int u = s; u < end && !(a.cos && base + u >= a.rope_rows); ++u) {
        if (u > s)
          turn<D, kFp8, kHalf>(a, a.k + b * a.ks[0] + u * a.ks[1] + h * a.ks[2], a.gamma_k,
                               base + u, y);
        for (int d = 0; d < D; ++d) z[d] += y[d];
      }
      for (int d = 0; d < D; ++d) out[d] = z[d];
    }
  }
  if (status && a.dev_status) atomicOr(a.dev_status, status);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int D, bool fp8, bool half, cudaStream_t st) {
  const dim3 grid(a.B, a.Hkv + (a.q ? a.H : 0));
  const int threads = a.S >= 128 ? 128 : 32;
  auto run = [&](auto kernel) {
    kernel<<<grid, threads, 0, st>>>(a);
    return cudaGetLastError();
  };
  if (D == 64) {
    if (fp8) return half ? run(append_kernel<64, true, true>) : run(append_kernel<64, true, false>);
    return half ? run(append_kernel<64, false, true>) : run(append_kernel<64, false, false>);
  }
  if (fp8) return half ? run(append_kernel<128, true, true>) : run(append_kernel<128, true, false>);
  return half ? run(append_kernel<128, false, true>) : run(append_kernel<128, false, false>);
}

}  // namespace sa
