// decode.cu -- attention of one new token per sequence over the paged cache.
#include "decode_kernel.cuh"

namespace sa {

int decode_row_tiles(int rows) {
  const int held = 16 * row_groups(rows);
  return (rows + held - 1) / held;
}

size_t decode_ws_bytes(int rows, int D) {
  // two partials of every run
  const int groups = row_groups(rows);
  const size_t held = static_cast<size_t>(max_runs(groups)) * 16 * groups;
  return cuts_bytes() + 2 * held * (D + 2) * sizeof(float);
}

cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          bool fp8, cudaStream_t st) {
  if (a.D == 64)
    return fp8 ? launch_d<64, true, false>(a, kmap, vmap, st) : launch_d<64, false, false>(a, kmap, vmap, st);
  return fp8 ? launch_d<128, true, false>(a, kmap, vmap, st) : launch_d<128, false, false>(a, kmap, vmap, st);
}

}  // namespace sa
