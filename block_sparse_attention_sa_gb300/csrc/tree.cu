// tree.cu -- attention of a few new tokens per sequence, a tree of drafted ones, over
// the paged cache.
#include "decode_kernel.cuh"

namespace sa {

// Rows (pairs of a new token and a query head) on a key-value head from which tcgen05
// takes them, 128 at a time; up to there a CTA of decode_kernel holds them all.
constexpr int kMostRows = 64;

size_t tree_ws_bytes(int rows, int D) {
  return rows > kMostRows ? tree_tile_ws_bytes(rows, D) : decode_ws_bytes(rows, D);
}

cudaError_t launch_tree(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        bool fp8, cudaStream_t st) {
  if (a.S * (a.H / a.Hkv) > kMostRows) return launch_tree_tile(a, kmap, vmap, fp8, st);
  if (a.D == 64)
    return fp8 ? launch_d<64, true, true>(a, kmap, vmap, st) : launch_d<64, false, true>(a, kmap, vmap, st);
  return fp8 ? launch_d<128, true, true>(a, kmap, vmap, st) : launch_d<128, false, true>(a, kmap, vmap, st);
}

}  // namespace sa
