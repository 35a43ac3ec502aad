// tree.cu -- attention of a few new tokens per sequence, a tree of drafted ones, over
// the paged cache.
#include "decode_kernel.cuh"

namespace sa {

cudaError_t launch_tree(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        bool fp8, cudaStream_t st) {
  if (a.D == 64)
    return fp8 ? launch_d<64, true, true>(a, kmap, vmap, st) : launch_d<64, false, true>(a, kmap, vmap, st);
  return fp8 ? launch_d<128, true, true>(a, kmap, vmap, st) : launch_d<128, false, true>(a, kmap, vmap, st);
}

}  // namespace sa
