// tree.cu -- attention of a few new tokens per sequence, a tree of drafted ones, over
// the paged cache.
#include <algorithm>

#include "decode_kernel.cuh"

namespace sa {

// Whether tcgen05 takes a tree, 128 rows (pairs of a new token and a query head) of a
// key-value head at a time, or decode_kernel, whose products are those of 16 rows. 64
// sequences of 3,000 tokens, 8 heads of 128 in bf16: 16 rows 162 us with the latter and 152
// with the former, 17 rows 191 and 154, 64 rows 394 and 156; of 6,000 in e4m3: 16 rows 188
// and 269, 33 rows 605 and 275 (heads of 64: 32 rows 199 and 232, 33 rows 359 and 234). Up
// to 32 rows decode_kernel starts sooner (777 tokens, 32/8 heads, 8 new ones: 17 us and
// 19), which decides where a run is a page or two, as far as the table's size tells.
static bool in_tiles(int rows, int D, bool fp8, int64_t pages) {
  if (rows <= 16) return false;
  return rows > 32 || !((fp8 && D == 64) || pages <= 2 * kSms);
}

size_t tree_ws_bytes(int rows, int D) {
  return rows <= 16 ? decode_ws_bytes(rows, D)
                    : (rows > 32 ? tree_tile_ws_bytes(rows, D)
                                 : std::max(tree_tile_ws_bytes(rows, D), decode_ws_bytes(rows, D)));
}

cudaError_t launch_tree(const DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap,
                        bool fp8, cudaStream_t st) {
  if (in_tiles(a.S * (a.H / a.Hkv), a.D, fp8, static_cast<int64_t>(a.B) * a.Hkv * a.pm.max_pages))
    return launch_tree_tile(a, kmap, vmap, fp8, st);
  if (a.D == 64)
    return fp8 ? launch_d<64, true, true>(a, kmap, vmap, st) : launch_d<64, false, true>(a, kmap, vmap, st);
  return fp8 ? launch_d<128, true, true>(a, kmap, vmap, st) : launch_d<128, false, true>(a, kmap, vmap, st);
}

}  // namespace sa
