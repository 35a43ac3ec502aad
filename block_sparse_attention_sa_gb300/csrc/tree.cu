// tree.cu -- attention of a few new tokens per sequence, a tree of drafted ones, over
// the paged cache.
#include <algorithm>

#include "decode_kernel.cuh"

namespace sa {

// Whether tcgen05 takes a tree, 128 rows (pairs of a new token and a query head) of a
// key-value head at a time, or decode_kernel, whose products are those of 16 rows. In us,
// decode_kernel and tiles (L2 flushed before each call):
//   rows a key-value head              8         16        17        32        33 and more
//   64 x 3,000, 8 heads of 128, bf16   154 146   162 150   191 150   207 152   64 rows: 394 156
//     heads of 64                       97  97   105 100   123 100   141 100
//   64 x 6,000, 8 heads of 128, e4m3   160 263   188 263   287 269   303 269   605 275
//     heads of 64                      103 233   128 233   181 238   199 237   359 234
//   8 x 1,500, 8 heads of 128, bf16     28  31    33  31    35  31    41  31
//   3 x 38,247, 2 heads of 128, bf16    42  48    42  46    46  48    48  45
//   1 x 777, 8 heads of 128, bf16       16  19    17  19    17  19    17  19
//     e4m3                              16  21    17  21    17  22    19  21
// Up to 16 rows decode_kernel, which reads a page once: it loses 5 to 8% in large batches in
// bf16 from 12 rows on and wins elsewhere, in e4m3 by 20 to 45%. Above 32 tiles. Between, a
// product of 32 rows costs decode_kernel more than the tiles' start, but for e4m3 with heads
// of 64, where turning codes into fp16 bounds the tiles, and where a run is a page or two, as
// far as the table's size tells.
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
