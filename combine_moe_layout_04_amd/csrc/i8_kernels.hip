// Which tiles a product of 8-bit rows takes (the kernel is i8_tile.h), and the large ones.
#include "i8_tile.h"

namespace moe {

// Tiles of 128 x 256, one workgroup a CU, where there are enough of them; else of 64 x
// 128, two workgroups a CU; else of 64 x 64.  Rows of 2 KiB and more hide a tile's
// beginning and end better, so fewer large ones will do.  In us, large / middle / small:
//   64 tokens of 8 of 128 experts, 2048 x 1536 (792 large tiles at most): 73 / 71 / 70
//   1500 rows, 7168 x 4096 (192): 49 / 55 / 71;   1024 rows (128): 51 / 41 / 49
//   2000 tokens of 2 of 8, 1024 x 2048 (312): 26 / 21 / 25
//   4096 rows, 768 x 1024 (128; 512 of the middle size): 13 / 10 / 13
//   64 tokens of 2 of 8, 4096 x 2048 (72; 160): 19 / 15 / 14;   1 token of 8 of 128: 13 / 10 / 9
hipError_t launch_i8(const I8Args& a, hipStream_t s) {
  if (most_tiles(a, 128, 256) >= (a.kch >= 128 ? 192 : 400)) return launch_i8_large(a, s);
  if (most_tiles(a, 64, 128) >= 256) return launch_i8_middle(a, s);
  return launch_i8_small(a, s);
}

hipError_t launch_i8_large(const I8Args& a, hipStream_t s) { return launch_tile<4, 4, 2, 4, 2>(a, s); }

}  // namespace moe
