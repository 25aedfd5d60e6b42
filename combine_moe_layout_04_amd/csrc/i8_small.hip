// Products of 8-bit rows in small tiles.
#include "i8_tile.h"

namespace moe {

hipError_t launch_i8_small(const I8Args& a, hipStream_t s) { return launch_tile<1, 2, 4, 2, 4>(a, s); }

}  // namespace moe
