// Products of 8-bit rows in middle-sized tiles.
#include "i8_tile.h"

namespace moe {

hipError_t launch_i8_middle(const I8Args& a, hipStream_t s) { return launch_tile<2, 4, 2, 2, 2>(a, s); }

}  // namespace moe
