// Tiles of the grouped product of 16-bit rows: the weights' gradient from rows held in 8 bits.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_weights_held(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmWeights, g16::kHeld>(a, st); }

}  // namespace mok
