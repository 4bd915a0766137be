// Tiles of the grouped product of 16-bit rows: the weights' gradient.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_weights(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmWeights, g16::kAcross>(a, st); }

}  // namespace mok
