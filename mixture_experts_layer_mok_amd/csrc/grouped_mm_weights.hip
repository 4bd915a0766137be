// Tiles of the grouped product of 16-bit rows: weights.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_weights(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmWeights>(a, st); }

}  // namespace mok
