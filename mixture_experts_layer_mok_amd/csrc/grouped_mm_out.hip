// Tiles of the grouped product of 16-bit rows: out.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_out(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmOut, g16::kAlong>(a, st); }

}  // namespace mok
