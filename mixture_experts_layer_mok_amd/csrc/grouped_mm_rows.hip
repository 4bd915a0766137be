// Tiles of the grouped product of 16-bit rows: the rows' gradient.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_rows(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmRows, g16::kAcross>(a, st); }

}  // namespace mok
