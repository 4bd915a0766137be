// Tiles of the grouped product of 16-bit rows: rows.
#include "grouped_mm_tiles.h"

namespace mok {

mok_status_t launch_mm_rows(const MmArgs& a, hipStream_t st) { return g16::launch_tiles<kMmRows>(a, st); }

}  // namespace mok
