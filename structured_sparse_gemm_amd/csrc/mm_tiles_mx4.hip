// mm_tiles_mx4.hip -- the tiled products of mx4 weights (see mm_tiles.hpp).
#include "mm_tiles.hpp"

namespace ssg {

hipError_t launch_mm_tiles_mx4(const MmArgs& a, int size, hipStream_t s) {
    if (a.mode == MM_MX4) return mm_tiles_size<MM_MX4, DT_F16, false, false>(a, size, s);
    return a.dt == DT_F16 ? mm_tiles_size<MM_W4, DT_F16, false, false>(a, size, s)
                          : mm_tiles_size<MM_W4, DT_BF16, false, false>(a, size, s);
}

}  // namespace ssg
