// mm_tiles_16.hip -- the tiled 16-bit products: Y = X W^T, dX = dY W,
// dW = dY^T X (see mm_tiles.hpp).
#include "mm_tiles.hpp"

namespace ssg {

template <int DT>
static hipError_t by_layout(const MmArgs& a, int size, hipStream_t s) {
    if (a.pt) return mm_tiles_size<MM_16, DT, true, true>(a, size, s);
    if (a.qt) return mm_tiles_size<MM_16, DT, true, false>(a, size, s);
    return mm_tiles_size<MM_16, DT, false, false>(a, size, s);
}

hipError_t launch_mm_tiles_16(const MmArgs& a, int size, hipStream_t s) {
    return a.dt == DT_F16 ? by_layout<DT_F16>(a, size, s) : by_layout<DT_BF16>(a, size, s);
}

}  // namespace ssg
