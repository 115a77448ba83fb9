// Partial products of the split microscaled product: every pair of formats and both
// tiles.
#include "mx_product.h"

namespace pgemm {
namespace layer {
namespace {

template <class TL>
hipError_t launch(const MxArgs& a, int splits, hipStream_t stream) {
    hipLaunchKernelGGL((mxp::product_kernel<TL, lp::StorePart>),
                       dim3((unsigned)(a.tiles_m * a.tiles_n), (unsigned)splits), dim3(TL::T), 0,
                       stream, a, lp::StorePart{});
    return hipGetLastError();
}

template <int FX, int FW>
hipError_t split_as(bool big, const MxArgs& a, int splits, hipStream_t stream) {
    using T = MxTiles<FX, FW>;
    return big ? launch<typename T::Big>(a, splits, stream)
               : launch<typename T::Small>(a, splits, stream);
}

}  // namespace

hipError_t mx_split(int xformat, int wformat, bool big, const MxArgs& a, int splits,
                    hipStream_t stream) {
    if (xformat == PMX_E2M1)
        return wformat == PMX_E2M1 ? split_as<PMX_E2M1, PMX_E2M1>(big, a, splits, stream)
                                   : split_as<PMX_E2M1, PMX_E4M3>(big, a, splits, stream);
    return wformat == PMX_E2M1 ? split_as<PMX_E4M3, PMX_E2M1>(big, a, splits, stream)
                               : split_as<PMX_E4M3, PMX_E4M3>(big, a, splits, stream);
}

}  // namespace layer
}  // namespace pgemm
