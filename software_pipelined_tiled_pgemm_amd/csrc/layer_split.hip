// Partial products of the layer operators' split-K launches: every operand
// layout and type, the fp32 partials stored row by row for a finish kernel.
#include "layer_pipe.h"

namespace pgemm {
namespace layer {

namespace {
template <class E, bool AKC, bool BKC>
hipError_t run(const Args& g, const Cut& cut, hipStream_t stream) {
    using T = lp::Tiles<E, AKC, BKC>;
    const lp::StorePart sp = {g.part, g.part_ld};
    return cut.big ? lp::launch_tiles<typename T::Big, lp::StorePart, true>(g, cut.splits, sp, stream)
                   : lp::launch_tiles<typename T::Small, lp::StorePart, true>(g, cut.splits, sp,
                                                                              stream);
}

template <class E>
hipError_t run_layout(int layout, const Args& g, const Cut& cut, hipStream_t stream) {
    switch (layout) {
        case kNN: return run<E, true, false>(g, cut, stream);
        case kNT: return run<E, true, true>(g, cut, stream);
        default: return run<E, false, false>(g, cut, stream);
    }
}
}  // namespace

hipError_t launch_split(int dtype, int layout, const Args& g, const Cut& cut, hipStream_t stream) {
    Args a = g;
    a.chunk = (int)cut.chunk;
    return dtype == kBF16 ? run_layout<BF16>(layout, a, cut, stream)
                          : run_layout<F16>(layout, a, cut, stream);
}

}  // namespace layer
}  // namespace pgemm
