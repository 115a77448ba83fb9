// The microscaled product with y in bf16.
#include "mx_product_impl.h"

namespace pgemm {
namespace layer {

hipError_t mx_product_bf16(int xformat, int wformat, const MxArgs& a, const MxCut& cut,
                          const MxLinearCall& c, hipStream_t stream) {
    return product<BF16>(xformat, wformat, a, cut, c, stream);
}

}  // namespace layer
}  // namespace pgemm
