// The linear layer on microscaled matrices: x's quantisation where it is not yet
// microscaled, the choice of kernel, workspace.
#include <algorithm>

#include "internal.h"
#include "mx.h"
#include "mx_math.h"

namespace pgemm {
namespace layer {
namespace {

MxCut choose_mx_cut(int xformat, int wformat, int64_t M, int64_t N, int steps, int cus) {
    if (M <= 64) return {true, false, 1, steps};
    const int64_t bn = xformat == PMX_E4M3 && wformat == PMX_E4M3 ? 128 : 256;
    const int64_t big = ((M + 255) / 256) * ((N + bn - 1) / bn);
    return {false, big >= cus, 1, steps};
}

}  // namespace

hipError_t mx_linear(const MxLinearCall& c, Arena& ar, hipStream_t stream) {
    if (c.M == 0 || c.N == 0) return hipSuccess;
    MxRows x = c.x;
    if (c.x16) {
        x.ld = mx_row_bytes(x.format, c.K);
        x.lds = round_up(mx_scale_bytes(c.K), 16);
        x.codes = static_cast<uint8_t*>(ar.take(c.M * x.ld));
        x.scales = static_cast<uint8_t*>(ar.take(c.M * x.lds));
        if (!ar.dry()) {
            const hipError_t rc = mx_quantize(c.dtype, c.x16, c.ldx16, x, c.M, c.K, stream);
            if (rc != hipSuccess) return rc;
        }
    }
    MxArgs a = {};
    a.x = x.codes, a.xs = x.scales, a.w = c.w.codes, a.ws = c.w.scales;
    a.ldx = x.ld, a.ldxs = x.lds, a.ldw = c.w.ld, a.ldws = c.w.lds;
    a.M = (int)c.M, a.N = (int)c.N, a.steps = (int)(mx_padded(c.K) / kMxGroup);
    const MxCut cut = choose_mx_cut(x.format, c.w.format, c.M, c.N, a.steps, compute_units());
    a.chunk = cut.chunk;
    if (cut.splits > 1) {
        a.part_ld = (int)round_up(a.N, 8);
        a.part = static_cast<float*>(ar.take((int64_t)cut.splits * a.M * a.part_ld * 4));
    }
    if (ar.dry()) return hipSuccess;
    return c.dtype == kBF16 ? mx_product_bf16(x.format, c.w.format, a, cut, c, stream)
                            : mx_product_f16(x.format, c.w.format, a, cut, c, stream);
}

}  // namespace layer
}  // namespace pgemm
