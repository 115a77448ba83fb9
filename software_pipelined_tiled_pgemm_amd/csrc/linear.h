// Calls of the linear layer, as the C entry points hand them on (validated).
#pragma once

#include "layer.h"

namespace pgemm {
namespace layer {

struct LinearCall {
    int dtype;
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;
    const void* bias;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    void* preact;
    int64_t ldp;
    int64_t M, N, K;
    int act;
};

struct LinearGradCall {
    int dtype;
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;
    const void* preact;
    int64_t ldp;
    const void* add;  // added to dx
    int64_t ldadd;
    void* dx;
    int64_t lddx;
    void* dw;
    int64_t lddw;
    void* dbias;
    int64_t M, N, K;
    int act;
};

// Where a product's values go: y = act(v + bias) + residual, v + bias to
// preact; null members are left out.  NT and TN products (gradients) take
// residual only.  half > 0 (not NN): the product's columns are two halves, each
// padded from `half` to round_up(half, 8) columns, which y holds without the
// padding (no residual then).
struct Sink {
    void* y;
    int64_t ldy;
    const void* residual;
    int64_t ldr;
    void* preact;
    int64_t ldp;
    const void* bias;
    int act;
    int half;
};
hipError_t launch_linear(int dtype, int layout, const Args& g, const Cut& cut, const Sink& sink,
                         hipStream_t stream);

// With a dry arena nothing is launched and only the workspace is counted.
hipError_t linear_forward(const LinearCall& c, Arena& ar, hipStream_t stream);
hipError_t linear_backward(const LinearGradCall& c, Arena& ar, hipStream_t stream);

// The operand [rows, cols] as the pipeline can copy it: itself, or a padded
// copy in the workspace.
inline hipError_t operand(const void* p, int64_t ld, int64_t rows, int64_t cols, Arena& ar,
                          hipStream_t stream, View& out) {
    if (direct(p, ld, cols)) {
        out = {static_cast<const uint16_t*>(p), (int)ld};
        return hipSuccess;
    }
    const int64_t c8 = round_up(cols, 8);
    uint16_t* dst = static_cast<uint16_t*>(ar.take(rows * c8 * 2));
    out = {dst, (int)c8};
    if (ar.dry()) return hipSuccess;
    return launch_pack(static_cast<const uint16_t*>(p), ld, dst, c8, rows, cols, stream);
}

// The arguments of C[M, N] = a . b over K, with room for the cut's partials.
inline Args args(View a, View b, int64_t M, int64_t N, int64_t K, const Cut& cut, Arena& ar) {
    Args g = {};
    g.a = a;
    g.b = b;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    const int64_t pb = part_bytes(cut, M, N);
    if (pb > 0) {
        g.part = static_cast<float*>(ar.take(pb));
        g.part_ld = (int)round_up(N, 8);
    }
    return g;
}

}  // namespace layer
}  // namespace pgemm
