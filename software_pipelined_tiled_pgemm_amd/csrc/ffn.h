// Calls of the gated feed-forward block, as the C entry points hand them on
// (validated).
#pragma once

#include "layer.h"

namespace pgemm {
namespace layer {

struct FfnCall {
    int dtype;
    const void* x;
    int64_t ldx;
    const void* w_in;
    int64_t ldwi;
    const void* w_out;
    int64_t ldwo;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    void* gate_up;
    int64_t ldgu;
    int64_t M, D, F, N;  // x [M,D], w_in [D,2F], w_out [F,N], y [M,N]
    int act;
};

struct FfnGradCall {
    int dtype;
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const void* w_in;
    int64_t ldwi;
    const void* w_out;
    int64_t ldwo;
    const void* gate_up;
    int64_t ldgu;
    const void* add;  // added to dx
    int64_t ldadd;
    void* dx;
    int64_t lddx;
    void* dw_in;
    int64_t lddwi;
    void* dw_out;
    int64_t lddwo;
    int64_t M, D, F, N;
    int act;
};

hipError_t ffn_forward(const FfnCall& c, Arena& ar, hipStream_t stream);
hipError_t ffn_backward(const FfnGradCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
