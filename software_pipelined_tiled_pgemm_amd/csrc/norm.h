// Calls of the root-mean-square norm, as the C entry points hand them on
// (validated).
#pragma once

#include "layer.h"
#include "mx.h"

namespace pgemm {
namespace layer {

struct NormCall {
    int dtype;
    const void* x;
    int64_t ldx;
    const void* residual;
    int64_t ldr;
    const void* weight;
    void* h;
    int64_t ldh;
    int format;  // below 0: y; else mx
    void* y;
    int64_t ldy;
    MxRows mx;
    int64_t M, D;
    float eps;
};
hipError_t norm_forward(const NormCall& c, hipStream_t stream);

struct NormGradCall {
    int dtype;
    const void* dy;
    int64_t lddy;
    const void* h;
    int64_t ldh;
    const void* residual;  // where not NULL, added to h in fp32
    int64_t ldr;
    const void* weight;
    const void* dh;
    int64_t lddh;
    void* dx;
    int64_t lddx;
    void* dw;
    int64_t M, D;
    float eps;
};
// With a dry arena nothing is launched and only the workspace is counted.
hipError_t norm_backward(const NormGradCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
