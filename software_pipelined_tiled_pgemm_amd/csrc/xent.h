// Calls of the vocabulary cross entropy, as the C entry points hand them on
// (validated).
#pragma once

#include "layer.h"

namespace pgemm {
namespace layer {

struct XentCall {
    int dtype;
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;
    const int64_t* target;
    int64_t ignore_index;
    int reduction;
    float* loss;
    float* lse;
    int64_t M, V, D;  // x [M,D], w [V,D]
};

struct XentGradCall {
    int dtype;
    const void* x;
    int64_t ldx;
    const void* w;
    int64_t ldw;
    const int64_t* target;
    int64_t ignore_index;
    int reduction;
    const float* lse;
    const float* dloss;
    void* dx;
    int64_t lddx;
    void* dw;
    int64_t lddw;
    int64_t M, V, D;
};

hipError_t xent_forward(const XentCall& c, Arena& ar, hipStream_t stream);
hipError_t xent_backward(const XentGradCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
