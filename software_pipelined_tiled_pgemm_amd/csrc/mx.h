// Calls of the microscaled operators, as the C entry points hand them on
// (validated).
#pragma once

#include "layer.h"

namespace pgemm {
namespace layer {

// A microscaled matrix: rows of elements and rows of scales, pitches in bytes.
struct MxRows {
    int format;
    uint8_t* codes;
    int64_t ld;
    uint8_t* scales;
    int64_t lds;
};

hipError_t mx_quantize(int dtype, const void* x, int64_t ldx, const MxRows& out, int64_t rows,
                       int64_t cols, hipStream_t stream);
hipError_t mx_dequantize(const MxRows& x, int dtype, void* y, int64_t ldy, int64_t rows,
                         int64_t cols, hipStream_t stream);

// y [M, N] = act(x w^T + bias) + residual.  x16: the 16-bit matrix that x's
// elements are made of first, in the workspace (x.codes is NULL then).
struct MxLinearCall {
    int dtype;
    MxRows x;
    const void* x16;
    int64_t ldx16;
    MxRows w;
    const void* bias;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    int64_t M, N, K;
    int act;
};
// With a dry arena nothing is launched and only the workspace is counted.
hipError_t mx_linear(const MxLinearCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
