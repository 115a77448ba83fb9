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

// A product x w^T and its tile grid, as the kernels take it.
struct MxArgs {
    const uint8_t *x, *xs, *w, *ws;
    int64_t ldx, ldxs, ldw, ldws;
    int M, N, steps;  // steps of 128 columns
    // where not NULL, x in 16 bits, `cols` columns, which the kernel quantises
    const uint16_t* x16;
    int64_t ldx16;
    int cols;
    int tiles_m, tiles_n;
    int chunk;    // split: steps per split, a multiple of 4
    float* part;  // split: partials [split][M][part_ld]
    int part_ld;
};

// Values of x (padded) that the kernel for few rows quantises itself.
constexpr int64_t kMxFewValues = 16384;

// How a product is cut: the kernel for few rows, or tiles (256 or 128 rows) with the
// contraction in `splits` parts of `chunk` steps.
struct MxCut {
    bool few, big;
    int splits, chunk;
};

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
// The kernels, with y in fp16 (mx_product_f16.hip) or bf16 (mx_product_bf16.hip), and
// the partial products of a split one (mx_split.hip; a has its tiles counted).
hipError_t mx_product_f16(int xformat, int wformat, const MxArgs& a, const MxCut& cut,
                          const MxLinearCall& c, hipStream_t stream);
hipError_t mx_product_bf16(int xformat, int wformat, const MxArgs& a, const MxCut& cut,
                           const MxLinearCall& c, hipStream_t stream);
hipError_t mx_split(int xformat, int wformat, bool big, const MxArgs& a, int splits,
                    hipStream_t stream);
// With a dry arena nothing is launched and only the workspace is counted.
hipError_t mx_linear(const MxLinearCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
