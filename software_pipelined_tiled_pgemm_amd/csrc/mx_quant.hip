// Microscaled quantisation of 16-bit matrices, and back.
//
// A lane takes 8 columns (16 bytes of 16-bit values), 4 neighbouring lanes a
// block of 32: the block's largest magnitude is two lane exchanges.  Bound by
// memory.
#include <algorithm>

#include "layer_math.h"
#include "mx.h"
#include "mx_math.h"

namespace pgemm {
namespace layer {
namespace {

// Chunks of 8 columns from any 2-byte boundary, zeros from cols on.
__device__ __forceinline__ u4_t chunk_bits(const uint16_t* row, int col, int cols) {
    const int nv = min(8, cols - col);
    u4_t w = {};
    if (nv == 8) {
        __builtin_memcpy(&w, row + col, 16);
    } else if (nv > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            w[q >> 1] |= (uint32_t)(q < nv ? row[col + q] : 0) << (16 * (q & 1));
    }
    return w;
}

template <class E, int FORMAT>
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                       const MxRows out, int64_t rows, int cols,
                                                       int cpr) {
    typedef Mx<FORMAT> F;
    const int64_t total = rows * cpr;  // a multiple of 4: blocks do not straddle the end
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cpr;
        const int c = (int)(i - r * cpr);
        float v[8];
        unpack8<E>(chunk_bits(x + r * ldx, c * 8, cols), v);
        const uint32_t code = F::scale_code(most_of_quad(most8(v)));
        uint32_t w[F::kWords];
        F::encode8(v, code, w);
        __builtin_memcpy(out.codes + r * out.ld + c * 4 * F::kWords, w, 4 * F::kWords);
        if ((c & 3) == 0) out.scales[r * out.lds + (c >> 2)] = (uint8_t)code;
    }
}

template <class E, int FORMAT>
__global__ __launch_bounds__(256) void dequantize_kernel(const MxRows x, uint16_t* __restrict__ y,
                                                         int64_t ldy, int64_t rows, int cols,
                                                         int cpr) {
    typedef Mx<FORMAT> F;
    const int64_t total = rows * cpr;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cpr;
        const int c = (int)(i - r * cpr);
        uint32_t w[F::kWords];
        __builtin_memcpy(w, x.codes + r * x.ld + c * 4 * F::kWords, 4 * F::kWords);
        float v[8];
        F::decode8(w, mx_scale(x.scales[r * x.lds + (c >> 2)]), v);
        store8<E, false>(Rows{y + r * ldy, 0, 0}, 0, c * 8, min(8, cols - c * 8), v);
    }
}

constexpr int64_t kMostBlocks = 1 << 16;

template <class Run>
hipError_t with_types(int dtype, int format, Run&& run) {
    if (dtype == kBF16)
        format == PMX_E2M1 ? run(BF16{}, std::integral_constant<int, PMX_E2M1>{})
                           : run(BF16{}, std::integral_constant<int, PMX_E4M3>{});
    else
        format == PMX_E2M1 ? run(F16{}, std::integral_constant<int, PMX_E2M1>{})
                           : run(F16{}, std::integral_constant<int, PMX_E4M3>{});
    return hipGetLastError();
}

}  // namespace

hipError_t mx_quantize(int dtype, const void* x, int64_t ldx, const MxRows& out, int64_t rows,
                       int64_t cols, hipStream_t stream) {
    const int cpr = (int)(mx_padded(cols) / 8);
    const int64_t chunks = rows * cpr;
    if (chunks == 0) return hipSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>((chunks + 255) / 256, kMostBlocks);
    return with_types(dtype, out.format, [&](auto e, auto f) {
        hipLaunchKernelGGL((quantize_kernel<decltype(e), decltype(f)::value>), dim3(blocks),
                           dim3(256), 0, stream, static_cast<const uint16_t*>(x), ldx, out, rows,
                           (int)cols, cpr);
    });
}

hipError_t mx_dequantize(const MxRows& x, int dtype, void* y, int64_t ldy, int64_t rows,
                         int64_t cols, hipStream_t stream) {
    const int cpr = (int)((cols + 7) / 8);
    const int64_t chunks = rows * cpr;
    if (chunks == 0) return hipSuccess;
    const unsigned blocks = (unsigned)std::min<int64_t>((chunks + 255) / 256, kMostBlocks);
    return with_types(dtype, x.format, [&](auto e, auto f) {
        hipLaunchKernelGGL((dequantize_kernel<decltype(e), decltype(f)::value>), dim3(blocks),
                           dim3(256), 0, stream, x, static_cast<uint16_t*>(y), ldy, rows,
                           (int)cols, cpr);
    });
}

}  // namespace layer
}  // namespace pgemm
