// Microscaled quantisation of 16-bit matrices, and back.
//
// A lane takes 8 columns (16 bytes of 16-bit values), 4 neighbouring lanes a
// block of 32: the block's largest magnitude is two lane exchanges.  Bound by
// memory: 16384 x 4096 bf16 to e2m1 28-33 us (5.2-6.0 TB/s), back 26 (6.5).
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

// A workgroup takes 2^shift lanes of chunks and 256 >> shift rows at a time, AHEAD times
// that many rows with all loads under way at once, and walks the rows; its columns
// are blockIdx.x's.  (A division per chunk to find its row took a tenth of the time:
// 16384 x 4096 bf16 to e2m1 37 -> 33 us.)  AHEAD is 4, or 1 where that leaves fewer than
// 2048 workgroups (67 x 2050: 4.0 us with 4, 2.9 with 1).
template <int AHEAD>
struct Walk {
    static constexpr int kAhead = AHEAD;
    int64_t rows;
    int chunks, shift;
    __device__ __forceinline__ int chunk() const {
        return (blockIdx.x << shift) + (threadIdx.x & ((1 << shift) - 1));
    }
    // f(row), g(row) for AHEAD rows at a time: all f before the first g.
    template <class F, class G>
    __device__ __forceinline__ void each(F&& f, G&& g) const {
        const int per = 256 >> shift;
        for (int64_t r0 = (int64_t)blockIdx.y * per * AHEAD + (threadIdx.x >> shift); r0 < rows;
             r0 += (int64_t)gridDim.y * per * AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (r0 + u * per < rows) f(u, r0 + u * per);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (r0 + u * per < rows) g(u, r0 + u * per);
        }
    }
};

template <class E, int FORMAT, int AHEAD>
__global__ __launch_bounds__(256) void quantize_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                       const MxRows out, const Walk<AHEAD> walk, int cols) {
    typedef Mx<FORMAT> F;
    const int c = walk.chunk();
    if (c >= walk.chunks) return;  // chunks are whole blocks: four lanes at a time
    u4_t b[AHEAD];
    walk.each([&](int u, int64_t r) __attribute__((always_inline)) {
                  b[u] = chunk_bits(x + r * ldx, c * 8, cols);
              },
              [&](int u, int64_t r) __attribute__((always_inline)) {
                  float v[8];
                  unpack8<E>(b[u], v);
                  const uint32_t code = F::scale_code(most_of_quad(most8(v)));
                  uint32_t w[F::kWords];
                  F::encode8(v, code, w);
                  __builtin_memcpy(out.codes + r * out.ld + c * 4 * F::kWords, w, 4 * F::kWords);
                  if ((c & 3) == 0) out.scales[r * out.lds + (c >> 2)] = (uint8_t)code;
              });
}

template <class E, int FORMAT, int AHEAD>
__global__ __launch_bounds__(256) void dequantize_kernel(const MxRows x, uint16_t* __restrict__ y,
                                                         int64_t ldy, const Walk<AHEAD> walk, int cols,
                                                         bool past) {
    typedef Mx<FORMAT> F;
    const int c = walk.chunk();
    if (c >= walk.chunks) return;
    uint32_t w[AHEAD][F::kWords];
    uint8_t s[AHEAD];
    walk.each([&](int u, int64_t r) __attribute__((always_inline)) {
                  __builtin_memcpy(w[u], x.codes + r * x.ld + c * 4 * F::kWords, 4 * F::kWords);
                  s[u] = x.scales[r * x.lds + (c >> 2)];
              },
              [&](int u, int64_t r) __attribute__((always_inline)) {
                  float v[8];
                  F::decode8(w[u], mx_scale(s[u]), v);
                  const Rows to = {y + r * ldy, 0, 0};
                  if (past)
                      store8<E, true>(to, 0, c * 8, min(8, cols - c * 8), v);
                  else
                      store8<E, false>(to, 0, c * 8, min(8, cols - c * 8), v);
              });
}

// run(walk, grid) with the walk over `chunks` columns of 8.
template <class Run>
void with_walk(int64_t rows, int chunks, Run&& run) {
    int shift = 4;
    while (shift < 8 && (1 << shift) < chunks) ++shift;
    const unsigned x = (unsigned)((chunks + (1 << shift) - 1) >> shift);
    const int64_t per = 256 >> shift, most = 65535;
    if ((rows + 4 * per - 1) / (4 * per) * x >= 2048)
        run(Walk<4>{rows, chunks, shift},
            dim3(x, (unsigned)std::min((rows + 4 * per - 1) / (4 * per), most)));
    else
        run(Walk<1>{rows, chunks, shift}, dim3(x, (unsigned)std::min((rows + per - 1) / per, most)));
}
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
    if (rows == 0 || cols == 0) return hipSuccess;
    return with_types(dtype, out.format, [&](auto e, auto f) {
        with_walk(rows, (int)(mx_padded(cols) / 8), [&](auto walk, dim3 grid) {
            hipLaunchKernelGGL((quantize_kernel<decltype(e), decltype(f)::value, decltype(walk)::kAhead>),
                               grid, dim3(256), 0, stream, static_cast<const uint16_t*>(x), ldx, out,
                               walk, (int)cols);
        });
    });
}

// Values that take half of the memory-side cache and more are stored past the caches: what
// their reader makes of them, as large again, would push them out.  us with the product that
// reads them (4096 outputs; 256 outputs), kept / past, rows of 4096 bf16 from e2m1:
//      8192 rows (64 MB)   194.7 / 196.9   44.1 / 50.5
//     12288 (96)           287.2 / 294.1   54.4 / 69.6
//     14336 (112)          366.9 / 376.2   68.0 / 75.2
//     16384 (128)          395.5 / 393.2   89.8 / 80.9
//     20480 (160)          484.5 / 488.4  106.9 / 103.6
constexpr int64_t kPast = kMemorySide / 2;

hipError_t mx_dequantize(const MxRows& x, int dtype, void* y, int64_t ldy, int64_t rows,
                         int64_t cols, hipStream_t stream) {
    if (rows == 0 || cols == 0) return hipSuccess;
    return with_types(dtype, x.format, [&](auto e, auto f) {
        with_walk(rows, (int)((cols + 7) / 8), [&](auto walk, dim3 grid) {
            hipLaunchKernelGGL(
                (dequantize_kernel<decltype(e), decltype(f)::value, decltype(walk)::kAhead>), grid,
                dim3(256), 0, stream, x, static_cast<uint16_t*>(y), ldy, walk, (int)cols,
                rows * cols * 2 >= kPast);
        });
    });
}

}  // namespace layer
}  // namespace pgemm
