// Shared small kernels and host rules of the layer operators.
#include "layer.h"

#include <algorithm>

#include "layer_math.h"

namespace pgemm {
namespace layer {
namespace {

// Packing an operand whose rows are not whole 16-byte pieces: one thread
// writes 16 bytes of the padded copy.  Reads are 16 bytes from any 2-byte
// boundary (the compiler's unaligned global load), element by element at
// the row's end.  Bound by memory: each value is read and written once (2039
// x 1025: 2.4-5 us for 8 MB, mostly the launch).
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* __restrict__ src, int64_t ld,
                                                   uint16_t* __restrict__ dst, int64_t dst_ld,
                                                   int64_t rows, int cols) {
    const int cpr = (cols + 7) / 8;
    const int64_t total = rows * cpr;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / cpr;
        const int c = (int)(i - r * cpr) * 8;
        const uint16_t* p = src + r * ld + c;
        u4_t w;
        if (c + 8 <= cols) {
            __builtin_memcpy(&w, p, 16);
        } else {
            uint16_t e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = p[c + q < cols ? q : 0];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = c + q < cols ? e[q] : (uint16_t)0;
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = e[2 * q] | ((uint32_t)e[2 * q + 1] << 16);
        }
        *reinterpret_cast<u4_t*>(dst + r * dst_ld + c) = w;
    }
}

// out[c] = sum over r of part[r][c]: 64 columns per workgroup, its 16 waves
// each adding a sixteenth of the rows in ascending order (8 loads in flight),
// the sixteenths then in order.  Bound by latency: 128 rows of 4096 in 4 us
// (with 4 waves and one load in flight 12).
constexpr int kSegs = 16;
template <class E>
__global__ __launch_bounds__(64 * kSegs) void column_sum_kernel(const float* __restrict__ part,
                                                                int64_t parts, int64_t cols,
                                                                uint16_t* __restrict__ out) {
    __shared__ float sums[kSegs][64];
    const int lane = threadIdx.x & 63, seg = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < cols) {
        const int64_t per = (parts + kSegs - 1) / kSegs;
        const int64_t r1 = parts < (seg + 1) * per ? parts : (seg + 1) * per;
        int64_t r = seg * per;
        for (; r + 8 <= r1; r += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = part[(r + u) * cols + c];
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        for (; r < r1; ++r) s += part[r * cols + c];
    }
    sums[seg][lane] = s;
    __syncthreads();
    if (seg == 0 && c < cols) {
        float t = sums[0][lane];
        for (int k = 1; k < kSegs; ++k) t += sums[k][lane];
        out[c] = E::put(t);
    }
}

}  // namespace

hipError_t launch_pack(const uint16_t* src, int64_t ld, uint16_t* dst, int64_t dst_ld, int64_t rows,
                       int64_t cols, hipStream_t stream) {
    const int64_t chunks = rows * ((cols + 7) / 8);
    if (chunks == 0) return hipSuccess;
    const int64_t blocks = std::min<int64_t>((chunks + 255) / 256, 1 << 16);
    hipLaunchKernelGGL(pack_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, src, ld, dst, dst_ld,
                       rows, (int)cols);
    return hipGetLastError();
}

hipError_t launch_column_sum(int dtype, const float* part, int64_t parts, int64_t cols, void* out,
                             hipStream_t stream) {
    const dim3 grid((unsigned)((cols + 63) / 64));
    if (dtype == kBF16)
        hipLaunchKernelGGL(column_sum_kernel<BF16>, grid, dim3(64 * kSegs), 0, stream, part, parts, cols,
                           static_cast<uint16_t*>(out));
    else
        hipLaunchKernelGGL(column_sum_kernel<F16>, grid, dim3(64 * kSegs), 0, stream, part, parts, cols,
                           static_cast<uint16_t*>(out));
    return hipGetLastError();
}

namespace {
// Estimated microseconds of a cut, with the constants measured on MI355X at long
// K: a 256x256 tile takes 0.65 us per K step of 32, two 128x128 tiles on a CU 0.57
// (their LDS reads bound them: half the product for nearly the time), one
// alone 0.33; a round of workgroups adds its prologue and epilogue, and a
// split a second launch and the partials' traffic.  It ranks cuts and is no
// forecast: 2039 x 2047 x 1025, where launch and edges count, is 14.5 by it and
// takes 20; reading the weights of a few rows has no term of its own.
double cut_time(int64_t M, int64_t N, int64_t K, int cus, bool big, int splits) {
    const int64_t b = big ? 256 : 128;
    const int64_t wgs = ((M + b - 1) / b) * ((N + b - 1) / b) * splits;
    const int64_t slots = big ? cus : 2 * cus;
    const double step = big ? 0.65 : wgs <= cus ? 0.33 : 0.57;
    const double rounds = (double)((wgs + slots - 1) / slots);
    const double steps = (double)((K + splits * 32 - 1) / (splits * 32)) + 2;
    double t = rounds * (steps * step + (big ? 6.0 : 3.0));
    if (splits > 1) t += 3.0 + (double)splits * M * N * 8.0 / 4.0e6;
    return t;
}
}  // namespace

Cut choose_cut(int64_t M, int64_t N, int64_t K, int cus, int max_splits) {
    static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
    Cut best = {false, 1, K};
    double best_t = 1e300;
    for (int s : kSplits) {
        if (s > max_splits || (s > 1 && K / s < 256)) break;
        const int64_t chunk = round_up((K + s - 1) / s, 64);
        const int parts = s == 1 ? 1 : (int)((K + chunk - 1) / chunk);
        for (int big = 0; big < 2; ++big) {
            const double t = cut_time(M, N, K, cus, big != 0, parts);
            if (t < best_t) {
                best_t = t;
                best = {big != 0, parts, parts > 1 ? chunk : K};
            }
        }
    }
    return best;
}

}  // namespace layer
}  // namespace pgemm
