// The product of microscaled matrices with the linear layer's epilogue:
//   y = act(x w^T + bias) + residual,   x [M, K], w [N, K], each value its
// element times 2^(scale of its block of 32).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 contracts 128 columns: lane (r, g) = (l % 16,
// l / 16) holds row r's elements of columns 32 g .. + 31 in 4 bits (16 bytes), in 8
// bits those of columns 16 g .. + 15 and 64 + 16 g .. + 15 (two times 16 bytes),
// and the scale of columns 32 g .. + 31 in one byte of a register (layout checked
// on gfx950 against products in binary64).  As in the 16-bit products w is the
// row operand, so a lane ends up with 4 consecutive columns of one row of y.
//
// The instruction adds the products of 4-bit elements without loss.  With 8-bit
// ones on either side a product far below the largest of its 128 loses bits:
// up to 2^-11 of the largest product was measured for elements over the whole
// range of the type, 2^-16 of the result for normally distributed values.
#include <algorithm>

#include "linear_epi.h"
#include "mx.h"
#include "mx_math.h"

namespace pgemm {
namespace layer {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// The elements of a lane: 16 bytes (e2m1) or 32 (e4m3).
template <int FORMAT>
struct Frag {
    static constexpr int kChunks = FORMAT == PMX_E2M1 ? 1 : 2;
    static constexpr int kCode = FORMAT == PMX_E2M1 ? 4 : 0;  // of the instruction's operand type
    i32x4 c[kChunks];
    __device__ __forceinline__ i32x8 operand() const {
        const i32x4 hi = c[kChunks - 1];
        return {c[0][0], c[0][1], c[0][2], c[0][3], hi[0], hi[1], hi[2], hi[3]};
    }
};

// c + w x^T for one 128 columns; BYTE: which byte of the scales.
template <int FW, int FX, int BYTE_W, int BYTE_X>
__device__ __forceinline__ floatx4 mx_mma(const Frag<FW>& w, const Frag<FX>& x, floatx4 c,
                                          uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        w.operand(), x.operand(), c, Frag<FW>::kCode, Frag<FX>::kCode, BYTE_W, (int)sw, BYTE_X,
        (int)sx);
}

struct MxArgs {
    const uint8_t *x, *xs, *w, *ws;
    int64_t ldx, ldxs, ldw, ldws;
    int M, N, steps;  // steps of 128 columns
};

// Few rows: a workgroup takes 16 rows of w (columns of y) and MB blocks of 16
// rows of x; its waves take turns at groups of 4 steps, and their sums are joined
// in LDS in a fixed order.
constexpr int kFewWaves = 8;

template <class E, int FX, int FW, int MB>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(const MxArgs a,
                                                                  const LinearEpi<E> epi) {
    __shared__ __attribute__((aligned(16))) floatx4 sums[kFewWaves][MB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MB);
    // rows past the end read the last one and are not stored
    const uint8_t* const w = a.w + (int64_t)min(n0 + r, a.N - 1) * a.ldw + g * 16;
    const uint8_t* const ws = a.ws + (int64_t)min(n0 + r, a.N - 1) * a.ldws;
    const uint8_t *x[MB], *xs[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t row = min(m0 + 16 * b + r, (int64_t)a.M - 1);
        x[b] = a.x + row * a.ldx + g * 16;
        xs[b] = a.xs + row * a.ldxs;
    }
    floatx4 acc[MB] = {};
    for (int s0 = wave * 4; s0 < a.steps; s0 += kFewWaves * 4) {
        const u32x4 sw = *reinterpret_cast<const u32x4*>(ws + s0 * 4);
        u32x4 sx[MB];
#pragma unroll
        for (int b = 0; b < MB; ++b) sx[b] = *reinterpret_cast<const u32x4*>(xs[b] + s0 * 4);
        Frag<FW> fw[4];
        Frag<FX> fx[4][MB];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t s = min(s0 + q, a.steps - 1);
#pragma unroll
            for (int h = 0; h < Frag<FW>::kChunks; ++h)
                fw[q].c[h] = *reinterpret_cast<const i32x4*>(
                    w + (s * Frag<FW>::kChunks + h) * 64);
#pragma unroll
            for (int b = 0; b < MB; ++b)
#pragma unroll
                for (int h = 0; h < Frag<FX>::kChunks; ++h)
                    fx[q][b].c[h] = *reinterpret_cast<const i32x4*>(
                        x[b] + (s * Frag<FX>::kChunks + h) * 64);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (s0 + q < a.steps) {
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    acc[b] = mx_mma<FW, FX, 0, 0>(fw[q], fx[q][b], acc[b], sw[q] >> (8 * g),
                                                  sx[b][q] >> (8 * g));
            }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) sums[wave][b][lane] = acc[b];
    __syncthreads();
    // Two neighbouring lane groups hold 8 consecutive columns of a row.
    for (int i = threadIdx.x; i < MB * 32; i += 64 * kFewWaves) {
        const int b = i >> 5, c = (i >> 4) & 1, rr = i & 15;
        const int64_t row = m0 + 16 * b + rr;
        const int col = n0 + 8 * c, nv = min(8, a.N - col);
        if (row >= a.M || nv <= 0) continue;
        float v[8] = {};
#pragma unroll
        for (int k = 0; k < kFewWaves; ++k) {
            const floatx4 lo = sums[k][b][32 * c + rr], hi = sums[k][b][32 * c + 16 + rr];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] += lo[q];
                v[4 + q] += hi[q];
            }
        }
        const LinearEpi<E> at = epi.from(row);
        const auto column = at.column(col, nv);
        const auto aux = at.load(0, col, nv);
        at.template with<false>([&](const auto& f) __attribute__((always_inline)) {
            f(0, col, nv, v, column, aux);
        });
    }
}

template <class E, int FX, int FW>
hipError_t launch(const MxArgs& a, const LinearEpi<E>& epi, hipStream_t stream) {
    const unsigned strips = (unsigned)((a.N + 15) / 16);
    // blocks of rows, in launches of at most 65535 (grid y)
    auto go = [&](auto mb) {
        constexpr int MB = decltype(mb)::value;
        constexpr int64_t kMost = (int64_t)65535 * 16 * MB;
        for (int64_t r0 = 0; r0 < a.M; r0 += kMost) {
            MxArgs p = a;
            p.x += r0 * a.ldx;
            p.xs += r0 * a.ldxs;
            p.M = (int)std::min<int64_t>(a.M - r0, kMost);
            LinearEpi<E> e = epi;
            e.y.ptr += r0 * e.y.ld;
            if (e.res.ptr) e.res.ptr += r0 * e.res.ld;
            hipLaunchKernelGGL((few_rows_kernel<E, FX, FW, MB>),
                               dim3(strips, (unsigned)((p.M + 16 * MB - 1) / (16 * MB))),
                               dim3(64 * kFewWaves), 0, stream, p, e);
        }
    };
    if (a.M <= 16) go(std::integral_constant<int, 1>{});
    else if (a.M <= 32) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 4>{});
    return hipGetLastError();
}

template <class E>
hipError_t linear_as(const MxLinearCall& c, Arena& ar, hipStream_t stream) {
    MxRows x = c.x;
    if (c.x16) {
        x.ld = mx_row_bytes(x.format, c.K);
        x.lds = round_up(mx_scale_bytes(c.K), 16);
        x.codes = static_cast<uint8_t*>(ar.take(c.M * x.ld));
        x.scales = static_cast<uint8_t*>(ar.take(c.M * x.lds));
    }
    if (ar.dry()) return hipSuccess;
    if (c.x16) {
        const hipError_t rc = mx_quantize(c.dtype, c.x16, c.ldx16, x, c.M, c.K, stream);
        if (rc != hipSuccess) return rc;
    }
    const MxArgs a = {x.codes, x.scales, c.w.codes, c.w.scales, x.ld, x.lds, c.w.ld, c.w.lds,
                      (int)c.M, (int)c.N, (int)(mx_padded(c.K) / kMxGroup)};
    const LinearEpi<E> epi = {make_rows(c.y, c.ldy), make_rows(c.residual, c.ldr),
                              make_rows(nullptr, 0), static_cast<const uint16_t*>(c.bias), c.act};
    if (x.format == PMX_E2M1)
        return c.w.format == PMX_E2M1 ? launch<E, PMX_E2M1, PMX_E2M1>(a, epi, stream)
                                      : launch<E, PMX_E2M1, PMX_E4M3>(a, epi, stream);
    return c.w.format == PMX_E2M1 ? launch<E, PMX_E4M3, PMX_E2M1>(a, epi, stream)
                                  : launch<E, PMX_E4M3, PMX_E4M3>(a, epi, stream);
}

}  // namespace

hipError_t mx_linear(const MxLinearCall& c, Arena& ar, hipStream_t stream) {
    if (c.M == 0 || c.N == 0) return hipSuccess;
    return c.dtype == kBF16 ? linear_as<BF16>(c, ar, stream) : linear_as<F16>(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
