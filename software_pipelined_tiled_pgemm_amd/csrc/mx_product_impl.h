// The kernels of the product of microscaled matrices with the linear layer's
// epilogue, for one element type of y (mx_product_f16.hip, mx_product_bf16.hip):
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
// range of the type, 2^-16 of the result for normally distributed values.  That is below
// the result's rounding to 16 bits (2^-11, 2^-8); whole fp32 sums would take the 16-bit
// instruction, at a quarter of the rate.
#pragma once

#include "linear_epi.h"
#include "mx_math.h"
#include "mx_product.h"

namespace pgemm {
namespace layer {
namespace {

using mxp::Frag;

// Few rows: a workgroup takes 16 rows of w (columns of y) and MB blocks of 16
// rows of x; its waves take turns at groups of 4 steps, and their sums are joined
// in LDS in a fixed order.  QUANTIZE: x comes in 16 bits (a few rows of it), and every
// workgroup quantises it for itself into LDS, while its first weights are on their
// way.
//
// Bound by the weights' way from memory, a token's also by the launch: 1 x 4096 x
// 8192 e4m3 x e2m1 6.3 us (17.8 MB at 2.8 TB/s).  (16 waves for long rows and few strips
// were no faster, and half as fast with 4 blocks of rows, which need the registers.)
constexpr int kFewWaves = 8;

template <class E, int FX, int FW, int MB, bool QUANTIZE>
__global__ __launch_bounds__(64 * kFewWaves) void few_rows_kernel(const MxArgs a, const LinearEpi<E> epi) {
    constexpr int W = kFewWaves;
    typedef Mx<FX> F;
    typedef mxp::i32x4 i32x4;
    __shared__ __attribute__((aligned(16))) floatx4 sums[W][MB][64];
    __shared__ __attribute__((aligned(16))) uint8_t codes[QUANTIZE ? kMxFewValues * F::kWords / 2 : 16];
    __shared__ __attribute__((aligned(16))) uint8_t scales[QUANTIZE ? kMxFewValues / 32 : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    u32x4 sw;
    Frag<FW> fw[4];
    auto load_w = [&](int s0) __attribute__((always_inline)) {
        sw = *reinterpret_cast<const u32x4*>(ws + s0 * 4);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int h = 0; h < Frag<FW>::kChunks; ++h)
                fw[q].c[h] = *reinterpret_cast<const i32x4*>(
                    w + ((int64_t)min(s0 + q, a.steps - 1) * Frag<FW>::kChunks + h) * 64);
    };
    const int group0 = wave * 4;
    if (group0 < a.steps) load_w(group0);
    if constexpr (QUANTIZE) {
        // rows of codes and of scales without gaps
        const int cpr = a.steps * 16;
        for (int row = 0; row < a.M; ++row)
            for (int c = threadIdx.x; c < cpr; c += 64 * W) {
                float v[8];
                u4_t bits = {};
                const int nv = min(8, a.cols - c * 8);
                if (nv > 0)
                    bits = load8_bits(Rows{const_cast<uint16_t*>(a.x16) + row * a.ldx16, 0, 0}, 0,
                                      c * 8, nv);
                unpack8<E>(bits, v);
                const uint32_t code = F::scale_code(most_of_quad(most8(v)));
                uint32_t out[F::kWords];
                F::encode8(v, code, out);
                __builtin_memcpy(codes + (row * cpr + c) * 4 * F::kWords, out, 4 * F::kWords);
                if ((c & 3) == 0) scales[(row * cpr + c) >> 2] = (uint8_t)code;
            }
        __syncthreads();
    }
    floatx4 acc[MB] = {};
    for (int s0 = group0; s0 < a.steps; s0 += W * 4) {
        if (s0 != group0) load_w(s0);
        uint32_t sx[4][MB];
        Frag<FX> fx[4][MB];
        if constexpr (QUANTIZE) {
            const int row = min(r, a.M - 1);
            const uint8_t* const at = codes + row * a.steps * Frag<FX>::kChunks * 64 + g * 16;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int s = min(s0 + q, a.steps - 1);
                sx[q][0] = *reinterpret_cast<const uint32_t*>(scales + (row * a.steps + s) * 4);
#pragma unroll
                for (int h = 0; h < Frag<FX>::kChunks; ++h)
                    fx[q][0].c[h] =
                        *reinterpret_cast<const i32x4*>(at + (s * Frag<FX>::kChunks + h) * 64);
            }
        } else {
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const u32x4 v = *reinterpret_cast<const u32x4*>(xs[b] + s0 * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    sx[q][b] = v[q];
#pragma unroll
                    for (int h = 0; h < Frag<FX>::kChunks; ++h)
                        fx[q][b].c[h] = *reinterpret_cast<const i32x4*>(
                            x[b] + ((int64_t)min(s0 + q, a.steps - 1) * Frag<FX>::kChunks + h) * 64);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (s0 + q < a.steps) {
#pragma unroll
                for (int b = 0; b < MB; ++b)
                    acc[b] = mxp::mma<FW, FX, 0>(fw[q], fx[q][b], acc[b], sw[q] >> (8 * g),
                                                 sx[q][b] >> (8 * g));
            }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) sums[wave][b][lane] = acc[b];
    __syncthreads();
    // Two neighbouring lane groups hold 8 consecutive columns of a row.
    for (int i = threadIdx.x; i < MB * 32; i += 64 * W) {
        const int b = i >> 5, c = (i >> 4) & 1, rr = i & 15;
        const int64_t row = m0 + 16 * b + rr;
        const int col = n0 + 8 * c, nv = min(8, a.N - col);
        if (row >= a.M || nv <= 0) continue;
        float v[8] = {};
#pragma unroll
        for (int k = 0; k < W; ++k) {
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
hipError_t launch_few(const MxArgs& a, const LinearEpi<E>& epi, hipStream_t stream) {
    const unsigned strips = (unsigned)((a.N + 15) / 16);
    auto go = [&](auto mb, auto quantize) {
        constexpr int MB = decltype(mb)::value;
        hipLaunchKernelGGL((few_rows_kernel<E, FX, FW, MB, decltype(quantize)::value>),
                           dim3(strips, (unsigned)((a.M + 16 * MB - 1) / (16 * MB))),
                           dim3(64 * kFewWaves), 0, stream, a, epi);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    if (a.x16) go(one, std::true_type{});
    else if (a.M <= 16) go(one, std::false_type{});
    else if (a.M <= 32) go(two, std::false_type{});
    else go(four, std::false_type{});
    return hipGetLastError();
}

template <class TL, int FX, int FW, class E>
hipError_t launch_tiles(MxArgs a, int splits, const LinearEpi<E>& epi, hipStream_t stream) {
    a.tiles_m = (a.M + TL::BM - 1) / TL::BM;
    a.tiles_n = (a.N + TL::BN - 1) / TL::BN;
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n), (unsigned)splits);
    if (splits == 1) {
        hipLaunchKernelGGL((mxp::product_kernel<TL, LinearEpi<E>>), grid, dim3(TL::T), 0,
                           stream, a, epi);
        return hipGetLastError();
    }
    const hipError_t rc = mx_split(FX, FW, TL::BM == 256, a, splits, stream);
    if (rc != hipSuccess) return rc;
    Args f = {};
    f.M = a.M, f.N = a.N, f.part = a.part, f.part_ld = a.part_ld;
    return lp::launch_finish(f, splits, 0, nullptr, epi, stream);
}

template <class E, int FX, int FW>
hipError_t product_as(const MxArgs& a, const MxCut& cut, const LinearEpi<E>& epi,
                      hipStream_t stream) {
    using T = MxTiles<FX, FW>;
    if (cut.few) return launch_few<E, FX, FW>(a, epi, stream);
    return cut.big ? launch_tiles<typename T::Big, FX, FW>(a, cut.splits, epi, stream)
                   : launch_tiles<typename T::Small, FX, FW>(a, cut.splits, epi, stream);
}

template <class E>
hipError_t product(int xformat, int wformat, const MxArgs& a, const MxCut& cut,
                   const MxLinearCall& c, hipStream_t stream) {
    const LinearEpi<E> epi = {make_rows(c.y, c.ldy), make_rows(c.residual, c.ldr),
                              make_rows(nullptr, 0), static_cast<const uint16_t*>(c.bias), c.act};
    if (xformat == PMX_E2M1)
        return wformat == PMX_E2M1 ? product_as<E, PMX_E2M1, PMX_E2M1>(a, cut, epi, stream)
                                   : product_as<E, PMX_E2M1, PMX_E4M3>(a, cut, epi, stream);
    return wformat == PMX_E2M1 ? product_as<E, PMX_E4M3, PMX_E2M1>(a, cut, epi, stream)
                               : product_as<E, PMX_E4M3, PMX_E4M3>(a, cut, epi, stream);
}

}  // namespace
}  // namespace layer
}  // namespace pgemm
