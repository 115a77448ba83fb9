// The root-mean-square norm with the residual's addition, and its backward pass.
//
//   forward    h = x + r,  n = h / sqrt(mean(h^2) + eps),  y = n w
//   backward   g = dy w,  dx = (g - n mean(g n)) / sqrt(mean(h^2) + eps) + dh,
//              dw = sum over rows of dy n
//
// h is summed in fp32 and normed as it is; what is stored of it is rounded once.
// The backward pass takes the stored h and computes the mean square again (the
// row is in registers anyway), so the forward pass keeps nothing else.  That h is
// rounded costs dw a rounding (16384 rows of bf16: 2.4e-3 of its norm off instead of
// 1.6e-3) and saves a matrix; a caller who wants it exact gives x and r, whose sum is
// taken again (SUM: 16384 x 4096 bf16 115 us with dw's sum instead of 93).  dw adds fp32
// products in a fixed order.
//
// A row of up to 32768 columns (backward: 16384) is held in registers by 64 lanes (no
// barrier) or by a workgroup; all passes over it after the first are free of memory, which
// bounds both (longer rows are read again for each pass):
//   16384 x 4096 bf16 (134 MB a matrix)   forward 93-106 us (5.1-5.8 TB/s), backward at
//   x + r 102-113 (5.9-6.6) and 5 for the sum of dw's parts, each after the other;
//   4096 x 4096 bf16 to e4m3   21-23 us (5.1-5.6 TB/s).
// Small ones are bound by latency: 1 x 4096 2.5 us, 2039 x 1025 fp16 8 and 11 (at x + r).
//
// Squares leave fp32's range for |h| around 2^64 (bf16) and lose bits below
// 2^-60: a row whose sum of squares says so is summed again, scaled by a power of
// two k; what is computed then is n = (k h) / sqrt(mean((k h)^2) + k^2 eps).
#include "norm.h"

#include <algorithm>

#include "layer_math.h"
#include "mx_math.h"

namespace pgemm {
namespace layer {
namespace {

// 8 columns of a row from any 2-byte boundary, zeros from `cols` on.  PAST: past the
// caches.
template <bool PAST = false>
__device__ __forceinline__ u4_t chunk_bits(const uint16_t* row, int col, int cols) {
    const int nv = min(8, cols - col);
    u4_t w = {};
    if (nv == 8) {
        typedef u4_t u4_any __attribute__((aligned(2)));
        if constexpr (PAST)
            w = __builtin_nontemporal_load(reinterpret_cast<const u4_any*>(row + col));
        else
            __builtin_memcpy(&w, row + col, 16);
    } else if (nv > 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            w[q >> 1] |= (uint32_t)(q < nv ? row[col + q] : 0) << (16 * (q & 1));
    }
    return w;
}
// past: past the caches.
template <class E>
__device__ __forceinline__ void put_chunk(uint16_t* row, int col, int cols, const float (&v)[8],
                                          bool past = false) {
    if (col >= cols) return;
    if (past)
        store8<E, true>(Rows{row, 0, 0}, 0, col, min(8, cols - col), v);
    else
        store8<E, false>(Rows{row, 0, 0}, 0, col, min(8, cols - col), v);
}

struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Most {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
        return max(a, b);
    }
};
// v combined over the T lanes of a row, the same in each of them.  slots: 2 T / 64
// words of LDS; `turn` says which half, and changes (so that one barrier a call
// is enough).
template <int T, class Op, class V>
__device__ __forceinline__ V over_row(V v, V* slots, int& turn, Op op) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = op(v, __shfl_xor(v, o, 64));
    if constexpr (T > 64) {
        constexpr int W = T / 64;
        V* const s = slots + turn * W;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
        __syncthreads();
        v = s[0];
#pragma unroll
        for (int i = 1; i < W; ++i) v = op(v, s[i]);
    }
    return v;
}
template <int T>
struct RowSums {
    uint32_t slots[T > 64 ? 2 * T / 64 : 1];
};
template <int T>
__device__ __forceinline__ float sum_over_row(float v, RowSums<T>& s, int& turn) {
    return over_row<T>(v, reinterpret_cast<float*>(s.slots), turn, Add{});
}

// Whether a row's sum of squares needs the scaled sum, and the scale for a row
// whose largest magnitude has the bits `most` (1 where no scale helps).
__device__ __forceinline__ bool needs_scale(float squares, float eps, int D) {
    return !(squares < INFINITY) || squares + eps * (float)D < 1e-25f;
}
__device__ __forceinline__ float scale_of(uint32_t most) {
    if (most >= 0x7F800000u) return 1.0f;
    const int e = min(128 - (int)(most >> 23), 75);  // k most is below 4
    return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ float inverse_root(float squares, float k, float eps, int D) {
    return __builtin_amdgcn_rsqf(squares * (1.0f / (float)D) + eps * k * k);
}

// T lanes a row, NC chunks of 8 columns a lane.  FORMAT below 0: y in 16 bits.  past: the
// larger result that is not read first, y in 16 bits or h beside a microscaled y, is stored
// past the caches (stores_past()).
template <class E, int T, int NC, int FORMAT>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(
    const uint16_t* x, int64_t ldx, const uint16_t* r, int64_t ldr, const uint16_t* __restrict__ w,
    uint16_t* h, int64_t ldh, uint16_t* y, int64_t ldy, const MxRows mx, int64_t M, int D,
    float eps, bool past) {
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ RowSums<T> sums;
    int turn = 0;
    const int t = threadIdx.x % T;
    u4_t wb[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (w) wb[i] = chunk_bits(w, (t + T * i) * 8, D);
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T; row < M;
         row += (int64_t)gridDim.x * RPB) {
        u4_t xb[NC], rb[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = (t + T * i) * 8;
            xb[i] = chunk_bits(x + row * ldx, col, D);
            if (r) rb[i] = chunk_bits(r + row * ldr, col, D);
        }
        float s[NC][8];
        float squares = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            unpack8<E>(xb[i], s[i]);
            if (r) {
                float v[8];
                unpack8<E>(rb[i], v);
#pragma unroll
                for (int q = 0; q < 8; ++q) s[i][q] += v[q];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) squares = fmaf(s[i][q], s[i][q], squares);
        }
        squares = sum_over_row<T>(squares, sums, turn);
        float k = 1.0f;
        if (needs_scale(squares, eps, D)) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) most = max(most, most8(s[i]));
            k = scale_of(over_row<T>(most, sums.slots, turn, Most{}));
            squares = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int q = 0; q < 8; ++q) squares += (s[i][q] * k) * (s[i][q] * k);
            squares = sum_over_row<T>(squares, sums, turn);
        }
        const float inv = inverse_root(squares, k, eps, D);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = (t + T * i) * 8;
            if (h) put_chunk<E>(h + row * ldh, col, D, s[i], past && FORMAT >= 0);
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = s[i][q] * k * inv;
            if (w) {
                float f[8];
                unpack8<E>(wb[i], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= f[q];
            }
            if constexpr (FORMAT < 0) {
                put_chunk<E>(y + row * ldy, col, D, v, past);
            } else {
                typedef Mx<FORMAT> F;
                // An infinite inv (0 / 0) leaves NaN in the padding too: none there.
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = col + q < D ? v[q] : 0.0f;
                const uint32_t code = F::scale_code(most_of_quad(most8(v)));
                uint32_t c[F::kWords];
                F::encode8(v, code, c);
                if (col < (D + kMxGroup - 1) / kMxGroup * kMxGroup) {
                    __builtin_memcpy(mx.codes + row * mx.ld + (col >> 3) * 4 * F::kWords, c,
                                     4 * F::kWords);
                    if (((col >> 3) & 3) == 0)
                        mx.scales[row * mx.lds + (col >> 5)] = (uint8_t)code;
                }
            }
        }
    }
}

// Rows longer than what registers hold: read again for each pass.
constexpr int kLongT = 1024;
// Most workgroups of a launch (of up to 1024 lanes: under 2^32 work-items); they
// walk the rows.
constexpr int64_t kMostBlocks = 1 << 20;
template <class E, int FORMAT>
__global__ __launch_bounds__(kLongT) void norm_long_kernel(
    const uint16_t* x, int64_t ldx, const uint16_t* r, int64_t ldr, const uint16_t* __restrict__ w,
    uint16_t* h, int64_t ldh, uint16_t* y, int64_t ldy, const MxRows mx, int64_t M, int D,
    float eps, bool past) {
    __shared__ RowSums<kLongT> sums;
    int turn = 0;
    const int padded = (D + kMxGroup - 1) / kMxGroup * kMxGroup;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        auto each = [&](auto&& f) __attribute__((always_inline)) {
            for (int col = threadIdx.x * 8; col < padded; col += kLongT * 8) {
                float s[8];
                unpack8<E>(chunk_bits(x + row * ldx, col, D), s);
                if (r) {
                    float v[8];
                    unpack8<E>(chunk_bits(r + row * ldr, col, D), v);
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[q] += v[q];
                }
                f(col, s);
            }
        };
        auto sum = [&](float k) __attribute__((always_inline)) {
            float squares = 0.0f;
            each([&](int, const float(&s)[8]) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < 8; ++q) squares += (s[q] * k) * (s[q] * k);
            });
            return sum_over_row<kLongT>(squares, sums, turn);
        };
        float squares = sum(1.0f), k = 1.0f;
        if (needs_scale(squares, eps, D)) {
            uint32_t most = 0;
            each([&](int, const float(&s)[8]) __attribute__((always_inline)) {
                most = max(most, most8(s));
            });
            k = scale_of(over_row<kLongT>(most, sums.slots, turn, Most{}));
            squares = sum(k);
        }
        const float inv = inverse_root(squares, k, eps, D);
        // Each chunk is read, then written, by one lane: h and y may be x or r.
        each([&](int col, const float(&s)[8]) __attribute__((always_inline)) {
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = s[q] * k * inv;
            if (w) {
                float f[8];
                unpack8<E>(chunk_bits(w, col, D), f);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= f[q];
            }
            if (h) put_chunk<E>(h + row * ldh, col, D, s, past && FORMAT >= 0);
            if constexpr (FORMAT < 0) {
                put_chunk<E>(y + row * ldy, col, D, v, past);
            } else {
                typedef Mx<FORMAT> F;
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = col + q < D ? v[q] : 0.0f;
                const uint32_t code = F::scale_code(most_of_quad(most8(v)));
                uint32_t c[F::kWords];
                F::encode8(v, code, c);
                __builtin_memcpy(mx.codes + row * mx.ld + (col >> 3) * 4 * F::kWords, c,
                                 4 * F::kWords);
                if (((col >> 3) & 3) == 0) mx.scales[row * mx.lds + (col >> 5)] = (uint8_t)code;
            }
        });
    }
}

// Backward: a workgroup takes rows blockIdx.x * RPB + .., gridDim.x * RPB apart,
// and leaves its part of dw in part[blockIdx.x][D].  SUM: h is h + r in fp32.
// READS_PAST: dy, h, r and dh too are read past the caches.  (The next row's loads issued
// ahead made 16384 x 4096 3% slower, and 2039 x 1025 15 us instead of 10.)
template <class E, int T, int NC, bool SUM, bool READS_PAST>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_grad_kernel(
    const uint16_t* dy, int64_t lddy, const uint16_t* __restrict__ h, int64_t ldh,
    const uint16_t* __restrict__ r, int64_t ldr, const uint16_t* __restrict__ w, const uint16_t* dh,
    int64_t lddh, uint16_t* dx, int64_t lddx, float* __restrict__ part, int64_t M, int D,
    float eps) {
    constexpr int RPB = T < 256 ? 256 / T : 1;
    __shared__ RowSums<T> sums;
    __shared__ float joined[RPB > 1 ? RPB : 1][RPB > 1 ? T * 8 : 1];
    int turn = 0;
    const int t = threadIdx.x % T;
    u4_t wb[NC];
    float dw[NC][8] = {};
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if (w) wb[i] = chunk_bits(w, (t + T * i) * 8, D);
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / T; row < M;
         row += (int64_t)gridDim.x * RPB) {
        u4_t yb[NC], hb[NC], rb[NC], ab[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int col = (t + T * i) * 8;
            yb[i] = chunk_bits<READS_PAST>(dy + row * lddy, col, D);
            hb[i] = chunk_bits<READS_PAST>(h + row * ldh, col, D);
            if constexpr (SUM) rb[i] = chunk_bits<READS_PAST>(r + row * ldr, col, D);
        }
        if (dh) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                ab[i] = chunk_bits<READS_PAST>(dh + row * lddh, (t + T * i) * 8, D);
        }
        auto normed = [&](int i, float(&n)[8]) __attribute__((always_inline)) {
            unpack8<E>(hb[i], n);
            if constexpr (SUM) {
                float v[8];
                unpack8<E>(rb[i], v);
#pragma unroll
                for (int q = 0; q < 8; ++q) n[q] += v[q];
            }
        };
        // g of a chunk (times 1 without a weight), and h times k.
        auto chunk = [&](int i, float k, float(&g)[8], float(&n)[8]) __attribute__((always_inline)) {
            unpack8<E>(yb[i], g);
            normed(i, n);
            if (w) {
                float f[8];
                unpack8<E>(wb[i], f);
#pragma unroll
                for (int q = 0; q < 8; ++q) g[q] *= f[q];
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) n[q] *= k;
        };
        float k = 1.0f, squares, along;
        auto sum = [&]() __attribute__((always_inline)) {
            squares = 0.0f, along = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float g[8], n[8];
                chunk(i, k, g, n);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    squares = fmaf(n[q], n[q], squares);
                    along = fmaf(g[q], n[q], along);
                }
            }
            squares = sum_over_row<T>(squares, sums, turn);
            along = sum_over_row<T>(along, sums, turn);
        };
        sum();
        if (needs_scale(squares, eps, D)) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float v[8];
                normed(i, v);
                most = max(most, most8(v));
            }
            k = scale_of(over_row<T>(most, sums.slots, turn, Most{}));
            sum();
        }
        const float inv = inverse_root(squares, k, eps, D);
        const float mean = along * inv * (1.0f / (float)D);
        const float factor = inv * k;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float g[8], n[8];
            chunk(i, k, g, n);
            float d[8];
            unpack8<E>(yb[i], d);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                n[q] *= inv;
                dw[i][q] = fmaf(d[q], n[q], dw[i][q]);
            }
            if (dx) {
                float a[8] = {};
                if (dh) unpack8<E>(ab[i], a);
#pragma unroll
                for (int q = 0; q < 8; ++q) a[q] += (g[q] - n[q] * mean) * factor;
                put_chunk<E>(dx + row * lddx, (t + T * i) * 8, D, a);
            }
        }
    }
    if (!part) return;
    float* const out = part + (int64_t)blockIdx.x * D;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if constexpr (RPB > 1) {
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 8; ++q) joined[threadIdx.x / T][t * 8 + q] = dw[i][q];
            __syncthreads();
            for (int c = threadIdx.x; c < T * 8; c += RPB * T) {
                float v = joined[0][c];
#pragma unroll
                for (int p = 1; p < RPB; ++p) v += joined[p][c];
                if (T * i * 8 + c < D) out[T * i * 8 + c] = v;
            }
        } else {
            const int col = (t + T * i) * 8;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (col + q < D) out[col + q] = dw[i][q];
        }
    }
}

// h of a chunk, with r (where not NULL) added.
template <class E>
__device__ __forceinline__ void sum_chunk(const uint16_t* h, const uint16_t* r, int col, int cols,
                                          float (&n)[8]) {
    unpack8<E>(chunk_bits(h, col, cols), n);
    if (r) {
        float v[8];
        unpack8<E>(chunk_bits(r, col, cols), v);
#pragma unroll
        for (int q = 0; q < 8; ++q) n[q] += v[q];
    }
}

// Rows longer than what registers hold: dx, and the factors k and inv of each row,
// from which the columns' sums are made.
template <class E>
__global__ __launch_bounds__(kLongT) void norm_grad_long_kernel(
    const uint16_t* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ h, int64_t ldh,
    const uint16_t* __restrict__ r, int64_t ldr, const uint16_t* __restrict__ w, const uint16_t* dh,
    int64_t lddh, uint16_t* dx, int64_t lddx, float* __restrict__ factors, int64_t M, int D,
    float eps) {
    __shared__ RowSums<kLongT> sums;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        auto each = [&](float k, auto&& f) __attribute__((always_inline)) {
            for (int col = threadIdx.x * 8; col < D; col += kLongT * 8) {
                float g[8], n[8];
                unpack8<E>(chunk_bits(dy + row * lddy, col, D), g);
                sum_chunk<E>(h + row * ldh, r ? r + row * ldr : nullptr, col, D, n);
                if (w) {
                    float v[8];
                    unpack8<E>(chunk_bits(w, col, D), v);
#pragma unroll
                    for (int q = 0; q < 8; ++q) g[q] *= v[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) n[q] *= k;
                f(col, g, n);
            }
        };
        float squares, along, k = 1.0f;
        auto sum = [&]() __attribute__((always_inline)) {
            squares = 0.0f, along = 0.0f;
            each(k, [&](int, const float(&g)[8], const float(&n)[8]) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    squares = fmaf(n[q], n[q], squares);
                    along = fmaf(g[q], n[q], along);
                }
            });
            squares = sum_over_row<kLongT>(squares, sums, turn);
            along = sum_over_row<kLongT>(along, sums, turn);
        };
        sum();
        if (needs_scale(squares, eps, D)) {
            uint32_t most = 0;
            each(1.0f, [&](int, const float(&)[8], const float(&n)[8]) __attribute__((always_inline)) {
                most = max(most, most8(n));
            });
            k = scale_of(over_row<kLongT>(most, sums.slots, turn, Most{}));
            sum();
        }
        const float inv = inverse_root(squares, k, eps, D);
        const float mean = along * inv * (1.0f / (float)D);
        if (threadIdx.x == 0 && factors) {
            factors[2 * row] = k;
            factors[2 * row + 1] = inv;
        }
        if (!dx) continue;
        each(k, [&](int col, const float(&g)[8], const float(&n)[8]) __attribute__((always_inline)) {
            float a[8] = {};
            if (dh) unpack8<E>(chunk_bits(dh + row * lddh, col, D), a);
#pragma unroll
            for (int q = 0; q < 8; ++q) a[q] += (g[q] - n[q] * inv * mean) * (inv * k);
            put_chunk<E>(dx + row * lddx, col, D, a);
        });
    }
}

// part[b][c] = sum over the block's rows of dy n, 2048 columns a workgroup.
constexpr int kLongRows = 64;
template <class E>
__global__ __launch_bounds__(256) void norm_columns_kernel(
    const uint16_t* __restrict__ dy, int64_t lddy, const uint16_t* __restrict__ h, int64_t ldh,
    const uint16_t* __restrict__ res, int64_t ldr, const float* __restrict__ factors,
    float* __restrict__ part, int64_t M, int D) {
    const int col = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (col >= D) return;
    float s[8] = {};
    const int64_t blocks = (M + kLongRows - 1) / kLongRows;
    for (int64_t b = blockIdx.y; b < blocks; b += gridDim.y) {
        const int64_t r1 = min(M, (b + 1) * kLongRows);
        for (int64_t r = b * kLongRows; r < r1; ++r) {
            float d[8], n[8];
            unpack8<E>(chunk_bits(dy + r * lddy, col, D), d);
            sum_chunk<E>(h + r * ldh, res ? res + r * ldr : nullptr, col, D, n);
            const float k = factors[2 * r], inv = factors[2 * r + 1];
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] = fmaf(d[q], n[q] * k * inv, s[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (col + q < D) part[(int64_t)blockIdx.y * D + col + q] = s[q];
}

template <int T_, int NC_>
struct Shape {
    static constexpr int T = T_, NC = NC_;
};
// run(Shape) for the lanes and chunks that hold `cols` columns; false where none
// does.  WIDE: up to 32768 columns, else 16384.  (The backward pass holds three times as
// much of a row and dw's part besides, which the 128 registers that 1024 lanes leave each
// other do not take: with 162-197 of them spilled 2016 x 16640 bf16 took 411 us, 1024 x
// 32768 281 and 8 x 32768 46; read again for each pass 136, 124 and 21.)
template <bool WIDE, class Run>
bool with_shape(int64_t cols, Run&& run) {
    const int64_t chunks = (cols + 7) / 8;
    if (chunks <= 64) run(Shape<64, 1>{});
    else if (chunks <= 128) run(Shape<64, 2>{});
    else if (chunks <= 256) run(Shape<64, 4>{});
    else if (chunks <= 512) run(Shape<256, 2>{});
    else if (chunks <= 1024) run(Shape<256, 4>{});
    else if (chunks <= 2048) run(Shape<512, 4>{});
    else if (!WIDE || chunks > 4096) return false;
    else if constexpr (WIDE) run(Shape<1024, 4>{});
    return true;
}

// What goes past the caches, chosen with the readers of the results in the measurement (a
// chain of norms, each with the projection that reads its y, the next norm taking h as its
// residual); us a norm and its readers, rows of 4096 bf16.
//
// y in 16 bits, from the size on at which the call's matrices together fill the memory-side
// cache and push each other out (kept / y past / h past too; 4096 outputs, 256 outputs):
//      4096 rows (128 MB)   122.5 / 122.9 / 123.9    47.7 /  48.3 /  48.9
//      8192 (256)           240.0 / 236.8 / 238.8    86.9 /  80.1 /  80.7
//     12288 (384)           349.2 / 352.2 / 352.6   124.0 / 116.9 / 116.3
//     16384 (512)           471.4 / 470.5 / 473.5   147.0 / 143.1 / 143.0
// and the backward pass reads past them from that size on (the norm's backward pass and the
// product on dx; kept / read past / dx past too): 4096 rows 112.1 / 110.7 / 113.2, 8192
// 210.1 / 202.4 / 207.1, 16384 413.1 / 388.6 / 409.7; 16384 x 1024 (128 MB) 54.8 / 55.1 /
// 56.0.  dx stays for its reader.  Norm, projection and both backward passes, 16384 rows: all
// kept 1301, y and the reads past 1265, h too 1269, dx too 1308; alone, without the
// products, dx past is the faster (176 instead of 184).
//
// h beside a microscaled y, where it is larger than the L2s together (32 MB): what is read
// first is y, and h would push it out.  Kept / past: 2048 rows (16 MB) 47.7 / 48.0, 3584
// (28 MB) 70.1 / 70.1, 4096 75.3 / 74.9, 8192 146.6 / 147.1, 12288 223.4 / 207.2, 16384 296.7 /
// 293.9; with two products of 16384 between h and its reader 4096 445.7 / 443.5, 6144 704.0 /
// 695.8, 12288 1332 / 1324.  Nothing reading it, 4096 rows to e4m3 and back: 32.4 / 31.2.
constexpr int64_t kL2 = 32 << 20;
inline bool stores_past(int format, int64_t bytes, int matrices) {
    return format < 0 ? bytes * matrices >= kMemorySide : bytes >= kL2;
}

template <class E, int FORMAT>
hipError_t forward_as(const NormCall& c, hipStream_t stream) {
    const uint16_t* x = static_cast<const uint16_t*>(c.x);
    const uint16_t* r = static_cast<const uint16_t*>(c.residual);
    const uint16_t* w = static_cast<const uint16_t*>(c.weight);
    uint16_t* h = static_cast<uint16_t*>(c.h);
    uint16_t* y = static_cast<uint16_t*>(c.y);
    const int D = (int)c.D;
    const bool past = stores_past(FORMAT, c.M * c.D * 2, 2 + (r ? 1 : 0) + (h ? 1 : 0));
    const bool held = with_shape<true>(FORMAT < 0 ? c.D : mx_padded(c.D), [&](auto s) {
        constexpr int T = decltype(s)::T, NC = decltype(s)::NC;
        constexpr int RPB = T < 256 ? 256 / T : 1;
        const unsigned blocks = (unsigned)std::min((c.M + RPB - 1) / RPB, kMostBlocks);
        hipLaunchKernelGGL((norm_kernel<E, T, NC, FORMAT>), dim3(blocks), dim3(RPB * T), 0, stream, x,
                           c.ldx, r, c.ldr, w, h, c.ldh, y, c.ldy, c.mx, c.M, D, c.eps, past);
    });
    if (!held)
        hipLaunchKernelGGL((norm_long_kernel<E, FORMAT>),
                           dim3((unsigned)std::min(c.M, kMostBlocks)), dim3(kLongT), 0, stream, x,
                           c.ldx, r, c.ldr, w, h, c.ldh, y, c.ldy, c.mx, c.M, D, c.eps, past);
    return hipGetLastError();
}

// Most parts of dw (256, 768, 1024 and 2048 were slower at 16384 x 4096).
constexpr int64_t kGradBlocks = 512;

template <class E>
hipError_t backward_as(const NormGradCall& c, Arena& ar, hipStream_t stream) {
    const uint16_t* dy = static_cast<const uint16_t*>(c.dy);
    const uint16_t* h = static_cast<const uint16_t*>(c.h);
    const uint16_t* r = static_cast<const uint16_t*>(c.residual);
    const uint16_t* w = static_cast<const uint16_t*>(c.weight);
    const uint16_t* dh = static_cast<const uint16_t*>(c.dh);
    uint16_t* dx = static_cast<uint16_t*>(c.dx);
    const int D = (int)c.D;
    const int dtype = std::is_same<E, BF16>::value ? kBF16 : kF16;
    const bool reads_past =
        c.M * c.D * 2 * (2 + (r ? 1 : 0) + (dh ? 1 : 0) + (dx ? 1 : 0)) >= kMemorySide;
    int64_t parts = 0;
    float* part = nullptr;
    const bool held = with_shape<false>(c.D, [&](auto s) {
        constexpr int T = decltype(s)::T, NC = decltype(s)::NC;
        constexpr int RPB = T < 256 ? 256 / T : 1;
        parts = std::min<int64_t>((c.M + RPB - 1) / RPB, kGradBlocks);
        if (c.dw) part = static_cast<float*>(ar.take(std::max<int64_t>(parts, 1) * c.D * 4));
        if (ar.dry() || parts == 0) return;
        auto go = [&](auto sum, auto reads_past) {
            hipLaunchKernelGGL(
                (norm_grad_kernel<E, T, NC, decltype(sum)::value, decltype(reads_past)::value>),
                dim3((unsigned)parts), dim3(RPB * T), 0, stream, dy, c.lddy, h, c.ldh, r, c.ldr, w,
                dh, c.lddh, dx, c.lddx, part, c.M, D, c.eps);
        };
        auto with_sum = [&](auto reads_past) {
            if (r) go(std::true_type{}, reads_past);
            else go(std::false_type{}, reads_past);
        };
        if (reads_past) with_sum(std::true_type{});
        else with_sum(std::false_type{});
    });
    if (!held) {
        parts = std::min<int64_t>((c.M + kLongRows - 1) / kLongRows, 64);
        float* factors = nullptr;
        if (c.dw) {
            part = static_cast<float*>(ar.take(std::max<int64_t>(parts, 1) * c.D * 4));
            factors = static_cast<float*>(ar.take(std::max<int64_t>(c.M, 1) * 8));
        }
        if (!ar.dry() && c.M > 0) {
            hipLaunchKernelGGL((norm_grad_long_kernel<E>),
                               dim3((unsigned)std::min(c.M, kMostBlocks)), dim3(kLongT), 0, stream, dy,
                               c.lddy, h, c.ldh, r, c.ldr, w, dh, c.lddh, dx, c.lddx, factors, c.M, D,
                               c.eps);
            if (c.dw)
                hipLaunchKernelGGL((norm_columns_kernel<E>),
                                   dim3((unsigned)((c.D + 2047) / 2048), (unsigned)parts), dim3(256),
                                   0, stream, dy, c.lddy, h, c.ldh, r, c.ldr, factors, part, c.M, D);
        }
    }
    if (ar.dry()) return hipSuccess;
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess || !c.dw) return rc;
    return launch_column_sum(dtype, part, c.M > 0 ? parts : 0, c.D, c.dw, stream);
}

}  // namespace

hipError_t norm_forward(const NormCall& c, hipStream_t stream) {
    const bool b = c.dtype == kBF16;
    if (c.format < 0) return b ? forward_as<BF16, -1>(c, stream) : forward_as<F16, -1>(c, stream);
    if (c.format == PMX_E2M1)
        return b ? forward_as<BF16, PMX_E2M1>(c, stream) : forward_as<F16, PMX_E2M1>(c, stream);
    return b ? forward_as<BF16, PMX_E4M3>(c, stream) : forward_as<F16, PMX_E4M3>(c, stream);
}

hipError_t norm_backward(const NormGradCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? backward_as<BF16>(c, ar, stream) : backward_as<F16>(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
