// Element types, activations and 8-wide row accesses of the layer operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pgemm.h"

namespace pgemm {
namespace {

// fp16 and bf16 as the kernels see them: 16-bit patterns in memory, fp32 in
// registers.  put() rounds once to nearest even (fp16: overflow to infinity,
// subnormals kept).
struct F16 {
    typedef _Float16 frag8 __attribute__((ext_vector_type(8)));
    typedef float f4 __attribute__((ext_vector_type(4)));
    __device__ static __forceinline__ f4 mma(frag8 row_op, frag8 col_op, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(row_op, col_op, c, 0, 0, 0);
    }
    __device__ static __forceinline__ uint32_t put2(float a, float b) {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        typedef float f2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), h2));
    }
    __device__ static __forceinline__ uint16_t put(float a) {
        return __builtin_bit_cast(uint16_t, (_Float16)a);
    }
    __device__ static __forceinline__ float get(uint16_t u) {
        return (float)__builtin_bit_cast(_Float16, u);
    }
};

struct BF16 {
    typedef _Float16 frag8 __attribute__((ext_vector_type(8)));  // container of 8 patterns
    typedef float f4 __attribute__((ext_vector_type(4)));
    __device__ static __forceinline__ f4 mma(frag8 row_op, frag8 col_op, f4 c) {
        typedef __bf16 b8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, row_op),
                                                       __builtin_bit_cast(b8, col_op), c, 0, 0, 0);
    }
    __device__ static __forceinline__ uint32_t put2(float a, float b) {
        typedef __bf16 h2 __attribute__((ext_vector_type(2)));
        typedef float f2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), h2));
    }
    __device__ static __forceinline__ uint16_t put(float a) {
        return __builtin_bit_cast(uint16_t, (__bf16)a);
    }
    __device__ static __forceinline__ float get(uint16_t u) {
        return __builtin_bit_cast(float, (uint32_t)u << 16);
    }
};

// How pffn keeps g and u for its backward pass, in 16 bits.  The gradients
// take products of them, so their rounding shows there: rounded to bf16 they
// double the error of dW_out (2.1 roundings of its size in all, against 1.4
// for h and the output alone).  fp16 keeps the values themselves.  bf16 keeps
// them with 6 exponent and 9 fraction bits (bias 31), a quarter of bf16's
// rounding (1.5 in all).
//
// What a form does not hold is marked, and the backward pass computes it again
// from x and W_in: in fp16 the infinities; in bf16 exponent field 0 (magnitudes
// below 2^-30, with gradual underflow; only 0 itself is code 0) and the
// topmost code (those that round to 2^33 - 2^23 and more, infinities, NaN).
// beyond(c) is 1 for a marked code, any_beyond(g, u) where one of 16 is (or, in
// fp16, is NaN); as_kept(c) is what it stands for where x or W_in is not at
// hand.  Both are computed as integers: 16 lane masks would not fit in scalar
// registers beside those of the copies.
typedef uint16_t us2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

template <class E>
struct Kept16 {
    __device__ static __forceinline__ uint32_t put2(float a, float b) { return E::put2(a, b); }
    __device__ static __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
        a = E::get((uint16_t)w);
        b = E::get((uint16_t)(w >> 16));
    }
    __device__ static __forceinline__ uint32_t beyond(uint32_t c) {
        return 1u - min((c & 0x7FFFu) ^ 0x7C00u, 1u);
    }
    __device__ static __forceinline__ uint32_t any_beyond(const u4_t& g, const u4_t& u) {
        us2_t top = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            top = __builtin_elementwise_max(top, __builtin_bit_cast(us2_t, g[q] & 0x7FFF7FFFu));
            top = __builtin_elementwise_max(top, __builtin_bit_cast(us2_t, u[q] & 0x7FFF7FFFu));
        }
        return ((uint32_t)max(top[0], top[1]) + 0x400u) >> 15;
    }
    __device__ static __forceinline__ float as_kept(uint32_t c) { return E::get((uint16_t)c); }
};
template <>
struct Kept16<BF16> {
    // The code is the top of an fp32 pattern 2^96 below the value: exact both
    // ways in the normal range.  Rounds to nearest, ties away from zero.
    __device__ static __forceinline__ uint32_t put(float f) {
        const uint32_t bits = __builtin_bit_cast(uint32_t, f * 0x1p-96f);
        const uint32_t least = f != 0.0f ? 1u << 14 : 0u;
        const uint32_t a = max((bits & 0x7FFFFFFFu) + 0x2000u, least);
        return (min(a, 0x7FFFu << 14) >> 14) | ((bits >> 16) & 0x8000u);
    }
    __device__ static __forceinline__ uint32_t put2(float a, float b) {
        return put(a) | (put(b) << 16);
    }
    // A code in the high half of w; the topmost one comes out as a number.
    __device__ static __forceinline__ float high(uint32_t w) {
        return __builtin_bit_cast(float, (uint32_t)((int32_t)w >> 2) & 0x9FFFC000u) * 0x1p96f;
    }
    __device__ static __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
        a = high(w << 16);
        b = high(w);
    }
    __device__ static __forceinline__ uint32_t beyond(uint32_t c) {
        c &= 0x7FFFu;
        return ((c + 1u) >> 15) | (((c - 0x200u) >> 31) & min(c, 1u));
    }
    __device__ static __forceinline__ uint32_t any_beyond(const u4_t& g, const u4_t& u) {
        const us2_t one = {1, 1};
        us2_t top = {}, low = {0xFFFF, 0xFFFF};  // low: of code - 1, so that 0 passes
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const us2_t c = __builtin_bit_cast(us2_t, (q < 4 ? g[q & 3] : u[q & 3]) & 0x7FFF7FFFu);
            top = __builtin_elementwise_max(top, c);
            low = __builtin_elementwise_min(low, (us2_t)(c - one));
        }
        return (((uint32_t)max(top[0], top[1]) + 1u) >> 15) |
               (((uint32_t)min(low[0], low[1]) - 0x1FFu) >> 31);
    }
    __device__ static __forceinline__ float as_kept(uint32_t c) {
        return (c & 0x7FFFu) == 0x7FFFu ? __builtin_nanf("") : high(c << 16);
    }
};

// ---- activations -----------------------------------------------------------
// exp2 and reciprocal are the hardware's (1 ulp), so an activation costs two
// quarter-rate instructions and a few ordinary ones per value.

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}

// Standard normal distribution and density at z.  The tail
// Phi(-|z|) = exp(-x^2) t P(t), x = |z| / sqrt 2, t = 1 / (1 + 0.375 x): the form
// of Abramowitz and Stegun 7.1.26, with a P of degree 6 fitted here for the
// relative error, since the activation's value for z < 0 is this tail (least
// squares on exp(x^2) erfc(x) / 2 for x <= 9.6, reweighted towards the largest
// relative error: 6.4e-7; in fp32 1.8e-6 at z = -4, 2e-5 at -13, where the
// argument of the exponential is rounded).  It serves the density too.
__device__ __forceinline__ void normal_cdf_pdf(float z, float& cdf, float& pdf) {
    const float x = fabsf(z) * 0.70710678f;
    const float t = __builtin_amdgcn_rcpf(fmaf(x, 0.375f, 1.0f));
    const float e = exp_fast(-x * x);
    float p = fmaf(t, -0.067547955f, 0.19396894f);
    p = fmaf(t, p, -0.064798675f);
    p = fmaf(t, p, 0.14153078f);
    p = fmaf(t, p, 0.08333228f);
    p = fmaf(t, p, 0.10784459f);
    p = fmaf(t, p, 0.10566972f);
    const float tail = t * p * e;
    cdf = z < 0.0f ? tail : 1.0f - tail;
    pdf = 0.3989422804f * e;
}

constexpr float kGeluA = 1.5957691216f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float relu_of(float z) {
    return z > 0.0f ? z : (z != z ? z : 0.0f);
}
__device__ __forceinline__ float gelu_of(float z) {
    float c, d;
    normal_cdf_pdf(z, c, d);
    return z * c;
}
// 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u)); the constants carry log2 e.
__device__ __forceinline__ float gelu_tanh_of(float z) {
    const float k = fmaf(z * z, -kGeluA * kGeluB * kLog2e, -kGeluA * kLog2e);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * k));
}
__device__ __forceinline__ float silu_of(float z) { return z * sigmoid(z); }

// The derivative, and with it the value (for the gated product, which needs
// both).  z is as a forward pass stored it, so in fp16 it is infinite where
// the sum was beyond 65504: the smooth activations' limits there are the
// values 0 and z, the derivatives 0 and 1.  They come from a distribution
// function that is exactly 0 or 1, which takes z itself (so NaN stays NaN),
// and from factors of z that are held to finite values.
__device__ __forceinline__ float not_minus_inf(float z) { return fmaxf(z, -1e30f); }

__device__ __forceinline__ float relu_grad(float z, float& value) {
    value = relu_of(z);
    return z > 0.0f ? 1.0f : 0.0f;
}
__device__ __forceinline__ float gelu_grad(float z, float& value) {
    float c, d;
    normal_cdf_pdf(z, c, d);
    value = not_minus_inf(z) * c;
    return d > 0.0f ? fmaf(z, d, c) : c;
}
// Far out the polynomial of the derivative is evaluated at +-30, where it is
// multiplied by 0.
__device__ __forceinline__ float gelu_tanh_grad(float z, float& value) {
    const float h = fminf(fmaxf(z, -30.0f), 30.0f);
    const float s = sigmoid(kGeluA * (z + kGeluB * z * z * z));
    value = not_minus_inf(z) * s;
    return s + h * s * (1.0f - s) * kGeluA * (1.0f + 3.0f * kGeluB * h * h);
}
__device__ __forceinline__ float silu_grad(float z, float& value) {
    const float s = sigmoid(z);
    const float h = not_minus_inf(z);
    value = h * s;
    return s * fmaf(fminf(h, 1e30f), 1.0f - s, 1.0f);
}

// An activation as a compile-time choice.
template <int ACT>
struct Act {
    __device__ static __forceinline__ float value(float z) {
        if constexpr (ACT == PGEMM_ACT_RELU) return relu_of(z);
        if constexpr (ACT == PGEMM_ACT_GELU) return gelu_of(z);
        if constexpr (ACT == PGEMM_ACT_GELU_TANH) return gelu_tanh_of(z);
        if constexpr (ACT == PGEMM_ACT_SILU) return silu_of(z);
        return z;
    }
    __device__ static __forceinline__ float grad(float z, float& value) {
        if constexpr (ACT == PGEMM_ACT_RELU) return relu_grad(z, value);
        if constexpr (ACT == PGEMM_ACT_GELU) return gelu_grad(z, value);
        if constexpr (ACT == PGEMM_ACT_GELU_TANH) return gelu_tanh_grad(z, value);
        if constexpr (ACT == PGEMM_ACT_SILU) return silu_grad(z, value);
        value = z;
        return 1.0f;
    }
};

// run(Act<act>{}): one uniform branch.
template <class Run>
__device__ __forceinline__ void with_act(int act, Run&& run) {
    switch (act) {
        case PGEMM_ACT_RELU: run(Act<PGEMM_ACT_RELU>{}); break;
        case PGEMM_ACT_GELU: run(Act<PGEMM_ACT_GELU>{}); break;
        case PGEMM_ACT_GELU_TANH: run(Act<PGEMM_ACT_GELU_TANH>{}); break;
        case PGEMM_ACT_SILU: run(Act<PGEMM_ACT_SILU>{}); break;
        default: run(Act<PGEMM_ACT_NONE>{}); break;
    }
}

// ---- rows of 16-bit values ---------------------------------------------------
// A row-major matrix of 16-bit values: 8 consecutive values of a row at a
// time, as one 16-byte access from any 2-byte boundary (the compiler's
// unaligned global access; an aligned one where `vec` says that the pointer
// is 16-byte aligned and ld a multiple of 8), one by one at the right edge
// (nv < 8).
struct Rows {
    uint16_t* ptr;
    int ld;        // below 2^22
    int aligned;  // whole chunks are 16-byte aligned
    // Element (row, col): row < 256 and ld < 2^24, a full-rate 24-bit product.
    __device__ __forceinline__ uint32_t at(int row, int col) const {
        return __umul24((uint32_t)row, (uint32_t)ld) + (uint32_t)col;
    }
    __host__ __device__ explicit operator bool() const { return ptr != nullptr; }
    // The same matrix from row r on.  Kernels address the rows of a tile (at
    // most 256) from its first one: a uniform 64-bit base and a 32-bit offset.
    __device__ __forceinline__ Rows from(int64_t r) const {
        return {ptr ? ptr + r * ld : ptr, ld, aligned};
    }
};

inline Rows make_rows(const void* p, int64_t ld) {
    return {static_cast<uint16_t*>(const_cast<void*>(p)), (int)ld,
            (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0};
}

template <class E>
__device__ __forceinline__ void unpack8(const u4_t& w, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = E::get((uint16_t)w[q]);
        v[2 * q + 1] = E::get((uint16_t)(w[q] >> 16));
    }
}

template <class E>
__device__ __forceinline__ void unpack8_kept(const u4_t& w, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) Kept16<E>::unpack2(w[q], v[2 * q], v[2 * q + 1]);
}

// The bits of 8 values, zeros from nv >= 1 on; row < 256.  At the edge the
// loads past nv take the first value's address, so that all are issued at once
// instead of one behind the other's branch.
__device__ __forceinline__ u4_t load8_bits(const Rows& m, int row, int col, int nv) {
    const uint16_t* p = m.ptr + m.at(row, col);
    u4_t w = {};
    if (nv == 8) {
        __builtin_memcpy(&w, p, 16);
    } else {
        uint32_t e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = p[q < nv ? q : 0];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            w[q >> 1] |= (q < nv ? e[q] : 0u) << (16 * (q & 1));
    }
    return w;
}

template <class E>
__device__ __forceinline__ void load8(const Rows& m, int row, int col, int nv, float (&v)[8]) {
    unpack8<E>(load8_bits(m, row, col, nv), v);
}

// F: how a pair of values is put (an element type, or Kept16 of one).  STREAM:
// past the caches, which keeps them for the operands that other workgroups
// still fetch (4096^3 with its epilogue 118 -> 114 us, the vocabulary
// gradients 1.6% faster); not for what the block's next products or its
// backward pass read again (1% of its step), and not for chunks that straddle
// lines, whose halves the caches join (a step of 2039 x 1025 x 2047: 86 us, past
// the caches 94).
template <class F, bool STREAM>
__device__ __forceinline__ void store8(const Rows& m, int row, int col, int nv,
                                       const float (&v)[8]) {
    typedef u4_t u4_any __attribute__((aligned(2)));
    uint16_t* p = m.ptr + m.at(row, col);
    const u4_t w = {F::put2(v[0], v[1]), F::put2(v[2], v[3]), F::put2(v[4], v[5]),
                    F::put2(v[6], v[7])};
    if (nv == 8) {
        if constexpr (STREAM)
            __builtin_nontemporal_store(w, reinterpret_cast<u4_any*>(p));
        else
            *reinterpret_cast<u4_any*>(p) = w;
    } else {
#pragma unroll
        for (int q = 0; q < 7; ++q)
            if (q < nv) p[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
    }
}

}  // namespace
}  // namespace pgemm
