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

// ---- activations -----------------------------------------------------------
// exp2 and reciprocal are the hardware's (1 ulp), so an activation costs two
// quarter-rate instructions and a few ordinary ones per value.

__device__ __forceinline__ float exp_fast(float x) {
    return __builtin_amdgcn_exp2f(x * 1.4426950408889634f);
}

__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}

// Standard normal distribution and density at z.  The tail
// Phi(-|z|) = erfc(|z| / sqrt 2) / 2 is Abramowitz and Stegun 7.1.26 (absolute
// error of erfc at most 1.5e-7, and its error shrinks with the factor
// exp(-z^2 / 2)); the exponential serves the density too.
__device__ __forceinline__ void normal_cdf_pdf(float z, float& cdf, float& pdf) {
    const float x = fabsf(z) * 0.70710678f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * x);
    const float e = exp_fast(-x * x);
    const float poly =
        t * (0.254829592f +
             t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    const float tail = 0.5f * poly * e;
    cdf = z < 0.0f ? tail : 1.0f - tail;
    pdf = 0.3989422804f * e;
}

constexpr float kGeluA = 1.5957691216f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case PGEMM_ACT_RELU:
            return z > 0.0f ? z : (z != z ? z : 0.0f);
        case PGEMM_ACT_GELU: {
            float c, d;
            normal_cdf_pdf(z, c, d);
            return z * c;
        }
        case PGEMM_ACT_GELU_TANH:  // 0.5 (1 + tanh u) = sigmoid(2 u)
            return z * sigmoid(kGeluA * (z + kGeluB * z * z * z));
        case PGEMM_ACT_SILU:
            return z * sigmoid(z);
        default:
            return z;
    }
}

// The derivative, and with it the value (for the gated product, which needs
// both).  Far out the derivative of the tanh form is 0 or 1 to the last bit;
// its polynomial is evaluated at z held to +-30, so that it stays finite.
__device__ __forceinline__ float act_grad(int act, float z, float& value) {
    switch (act) {
        case PGEMM_ACT_RELU:
            value = z > 0.0f ? z : (z != z ? z : 0.0f);
            return z > 0.0f ? 1.0f : 0.0f;
        case PGEMM_ACT_GELU: {
            float c, d;
            normal_cdf_pdf(z, c, d);
            value = z * c;
            return d > 0.0f ? c + z * d : c;
        }
        case PGEMM_ACT_GELU_TANH: {
            const float h = fminf(fmaxf(z, -30.0f), 30.0f);
            const float s = sigmoid(kGeluA * (h + kGeluB * h * h * h));
            value = z * s;
            return s + h * s * (1.0f - s) * kGeluA * (1.0f + 3.0f * kGeluB * h * h);
        }
        case PGEMM_ACT_SILU: {
            const float s = sigmoid(z);
            value = z * s;
            return s * (1.0f + z * (1.0f - s));
        }
        default:
            value = z;
            return 1.0f;
    }
}

// ---- rows of 16-bit values ---------------------------------------------------
// A row-major matrix of 16-bit values: 8 consecutive values of a row at a
// time.  vec: the pointer is 16-byte aligned and ld a multiple of 8, so whole
// chunks are single 16-byte accesses; otherwise, and at the right edge
// (nv < 8), values move one by one.
struct Rows {
    uint16_t* ptr;
    int64_t ld;
    int vec;
    __host__ __device__ explicit operator bool() const { return ptr != nullptr; }
};

inline Rows make_rows(const void* p, int64_t ld) {
    const bool vec = p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
    return {static_cast<uint16_t*>(const_cast<void*>(p)), ld, vec};
}

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));

template <class E>
__device__ __forceinline__ void load8(const Rows& m, int64_t row, int64_t col, int nv, float (&v)[8]) {
    const uint16_t* p = m.ptr + row * m.ld + col;
    if (m.vec && nv == 8) {
        const u4_t w = *reinterpret_cast<const u4_t*>(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = E::get((uint16_t)w[q]);
            v[2 * q + 1] = E::get((uint16_t)(w[q] >> 16));
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = q < nv ? E::get(p[q]) : 0.0f;
    }
}

template <class E>
__device__ __forceinline__ void store8(const Rows& m, int64_t row, int64_t col, int nv,
                                       const float (&v)[8]) {
    uint16_t* p = m.ptr + row * m.ld + col;
    if (m.vec && nv == 8) {
        const u4_t w = {E::put2(v[0], v[1]), E::put2(v[2], v[3]), E::put2(v[4], v[5]),
                        E::put2(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<u4_t*>(p));
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (q < nv) p[q] = E::put(v[q]);
    }
}

// A vector (bias) over columns: the same chunk of every row.
template <class E>
__device__ __forceinline__ void load8_vec(const uint16_t* b, int vec, int64_t col, int nv,
                                          float (&v)[8]) {
    const Rows r = {const_cast<uint16_t*>(b), 0, vec};
    load8<E>(r, 0, col, nv, v);
}

}  // namespace
}  // namespace pgemm
