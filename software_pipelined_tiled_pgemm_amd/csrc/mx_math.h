// Microscaled numbers (OCP MX): 4-bit (e2m1) or 8-bit (e4m3) elements in blocks
// of 32 along a row, each block with a scale 2^(code - 127) in 8 bits (e8m0,
// code 255: NaN).
//
// Rows are padded to whole groups of 128 columns (what one matrix instruction
// contracts): elements 0, scale code 0.  A row of elements takes 64 (e2m1, two
// a byte, the first one in the low half) or 128 (e4m3) bytes a group, a row of
// scales 4 bytes a group.
//
// The scale of a block is the smallest one that leaves no element beyond the
// element type's largest (6 or 448): with amax = m 2^k, 1 <= m < 2, and the
// largest element M 2^E, that is 2^(k - E), or 2^(k - E + 1) where m > M.  (Taking
// 2^(k - E) always would cut values of up to a quarter (e2m1) or an eighth
// (e4m3) off the block's largest.)  Codes below 0 become 0: values under about
// 2^-127 lose bits as subnormals do.  A block with an infinity or a NaN has no
// scale that holds it: it gets code 255 and elements 0, and stands for NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pgemm.h"

namespace pgemm {
namespace {

constexpr int kMxGroup = 128;  // columns that rows are padded to
constexpr int kMxBlock = 32;   // columns of a scale

inline int64_t mx_padded(int64_t cols) { return (cols + kMxGroup - 1) / kMxGroup * kMxGroup; }
// Bytes that the elements and the scales of a row take at least.
inline int64_t mx_row_bytes(int format, int64_t cols) {
    return format == PMX_E2M1 ? mx_padded(cols) / 2 : mx_padded(cols);
}
inline int64_t mx_scale_bytes(int64_t cols) { return mx_padded(cols) / kMxBlock; }

__device__ __forceinline__ uint32_t magnitude(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}
// The larger of the magnitudes' bits of 8 values: infinities and NaN count as
// the largest.
__device__ __forceinline__ uint32_t most8(const float (&v)[8]) {
    uint32_t m = magnitude(v[0]);
#pragma unroll
    for (int q = 1; q < 8; ++q) m = max(m, magnitude(v[q]));
    return m;
}
// The largest of 4 neighbouring lanes (those of a block).
__device__ __forceinline__ uint32_t most_of_quad(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
}

__device__ __forceinline__ float mx_scale(uint32_t code) {
    if (code == 255) return __builtin_nanf("");
    return __builtin_bit_cast(float, code == 0 ? 0x00400000u : code << 23);
}

template <int FORMAT>
struct Mx {
    static constexpr bool kFour = FORMAT == PMX_E2M1;
    static constexpr int kWords = kFour ? 1 : 2;  // 32-bit words of 8 elements

    // The scale code of a block whose largest magnitude has the bits `most`.
    __device__ static __forceinline__ uint32_t scale_code(uint32_t most) {
        if (most >= 0x7F800000u) return 255;
        constexpr int E = kFour ? 2 : 8;
        constexpr uint32_t over = kFour ? 0x400000u : 0x600000u;  // fraction of 1.5, 1.75
        const int c = (int)(most >> 23) - E + ((most & 0x7FFFFFu) > over ? 1 : 0);
        return (uint32_t)max(c, 0);
    }
    // 8 values over the scale, rounded to nearest even.  (The reciprocal of the
    // scale is a power of two, at most 2^127, so the products are exact but
    // where they end below 2^-126, far under the smallest element.)
    __device__ static __forceinline__ void encode8(const float (&v)[8], uint32_t code,
                                                   uint32_t (&w)[kWords]) {
        if (code == 255) {
#pragma unroll
            for (int q = 0; q < kWords; ++q) w[q] = 0;
            return;
        }
        const float inv = __builtin_bit_cast(float, (254u - code) << 23);
        if constexpr (kFour) {
            uint32_t r = 0;
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
            r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
            w[0] = r;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int r = 0;
                r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, r, false);
                r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, r, true);
                w[h] = (uint32_t)r;
            }
        }
    }
    __device__ static __forceinline__ void decode8(const uint32_t (&w)[kWords], float scale,
                                                   float (&v)[8]) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        f2 p[4];
        if constexpr (kFour) {
            p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 0);
            p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 1);
            p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 2);
            p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[0], 1.0f, 3);
        } else {
            p[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], false);
            p[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[0], true);
            p[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], false);
            p[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[1], true);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = p[q >> 1][q & 1] * scale;
    }
};

}  // namespace
}  // namespace pgemm
