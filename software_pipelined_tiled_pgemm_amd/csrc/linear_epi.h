// The epilogue of the linear layer's product, which the microscaled product has
// too.
#pragma once

#include "layer_pipe.h"

namespace pgemm {
namespace layer {
namespace {

// y = act(v + bias) + residual; z = v + bias is stored too where asked for.  At
// 4096^3 fp16 (bias, tanh GELU, residual) it adds 4-9 us to the product's 105:
// 12 instructions a value and two streams, in all CUs at the same time.
template <class E>
struct LinearEpi {
    static constexpr lp::EpiKind kind = lp::kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 4;
    Rows y, res, pre;
    const uint16_t* bias;
    int act;
    __device__ __forceinline__ LinearEpi from(int64_t r) const {
        return {y.from(r), res.from(r), pre.from(r), bias, act};
    }
    struct Column {
        float bias[8];
    };
    __device__ __forceinline__ Column column(int col, int nv) const {
        Column c = {};
        if (bias) load8<E>(Rows{const_cast<uint16_t*>(bias), 0, 0}, 0, col, nv, c.bias);
        return c;
    }
    __device__ __forceinline__ u4_t load(int row, int col, int nv) const {
        return res ? load8_bits(res, row, col, nv) : u4_t{};
    }
    __device__ __forceinline__ bool aligned() const { return y.aligned && (!pre || pre.aligned); }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        with_act(act, [&](auto a) __attribute__((always_inline)) {
            run([&](int row, int col, int nv, float(&v)[8], const Column& c, u4_t r)
                    __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += c.bias[q];
                if (pre) store8<E, STREAM>(pre, row, col, nv, v);
                float t[8];
                unpack8<E>(r, t);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = decltype(a)::value(v[q]);
                if (res) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] += t[q];
                }
                store8<E, STREAM>(y, row, col, nv, v);
            });
        });
    }
};

}  // namespace
}  // namespace layer
}  // namespace pgemm
