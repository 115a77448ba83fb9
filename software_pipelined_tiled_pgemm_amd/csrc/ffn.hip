// The gated feed-forward block and its backward pass.
//
//   forward    [g | u] = x W_in,  h = act(g) * u,  y = h W_out + r
//              x [M,D], W_in [D,2F] (gate columns, then up columns), W_out [F,N]
//   backward   dh = dy W_out^T
//              dg = dh * u * act'(g),  du = dh * act(g)
//              dx = [dg | du] W_in^T (+ a),  dW_in = x^T [dg | du],  dW_out = h^T dy
//
// Both projections, the activation and the product are one kernel (the sums of
// a split contraction are joined, and the rest done, by the finish kernel): a
// tile's columns are 32 gate columns and the same 32 up columns per wave, so g
// and u of a value meet in the epilogue, and only h is written (and g, u for a
// backward pass).  The backward pass computes dg, du and h (again, from g
// and u) in the epilogue of dh, which is never written.  Since [dg | du] and
// W_in lie side by side, dx and dW_in are one product each.
//
// Roundings beyond one per output: h and [dg | du], once each, as operands of
// the next product; g and u as kept for the backward pass (Kept16).
#include "ffn.h"

#include "layer_pipe.h"
#include "linear.h"

namespace pgemm {
namespace layer {
namespace {

// h, and g and u where they are kept.  4096 x 4096 -> 2 x 8192 fp16: 391-470 us
// for the launch (1170-1400 TFLOP/s, as the power limit allows).
template <class E>
struct GluEpi {
    static constexpr lp::EpiKind kind = lp::kPaired;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 1;
    Rows h;  // padded rows: whole chunks
    Rows gate, up;
    int act;
    __device__ __forceinline__ GluEpi from(int64_t r) const {
        return {h.from(r), gate.from(r), up.from(r), act};
    }
    __device__ __forceinline__ lp::Nothing column(int, int) const { return {}; }
    __device__ __forceinline__ lp::Nothing load(int, int, int) const { return {}; }
    __device__ __forceinline__ bool aligned() const {
        return !gate || (gate.aligned && up.aligned);
    }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        with_act(act, [&](auto a) __attribute__((always_inline)) {
            run([&](int row, int col, int nv, float(&g)[8], float(&u)[8], lp::Nothing, lp::Nothing)
                    __attribute__((always_inline)) {
                if (gate) {
                    store8<Kept16<E>, false>(gate, row, col, nv, g);
                    store8<Kept16<E>, false>(up, row, col, nv, u);
                }
                // 0 past F, where an infinite row of x has NaN
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] = q < nv ? u[q] * decltype(a)::value(g[q]) : 0.0f;
                store8<E, STREAM>(h, row, col, 8, u);
            });
        });
    }
};

// g and u summed again in fp32, for the kept codes that do not hold them: one
// dot product of a row of x and a column of W_in per value, by one lane.  At
// ordinary scales a block has no such values; NaN takes the same way, and ends
// its sum at once.
template <class E>
struct Source {
    const uint16_t* x;  // NULL where x or W_in is not at hand
    int64_t ldx;
    const uint16_t* w;
    int64_t ldw;
    int D, F;
    __device__ __forceinline__ Source from(int64_t r) const {
        return {x ? x + r * ldx : x, ldx, w, ldw, D, F};
    }
    __device__ __forceinline__ void again(int row, int col, const u4_t& gc, const u4_t& uc,
                                          float (&g)[8], float (&u)[8]) const {
        uint32_t todo = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t cg = gc[q >> 1] >> (16 * (q & 1)), cu = uc[q >> 1] >> (16 * (q & 1));
            todo |= Kept16<E>::beyond(cg) << q | Kept16<E>::beyond(cu) << (8 + q);
            if (!x) {
                g[q] = Kept16<E>::as_kept(cg);
                u[q] = Kept16<E>::as_kept(cu);
            }
        }
        if (!x) return;
        while (todo) {
            const int q = __builtin_ctz(todo);
            todo &= todo - 1;
            const uint16_t* px = x + row * ldx;
            const uint16_t* pw = w + col + (q & 7) + (q >= 8 ? F : 0);
            float sum = 0.0f;
            for (int d = 0; d < D && sum == sum; d += 32) {  // a NaN stays one
                const int end = min(D, d + 32);
#pragma unroll 4
                for (int e = d; e < end; ++e, pw += ldw) sum = fmaf(E::get(px[e]), E::get(*pw), sum);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = q == k ? sum : g[k];
                u[k] = q == k + 8 ? sum : u[k];
            }
        }
    }
};

// dg, du and h from dh and the kept g and u.  Bound by the epilogue itself:
// 45 instructions a value (4 each to decode g and u, 4 to look for marked codes,
// 20 for the activation's derivative) and five streams of memory; 4093 x 8192
// at K = 2048 212-224 us, of which the product takes 95.  128x128 tiles, whose
// two workgroups per CU overlap better, took 40 us more.
template <class E>
struct GluGradEpi {
    static constexpr lp::EpiKind kind = lp::kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = true;
    static constexpr int kAhead = 2;
    Rows gate, up;       // as the forward pass kept them
    Rows h, dgate, dup;  // padded rows: whole chunks, zeros past F
    int act;
    Source<E> source;
    __device__ __forceinline__ GluGradEpi from(int64_t r) const {
        return {gate.from(r), up.from(r), h.from(r), dgate.from(r), dup.from(r), act,
                source.from(r)};
    }
    struct Kept {
        u4_t g, u;
    };
    __device__ __forceinline__ lp::Nothing column(int, int) const { return {}; }
    __device__ __forceinline__ Kept load(int row, int col, int nv) const {
        return {load8_bits(gate, row, col, nv), load8_bits(up, row, col, nv)};
    }
    __device__ __forceinline__ bool aligned() const { return true; }
    // STREAM (whole tiles): a chunk with a code that does not hold its value
    // only says so, and its tile is done again in the other form.
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        with_act(act, [&](auto a) __attribute__((always_inline)) {
            run([&](int row, int col, int nv, float(&d)[8], lp::Nothing, const Kept& k)
                    __attribute__((always_inline)) {
                const uint32_t odd = Kept16<E>::any_beyond(k.g, k.u);
                float g[8], u[8], s[8];
                unpack8_kept<E>(k.g, g);
                unpack8_kept<E>(k.u, u);
                if constexpr (!STREAM)
                    if (odd) source.again(row, col, k.g, k.u, g, u);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float v;
                    s[q] = decltype(a)::grad(g[q], v) * d[q] * u[q];  // dg
                    u[q] *= v;                                        // h
                    d[q] *= v;                                        // du
                    if (q >= nv) s[q] = d[q] = 0.0f;  // where an infinite row of dy has NaN
                }
                store8<E, false>(h, row, col, 8, u);
                store8<E, false>(dgate, row, col, 8, s);
                store8<E, false>(dup, row, col, 8, d);
                return odd;
            });
        });
    }
};

// W_in as a product's operand: both halves in rows of whole chunks, the up
// half `shift` columns after the gate half.
hipError_t halves(const void* w, int64_t ld, int64_t rows, int64_t F, Arena& ar, hipStream_t stream,
                  View& out) {
    const uint16_t* p = static_cast<const uint16_t*>(w);
    if (direct(w, ld, F)) {
        out = {p, (int)ld};
        return hipSuccess;
    }
    const int64_t f8 = round_up(F, 8);
    uint16_t* dst = static_cast<uint16_t*>(ar.take(rows * 2 * f8 * 2));
    out = {dst, (int)(2 * f8)};
    if (ar.dry()) return hipSuccess;
    const hipError_t rc = launch_pack(p, ld, dst, 2 * f8, rows, F, stream);
    if (rc != hipSuccess) return rc;
    return launch_pack(p + F, ld, dst + f8, 2 * f8, rows, F, stream);
}

template <class E>
struct Ffn {
    static constexpr int dtype = std::is_same<E, BF16>::value ? kBF16 : kF16;

    static hipError_t forward(const FfnCall& c, Arena& ar, hipStream_t stream) {
        const int cus = compute_units();
        const int64_t f8 = round_up(c.F, 8);
        hipError_t rc;
        uint16_t* h = static_cast<uint16_t*>(ar.take(c.M * f8 * 2));
        const Sink s = {c.y, c.ldy, c.residual, c.ldr, nullptr, 0, nullptr, 0, 0};
        uint16_t* gu = static_cast<uint16_t*>(c.gate_up);
        const GluEpi<E> epi = {{h, (int)f8, 1},
                               make_rows(gu, c.ldgu),
                               make_rows(gu ? gu + c.F : nullptr, c.ldgu),
                               c.act};
        if (c.F > 0) {
            View x, w;
            if ((rc = operand(c.x, c.ldx, c.M, c.D, ar, stream, x)) != hipSuccess) return rc;
            if ((rc = halves(c.w_in, c.ldwi, c.D, c.F, ar, stream, w)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.M, 2 * f8, c.D, cus, 16);
            Args g = args(x, w, c.M, 2 * f8, c.D, cut, ar);
            g.N = (int)c.F;
            g.pair_shift = (int)f8;
            if (!ar.dry()) {
                rc = lp::launch_product<E, true, false>(g, cut, epi, stream);
                if (rc != hipSuccess) return rc;
            }
        }
        if (c.N == 0) return hipSuccess;  // only gate_up was asked for
        View wo;
        if ((rc = operand(c.w_out, c.ldwo, c.F, c.N, ar, stream, wo)) != hipSuccess) return rc;
        const Cut cut = choose_cut(c.M, c.N, c.F, cus, 16);
        const Args g = args({h, (int)f8}, wo, c.M, c.N, c.F, cut, ar);
        if (ar.dry()) return hipSuccess;
        return launch_linear(dtype, kNN, g, cut, s, stream);
    }

    static hipError_t backward(const FfnGradCall& c, Arena& ar, hipStream_t stream) {
        const int cus = compute_units();
        const int64_t f8 = round_up(c.F, 8);
        hipError_t rc;
        View dy = {}, wo = {};
        if ((rc = operand(c.dy, c.lddy, c.M, c.N, ar, stream, dy)) != hipSuccess) return rc;
        uint16_t* h = static_cast<uint16_t*>(ar.take(c.M * f8 * 2));
        uint16_t* d = static_cast<uint16_t*>(ar.take(c.M * 2 * f8 * 2));
        if (c.M > 0 && c.F > 0) {
            if ((rc = operand(c.w_out, c.ldwo, c.F, c.N, ar, stream, wo)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.M, c.F, c.N, cus, 16);
            const Args g = args(dy, wo, c.M, c.F, c.N, cut, ar);
            if (!ar.dry()) {
                const uint16_t* gu = static_cast<const uint16_t*>(c.gate_up);
                const bool source = c.x && c.w_in;
                const GluGradEpi<E> epi = {
                    make_rows(gu, c.ldgu), make_rows(gu + c.F, c.ldgu), {h, (int)f8, 1},
                    {d, (int)(2 * f8), 1}, {d + f8, (int)(2 * f8), 1}, c.act,
                    {source ? static_cast<const uint16_t*>(c.x) : nullptr, c.ldx,
                     static_cast<const uint16_t*>(c.w_in), c.ldwi, (int)c.D, (int)c.F}};
                rc = lp::launch_product<E, true, true>(g, cut, epi, stream);
                if (rc != hipSuccess) return rc;
            }
        }
        const View dv = {d, (int)(2 * f8)};
        if (c.dw_out && c.F > 0 && c.N > 0) {
            const Cut cut = choose_cut(c.F, c.N, c.M, cus, 16);
            const Args g = args({h, (int)f8}, dy, c.F, c.N, c.M, cut, ar);
            if (!ar.dry()) {
                const Sink s = {c.dw_out, c.lddwo, nullptr, 0, nullptr, 0, nullptr, 0, 0};
                if ((rc = launch_linear(dtype, kTN, g, cut, s, stream)) != hipSuccess) return rc;
            }
        }
        if (c.dx && c.M > 0 && c.D > 0) {
            View wi;
            if ((rc = halves(c.w_in, c.ldwi, c.D, c.F, ar, stream, wi)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.M, c.D, 2 * f8, cus, 16);
            const Args g = args(dv, wi, c.M, c.D, 2 * f8, cut, ar);
            if (!ar.dry()) {
                const Sink s = {c.dx, c.lddx, c.add, c.ldadd, nullptr, 0, nullptr, 0, 0};
                if ((rc = launch_linear(dtype, kNT, g, cut, s, stream)) != hipSuccess) return rc;
            }
        }
        if (c.dw_in && c.D > 0 && c.F > 0) {
            View x;
            if ((rc = operand(c.x, c.ldx, c.M, c.D, ar, stream, x)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.D, 2 * f8, c.M, cus, 16);
            const Args g = args(x, dv, c.D, 2 * f8, c.M, cut, ar);
            if (!ar.dry()) {
                const Sink s = {c.dw_in, c.lddwi, nullptr, 0, nullptr, 0, nullptr, 0, (int)c.F};
                if ((rc = launch_linear(dtype, kTN, g, cut, s, stream)) != hipSuccess) return rc;
            }
        }
        return hipSuccess;
    }
};

}  // namespace

hipError_t ffn_forward(const FfnCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Ffn<BF16>::forward(c, ar, stream) : Ffn<F16>::forward(c, ar, stream);
}

hipError_t ffn_backward(const FfnGradCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Ffn<BF16>::backward(c, ar, stream)
                            : Ffn<F16>::backward(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
