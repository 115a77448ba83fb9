// The linear layer with its epilogue, and its backward pass.
//
//   forward    z = x W + b,  y = act(z) + r           x [M,K], W [K,N]
//   backward   dz = dy * act'(z)
//              dx = dz W^T (+ a),  dW = x^T dz,  db = sum over rows of dz
//
// z is summed in fp32 and y rounded once; the backward pass takes z as the
// forward pass stored it (rounded to the type, which moves act' by no more
// than a rounding of dy would), computes dz in fp32 and rounds it once, as
// the operand of two products.  db adds the unrounded dz in fp32, in a fixed
// order.
#include "linear.h"
#include "linear_epi.h"

namespace pgemm {
namespace layer {
namespace {

// y = v + add, the gradients' epilogue; half > 0: two padded halves of
// columns (Sink).
template <class E>
struct GradEpi {
    static constexpr lp::EpiKind kind = lp::kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 4;
    Rows y, add;
    int half;
    __device__ __forceinline__ GradEpi from(int64_t r) const {
        return {y.from(r), add.from(r), half};
    }
    __device__ __forceinline__ lp::Nothing column(int, int) const { return {}; }
    __device__ __forceinline__ u4_t load(int row, int col, int nv) const {
        return add ? load8_bits(add, row, col, nv) : u4_t{};
    }
    __device__ __forceinline__ bool aligned() const { return y.aligned && half % 8 == 0; }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        run([&](int row, int col, int nv, float(&v)[8], lp::Nothing, u4_t r)
                __attribute__((always_inline)) {
            if (add) {
                float t[8];
                unpack8<E>(r, t);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += t[q];
            }
            if (half > 0) {
                const int h8 = (half + 7) & ~7;
                const int second = col >= h8;
                const int c = col - (second ? h8 : 0);
                nv = min(8, half - c);
                col = c + (second ? half : 0);
            }
            store8<E, STREAM>(y, row, col, nv, v);
        });
    }
};

// dz = dy * act'(z), and the column sums of each block of `per` rows.  A
// workgroup covers 512 columns (64 lanes of 8) in 4 row lanes.  Memory
// bound: reads dy and z, writes dz, once each (8192 x 4096 bf16: 45-50 us for
// 201 MB, 4.0-4.5 TB/s).
constexpr int64_t kDzRows = 64;
constexpr int64_t kDzBlocks = 32768;  // most row blocks of a launch (grid y)

template <class E>
__global__ __launch_bounds__(256) void dz_kernel(const Rows dy0, const Rows pre0, const Rows dz0,
                                                 float* __restrict__ part, int64_t M, int N,
                                                 int dz_cols, int64_t per, int act) {
    __shared__ float sums[4][512];
    const int cl = threadIdx.x & 63, rl = threadIdx.x >> 6;
    const int col = (blockIdx.x * 64 + cl) * 8;
    const int nv = min(8, N - col);
    const int64_t r0 = (int64_t)blockIdx.y * per;
    const int64_t end = r0 + per < M ? r0 + per : M;
    float s[8] = {};
    if (col < dz_cols) {
        with_act(act, [&](auto a) __attribute__((always_inline)) {
            auto one = [&](const Rows& dz, int r, const u4_t& db, const u4_t& zb) __attribute__((always_inline)) {
                float d[8], z[8];
                unpack8<E>(db, d);
                unpack8<E>(zb, z);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float value;
                    if (pre0) d[q] *= decltype(a)::grad(z[q], value);
                    if (q >= nv) d[q] = 0.0f;
                    s[q] += d[q];
                }
                // dz rows are padded with zeros to whole chunks
                if (dz) store8<E, true>(dz, r, col, 8, d);
            };
            // kDzRows rows at a time, 4 rows' loads in flight per lane
            for (int64_t rb = r0; rb < end; rb += kDzRows) {
                const int rows = (int)(end - rb < kDzRows ? end - rb : kDzRows);
                const Rows dy = dy0.from(rb), pre = pre0.from(rb), dz = dz0.from(rb);
                int r = rl;
                for (; r + 12 < rows; r += 16) {
                    u4_t db[4], zb[4] = {};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        db[u] = load8_bits(dy, r + 4 * u, col, nv);
                        if (pre) zb[u] = load8_bits(pre, r + 4 * u, col, nv);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) one(dz, r + 4 * u, db[u], zb[u]);
                }
                for (; r < rows; r += 4)
                    one(dz, r, load8_bits(dy, r, col, nv),
                        pre ? load8_bits(pre, r, col, nv) : u4_t{});
            }
        });
    }
    if (part) {
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[rl][cl * 8 + q] = s[q];
        __syncthreads();
        for (int c = threadIdx.x; c < 512; c += 256) {
            const int64_t gc = (int64_t)blockIdx.x * 512 + c;
            if (gc < N)
                part[blockIdx.y * (int64_t)N + gc] =
                    ((sums[0][c] + sums[1][c]) + sums[2][c]) + sums[3][c];
        }
    }
}

template <class E>
hipError_t launch_linear_as(int layout, const Args& g, const Cut& cut, const Sink& s,
                            hipStream_t stream) {
    const Rows y = make_rows(s.y, s.ldy), res = make_rows(s.residual, s.ldr);
    if (layout == kNN) {
        const LinearEpi<E> epi = {y, res, make_rows(s.preact, s.ldp),
                                  static_cast<const uint16_t*>(s.bias), s.act};
        return lp::launch_product<E, true, false>(g, cut, epi, stream);
    }
    const GradEpi<E> epi = {y, res, s.half};
    return layout == kNT ? lp::launch_product<E, true, true>(g, cut, epi, stream)
                         : lp::launch_product<E, false, false>(g, cut, epi, stream);
}

template <class E>
struct Linear {
    static hipError_t forward(const LinearCall& c, Arena& ar, hipStream_t stream) {
        View x, w;
        hipError_t rc;
        if ((rc = operand(c.x, c.ldx, c.M, c.K, ar, stream, x)) != hipSuccess) return rc;
        if ((rc = operand(c.w, c.ldw, c.K, c.N, ar, stream, w)) != hipSuccess) return rc;
        const Cut cut = choose_cut(c.M, c.N, c.K, compute_units(), 16);
        const Args g = args(x, w, c.M, c.N, c.K, cut, ar);
        if (ar.dry()) return hipSuccess;
        const Sink s = {c.y, c.ldy, c.residual, c.ldr, c.preact, c.ldp, c.bias, c.act, 0};
        return launch_linear_as<E>(kNN, g, cut, s, stream);
    }

    static hipError_t backward(const LinearGradCall& c, Arena& ar, hipStream_t stream) {
        hipError_t rc;
        const bool act = c.act != PGEMM_ACT_NONE;
        // dz: dy itself where there is no activation and it can be copied
        // from where it lies, else a padded copy in the workspace.
        View dz = {static_cast<const uint16_t*>(c.dy), (int)c.lddy};
        const bool need_dz = (c.dx || c.dw) && (act || !direct(c.dy, c.lddy, c.N));
        const int64_t n8 = round_up(c.N, 8);
        uint16_t* dzw = nullptr;
        if (need_dz) {
            dzw = static_cast<uint16_t*>(ar.take(c.M * n8 * 2));
            dz = {dzw, (int)n8};
        }
        // Rows per workgroup: fewer where there would be too few workgroups.
        const int64_t strips = (n8 + 511) / 512;
        int64_t per = kDzRows * std::max<int64_t>(1, (c.M + kDzRows * kDzBlocks - 1) /
                                                        (kDzRows * kDzBlocks));
        while (per > 16 && strips * ((c.M + per - 1) / per) < 1024) per /= 2;
        const int64_t blocks = (c.M + per - 1) / per;
        float* part = nullptr;
        if (c.dbias) part = static_cast<float*>(ar.take(std::max<int64_t>(blocks, 1) * c.N * 4));
        if (!ar.dry() && c.M > 0 && c.N > 0 && (need_dz || c.dbias)) {
            const dim3 grid((unsigned)((n8 + 511) / 512), (unsigned)blocks);
            hipLaunchKernelGGL(dz_kernel<E>, grid, dim3(256), 0, stream, make_rows(c.dy, c.lddy),
                               act ? make_rows(c.preact, c.ldp) : Rows{nullptr, 0, 0},
                               need_dz ? Rows{dzw, (int)n8, 1} : Rows{nullptr, 0, 0}, part, c.M,
                               (int)c.N, need_dz ? (int)n8 : (int)c.N, per, c.act);
            if ((rc = hipGetLastError()) != hipSuccess) return rc;
        }
        if (!ar.dry() && c.dbias && c.N > 0) {
            rc = launch_column_sum(dtype(), part, c.M > 0 ? blocks : 0, c.N, c.dbias, stream);
            if (rc != hipSuccess) return rc;
        }
        if (c.dx && c.M > 0 && c.K > 0) {
            View w;
            if ((rc = operand(c.w, c.ldw, c.K, c.N, ar, stream, w)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.M, c.K, c.N, compute_units(), 16);
            const Args g = args(dz, w, c.M, c.K, c.N, cut, ar);
            if (!ar.dry()) {
                const Sink s = {c.dx, c.lddx, c.add, c.ldadd, nullptr, 0, nullptr, 0, 0};
                rc = launch_linear_as<E>(kNT, g, cut, s, stream);
                if (rc != hipSuccess) return rc;
            }
        }
        if (c.dw && c.K > 0 && c.N > 0) {
            View x;
            if ((rc = operand(c.x, c.ldx, c.M, c.K, ar, stream, x)) != hipSuccess) return rc;
            const Cut cut = choose_cut(c.K, c.N, c.M, compute_units(), 16);
            const Args g = args(x, dz, c.K, c.N, c.M, cut, ar);
            if (!ar.dry()) {
                const Sink s = {c.dw, c.lddw, nullptr, 0, nullptr, 0, nullptr, 0, 0};
                rc = launch_linear_as<E>(kTN, g, cut, s, stream);
                if (rc != hipSuccess) return rc;
            }
        }
        return hipSuccess;
    }

    static constexpr int dtype() { return std::is_same<E, BF16>::value ? kBF16 : kF16; }
};

}  // namespace

hipError_t launch_linear(int dtype, int layout, const Args& g, const Cut& cut, const Sink& sink,
                         hipStream_t stream) {
    return dtype == kBF16 ? launch_linear_as<BF16>(layout, g, cut, sink, stream)
                          : launch_linear_as<F16>(layout, g, cut, sink, stream);
}

hipError_t linear_forward(const LinearCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Linear<BF16>::forward(c, ar, stream)
                            : Linear<F16>::forward(c, ar, stream);
}

hipError_t linear_backward(const LinearGradCall& c, Arena& ar, hipStream_t stream) {
    return c.dtype == kBF16 ? Linear<BF16>::backward(c, ar, stream)
                            : Linear<F16>::backward(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
