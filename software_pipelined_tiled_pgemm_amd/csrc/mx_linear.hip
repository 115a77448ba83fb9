// The linear layer on microscaled matrices: x's quantisation where it is not yet
// microscaled, the choice of kernel, workspace.
#include <algorithm>

#include "internal.h"
#include "mx.h"
#include "mx_math.h"

namespace pgemm {
namespace layer {
namespace {

// Estimated microseconds of tiles, with constants measured on MI355X: a step of 128
// columns takes `step` in the 256 x 256 tiles (256 x 128 for 8-bit elements on both
// sides), `pair` in two 128 x 128 tiles on a CU and `alone` in a single one; a round of
// workgroups adds its first copies and its epilogue, and a split a second launch and
// the partials' traffic.
struct Rates {
    int columns;
    double step, pair, alone;
};
double cut_time(const Rates& q, int64_t M, int64_t N, int steps, int cus, bool big, int splits) {
    const int64_t bm = big ? 256 : 128, bn = big ? q.columns : 128;
    const int64_t wgs = ((M + bm - 1) / bm) * ((N + bn - 1) / bn) * splits;
    const int64_t slots = big ? cus : 2 * cus;
    const double step = big ? q.step : wgs <= cus ? q.alone : q.pair;
    const double rounds = (double)((wgs + slots - 1) / slots);
    double t = rounds * ((double)((steps + splits - 1) / splits) * step + (big ? 8.0 : 3.0));
    if (splits > 1) t += 8.0 + (double)splits * M * N * 8.0 / 4.0e6;
    return t;
}

// Estimated microseconds of the kernel for few rows: a workgroup takes 16 columns of y, and
// each of its steps the reading of w and the multiplications of its rows.  (Fitted to 352
// measured products of 1-64 rows, 512-131072 columns, 8-128 steps and every pair of formats,
// from which it is 8% off.)
double few_time(int xformat, int wformat, int64_t M, int64_t N, int steps, int cus) {
    const double read = wformat == PMX_E2M1 ? 0.059 : 0.098,
                 row = xformat == PMX_E2M1 ? 0.00225 : 0.0039;
    const double rounds = std::max(1.0, (double)((N + 15) / 16) / cus);
    return 2.4 + rounds * (0.2 + steps * (read + row * (double)M));
}

// Up to 64 rows go by the kernel for few rows or by tiles, whichever is estimated the
// faster: tiles hold more of w at a time, and win where there are many columns.  Few rows /
// tiles, us, e4m3 x e2m1, K 4096:
//     columns      1 row         16 rows        32 rows        64 rows
//       4096      5.0 / 10.0    6.6 / 10.8     8.5 / 11.1    12.4 / 12.7
//       8192      7.0 / 10.8    9.7 / 11.7    13.7 / 13.2    23.0 / 19.0
//      16384     11.6 / 18.8   16.8 / 18.9    24.5 / 19.2    43.5 / 20.1
//     131072     72.0 / 64.9  111.8 / 66.9   169.9 / 69.6   325.4 / 76.7
// (The choice takes 1% longer than the better of both in the mean of the 352, up to 41% where
// tiles are estimated too low; the kernel for few rows in all of them 20%, up to 4.2 times.)
// From 65 rows on it takes a second block of rows: 96 rows x 4096 19.4 / 19.1, x 8192 36.0 /
// 19.6.
constexpr int64_t kMxFewRows = 64;

MxCut choose_mx_cut(int xformat, int wformat, int64_t M, int64_t N, int steps, int cus) {
    const int eights = (xformat == PMX_E4M3) + (wformat == PMX_E4M3);
    const Rates q = eights == 0   ? Rates{256, 0.85, 0.75, 0.33}
                    : eights == 1 ? Rates{256, 1.35, 0.97, 0.45}
                                  : Rates{128, 0.95, 1.05, 0.70};
    MxCut best = {M <= kMxFewRows, false, 1, steps};
    double best_t = best.few ? few_time(xformat, wformat, M, N, steps, cus) : 1e300;
    for (int s : {1, 2, 3, 4, 6, 8}) {
        // at least 8 steps a split, whole groups of 4
        const int chunk = s == 1 ? steps : ((steps + s - 1) / s + 3) / 4 * 4;
        if (s > 1 && chunk < 8) break;
        const int parts = s == 1 ? 1 : (steps + chunk - 1) / chunk;
        for (bool big : {false, true}) {
            const double t = cut_time(q, M, N, steps, cus, big, parts);
            if (t < best_t) {
                best_t = t;
                best = {false, big, parts, parts > 1 ? chunk : steps};
            }
        }
    }
    return best;
}

}  // namespace

hipError_t mx_linear(const MxLinearCall& c, Arena& ar, hipStream_t stream) {
    if (c.M == 0 || c.N == 0) return hipSuccess;
    MxRows x = c.x;
    MxArgs a = {};
    a.M = (int)c.M, a.N = (int)c.N, a.steps = (int)(mx_padded(c.K) / kMxGroup);
    const MxCut cut = choose_mx_cut(x.format, c.w.format, c.M, c.N, a.steps, compute_units());
    a.chunk = cut.chunk;
    if (c.x16 && cut.few && c.M <= 4 && c.M * mx_padded(c.K) <= kMxFewValues) {
        // quantised by the kernel: 1 x 4096 x 8192 16.9 -> 12.8 us a call, since a launch
        // of its own costs more than every workgroup's doing it, up to 4 rows (in the kernel /
        // by a launch, us, to e4m3: 4 x 4096 x 8192 9.1 / 10.3, 4 x 2048 x 16384 11.2 / 11.1, 4 x
        // 1024 x 4096 5.2 / 6.1; 6 x 2048 x 16384 12.9 / 11.3, 6 x 500 x 1000 6.6 / 6.0, 8 x 1024
        // x 4096 6.7 / 6.2)
        a.x16 = static_cast<const uint16_t*>(c.x16);
        a.ldx16 = c.ldx16;
        a.cols = (int)c.K;
    } else if (c.x16) {
        x.ld = mx_row_bytes(x.format, c.K);
        x.lds = round_up(mx_scale_bytes(c.K), 16);
        x.codes = static_cast<uint8_t*>(ar.take(c.M * x.ld));
        x.scales = static_cast<uint8_t*>(ar.take(c.M * x.lds));
        if (!ar.dry()) {
            const hipError_t rc = mx_quantize(c.dtype, c.x16, c.ldx16, x, c.M, c.K, stream);
            if (rc != hipSuccess) return rc;
        }
    }
    a.x = x.codes, a.xs = x.scales, a.w = c.w.codes, a.ws = c.w.scales;
    a.ldx = x.ld, a.ldxs = x.lds, a.ldw = c.w.ld, a.ldws = c.w.lds;
    if (cut.splits > 1) {
        a.part_ld = (int)round_up(a.N, 8);
        a.part = static_cast<float*>(ar.take((int64_t)cut.splits * a.M * a.part_ld * 4));
    }
    if (ar.dry()) return hipSuccess;
    return c.dtype == kBF16 ? mx_product_bf16(x.format, c.w.format, a, cut, c, stream)
                            : mx_product_f16(x.format, c.w.format, a, cut, c, stream);
}

}  // namespace layer
}  // namespace pgemm
