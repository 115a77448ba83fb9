// C entry points of the norm, the microscaled matrices and sampling: argument
// checks, workspace, status.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "layer_check.h"
#include "mx.h"
#include "mx_math.h"
#include "norm.h"
#include "sample.h"

using namespace pgemm;
using namespace pgemm::layer;

namespace {

bool known_format(int f) { return f == PMX_E2M1 || f == PMX_E4M3; }

// The codes and scales of a microscaled matrix as byte matrices.
struct MxMat {
    Mat codes, scales;
};
MxMat mx_mat(int format, const void* codes, int64_t ldc, const void* scales, int64_t lds,
             int64_t rows, int64_t cols) {
    // scales are read 16 bytes at a time; a single row's pitch is not looked at
    const int64_t c = mx_row_bytes(format, cols), s = round_up(mx_scale_bytes(cols), 16);
    return {{codes, rows, c, rows > 1 ? ldc : c, 1}, {scales, rows, s, rows > 1 ? lds : s, 1}};
}
int check_pitched(const Mat& m) {
    const int rc = check(m, true);
    if (rc != PGEMM_OK || m.rows == 0 || m.cols == 0) return rc;
    if (m.ld >= kMaxCols || m.ld % 16 || !aligned16(m.p)) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}
int check_mx(const MxMat& m) {
    const int rc = check_pitched(m.codes);
    return rc != PGEMM_OK ? rc : check_pitched(m.scales);
}
MxRows mx_rows(int format, const MxMat& m) {
    return {format, static_cast<uint8_t*>(const_cast<void*>(m.codes.p)), m.codes.ld,
            static_cast<uint8_t*>(const_cast<void*>(m.scales.p)), m.scales.ld};
}

// A matrix's sizes.
int check_sizes(int dtype, int64_t M, int64_t D) {
    if (M < 0 || D < 0) return PGEMM_EINVAL;
    if (!known(dtype, PGEMM_ACT_NONE) || M >= kMaxRows || D >= kMaxCols) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}
constexpr int64_t kMaxTiles = (int64_t)1 << 23;
bool valid_eps(float eps) { return eps >= 0.0f && eps < INFINITY; }

int check_mx_linear(int dtype, int xformat, int wformat, int64_t M, int64_t N, int64_t K, int act) {
    if (M < 0 || N < 0 || K < 0) return PGEMM_EINVAL;
    if (!known(dtype, act) || !known_format(xformat) || !known_format(wformat))
        return PGEMM_EUNSUPPORTED;
    // rows of codes have pitches below 2^22 bytes
    if (M >= kMaxRows || N >= kMaxCols || mx_padded(K) >= kMaxCols) return PGEMM_EUNSUPPORTED;
    if (K > 0 && (M > kMaxElems / K || N > kMaxElems / K)) return PGEMM_EUNSUPPORTED;
    // a launch has fewer than 2^32 lanes: tiles of 128 x 128 by 256 lanes
    if (((M + 127) / 128) * ((N + 127) / 128) >= kMaxTiles) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}

// The norm's backward pass; `sum`: at h + residual.
int norm_bwd(NormGradCall c, bool sum, void* workspace, int64_t workspace_bytes,
             pgemm_stream_t stream) {
    const int rc = check_sizes(c.dtype, c.M, c.D);
    if (rc != PGEMM_OK) return rc;
    if (!valid_eps(c.eps)) return PGEMM_EINVAL;
    if (c.D == 0 || (!c.dx && !c.dw)) return PGEMM_OK;
    const int64_t M = c.M, D = c.D;
    const Mat mdy = mat(c.dy, M, D, c.lddy), mh = mat(c.h, M, D, c.ldh),
              mr = mat(c.residual, M, D, c.ldr), mw = flat(c.weight, D, 2),
              mdh = mat(c.dh, M, D, c.lddh), mdx = mat(c.dx, M, D, c.lddx), mdw = flat(c.dw, D, 2);
    Outputs o;
    o.add(check(mdy, true));
    o.add(check(mh, true));
    o.add(check(mr, sum));
    for (const Mat* m : {&mw, &mdh, &mdx, &mdw}) o.add(check(*m, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* out : {&mdx, &mdw}) {
        for (const Mat* in : {&mdy, &mh, &mr, &mw}) o.apart(*out, *in);
        o.apart(*out, mdh, out == &mdx);
    }
    o.apart(mdx, mdw);
    if (o.rc != PGEMM_OK) return o.rc;
    c.lddy = mdy.ld, c.ldh = mh.ld, c.ldr = mr.ld, c.lddh = mdh.ld, c.lddx = mdx.ld;
    const Mat all[] = {mdy, mh, mr, mw, mdh, mdx, mdw};
    return with_workspace(
        [&](Arena& ar) { return norm_backward(c, ar, static_cast<hipStream_t>(stream)); },
        workspace, workspace_bytes, all, 7);
}

}  // namespace

extern "C" {

int64_t pmx_codes_pitch(int format, int64_t cols) {
    if (cols < 0) return PGEMM_EINVAL;
    if (!known_format(format) || mx_padded(cols) >= kMaxCols) return PGEMM_EUNSUPPORTED;
    return mx_row_bytes(format, cols);
}

int64_t pmx_scales_pitch(int64_t cols) {
    if (cols < 0) return PGEMM_EINVAL;
    if (mx_padded(cols) >= kMaxCols) return PGEMM_EUNSUPPORTED;
    return round_up(mx_scale_bytes(cols), 16);
}

int prmsnorm(int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr,
             const void* weight, void* h, int64_t ldh, int format, void* y, int64_t ldy,
             void* scales, int64_t lds, int64_t M, int64_t D, float eps, pgemm_stream_t stream) {
    const int rc = check_sizes(dtype, M, D);
    if (rc != PGEMM_OK) return rc;
    if (!valid_eps(eps)) return PGEMM_EINVAL;
    const bool mx = format != PMX_NONE;
    if (mx && !known_format(format)) return PGEMM_EUNSUPPORTED;
    if (M == 0 || D == 0) return PGEMM_OK;
    const Mat mx_ = mat(x, M, D, ldx), mr = mat(residual, M, D, ldr), mw = flat(weight, D, 2),
              mh = mat(h, M, D, ldh);
    Outputs o;
    o.add(check(mx_, true));
    o.add(check(mr, false));
    o.add(check(mw, false));
    o.add(check(mh, false));
    Mat my = mat(y, M, D, ldy), ms = flat(nullptr, 0, 1);
    MxMat out = {};
    if (mx) {
        out = mx_mat(format, y, ldy, scales, lds, M, D);
        o.add(check_mx(out));
        my = out.codes, ms = out.scales;
    } else {
        o.add(check(my, true));
    }
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* in : {&mx_, &mr}) {
        // a lane reads its part of a row before it writes it
        o.apart(my, *in, !mx);
        o.apart(mh, *in, true);
        o.apart(ms, *in);
    }
    for (const Mat& out_ : {my, mh, ms}) o.apart(out_, mw);
    o.apart(my, mh);
    o.apart(ms, mh);
    o.apart(ms, my);
    if (o.rc != PGEMM_OK) return o.rc;
    NormCall c = {};
    c.dtype = dtype;
    c.x = x, c.ldx = mx_.ld, c.residual = residual, c.ldr = mr.ld, c.weight = weight;
    c.h = h, c.ldh = mh.ld, c.format = mx ? format : -1;
    c.y = y, c.ldy = my.ld;
    if (mx) c.mx = mx_rows(format, out);
    c.M = M, c.D = D, c.eps = eps;
    return hip_status(norm_forward(c, static_cast<hipStream_t>(stream)));
}

int prmsnorm_bwd(int dtype, const void* dy, int64_t lddy, const void* h, int64_t ldh,
                 const void* weight, const void* dh, int64_t lddh, void* dx, int64_t lddx,
                 void* dweight, int64_t M, int64_t D, float eps, void* workspace,
                 int64_t workspace_bytes, pgemm_stream_t stream) {
    return norm_bwd({dtype, dy, lddy, h, ldh, nullptr, 0, weight, dh, lddh, dx, lddx, dweight, M, D,
                     eps},
                    false, workspace, workspace_bytes, stream);
}

int prmsnorm_bwd_sum(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                     const void* residual, int64_t ldr, const void* weight, const void* dh,
                     int64_t lddh, void* dx, int64_t lddx, void* dweight, int64_t M, int64_t D,
                     float eps, void* workspace, int64_t workspace_bytes, pgemm_stream_t stream) {
    return norm_bwd({dtype, dy, lddy, x, ldx, residual, ldr, weight, dh, lddh, dx, lddx, dweight, M,
                     D, eps},
                    true, workspace, workspace_bytes, stream);
}

int64_t prmsnorm_bwd_workspace_bytes(int dtype, int64_t M, int64_t D, int need_dx,
                                     int need_dweight) {
    const int rc = check_sizes(dtype, M, D);
    if (rc != PGEMM_OK) return rc;
    if (D == 0 || (!need_dx && !need_dweight)) return 0;
    if (M > kMaxElems / D) return PGEMM_EUNSUPPORTED;
    void* const some = reinterpret_cast<void*>(16);  // stands for an output; never touched
    NormGradCall c = {};
    c.dtype = dtype;
    c.dx = need_dx ? some : nullptr;
    c.dw = need_dweight ? some : nullptr;
    c.M = M, c.D = D;
    Arena dry = {nullptr, 0};
    const hipError_t e = norm_backward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int pmx_quantize(int dtype, const void* x, int64_t ldx, int format, void* codes, int64_t ldc,
                 void* scales, int64_t lds, int64_t M, int64_t K, pgemm_stream_t stream) {
    const int rc = check_sizes(dtype, M, K);
    if (rc != PGEMM_OK) return rc;
    if (!known_format(format) || mx_padded(K) >= kMaxCols) return PGEMM_EUNSUPPORTED;
    if (M == 0 || K == 0) return PGEMM_OK;
    const Mat mx = mat(x, M, K, ldx);
    const MxMat out = mx_mat(format, codes, ldc, scales, lds, M, K);
    Outputs o;
    o.add(check(mx, true));
    o.add(check_mx(out));
    if (o.rc != PGEMM_OK) return o.rc;
    o.apart(out.codes, mx);
    o.apart(out.scales, mx);
    o.apart(out.codes, out.scales);
    if (o.rc != PGEMM_OK) return o.rc;
    return hip_status(mx_quantize(dtype, x, mx.ld, mx_rows(format, out), M, K,
                                  static_cast<hipStream_t>(stream)));
}

int pmx_dequantize(int format, const void* codes, int64_t ldc, const void* scales, int64_t lds,
                   int dtype, void* y, int64_t ldy, int64_t M, int64_t K, pgemm_stream_t stream) {
    const int rc = check_sizes(dtype, M, K);
    if (rc != PGEMM_OK) return rc;
    if (!known_format(format) || mx_padded(K) >= kMaxCols) return PGEMM_EUNSUPPORTED;
    if (M == 0 || K == 0) return PGEMM_OK;
    const Mat my = mat(y, M, K, ldy);
    const MxMat in = mx_mat(format, codes, ldc, scales, lds, M, K);
    Outputs o;
    o.add(check(my, true));
    o.add(check_mx(in));
    if (o.rc != PGEMM_OK) return o.rc;
    o.apart(my, in.codes);
    o.apart(my, in.scales);
    if (o.rc != PGEMM_OK) return o.rc;
    return hip_status(mx_dequantize(mx_rows(format, in), dtype, y, my.ld, M, K,
                                    static_cast<hipStream_t>(stream)));
}

int pmx_linear(int dtype, int xformat, const void* x, int64_t ldx, const void* xscales,
               int64_t ldxs, int wformat, const void* w, int64_t ldw, const void* wscales,
               int64_t ldws, const void* bias, const void* residual, int64_t ldr, void* y,
               int64_t ldy, int64_t M, int64_t N, int64_t K, int act, void* workspace,
               int64_t workspace_bytes, pgemm_stream_t stream) {
    const int rc = check_mx_linear(dtype, xformat, wformat, M, N, K, act);
    if (rc != PGEMM_OK) return rc;
    if (M == 0 || N == 0) return PGEMM_OK;
    const bool quantizes = xscales == nullptr && K > 0;
    Mat mx = mat(x, M, K, ldx), mxs = flat(nullptr, 0, 1);
    MxMat xin = {};
    Outputs o;
    if (quantizes) {
        o.add(check(mx, true));
    } else {
        xin = mx_mat(xformat, x, ldx, xscales, ldxs, M, K);
        o.add(check_mx(xin));
        mx = xin.codes, mxs = xin.scales;
    }
    const MxMat win = mx_mat(wformat, w, ldw, wscales, ldws, N, K);
    const Mat mb = flat(bias, N, 2), mr = mat(residual, M, N, ldr), my = mat(y, M, N, ldy);
    o.add(check_mx(win));
    o.add(check(mb, false));
    o.add(check(mr, false));
    o.add(check(my, true));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat& in : {mx, mxs, win.codes, win.scales, mb}) o.apart(my, in);
    o.apart(my, mr, true);
    if (o.rc != PGEMM_OK) return o.rc;
    MxLinearCall c = {};
    c.dtype = dtype;
    c.x = mx_rows(xformat, xin);
    c.x16 = quantizes ? x : nullptr;
    c.ldx16 = mx.ld;
    c.w = mx_rows(wformat, win);
    c.bias = bias, c.residual = residual, c.ldr = mr.ld, c.y = y, c.ldy = my.ld;
    c.M = M, c.N = N, c.K = K, c.act = act;
    const Mat all[] = {mx, mxs, win.codes, win.scales, mb, mr, my};
    return with_workspace(
        [&](Arena& ar) { return mx_linear(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 7);
}

int64_t pmx_linear_workspace_bytes(int dtype, int xformat, int quantizes, int wformat, int64_t M,
                                   int64_t N, int64_t K) {
    const int rc = check_mx_linear(dtype, xformat, wformat, M, N, K, PGEMM_ACT_NONE);
    if (rc != PGEMM_OK) return rc;
    MxLinearCall c = {};
    c.dtype = dtype;
    c.x.format = xformat, c.w.format = wformat;
    c.x16 = quantizes && K > 0 ? reinterpret_cast<void*>(16) : nullptr;  // never touched
    c.M = M, c.N = N, c.K = K;
    Arena dry = {nullptr, 0};
    const hipError_t e = mx_linear(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int psample(int dtype, const void* logits, int64_t ld, const float* u, float temperature,
            const float* temperatures, int32_t top_k, const int32_t* top_ks, float top_p,
            const float* top_ps, float min_p, const float* min_ps, int64_t* tokens,
            float* logprobs, int64_t M, int64_t V, void* workspace, int64_t workspace_bytes,
            pgemm_stream_t stream) {
    if (M < 0 || V < 1) return PGEMM_EINVAL;
    if (!temperatures && !(temperature >= 0.0f)) return PGEMM_EINVAL;
    if (!top_ps && !(top_p >= 0.0f)) return PGEMM_EINVAL;
    if (!min_ps && !(min_p >= 0.0f && min_p <= 1.0f)) return PGEMM_EINVAL;
    if (dtype != PGEMM_F16 && dtype != PGEMM_BF16 && dtype != PGEMM_F32) return PGEMM_EUNSUPPORTED;
    if (M >= kMaxRows || V >= kMaxCols) return PGEMM_EUNSUPPORTED;
    if (M == 0) return PGEMM_OK;
    Mat ml = mat(logits, M, V, ld);
    ml.bytes = dtype == PGEMM_F32 ? 4 : 2;
    const Mat in[] = {ml, flat(u, M, 4), flat(temperatures, M, 4), flat(top_ks, M, 4),
                      flat(top_ps, M, 4), flat(min_ps, M, 4)};
    const Mat out[] = {flat(tokens, M, 8), flat(logprobs, M, 4)};
    Outputs o;
    for (int i = 0; i < 6; ++i) o.add(check(in[i], i < 2));
    for (int i = 0; i < 2; ++i) o.add(check(out[i], i == 0));
    if (o.rc != PGEMM_OK) return o.rc;
    if (ml.ld >= kMaxCols) return PGEMM_EUNSUPPORTED;
    for (const Mat& a : out)
        for (const Mat& b : in) o.apart(a, b);
    o.apart(out[0], out[1]);
    if (o.rc != PGEMM_OK) return o.rc;
    SampleCall c = {};
    c.dtype = dtype, c.logits = logits, c.ld = ml.ld, c.u = u;
    c.temperature = {temperature, temperatures};
    c.top_p = {top_p, top_ps};
    c.min_p = {min_p, min_ps};
    c.top_k = {top_k, top_ks};
    c.tokens = tokens, c.logprobs = logprobs, c.M = M, c.V = V;
    const Mat all[] = {in[0], in[1], in[2], in[3], in[4], in[5], out[0], out[1]};
    return with_workspace(
        [&](Arena& ar) { return sample(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 8);
}

int64_t psample_workspace_bytes(int dtype, int64_t M, int64_t V) {
    if (M < 0 || V < 1) return PGEMM_EINVAL;
    if (dtype != PGEMM_F16 && dtype != PGEMM_BF16 && dtype != PGEMM_F32) return PGEMM_EUNSUPPORTED;
    if (M >= kMaxRows || V >= kMaxCols || M > kMaxElems / V) return PGEMM_EUNSUPPORTED;
    SampleCall c = {};
    c.dtype = dtype, c.M = M, c.V = V;
    Arena dry = {nullptr, 0};
    const hipError_t e = sample(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

}  // extern "C"
