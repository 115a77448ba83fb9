// C entry points of the layer operators: argument checks, workspace, status.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pgemm.h"
#include <algorithm>
#include <memory>
#include <new>

#include "clip.h"
#include "ffn.h"
#include "linear.h"
#include "xent.h"

namespace {

using namespace pgemm::layer;

constexpr int64_t kMaxCols = (int64_t)1 << 22;  // row lengths and pitches
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 256;
constexpr int64_t kMaxElems = (int64_t)1 << 37;

// A matrix argument: what overlap and size checks need of it.
struct Mat {
    const void* p;
    int64_t rows, cols, ld;  // ld in elements
    int bytes;               // per element
    bool empty() const { return !p || rows == 0 || cols == 0; }
    int64_t extent() const { return ((rows - 1) * ld + cols) * bytes; }
};

Mat mat(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {p, rows, cols, rows > 1 ? ld : cols, 2};
}
Mat flat(const void* p, int64_t n, int bytes) { return {p, 1, n, n, bytes}; }

// Status of a matrix's own description; `needed`: it must not be NULL unless
// it is empty.
int check(const Mat& m, bool needed) {
    if (m.rows < 0 || m.cols < 0) return PGEMM_EINVAL;
    if (m.rows == 0 || m.cols == 0) return PGEMM_OK;
    if (!m.p) return needed ? PGEMM_EINVAL : PGEMM_OK;
    if (m.ld < m.cols) return PGEMM_EINVAL;
    if (m.bytes == 2 && (m.ld >= kMaxCols || m.cols >= kMaxCols)) return PGEMM_EUNSUPPORTED;
    if (m.rows >= kMaxRows || m.rows > kMaxElems / m.cols) return PGEMM_EUNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(m.p) % (uintptr_t)m.bytes) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}

// The two matrices share an element.  Column ranges of one buffer (the same
// pitch) are told apart by their column offsets.
bool shares(const Mat& a, const Mat& b) {
    if (a.empty() || b.empty()) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (a0 >= b0 + (uintptr_t)b.extent() || b0 >= a0 + (uintptr_t)a.extent()) return false;
    if (a.rows > 1 && b.rows > 1 && a.ld == b.ld && a.bytes == b.bytes) {
        const int64_t pitch = a.ld * a.bytes;
        int64_t d = (int64_t)(b0 - a0) % pitch;
        if (d < 0) d += pitch;
        if (d >= a.cols * a.bytes && d + b.cols * b.bytes <= pitch) return false;
    }
    return true;
}

// Outputs against everything: `same` names an input that an output may equal
// exactly.
struct Outputs {
    int rc = PGEMM_OK;
    void fail(int status) {
        if (rc == PGEMM_OK) rc = status;
    }
    void apart(const Mat& out, const Mat& other, bool may_equal = false) {
        if (may_equal && out.p == other.p && out.ld == other.ld && out.cols == other.cols) return;
        if (shares(out, other)) fail(PGEMM_EINVAL);
    }
    void add(int status) { if (status != PGEMM_OK) fail(status); }
};

int hip_status(hipError_t e) { return pgemm::record_hip_status(e); }

bool known(int dtype, int act) {
    return (dtype == PGEMM_F16 || dtype == PGEMM_BF16) && act >= PGEMM_ACT_NONE &&
           act <= PGEMM_ACT_SILU;
}

// Runs `f` once dry, to size the workspace, and then on it.  `others`: the
// call's buffers, which the workspace must not share memory with.
template <class F>
int with_workspace(F&& f, void* workspace, int64_t workspace_bytes, const Mat* others, int n) {
    Arena dry = {nullptr, 0};
    hipError_t e = f(dry);
    if (e != hipSuccess) return hip_status(e);
    Arena ar = {static_cast<char*>(workspace), 0};
    if (dry.used > 0) {
        if (!workspace || workspace_bytes < dry.used) return PGEMM_EINVAL;
        if (!aligned16(workspace)) return PGEMM_EUNSUPPORTED;
        const Mat ws = flat(workspace, dry.used, 1);
        for (int i = 0; i < n; ++i)
            if (shares(ws, others[i])) return PGEMM_EINVAL;
    } else {
        // nothing will be taken, but a null base would mean a dry run
        static char none;
        ar.base = &none;
    }
    return hip_status(f(ar));
}

int check_linear(int dtype, int act, int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0) return PGEMM_EINVAL;
    if (!known(dtype, act)) return PGEMM_EUNSUPPORTED;
    if (M >= kMaxRows || N >= kMaxCols || K >= kMaxCols) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}

int check_ffn(int dtype, int act, int64_t M, int64_t D, int64_t F, int64_t N) {
    if (F < 0 || N < 0) return PGEMM_EINVAL;
    const int rc = check_linear(dtype, act, M, D, N);
    if (rc != PGEMM_OK) return rc;
    // [g | u] in padded halves is a matrix like the others
    if (F > kMaxCols / 2 - 8 || (F > 0 && M > kMaxElems / (2 * F))) return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}

// Gradient clipping.
constexpr int64_t kMaxTensors = (int64_t)1 << 20;
constexpr int64_t kMaxTensorElems = (int64_t)1 << 40;
struct Range {
    uintptr_t begin, end;
    bool writes;
};

int check_xent(int dtype, int reduction, int64_t M, int64_t V, int64_t D) {
    if (M < 0 || V < 1 || D < 0) return PGEMM_EINVAL;
    if (!known(dtype, PGEMM_ACT_NONE) || reduction < PGEMM_REDUCE_NONE ||
        reduction > PGEMM_REDUCE_SUM)
        return PGEMM_EUNSUPPORTED;
    if (M >= kMaxRows || V >= kMaxRows || D >= kMaxCols || M > kMaxElems / V)
        return PGEMM_EUNSUPPORTED;
    return PGEMM_OK;
}

}  // namespace

extern "C" {

int plinear(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
            const void* residual, int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldp,
            int64_t M, int64_t N, int64_t K, int act, void* workspace, int64_t workspace_bytes,
            pgemm_stream_t stream) {
    int rc = check_linear(dtype, act, M, N, K);
    if (rc != PGEMM_OK) return rc;
    if (M == 0 || N == 0) return PGEMM_OK;
    const Mat mx = mat(x, M, K, ldx), mw = mat(w, K, N, ldw), mb = flat(bias, N, 2),
              mr = mat(residual, M, N, ldr), my = mat(y, M, N, ldy), mp = mat(preact, M, N, ldp);
    Outputs o;
    o.add(check(mx, true));
    o.add(check(mw, true));
    o.add(check(mb, false));
    o.add(check(mr, false));
    o.add(check(my, true));
    o.add(check(mp, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* in : {&mx, &mw, &mb}) {
        o.apart(my, *in);
        o.apart(mp, *in);
    }
    o.apart(my, mr, true);
    o.apart(mp, mr);
    o.apart(mp, my);
    if (o.rc != PGEMM_OK) return o.rc;
    const LinearCall c = {dtype, x, mx.ld, w, mw.ld, bias, residual, mr.ld, y, my.ld, preact, mp.ld,
                          M, N, K, act};
    const Mat all[] = {mx, mw, mb, mr, my, mp};
    return with_workspace(
        [&](Arena& ar) { return linear_forward(c, ar, static_cast<hipStream_t>(stream)); },
        workspace, workspace_bytes, all, 6);
}

int64_t plinear_workspace_bytes(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                int64_t M, int64_t N, int64_t K) {
    int rc = check_linear(dtype, PGEMM_ACT_NONE, M, N, K);
    if (rc != PGEMM_OK) return rc;
    if (M == 0 || N == 0) return 0;
    const Mat mx = mat(x, M, K, ldx), mw = mat(w, K, N, ldw);
    if ((rc = check(mx, true)) != PGEMM_OK || (rc = check(mw, true)) != PGEMM_OK) return rc;
    LinearCall c = {};
    c.dtype = dtype;
    c.x = x, c.ldx = mx.ld, c.w = w, c.ldw = mw.ld;
    c.M = M, c.N = N, c.K = K;
    Arena dry = {nullptr, 0};
    const hipError_t e = linear_forward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int plinear_bwd(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                int64_t ldw, const void* preact, int64_t ldp, const void* add, int64_t ldadd,
                void* dx, int64_t lddx, void* dw, int64_t lddw, void* dbias, int64_t M, int64_t N,
                int64_t K, int act, void* workspace, int64_t workspace_bytes,
                pgemm_stream_t stream) {
    int rc = check_linear(dtype, act, M, N, K);
    if (rc != PGEMM_OK) return rc;
    const Mat mdy = mat(dy, M, N, lddy), mx = mat(x, M, K, ldx), mw = mat(w, K, N, ldw),
              mp = mat(preact, M, N, ldp), ma = mat(add, M, K, ldadd), mdx = mat(dx, M, K, lddx),
              mdw = mat(dw, K, N, lddw), mdb = flat(dbias, N, 2);
    Outputs o;
    o.add(check(mdy, dx || dw || dbias));
    o.add(check(mx, dw != nullptr));
    o.add(check(mw, dx != nullptr));
    o.add(check(mp, act != PGEMM_ACT_NONE && (dx || dw || dbias)));
    o.add(check(ma, false));
    o.add(check(mdx, false));
    o.add(check(mdw, false));
    o.add(check(mdb, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* out : {&mdx, &mdw, &mdb}) {
        for (const Mat* in : {&mdy, &mx, &mw, &mp}) o.apart(*out, *in);
        o.apart(*out, ma, out == &mdx);
    }
    o.apart(mdx, mdw);
    o.apart(mdx, mdb);
    o.apart(mdw, mdb);
    if (o.rc != PGEMM_OK) return o.rc;
    const LinearGradCall c = {dtype, dy, mdy.ld, x, mx.ld, w, mw.ld, preact, mp.ld, add, ma.ld,
                              dx, mdx.ld, dw, mdw.ld, dbias, M, N, K, act};
    const Mat all[] = {mdy, mx, mw, mp, ma, mdx, mdw, mdb};
    return with_workspace(
        [&](Arena& ar) { return linear_backward(c, ar, static_cast<hipStream_t>(stream)); },
        workspace, workspace_bytes, all, 8);
}

int64_t plinear_bwd_workspace_bytes(int dtype, const void* dy, int64_t lddy, const void* x,
                                    int64_t ldx, const void* w, int64_t ldw, int64_t M, int64_t N,
                                    int64_t K, int act, int need_dx, int need_dw, int need_dbias) {
    int rc = check_linear(dtype, act, M, N, K);
    if (rc != PGEMM_OK) return rc;
    const Mat mdy = mat(dy, M, N, lddy), mx = mat(x, M, K, ldx), mw = mat(w, K, N, ldw);
    if ((rc = check(mdy, need_dx || need_dw || need_dbias)) != PGEMM_OK ||
        (rc = check(mx, need_dw != 0)) != PGEMM_OK || (rc = check(mw, need_dx != 0)) != PGEMM_OK)
        return rc;
    LinearGradCall c = {};
    void* const some = reinterpret_cast<void*>(16);  // stands for an output; never touched
    c.dtype = dtype;
    c.dy = dy, c.lddy = mdy.ld, c.x = x, c.ldx = mx.ld, c.w = w, c.ldw = mw.ld;
    c.dx = need_dx ? some : nullptr;
    c.dw = need_dw ? some : nullptr;
    c.dbias = need_dbias ? some : nullptr;
    c.M = M, c.N = N, c.K = K, c.act = act;
    Arena dry = {nullptr, 0};
    const hipError_t e = linear_backward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int pffn(int dtype, const void* x, int64_t ldx, const void* w_in, int64_t ldwi, const void* w_out,
         int64_t ldwo, const void* residual, int64_t ldr, void* y, int64_t ldy, void* gate_up,
         int64_t ldgu, int64_t M, int64_t D, int64_t F, int64_t N, int act, void* workspace,
         int64_t workspace_bytes, pgemm_stream_t stream) {
    const int rc = check_ffn(dtype, act, M, D, F, N);
    if (rc != PGEMM_OK) return rc;
    if (M == 0 || (N == 0 && !gate_up)) return PGEMM_OK;
    const Mat mx = mat(x, M, D, ldx), mwi = mat(w_in, D, 2 * F, ldwi), mwo = mat(w_out, F, N, ldwo),
              mr = mat(residual, M, N, ldr), my = mat(y, M, N, ldy),
              mgu = mat(gate_up, M, 2 * F, ldgu);
    Outputs o;
    o.add(check(mx, F > 0));
    o.add(check(mwi, true));
    o.add(check(mwo, true));
    o.add(check(mr, false));
    o.add(check(my, true));
    o.add(check(mgu, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* in : {&mx, &mwi, &mwo}) {
        // y is written by the last launch, which no longer reads x: y may
        // take the place of x where x is the residual
        o.apart(my, *in, in == &mx);
        o.apart(mgu, *in);
    }
    o.apart(my, mr, true);
    o.apart(mgu, mr);
    o.apart(mgu, my);
    if (o.rc != PGEMM_OK) return o.rc;
    const FfnCall c = {dtype, x, mx.ld, w_in, mwi.ld, w_out, mwo.ld, residual, mr.ld, y, my.ld,
                       gate_up, mgu.ld, M, D, F, N, act};
    const Mat all[] = {mx, mwi, mwo, mr, my, mgu};
    return with_workspace(
        [&](Arena& ar) { return ffn_forward(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 6);
}

int64_t pffn_workspace_bytes(int dtype, const void* x, int64_t ldx, const void* w_in, int64_t ldwi,
                             const void* w_out, int64_t ldwo, int64_t M, int64_t D, int64_t F,
                             int64_t N) {
    const int rc = check_ffn(dtype, PGEMM_ACT_NONE, M, D, F, N);
    if (rc != PGEMM_OK) return rc;
    if (M == 0) return 0;
    const Mat mx = mat(x, M, D, ldx), mwi = mat(w_in, D, 2 * F, ldwi), mwo = mat(w_out, F, N, ldwo);
    Outputs o;
    o.add(check(mx, F > 0));
    o.add(check(mwi, true));
    o.add(check(mwo, true));
    if (o.rc != PGEMM_OK) return o.rc;
    FfnCall c = {};
    c.dtype = dtype;
    c.x = x, c.ldx = mx.ld, c.w_in = w_in, c.ldwi = mwi.ld, c.w_out = w_out, c.ldwo = mwo.ld;
    c.M = M, c.D = D, c.F = F, c.N = N;
    Arena dry = {nullptr, 0};
    const hipError_t e = ffn_forward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int pffn_bwd(int dtype, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_in,
             int64_t ldwi, const void* w_out, int64_t ldwo, const void* gate_up, int64_t ldgu,
             const void* add, int64_t ldadd, void* dx, int64_t lddx, void* dw_in, int64_t lddwi,
             void* dw_out, int64_t lddwo, int64_t M, int64_t D, int64_t F, int64_t N, int act,
             void* workspace, int64_t workspace_bytes, pgemm_stream_t stream) {
    const int rc = check_ffn(dtype, act, M, D, F, N);
    if (rc != PGEMM_OK) return rc;
    if (!dx && !dw_in && !dw_out) return PGEMM_OK;
    const Mat mdy = mat(dy, M, N, lddy), mx = mat(x, M, D, ldx), mwi = mat(w_in, D, 2 * F, ldwi),
              mwo = mat(w_out, F, N, ldwo), mgu = mat(gate_up, M, 2 * F, ldgu),
              ma = mat(add, M, D, ldadd), mdx = mat(dx, M, D, lddx),
              mdwi = mat(dw_in, D, 2 * F, lddwi), mdwo = mat(dw_out, F, N, lddwo);
    Outputs o;
    o.add(check(mdy, true));
    o.add(check(mx, dw_in != nullptr));
    o.add(check(mwi, dx != nullptr));
    o.add(check(mwo, true));
    o.add(check(mgu, true));
    for (const Mat* m : {&ma, &mdx, &mdwi, &mdwo}) o.add(check(*m, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* out : {&mdx, &mdwi, &mdwo}) {
        for (const Mat* in : {&mdy, &mx, &mwi, &mwo, &mgu}) o.apart(*out, *in);
        o.apart(*out, ma, out == &mdx);
    }
    o.apart(mdx, mdwi);
    o.apart(mdx, mdwo);
    o.apart(mdwi, mdwo);
    if (o.rc != PGEMM_OK) return o.rc;
    const FfnGradCall c = {dtype, dy, mdy.ld, x, mx.ld, w_in, mwi.ld, w_out, mwo.ld, gate_up,
                           mgu.ld, add, ma.ld, dx, mdx.ld, dw_in, mdwi.ld, dw_out, mdwo.ld,
                           M, D, F, N, act};
    const Mat all[] = {mdy, mx, mwi, mwo, mgu, ma, mdx, mdwi, mdwo};
    return with_workspace(
        [&](Arena& ar) { return ffn_backward(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 9);
}

int64_t pffn_bwd_workspace_bytes(int dtype, const void* dy, int64_t lddy, const void* x,
                                 int64_t ldx, const void* w_in, int64_t ldwi, const void* w_out,
                                 int64_t ldwo, int64_t M, int64_t D, int64_t F, int64_t N,
                                 int need_dx, int need_dw_in, int need_dw_out) {
    const int rc = check_ffn(dtype, PGEMM_ACT_NONE, M, D, F, N);
    if (rc != PGEMM_OK) return rc;
    if (!need_dx && !need_dw_in && !need_dw_out) return 0;
    const Mat mdy = mat(dy, M, N, lddy), mx = mat(x, M, D, ldx), mwi = mat(w_in, D, 2 * F, ldwi),
              mwo = mat(w_out, F, N, ldwo);
    Outputs o;
    o.add(check(mdy, true));
    o.add(check(mx, need_dw_in != 0));
    o.add(check(mwi, need_dx != 0));
    o.add(check(mwo, true));
    if (o.rc != PGEMM_OK) return o.rc;
    FfnGradCall c = {};
    void* const some = reinterpret_cast<void*>(16);  // stands for an output; never touched
    c.dtype = dtype;
    c.dy = dy, c.lddy = mdy.ld, c.x = x, c.ldx = mx.ld;
    c.w_in = w_in, c.ldwi = mwi.ld, c.w_out = w_out, c.ldwo = mwo.ld;
    c.dx = need_dx ? some : nullptr;
    c.dw_in = need_dw_in ? some : nullptr;
    c.dw_out = need_dw_out ? some : nullptr;
    c.M = M, c.D = D, c.F = F, c.N = N;
    Arena dry = {nullptr, 0};
    const hipError_t e = ffn_backward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int pxent(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw, const int64_t* target,
          int64_t ignore_index, int reduction, float* loss, float* lse, int64_t M, int64_t V,
          int64_t D, void* workspace, int64_t workspace_bytes, pgemm_stream_t stream) {
    const int rc = check_xent(dtype, reduction, M, V, D);
    if (rc != PGEMM_OK) return rc;
    const bool each = reduction == PGEMM_REDUCE_NONE;
    if (M == 0 && each) return PGEMM_OK;
    const Mat mx = mat(x, M, D, ldx), mw = mat(w, V, D, ldw), mt = flat(target, M, 8),
              ml = flat(loss, each ? M : 1, 4), ms = flat(lse, M, 4);
    Outputs o;
    o.add(check(mx, true));
    o.add(check(mw, true));
    o.add(check(mt, true));
    o.add(check(ml, true));
    o.add(check(ms, true));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* in : {&mx, &mw, &mt}) {
        o.apart(ml, *in);
        o.apart(ms, *in);
    }
    o.apart(ml, ms);
    if (o.rc != PGEMM_OK) return o.rc;
    const XentCall c = {dtype, x, mx.ld, w, mw.ld, target, ignore_index, reduction, loss, lse,
                        M, V, D};
    const Mat all[] = {mx, mw, mt, ml, ms};
    return with_workspace(
        [&](Arena& ar) { return xent_forward(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 5);
}

int64_t pxent_workspace_bytes(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              int reduction, int64_t M, int64_t V, int64_t D) {
    const int rc = check_xent(dtype, reduction, M, V, D);
    if (rc != PGEMM_OK) return rc;
    const Mat mx = mat(x, M, D, ldx), mw = mat(w, V, D, ldw);
    Outputs o;
    o.add(check(mx, true));
    o.add(check(mw, true));
    if (o.rc != PGEMM_OK) return o.rc;
    XentCall c = {};
    c.dtype = dtype;
    c.x = x, c.ldx = mx.ld, c.w = w, c.ldw = mw.ld, c.reduction = reduction;
    c.M = M, c.V = V, c.D = D;
    Arena dry = {nullptr, 0};
    const hipError_t e = xent_forward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int pxent_bwd(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
              const int64_t* target, int64_t ignore_index, int reduction, const float* lse,
              const float* dloss, void* dx, int64_t lddx, void* dw, int64_t lddw, int64_t M,
              int64_t V, int64_t D, void* workspace, int64_t workspace_bytes,
              pgemm_stream_t stream) {
    const int rc = check_xent(dtype, reduction, M, V, D);
    if (rc != PGEMM_OK) return rc;
    if (!dx && !dw) return PGEMM_OK;
    const bool each = reduction == PGEMM_REDUCE_NONE;
    const Mat mx = mat(x, M, D, ldx), mw = mat(w, V, D, ldw), mt = flat(target, M, 8),
              ms = flat(lse, M, 4), mg = flat(dloss, each ? M : 1, 4), mdx = mat(dx, M, D, lddx),
              mdw = mat(dw, V, D, lddw);
    Outputs o;
    o.add(check(mx, true));
    o.add(check(mw, true));
    o.add(check(mt, true));
    o.add(check(ms, true));
    o.add(check(mg, false));
    o.add(check(mdx, false));
    o.add(check(mdw, false));
    if (o.rc != PGEMM_OK) return o.rc;
    for (const Mat* in : {&mx, &mw, &mt, &ms, &mg}) {
        o.apart(mdx, *in);
        o.apart(mdw, *in);
    }
    o.apart(mdx, mdw);
    if (o.rc != PGEMM_OK) return o.rc;
    const XentGradCall c = {dtype, x, mx.ld, w, mw.ld, target, ignore_index, reduction, lse, dloss,
                            dx, mdx.ld, dw, mdw.ld, M, V, D};
    const Mat all[] = {mx, mw, mt, ms, mg, mdx, mdw};
    return with_workspace(
        [&](Arena& ar) { return xent_backward(c, ar, static_cast<hipStream_t>(stream)); }, workspace,
        workspace_bytes, all, 7);
}

int64_t pxent_bwd_workspace_bytes(int dtype, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                  int64_t M, int64_t V, int64_t D, int need_dx, int need_dw) {
    const int rc = check_xent(dtype, PGEMM_REDUCE_MEAN, M, V, D);
    if (rc != PGEMM_OK) return rc;
    if (!need_dx && !need_dw) return 0;
    const Mat mx = mat(x, M, D, ldx), mw = mat(w, V, D, ldw);
    Outputs o;
    o.add(check(mx, true));
    o.add(check(mw, true));
    if (o.rc != PGEMM_OK) return o.rc;
    XentGradCall c = {};
    void* const some = reinterpret_cast<void*>(16);  // stands for an output; never touched
    c.dtype = dtype;
    c.x = x, c.ldx = mx.ld, c.w = w, c.ldw = mw.ld;
    c.dx = need_dx ? some : nullptr;
    c.dw = need_dw ? some : nullptr;
    c.M = M, c.V = V, c.D = D;
    Arena dry = {nullptr, 0};
    const hipError_t e = xent_backward(c, dry, nullptr);
    return e == hipSuccess ? dry.used : hip_status(e);
}

int64_t pclip_grad_norm_workspace_bytes(int64_t count) {
    if (count < 0) return PGEMM_EINVAL;
    return clip_workspace_bytes(count);
}

int pclip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes,
                    const int* dtypes, int64_t count, float max_norm, float* norm, void* workspace,
                    int64_t workspace_bytes, pgemm_stream_t stream) {
    if (count < 0 || !norm || !(max_norm >= 0.0f)) return PGEMM_EINVAL;
    if (count > 0 && (!grads || !sizes || !dtypes)) return PGEMM_EINVAL;
    if (count > kMaxTensors || reinterpret_cast<uintptr_t>(norm) % 4) return PGEMM_EUNSUPPORTED;
    const int64_t need = clip_workspace_bytes(count);
    if (!workspace || workspace_bytes < need) return PGEMM_EINVAL;
    if (!aligned16(workspace)) return PGEMM_EUNSUPPORTED;
    // Every byte range of the call, to be sorted by address: written ranges
    // (outputs, norm, workspace) may meet no other, but for an output that is
    // its own gradient, which counts once.
    std::unique_ptr<Range[]> ranges(new (std::nothrow) Range[2 * count + 2]);
    if (!ranges) return hip_status(hipErrorOutOfMemory);
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t size = sizes[i];
        if (size < 0) return PGEMM_EINVAL;
        if (dtypes[i] != PGEMM_F16 && dtypes[i] != PGEMM_BF16 && dtypes[i] != PGEMM_F32)
            return PGEMM_EUNSUPPORTED;
        if (size == 0) continue;
        if (size > kMaxTensorElems) return PGEMM_EUNSUPPORTED;
        const void* in = grads[i];
        const void* out = outs ? outs[i] : in;
        if (!in || !out) return PGEMM_EINVAL;
        const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
        const int bytes = dtypes[i] == PGEMM_F32 ? 4 : 2;
        if (a % bytes || b % bytes) return PGEMM_EUNSUPPORTED;
        if (a != b) ranges[n++] = {a, a + (uintptr_t)(size * bytes), false};
        ranges[n++] = {b, b + (uintptr_t)(size * bytes), true};
    }
    const uintptr_t nb = reinterpret_cast<uintptr_t>(norm), wb = reinterpret_cast<uintptr_t>(workspace);
    ranges[n++] = {nb, nb + 4, true};
    ranges[n++] = {wb, wb + (uintptr_t)need, true};
    std::sort(ranges.get(), ranges.get() + n,
              [](const Range& u, const Range& v) { return u.begin < v.begin; });
    uintptr_t any = 0, written = 0;  // furthest ends so far
    for (int64_t i = 0; i < n; ++i) {
        if (ranges[i].begin < (ranges[i].writes ? any : written)) return PGEMM_EINVAL;
        any = std::max(any, ranges[i].end);
        if (ranges[i].writes) written = std::max(written, ranges[i].end);
    }
    const ClipCall c = {grads, outs, sizes, dtypes, count, (double)max_norm, norm};
    return hip_status(clip(c, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
