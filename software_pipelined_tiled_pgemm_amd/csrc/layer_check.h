// Argument checks shared by the C entry points of the layer operators
// (layer_api.hip) and of the serving operators (serving_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pgemm.h"
#include "layer.h"

namespace pgemm {
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

inline Mat mat(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {p, rows, cols, rows > 1 ? ld : cols, 2};
}
inline Mat flat(const void* p, int64_t n, int bytes) { return {p, 1, n, n, bytes}; }

// Status of a matrix's own description; `needed`: it must not be NULL unless
// it is empty.
inline int check(const Mat& m, bool needed) {
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
inline bool shares(const Mat& a, const Mat& b) {
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

inline int hip_status(hipError_t e) { return pgemm::record_hip_status(e); }

inline bool known(int dtype, int act) {
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

}  // namespace
}  // namespace pgemm
