// The call of gradient clipping, as the C entry point hands it on (validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pgemm {
namespace layer {

struct ClipCall {
    const void* const* grads;  // host arrays of `count`
    void* const* outs;         // NULL: in place
    const int64_t* sizes;
    const int* dtypes;
    int64_t count;
    double max_norm;
    float* norm;
};

int64_t clip_workspace_bytes(int64_t count);
hipError_t clip(const ClipCall& c, void* workspace, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
