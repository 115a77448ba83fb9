// Sampling calls, as the C entry point hands them on (validated).
#pragma once

#include "layer.h"

namespace pgemm {
namespace layer {

// One number for every row, or (each not NULL) one of each row on the device.
template <class V>
struct Setting {
    V value;
    const V* each;
};

struct SampleCall {
    int dtype;  // f16, bf16 or f32 (enum pgemm_dtype)
    const void* logits;
    int64_t ld;
    const float* u;
    Setting<float> temperature, top_p, min_p;
    Setting<int32_t> top_k;
    int64_t* tokens;
    float* logprobs;
    int64_t M, V;
};
// With a dry arena nothing is launched and only the workspace is counted.
hipError_t sample(const SampleCall& c, Arena& ar, hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
