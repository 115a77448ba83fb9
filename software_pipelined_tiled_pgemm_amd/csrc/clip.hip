// Gradient clipping by the global norm over many tensors.
//
//   norm = sqrt(sum over all tensors of sum of g^2)
//   g' = g * min(1, max_norm / (norm + 1e-6))
//
// Three kinds of launches: partial sums of squares (a table of up to
// kTensors tensors travels in the kernel's arguments, cut into chunks that
// the workgroups walk), one workgroup that adds the partials and derives the
// factor, and the scaling over the same chunks.  Bound by memory: two reads
// and one write of every gradient.  The scaling walks the chunks backwards,
// so that what the first pass read last is read again first, while it is
// still in the last-level cache.
//
// Squares: fp16 ones are exact in fp32, where 8 of them are added (rounding by
// at most 7 2^-24 of the sum) before joining an fp64 sum; bf16 and fp32 values are
// squared in fp64, where none overflows or vanishes.  The order of all sums is
// fixed.  7e8 bf16 values: 826 us (4.2 GB, 5.1 TB/s; with stores through the
// caches 898); 60 tensors of 2^20 fp32 values in all: 12.5 us of kernels.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/pgemm.h"
#include "clip.h"
#include "layer_math.h"

namespace pgemm {
namespace layer {
namespace {

constexpr int kThreads = 256;
constexpr int kTensors = 112;
constexpr int kBlocks = 2048;  // most workgroups of a launch: 8 per CU

struct Table {
    const void* in[kTensors];
    void* out[kTensors];
    int64_t n[kTensors];
    int end[kTensors];  // chunks up to and including this tensor's last
    uint8_t dtype[kTensors];
    int count;
    int chunk;  // elements, a multiple of 8 * kThreads
};
static_assert(sizeof(Table) + 64 <= 4096, "kernel argument size");

// Tensor of a chunk, and the chunk's index in it.
__device__ __forceinline__ int locate(const Table& t, int chunk, int& index) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (chunk < t.end[mid])
            hi = mid;
        else
            lo = mid + 1;
    }
    index = chunk - (lo > 0 ? t.end[lo - 1] : 0);
    return lo;
}

// Loads and stores of 8 values from any element-aligned address (the
// compiler's unaligned 16-byte accesses); stores go past the caches.
typedef u4_t u4_any __attribute__((aligned(2)));
__device__ __forceinline__ u4_t get16(const void* p) {
    const u4_any* q = static_cast<const u4_any*>(p);
    return *q;
}
__device__ __forceinline__ void put16(void* p, u4_t w) {
    __builtin_nontemporal_store(w, static_cast<u4_any*>(p));
}
template <class E>
struct Vec8 {
    typedef uint16_t elem;
    __device__ static __forceinline__ void load(const elem* p, float (&v)[8]) {
        const u4_t w = get16(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = E::get((uint16_t)w[q]);
            v[2 * q + 1] = E::get((uint16_t)(w[q] >> 16));
        }
    }
    __device__ static __forceinline__ void store(elem* p, const float (&v)[8]) {
        const u4_t w = {E::put2(v[0], v[1]), E::put2(v[2], v[3]), E::put2(v[4], v[5]),
                        E::put2(v[6], v[7])};
        put16(p, w);
    }
    __device__ static __forceinline__ float get(const elem* p) { return E::get(*p); }
    __device__ static __forceinline__ void put(elem* p, float v) { *p = E::put(v); }
};
struct F32 {};
template <>
struct Vec8<F32> {
    typedef float elem;
    __device__ static __forceinline__ void load(const elem* p, float (&v)[8]) {
        const u4_t lo = get16(p), hi = get16(p + 4);
        __builtin_memcpy(v, &lo, 16);
        __builtin_memcpy(v + 4, &hi, 16);
    }
    __device__ static __forceinline__ void store(elem* p, const float (&v)[8]) {
        u4_t lo, hi;
        __builtin_memcpy(&lo, v, 16);
        __builtin_memcpy(&hi, v + 4, 16);
        put16(p, lo);
        put16(p + 4, hi);
    }
    __device__ static __forceinline__ float get(const elem* p) { return *p; }
    __device__ static __forceinline__ void put(elem* p, float v) { *p = v; }
};

template <class E>
__device__ __forceinline__ double squares(const float (&v)[8]) {
    if constexpr (std::is_same<E, F16>::value) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s = fmaf(v[q], v[q], s);
        return (double)s;
    } else {
        double s = 0.0;
#pragma unroll
        for (int q = 0; q < 8; ++q) s = fma((double)v[q], (double)v[q], s);
        return s;
    }
}

template <class E>
__device__ __forceinline__ double chunk_squares(const void* in, int64_t from, int64_t to) {
    const typename Vec8<E>::elem* p = static_cast<const typename Vec8<E>::elem*>(in);
    double s = 0.0;
    int64_t i = from + threadIdx.x * 8;
    for (; i + 3 * 8 * kThreads + 8 <= to; i += 4 * 8 * kThreads) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) Vec8<E>::load(p + i + u * 8 * kThreads, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) s += squares<E>(v[u]);
    }
    for (; i < to; i += 8 * kThreads) {
        float v[8];
        if (i + 8 <= to) {
            Vec8<E>::load(p + i, v);
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = i + q < to ? Vec8<E>::get(p + i + q) : 0.0f;
        }
        s += squares<E>(v);
    }
    return s;
}

__global__ __launch_bounds__(kThreads) void squares_kernel(const Table t, double* __restrict__ part) {
    const int chunks = t.end[t.count - 1];
    double s = 0.0;
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        int index;
        const int k = locate(t, c, index);
        const int64_t from = (int64_t)index * t.chunk;
        const int64_t to = from + t.chunk < t.n[k] ? from + t.chunk : t.n[k];
        if (t.dtype[k] == PGEMM_F16)
            s += chunk_squares<F16>(t.in[k], from, to);
        else if (t.dtype[k] == PGEMM_BF16)
            s += chunk_squares<BF16>(t.in[k], from, to);
        else
            s += chunk_squares<F32>(t.in[k], from, to);
    }
    __shared__ double sums[kThreads];
    sums[threadIdx.x] = s;
    for (int h = kThreads / 2; h > 0; h >>= 1) {
        __syncthreads();
        if (threadIdx.x < h) sums[threadIdx.x] += sums[threadIdx.x + h];
    }
    if (threadIdx.x == 0) part[blockIdx.x] = sums[0];
}

// norm and the factor, from the partials of every launch.
__global__ __launch_bounds__(1024) void norm_kernel(const double* __restrict__ part, int64_t parts,
                                                    double max_norm, float* __restrict__ norm,
                                                    float* __restrict__ factor) {
    __shared__ double sums[1024];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += 1024) s += part[i];
    sums[threadIdx.x] = s;
    for (int h = 512; h > 0; h >>= 1) {
        __syncthreads();
        if (threadIdx.x < h) sums[threadIdx.x] += sums[threadIdx.x + h];
    }
    if (threadIdx.x == 0) {
        const double n = sqrt(sums[0]);
        const double f = max_norm / (n + 1e-6);
        norm[0] = (float)n;
        factor[0] = f > 1.0 ? 1.0f : (float)f;  // a NaN norm gives a NaN factor
    }
}

template <class E>
__device__ __forceinline__ void chunk_scale(const void* in, void* out, int64_t from, int64_t to,
                                            float f) {
    typedef typename Vec8<E>::elem elem;
    const elem* p = static_cast<const elem*>(in);
    elem* o = static_cast<elem*>(out);
    int64_t i = from + threadIdx.x * 8;
    for (; i + 3 * 8 * kThreads + 8 <= to; i += 4 * 8 * kThreads) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) Vec8<E>::load(p + i + u * 8 * kThreads, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[u][q] *= f;
            Vec8<E>::store(o + i + u * 8 * kThreads, v[u]);
        }
    }
    for (; i < to; i += 8 * kThreads) {
        if (i + 8 <= to) {
            float v[8];
            Vec8<E>::load(p + i, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] *= f;
            Vec8<E>::store(o + i, v);
        } else {
            for (int64_t j = i; j < to; ++j) Vec8<E>::put(o + j, Vec8<E>::get(p + j) * f);
        }
    }
}

__global__ __launch_bounds__(kThreads) void scale_kernel(const Table t,
                                                         const float* __restrict__ factor) {
    const float f = factor[0];
    const int chunks = t.end[t.count - 1];
    for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
        int index;
        const int k = locate(t, c, index);
        if (f == 1.0f && t.in[k] == t.out[k]) continue;  // in place, nothing to scale
        const int64_t from = (int64_t)index * t.chunk;
        const int64_t to = from + t.chunk < t.n[k] ? from + t.chunk : t.n[k];
        if (t.dtype[k] == PGEMM_F16)
            chunk_scale<F16>(t.in[k], t.out[k], from, to, f);
        else if (t.dtype[k] == PGEMM_BF16)
            chunk_scale<BF16>(t.in[k], t.out[k], from, to, f);
        else
            chunk_scale<F32>(t.in[k], t.out[k], from, to, f);
    }
}

}  // namespace

int64_t clip_workspace_bytes(int64_t count) {
    return 256 + (count + kTensors - 1) / kTensors * kBlocks * (int64_t)sizeof(double);
}

hipError_t clip(const ClipCall& c, void* workspace, hipStream_t stream) {
    float* const factor = static_cast<float*>(workspace);
    double* const part = reinterpret_cast<double*>(static_cast<char*>(workspace) + 256);
    // Short lists in short chunks, so that they spread over the CUs.
    int64_t total = 0;
    for (int64_t i = 0; i < c.count; ++i) total += c.sizes[i];
    const int chunk = total < ((int64_t)1 << 24) ? 4096 : 32768;
    Table t;
    t.chunk = chunk;
    int64_t parts = 0;
    hipError_t rc = hipSuccess;
    // Runs `f` on each table of the list, forwards or backwards; empty
    // tensors are left out.
    auto tables = [&](bool backwards, auto&& f) {
        const int64_t groups = (c.count + kTensors - 1) / kTensors;
        for (int64_t k = 0; k < groups && rc == hipSuccess; ++k) {
            const int64_t first = (backwards ? groups - 1 - k : k) * kTensors;
            const int64_t last = std::min<int64_t>(c.count, first + kTensors);
            int64_t chunks = 0;
            t.count = 0;
            for (int64_t i = first; i < last; ++i) {
                if (c.sizes[i] == 0) continue;
                chunks += (c.sizes[i] + chunk - 1) / chunk;
                t.in[t.count] = c.grads[i];
                t.out[t.count] = c.outs ? c.outs[i] : const_cast<void*>(c.grads[i]);
                t.n[t.count] = c.sizes[i];
                t.dtype[t.count] = (uint8_t)c.dtypes[i];
                t.end[t.count++] = (int)chunks;
            }
            if (t.count > 0) {
                f((unsigned)std::min<int64_t>(chunks, kBlocks));
                rc = hipGetLastError();
            }
        }
    };
    tables(false, [&](unsigned grid) {
        hipLaunchKernelGGL(squares_kernel, dim3(grid), dim3(kThreads), 0, stream, t, part + parts);
        parts += grid;
    });
    if (rc != hipSuccess) return rc;
    hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(1024), 0, stream, part, parts, c.max_norm, c.norm,
                       factor);
    if ((rc = hipGetLastError()) != hipSuccess) return rc;
    tables(true, [&](unsigned grid) {
        hipLaunchKernelGGL(scale_kernel, dim3(grid), dim3(kThreads), 0, stream, t, factor);
    });
    return rc;
}

}  // namespace layer
}  // namespace pgemm
