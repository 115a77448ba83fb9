// Sampling tokens from rows of logits, with given random numbers.
//
// In descending order of the logits (equal ones by index), with weights w =
// exp((l - max) / temperature) and W(j) their sum up to the j-th:
//   top-k   keeps the first k,             sum Zk = W(k)
//   top-p   keeps up to the first j with W(j) >= p Zk,  sum Zp = W(j)
//   min-p   keeps those with w >= min_p,   sum Zm
// All three keep a beginning of the same order, so together they keep the one
// with the smallest sum Z, and the token is the first j with W(j) > u Z.  So
// every step is one kind of search: the first j whose running sum (of weights, or
// of ones) reaches a given value.
//
// Weights are whole numbers, exp(..) 2^40 rounded, and their sums (below 2^62)
// exact: they do not depend on the order of the additions, and two tokens
// are told apart by less than 2^-40 of the largest weight.  (With fp32 sums a
// row of 10^5 tokens gives another token than the definition for one u in about a
// hundred.)
//
// The search: a histogram of counts and sums over bins of 1/64 in (max - l) /
// temperature, in LDS; the bin that holds the wanted place is gathered and its
// elements ranked by comparison with each other.  A bin of more elements than
// the list takes is cut into bins of its own, down to equal logits, which are
// taken by index.
#include "sample.h"

#include "layer_math.h"

namespace pgemm {
namespace layer {
namespace {

struct F32 {};  // logits of 32 bits

template <class E>
struct Logits {
    static constexpr int kWidth = 8;  // logits of 16 bytes
    typedef uint16_t Bits;
    __device__ static __forceinline__ float get(uint16_t b) { return E::get(b); }
};
template <>
struct Logits<F32> {
    static constexpr int kWidth = 4;
    typedef uint32_t Bits;
    __device__ static __forceinline__ float get(uint32_t b) { return __builtin_bit_cast(float, b); }
};

constexpr int kT = 1024;       // lanes of a row's workgroup
constexpr int kBins = 2048;    // bins of a histogram
constexpr int kList = 1024;    // elements that are ranked at once
constexpr float kPerUnit = 64.0f;  // bins per unit of (max - l) / temperature
constexpr double kOne = 1099511627776.0;  // 2^40, the largest weight

typedef unsigned long long u64;

struct Histogram {
    u64 sum[kBins];
    uint32_t count[kBins];
};

// What a search found: the sum of the weights up to and with the element, its
// index and its logit.
struct Found {
    u64 sum;
    int64_t index;
    float logit;
};

struct Shared {
    Histogram all, part;
    float logit[kList];
    uint32_t index[kList];
    u64 weight[kList];
    u64 wave_sum[kT / 64];
    uint32_t wave_count[kT / 64];
    float wave_min[kT / 64], wave_max[kT / 64];
    int flag;
    uint32_t listed;
    int bin;
    u64 before_sum, before_count;
    Found found;
};

// A row's logits and what its weights are made with.
template <class E>
struct Row {
    typedef Logits<E> L;
    const typename L::Bits* ptr;
    int V;
    float most;
    double inverse;  // 1 / temperature
    float per;       // bins per unit of max - l

    // f(index, logit) for this lane's elements.
    template <class Fn>
    __device__ __forceinline__ void each(Fn&& f) const {
        for (int64_t c = (int64_t)threadIdx.x * L::kWidth; c < V; c += kT * L::kWidth) {
            typename L::Bits b[L::kWidth];
            if (c + L::kWidth <= V) {
                __builtin_memcpy(b, ptr + c, 16);
#pragma unroll
                for (int q = 0; q < L::kWidth; ++q) f((int)c + q, L::get(b[q]));
            } else {
                for (int q = 0; c + q < V; ++q) f((int)c + q, L::get(ptr[c + q]));
            }
        }
    }
    // exp((l - max) / temperature); 0 where it is below 2^-41.
    __device__ __forceinline__ double weight(float l) const {
        if (l == most) return 1.0;
        const double x = ((double)l - (double)most) * inverse;
        return x > -28.5 ? exp(x) : 0.0;  // NaN (a masked logit, no temperature): 0
    }
    __device__ __forceinline__ int bin(float l) const {
        return l == most ? 0 : (int)fminf((most - l) * per, (float)(kBins - 1));
    }
};
__device__ __forceinline__ u64 whole(double w) { return (u64)__builtin_rint(w * kOne); }

template <class V, class Op>
__device__ __forceinline__ V over_block(V v, V* slots, Op op) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = op(v, __shfl_xor(v, o, 64));
    __syncthreads();  // the slots' last readers are done
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < kT / 64; ++i) v = op(v, slots[i]);
    return v;
}

__device__ __forceinline__ void clear(Histogram& h) {
    for (int i = threadIdx.x; i < kBins; i += kT) {
        h.sum[i] = 0;
        h.count[i] = 0;
    }
}

// The bin in which the running sum (by_count: count) first reaches `goal`, and
// what comes before it: s.bin, s.before_sum, s.before_count.  Bins run in
// descending order of the logits.
__device__ __forceinline__ void find_bin(Shared& s, const Histogram& h, bool by_count, u64 goal,
                                         u64 sum0, u64 count0) {
    constexpr int PER = kBins / kT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 sum = 0;
    uint32_t count = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        sum += h.sum[threadIdx.x * PER + i];
        count += h.count[threadIdx.x * PER + i];
    }
    u64 sums = sum;
    uint32_t counts = count;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const u64 a = __shfl_up(sums, o, 64);
        const uint32_t b = __shfl_up(counts, o, 64);
        if (lane >= o) {
            sums += a;
            counts += b;
        }
    }
    __syncthreads();
    if (lane == 63) {
        s.wave_sum[wave] = sums;
        s.wave_count[wave] = counts;
    }
    __syncthreads();
    u64 bs = sum0 + sums - sum, bc = count0 + counts - count;
    for (int i = 0; i < wave; ++i) {
        bs += s.wave_sum[i];
        bc += s.wave_count[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const u64 hs = h.sum[threadIdx.x * PER + i];
        const uint32_t hc = h.count[threadIdx.x * PER + i];
        const u64 before = by_count ? bc : bs, own = by_count ? hc : hs;
        if (before < goal && goal <= before + own) {
            s.bin = threadIdx.x * PER + i;
            s.before_sum = bs;
            s.before_count = bc;
        }
        bs += hs;
        bc += hc;
    }
    __syncthreads();
}

// The first element, in the order, at which the running sum (by_count: count)
// reaches `goal`, which lies between 1 and the whole row's.
template <class E>
__device__ __forceinline__ void search(Shared& s, const Row<E>& row, bool by_count, u64 goal) {
    find_bin(s, s.all, by_count, goal, 0, 0);
    const int bin = s.bin;
    u64 before_sum = s.before_sum, before_count = s.before_count;
    uint32_t count = s.all.count[bin];
    // The elements looked at: those of the bin, then those of lo <= l <= hi.
    float lo = 0.0f, hi = 0.0f;
    bool ranged = false;
    auto in = [&](float l) __attribute__((always_inline)) {
        if (ranged) return l >= lo && l <= hi;
        // a bin far out may hold logits without weight, which do not count
        return row.bin(l) == bin && (bin < kBins * 7 / 8 || whole(row.weight(l)) != 0);
    };
    // fp32's range holds 278 doublings, and a pass takes off almost 11: the bound
    // is never reached.
    for (int pass = 0; pass < 40 && count > kList; ++pass) {
        float least = INFINITY, top = -INFINITY;
        row.each([&](int, float l) __attribute__((always_inline)) {
            if (in(l)) {
                least = fminf(least, l);
                top = fmaxf(top, l);
            }
        });
        least = over_block(least, s.wave_min, [](float a, float b) { return fminf(a, b); });
        top = over_block(top, s.wave_max, [](float a, float b) { return fmaxf(a, b); });
        lo = least, hi = top;
        ranged = true;
        if (lo == hi) break;
        // 2048 bins over hi - lo, in binary64, where the difference of two logits,
        // its reciprocal and their products neither vanish nor overflow: hi goes
        // to bin 0 and lo to one of the last two, so that every pass leaves out
        // one of them at least (and all but about 1/2047 of the range).
        const double scale = (double)(kBins - 1) / ((double)hi - (double)lo);
        auto sub = [&](float l) __attribute__((always_inline)) {
            return (int)fmin(((double)hi - (double)l) * scale, (double)(kBins - 1));
        };
        __syncthreads();
        clear(s.part);
        __syncthreads();
        row.each([&](int, float l) __attribute__((always_inline)) {
            if (l >= lo && l <= hi) {
                const int b = sub(l);
                atomicAdd(&s.part.sum[b], whole(row.weight(l)));
                atomicAdd(&s.part.count[b], 1u);
            }
        });
        __syncthreads();
        find_bin(s, s.part, by_count, goal, before_sum, before_count);
        before_sum = s.before_sum, before_count = s.before_count;
        count = s.part.count[s.bin];
        // the ends of that bin's logits
        const int want = s.bin;
        least = INFINITY, top = -INFINITY;
        row.each([&](int, float l) __attribute__((always_inline)) {
            if (l >= lo && l <= hi && sub(l) == want) {
                least = fminf(least, l);
                top = fmaxf(top, l);
            }
        });
        lo = over_block(least, s.wave_min, [](float a, float b) { return fminf(a, b); });
        hi = over_block(top, s.wave_max, [](float a, float b) { return fmaxf(a, b); });
        if (lo == hi) break;
    }
    __syncthreads();
    if (count > kList) {
        // `count` equal logits: the r-th of them by index.
        const u64 w = whole(row.weight(lo));
        const u64 r = by_count ? goal - before_count : (goal - before_sum + w - 1) / w;
        // Lane t looks at the t-th stretch of the row.
        const int64_t per = ((int64_t)row.V + kT - 1) / kT;
        const int64_t i0 = threadIdx.x * per, i1 = min(i0 + per, (int64_t)row.V);
        uint32_t mine = 0;
        for (int64_t i = i0; i < i1; ++i) mine += Logits<E>::get(row.ptr[i]) == lo;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t b = __shfl_up(upto, o, 64);
            if (lane >= o) upto += b;
        }
        if (lane == 63) s.wave_count[wave] = upto;
        __syncthreads();
        u64 n = upto - mine;
        for (int i = 0; i < wave; ++i) n += s.wave_count[i];
        if (n < r && r <= n + mine)
            for (int64_t i = i0; i < i1; ++i)
                if (Logits<E>::get(row.ptr[i]) == lo && ++n == r) {
                    s.found.sum = before_sum + r * w;
                    s.found.index = i;
                    s.found.logit = lo;
                }
        __syncthreads();
        return;
    }
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    row.each([&](int i, float l) __attribute__((always_inline)) {
        if (in(l)) {
            const uint32_t at = atomicAdd(&s.listed, 1u);
            if (at < kList) {
                s.logit[at] = l;
                s.index[at] = (uint32_t)i;
                s.weight[at] = whole(row.weight(l));
            }
        }
    });
    __syncthreads();
    if (threadIdx.x < count) {
        const float l = s.logit[threadIdx.x];
        const uint32_t i = s.index[threadIdx.x];
        u64 bs = before_sum, bc = before_count;
        for (uint32_t j = 0; j < count; ++j) {
            const float lj = s.logit[j];
            if (lj > l || (lj == l && s.index[j] < i)) {
                bs += s.weight[j];
                ++bc;
            }
        }
        const u64 w = s.weight[threadIdx.x];
        const u64 before = by_count ? bc : bs, own = by_count ? 1 : w;
        if (before < goal && goal <= before + own) {
            s.found.sum = bs + w;
            s.found.index = i;
            s.found.logit = l;
        }
    }
    __syncthreads();
}

// The least sum that is at least `goal`, or (beyond) above it, between 1 (also for
// NaN) and Z.
__device__ __forceinline__ u64 least_sum(double goal, bool beyond, u64 Z) {
    if (goal >= (double)Z) return Z;
    if (!(goal > 0.0)) return 1;
    // (added as whole numbers: a goal beyond 2^53 has no room for the 1)
    return min(beyond ? (u64)goal + 1 : (u64)ceil(goal), Z);
}

template <class V>
__device__ __forceinline__ V at(const Setting<V>& s, int64_t row) {
    return s.each ? s.each[row] : s.value;
}

template <class E>
__global__ __launch_bounds__(kT) void sample_kernel(
    const typename Logits<E>::Bits* __restrict__ logits, int64_t ld, const float* __restrict__ u,
    const Setting<float> temperature, const Setting<float> top_p, const Setting<float> min_p,
    const Setting<int32_t> top_k, int64_t* __restrict__ tokens, float* __restrict__ logprobs,
    int64_t M, int V) {
    __shared__ Shared s;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        Row<E> row = {logits + m * ld, V, 0.0f, 0.0, 0.0f};
        // The largest logit, and whether there is a NaN.
        float most = -INFINITY;
        int bad = 0;
        row.each([&](int, float l) __attribute__((always_inline)) {
            most = fmaxf(most, l);
            bad |= l != l;
        });
        __syncthreads();  // the row before is done
        if (threadIdx.x == 0) s.flag = 0;
        clear(s.all);
        most = over_block(most, s.wave_max, [](float a, float b) { return fmaxf(a, b); });
        if (bad) s.flag = 1;
        __syncthreads();
        if (s.flag || most == -INFINITY) {
            if (threadIdx.x == 0) {
                tokens[m] = -1;
                if (logprobs) logprobs[m] = __builtin_nanf("");
            }
            continue;
        }
        const float t = at(temperature, m);
        row.most = most;
        if (!(t > 0.0f)) {
            // Greedy: the first of the largest.
            uint32_t first = 0xFFFFFFFFu;
            row.each([&](int i, float l) __attribute__((always_inline)) {
                if (l == most) first = min(first, (uint32_t)i);
            });
            first = over_block(first, s.wave_count,
                               [](uint32_t a, uint32_t b) { return a < b ? a : b; });
            if (threadIdx.x == 0) {
                tokens[m] = first;
                if (logprobs) logprobs[m] = 0.0f;
            }
            continue;
        }
        row.inverse = 1.0 / (double)t;
        row.per = kPerUnit / t;
        // The histogram; the sum of what min-p keeps.
        const float least = at(min_p, m);
        const double bound = least > 0.0f ? fmin((double)least, 1.0) : 0.0;
        u64 kept = 0;
        row.each([&](int, float l) __attribute__((always_inline)) {
            const double e = row.weight(l);
            const u64 w = whole(e);
            if (w != 0) {
                const int b = row.bin(l);
                atomicAdd(&s.all.sum[b], w);
                atomicAdd(&s.all.count[b], 1u);
                if (e >= bound) kept += w;
            }
        });
        __syncthreads();
        u64 total = 0;
        uint32_t n = 0;
        for (int i = threadIdx.x; i < kBins; i += kT) {
            total += s.all.sum[i];
            n += s.all.count[i];
        }
        auto add = [](auto a, auto b) { return a + b; };
        kept = over_block(kept, s.wave_sum, add);
        total = over_block(total, s.wave_sum, add);
        n = over_block(n, s.wave_count, add);
        u64 Z = total;
        const int32_t k = at(top_k, m);
        if (k > 0 && (uint32_t)k < n) {
            search(s, row, true, (u64)k);
            Z = s.found.sum;
        }
        const float p = at(top_p, m);
        if (p < 1.0f) {
            search(s, row, false, least_sum((double)p * (double)Z, false, Z));
            Z = min(Z, s.found.sum);
        }
        Z = min(Z, kept);
        search(s, row, false, least_sum((double)u[m] * (double)Z, true, Z));
        if (threadIdx.x == 0) {
            tokens[m] = s.found.index;
            if (logprobs) {
                const double x = s.found.logit == most
                                     ? 0.0
                                     : ((double)s.found.logit - (double)most) * row.inverse;
                logprobs[m] = (float)(x - log((double)Z / kOne));
            }
        }
    }
}

template <class E>
hipError_t launch(const SampleCall& c, hipStream_t stream) {
    const unsigned blocks = (unsigned)(c.M < (1 << 20) ? c.M : 1 << 20);
    hipLaunchKernelGGL(sample_kernel<E>, dim3(blocks), dim3(kT), 0, stream,
                       static_cast<const typename Logits<E>::Bits*>(c.logits), c.ld, c.u,
                       c.temperature, c.top_p, c.min_p, c.top_k, c.tokens, c.logprobs, c.M,
                       (int)c.V);
    return hipGetLastError();
}

}  // namespace

hipError_t sample(const SampleCall& c, Arena& ar, hipStream_t stream) {
    if (ar.dry() || c.M == 0) return hipSuccess;
    if (c.dtype == PGEMM_F32) return launch<F32>(c, stream);
    return c.dtype == PGEMM_BF16 ? launch<BF16>(c, stream) : launch<F16>(c, stream);
}

}  // namespace layer
}  // namespace pgemm
