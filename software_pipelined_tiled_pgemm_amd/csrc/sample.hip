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
// The search: a histogram over bins of 1/64 in (max - l) / temperature, in LDS;
// the bins that hold the wanted places are gathered and sorted.  Three ways:
//  - up to 512 kept by top-k (the usual case): counts alone find the bin of the
//    k-th; everything up to it is gathered, weighed and sorted.  No other
//    logit is weighed.
//  - no top-k: sums of the weights; the bin where top-p ends and those where the
//    token may lie are gathered and sorted.
//  - more than 512, or more elements in those bins than the list takes (many
//    logits next to each other): one search after the other, each cutting its
//    bin into bins of its own until the list takes what is left, down to equal
//    logits, which are taken by index.
// A row is kept in LDS where it fits; few long rows are cut into pieces, a workgroup
// each, with the histogram and the list in the workspace.  Long rows of 16 bits
// go another way, by a counter for each of the 65536 patterns.
#include "sample.h"

#include <type_traits>

#include "layer_math.h"

namespace pgemm {
namespace layer {
namespace {

struct F32 {};  // logits of 32 bits

// Logits as whole numbers of the same order (-0 as 0), and back.
__device__ __forceinline__ uint32_t order_of(float l) {
    const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float logit_in_order(uint32_t o) {
    return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Pieces of 16 bytes; the largest and the smallest of many pieces, as whole numbers
// in the logits' order, two at a time in 16 bits (NaN come out beyond the
// infinities).
typedef int16_t s2_t __attribute__((ext_vector_type(2)));
template <class E>
struct Logits {
    static constexpr int kWidth = 8;  // logits of 16 bytes
    typedef uint16_t Bits;
    __device__ static __forceinline__ float get(uint16_t b) { return E::get(b); }
    static constexpr bool kBrain = std::is_same<E, BF16>::value;
    static constexpr uint32_t kLeast = kBrain ? 0xFF80FF80u : 0xFC00FC00u;  // -infinity, twice
    struct Ends {
        static constexpr int16_t kTop = (int16_t)((uint16_t)kLeast ^ 0x7FFF),
                                 kLow = (int16_t)((uint16_t)kLeast & 0x7FFF);  // +- infinity
        s2_t top = {kTop, kTop}, low = {kLow, kLow};
        __device__ __forceinline__ void add(u4_t w) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t word = w[q];  // (a bit_cast of an element takes element 0)
                const s2_t b = __builtin_bit_cast(s2_t, word);
                const s2_t flip = (b >> 15) & 0x7FFF;
                top = __builtin_elementwise_max(top, (s2_t)(b ^ flip));
                low = __builtin_elementwise_min(low, (s2_t)(b ^ flip));
            }
        }
        __device__ static __forceinline__ float value(int v) {
            return E::get((uint16_t)(v < 0 ? v ^ 0x7FFF : v));
        }
        // The largest as order_of() has it; a NaN's is above all.
        __device__ __forceinline__ uint32_t order() const {
            const float most = value(max(top[0], top[1])), least = value(min(low[0], low[1]));
            return most != most || least != least ? 0xFFFFFFFFu : order_of(most);
        }
    };
};
template <>
struct Logits<F32> {
    static constexpr int kWidth = 4;
    typedef uint32_t Bits;
    __device__ static __forceinline__ float get(uint32_t b) { return __builtin_bit_cast(float, b); }
    static constexpr uint32_t kLeast = 0xFF800000u;
    struct Ends {
        int top = (int)(kLeast ^ 0x7FFFFFFFu), low = (int)(kLeast & 0x7FFFFFFFu);
        __device__ __forceinline__ void add(u4_t w) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int b = (int)w[q], v = b ^ ((b >> 31) & 0x7FFFFFFF);
                top = max(top, v);
                low = min(low, v);
            }
        }
        __device__ static __forceinline__ float value(int v) {
            return __builtin_bit_cast(float, v < 0 ? v ^ 0x7FFFFFFF : v);
        }
        __device__ __forceinline__ uint32_t order() const {
            const float most = value(top), least = value(low);
            return most != most || least != least ? 0xFFFFFFFFu : order_of(most);
        }
    };
};

constexpr int kT = 1024;       // lanes of a row's workgroup
constexpr int kMaxRow = 1 << 22;  // a row's logits are fewer
constexpr int kBins = 2048;    // bins of a histogram
constexpr int kList = 1024;    // elements that are sorted at once
constexpr int kSmallK = 512;   // most of top-k for the way of counts alone
// Bins from here on hold no weight: exp(-28.5) 2^40 is below a half.
constexpr int kLightBin = 1824;
constexpr float kPerUnit = 64.0f;  // bins per unit of (max - l) / temperature
constexpr int kStepBits = 8, kSteps = 1 << kStepBits;  // of the exponential's table
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

// LDS: what every way needs, and the histograms; a kept row takes the place of those
// of the searches, which read the row from memory.
struct Shared {
    double power[kSteps];  // 2^(i / kSteps)
    u64 list[kList];   // sorted keys (key_of)
    u64 wave_sum[kT / 64];
    uint32_t wave_count[kT / 64];
    float wave_min[kT / 64], wave_max[kT / 64];
    u64 before_sum, before_count;
    // of the ways of one histogram: each place is written once a row
    u64 slots[4][kT / 64], picked[2];
    struct At {
        u64 before, own;
        int bin;
    } at[3];
    uint32_t fewest[kT / 64];
    Found found;
    uint32_t listed;
    int flag, bin;
};
struct Searches {
    Histogram all, part;
};
// A histogram of sums or of counts alone.
union Single {
    u64 sum[kBins];
    uint32_t count[kBins];
};

// What a row's weights are made with.
struct Scale {
    float most;
    double inverse;       // 1 / temperature
    float per;            // bins per unit of max - l
    const double* power;  // 2^(i / kSteps) in LDS

    // exp((l - max) / temperature), 2^-42 of it off; 0 where it is below 2^-41.  With
    // n = 256 x / log 2 rounded: 2^(n / 256) from the table times e^r, |r| < 0.00136, to
    // r^3.
    __device__ __forceinline__ double weight(float l) const {
        double x = ((double)l - (double)most) * inverse;
        if (l == most) x = 0.0;
        const bool some = x > -28.5;  // NaN (a masked logit, no temperature): none
        x = some ? x : 0.0;
        const double shift = 0x1.8p52;
        const double s = fma(x, kSteps / 0.693147180559945309417232, shift);
        const int n = (int)(uint32_t)__builtin_bit_cast(u64, s);
        const double r = fma(s - shift, -0.693147180559945309417232 / kSteps, x);
        const double p = r * fma(r, fma(r, 1.0 / 6, 0.5), 1.0);
        const double t = power[n & (kSteps - 1)];
        const double e = __builtin_amdgcn_ldexp(fma(t, p, t), n >> kStepBits);
        return some ? e : 0.0;
    }
    __device__ __forceinline__ int bin(float l) const {
        return l == most ? 0 : (int)fminf((most - l) * per, (float)(kBins - 1));
    }
    // Where the largest logit is finite, and the bins' width too and not so large that a
    // difference beyond fp32's largest has weight (kLightBin / per is 2^127 then), the
    // difference needs no second look: a logit's place in bins is the quotient
    // (-infinity, and a difference that overflows: infinity), and what lies past kLightBin
    // has no weight.
    __device__ __forceinline__ bool ordinary() const {
        return fabsf(most) < INFINITY && per < INFINITY && per >= kLightBin * 0x1p-127f;
    }
    __device__ __forceinline__ float place(float l) const { return (most - l) * per; }
    // Of a logit whose place is below kLightBin: no clamp.
    __device__ __forceinline__ u64 whole_weight(float l) const {
        const double x = ((double)l - (double)most) * inverse;
        const double shift = 0x1.8p52;
        const double s = fma(x, kSteps / 0.693147180559945309417232, shift);
        const int n = (int)(uint32_t)__builtin_bit_cast(u64, s);
        const double r = fma(s - shift, -0.693147180559945309417232 / kSteps, x);
        const double p = r * fma(r, fma(r, 1.0 / 6, 0.5), 1.0);
        const double t = power[n & (kSteps - 1)];
        // 2^40 2^(n / kSteps's whole part)
        const double up =
            __builtin_bit_cast(double, (u64)(uint32_t)((n >> kStepBits) + 1063) << 52);
        return __builtin_bit_cast(u64, fma(fma(t, p, t), up, 0x1p52)) - 0x4330000000000000ull;
    }
};
__device__ __forceinline__ u64 whole(double w) {
    // below 2^52: the rounded value is the low half of w 2^40 + 2^52
    return __builtin_bit_cast(u64, fma(w, kOne, 0x1p52)) - 0x4330000000000000ull;
}

// Logits and indices as keys in the order of the search (ascending), and back.
__device__ __forceinline__ u64 key_of(float l, uint32_t index) {
    return ((u64)~order_of(l) << 32) | index;
}
__device__ __forceinline__ float logit_of(u64 key) {
    return logit_in_order(~(uint32_t)(key >> 32));
}

// A row's elements, 16 bytes at a time, read from memory for each pass, or (HELD)
// kept in LDS by the first one.
template <class E, bool HELD>
struct Row {
    typedef Logits<E> L;
    typedef typename L::Bits Bits;
    static constexpr int W = L::kWidth;
    const Bits* ptr;
    int V;
    u4_t* kept;

    // Past the row's end: -infinity, which no pass takes.
    __device__ __forceinline__ u4_t piece(int c) const {
        u4_t w = {L::kLeast, L::kLeast, L::kLeast, L::kLeast};
        if (c + W <= V) {
            __builtin_memcpy(&w, ptr + c, 16);
        } else if (c < V) {
            Bits b[W];
#pragma unroll
            for (int q = 0; q < W; ++q) {
                const Bits v = ptr[c + q < V ? c + q : c];
                b[q] = c + q < V ? v : (Bits)L::kLeast;
            }
            __builtin_memcpy(&w, b, 16);
        }
        return w;
    }
    // Calls that take long expressions are kept apart two by two: with all of a
    // piece's at once in registers they would not fit.
    template <class Fn>
    __device__ __forceinline__ void visit(u4_t w, int c, Fn&& f) const {
        Bits b[W];
        __builtin_memcpy(b, &w, 16);
#pragma unroll
        for (int q = 0; q < W; ++q) {
            f(c + q, L::get(b[q]));
            if (q & 1) __builtin_amdgcn_sched_barrier(0);
        }
    }
    // f(index, logit) for this lane's elements, and for -infinity behind the row's
    // end.
    template <class Fn>
    __device__ __forceinline__ void each(Fn&& f) const {
#pragma unroll 1
        for (int p = threadIdx.x; p * W < V; p += kT) visit(HELD ? kept[p] : piece(p * W), p * W, f);
    }
    // The first pass, 4 pieces on their way at once: keeps the row, and returns the
    // ends of this lane's elements.
    __device__ __forceinline__ typename L::Ends first_pass() const {
        typename L::Ends ends;
#pragma unroll 1
        for (int p = threadIdx.x; p * W < V; p += 4 * kT) {
            u4_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = piece((p + i * kT) * W);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (HELD && (p + i * kT) * W < V) kept[p + i * kT] = w[i];
                ends.add(w[i]);
            }
        }
        return ends;
    }
};

// Sums and the like over the 64 lanes of a wave, by moves between neighbours,
// rows of 16 and their ends (row_shr 1, 2, 4, 8, then row_bcast 15 and 31): each is a
// few cycles where an exchange through LDS is a hundred.  Lanes without a source get
// `none`.
template <int CTRL, int ROWS, class V>
__device__ __forceinline__ V moved(V none, V v) {
    if constexpr (sizeof(V) == 8) {
        const u64 n = __builtin_bit_cast(u64, none), w = __builtin_bit_cast(u64, v);
        const uint32_t lo = moved<CTRL, ROWS>((uint32_t)n, (uint32_t)w);
        const uint32_t hi = moved<CTRL, ROWS>((uint32_t)(n >> 32), (uint32_t)(w >> 32));
        return __builtin_bit_cast(V, ((u64)hi << 32) | lo);
    } else {
        return __builtin_bit_cast(
            V, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, v),
                                           CTRL, ROWS, 0xF, false));
    }
}
// v combined with those of the lanes before.
template <class V, class Op>
__device__ __forceinline__ V wave_scan(V v, V none, Op op) {
    v = op(v, moved<0x111, 0xF>(none, v));
    v = op(v, moved<0x112, 0xF>(none, v));
    v = op(v, moved<0x114, 0xF>(none, v));
    v = op(v, moved<0x118, 0xF>(none, v));
    v = op(v, moved<0x142, 0xA>(none, v));
    return op(v, moved<0x143, 0xC>(none, v));
}
template <class V>
__device__ __forceinline__ V from_lane(V v, int lane) {
    if constexpr (sizeof(V) == 8) {
        const u64 w = __builtin_bit_cast(u64, v);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)w, lane);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(w >> 32), lane);
        return __builtin_bit_cast(V, ((u64)hi << 32) | lo);
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    }
}
struct Plus {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Larger {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};
struct Smaller {
    __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return min(a, b); }
};

constexpr int kWaves = kT / 64;

// v combined over the workgroup.  The slots are free: nothing has read them since
// the last barrier.
template <class V, class Op>
__device__ __forceinline__ V over_block_once(V v, V none, V* slots, Op op) {
    v = from_lane(wave_scan(v, none, op), 63);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v = op(v, slots[i]);
    return v;
}
template <class V, class Op>
__device__ __forceinline__ V over_block(V v, V none, V* slots, Op op) {
    __syncthreads();
    return over_block_once(v, none, slots, op);
}

__device__ __forceinline__ void clear(Histogram& h) {
    for (int i = threadIdx.x; i < kBins; i += kT) {
        h.sum[i] = 0;
        h.count[i] = 0;
    }
}
__device__ __forceinline__ void clear(Single& h) {
    for (int i = threadIdx.x; i < kBins; i += kT) h.sum[i] = 0;
}

// The bin in which the running sum (by_count: count) first reaches `goal`, and
// what comes before it: s.bin, s.before_sum, s.before_count.  Bins run in
// descending order of the logits.
__device__ __forceinline__ void find_bin(Shared& s, const Histogram& h, bool by_count, u64 goal,
                                         u64 sum0, u64 count0) {
    constexpr int PER = kBins / kT;
    const int wave = threadIdx.x >> 6;
    u64 own_sum = 0;
    uint32_t own_count = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        own_sum += h.sum[threadIdx.x * PER + i];
        own_count += h.count[threadIdx.x * PER + i];
    }
    const u64 sums = wave_scan(own_sum, (u64)0, Plus{});
    const uint32_t counts = wave_scan(own_count, 0u, Plus{});
    __syncthreads();
    if ((threadIdx.x & 63) == 63) {
        s.wave_sum[wave] = sums;
        s.wave_count[wave] = counts;
    }
    __syncthreads();
    u64 bs = sum0 + sums - own_sum, bc = count0 + counts - own_count;
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

// The sum of v over the lanes up to and with this one.  The slots are free.
__device__ __forceinline__ u64 running_sum(u64 v, u64* slots) {
    const int wave = threadIdx.x >> 6;
    v = wave_scan(v, (u64)0, Plus{});
    if ((threadIdx.x & 63) == 63) slots[wave] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves - 1; ++i) v += i < wave ? slots[i] : 0;
    return v;
}

// Appends the row's elements that `in` takes to the list (s.listed is 0); those
// that it has no room for are counted.
template <class R, class In>
__device__ __forceinline__ void gather(Shared& s, const R& row, In&& in) {
    row.each([&](int i, float l) __attribute__((always_inline)) {
        if (in(l)) {
            const uint32_t at = atomicAdd(&s.listed, 1u);
            if (at < kList) s.list[at] = key_of(l, (uint32_t)i);
        }
    });
    __syncthreads();
}

// Sorts the first n (at most kList) keys of the list.  Up to 256 each key counts the
// smaller ones (n reads that all lanes of a wave share); more take a bitonic network,
// a key a lane, between lanes of a wave by exchanges and between waves through LDS.
__device__ __forceinline__ void sort_list(Shared& s, uint32_t n) {
    static_assert(kList == kT, "a key a lane");
    const uint32_t t = threadIdx.x;
    if (n <= 256) {
        if (t >= n && t < ((n + 7) & ~7u)) s.list[t] = ~0ull;
        __syncthreads();
        u64 key = 0;
        uint32_t rank = 0;
        if (t < n) {
            key = s.list[t];
            for (uint32_t j = 0; j < n; j += 8) {
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) rank += s.list[j + i] < key ? 1 : 0;
            }
        }
        __syncthreads();
        if (t < n) s.list[rank] = key;
        __syncthreads();
        return;
    }
    u64 key = t < n ? s.list[t] : ~0ull;
    for (uint32_t size = 2; size < 2 * n; size <<= 1)
        for (uint32_t half = size / 2; half > 0; half >>= 1) {
            u64 other;
            if (half < 64) {
                other = __shfl_xor(key, (int)half, 64);
            } else {
                __syncthreads();
                s.list[t] = key;
                __syncthreads();
                other = s.list[t ^ half];
            }
            const bool least = ((t & half) == 0) == ((t & size) == 0);
            key = least == (key < other) ? key : other;
        }
    __syncthreads();
    s.list[t] = key;
    __syncthreads();
}

// The first element, in the order, at which the running sum (by_count: count)
// reaches `goal`, which lies between 1 and the whole row's.
template <class R>
__device__ __forceinline__ void search(Shared& s, Searches& h, const R& row, const Scale& sc,
                                       bool by_count, u64 goal) {
    find_bin(s, h.all, by_count, goal, 0, 0);
    const int bin = s.bin;
    u64 before_sum = s.before_sum, before_count = s.before_count;
    uint32_t count = h.all.count[bin];
    // The elements looked at: those of the bin, then those of lo <= l <= hi.
    float lo = 0.0f, hi = 0.0f;
    bool ranged = false;
    auto in = [&](float l) __attribute__((always_inline)) {
        if (ranged) return l >= lo && l <= hi;
        // a bin far out may hold logits without weight, which do not count
        return sc.bin(l) == bin && (bin < kBins * 7 / 8 || whole(sc.weight(l)) != 0);
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
        least = over_block(least, (float)INFINITY, s.wave_min, Smaller{});
        top = over_block(top, -(float)INFINITY, s.wave_max, Larger{});
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
        clear(h.part);
        __syncthreads();
        row.each([&](int, float l) __attribute__((always_inline)) {
            if (l >= lo && l <= hi) {
                const int b = sub(l);
                atomicAdd(&h.part.sum[b], whole(sc.weight(l)));
                atomicAdd(&h.part.count[b], 1u);
            }
        });
        __syncthreads();
        find_bin(s, h.part, by_count, goal, before_sum, before_count);
        before_sum = s.before_sum, before_count = s.before_count;
        count = h.part.count[s.bin];
        // the ends of that bin's logits
        const int want = s.bin;
        least = INFINITY, top = -INFINITY;
        row.each([&](int, float l) __attribute__((always_inline)) {
            if (l >= lo && l <= hi && sub(l) == want) {
                least = fminf(least, l);
                top = fmaxf(top, l);
            }
        });
        lo = over_block(least, (float)INFINITY, s.wave_min, Smaller{});
        hi = over_block(top, -(float)INFINITY, s.wave_max, Larger{});
        if (lo == hi) break;
    }
    __syncthreads();
    if (count > kList) {
        // `count` equal logits: the r-th of them by index.
        const u64 w = whole(sc.weight(lo));
        const u64 r = by_count ? goal - before_count : (goal - before_sum + w - 1) / w;
        // Lane t looks at the t-th stretch of the row.
        const int64_t per = ((int64_t)row.V + kT - 1) / kT;
        const int64_t i0 = threadIdx.x * per, i1 = min(i0 + per, (int64_t)row.V);
        uint32_t mine = 0;
        for (int64_t i = i0; i < i1; ++i) mine += R::L::get(row.ptr[i]) == lo;
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
                if (R::L::get(row.ptr[i]) == lo && ++n == r) {
                    s.found.sum = before_sum + r * w;
                    s.found.index = i;
                    s.found.logit = lo;
                }
        __syncthreads();
        return;
    }
    if (threadIdx.x == 0) s.listed = 0;
    __syncthreads();
    gather(s, row, in);
    sort_list(s, count);
    // the running sums over the list
    const bool mine = threadIdx.x < count;
    const u64 key = mine ? s.list[threadIdx.x] : 0;
    const float l = logit_of(key);
    const u64 w = mine ? whole(sc.weight(l)) : 0;
    __syncthreads();
    const u64 upto = before_sum + running_sum(w, s.wave_sum);
    const u64 reach = by_count ? before_count + threadIdx.x + 1 : upto;
    if (mine && reach >= goal && reach - (by_count ? 1 : w) < goal) {
        s.found.sum = upto;
        s.found.index = (uint32_t)key;
        s.found.logit = l;
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

// The least weight that min-p keeps.
__device__ __forceinline__ u64 least_weight(float min_p) {
    return min_p > 0.0f ? (u64)ceil(fmin((double)min_p, 1.0) * kOne) : 0;
}


struct Settings {
    float u, temperature, top_p, min_p;
    int32_t top_k;
};

// The row by one search after the other.
template <class R>
__device__ __forceinline__ void sample_searching(Shared& s, Searches& h, const R& row,
                                                 const Scale& sc, const Settings& set) {
    __syncthreads();
    clear(h.all);
    __syncthreads();
    const u64 bound = least_weight(set.min_p);
    u64 kept = 0, total = 0;
    uint32_t n = 0;
    row.each([&](int, float l) __attribute__((always_inline)) {
        const u64 w = whole(sc.weight(l));
        if (w != 0) {
            const int b = sc.bin(l);
            atomicAdd(&h.all.sum[b], w);
            atomicAdd(&h.all.count[b], 1u);
            total += w;
            ++n;
            if (w >= bound) kept += w;
        }
    });
    kept = over_block(kept, (u64)0, s.wave_sum, Plus{});
    total = over_block(total, (u64)0, s.wave_sum, Plus{});
    n = over_block(n, 0u, s.wave_count, Plus{});
    u64 Z = total;
    // top-k, top-p, the token
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        u64 goal = (u64)set.top_k;
        if (step == 0 && !(set.top_k > 0 && (uint32_t)set.top_k < n)) continue;
        if (step == 1) {
            if (!(set.top_p < 1.0f)) continue;
            goal = least_sum((double)set.top_p * (double)Z, false, Z);
        }
        if (step == 2) {
            Z = min(Z, kept);
            goal = least_sum((double)set.u * (double)Z, true, Z);
        }
        search(s, h, row, sc, step == 0, goal);
        if (step < 2) Z = min(Z, s.found.sum);
    }
    __syncthreads();
    if (threadIdx.x == 0) s.found.sum = Z;
    __syncthreads();
}

// Which bins a row's token and the end of top-p lie in: those of first .. last, and
// `end` (behind them, or -1), and the sums before first and before end.
struct Wanted {
    int first, last, end;
    u64 before, before_end;
    u64 total, kept;  // the sums of all and of what min-p keeps (without top-k)
};

__device__ __forceinline__ bool by_counts(const Settings& set, int V) {
    return set.top_k > 0 && set.top_k <= kSmallK && set.top_k < V;
}

// From the histogram: of counts (`counts`: the bins up to the k-th's), or of sums.  kept:
// the sum that min-p keeps, where it is on.
__device__ __forceinline__ Wanted wanted_bins(Shared& s, const Single& h, bool counts,
                                              const Settings& set, u64 kept) {
    constexpr int PER = kBins / kT;
    const int first_bin = threadIdx.x * PER, wave = threadIdx.x >> 6;
    u64 own[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        sum += own[i] = counts ? h.count[first_bin + i] : h.sum[first_bin + i];
    const u64 upto = wave_scan(sum, (u64)0, Plus{});
    if ((threadIdx.x & 63) == 63) s.slots[0][wave] = upto;
    __syncthreads();
    u64 before = upto - sum, total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        const u64 v = s.slots[0][i];
        before += i < wave ? v : 0;
        total += v;
    }
    // The bin in which the running sum first reaches `goal`, to s.at[k].
    auto find = [&](u64 goal, int k) __attribute__((always_inline)) {
        u64 b = before;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (b < goal && goal <= b + own[i]) s.at[k] = {b, own[i], first_bin + i};
            b += own[i];
        }
    };
    Wanted w = {0, 0, -1, 0, 0, total, set.min_p > 0.0f ? kept : total};
    if (counts) {
        // fewer with weight than k: all of them
        w.last = kLightBin - 1;
        if ((u64)set.top_k <= total) {
            find((u64)set.top_k, 0);
            __syncthreads();
            w.last = s.at[0].bin;
        }
        return w;
    }
    u64 low = total, high = total;  // bounds of what top-p keeps
    if (set.top_p < 1.0f) {
        find(least_sum((double)set.top_p * (double)total, false, total), 0);
        __syncthreads();
        w.end = s.at[0].bin;
        w.before_end = s.at[0].before;
        low = w.before_end + 1, high = w.before_end + s.at[0].own;
    }
    low = min(low, w.kept), high = min(high, w.kept);
    find(least_sum((double)set.u * (double)low, true, low), 1);
    if (high != low) find(least_sum((double)set.u * (double)high, true, high), 2);
    __syncthreads();
    w.first = s.at[1].bin;
    w.before = s.at[1].before;
    // high is at most the sum up to the end of top-p's bin, and the token's goal at most
    // high: first <= last, and last <= end where top-p is on.
    w.last = high != low ? s.at[2].bin : w.first;
    return w;
}

// The token of a row whose wanted elements are the first n of the list (n at most
// kList): s.found, with the sum kept for found.sum.  Up to 64 are the first wave's
// alone.
__device__ __forceinline__ void sample_list(Shared& s, uint32_t n, bool counts, const Wanted& want,
                                            const Scale& sc, const Settings& set) {
    sort_list(s, n);
    const uint32_t t = threadIdx.x;
    const bool alone = n <= 64;
    if (!alone || t < 64) {
        const bool mine = t < n;
        const u64 key = mine ? s.list[t] : 0;
        const float l = logit_of(key);
        const u64 w = mine ? whole(sc.weight(l)) : 0;
        u64 upto = alone ? wave_scan(w, (u64)0, Plus{}) : running_sum(w, s.slots[1]);
        // v of the one lane that has `here`
        auto pick = [&](bool here, u64 v, u64* slot) __attribute__((always_inline)) {
            if (alone) {
                const u64 lanes = __ballot(here);
                return lanes != 0 ? from_lane(v, __builtin_ctzll(lanes)) : 0;
            }
            if (here) *slot = v;
            __syncthreads();
            return *slot;
        };
        auto reaches = [&](u64 goal) __attribute__((always_inline)) {
            return mine && upto >= goal && upto - w < goal;
        };
        u64 Z = want.total, kept = want.kept;
        bool ends = true;  // whether this element may be where top-p ends
        if (counts) {
            // the list is the beginning of the order
            const uint32_t k = min((uint32_t)set.top_k, n);
            Z = kept = pick(t == k - 1, upto, &s.picked[0]);
            if (set.min_p > 0.0f) {
                const u64 v = t < k && w >= least_weight(set.min_p) ? w : 0;
                kept = alone ? from_lane(wave_scan(v, (u64)0, Plus{}), 63)
                             : over_block_once(v, (u64)0, s.slots[2], Plus{});
            }
        } else {
            // The bins first .. last, then `end`: the sums before them come from the
            // histogram.
            const int bin = mine ? (int)sc.place(l) : 0;
            const bool behind = bin > want.last;
            ends = bin == want.end;
            u64 front = 0;
            if (want.end > want.last)
                front = pick(mine && !behind &&
                                 (t == n - 1 || (int)sc.place(logit_of(s.list[t + 1])) > want.last),
                             upto, &s.picked[0]);
            upto += behind ? want.before_end - front : want.before;
        }
        if (set.top_p < 1.0f) {
            const u64 goal = least_sum((double)set.top_p * (double)Z, false, Z);
            Z = min(Z, pick(ends && reaches(goal), upto, &s.picked[1]));
        }
        Z = min(Z, kept);
        if (reaches(least_sum((double)set.u * (double)Z, true, Z))) {
            s.found.sum = Z;
            s.found.index = (uint32_t)key;
            s.found.logit = l;
        }
    }
    __syncthreads();
}

struct SampleArgs {
    const void* logits;
    int64_t ld;
    const float* u;
    Setting<float> temperature, top_p, min_p;
    Setting<int32_t> top_k;
    int64_t* tokens;
    float* logprobs;
    int64_t M;
    int V;
    // (All loads on their way at once: what has no array reads u's.)
    template <class V>
    __device__ __forceinline__ V of_row(const Setting<V>& s, int64_t m) const {
        static_assert(sizeof(V) == sizeof(float), "");
        V v;
        __builtin_memcpy(&v, (s.each ? (const char*)s.each : (const char*)u) + 4 * m, 4);
        return s.each ? v : s.value;
    }
    __device__ __forceinline__ Settings settings(int64_t m) const {
        // a number of 1 and more is the largest fp32 below 1 (below 0, and NaN: least_sum)
        const float n = u[m];
        return {n >= 1.0f ? 0x1.fffffep-1f : n, of_row(temperature, m), of_row(top_p, m), of_row(min_p, m), of_row(top_k, m)};
    }
    __device__ __forceinline__ void put(int64_t m, int64_t token, float logprob) const {
        tokens[m] = token;
        if (logprobs) logprobs[m] = logprob;
    }
    __device__ __forceinline__ void put_found(int64_t m, const Found& f, const Scale& sc) const {
        const double x =
            f.logit == sc.most ? 0.0 : ((double)f.logit - (double)sc.most) * sc.inverse;
        put(m, f.index, (float)(x - log((double)f.sum / kOne)));
    }
};

__device__ __forceinline__ Scale scale_for(const Shared& s, float most, float temperature) {
    return {most, 1.0 / (double)temperature, kPerUnit / temperature, s.power};
}
__device__ __forceinline__ void fill_powers(Shared& s) {
    if (threadIdx.x < kSteps) s.power[threadIdx.x] = exp2(threadIdx.x / (double)kSteps);
}

// This lane's part of the histogram, of counts or of sums, and of the sum that min-p
// keeps.  An ordinary row's (Scale).
template <class R>
__device__ __forceinline__ void add_to_histogram(Single& h, const R& row, const Scale& sc,
                                                 const Settings& set, bool counts, u64& kept) {
    if (counts) {
        row.each([&](int, float l) __attribute__((always_inline)) {
            const float d = sc.place(l);
            if (d < (float)kLightBin) atomicAdd(&h.count[(int)d], 1u);
        });
    } else if (set.min_p > 0.0f) {
        const u64 bound = least_weight(set.min_p);
        row.each([&](int, float l) __attribute__((always_inline)) {
            const float d = sc.place(l);
            if (d < (float)kLightBin) {
                const u64 w = sc.whole_weight(l);
                atomicAdd(&h.sum[(int)d], w);
                kept += w >= bound ? w : 0;
            }
        });
    } else {
        row.each([&](int, float l) __attribute__((always_inline)) {
            const float d = sc.place(l);
            if (d < (float)kLightBin) atomicAdd(&h.sum[(int)d], sc.whole_weight(l));
        });
    }
}
// Whether a row's settings and scale allow the ways of one histogram.
__device__ __forceinline__ bool one_histogram(const Scale& sc, const Settings& set, int V) {
    return sc.ordinary() && (by_counts(set, V) || !(set.top_k > 0 && set.top_k < V));
}

template <class R>
__device__ __forceinline__ void gather_wanted(Shared& s, const R& row, const Scale& sc,
                                              const Wanted& want) {
    const float lo = (float)want.first, hi = (float)(want.last + 1), lo2 = (float)want.end,
                hi2 = (float)(want.end + 1);
    if (want.end > want.last)
        gather(s, row, [&](float l) __attribute__((always_inline)) {
            const float d = sc.place(l);
            return (d >= lo && d < hi) || (d >= lo2 && d < hi2);
        });
    else
        gather(s, row, [&](float l) __attribute__((always_inline)) {
            const float d = sc.place(l);
            return d >= lo && d < hi;
        });
}

// A workgroup per row.  HELD: bytes of LDS that keep the row (0: none).  Bound by
// instructions, 45 an element where each is weighed.  256 rows of bf16: 12 us of 8192
// (top-k 50), 20 of 32768, 27 of 65536.  (Up to 15 registers spill: constants that the
// compiler works out before the loop over rows and reads once a row.)
template <class E, int HELD>
__global__ __launch_bounds__(kT) void sample_kernel(const SampleArgs a) {
    __shared__ Shared s;
    __shared__ union {
        Searches searches;
        struct {
            Single single;
            u4_t row[HELD > 0 ? HELD / 16 : 1];
        };
    } h;
    typedef Row<E, (HELD > 0)> R;
    fill_powers(s);
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const R row = {static_cast<const typename R::Bits*>(a.logits) + m * a.ld, a.V, h.row};
        const Settings set = a.settings(m);
        __syncthreads();  // the row before is done
        // The largest logit, and whether there is a NaN.
        const auto ends = row.first_pass();
        if (threadIdx.x == 0) s.listed = 0;
        clear(h.single);
        const float most =
            logit_in_order(over_block_once(ends.order(), 0u, s.fewest, Larger{}));
        if (!(most > -INFINITY)) {
            if (threadIdx.x == 0) a.put(m, -1, __builtin_nanf(""));
            continue;
        }
        if (!(set.temperature > 0.0f)) {
            // Greedy: the first of the largest.
            uint32_t first = 0xFFFFFFFFu;
            row.each([&](int i, float l) __attribute__((always_inline)) {
                if (l == most) first = min(first, (uint32_t)i);
            });
            first = over_block_once(first, 0xFFFFFFFFu, s.wave_count, Smaller{});
            if (threadIdx.x == 0) a.put(m, first, 0.0f);
            continue;
        }
        const Scale sc = scale_for(s, most, set.temperature);
        const bool counts = by_counts(set, a.V);
        bool done = false;
        if (one_histogram(sc, set, a.V)) {
            u64 kept = 0;
            add_to_histogram(h.single, row, sc, set, counts, kept);
            if (set.min_p > 0.0f && !counts)
                kept = over_block_once(kept, (u64)0, s.slots[3], Plus{});
            else
                __syncthreads();
            const Wanted want = wanted_bins(s, h.single, counts, set, kept);
            gather_wanted(s, row, sc, want);
            const uint32_t n = s.listed;
            if (n <= kList) {
                sample_list(s, n, counts, want, sc, set);
                done = true;
            }
        }
        if (!done) {
            const Row<E, false> all = {row.ptr, a.V, nullptr};
            sample_searching(s, h.searches, all, sc, set);
        }
        if (threadIdx.x == 0) a.put_found(m, s.found, sc);
    }
}

// 16-bit logits, a workgroup per row: a counter for each of the 65536 patterns.  Then
// only the patterns that occur are weighed, once each, a search ends at a pattern, and
// equal logits need no list: the r-th of them by index is found in a last pass.  The
// time hardly depends on the settings or on how the logits lie (by_patterns()).
//
// Patterns in descending order of their logits: d = 32767 - key, the key being the
// pattern as a whole number of the same order, +0 and -0 the same.  A wave looks at
// 64 of them, a group; groups[g] holds a group's sums.
//
// 256 x 65536 bf16: 33 us for 33.5 MB (1.0 TB/s).  A wave's 2300 vector instructions, most
// of them in three passes over the row, which stays in registers up to 65536, are 15
// us of it with four waves a SIMD; the rest is the first read, 143 KB of counters
// cleared, and the searches, chains of LDS reads and scans of one wave.  (With all waves
// searching, and barriers between, 38 us.)  Of the 128 registers that 1024 lanes leave each
// other 21-30 spill: constants from before the loop over rows, read once or twice a row,
// and with HELD 8 one of its pieces.
struct Groups {
    u64 sum[1024];
    uint32_t count[1024];
};
struct Patterns {
    uint32_t counts[32768];  // d even in the low half
    Groups groups;
};

// Where a search ended: the pattern, what comes before it, its weight and count.
struct Place {
    int d;
    uint32_t count, before_count;
    u64 weight, before;
};

template <class E>
struct PatternSearch {
    typedef Logits<E> L;
    Shared& s;
    Patterns& h;
    const Scale& sc;
    u64 upto;  // of lane i (of the first 16): the sum of the first i + 1 waves' groups
    uint32_t upto_n;

    __device__ static __forceinline__ float value(int d) {
        const int key = 32767 - d;
        return L::Ends::value(key < 0 ? key - 1 : key);
    }
    // The pattern nearest to l.
    __device__ static __forceinline__ int pattern(float l) {
        const int b = (int16_t)E::put(l), sign = b >> 15;
        return 32767 - ((b ^ (sign & 0x7FFF)) - sign);
    }
    __device__ __forceinline__ uint32_t count(int d) const {
        return (h.counts[d >> 1] >> (16 * (d & 1))) & 0xFFFFu;
    }
    __device__ __forceinline__ u64 weight(int d, uint32_t n) const {
        if (n == 0) return 0;
        const float l = value(d);
        return sc.place(l) < (float)kLightBin ? sc.whole_weight(l) : 0;
    }
    // The sums of the groups first .. last, in turns of the waves; returns this lane's
    // part of what min-p keeps.
    __device__ __forceinline__ u64 weigh(int first, int last, u64 bound) {
        u64 kept = 0;
        const int lane = threadIdx.x & 63;
#pragma unroll 1
        for (int g0 = first + (threadIdx.x >> 6); g0 <= last; g0 += 4 * kWaves) {
            uint32_t n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                n[i] = g0 + i * kWaves <= last ? count(64 * (g0 + i * kWaves) + lane) : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (__ballot(n[i] != 0) == 0) continue;
                const int g = g0 + i * kWaves;
                const u64 w = weight(64 * g + lane, n[i]), m = w * n[i];
                kept += w >= bound ? m : 0;
                const u64 sum = wave_scan(m, (u64)0, Plus{});
                const uint32_t all = wave_scan(n[i], 0u, Plus{});
                if (lane == 63) {
                    h.groups.sum[g] = sum;
                    h.groups.count[g] = all;
                }
            }
        }
        return kept;
    }
    // The running sums of each wave's groups, in their place.
    __device__ __forceinline__ void sum_up() {
        static_assert(kT == 1024, "a group a lane");
        const int wave = threadIdx.x >> 6;
        const u64 sum = wave_scan(h.groups.sum[threadIdx.x], (u64)0, Plus{});
        const uint32_t n = wave_scan(h.groups.count[threadIdx.x], 0u, Plus{});
        h.groups.sum[threadIdx.x] = sum;
        h.groups.count[threadIdx.x] = n;
        if ((threadIdx.x & 63) == 63) {
            s.slots[0][wave] = sum;
            s.slots[1][wave] = n;
        }
        __syncthreads();
    }
    // From here on the first wave's alone.
    __device__ __forceinline__ void begin(u64& total, uint32_t& n) {
        const int lane = threadIdx.x;
        upto = wave_scan(lane < kWaves ? s.slots[0][lane] : 0, (u64)0, Plus{});
        upto_n = wave_scan(lane < kWaves ? (uint32_t)s.slots[1][lane] : 0, 0u, Plus{});
        total = from_lane(upto, 63);
        n = from_lane(upto_n, 63);
    }
    // The first pattern at which the running sum (COUNT: count) reaches `goal`, at most
    // the total.
    template <bool COUNT>
    __device__ __forceinline__ Place find(u64 goal) const {
        const int lane = threadIdx.x;
        // the wave, its group, the pattern
        int at = __builtin_ctzll(__ballot(COUNT ? upto_n >= goal : upto >= goal) | 1ull << 15);
        const int wave = at;
        u64 before = at > 0 ? from_lane(upto, at - 1) : 0;
        uint32_t before_n = at > 0 ? from_lane(upto_n, at - 1) : 0;
        const u64 sum = before + h.groups.sum[64 * wave + lane];
        const uint32_t num = before_n + h.groups.count[64 * wave + lane];
        at = __builtin_ctzll(__ballot(COUNT ? num >= goal : sum >= goal) | 1ull << 63);
        const int g = 64 * wave + at;
        before = at > 0 ? from_lane(sum, at - 1) : before;
        before_n = at > 0 ? from_lane(num, at - 1) : before_n;
        const uint32_t n = count(64 * g + lane);
        const u64 w = weight(64 * g + lane, n), m = w * n;
        const u64 sum1 = before + wave_scan(m, (u64)0, Plus{});
        const uint32_t num1 = before_n + wave_scan(n, 0u, Plus{});
        at = __builtin_ctzll(__ballot(COUNT ? num1 >= goal : sum1 >= goal) | 1ull << 63);
        return {64 * g + at, from_lane(n, at), from_lane(num1 - n, at), from_lane(w, at),
                from_lane(sum1 - m, at)};
    }
};

// A row's pieces, the workgroup's i-th 1024 in turn; up to HELD of them stay in
// registers.  (HELD 0: read for each pass, 4 on their way at once.)
template <class E, int HELD>
struct Pieces {
    typedef Row<E, false> R;
    R row;
    int t;
    u4_t held[HELD > 0 ? HELD : 1];
    __device__ __forceinline__ explicit Pieces(const R& r) : row(r), t(threadIdx.x) {
        // What depends on the lane is not worked out ahead of the loop over rows, where
        // it would fill the registers.
        asm volatile("" : "+v"(t));
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) held[i] = row.piece((t + i * kT) * 8);
        }
    }
    // f(piece's bits, its first index): whole waves, with pieces of -infinity behind
    // the row's end.
    template <class Fn>
    __device__ __forceinline__ void each(Fn&& f) const {
        const int first = __builtin_amdgcn_readfirstlane(t) * 8, own = (t & 63) * 8;
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const int c = first + i * kT * 8;
                if (c < row.V) f(held[i], c + own);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll 1
            for (int c = first; c < row.V; c += 4 * kT * 8) {
                u4_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = row.piece(c + i * kT * 8 + own);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i * kT * 8 < row.V) f(w[i], c + i * kT * 8 + own);
            }
        }
    }
};

template <class E, int HELD>
__global__ __launch_bounds__(kT) void sample_patterns_kernel(const SampleArgs a) {
    __shared__ Shared s;
    __shared__ __attribute__((aligned(16))) union {
        Patterns patterns;
        Searches searches;
        uint32_t matches[8192];  // of each wave's pieces
    } h;
    static_assert(sizeof(h.matches) / 4 * 64 * 8 >= (size_t)kMaxRow, "a place for each");
    typedef Row<E, false> R;
    typedef PatternSearch<E> P;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const R row = {static_cast<const uint16_t*>(a.logits) + m * a.ld, a.V, nullptr};
        const Pieces<E, HELD> pieces(row);
        const int wave = pieces.t >> 6, lane = pieces.t & 63;
        const Settings set = a.settings(m);
        __syncthreads();  // the row before is done
        if (m == blockIdx.x) fill_powers(s);
        for (int i = threadIdx.x; i < (int)(sizeof(Patterns) / 16); i += kT)
            reinterpret_cast<u4_t*>(&h.patterns)[i] = u4_t{};
        typename Logits<E>::Ends ends;
        pieces.each([&](u4_t w, int) __attribute__((always_inline)) { ends.add(w); });
        const float most = logit_in_order(over_block_once(ends.order(), 0u, s.fewest, Larger{}));
        if (!(most > -INFINITY)) {
            if (threadIdx.x == 0) a.put(m, -1, __builtin_nanf(""));
            continue;
        }
        // The elements whose logit is l, a bit for each.
        auto matches = [](u4_t w, float l) __attribute__((always_inline)) {
            const uint32_t pair = E::put(l) * 0x10001u, mask = l == 0.0f ? 0x7FFF7FFFu : 0xFFFFFFFFu;
            uint32_t found = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t x = (w[q] ^ pair) & mask;
                found |= (x & 0xFFFFu) == 0 ? 1u << (2 * q) : 0;
                found |= x < 0x10000u ? 2u << (2 * q) : 0;
            }
            return found;
        };
        if (!(set.temperature > 0.0f)) {
            // Greedy: the first of the largest.
            uint32_t first = 0xFFFFFFFFu;
            pieces.each([&](u4_t w, int c) __attribute__((always_inline)) {
                const uint32_t f = matches(w, most);
                if (f) first = min(first, (uint32_t)(c + __builtin_ctz(f)));
            });
            first = over_block_once(first, 0xFFFFFFFFu, s.wave_count, Smaller{});
            if (threadIdx.x == 0) a.put(m, first, 0.0f);
            continue;
        }
        const Scale sc = scale_for(s, most, set.temperature);
        bool counted = false;
        // The last pattern that may have weight; -infinity has none.
        const int last =
            min(P::pattern(most - (float)kLightBin / sc.per) + 2, P::pattern(-INFINITY) - 1);
        if (sc.ordinary()) {
            uint32_t all = 0;
            pieces.each([&](u4_t w, int) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t word = w[q];
                    const s2_t b = __builtin_bit_cast(s2_t, word);
                    const s2_t sign = b >> 15;
                    const s2_t d = (s2_t)0x7FFF - ((b ^ (sign & (s2_t)0x7FFF)) - sign);
                    const uint32_t two = __builtin_bit_cast(uint32_t, d);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t p = e ? two >> 16 : two & 0xFFFFu;
                        if (p <= (uint32_t)last) {
                            atomicAdd(&h.patterns.counts[p >> 1], p & 1 ? 0x10000u : 1u);
                            ++all;
                        }
                    }
                }
            });
            __syncthreads();
            counted = true;
            if (a.V >= 65536) {
                // A pattern that occurs more often than its counter holds takes 65535 or
                // 65536 off the counters' sum each time, which nothing makes up for.
                for (int i = threadIdx.x; i < 32768; i += kT) {
                    const uint32_t v = h.patterns.counts[i];
                    all -= (v & 0xFFFFu) + (v >> 16);
                }
                counted = over_block_once(all, 0u, s.wave_count, Plus{}) == 0;
            }
        }
        if (__builtin_expect(!counted, 0)) {
            sample_searching(s, h.searches, row, sc, set);
            if (threadIdx.x == 0) a.put_found(m, s.found, sc);
            continue;
        }
        P ps = {s, h.patterns, sc};
        u64 kept = ps.weigh(P::pattern(most) >> 6, last >> 6, least_weight(set.min_p));
        if (set.min_p > 0.0f) {
            kept = wave_scan(kept, (u64)0, Plus{});
            if (lane == 63) s.slots[2][wave] = kept;
        }
        __syncthreads();
        ps.sum_up();
        if (wave == 0) {
            u64 Z;
            uint32_t n;
            ps.begin(Z, n);
            // the first to reach a sum is the r-th of a pattern's equal logits
            auto rank = [](const Place& at, u64 goal) __attribute__((always_inline)) {
                const u64 x = goal - at.before;
                u64 r = (u64)((double)x / (double)at.weight);  // off by one at most
                r += r * at.weight < x ? 1 : 0;
                r += r * at.weight < x ? 1 : 0;
                return r - ((r - 1) * at.weight >= x ? 1 : 0);
            };
            if (set.top_k > 0 && (uint32_t)set.top_k < n) {
                const Place at = ps.template find<true>((u64)set.top_k);
                Z = at.before + ((u64)set.top_k - at.before_count) * at.weight;
            }
            if (set.top_p < 1.0f) {
                const u64 goal = least_sum((double)set.top_p * (double)Z, false, Z);
                const Place at = ps.template find<false>(goal);
                Z = at.before + rank(at, goal) * at.weight;
            }
            if (set.min_p > 0.0f)
                Z = min(Z, from_lane(wave_scan(lane < kWaves ? s.slots[2][lane] : 0, (u64)0, Plus{}),
                                     63));
            const u64 goal = least_sum((double)set.u * (double)Z, true, Z);
            const Place at = ps.template find<false>(goal);
            if (lane == 0) {
                s.found.sum = Z;
                s.found.logit = P::value(at.d);
                s.before_count = rank(at, goal);
                s.flag = at.count == 1;
            }
        }
        __syncthreads();
        // The r-th one by index.
        const float l = s.found.logit;
        if (s.flag) {
            pieces.each([&](u4_t w, int c) __attribute__((always_inline)) {
                const uint32_t f = matches(w, l);
                if (f) s.found.index = c + __builtin_ctz(f);
            });
        } else {
            const uint32_t r = (uint32_t)s.before_count;
            pieces.each([&](u4_t w, int c) __attribute__((always_inline)) {
                const uint32_t n =
                    wave_scan((uint32_t)__builtin_popcount(matches(w, l)), 0u, Plus{});
                if (lane == 63) h.matches[c / (64 * 8)] = n;
            });
            __syncthreads();
            // The 64 pieces that hold it: each lane sums a stretch of theirs.
            const int entries = (a.V + 64 * 8 - 1) / (64 * 8), per = (entries + kT - 1) / kT;
            const int e0 = min((int)threadIdx.x * per, entries), e1 = min(e0 + per, entries);
            uint32_t mine = 0;
            for (int e = e0; e < e1; ++e) mine += h.matches[e];
            uint32_t upto = (uint32_t)running_sum(mine, s.slots[3]) - mine;
            for (int e = e0; e < e1; ++e) {
                const uint32_t n = h.matches[e];
                if (upto < r && r <= upto + n) {
                    s.bin = e;
                    s.flag = (int)(r - upto);
                }
                upto += n;
            }
            __syncthreads();
            if (wave == 0) {
                const int c = (s.bin * 64 + lane) * 8;
                uint32_t f = matches(row.piece(c), l);
                const uint32_t own = __builtin_popcount(f);
                const uint32_t sum = wave_scan(own, 0u, Plus{});
                uint32_t left = (uint32_t)s.flag;
                if (sum >= left && sum - own < left) {
                    for (left -= sum - own; left > 1; --left) f &= f - 1;
                    s.found.index = c + __builtin_ctz(f);
                }
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) a.put_found(m, s.found, sc);
    }
}

// Few long rows: pieces of kT * 16 bytes, a workgroup each, in three launches, with a
// row's histogram and list in the workspace.
struct Space {
    Single hist;
    u64 list[kList];
    u64 kept;
    uint32_t listed, done;  // entries of the list; workgroups that have added theirs
    uint32_t first;         // of the largest logits (greedy)
    float most;
};
struct Spaces {
    Space* rows;
    uint32_t* most;  // of each piece (order_of): [M][pieces], the largest for a NaN
    int pieces;
};

// A piece of a row.
template <class E>
struct Piece {
    typedef Row<E, false> R;
    typedef typename R::L L;
    R row;
    u4_t bits;
    int c;
    __device__ __forceinline__ Piece(const SampleArgs& a, int64_t m, int p)
        : row{static_cast<const typename R::Bits*>(a.logits) + m * a.ld, a.V, nullptr},
          c((p * kT + (int)threadIdx.x) * R::W) {
        bits = row.piece(c);
    }
    template <class Fn>
    __device__ __forceinline__ void each(Fn&& f) const {
        row.visit(bits, c, f);
    }
};

// The largest logit of each piece; the spaces cleared.  (1 x 131072 fp32, top-k 50: 2.4,
// 3.5 and 8.5 us in the three launches: latency, the last one with one workgroup at its
// end that sorts and sums.)
template <class E>
__global__ __launch_bounds__(kT) void piece_most_kernel(const SampleArgs a, const Spaces ws) {
    __shared__ uint32_t slots[kT / 64];
    const int p = blockIdx.x;
    const int64_t m = blockIdx.y;
    const Piece<E> piece(a, m, p);
    Space& space = ws.rows[m];
    for (int i = p * kT + threadIdx.x; i < kBins; i += ws.pieces * kT) space.hist.sum[i] = 0;
    if (p == 0 && threadIdx.x == 0) {
        space.kept = 0;
        space.listed = 0;
        space.done = 0;
        space.first = 0xFFFFFFFFu;
    }
    typename Logits<E>::Ends ends;
    ends.add(piece.bits);
    const uint32_t most = over_block_once(ends.order(), 0u, slots, Larger{});
    if (threadIdx.x == 0) ws.most[m * ws.pieces + p] = most;
}

// The largest logit of a row, NaN where it has one.
__device__ __forceinline__ float most_of_row(uint32_t* slots, const Spaces& ws, int64_t m) {
    uint32_t most = 0;
    for (int i = threadIdx.x; i < ws.pieces; i += kT) most = max(most, ws.most[m * ws.pieces + i]);
    return logit_in_order(over_block_once(most, 0u, slots, Larger{}));
}

template <class E>
__global__ __launch_bounds__(kT) void piece_histogram_kernel(const SampleArgs a, const Spaces ws) {
    __shared__ Shared s;
    __shared__ Single h;
    const int64_t m = blockIdx.y;
    const Piece<E> piece(a, m, blockIdx.x);
    Space& space = ws.rows[m];
    const Settings set = a.settings(m);
    fill_powers(s);
    clear(h);
    const float most = most_of_row(s.fewest, ws, m);
    if (blockIdx.x == 0 && threadIdx.x == 0) space.most = most;
    if (!(most > -INFINITY)) return;
    if (!(set.temperature > 0.0f)) {
        uint32_t first = 0xFFFFFFFFu;
        piece.each([&](int i, float l) __attribute__((always_inline)) {
            if (l == most) first = min(first, (uint32_t)i);
        });
        if (first != 0xFFFFFFFFu) atomicMin(&space.first, first);
        return;
    }
    const Scale sc = scale_for(s, most, set.temperature);
    if (!one_histogram(sc, set, a.V)) return;
    const bool counts = by_counts(set, a.V);
    u64 kept = 0;
    add_to_histogram(h, piece, sc, set, counts, kept);
    if (set.min_p > 0.0f && !counts) {
        kept = over_block_once(kept, (u64)0, s.slots[3], Plus{});
        if (threadIdx.x == 0 && kept != 0) atomicAdd(&space.kept, kept);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kT) {
        if (counts) {
            if (h.count[i] != 0) atomicAdd(&space.hist.count[i], h.count[i]);
        } else if (h.sum[i] != 0) {
            atomicAdd(&space.hist.sum[i], h.sum[i]);
        }
    }
}

// Gathers the wanted elements; the workgroup of a row that is done last takes the
// token.
template <class E>
__global__ __launch_bounds__(kT) void piece_gather_kernel(const SampleArgs a, const Spaces ws) {
    __shared__ Shared s;
    __shared__ union {
        Single single;
        Searches searches;
    } h;
    const int64_t m = blockIdx.y;
    const Piece<E> piece(a, m, blockIdx.x);
    Space& space = ws.rows[m];
    const Settings set = a.settings(m);
    const float most = space.most;
    if (!(most > -INFINITY) || !(set.temperature > 0.0f)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) {
            if (most > -INFINITY)
                a.put(m, space.first, 0.0f);
            else
                a.put(m, -1, __builtin_nanf(""));
        }
        return;
    }
    fill_powers(s);
    const Scale sc = scale_for(s, most, set.temperature);
    const bool counts = by_counts(set, a.V);
    bool searching = !one_histogram(sc, set, a.V);
    Wanted want = {};
    uint32_t n = 0;
    if (!searching) {
        for (int i = threadIdx.x; i < kBins; i += kT) h.single.sum[i] = space.hist.sum[i];
        if (threadIdx.x == 0) s.listed = 0;
        __syncthreads();
        want = wanted_bins(s, h.single, counts, set, space.kept);
        gather_wanted(s, piece, sc, want);
        n = s.listed;
        if (n > 0) {
            if (threadIdx.x == 0) s.flag = (int)atomicAdd(&space.listed, n);
            __syncthreads();
            const uint32_t to = (uint32_t)s.flag;
            if (threadIdx.x < n && threadIdx.x + to < kList)
                __hip_atomic_store(&space.list[to + threadIdx.x], s.list[threadIdx.x],
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    // This workgroup's entries are written before it counts itself, and the last
    // one's reads come after its count: every wave waits until its own stores, which go
    // past its CU's cache, are done; then one lane counts for all.  (The barrier alone
    // waits for LDS, and the lane's release for its own wave's stores.  A release of every
    // wave took 10 us.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        s.bin = __hip_atomic_fetch_add(&space.done, 1u, __ATOMIC_ACQ_REL,
                                       __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)ws.pieces - 1;
    __syncthreads();
    if (!s.bin) return;
    if (!searching) {
        n = __hip_atomic_load(&space.listed, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        searching = n > kList;
    }
    if (searching) {
        const Row<E, false> row = {piece.row.ptr, a.V, nullptr};
        sample_searching(s, h.searches, row, sc, set);
    } else {
        if (threadIdx.x < n)
            s.list[threadIdx.x] = __hip_atomic_load(&space.list[threadIdx.x], __ATOMIC_RELAXED,
                                                    __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        sample_list(s, n, counts, want, sc, set);
    }
    if (threadIdx.x == 0) a.put_found(m, s.found, sc);
}

// Whether rows are cut into pieces: up to 16 of them.  In pieces / a workgroup each, us:
//                        top-k 50                    top-p 0.9
//     rows           8      16      32      64      16      32      64
//     65536 fp32   18/22   21/23   32/24   53/24   23/34   36/37   60/38
//     131072       21/35   31/35   50/35   92/36   40/60   63/61  114/61
//     65536 bf16   17/22   18/22   22/23   32/23   24/29   28/30   44/30
//     131072       18/29   21/30   32/31   54/31   32/38   45/39   74/39
// Rows that the list does not take are left to the last workgroup, which searches them
// alone: 1 x 131072 fp32 98 us with top-k 1000 and 222 crowded (temperature 8), bf16 crowded
// 225 where patterns take 37.
bool cuts(int dtype, int64_t M, int64_t V) {
    const int64_t bytes = V * (dtype == PGEMM_F32 ? 4 : 2);
    return bytes > 32768 && M <= 16;
}

// Whether top-k keeps more than the histogram's counts find.
bool keeps_many(const SampleCall& c) {
    return !c.top_k.each && c.top_k.value > kSmallK && c.top_k.value < c.V && c.V >= 8192;
}
// Whether rows of 16 bits, a workgroup each, go by patterns: long ones, and shorter ones
// of which top-k keeps many.  Not where all of them keep up to kSmallK.  256 rows of
// bf16, us, by histogram / by patterns:
//     V         top-k 50    top-p 0.9   top-k 1000   crowded (temperature 8)
//     8192      12 / 19     12 / 18     26 / 18      20 / 18
//     32768     20 / 26     26 / 25     51 / 26      73 / 25
//     65536     27 / 34     38 / 33     78 / 33      136 / 33
//     131072    40 / 50     63 / 50     132 / 50     298 / 50
// (By patterns also where each row has a top-k of its own, which the host does not know:
// 65536 with 50 in every row 36 instead of 29.)
bool by_patterns(const SampleCall& c) {
    const int64_t k = c.top_k.each ? 0 : c.top_k.value;
    return keeps_many(c) || (c.V >= 32768 && !(k > 0 && k <= kSmallK));
}

template <class E>
hipError_t launch_pieces(const SampleArgs& a, const Spaces& ws, hipStream_t stream) {
    const dim3 grid((unsigned)ws.pieces, (unsigned)a.M);
    hipLaunchKernelGGL(piece_most_kernel<E>, grid, dim3(kT), 0, stream, a, ws);
    hipLaunchKernelGGL(piece_histogram_kernel<E>, grid, dim3(kT), 0, stream, a, ws);
    hipLaunchKernelGGL(piece_gather_kernel<E>, grid, dim3(kT), 0, stream, a, ws);
    return hipGetLastError();
}

template <class E>
hipError_t launch(const SampleCall& c, Arena& ar, hipStream_t stream) {
    Spaces ws = {};
    const bool cut = cuts(c.dtype, c.M, c.V);
    if (cut) {
        ws.pieces = (int)((c.V + kT * Logits<E>::kWidth - 1) / (kT * Logits<E>::kWidth));
        ws.rows = static_cast<Space*>(ar.take(c.M * (int64_t)sizeof(Space)));
        ws.most = static_cast<uint32_t*>(ar.take(c.M * ws.pieces * 4));
    }
    if (ar.dry()) return hipSuccess;
    const unsigned blocks = (unsigned)(c.M < (1 << 20) ? c.M : 1 << 20);
    const SampleArgs a = {c.logits, c.ld, c.u, c.temperature, c.top_p, c.min_p, c.top_k,
                          c.tokens, c.logprobs, c.M, (int)c.V};
    // (16-bit rows of which top-k keeps many would be left to one workgroup in the end.)
    if (cut && !(!std::is_same<E, F32>::value && keeps_many(c)))
        return launch_pieces<E>(a, ws, stream);
    if constexpr (!std::is_same<E, F32>::value) {
        auto go = [&](auto held) {
            hipLaunchKernelGGL((sample_patterns_kernel<E, decltype(held)::value>), dim3(blocks),
                               dim3(kT), 0, stream, a);
            return hipGetLastError();
        };
        if (by_patterns(c)) {
            const int64_t rounds = (c.V + kT * 8 - 1) / (kT * 8);
            if (rounds <= 2) return go(std::integral_constant<int, 2>{});
            if (rounds <= 4) return go(std::integral_constant<int, 4>{});
            if (rounds <= 8) return go(std::integral_constant<int, 8>{});
            return go(std::integral_constant<int, 0>{});
        }
    }
    const int64_t bytes = (c.V + Logits<E>::kWidth - 1) / Logits<E>::kWidth * 16;
    auto go = [&](auto held) {
        hipLaunchKernelGGL((sample_kernel<E, decltype(held)::value>), dim3(blocks), dim3(kT), 0,
                           stream, a);
    };
    if (bytes <= 32768) go(std::integral_constant<int, 32768>{});
    else if (bytes <= 131072) go(std::integral_constant<int, 131072>{});
    else go(std::integral_constant<int, 0>{});
    return hipGetLastError();
}

}  // namespace

hipError_t sample(const SampleCall& c, Arena& ar, hipStream_t stream) {
    if (c.M == 0) return hipSuccess;
    if (c.dtype == PGEMM_F32) return launch<F32>(c, ar, stream);
    return c.dtype == PGEMM_BF16 ? launch<BF16>(c, ar, stream) : launch<F16>(c, ar, stream);
}

}  // namespace layer
}  // namespace pgemm
