// Products of either operand layout with a fused epilogue, for gfx950: the
// LDS-DMA pipeline of gemm_kernels.h (16x16x32 matrix instruction, 5-stage
// ring, copies up to 4 steps of K 32 ahead) for fp16 and bf16 operands whose
// contraction index runs along rows or down columns, followed by an epilogue
// functor on fp32 values.  Included by the layer operators (linear.hip,
// ffn.hip, xent.hip).
//
// A training step needs three products of the same matrices:
//   y  = x . W          x [M,K] rows of K, W [K,N] columns   ("NN")
//   dx = dz . W^T       dz [M,N] rows of N, W [K,N] rows of N ("NT")
//   dW = x^T . dz       x [M,K], dz [M,N], both down M        ("TN")
// so each operand of a product is either K-contiguous (KC: the contraction
// index is the memory-contiguous one) or K-rows (KR: each row of memory holds
// one contraction index).  A KC operand is staged and read like the A of the
// plain GEMM, a KR operand like its B (transposing LDS reads), whichever
// side of the product it is on: the MFMA's row and column operands hold the
// same lane layout.  No operand is transposed in memory.
//
// What bounds it: the matrix cores (a 256x256 tile reads 32 B per clock and
// CU against the 58 B a copy can sustain); at 4096^3 and above the loop runs
// at the chip's power limit, as the plain GEMM does, where a product's first
// launches are 10-20% faster than steady ones.  Measured, bf16 without an
// epilogue's extras, the fastest run of ten launches and the median: 8192^3 758
// and 788 us (1451 and 1395 TFLOP/s); 8192 x 4096 x 4096 NN 198 and 212 (1388 and
// 1297), NT 202 and 212, TN 202 and 214-222.
//
// Registers: the 256x256 tiles use all 256 vector registers of a wave, and some
// spill: in NN 2 (LinearEpi fp16, SumEpi), 5 (GluEpi) or 22 (StorePart, with four
// scratch loads in the loop of 10 steps), in NT the walking StatsEpi 1.

#pragma once

#include <algorithm>

#include "gemm_kernels.h"
#include "layer.h"
#include "layer_math.h"

namespace pgemm {
namespace {
namespace lp {

using dm::BK;

using layer::Args;
using layer::View;

// A descriptor, which is the same in every lane, as the scalar registers that
// a copy takes it in, wherever the compiler keeps it.
__device__ __forceinline__ u32x4 scalar4(u32x4 r) {
#pragma unroll
    for (int c = 0; c < 4; ++c) r[c] = __builtin_amdgcn_readfirstlane(r[c]);
    return r;
}

// The copies of one operand's stage (ROWS x 32 values, 64 * ROWS bytes) by
// NW waves, CP copies of 1 KiB per wave and step.
//  KC: stage [ROWS][32], chunk c of row r at c ^ aswz16(r); copies of steps
//      2j and 2j+1 should be issued in pairs (the two halves of 128-byte
//      lines).
//  KR: stage [32][ROWS], chunk c of row r at c ^ bswz16(r).
template <int ROWS, bool KC, int NW>
struct Operand {
    static constexpr int BYTES = ROWS * BK * 2;
    static constexpr int CP = BYTES / 1024 / NW;
    uint32_t off[CP];
    int kc;  // KC: K coordinate of this lane's chunks
    int ld;
    const uint16_t* base;  // tile origin at K = 0
    int rows_valid;        // KC: rows of the tile inside the operand
    int col0;              // KR: first column of the tile (descriptor size)
    u32x4 fix;             // KC: descriptor over the tile's rows from K = 0
    uint32_t fix_size;     // KR: descriptor size of a full step

    // `origin`: first row (KC) or column (KR) of the tile; `extent`: rows or
    // columns of the operand.  pair_shift > 0 (KR only): the stage's columns
    // come in 64-column groups of 32 columns of the first half matrix and the
    // same 32 of the second, which starts pair_shift columns further on;
    // origin and extent then count columns of one half.
    __device__ __forceinline__ void place(int lane, int wave, View v, int origin, int extent,
                                          int pair_shift) {
        ld = v.ld;
        if constexpr (KC) {
            const int row = (wave * CP) * 16 + (lane >> 2);
            const int c = (lane & 3) ^ dm::aswz16(lane >> 2);
            kc = c * 8;
#pragma unroll
            for (int t = 0; t < CP; ++t) off[t] = (uint32_t)(((row + 16 * t) * ld + c * 8) * 2);
        } else {
#pragma unroll
            for (int t = 0; t < CP; ++t) {
                const int p = (wave * CP + t) * 64 + lane;
                const int row = p / (ROWS / 8);
                const int c = ((p % (ROWS / 8)) ^ dm::bswz16(row)) * 8;
                int col = c, src = c;
                if (pair_shift > 0) {
                    col = (c >> 6) * 32 + (c & 31);
                    src = col + ((c >> 5) & 1) * pair_shift;
                }
                off[t] = (origin + col < extent) ? (uint32_t)((row * ld + src) * 2) : kOOB;
            }
        }
    }
    __device__ __forceinline__ void init(int lane, int wave, View v, int origin, int extent,
                                         int pair_shift) {
        place(lane, wave, v, origin, extent, pair_shift);
        if constexpr (KC) {
            base = v.ptr + (int64_t)origin * ld;
            rows_valid = min(ROWS, extent - origin);
            fix = rsrc_words(base, (int64_t)rows_valid * ld * 2);
        } else {
            base = v.ptr + origin;
            col0 = origin;
            fix_size = (uint32_t)(((int64_t)BK * ld - origin) * 2);
        }
    }
    // Copy t of the step at k0, any part of which may lie past K (zeros).
    __device__ __forceinline__ void general(int t, int K, int k0, uint32_t stage, int wave) const {
        const uint32_t dst = stage + (wave * CP + t) * 1024;
        if constexpr (KC) {
            const u32x4 r = rsrc_words(base + k0, ((int64_t)rows_valid * ld - k0) * 2);
            dma16(scalar4(r), kc < K - k0 ? off[t] : kOOB, dst);
        } else {
            const int kv = min(BK, K - k0);
            const u32x4 r = rsrc_words(base + (int64_t)k0 * ld, ((int64_t)kv * ld - col0) * 2);
            dma16(scalar4(r), off[t], dst);
        }
    }
    // Copy t of a step that lies inside K: k_byte = 2 * k0 (KC), row = the
    // operand at row k0 of the tile's columns (KR).
    __device__ __forceinline__ void fast(int t, uint32_t k_byte, const uint16_t* row,
                                         uint32_t stage, int wave) const {
        const uint32_t dst = stage + (wave * CP + t) * 1024;
        if constexpr (KC) {
            dma16s(scalar4(fix), off[t], k_byte, dst);
        } else {
            const uint64_t a = reinterpret_cast<uint64_t>(row);
            u32x4 r;
            r[0] = (uint32_t)a;
            r[1] = (uint32_t)(a >> 32) & 0xFFFFu;
            r[2] = fix_size;
            r[3] = (uint32_t)kRsrcWord3;
            dma16(scalar4(r), off[t], dst);
        }
    }
    // This lane's byte offset in a stage for block 0 of the wave's rows
    // (columns), which start at w0; block i is 16 rows (columns) further on.
    // A fragment gives lane (r, g) = (l % 16, l / 16) row r of the block and
    // K values 8g .. 8g+7.
    __device__ static __forceinline__ int lane_offset(int w0, int lane) {
        const int g = lane >> 4, r = lane & 15;
        if constexpr (KC) return (w0 + r) * (BK * 2) + (g ^ dm::aswz16(r)) * 16;
        const int row = 8 * g + (r >> 2);
        return row * (ROWS * 2) + (((w0 / 8 + ((r >> 1) & 1)) ^ dm::bswz16(row)) * 16) + (r & 1) * 8;
    }
    // Block i (below 8): in a KR stage its chunks differ from block 0's in
    // the three bits that the swizzle flips, so the offset is an exclusive or.
    __device__ static __forceinline__ half8 read(const char* st, int offset, int i) {
        if constexpr (KC) return *reinterpret_cast<const half8*>(st + offset + i * 16 * (BK * 2));
        const char* q = st + (offset ^ (i << 5));
        const fp16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((LDS_AS fp16x4_t*)q);
        const fp16x4_t hi =
            __builtin_amdgcn_ds_read_tr16_b64_v4f16((LDS_AS fp16x4_t*)(q + 4 * ROWS * 2));
        const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
        return __builtin_bit_cast(half8, u32x4{l2[0], l2[1], h2[0], h2[1]});
    }
};

// E: element type (F16 or BF16 of layer_math.h); AKC, BKC: operand layouts.
template <class E_, int BM_, int BN_, int WM_, int WN_, bool AKC_, bool BKC_>
struct Tile {
    using E = E_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool AKC = AKC_, BKC = BKC_;
    static constexpr int S = 5;
    static constexpr int NW = WM * WN;
    static constexpr int T = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN;
    static constexpr int FM = TM / 16, FN = TN / 16;
    using OpA = Operand<BM, AKC, NW>;
    using OpB = Operand<BN, BKC, NW>;
    static constexpr int A_BYTES = OpA::BYTES;
    static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
    static constexpr int LDS = S * STAGE;
    static constexpr int H = OpA::CP;  // copies of one operand per wave and step
    static_assert(OpB::CP == H && H % 2 == 0, "the copy schedule moves one operand per half-step");
    static_assert(LDS <= 160 * 1024, "LDS of one CU");
    static_assert(FN % 2 == 0, "a step's MFMAs are split by B block");
    // vmcnt thresholds of the two waits of a period (see the copy schedule).
    static constexpr int W0 = BKC ? 2 * H * (S - 3) : H * (2 * S - 5);
    static constexpr int W1 = (BKC || AKC) ? 2 * H * (S - 3) : H * (2 * S - 5);
    static_assert(!BKC || AKC, "layouts NN, NT and TN");
};

// MFMA slot after which copy c of nc goes (see copy_slot of gemm_kernels.h).
template <class TL>
__device__ __forceinline__ constexpr int slot_of_copy(int c, int nc, int ns) {
    return TL::BM == 128 ? ns - 1 - nc + c : (2 * c + 1) * ns / (2 * (nc > 0 ? nc : 1));
}

template <class TL>
struct Product {
    using E = typename TL::E;
    floatx4 acc[TL::FN][TL::FM];
    half8 fa[2][TL::FM], fb[TL::FN];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
            for (int i = 0; i < TL::FM; ++i) acc[j][i] = floatx4{};
    }
    int oa, ob;  // this lane's offsets of A's and B's block 0 in a stage
    __device__ __forceinline__ void place(int wm, int wn, int lane) {
        oa = TL::OpA::lane_offset(wm * TL::TM, lane);
        ob = TL::OpB::lane_offset(wn * TL::TN, lane);
    }
    __device__ __forceinline__ half8 read_a(const char* st, int i) const {
        return TL::OpA::read(st, oa, i);
    }
    __device__ __forceinline__ half8 read_b(const char* st, int j) const {
        return TL::OpB::read(st + TL::A_BYTES, ob, j);
    }
    __device__ __forceinline__ void first_reads(const char* st) {
#pragma unroll
        for (int j = 0; j < TL::FN / 2; ++j) fb[j] = read_b(st, j);
#pragma unroll
        for (int i = 0; i < TL::FM; ++i) fa[0][i] = read_a(st, i);
    }
    // Call c = 0..3 of a period: half c&1 of its step with A buffer c>>1, the
    // order of half16 in gemm_kernels.h (the same sums, bit for bit).
    template <int CALL, int NC, class CopyFn>
    __device__ __forceinline__ void half(const char* rst, CopyFn copy) {
        // A KR operand's block offsets for every slot of the ring would not fit
        // in registers; hiding the offset's value keeps their derivation here.
        if constexpr (!TL::AKC) asm volatile("" : "+v"(oa));
        if constexpr (!TL::BKC) asm volatile("" : "+v"(ob));
        constexpr int HALF = CALL & 1, b = CALL >> 1;
        constexpr int FM = TL::FM, JH = TL::FN / 2;
        constexpr int NS = JH * FM;
        constexpr int NR = HALF == 0 ? JH : FM + JH;
        half8(&na)[FM] = fa[b ^ 1];
#pragma unroll
        for (int q = 0; q < NS; ++q) {
            const int jj = q / FM, ii = q % FM;
            const int j = HALF * JH + jj;
            const int i = (jj & 1) ? FM - 1 - ii : ii;
            acc[j][i] = E::mma(fb[j], fa[b][i], acc[j][i]);
            if (q < NR) {
                if (HALF == 0)
                    fb[JH + q] = read_b(rst, JH + q);
                else if (q == 0)
                    fb[0] = read_b(rst, 0);
                else if (q <= FM)
                    na[q - 1] = read_a(rst, q - 1);
                else
                    fb[q - FM] = read_b(rst, q - FM);
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (q == slot_of_copy<TL>(c, NC, NS)) copy(c);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// Copy schedule.  As in gemm_kernels.h a period of two steps (kt even, kt+1)
// issues the copies of steps kt+S-1 (h = 0, into the slot of kt-1, free
// since the middle of step kt-1) and kt+S (h = 1, into the slot of kt, free
// since the middle of step kt), per half-step (call 0..3):
//         call 0      call 1       call 2       call 3      (H copies each
//   NN    B h=0       A pairs      A pairs      B h=1        unless noted)
//   TN    B h=0       A h=0        A h=1        B h=1
//   NT    -           A pairs, 2H  B pairs, 2H  -
// KC operands are copied in pairs (h = 0, 1 back to back), which need both
// slots free: in NT that leaves calls 1 and 2 for everything (call 3 would
// do too, but a copy issued there has one half-step less to land).
// Waits, counting the copies issued after the last one of the awaited step:
//  middle of step kt, for step kt+1 (h = 1 of period kt+1-S): the (S-3)/2
//  periods between, 4H each, plus call 0 of this one: W0 = H(2S-5) in NN and
//  TN; in NT call 0 is empty: W0 = 2H(S-3).
//  middle of step kt+1, for step kt+2 (h = 0 of period kt+3-S): what follows
//  its last copy in that period, (S-5)/2 periods, and calls 0-2 of this one.
//  NN: 1 + H + 3H + 2H(S-5), waited to 2H(S-3); TN: 2H + 3H + 2H(S-5)
//  = H(2S-5); NT: 1 + 4H + 2H(S-5), waited to 2H(S-3).
// The prologue issues steps 0 .. S-2 in the same order, so the first wait
// (step 0) finds at least W0 later copies.
// Operand side (false: A, true: B), copy index and step parity of copy c of
// call CALL.
template <class TL, int CALL>
struct Plan {
    static constexpr bool NT = TL::AKC && TL::BKC, TN = !TL::AKC && !TL::BKC;
    static constexpr int NC = NT ? ((CALL == 1 || CALL == 2) ? 2 * TL::H : 0) : TL::H;
    static constexpr bool B = NT ? CALL == 2 : (CALL == 0 || CALL == 3);
    __device__ static constexpr int t(int c) {
        return NT ? c >> 1 : (TN || B) ? c : ((CALL - 1) * TL::H + c) >> 1;
    }
    __device__ static constexpr int h(int c) {
        return NT ? c & 1 : B ? (CALL == 3) : TN ? CALL - 1 : c & 1;
    }
};

// The copies of a tile, a and b having been initialised for it.
template <class TL>
struct Copies {
    typename TL::OpA a;
    typename TL::OpB b;
    int64_t astep, bstep;  // elements per step (KR)

    __device__ __forceinline__ void init(int lane, int wave, View va, View vb, int m0, int M, int n0,
                                         int N, int shift) {
        a.init(lane, wave, va, m0, M, 0);
        b.init(lane, wave, vb, n0, N, shift);
        astep = (int64_t)BK * va.ld;
        bstep = (int64_t)BK * vb.ld;
    }
    // Copy c of call CALL for steps (s, s+1) into the stages at LDS addresses
    // se and so; any part may lie past K.
    template <int CALL>
    __device__ __forceinline__ void general(int c, int K, int s, uint32_t se, uint32_t so,
                                            int wave) const {
        using P = Plan<TL, CALL>;
        const int t = P::t(c), h = P::h(c);
        const uint32_t st = h ? so : se;
        if constexpr (P::B)
            b.general(t, K, (s + h) * BK, st + TL::A_BYTES, wave);
        else
            a.general(t, K, (s + h) * BK, st, wave);
    }
    // The same for steps inside K: k_byte, ar, br belong to step s.
    template <int CALL>
    __device__ __forceinline__ void fast(int c, uint32_t k_byte, const uint16_t* ar,
                                         const uint16_t* br, uint32_t se, uint32_t so,
                                         int wave) const {
        using P = Plan<TL, CALL>;
        const int t = P::t(c), h = P::h(c);
        const uint32_t st = h ? so : se;
        if constexpr (P::B)
            b.fast(t, k_byte + h * (BK * 2), br + h * bstep, st + TL::A_BYTES, wave);
        else
            a.fast(t, k_byte + h * (BK * 2), ar + h * astep, st, wave);
    }
    template <int CALL, bool FAST>
    __device__ __forceinline__ void start_call(int e, int K, uint32_t se, uint32_t so,
                                               int wave) const {
#pragma unroll
        for (int c = 0; c < Plan<TL, CALL>::NC; ++c) {
            if constexpr (FAST)
                fast<CALL>(c, (uint32_t)(e * BK * 2), a.base + e * astep, b.base + e * bstep, se, so,
                           wave);
            else
                general<CALL>(c, K, e, se, so, wave);
        }
    }
    template <bool FAST>
    __device__ __forceinline__ void start_all(int K, uint32_t ring, int wave) const {
#pragma unroll
        for (int e = 0; e < TL::S - 1; e += 2) {
            const uint32_t se = ring + e * TL::STAGE, so = se + TL::STAGE;
            start_call<0, FAST>(e, K, se, so, wave);
            start_call<1, FAST>(e, K, se, so, wave);
            start_call<2, FAST>(e, K, se, so, wave);
            start_call<3, FAST>(e, K, se, so, wave);
        }
    }
    // The prologue: steps 0 .. S-2 into slots 0 .. S-2.
    __device__ __forceinline__ void start(int K, uint32_t ring, int wave) const {
        if (K >= (TL::S - 1) * BK)
            start_all<true>(K, ring, wave);
        else
            start_all<false>(K, ring, wave);
    }
};

// One output tile's K loop, its prologue copies having been issued: the
// periods, and the wait for the copies past K.  place(): recomputes the
// copies' per-lane offsets (so that the unrolled loop need not keep them for
// the tail).
template <class TL, int PH, class Place>
__device__ __forceinline__ void run_k(Product<TL>& pr, Copies<TL>& cp, char* smem, int K, int wave,
                                      int tid, Place&& place) {
    constexpr int S = TL::S;
    const uint32_t ring = lds_addr(smem);
    const int nk = (K + BK - 1) / BK;
    wait_vmcnt<TL::W0>();
    __syncthreads();
    pr.first_reads(smem);

    const uint16_t* ar = cp.a.base + (S - 1) * cp.astep;  // rows of step kt+S-1
    const uint16_t* br = cp.b.base + (S - 1) * cp.bstep;
    uint32_t k_byte = (S - 1) * BK * 2;
    auto period = [&](int kt, auto is_fast, auto slot) __attribute__((always_inline)) {
        constexpr bool F = decltype(is_fast)::value;
        const int se = slot;
        const int s1 = dm::wrap_slot<S>(se + 1), s2 = dm::wrap_slot<S>(se + 2);
        const int s4 = dm::wrap_slot<S>(se + S - 1);
        const uint32_t st4 = ring + s4 * TL::STAGE, st5 = ring + se * TL::STAGE;
        auto copy = [&](auto call) __attribute__((always_inline)) {
            constexpr int CALL = decltype(call)::value;
            return [&](int c) __attribute__((always_inline)) {
                if constexpr (F)
                    cp.template fast<CALL>(c, k_byte, ar, br, st4, st5, wave);
                else
                    cp.template general<CALL>(c, K, kt + S - 1, st4, st5, wave);
            };
        };
        const std::integral_constant<int, 0> c0;
        const std::integral_constant<int, 1> c1;
        const std::integral_constant<int, 2> c2;
        const std::integral_constant<int, 3> c3;
        dm::half_priority<PH, 0>();
        pr.template half<0, Plan<TL, 0>::NC>(smem + se * TL::STAGE, copy(c0));
        wait_vmcnt<TL::W0>();
        __syncthreads();  // step kt+1 published, slot se released
        if constexpr (PGEMM_POISON_LDS) {
            poison_stage<TL::STAGE, TL::T>(smem + se * TL::STAGE, tid);
            __syncthreads();
        }
        dm::half_priority<PH, 1>();
        pr.template half<1, Plan<TL, 1>::NC>(smem + s1 * TL::STAGE, copy(c1));
        dm::half_priority<PH, 2>();
        pr.template half<2, Plan<TL, 2>::NC>(smem + s1 * TL::STAGE, copy(c2));
        wait_vmcnt<TL::W1>();
        __syncthreads();  // step kt+2 published, slot s1 released
        if constexpr (PGEMM_POISON_LDS) {
            poison_stage<TL::STAGE, TL::T>(smem + s1 * TL::STAGE, tid);
            __syncthreads();
        }
        dm::half_priority<PH, 3>();
        pr.template half<3, Plan<TL, 3>::NC>(smem + s2 * TL::STAGE, copy(c3));
        ar += 2 * cp.astep;
        br += 2 * cp.bstep;
        k_byte += 2 * BK * 2;
        return s2;
    };
    const int fast_end = K / BK - S;  // kt < fast_end <=> step kt+S is a full step
    int kt = 0;
    for (; kt + 2 * (S - 1) < fast_end && kt + 2 * (S - 1) < nk; kt += 2 * S)
        dm::ring_pass<S>(
            [&](auto j, auto slot) __attribute__((always_inline)) {
                period(kt + 2 * decltype(j)::value, std::true_type{}, slot);
            },
            std::make_integer_sequence<int, S>{});
    place();
    int se = 0;
    for (; kt < fast_end && kt < nk; kt += 2) se = period(kt, std::true_type{}, se);
    for (; kt < nk; kt += 2) se = period(kt, std::false_type{}, se);
    if constexpr (PH >= 0) __builtin_amdgcn_s_setprio(0);
    wait_vmcnt<0>();  // the copies past the end of K
}

// Epilogue of a tile, straight from the accumulators.  Lane (r, g) = (l % 16,
// l / 16) of block (j, i) holds row 16 i + r, columns 16 j + 4 g .. + 3 of the
// wave's part.  Exchanging the odd 16-lane rows of block j with the even ones
// of block j + 1 (one v_permlane16_swap per register) leaves every lane with
// 8 consecutive columns, 16 (j + g % 2) + 8 (g / 2) .. + 7, of one row: a
// functor's loads and stores are 16 bytes a lane, 64 bytes a row, with no LDS
// and no barrier.
//
// Functors on chunks of 8 fp32 values (columns col .. col + nv - 1 of a row, nv <
// 8 only at the matrix's edge).  epi.from(m0) is the functor for the tile whose
// first row is m0; row counts from there:
//   kPlain:  f(row, col, nv, v, column, aux)
//   kPaired: f(row, col, nv, first half's v, second half's v, column, aux)
// with column = epi.column(col, nv), what a column chunk needs (bias), and aux
// = epi.load(row, col, nv), what the functor reads of memory for the chunk;
// these loads are issued kAhead chunks before their use, since a wait for
// memory per chunk would dominate.  epi.with<STREAM>(run) calls run(f) once with
// the functor proper, so that what is the same for all chunks (the activation,
// whether stores go past the caches) is decided before the first one;
// epi.aligned() says that chunks do not straddle 16-byte boundaries.  With kRedo f
// returns whether the chunk needs more than the functor of whole tiles
// (STREAM) does: such a tile is done again with the other one, in drain_edge.
// Functors on rows (kRows) see the accumulators themselves (see drain_rows).
enum EpiKind { kPlain, kPaired, kRows };
struct Nothing {};

__device__ __forceinline__ void swap_rows16(float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                    __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];  // (a bit_cast of an element takes element 0)
    a = __builtin_bit_cast(float, x);
    b = __builtin_bit_cast(float, y);
}

// 8 consecutive columns per lane out of two neighbouring blocks.
__device__ __forceinline__ void chunk8(const floatx4& a, const floatx4& b, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[q] = a[q];
        v[4 + q] = b[q];
        swap_rows16(v[q], v[4 + q]);
    }
}

// A tile inside the matrix whose chunks are aligned.  Not 0 where the functor
// (kRedo) found a chunk that it cannot do here.
template <class TL, class Acc, class Epi>
__device__ __forceinline__ uint32_t drain_full(const Acc& pr, const int row00, int col0,
                                               const Epi epi) {
    constexpr bool PAIR = Epi::kind == kPaired;
    constexpr int JP = TL::FN / (PAIR ? 4 : 2);  // column chunks per lane
    constexpr int FM = TL::FM;
    constexpr int AHEAD = Epi::kAhead < FM ? Epi::kAhead : FM;
    static_assert(!PAIR || TL::TN == 64, "32 columns of each half per wave");
    uint32_t redo = 0;
    epi.template with<true>([&](const auto& f) __attribute__((always_inline)) {
#pragma unroll
        for (int jp = 0; jp < JP; ++jp) {
            const int col = col0 + 32 * jp;
            const auto column = epi.column(col, 8);
            decltype(epi.load(0, 0, 0)) aux[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) aux[i] = epi.load(row00 + 16 * i, col, 8);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                // Hidden from the compiler, so that it does not keep the
                // addresses of all chunks in registers.
                int row0 = row00;
                asm volatile("" : "+v"(row0));
                const int row = row0 + 16 * i;
                const auto now = aux[i % AHEAD];
                if (i + AHEAD < FM) aux[i % AHEAD] = epi.load(row + 16 * AHEAD, col, 8);
                float v[8];
                chunk8(pr.acc[2 * jp][i], pr.acc[2 * jp + 1][i], v);
                if constexpr (PAIR) {
                    float u[8];
                    chunk8(pr.acc[2 * jp + 2][i], pr.acc[2 * jp + 3][i], u);
                    f(row, col, 8, v, u, column, now);
                } else if constexpr (Epi::kRedo) {
                    redo |= f(row, col, 8, v, column, now);
                    asm volatile("" : "+v"(redo));
                } else {
                    f(row, col, 8, v, column, now);
                }
                __builtin_amdgcn_sched_barrier(0);  // bounds what is in registers at once
            }
        }
    });
    return redo;
}

// A tile at the matrix's edge, of unaligned rows, or done again (kRedo): the
// accumulators go through the ring in bands of rows (half of each wave's at a
// time where the tile does not fit), and a loop over the band's chunks checks
// each against the edge.  (Checked chunks
// unrolled like drain_full's made the code of both so large that the
// registers of the K loop suffered.)  16-byte chunk c of LDS row r sits at
// (c & 1) * CH/2 + ((c >> 1) ^ (r mod CH/2)): the two halves of 8 columns are
// read from the two halves of the row, consecutive lanes consecutive chunks.
template <class TL, class Acc, class Epi>
__device__ __forceinline__ void drain_edge(char* smem, const Acc& pr, int rows, int N,
                                           int n0, int tid, int wm, int wn, const Epi epi) {
    constexpr bool PAIR = Epi::kind == kPaired;
    constexpr int CH = TL::BN / 4, ROWB = TL::BN * 4;
    constexpr int NB = TL::BM * ROWB <= TL::LDS ? 1 : 2;
    constexpr int RB = TL::BM / NB, WR = TL::TM / NB, IB = TL::FM / NB;
    static_assert(RB * ROWB <= TL::LDS && TL::FM % NB == 0, "a band fits in the ring");
    constexpr int LPR = (PAIR ? TL::BN / 2 : TL::BN) / 8;  // threads per row
    constexpr int STEP = TL::T / LPR;                      // rows per pass
    auto pos = [](int c, int row) {
        return row * ROWB + ((c & 1) * (CH / 2) + ((c >> 1) ^ (row & (CH / 2 - 1)))) * 16;
    };
    auto read8 = [&](int c, int row, float(&v)[8]) __attribute__((always_inline)) {
        const floatx4 lo = *reinterpret_cast<const floatx4*>(smem + pos(2 * c, row));
        const floatx4 hi = *reinterpret_cast<const floatx4*>(smem + pos(2 * c + 1, row));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[q] = lo[q];
            v[4 + q] = hi[q];
        }
    };
    const int r = tid & 15, g = (tid >> 4) & 3;
    const int cl = tid % LPR;
    const int col = n0 + cl * 8, nv = min(8, N - col);
    epi.template with<false>([&](const auto& f) __attribute__((always_inline)) {
#pragma unroll
        for (int p = 0; p < NB; ++p) {
            __syncthreads();  // the ring, or the band before, has been read
#pragma unroll
            for (int j = 0; j < TL::FN; ++j)
#pragma unroll
                for (int ii = 0; ii < IB; ++ii)
                    *reinterpret_cast<floatx4*>(
                        smem + pos((wn * TL::TN + 16 * j) / 4 + g, wm * WR + 16 * ii + r)) =
                        pr.acc[j][p * IB + ii];
            __syncthreads();
            if (nv > 0) {
                const auto column = epi.column(col, nv);
#pragma unroll 1
                for (int l = tid / LPR; l < RB; l += STEP) {
                    const int row = (l / WR) * TL::TM + p * WR + l % WR;
                    if (row >= rows) continue;
                    const auto aux = epi.load(row, col, nv);
                    float v[8];
                    if constexpr (PAIR) {
                        const int c = (cl >> 2) * 8 + (cl & 3);  // the first half's chunk
                        float u[8];
                        read8(c, l, v);
                        read8(c + 4, l, u);
                        f(row, col, nv, v, u, column, aux);
                    } else {
                        read8(cl, l, v);
                        f(row, col, nv, v, column, aux);
                    }
                }
            }
        }
    });
}

// Acc: what holds the accumulators acc[FN][FM] of a wave.
template <class TL, class Acc, class Epi>
__device__ __forceinline__ void drain_epi(char* smem, const Acc& pr, int M, int N, int m0, int n0,
                                          int tid, int wm, int wn, const Epi& epi) {
    constexpr bool PAIR = Epi::kind == kPaired;
    constexpr int COLS = PAIR ? TL::BN / 2 : TL::BN;
    if (m0 + TL::BM <= M && n0 + COLS <= N && epi.aligned()) {
        const int r = tid & 15, g = (tid >> 4) & 3;
        const uint32_t redo =
            drain_full<TL>(pr, wm * TL::TM + r,
                           n0 + wn * (PAIR ? 32 : TL::TN) + 16 * (g & 1) + 8 * (g >> 1), epi.from(m0));
        if constexpr (Epi::kRedo) {
            // Does any wave ask for the tile once more?  A word per wave in LDS.
            uint32_t* const asked = reinterpret_cast<uint32_t*>(smem);
            const bool mine = __any(redo != 0);
            __syncthreads();  // every wave is done with the ring
            if ((tid & 63) == 0) asked[tid >> 6] = mine;
            __syncthreads();
            bool any = false;
#pragma unroll
            for (int w = 0; w < TL::NW; ++w) any |= asked[w] != 0;
            if (any) {
                wait_vmcnt<0>();  // the first pass's stores, before any wave's second ones
                drain_edge<TL>(smem, pr, M - m0, N, n0, tid, wm, wn, epi.from(m0));
            }
        }
    } else {
        drain_edge<TL>(smem, pr, M - m0, N, n0, tid, wm, wn, epi.from(m0));
    }
}

// Row functors: each row of the tile is reduced over its columns, first in
// the lanes that hold it (values past column N are passed as -infinity), then
// over the 4 lanes (r, 0..3), then over the wave columns through LDS.
//   Acc a = epi.reduce<FN>(row, row < M, column of v[0][0], v), v[j] 16 columns
//   apart;
//   epi.join(a, other);  epi.finish(a, row, tile column).
// Acc is 8 bytes.
template <class TL, class Epi>
__device__ __forceinline__ void drain_rows(char* smem, const Product<TL>& pr, int M, int N, int m0,
                                           int tn, int tid, int wm, int wn, const Epi& epi) {
    typedef typename Epi::Acc Acc;
    static_assert(sizeof(Acc) == 8, "exchanged as two words");
    const int lane = tid & 63;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = tn * TL::BN + wn * TL::TN + 4 * g;
    Acc* const joined = reinterpret_cast<Acc*>(smem);  // [WN][BM]
    const bool whole = tn * TL::BN + TL::BN <= N;
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) {
        const int row = m0 + wm * TL::TM + 16 * i + r;
        float v[TL::FN][4];
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[j][q] = (whole || n0 + 16 * j + q < N) ? pr.acc[j][i][q] : -INFINITY;
        Acc a = epi.template reduce<TL::FN>(row, row < M, n0, v);
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {
            u32x2 w = __builtin_bit_cast(u32x2, a);
            w[0] = __shfl_xor((int)w[0], o, 64);
            w[1] = __shfl_xor((int)w[1], o, 64);
            epi.join(a, __builtin_bit_cast(Acc, w));
        }
        if (g == 0) joined[wn * TL::BM + wm * TL::TM + 16 * i + r] = a;
    }
    __syncthreads();
    for (int k = tid; k < TL::BM; k += TL::T) {
        if (m0 + k >= M) break;
        Acc a = joined[k];
#pragma unroll
        for (int c = 1; c < TL::WN; ++c) epi.join(a, joined[c * TL::BM + k]);
        epi.finish(a, m0 + k, tn);
    }
}

// Functor of a split-K launch: the partial product, rows of part_ld floats.
struct StorePart {
    static constexpr EpiKind kind = kPlain;
    static constexpr bool kWalk = false;
    static constexpr bool kRedo = false;
    static constexpr int kAhead = 1;
    float* part;
    int ld;
    __device__ __forceinline__ StorePart from(int64_t r) const { return {part + r * ld, ld}; }
    __device__ __forceinline__ bool aligned() const { return true; }
    template <bool STREAM, class Run>
    __device__ __forceinline__ void with(Run&& run) const {
        run(*this);
    }
    __device__ __forceinline__ Nothing column(int, int) const { return {}; }
    __device__ __forceinline__ Nothing load(int, int, int) const { return {}; }
    __device__ __forceinline__ void operator()(int row, int col, int nv, const float (&v)[8], Nothing,
                                               Nothing) const {
        // part_ld is a multiple of 8, so whole chunks always fit the row
        float* p = part + (uint32_t)(row * ld + col);
        *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(p + 4) = floatx4{v[4], v[5], v[6], v[7]};
    }
};

// One workgroup per tile; with a functor that says kWalk, a workgroup takes the
// tiles blockIdx.x, blockIdx.x + gridDim.x, ...: as many workgroups as the chip
// holds walk the tiles of a large product (see launch_tiles).  The copies of a
// tile's first steps are issued before the epilogue of the one before it, which
// needs no LDS (kRows: 8 KiB in the slot that the prologue leaves free).  They
// overlap only with what that epilogue does before its first load: loads return
// in order, so a functor that reads memory (StatsEpi: a target per row block)
// waits for these copies first.  The wait for step 0 counts the epilogue's
// stores too, which were issued later, and waits for more than it has to.
template <class TL, class Epi, bool SPLIT>
__global__ __launch_bounds__(TL::T, 1) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(const Args g, const Epi epi) {
    __shared__ __attribute__((aligned(1024))) char smem[TL::LDS];
    constexpr int COLS = Epi::kind == kPaired ? TL::BN / 2 : TL::BN;
    int M = g.M, Kfull = g.K, tiles_m = g.tiles_m;
    if (g.live) {
        const int n = *g.live;
        if constexpr (TL::AKC) {
            M = min(M, n);
            tiles_m = (M + TL::BM - 1) / TL::BM;
        } else {
            Kfull = min(Kfull, n);
        }
    }
    const int tiles = tiles_m * g.tiles_n;
    if ((int)blockIdx.x >= tiles) return;
    const int group_m = min(tiles_m, 4);  // bands of 4 tile rows, as in the plain GEMM
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / TL::WN, wn = wave % TL::WN;
    const uint32_t ring = lds_addr(smem);

    View va = g.a, vb = g.b;
    int K = Kfull;
    if constexpr (SPLIT) {
        const int kb = blockIdx.y * g.chunk;
        K = min(g.chunk, Kfull - kb);
        va.ptr += TL::AKC ? (int64_t)kb : (int64_t)kb * va.ld;
        vb.ptr += TL::BKC ? (int64_t)kb : (int64_t)kb * vb.ld;
    }
    const int shift = Epi::kind == kPaired ? g.pair_shift : 0;

    int blk = blockIdx.x, tm, tn;
    tile_of_block(blk, tiles, tiles_m, g.tiles_n, group_m, tm, tn);
    Product<TL> pr;
    pr.place(wm, wn, lane);
    Copies<TL> cp;
    if (K > 0) {
        cp.init(lane, wave, va, vb, tm * TL::BM, M, tn * COLS, g.N, shift);
        cp.start(K, ring, wave);
    }
    for (;;) {
        const int m0 = tm * TL::BM, n0 = tn * COLS;
        const int tn_now = tn;
        pr.zero();
        if (K > 0) {
            dm::with_priority_group<TL>(wave, [&](auto ph) __attribute__((always_inline)) {
                run_k<TL, decltype(ph)::value>(
                    pr, cp, smem, K, wave, tid, [&]() __attribute__((always_inline)) {
                        int l = lane;
                        asm volatile("" : "+v"(l));
                        cp.a.place(l, wave, va, m0, M, 0);
                        cp.b.place(l, wave, vb, n0, g.N, shift);
                    });
            });
        }
        bool more = false;
        if constexpr (Epi::kWalk) {
            blk += gridDim.x;
            more = blk < tiles;
        }
        if constexpr (Epi::kWalk || Epi::kind == kRows)
            __syncthreads();  // every wave is done with the ring
        // What follows derives its lane values afresh, so that none is kept
        // live across the K loop.
        int tid_d = tid;
        asm volatile("" : "+v"(tid_d));
        if (Epi::kWalk && more) {
            tile_of_block(blk, tiles, tiles_m, g.tiles_n, group_m, tm, tn);
            if (K > 0) {
                cp.init(tid_d & 63, wave, va, vb, tm * TL::BM, M, tn * COLS, g.N, shift);
                cp.start(K, ring, wave);
            }
        }
        if constexpr (SPLIT) {
            const StorePart sp = {g.part + (int64_t)blockIdx.y * g.M * g.part_ld, g.part_ld};
            drain_epi<TL>(smem, pr, M, g.N, m0, n0, tid_d, wm, wn, sp);
        } else if constexpr (Epi::kind == kRows) {
            drain_rows<TL>(smem + (TL::S - 1) * TL::STAGE, pr, M, g.N, m0, tn_now, tid_d, wm, wn,
                           epi);
        } else {
            drain_epi<TL>(smem, pr, M, g.N, m0, n0, tid_d, wm, wn, epi);
        }
        if (!more) break;
    }
}

// Split-K finish: the partials of 8 consecutive outputs added in ascending
// order, 4 in flight, then the epilogue functor; grid-stride over M * ceil(N /
// 8) chunks.  Bound by memory where it is large (4093 x 2048, 2 partials: 17-18
// us for 84 MB, 4.8 TB/s), by its launch for a few rows (3-4 us).
template <class Epi>
__global__ __launch_bounds__(256) void finish_kernel(const float* __restrict__ part, int64_t part_ld,
                                                     int splits, int M, int N, int pair_shift,
                                                     const int* live, const Epi epi) {
    const int cpr = (N + 7) / 8;
    const int64_t total = (int64_t)(live ? min(M, *live) : M) * cpr;
    const int64_t slice = (int64_t)M * part_ld;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / cpr);
        const int col = (int)(i - (int64_t)row * cpr) * 8;
        const int nv = min(8, N - col);
        const float* p = part + (int64_t)row * part_ld + col;
        auto sum = [&](const float* src, float(&v)[8]) __attribute__((always_inline)) {
            floatx4 lo = {}, hi = {};
            int s = 0;
            for (; s + 4 <= splits; s += 4) {
                floatx4 l[4], h[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    l[u] = *reinterpret_cast<const floatx4*>(src + (s + u) * slice);
                    h[u] = *reinterpret_cast<const floatx4*>(src + (s + u) * slice + 4);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    lo += l[u];
                    hi += h[u];
                }
            }
            for (; s < splits; ++s) {
                lo += *reinterpret_cast<const floatx4*>(src + s * slice);
                hi += *reinterpret_cast<const floatx4*>(src + s * slice + 4);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = lo[q];
                v[4 + q] = hi[q];
            }
        };
        const Epi at = epi.from(row);
        const auto column = at.column(col, nv);
        const auto aux = at.load(0, col, nv);
        float v[8];
        sum(p, v);
        at.template with<false>([&](const auto& f) __attribute__((always_inline)) {
            if constexpr (Epi::kind == kPaired) {
                float u[8];
                sum(p + pair_shift, u);
                f(0, col, nv, v, u, column, aux);
            } else {
                f(0, col, nv, v, column, aux);
            }
        });
    }
}

// ---- launches ----------------------------------------------------------------

template <class TL, class Epi, bool SPLIT>
hipError_t launch_tiles(Args g, int splits, const Epi& epi, hipStream_t stream) {
    constexpr int COLS = Epi::kind == kPaired ? TL::BN / 2 : TL::BN;
    g.tiles_m = (g.M + TL::BM - 1) / TL::BM;
    g.tiles_n = (g.N + COLS - 1) / COLS;
    // One 256x256 workgroup fills a CU's LDS: at most one per CU, each walking
    // several tiles (a multiple of 8 workgroups keeps tile_of_block's map of
    // tiles to XCDs).
    int grid = g.tiles_m * g.tiles_n;
    if (TL::BM == 256 && Epi::kWalk) {
        const int cus = compute_units();
        if (cus >= 8) grid = std::min(grid, cus & ~7);
    }
    hipLaunchKernelGGL((product_kernel<TL, Epi, SPLIT>), dim3(grid, splits), dim3(TL::T), 0, stream,
                       g, epi);
    return hipGetLastError();
}

template <class E, bool AKC, bool BKC>
struct Tiles {
    // TN: A blocks double-buffered and read through 2 addresses each, so the
    // wave takes 64 rows x 128 columns (16 fragment registers fewer).
    using Big = Tile<E, 256, 256, AKC ? 2 : 4, AKC ? 4 : 2, AKC, BKC>;
    using Small = Tile<E, 128, 128, 2, 2, AKC, BKC>;
};

template <class Epi>
hipError_t launch_finish(const Args& g, int splits, int pair_shift, const int* live,
                         const Epi& epi, hipStream_t stream) {
    const int64_t chunks = (int64_t)g.M * ((g.N + 7) / 8);
    const int64_t blocks = std::min<int64_t>((chunks + 255) / 256, 4096);
    hipLaunchKernelGGL((finish_kernel<Epi>), dim3((unsigned)blocks), dim3(256), 0, stream, g.part,
                       (int64_t)g.part_ld, splits, g.M, g.N, pair_shift, live, epi);
    return hipGetLastError();
}

// One product with its epilogue: a single launch, or partials and a finish.
template <class E, bool AKC, bool BKC, class Epi>
hipError_t launch_product(const Args& g, const layer::Cut& cut, const Epi& epi,
                          hipStream_t stream) {
    using T = Tiles<E, AKC, BKC>;
    if (cut.splits <= 1)
        return cut.big ? launch_tiles<typename T::Big, Epi, false>(g, 1, epi, stream)
                       : launch_tiles<typename T::Small, Epi, false>(g, 1, epi, stream);
    Args p = g;
    if (Epi::kind == kPaired) p.N = g.pair_shift + g.N;  // both halves as plain columns
    const int layout = BKC ? layer::kNT : AKC ? layer::kNN : layer::kTN;
    const hipError_t rc = layer::launch_split(std::is_same<E, BF16>::value ? layer::kBF16
                                                                           : layer::kF16,
                                              layout, p, cut, stream);
    if (rc != hipSuccess) return rc;
    return launch_finish(g, cut.splits, Epi::kind == kPaired ? g.pair_shift : 0,
                         AKC ? g.live : nullptr, epi, stream);
}

}  // namespace lp
}  // namespace
}  // namespace pgemm
