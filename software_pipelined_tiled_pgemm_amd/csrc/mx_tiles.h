// Output tiles of the microscaled product: both operands' elements go straight
// into an LDS ring, as in the 16-bit pipeline (layer_pipe.h), one slot per step of
// 128 columns, and the scales beside it.
//
// A slot holds each operand's rows as pieces of 64 bytes: one (e2m1) or two (e4m3:
// columns 0..63 and 64..127), 16-byte chunk c of row r at c ^ aswz16(r), which
// leaves the reads without bank conflicts.  Lane (r, g) reads chunk g of a piece:
// its elements as the instruction wants them.
//
// Scales: the instruction takes a lane's scale from one byte of a register, the
// same byte in all lanes.  A row's scales of 4 steps are 16 bytes, 4 for each
// step; turned around (4 x 4 bytes, on their way within LDS) each lane's dword
// holds its block's scale for all 4 steps, so a register is read once in 4
// steps and the step picks the byte.
//
// One barrier a step, after the last read of its slot: it releases that slot (the
// copies of step t + S follow at once) and publishes the next step's, whose
// first fragments are read while this step's last blocks are multiplied.
//
//   step t     blocks i = 0 .. FM-P: read the remaining fragments of x;
//              wait for the copies of step t+1; barrier;
//              blocks i = FM-P+1 .. FM-1: copies of step t+S, fragments of t+1
//
// Bound by the copies, LDS reads and multiplications of a step that two waves a SIMD do
// not overlap wholly, and by power.  4096 x 4096 x 32768, normal values, TFLOP/s: e2m1 both
// 4400-4520 (zeros 5900), e4m3 x e2m1 3200, e4m3 both 2240.  4096^3 e2m1 40 us: 27 in its 32
// steps, the rest the first copies and the epilogue, during which nothing is multiplied.
//
// Scales of steps 4u .. 4u+3: copied after the barrier of step 4u-4 (the prologue
// copies those of u = 0), turned after the barrier of 4u-2, read after that of 4u-1.
#pragma once

#include "layer_pipe.h"
#include "mx.h"
#include "mx_math.h"

namespace pgemm {
namespace {
namespace mxp {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// The elements of a lane: 16 bytes (e2m1) or 32 (e4m3).
template <int FORMAT>
struct Frag {
    static constexpr int kChunks = FORMAT == PMX_E2M1 ? 1 : 2;
    static constexpr int kCode = FORMAT == PMX_E2M1 ? 4 : 0;  // the instruction's operand type
    i32x4 c[kChunks];
    __device__ __forceinline__ i32x8 operand() const {
        const i32x4 hi = c[kChunks - 1];  // of 4-bit elements the first half counts
        return {c[0][0], c[0][1], c[0][2], c[0][3], hi[0], hi[1], hi[2], hi[3]};
    }
};

// c + w x^T over 128 columns; BYTE: which byte of the scales' registers.
template <int FW, int FX, int BYTE>
__device__ __forceinline__ floatx4 mma(const Frag<FW>& w, const Frag<FX>& x, floatx4 c, uint32_t sw,
                                       uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.operand(), x.operand(), c,
                                                            Frag<FW>::kCode, Frag<FX>::kCode, BYTE,
                                                            (int)sw, BYTE, (int)sx);
}

using Args = layer::MxArgs;

// ROWS rows of one operand, in PIECES of 64 bytes a step, copied by NW waves.
template <int ROWS, int PIECES, int NW>
struct Copy {
    static constexpr int BYTES = ROWS * 64 * PIECES;
    static constexpr int PER = ROWS / 16 / NW;  // copies of 1 KiB per wave and piece
    static constexpr int CP = PER * PIECES;
    static_assert(ROWS % (16 * NW) == 0, "whole copies per wave");
    uint32_t off[PER];
    u32x4 rsrc;

    // `rows` of the tile lie inside the operand: the descriptor ends behind the last
    // one, and rows past it read as zeros.
    __device__ __forceinline__ void init(int lane, int wave, const uint8_t* base, int64_t ld,
                                         int rows, int row_bytes) {
        const int r = wave * PER * 16 + (lane >> 2);
        const int c = (lane & 3) ^ dm::aswz16(lane >> 2);
#pragma unroll
        for (int t = 0; t < PER; ++t) off[t] = (uint32_t)((r + 16 * t) * (int)ld + c * 16);
        rsrc = lp::scalar4(rsrc_words(base, (int64_t)(min(rows, ROWS) - 1) * ld + row_bytes));
    }
    // Copy c of a step: its elements start at byte k of a row.
    __device__ __forceinline__ void go(int c, uint32_t k, uint32_t stage, int wave) const {
        const int t = c / PIECES, p = c % PIECES;
        dma16s(rsrc, off[t], k + p * 64,
               stage + p * (ROWS * 64) + (wave * PER + t) * 1024);
    }
    __device__ static __forceinline__ int lane_offset(int row0, int lane) {
        const int g = lane >> 4, r = lane & 15;
        return (row0 + r) * 64 + (g ^ dm::aswz16(r)) * 16;
    }
    template <int FORMAT>
    __device__ static __forceinline__ Frag<FORMAT> read(const char* stage, int offset, int i) {
        Frag<FORMAT> f;
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
            f.c[p] = *reinterpret_cast<const i32x4*>(stage + offset + p * (ROWS * 64) + i * 1024);
        return f;
    }
};

template <int FX_, int FW_, int BM_, int BN_, int WM_, int WN_, int S_, int P_>
struct Tile {
    static constexpr int FX = FX_, FW = FW_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int S = S_;  // slots of the ring
    static constexpr int P = P_;  // fragments of x in registers
    static constexpr int NW = WM * WN, T = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    using CX = Copy<BM, Frag<FX>::kChunks, NW>;
    using CW = Copy<BN, Frag<FW>::kChunks, NW>;
    static constexpr int STAGE = CX::BYTES + CW::BYTES;
    static constexpr int RING = S * STAGE;
    static constexpr int LDS = RING + (BM + BN) * 16;
    static constexpr int C = CX::CP + CW::CP;  // copies per wave and step
    static_assert(LDS <= 160 * 1024, "LDS of one CU");
    static_assert(BM + BN <= 64 * NW && BM % 64 == 0, "a wave copies the scales of 64 rows of one side");
    static_assert(FM % P == 0 && P >= 2, "a fragment's register does not depend on the step");
    static_assert(S >= 2 && S <= 4, "the scales land within two steps");
};

// 4 x 4 bytes turned around: dword g of the result holds byte g of each dword.
__device__ __forceinline__ u32x4 turned(const u32x4 d) {
    const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400);  // b0 b0' b1 b1'
    const uint32_t b = __builtin_amdgcn_perm(d[1], d[0], 0x07030602);  // b2 b2' b3 b3'
    const uint32_t c = __builtin_amdgcn_perm(d[3], d[2], 0x05010400);
    const uint32_t e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602);
    return {__builtin_amdgcn_perm(c, a, 0x05040100), __builtin_amdgcn_perm(c, a, 0x07060302),
            __builtin_amdgcn_perm(e, b, 0x05040100), __builtin_amdgcn_perm(e, b, 0x07060302)};
}

template <class TL>
struct Product {
    floatx4 acc[TL::FN][TL::FM];
};

// With lp::StorePart for Epi the contraction is split over blockIdx.y, and the partial
// products go to g.part.
template <class TL, class Epi>
__global__ __launch_bounds__(TL::T, 1) __attribute__((amdgpu_waves_per_eu(2, 2)))
void product_kernel(const Args g, const Epi epi) {
    constexpr bool SPLIT = std::is_same<Epi, lp::StorePart>::value;
    constexpr int FM = TL::FM, FN = TL::FN, P = TL::P, S = TL::S, C = TL::C;
    using CX = typename TL::CX;
    using CW = typename TL::CW;
    __shared__ __attribute__((aligned(1024))) char smem[TL::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / TL::WN, wn = wave % TL::WN;
    int tm, tn;
    tile_of_block(blockIdx.x, g.tiles_m * g.tiles_n, g.tiles_m, g.tiles_n, min(g.tiles_m, 4), tm, tn);
    const int m0 = tm * TL::BM, n0 = tn * TL::BN;
    const int first = SPLIT ? blockIdx.y * g.chunk : 0;
    const int nk = SPLIT ? min(g.chunk, g.steps - first) : g.steps;

    const uint32_t ring = lds_addr(smem);
    char* const scales = smem + TL::RING;
    Product<TL> pr;
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) pr.acc[j][i] = floatx4{};

    if (nk > 0) {
        CX cx;
        CW cw;
        cx.init(lane, wave, g.x + (int64_t)m0 * g.ldx, g.ldx, g.M - m0,
                g.steps * 64 * Frag<TL::FX>::kChunks);
        cw.init(lane, wave, g.w + (int64_t)n0 * g.ldw, g.ldw, g.N - n0,
                g.steps * 64 * Frag<TL::FW>::kChunks);
        // This wave's 64 rows of scales: rows of x, then rows of w.
        const int row_s = wave * 64;
        const bool has_s = row_s < TL::BM + TL::BN, of_x = row_s < TL::BM;
        const int row_o = of_x ? row_s : row_s - TL::BM;
        const int rows_s = of_x ? g.M - m0 - row_o : g.N - n0 - row_o;
        const int64_t ld_s = of_x ? g.ldxs : g.ldws;
        const int bytes_s = (g.steps + 3) / 4 * 16;
        const uint8_t* const base_s = of_x ? g.xs + (int64_t)(m0 + row_o) * g.ldxs
                                           : g.ws + (int64_t)(n0 + row_o) * g.ldws;
        // no rows inside: a descriptor of size 0
        const u32x4 rsrc_s = lp::scalar4(rsrc_words(
            base_s, has_s && rows_s > 0 ? (int64_t)(min(rows_s, 64) - 1) * ld_s + bytes_s : 0));
        const uint32_t off_s = (uint32_t)(lane * (int)ld_s);
        const int groups = (g.steps + 3) / 4, group0 = first / 4;
        // Scales of group u; past the last group the last one's again.
        auto copy_scales = [&](int u) __attribute__((always_inline)) {
            if (has_s)
                dma16s(rsrc_s, off_s, (uint32_t)(min(group0 + u, groups - 1) * 16),
                       ring + TL::RING + row_s * 16);
        };
        auto turn_scales = [&]() __attribute__((always_inline)) {
            if (has_s) {
                u32x4* const p = reinterpret_cast<u32x4*>(scales + (row_s + lane) * 16);
                *p = turned(*p);
            }
        };
        // Copy c of step t (past the last step the last one's again) into slot `to`.
        auto copy = [&](int c, int t, uint32_t to) __attribute__((always_inline)) {
            const uint32_t k = (uint32_t)(first + min(t, nk - 1)) * 64;
            if (c < CX::CP)
                cx.go(c, k * Frag<TL::FX>::kChunks, to, wave);
            else
                cw.go(c - CX::CP, k * Frag<TL::FW>::kChunks, to + CX::BYTES, wave);
        };
        copy_scales(0);
#pragma unroll
        for (int t = 0; t < S; ++t)
#pragma unroll
            for (int c = 0; c < C; ++c) copy(c, t, ring + t * TL::STAGE);

        const int ox = CX::lane_offset(wm * TL::TM, lane), ow = CW::lane_offset(wn * TL::TN, lane);
        Frag<TL::FX> fx[P];
        Frag<TL::FW> fw[2][FN];
        uint32_t sx[FM], sw[FN];
        auto read_x = [&](const char* st, int i) __attribute__((always_inline)) {
            fx[i % P] = CX::template read<TL::FX>(st, ox, i);
        };
        auto read_w = [&](const char* st, int b, int j) __attribute__((always_inline)) {
            fw[b][j] = CW::template read<TL::FW>(st + CX::BYTES, ow, j);
        };
        const char* const sx_at = scales + (wm * TL::TM + (lane & 15)) * 16 + (lane >> 4) * 4;
        const char* const sw_at =
            scales + (TL::BM + wn * TL::TN + (lane & 15)) * 16 + (lane >> 4) * 4;

        wait_vmcnt<S * C>();  // the scales, copied first
        asm volatile("" ::: "memory");  // no LDS access before the wait
        turn_scales();
        wait_vmcnt<(S - 1) * C>();  // step 0
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FM; ++i) sx[i] = *reinterpret_cast<const uint32_t*>(sx_at + i * 256);
#pragma unroll
        for (int j = 0; j < FN; ++j) sw[j] = *reinterpret_cast<const uint32_t*>(sw_at + j * 256);
#pragma unroll
        for (int j = 0; j < FN; ++j) read_w(smem, 0, j);
#pragma unroll
        for (int i = 0; i < P - 1; ++i) read_x(smem, i);

        int slot = 0;
        auto step = [&](int t, auto quarter) __attribute__((always_inline)) {
            constexpr int Q = decltype(quarter)::value;  // t % 4
            constexpr int B = Q & 1;                     // the buffer of w's fragments
            if constexpr (S == 4) slot = Q;  // the loop over t starts at slot 0
            const int next = slot + 1 == S ? 0 : slot + 1;
            const char* const cur = smem + slot * TL::STAGE;
            const char* const nxt = smem + next * TL::STAGE;
            const uint32_t to = ring + slot * TL::STAGE;
            auto block = [&](int i, auto between) __attribute__((always_inline)) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    pr.acc[j][i] = mma<TL::FW, TL::FX, Q>(fw[B][j], fx[i % P], pr.acc[j][i], sw[j],
                                                          sx[i]);
                    between(j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
#pragma unroll
            for (int i = 0; i <= FM - P; ++i)
                block(i, [&](int j) __attribute__((always_inline)) {
                    if (j == 0) read_x(cur, i + P - 1);
                });
            wait_vmcnt<(S - 2) * C>();  // step t + 1
            __syncthreads();            // published; slot of step t released
            if constexpr (PGEMM_POISON_LDS) {
                poison_stage<TL::STAGE, TL::T>(smem + slot * TL::STAGE, tid);
                __syncthreads();
            }
            if (Q == 0) copy_scales(t / 4 + 1);
            if (Q == 2) turn_scales();
            uint32_t nx[FM], nw[FN];
            if (Q == 3) {
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    nx[i] = *reinterpret_cast<const uint32_t*>(sx_at + i * 256);
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    nw[j] = *reinterpret_cast<const uint32_t*>(sw_at + j * 256);
            }
            constexpr int REST = (P - 1) * FN;  // multiplications after the barrier
#pragma unroll
            for (int i = FM - P + 1; i < FM; ++i)
                block(i, [&](int j) __attribute__((always_inline)) {
                    const int n = i - (FM - P + 1), q = n * FN + j;
                    if (q < FN) read_w(nxt, B ^ 1, q);
                    // fragment n's register is free since block FM - P + n
                    if (j == 0) read_x(nxt, n);
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (q == c * REST / C) copy(c, t + S, to);
                });
            if (Q == 3) {
#pragma unroll
                for (int i = 0; i < FM; ++i) sx[i] = nx[i];
#pragma unroll
                for (int j = 0; j < FN; ++j) sw[j] = nw[j];
            }
            slot = next;
        };
        for (int t = 0; t < nk; t += 4) {
            step(t, std::integral_constant<int, 0>{});
            if (t + 1 < nk) step(t + 1, std::integral_constant<int, 1>{});
            if (t + 2 < nk) step(t + 2, std::integral_constant<int, 2>{});
            if (t + 3 < nk) step(t + 3, std::integral_constant<int, 3>{});
        }
        wait_vmcnt<0>();  // the copies past the last step
    }
    int tid_d = tid;
    asm volatile("" : "+v"(tid_d));
    if constexpr (SPLIT) {
        const lp::StorePart sp = {g.part + (int64_t)blockIdx.y * g.M * g.part_ld, g.part_ld};
        lp::drain_epi<TL>(smem, pr, g.M, g.N, m0, n0, tid_d, wm, wn, sp);
    } else {
        lp::drain_epi<TL>(smem, pr, g.M, g.N, m0, n0, tid_d, wm, wn, epi);
    }
}

}  // namespace mxp
}  // namespace
}  // namespace pgemm
