// Host-side plumbing shared by the layer operators (linear, gated block,
// cross entropy): workspace carving, operand packing, the choice of tile and
// split, and the launch interfaces between their sources.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace pgemm {
namespace layer {

// An operand in memory: first element and row pitch in elements.
struct View {
    const uint16_t* ptr;
    int ld;
};

// A product C[M, N] = A . B over K and its tile grid, as the kernels take it.
struct Args {
    View a, b;
    int M, N, K;
    int tiles_m, tiles_n;
    int pair_shift;  // > 0: B's columns are paired (see Operand::place); N counts one half
    int chunk;       // split-K: contraction indices per split
    float* part;     // split-K: partials [split][M][part_ld]
    int part_ld;
    // Where not NULL, device memory with the number of rows in use, at most M
    // (NN, NT) or K (TN): the others are left out.
    const int* live;
};

// Layout of a product's operands (K-contiguous or K-rows).
enum Layout { kNN, kNT, kTN };
enum Dtype { kF16 = 0, kBF16 = 1 };

inline int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Carves the caller's workspace into 256-byte aligned pieces; with a null
// base it only counts, so that one function both sizes a call's workspace
// and uses it.
struct Arena {
    char* base;
    int64_t used;
    void* take(int64_t bytes) {
        void* p = base ? base + used : nullptr;
        used += round_up(bytes, 256);
        return p;
    }
    bool dry() const { return base == nullptr; }
};

// An operand that the pipeline can copy from where it lies: 16-byte aligned
// rows of whole 16-byte pieces.
inline bool direct(const void* p, int64_t ld, int64_t cols) {
    return aligned16(p) && ld % 8 == 0 && cols % 8 == 0;
}

// dst[r][c] = src[r][c], c < cols, zeros up to round_up(cols, 8); dst is
// 16-byte aligned, its pitch a multiple of 8 (layer_common.hip).
hipError_t launch_pack(const uint16_t* src, int64_t ld, uint16_t* dst, int64_t dst_ld, int64_t rows,
                       int64_t cols, hipStream_t stream);

// How a product is cut: 256x256 tiles (8 waves, one workgroup per CU) or
// 128x128 ones (4 waves, two per CU), and the number of K splits.
struct Cut {
    bool big;
    int splits;
    int64_t chunk;  // multiple of 64
};
// The cheapest cut by an estimate of its time (layer_common.hip).  max_splits 1:
// no split (the epilogue needs the whole sum of a tile at once).
Cut choose_cut(int64_t M, int64_t N, int64_t K, int cus, int max_splits);
// Bytes of the partials of a cut (0 without a split).
inline int64_t part_bytes(const Cut& c, int64_t M, int64_t N) {
    return c.splits > 1 ? c.splits * M * round_up(N, 8) * 4 : 0;
}

// The partial products of a split product (layer_split.hip).
hipError_t launch_split(int dtype, int layout, const Args& g, const Cut& cut, hipStream_t stream);

// Column sums: out[c] = sum over `parts` rows of part[r][c], rounded to the
// type (layer_common.hip).
hipError_t launch_column_sum(int dtype, const float* part, int64_t parts, int64_t cols, void* out,
                             hipStream_t stream);

}  // namespace layer
}  // namespace pgemm
