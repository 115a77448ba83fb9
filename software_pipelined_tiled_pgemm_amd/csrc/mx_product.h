// The products of microscaled matrices: the tiles of each pair of formats.
#pragma once

#include "mx_tiles.h"

namespace pgemm {
namespace layer {

namespace {
// Tiles: 256 x 256 where both operands' slots fit three times into LDS, 256 x 128 for 8-bit
// elements on both sides (256 x 256 with two slots spilled 38 registers: 1800 TFLOP/s
// instead of 2240 at 4096 x 4096 x 32768).
template <int FX, int FW>
struct MxTiles {
    static constexpr int kBytes = mxp::Frag<FX>::kChunks + mxp::Frag<FW>::kChunks;
    using Big = mxp::Tile<FX, FW, 256, kBytes == 4 ? 128 : 256, kBytes == 4 ? 4 : 2,
                          kBytes == 4 ? 2 : 4, kBytes == 2 ? 4 : 3, 4>;
    using Small = mxp::Tile<FX, FW, 128, 128, 2, 2, kBytes == 2 ? 4 : kBytes == 3 ? 3 : 2, 4>;
};
}  // namespace

}  // namespace layer
}  // namespace pgemm
