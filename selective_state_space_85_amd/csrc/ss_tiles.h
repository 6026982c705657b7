// Which tile forms a matrix product, and what a launch of tiles takes of a grid: plain host code,
// shared by the kernels' launchers (ss_gemm.h) and the C ABI's checks.  Internal to the library.
#pragma once

#include <stdint.h>

namespace ssk {
namespace {

enum class Tile { Large, Small, Mini };

constexpr uint32_t kCUs = 256;

inline uint32_t up(int64_t a, int64_t b) { return uint32_t((a + b - 1) / b); }

// Number of bm x bn tiles of a rows x cols output.
inline int64_t count(int64_t rows, int64_t cols, int bm, int bn) { return int64_t(up(rows, bm)) * up(cols, bn); }

// The fastest tile for launches of that many tiles of each kind, by what they take at k = 2048 on
// 256 CUs, in units of a round of large tiles (57 us; bf16) or of small ones (98 us; fp32):
// 1024 x 1024, 2048 x 2048 and 4096 x 4096 outputs, bf16: halves 28, 31, 69 us, small 24, 27, 79, mini
// 17, 24, 92; fp32: small 115, 132, 390, mini 86, 139, 451.  n: tiles on the busiest CU.
template <int DT>
inline Tile best_tile(int64_t large, int64_t small, int64_t mini)
{
    const double ns = double((small + kCUs - 1) / kCUs), nm = double((mini + kCUs - 1) / kCUs);
    if (DT == 0) {
        const double cs = ns == 1 ? 1.35 : ns, cm = nm == 1 ? 0.88 : nm == 2 ? 1.42 : 0.58 * nm;
        return cm < cs ? Tile::Mini : Tile::Small;
    }
    const int64_t rounds = large / kCUs, rest = large % kCUs;
    const double cl = double(rounds) + (rest == 0 ? 0.0 : rest <= kCUs / 2 ? 0.55 : rounds ? 1.0 : 0.75);
    const double cs = ns == 1 ? 0.46 : 0.35 * ns, cm = nm == 1 ? 0.30 : nm == 2 ? 0.42 : 0.20 * nm;
    if (cl <= cs && cl <= cm) return Tile::Large;
    return cm < cs ? Tile::Mini : Tile::Small;
}

// Threads of a launch of those tiles of the kind `t`; halving its last large ones adds less than a
// round of workgroups.
inline int64_t tile_threads(Tile t, int64_t large, int64_t small, int64_t mini)
{
    return t == Tile::Large ? 512 * (large + kCUs) : 256 * (t == Tile::Small ? small : mini);
}

}  // namespace
}  // namespace ssk
