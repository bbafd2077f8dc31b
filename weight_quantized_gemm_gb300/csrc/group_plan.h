// How a product of 4-bit or 16-bit operands (group_gemm.cuh) is cut into tiles; host code only.
#pragma once

#include "experts.h"

namespace qg {
namespace gg {

constexpr int kCh = 128;                           // channels per tile
constexpr int kMaxSplit = 8;

// Tile height and cluster size. A call's time beyond its launch is about
//   rounds * stages / split * (stage of this height) + (last tile's epilogue) + (joining the parts of K),
// rounds = tiles * split / blocks at a time, with the constants below (nanoseconds, fitted to MXFP4 calls;
// a stage is 128 bytes of K in every form, and the constants rank the other forms' heights too).
// Small tiles fill the GPU and end sooner; large ones read the operands fewer times:
//   4096 x 4096, us               M = 100    300    512   1024  |  N = 14336:  M = 64    256    512   1024
//   MXFP4    32 rows                  6.6   14.2   18.3         |                10.9   26.5   50.5
//            128 rows                 7.4    7.7    7.9   12.3  |                 8.3   12.6   17.0   30.7
//            256 rows, two blocks     7.6    9.8    9.9   10.6  |                 8.7   11.0   16.7   23.0
//   NVFP4    32 rows                  6.8   14.8   19.0         |                11.2   27.1   51.7
//            128 rows                 7.5    8.0    8.2   12.9  |                 8.7   13.3   18.0   32.2
//            256 rows, two blocks     9.4   11.9   11.9   12.5  |                10.1   12.8   20.9   29.1
//   16 bits (first column M = 128)
//            32 rows                 17.4   46.2   61.1         |                32.2   91.1  179
//            128 rows                18.2   18.2   18.8   34.1  |                23.1   35.5   50.3   96.2
//            256 rows, two blocks    17.8   22.2   22.4   23.2  |                23.5   27.0   42.5   65.1
// The rule's choice is the fastest of its column or within 2 % of it (M = 128 in 16 bits: 4 %).
// Joining pays for few tiles of long K. 77 x 9728 x 2560, us: MXFP4 11.5 with 32 rows a tile, 9.1 with K in two,
// 8.9 with 128 rows and K in four; NVFP4 11.5, 8.9, 9.2; 16 bits 36.8, 20.6, 17.1. M = 100 of 4096 x 4096 is no
// faster with it. A cluster has one tile, so a split call's tiles must all fit at once. K is cut by powers of two
// (a block's share of the channels is one), which leaves SMs idle: the 86 tiles of 11008 channels run on 86 of
// 152, since 172 blocks would not fit.
struct Choice {
    int bn, split;
    long long tiles;       // at least as many as the call has
};
inline Choice choose(const GroupGemmArgs& a, int fmt) {
    static const struct { int bn, channels, blocks; long long stage, last, join; } kHeights[3] = {
        {32, kCh, 1, 200, 500, 1200}, {128, kCh, 1, 280, 1500, 2500}, {256, 2 * kCh, 2, 360, 4000, 0}};
    const int stages = fmt == GF_F16 || fmt == GF_BF16 ? a.K / 64 : (a.K + 255) / 256;      // 128 bytes of K each
    const long long groups = a.offsets ? (a.M < a.E ? a.M : a.E) : 1;     // that can have rows
    Choice best{};
    long long least = -1;
    for (const auto& h : kHeights) {
        const long long n_tiles = (a.N + h.channels - 1) / h.channels;
        // the dense product's row tiles, or the most that ragged groups make, and about as many as they do
        const long long most = a.offsets ? a.M / h.bn + groups : (a.M + h.bn - 1) / h.bn;
        const long long mean = a.offsets ? (a.M / h.bn + groups / 2 > groups ? a.M / h.bn + groups / 2 : groups) : most;
        for (int split = 1; split <= (h.join ? kMaxSplit : 1); split *= 2) {
            if (split > 1 && (most * n_tiles * split > kTargetSms || stages / split < 2)) break;
            const long long at_once = kTargetSms / (split * h.blocks);
            const long long rounds = (mean * n_tiles + at_once - 1) / at_once;
            const long long t = rounds * ((stages + split - 1) / split) * h.stage + h.last + (split > 1 ? h.join : 0);
            if (least < 0 || t < least) {
                least = t;
                best = {h.bn, split, most * n_tiles};
            }
        }
    }
    return best;
}

// The kernel counts tiles, and the weights' scale tiles, in 32 bits (with room for a step past the last).
// (No height makes more tiles than the lowest, so most calls need no plan here.)
inline bool countable(const GroupGemmArgs& a, int fmt) {
    constexpr long long kMost = 1LL << 30;
    const long long ch_tiles = (a.N + kCh - 1) / kCh;
    if ((long long)a.E * ch_tiles * ((a.K + 63) / 64) > kMost) return false;
    return ((long long)a.M / 32 + (a.offsets ? a.E : 1)) * ch_tiles <= kMost || choose(a, fmt).tiles <= kMost;
}

}  // namespace gg
}  // namespace qg
