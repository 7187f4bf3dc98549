// i8_forms.h -- which form of the 8-bit product (i8_gemm.hip) a call takes: rules
// on sizes, pitches and alignment, on the host, with no device code, so that a
// host program can ask them.
#pragma once

#include <stdint.h>

namespace mxq {
namespace {

// Row tiles that any offsets can give: every group and the tail may end in a
// tile of its own.
inline int64_t tile_bound(int64_t M, int64_t TM, bool groups, int32_t G) {
    const int64_t full = M / TM;
    if (!groups) return (M + TM - 1) / TM;
    const int64_t parts = int64_t(G) + 1;
    return full + (parts < M ? parts : M);
}

// Row tiles that a grouped grid has room for: an XCD's share is at most a
// ceiling of the covered tiles and one of the tail's.
inline int64_t group_tiles(int64_t tiles_m) { return 8 * ((tiles_m + 7) / 8 + 1); }

// Columns per workgroup: at most 512 workgroups (two of about 64 KiB LDS on
// each CU) while that is 64 at most.  [8192, 8192] with one row: 16 columns
// 13.1 us, 32 19.0, 64 15.2; [14336, 4096]: 16 columns 14.7 us, 32 12.8, 64 12.4.
inline int ring_columns(int64_t N) { return N <= 16 * 512 ? 1 : (N <= 32 * 512 ? 2 : 4); }

// Which kernel.
enum class Kind { kSplit, kStaged, kRing, kPipe };
struct Form {
    Kind kind;
    int ms, ns;                  // kSplit, kRing: 16 rows and 16-column parts of a workgroup; kStaged, kPipe: 64-row, 64-column units
    uint64_t threads;            // of the grid
};

// What the operands allow: whole aligned 16-byte pieces, rows at any byte, rows
// so far apart that a tile's offsets leave 32 bits.
enum class Rows { kPieces, kBytes, kFar };
inline bool far(int64_t lda, int64_t ldb) { return lda >= (1 << 23) || ldb >= (1 << 23); }

// The tile with the least ceil(tiles / 256 CUs) (steps t + 1.2 us), t the time
// of one 128-code step with a tile on each CU.
struct Tile {
    int um, un;                  // 64-row, 64-column units
    double step;                 // us
};
template <int kN>
const Tile& best_tile(const Tile (&tiles)[kN], int64_t M, int64_t N, int64_t K, int64_t groups) {
    const Tile* best = nullptr;
    double least = 0;
    for (const Tile& t : tiles) {
        const int64_t n = groups * ((M + 64 * t.um - 1) / (64 * t.um)) * ((N + 64 * t.un - 1) / (64 * t.un));
        const double cost = double((n + 255) / 256) * (double((K + 127) / 128) * t.step + 1.2);
        if (!best || cost < least) {
            best = &t;
            least = cost;
        }
    }
    return *best;
}

// Row groups in whole pieces, by the mean rows of a group (64 experts of [2048,
// 5120], group sizes spread by e^0.6; us for tiles of 64, 128 and 256 rows):
//   rows   8: 106.3  111.9  126.6  rows  96:        154.7  169.6
//   rows  16: 108.4  112.8  125.5  rows 128:        164.1  175.3
//   rows  24: 133.7  113.4  124.4  rows 192:        217.3  204.4
//   rows  32: 135.1  116.8  131.9  rows 256:        262.9  236.8
//   rows  64:        152.9  137.6  rows 512:        482.1  411.4
// (64 rows to each expert alike: 120.8 and 136.0; the 671 MB of weights alone
// take 108 us at 6.2 TB/s).  The thresholds come from that one shape; few rows
// of few experts make too few tiles of 256 columns (1, 2, 4 and 8 tokens with 4
// picks of these experts: 33, 35, 38 and 47 us, the picked experts' weights
// alone 7, 14, 26 and 46).
//
// Dense in whole pieces: with the times below the choice is the fastest of the
// five tiles at each of the 42 shapes where all were timed (M 32 to 8192; N, K
// 14336 x 4096, 8192 x 8192 and 2048 x 5120).  No tile splits the contraction:
// past the ring's 16 rows each workgroup walks all of it, however few there are
// (16, 17 and 64 rows: [8192, 8192] 14.2, 23.3 and 24.1 us; [1024, 8192] 7.6, 21.4
// and 21.7).
//
// Rows at any byte, dense [8191, 4095] and the same (us for tiles of 64 x 64, 128
// x 64, 128 x 128, 128 x 256; the last form is 16 x 16 split):
//   rows   64: 19.4 24.7 30.9 47.6 30.9    rows  512: 60.2 48.7 36.2 54.3 202
//   rows  128: 20.3 24.6 32.1 51.7 55.2    rows 1024: 116  91.2 73.8 62.3 383
//   rows  256: 31.9 26.3 33.0 52.2 109     rows 4096: 410  329  262  227
// by expert, 64 of [2047, 5119]: rows 8 162, 188, 174, 158; 64 237, 248, 220,
// 230; 256 608, 492, 430, 381.  Twice to three times those of whole pieces: the
// loads of 16 bytes that straddle dwords take the address units as much longer.
// Splitting the contraction wins while there are few workgroups of it, against
// 64 x 64 tiles (us in a graph): dense, 16 x 16, 315 of them (77 x 1000 x 1111)
// 4.8 and 6.9, 512 (64 x 2047 x 8191) 16.9 and 26.4, 1008 (256 x 1000 x 1041) 7.7
// and 7.0, 1024 (64 x 4095 x 4095) 16.6 and 15.3; by expert, 16 x 32, 512 (8 of
// [2047, 5119]) 19.4 and 25.3, 640 (64 of [301, 701]) 9.9 and 10.0, 1408 (64 of
// [700, 513]) 15.6 and 11.9.
inline Form choose(int64_t M, int64_t N, int64_t K, bool groups, int32_t G, Rows rows) {
    auto split = [&](int ns) {
        return Form{Kind::kSplit, 1, ns,
                    uint64_t(tile_bound(M, 16, groups, G)) * uint64_t((N + 16 * ns - 1) / (16 * ns)) * 512u};
    };
    auto tiled = [&](Kind kind, int um, int un) {
        const int64_t tm = tile_bound(M, 64 * um, groups, G), tn = (N + 64 * un - 1) / (64 * un);
        return Form{kind, um, un, (groups ? uint64_t(group_tiles(tm)) * uint64_t(tn) : (uint64_t(tm) * uint64_t(tn) + 7) / 8 * 8) * 512};
    };
    const int64_t each = groups ? (M + G - 1) / G : M, parts = groups ? G : 1;   // rows of a group, groups
    if (rows == Rows::kPieces) {
        if (groups) return tiled(Kind::kPipe, each <= 16 ? 1 : each <= 160 ? 2 : 4, 4);
        if (M <= 16) return Form{Kind::kRing, 1, ring_columns(N), uint64_t((N + 15) / 16) * 512};
        constexpr Tile kTiles[] = {{4, 4, 1.25}, {2, 4, 0.80}, {2, 2, 0.57}, {2, 1, 0.51}, {1, 1, 0.33}};
        const Tile& t = best_tile(kTiles, M, N, K, 1);
        return tiled(Kind::kPipe, t.um, t.un);
    }
    if (groups ? parts * ((each + 15) / 16) * ((N + 31) / 32) <= 640 : ((M + 15) / 16) * ((N + 15) / 16) <= 768)
        return split(groups ? 2 : 1);
    if (rows == Rows::kFar) return split(2);
    constexpr Tile kTiles[] = {{2, 4, 1.85}, {2, 2, 0.98}, {2, 1, 0.74}, {1, 1, 0.56}};
    const Tile& t = best_tile(kTiles, each, N, K, parts);
    return tiled(Kind::kStaged, t.um, t.un);
}

// Activations that the product quantizes by itself: up to 16 rows of whole
// 16-byte pieces with the ring, or few tiles of short rows with the split.
constexpr int kFuseBytes = 16 * 1024;    // of activations at most (ring)
constexpr int64_t kFuseSplitCodes = 2048;                                   // two steps of 8 waves
constexpr int64_t kFuseSplitTiles = 384;

inline bool ring_fuses(const void* x, int64_t esz, int64_t ld_x, const int8_t* B, int64_t ldb, int64_t M, int64_t K) {
    return M <= 16 && K > 0 && K % 16 == 0 && M * K * esz <= kFuseBytes && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
           (M == 1 || ld_x * esz % 16 == 0) && (M - 1) * ld_x * esz < (1 << 30) && reinterpret_cast<uintptr_t>(B) % 16 == 0 &&
           ldb % 16 == 0 && ldb < (1 << 23);
}

inline bool split_fuses(int64_t M, int64_t N, int64_t K) {
    return K > 0 && K <= kFuseSplitCodes && ((M + 15) / 16) * ((N + 31) / 32) <= kFuseSplitTiles;
}

}  // namespace
}  // namespace mxq
