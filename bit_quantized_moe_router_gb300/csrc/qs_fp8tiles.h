// qs_fp8tiles.h -- which tiles a product of e4m3 rows runs in: a rule on its sizes and the number of SMs, on the host.
#pragma once

#include <algorithm>
#include <cstdint>

namespace qs {

constexpr int kTileRows = 128;
constexpr int kFewRows = 64;  // most rows that are copied by small boxes
constexpr int kFewTile = 16, kFewAverage = 4;  // rows of a tile of groups of few, and of their average group at most

// cols weight rows a tile; pair: 256 rows in two CTAs; few (0, 16, 32): that many rows, the weight rows down the
// accumulator; count: tiles there can be at most.
struct MmTiles {
    int cols;
    bool pair;
    int few;
    int64_t count;
};

// wide: whether tiles of 256 weight rows may be taken.
inline MmTiles pick_tiles(int n_rows, int n_cols, int n_experts, bool grouped, int n_sm, bool wide) {
    // Pairs of CTAs where tiles of 256 x 256 fill them: more than half of a tile's rows are there on
    // average, and there is a tile for each pair.
    const int64_t per = grouped ? n_rows / n_experts : n_rows;
    const int64_t pair_tiles = (grouped ? (int64_t)n_rows / 256 + n_experts : ((int64_t)n_rows + 255) / 256) *
                               (((int64_t)n_cols + 255) / 256);
    if (wide && per > kTileRows && pair_tiles >= n_sm / 2) return {256, true, 0, pair_tiles};
    // (Times here and below are of one call in a loop: weights that fit the L2 are read from it.  Those of uneven groups
    // are with three sets of weights in turn.)
    // Groups of few rows: weight rows down the accumulator, the group's across, 16 a tile.  Against the tiles below, 8 of
    // 256 experts: one token at 2048 x 1024 (columns x inner) 4.6 us against 6.3, eight 21.3 against 24.8, 128 80.1
    // against 84.7; sixty-four rows to two experts, 2048 x 2048, 5.3 against 5.6.  At eight rows an expert and more what is
    // gained where they spread evenly (82.5 against 86.8) is lost where they do not (31.5 against 24.4 if popularity
    // falls with rank^-1.5), since each 16 rows take an expert's weights again.  At four, 1024 x 2048, uneven groups gain
    // too, but where few experts have nearly all rows: 128 tokens to 8 of 256, popularity as rank^-0, -0.5, -1, -1.5, -2: 80,
    // 64, 32, 21, 18 us against 83, 70, 30, 25, 15; 32 tokens to 8 of 64: 24, 21, 17, 12, 10 against 26, 26, 24, 14, 13; one group
    // of 1000 rows and 24 of one 18 against 14, of 500 and 246 of one 79 against 81.  Tiles of 32 and 64 rows were slower (eight
    // tokens at 1024 x 2048 22.5 and 24.3 against 22.2).  64 weight rows a tile where those leave half of the SMs free
    // (one token at 512 x 2048 4.5 against 5.0 with 128; with more tiles they lose as often, 5.1 against 4.8 for two
    // tokens through 4 experts at 1024 x 2048).
    const int64_t few64 = ((int64_t)n_cols + 63) / 64, few128 = ((int64_t)n_cols + 127) / 128;
    if (grouped && n_rows <= std::max(kFewRows, kFewAverage * n_experts)) {
        const int64_t mt = (int64_t)n_rows / kFewTile + std::min(n_rows, n_experts);
        if (2 * mt * few64 <= n_sm) return {64, false, kFewTile, mt * few64};
        return {128, false, kFewTile, mt * few128};
    }
    // One matrix: the tiles of 64 weight rows if all have an SM, since one fills its SM with the K of 64 weight rows
    // faster than the tiles below with theirs: 1 x 4096 x 2048 4.0 us against 4.8, 16 x 9728 x 2048 4.5 against 5.5,
    // 100 x 1024 x 4096 5.5 against 7.0, 1 x 4096 x 16384 16.8 against 19.7; at K of 1024 and less the same or better.
    // Then the same with 32 rows: 64 x 4864 x 4096 6.4 against 7.9, 200 x 1024 x 2048 4.8 against 5.2, 512 x 512 x 1024
    // 4.0 against 4.1 (with 64 rows 4.5: slower than what follows in 60 of 80 such shapes).
    // Else those of 128 for 16 rows: 1 x 10000 x 2048 5.0 against 7.8, 1 x 32768 x 4096 22.9 against 25.0; 32 rows would
    // take the weights twice (29.3 against 25.4).
    if (!grouped) {
        const int64_t mt = ((int64_t)n_rows + kFewTile - 1) / kFewTile, mt32 = (mt + 1) / 2;
        if (mt * few64 <= n_sm) return {64, false, kFewTile, mt * few64};
        if (mt32 * few64 <= n_sm) return {64, false, 2 * kFewTile, mt32 * few64};
        if (mt == 1) return {128, false, kFewTile, few128};
    }
    // row tiles: those of one matrix, or for groups the most there can be if rows spread over the
    // experts (each group's last tile may be short)
    const int64_t mt = grouped ? (int64_t)n_rows / kTileRows + std::min(n_rows, n_experts)
                               : ((int64_t)n_rows + kTileRows - 1) / kTileRows;
    // the width whose waves of tiles take least, a tile taking its columns and a fixed part
    MmTiles best = {};
    int64_t best_cost = INT64_MAX;
    for (int cols = wide ? 256 : 128; cols >= 16; cols /= 2) {
        const int64_t tiles = mt * (((int64_t)n_cols + cols - 1) / cols);
        const int64_t cost = (tiles + n_sm - 1) / n_sm * (cols + 32);
        if (cost < best_cost) {
            best_cost = cost;
            best = {cols, false, 0, tiles};
        }
    }
    return best;
}

}  // namespace qs
