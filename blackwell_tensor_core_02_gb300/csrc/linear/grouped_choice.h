// grouped_choice.h -- how a grouped product or adapters run: the tile and the CTAs that share a tile's sum,
// by a fitted cost.  Host logic alone, of a call's sizes (`Params`: groups, rows, I, J, R and rank of GroupParams).
#pragma once

#include <stdint.h>

#include "grouped_ops.h"

namespace linear_ops {

enum GroupMode { kGroupNT = 0, kGroupNN = 1, kGroupTN = 2, kGroupLora = 3, kGroupDown = 4 };

// Tiles of `tile` rows that the groups have at most: each that has a row begins one, and
// the other rows fill more.
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t tile) {
    const int64_t some = groups < rows ? groups : rows;
    return some + (rows - some) / tile;
}

// How a call runs: its tile, and the CTAs that share a tile's sum, or 0 for a persistent grid.
struct Choice {
    int tile, split;
};

// Cycles that a choice takes, near enough to choose by: a stage (64 of the sum) of each
// tile, set by the rows that the copy engine brings and, of pairs, by the MMAs; tiles by
// the groups' average rows; whole waves of a persistent grid, but of clusters, two CTAs an
// SM that share what it brings, a share of one; and what a tile and a launch take besides.
// The numbers are fitted to the times of 85 shapes (1 to 8192 rows, 1 to 64 groups, 64 to
// 14336 columns, sums of 64 to 4096) with each of the 20 choices; on 85 others the chosen one is 4 % off
// the best on average, 30 % at most.  In microseconds, the choice and others, rows spread evenly but where said:
//   256 x 4096 x 4096, one group    128 rows, 2 CTAs a tile: 13.5   64, 1: 14.7   256, pairs: 22.9
//   512 x 2048 x 2048, one group    128, 2: 8.7                     64, 1: 8.9    256, pairs: 14.0
//   2000 x 2048 x 2048, 8 groups    256, pairs: 18.7                128, 1: 20.8  128, persistent: 21.1
//   the same, all rows in one       256, pairs: 15.3                128, 1: 17.9  128, persistent: 18.3
//   8192 x 1024 x 1024, 8 groups    256, pairs: 16.2                128, persistent: 19.9   64: 26.9
//   2 x 2048 x 1024, 64 groups      16, 4: 4.9                      32, 4: 5.3    256, pairs: 6.6
//   4096 x 1024 x 1024, 64 groups, all rows in one   128, persistent: 12.0        256, pairs: 10.9
// Sums over rows, of which 60 shapes were timed with each choice, the chosen one 2 % off the best; on 60
// others 4 %, at most 2.2 times (6098 rows, 10 groups, 184 x 88: 64, persistent 15.3; 64, 8 7.0):
//   8192 rows, 1024 x 1024          128, 2: 21.2                    64, 2: 23.4   256, pairs: 39.6
//   3855 rows, 208 x 208            64, 4: 6.9                      64, 8: 5.8    256, pairs: 20.5
//   8192 rows, 8 groups, 1024 x 1024  256, pairs: 16.2              128, persistent: 20.4   128, 2: 37.6
template <typename Params>
double cost_of(int mode, const Params &p, int sms, int tile, int split) {
    // of a sum over rows the groups have p.J columns each, and sums of as many rows as there are on average
    const bool sum = mode == kGroupTN;
    const double some = sum || p.groups < p.rows ? p.groups : p.rows, rows = sum ? some * p.J : p.rows, each = rows / some;
    const double k_tiles = sum ? (p.rows / some + 63) / 64 : (p.R + 63) / 64;
    const bool pair = tile == 256;
    // a group's rows fill its last tile by half
    double tiles = each > 0.5 * tile ? rows / tile + 0.5 * some : some;
    const double most = static_cast<double>(most_tiles(p.rows, p.groups, tile));
    if (!sum && tiles > most) tiles = most;
    if (sum) tiles = some * ((p.J + tile - 1) / tile);
    // rows of a stage in one CTA: 128 of P, and of Q boxes of 32 as far as a tile is filled
    const int filled = tiles > some ? tile : (each < tile ? static_cast<int>(each + 31) / 32 * 32 : tile);
    const int q = tile == 16 ? 16 : (filled / (pair ? 2 : 1) + 31) / 32 * 32;
    double stage = 1.6 * (128 + q) * (pair ? 1.13 : 1.0);
    if (stage < 450) stage = 450;
    const double n = tiles * ((p.I + (pair ? 255 : 127)) / (pair ? 256 : 128)) * (split > 0 ? split : 1);
    if (split == 0) {
        double waves = n / (pair ? sms / 2 : sms);
        waves = waves < 3 ? static_cast<double>(static_cast<int64_t>(waves + 1 - 1e-6)) : waves + 0.5;
        return waves * (k_tiles * stage + 1330) + 3500;
    }
    double load = n / sms;
    const double turns = static_cast<double>(static_cast<int64_t>(load / 2 + 1 - 1e-6));
    load = load <= 1 ? 1 : (load <= 2 ? 1 + load / 2 : 1.5 * (load + 0.5));
    return load * (k_tiles / split) * stage + turns * (3800 + 17 * tile + (split > 1 ? 600 + 20 * tile * split : 0));
}

template <typename Params>
Choice choose(int mode, const Params &p, int sms, const grouped_options &o) {
    const bool sum = mode == kGroupTN;
    // K tiles of a sum: of rows, as many as the groups have on average
    const int64_t k_tiles = sum ? (static_cast<int64_t>(p.rows) / p.groups + 63) / 64 : (static_cast<int64_t>(p.R) + 63) / 64;
    Choice best = {o.tile ? o.tile : 32, o.split > 0 ? o.split : 0};
    double least = -1;
    for (int tile = sum ? 64 : 16; tile <= 256; tile *= 2) {
        for (int split = 0; split <= 8; split = split ? 2 * split : 1) {
            // split 0: a persistent grid, of tiles from 32 on; clusters of tiles up to 128
            if ((o.tile && tile != o.tile) || (o.split && split != (o.split > 0 ? o.split : 0)) ||
                (split == 0 ? tile == 16 : tile == 256) || (split > 1 && split > k_tiles && !o.split) ||
                (sum && split == 1 && !o.split)) {
                continue;
            }
            const double cost = cost_of(mode, p, sms, tile, split);
            if (least < 0 || cost < least) least = cost, best = {tile, split};
        }
    }
    while (best.split > 1 && best.split > k_tiles) best.split /= 2;
    return best;
}

// As cost_of(), of a call with adapters behind its first launch: tiles of 256 rows have one request
// each and its ranks as more of the sum; others, of a CTA an SM, pieces, shared by the cluster.  Fitted to 65 shapes (1
// to 3600 rows, 1 to 128 requests, 512 to 8192 columns, sums of 704 to 4096) with each choice; on 65 others 1 %
// off the best on average, 15 % at most.  In microseconds, the choice and others, of 4096 x 4096 but where said:
//   64 requests of 1 row, rank 16   64 rows, 4 CTAs a tile: 16.8   128, 4: 17.6   32, 2: 17.6   16, 1: 21.1
//   8 of 100, 16                    256, pairs: 37.2               128, 1: 49.4   64, 1: 54.9
//   32 of 64, 16                    128, 1: 93.5                   256, pairs: 118
//   64 of 4, 32, 1024 x 1024        32, 2: 18.9                    16, 1: 18.5    128, 4: 22.0
//   1 of 1, 32, 2048 x 2048         16, 4: 5.9                     32, 4: 5.9     16, 1: 9.1
// (Of 152 SMs clusters of 8 and 4 have 120 and 144 at once.)
template <typename Params>
double lora_cost(const Params &p, int sms, int tile, int split) {
    const int requests = p.groups > 0 ? p.groups : 1;
    const double rows = p.rows, each = rows / requests, k_tiles = (p.R + 63) / 64;
    const int ranks = (p.rank + 63) / 64;
    auto whole = [](double v) { return static_cast<double>(static_cast<int64_t>(v + 1 - 1e-6)); };
    if (tile == 256) {
        const double tiles = each > 128 ? rows / 256 + 0.5 * requests : requests;
        const int filled = each >= 256 ? 256 : (static_cast<int>(each) + 31) / 32 * 32, q = (filled / 2 + 31) / 32 * 32;
        const double stage = 1.6 * (128 + q) * 1.13, waves = tiles * ((p.I + 255) / 256) / (sms / 2);
        return (waves < 3 ? whole(waves) : waves + 0.5) * ((k_tiles + 2 * ranks) * (stage < 450 ? 450 : stage) + 1330) + 3500;
    }
    const int filled = tile < p.rows ? tile : p.rows, q = tile == 16 ? 16 : (filled + 31) / 32 * 32;
    const int at_once = split == 8 ? sms * 15 / 19 : (split == 4 ? sms * 18 / 19 : sms);
    const double turns = whole(static_cast<double>((static_cast<int64_t>(p.rows) + tile - 1) / tile * ((p.I + 127) / 128) * split) / at_once);
    const double stage = 1.6 * (128 + q);
    double pieces = 0;
    if (p.groups > 0) {
        const int piece = tile < 64 ? 16 : tile / 2;  // FewShape::PIECE
        pieces = filled / each + 1 < filled ? filled / each + 1 : filled;
        if (pieces * piece < filled) pieces = static_cast<double>(filled) / piece;
        pieces = whole(pieces / split);
    }
    return turns * (k_tiles / split * (stage < 400 ? 400 : stage) + pieces * (800 + 200 * (ranks - 1)) + 3800 + 30 * tile +
                    (split > 1 ? 600 + 20.0 * filled * split : 0));
}

template <typename Params>
Choice choose_lora(const Params &p, int sms, const grouped_options &o) {
    const int64_t k_tiles = (static_cast<int64_t>(p.R) + 63) / 64;
    Choice best = {o.tile ? o.tile : 16, o.split > 0 ? o.split : 0};
    double least = -1;
    for (int tile = 16; tile <= 256; tile *= 2) {
        for (int split = tile == 256 ? 0 : 1; split <= (tile == 256 ? 0 : 8); split = split ? 2 * split : 1) {
            if ((o.tile && tile != o.tile) || (o.split && split != (o.split > 0 ? o.split : 0)) || (split > 1 && split > k_tiles && !o.split)) continue;
            const double cost = lora_cost(p, sms, tile, split);
            if (least < 0 || cost < least) least = cost, best = {tile, split};
        }
    }
    while (best.split > 1 && best.split > k_tiles) best.split /= 2;
    return best;
}

}  // namespace linear_ops
