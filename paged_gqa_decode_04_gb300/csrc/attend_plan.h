// How many CTAs share a piece of rows in paged_gqa_attend: host arithmetic alone.
#pragma once

#include <stdint.h>

namespace pgd {
namespace attend {

constexpr int kTile = 128;      // tokens of a key tile
constexpr int kRowShift = 8;    // log2 of the rows of a CTA

// The most key tiles a piece of rows meets, when sequences have at most `max_len` tokens.  With
// a window, its 256 rows (token, head of the group) lie in (254 + group) / group + 1 tokens or
// fewer, which see window - 1 tokens more, from anywhere in a tile on.
inline int64_t piece_tiles(int64_t max_len, int window, int group) {
    const int64_t all = (max_len + kTile - 1) / kTile;
    if (window <= 0) return all;
    const int64_t seen = window + ((1 << kRowShift) - 2 + group) / group;
    const int64_t tiles = (seen + kTile - 2) / kTile + 1;
    return tiles < all ? tiles : all;
}

// CTAs that share the keys of a piece of rows (a cluster of c).  With `units` pieces and `fit[i]`
// clusters of 1 << i on the GPU at once there are ceil(units / fit) rounds, each of tiles / c key
// tiles of `tile` us and a CTA's start and end, 10 us and for a join 1 us a doubling and, with
// more than 128 rows, 6 more.  The smallest sum is taken; tiles are those of the longest sequence
// that the table can hold, which may be far more than there are: where pieces fill the GPU four
// times, the uneven end is not worth that risk and c is 1 (4 prompts of up to 4096 behind a table
// for 131072: 265 us, 466 with c = 2).  Measured over c = 1, 2, 4, 8 (us; the choice is marked):
//     2 sequences, 2048 cached, 4 queries each     33   22   19*  32
//     8 sequences, up to 4096, 2-8 queries each    48   33*  44   75
//     one prompt of 512, 32/8 heads                21*  28   47  102
//     2048 queries of 32768, 64/8 heads          1349 1260* 1455
//     2048 queries of 8192, 64/8 heads            336* 379  522
inline int choose_cluster(const int (&fit)[4], int64_t units, int64_t most_tiles, bool few,
                          double tile) {
    const double tiles = double(most_tiles);
    int best = 0;
    double least = 0;
    for (int i = 0; i < 4; ++i) {
        if (fit[i] < 1 || (i && (tiles < (1 << i) || units > 4 * fit[0]))) break;
        const double us = double((units + fit[i] - 1) / fit[i]) *
                          (tiles / (1 << i) * tile + 10 + (i ? i + (few ? 0 : 6) : 0));
        if (i == 0 || us < least) best = i, least = us;
    }
    return 1 << best;
}

}  // namespace attend
}  // namespace pgd
