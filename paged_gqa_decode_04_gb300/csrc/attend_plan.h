// How many CTAs share a piece of rows in paged_gqa_attend: host arithmetic alone.
#pragma once

#include <stdint.h>

namespace pgd {
namespace attend {

constexpr int kTile = 128;      // tokens of a key tile
constexpr int kRowShift = 8;    // log2 of the rows of a CTA
// Query heads of a KV head in the kernels with shaped scores: a row's place among them comes from
// a float32 quotient, which is exact below 2^21.
constexpr int kMostGroup = 1 << 20;

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

// Parts that the `tokens` of a shared prefix are cut into: two key tiles each or more, at most
// `splits` (0 for no tokens).
#ifdef __CUDACC__
__host__ __device__
#endif
inline int prefix_parts(int tokens, int splits) {
    const int pairs = (tokens + 2 * kTile - 1) / (2 * kTile);
    return pairs < splits ? pairs : splits;
}

constexpr int kMostSplits = 64;

// CTAs that a piece of 256 query rows of one KV head is given for its group's prefix: as many
// as the GPU holds at once, for `rows` rows a KV head of `groups` groups.
inline int prefix_splits(int64_t rows, int groups, int hkv, int num_sms) {
    int64_t pieces = (rows + (1 << kRowShift) - 1) >> kRowShift;
    if (pieces < groups) pieces = groups;
    const int64_t splits = num_sms / (pieces * hkv);
    return splits < 1 ? 1 : splits > kMostSplits ? kMostSplits : int(splits);
}

// The most results of query heads, rows times prefix_splits, that a batch of at most `heads` query
// heads (rows of all KV heads) leaves, however many groups it has: a piece's 256 rows have no more
// than their share of the GPU.  Grows with the batch, so that a workspace serves smaller ones.
inline int64_t most_prefix_rows(int64_t heads, int num_sms) {
    const int64_t most = int64_t(num_sms) << kRowShift;
    const int64_t all = heads * kMostSplits;
    return heads > most ? heads : all < most ? all : most;
}

}  // namespace attend
}  // namespace pgd
