// Which kernel a call of the feed-forward block takes: rules on rows, experts, columns
// and compute units.  Plain C++, so that a host program can ask them as well.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace moegg {

// Row tiles of `rows` rows over E experts, at most.
inline int64_t row_tiles(int64_t rows, int E, int block)
{
    return rows <= E ? rows : (rows - E + 1 + block - 1) / block + E - 1;
}

// Tile shapes: small (32 rows: for a few row tiles of streamed weights), middle (128 x
// 128, two workgroups a compute unit), deep (the same with four stages, one workgroup)
// and large (256 x 256, one).
enum Shape { kSmallTiles, kMidTiles, kDeepTiles, kBigTiles };

// Which of them a launch takes.  Rows per expert are known on the device alone: an
// expert's last row tile counts as half full (one expert's is known).
//   small   where a launch is bound by latency: it has up to `most_small` rounds of
//           small tiles.  8 experts of 64 rows, 2048 into 2048: int8 16.2 us (middle
//           19.5, large 27.8), bf16 23.9 (29.5, 47.6).
//   deep    where the middle tiles leave each compute unit one: nothing else covers
//           a stage's way from memory.  3003 rows of 1008 into 2 x 520, A kept, 18.7 us
//           (middle 21.8); 2048 rows of 2048 into 2 x 768 25.8 (28.1); with 320 tiles for
//           256 units 45.0 (33.5).
//   large   where their rounds over the compute units cost less than the middle
//           tiles', 1.65 times as much a round, two tiles a unit in a middle one whose
//           last round costs what it fills: 60 experts, 2048 into 2048 int8, of 1024
//           rows 318 us (middle 362, small 690), of 128 rows 85 (66, 140).
// 256 x 128 and 128 x 256 tiles with 32-deep stages, two workgroups a unit, lose to
// both (8192 rows of 4096 int8 into 28672 1.19 ms, large 0.98; 65536 of 768 into
// 2048, each with 38 for their quantisation, 248 us, large 236).  Swept over 1, 8 and 60 experts of 16 to 1024 rows and 512
// to 8192 columns.
inline Shape tile_shape(int64_t S, int E, int cols, int small_cols, double most_small, int cus)
{
    auto rounds = [&](int64_t bm, int64_t bn, int a_round) {
        const int64_t rows =
            E == 1 ? (S + bm - 1) / bm
                   : std::min(S, std::max(std::min<int64_t>(S, E), S / bm + E / 2));
        return (double)(rows * ((cols + bn - 1) / bn)) / a_round;
    };
    if (rounds(32, small_cols, cus) <= most_small)
        return kSmallTiles;
    const double mid = std::max(0.6, rounds(128, 128, 2 * cus) + 0.2);
    if (1.65 * std::ceil(rounds(256, 256, cus)) < mid)
        return kBigTiles;
    return rounds(128, 128, cus) <= 1.0 ? kDeepTiles : kMidTiles;
}

// The backward's: as above, where its middle tiles leave registers for two workgroups a
// compute unit (`two`: 256 of them, which packed values in whole columns alone keep to;
// the other forms take 260 to 268).  Else four stages at the same one workgroup a unit,
// which cover a stage's way from memory where nothing else does: with A kept, 8 experts of
// 1024 rows, 4096 into 4096, 418 us (two stages 532), 60 of 256 rows, 2048 into 768, 113
// (133), 128 of 64, 768 into 512, 41 (40), the worst of 200 shapes 46 (45).  Held to 256
// registers, the two-stage form gains where there are many tiles and loses where there
// are up to two a unit (8 experts of 256 rows, 1024 into 2048, A kept: 34.4 us for 26.8).
inline Shape bwd_shape(int64_t S, int E, int cols, int small_cols, double most_small, bool two,
                       int cus)
{
    const Shape shape = tile_shape(S, E, cols, small_cols, most_small, cus);
    return shape == kMidTiles && !two ? kDeepTiles : shape;
}

// Up to about two rows for each expert (four where there are fewer), unless tiles of 32
// rows fill the card anyway: one of their rounds over the compute units is worth 1024
// bytes of a row of W, shorter rows leaving a wave little between its tables, loads
// and sums.  In a graph, other experts' weights from memory each time (tiles / vectors, us;
// int8 and gated unless said):
//   1 token of 1024 into 2 of 8 experts of 2048                    11.8 /  5.6
//   1 token of 2048 into 8 of 128 experts of 1536                  19.2 /  9.3
//   1 token of 4096 into 2 of 8 experts of 14336, 28672, 57344     36.3 / 26.8, 55.5 / 48.3, 110 / 89
//   1 token of 1024 into 2 of 8 experts of 32768                   20.6 / 20.1
//   4 tokens of 4096 into 2 of 8 experts of 4096, 14336            33.8 / 22.9, 88.8 / 64.6
//   8 tokens of 4096 into 2 of 8 experts of 4096, bf16             60.4 / 48.0
//   8 and 16 tokens of 2048 into 8 of 128 experts of 1536          47.7 / 40.2, 54.6 / 60.9
//   1 and 4 rows of 768 into 8 of 128 experts of 2048, plain       11.2 /  7.2, 16.3 / 20.3
// Where it is the wrong side: at two rows an expert of 2048 bytes (256 rows over 128 experts
// of 512 columns 28.3 / 33.4, of 1024 52.4 / 59.9); plain calls, whose tiles it counts by 128
// columns (30 tokens of 4096 into 4 of 60 experts of 2816: 152 / 118, and it takes tiles);
// and where routing, which the device alone knows, sends many rows to one expert, whose W
// is then read once for every four of them (256 of 2048 into 1024, all to one of 128 experts:
// 17.1 / 29.8; 128 of 8192 into 4096, all to one of 64: 48 / 95).  Fewer rows in all would bound
// that and lose more where they spread (those 128 over all experts: 393 / 319).
inline bool vec_pays(int64_t S, int E, int cols, bool gated, int64_t row_bytes, int cus)
{
    if (S > std::max<int64_t>(2 * (int64_t)E, 4))
        return false;
    const int tile = gated ? 256 : 128;
    const int64_t tiles = std::min<int64_t>(S, E) * ((cols + tile - 1) / tile);
    return tiles * 1024 <= row_bytes * cus;
}

}  // namespace moegg
