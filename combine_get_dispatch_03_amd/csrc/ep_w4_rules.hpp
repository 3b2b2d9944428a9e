// ep_w4_rules.hpp -- which kernel a product of the expert block with 4-bit weights takes: plain host code on the call's sizes.
#pragma once

#include <cstdint>

namespace ep {

enum W4Kernel { kW4Stream, kW4Tile32, kW4Tile64, kW4Tile128 };

struct W4Sizes {
    int T, K, E, El;
    int N;         // output channels of a projection
    bool up;       // gate and up: a tile holds 128 of them, otherwise 256
};

// us of the whole call (int4 in groups of 64, uniform routing), streamed / tiles of 32 / of 64 / of 128 rows, at so many rows per
// expert; in brackets the tiles of 32 rows of the gate and up product:
//                                       1 or 2 rows          12                   40                   64                   128
//    8 experts of 1024 x 512 (32)     10 / 18 / 19 / 22    11 / 18 / 18 / 21    16 / 21 / 23 / 27    19 / 21 / 26 / 30    26 / 21 / 26 / 35
//   16 of 2048 x 768 (96)             14 / 25 / 26 / 32    19 / 29 / 29 / 32    29 / 31 / 34 / 42    48 / 36 / 39 / 46    77 / 61 / 47 / 57
//    8 of 7168 x 2048 (128)           39 / 60 / 65 / 78    46 / 61 / 65 / 80    78 / 88 / 87 / 104  155 / 145 / 112 / 120 225 / 231 / 175 / 175
//   20 of 2112 x 1344 (198, 220)      26 / 29 / 30 / 38    37 / 35 / 34 / 39    58 / 56 / 42 / 49    92 / 85 / 72 / 60   132 / 107 / 90 / 130
//   64 of 2048 x 768 (384)            34 / 30 / 32 / 60    53 / 45 / 44 / 62    89 / 85 / 61 / 79   140 / 100 / 106 / 94 233 / 183 / 141 / 158
//   64 of 4096 x 1408 (704)           96 / 89 / 91 / 159  154 / 148 / 147 / 164 253 / 244 / 196 / 219 385 / 314 / 254 / 253 662 / 543 / 439 / 429
// 32 of 7168 x 2048, int4 in groups of 128: 2 rows 164 / 155 / 167 / 180, 16 rows 197 / 166 / 187 / 190, 24 rows 222 / 194 / 189 / 210.
// Tiles of 64 / of 128 rows there: 40 rows 229 / 268, 56 rows 297 / 278, 96 rows 391 / 365, 128 rows 510 / 538, 192 rows 689 / 647, 256 rows
// 870 / 792; 16 of 2048 x 768: 80 rows 36 / 47, 160 rows 61 / 52, 400 rows 119 / 110; 4 of 4096 x 1408: 256 rows 75 / 92, 400 rows 104 / 95.
// us of the down product, streamed / 32 / 64: 180 tiles (20 of 2112 x 1344), 12 rows 14.1 / 14.2 / 14.4, 40 rows 22.5 / 23.1 / 17.4; 224
// tiles (8 of 7168 x 2048), 1 row 14.8 / 16.2 / 16.8, 12 rows 18.6 / 17.3 / 17.8.
//   Streaming spreads a few tiles' work over idle CUs; tiles share the rows over 256 channels. A tile of 64 rows has twice a
// tile of 32's work, so there should be enough of them. A tile of 128 rows widens its codes once for twice the rows, but has a CU to
// itself where two of 64 share one: it is better where there is more than a round of work and the experts' rows fill it, or half of
// them do not fall just past its height (about 128 rows an expert).
inline W4Kernel w4_kernel(const W4Sizes& s) {
    const int64_t entries = (int64_t)s.T * s.K, busy = entries < s.El ? entries : s.El, cols = (s.N + (s.up ? 127 : 255)) / (s.up ? 128 : 256);
    const double rows = (double)entries / s.E;
    const double tiles = (double)(busy * cols);
    if (s.up ? tiles < 200 && rows <= 48 : tiles < 300 && rows * tiles < 2500) return kW4Stream;
    const double tiles64 = (rows / 64 + 0.5) * tiles;
    if (rows <= 20 || tiles64 < 150) return kW4Tile32;
    return (rows > 150 ? tiles64 > 290 : rows > 52 && rows <= 100 && tiles64 > 500) ? kW4Tile128 : kW4Tile64;
}

}  // namespace ep
