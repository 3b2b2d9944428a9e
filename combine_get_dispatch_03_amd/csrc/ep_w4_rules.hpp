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
//    8 experts of 1024 x 512 (32)     10 / 18 / 19 / 26    11 / 18 / 18 / 26    16 / 21 / 23 / 31    19 / 21 / 26 / 35    26 / 21 / 26 / 40
//   16 of 2048 x 768 (96)             14 / 25 / 26 / 40    19 / 29 / 29 / 40    29 / 31 / 34 / 47    48 / 36 / 39 / 54    77 / 61 / 47 / 62
//    8 of 7168 x 2048 (128)           39 / 60 / 65 / 108   46 / 61 / 65 / 107   78 / 88 / 87 / 128  155 / 145 / 112 / 144 225 / 231 / 175 / 202
//   20 of 2112 x 1344 (198, 220)      26 / 29 / 30 / 47    37 / 35 / 34 / 49    58 / 56 / 42 / 58    92 / 85 / 72 / 67   132 / 107 / 90 / 119
//   64 of 2048 x 768 (384)            34 / 30 / 32 / 51    53 / 45 / 44 / 76    89 / 85 / 61 / 93   140 / 100 / 106 / 106 233 / 183 / 141 / 174
//   64 of 4096 x 1408 (704)           96 / 89 / 91 / 150  154 / 148 / 147 / 214 253 / 244 / 196 / 256 385 / 314 / 254 / 292 662 / 543 / 439 / 461
// 32 of 7168 x 2048, int4 in groups of 128: 2 rows 164 / 155 / 167 / 259, 16 rows 197 / 166 / 187 / 258, 24 rows 222 / 194 / 189 / 270,
// 256 rows - / - / 970 / 975, 1024 rows - / - / 3257 / 3149; e2m1 in groups of 32 there - / - / 3483 / 3312.
// us of the down product, streamed / 32 / 64: 180 tiles (20 of 2112 x 1344), 12 rows 14.1 / 14.2 / 14.4, 40 rows 22.5 / 23.1 / 17.4; 224
// tiles (8 of 7168 x 2048), 1 row 14.8 / 16.2 / 16.8, 12 rows 18.6 / 17.3 / 17.8.
//   Streaming spreads a few tiles' work over idle CUs; tiles share the rows over 256 channels. A tile of 64 rows has twice a
// tile of 32's work, so there should be enough of them.
inline W4Kernel w4_kernel(const W4Sizes& s) {
    const int64_t entries = (int64_t)s.T * s.K, busy = entries < s.El ? entries : s.El, cols = (s.N + (s.up ? 127 : 255)) / (s.up ? 128 : 256);
    const double rows = (double)entries / s.E;
    const double tiles = (double)(busy * cols);
    if (s.up ? tiles < 200 && rows <= 48 : tiles < 300 && rows * tiles < 2500) return kW4Stream;
    if (rows <= 20 || (rows / 64 + 0.5) * tiles < 150) return kW4Tile32;
    return rows <= 300 ? kW4Tile64 : kW4Tile128;
}

}  // namespace ep
