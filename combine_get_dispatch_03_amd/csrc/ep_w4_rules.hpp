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

// us of the whole call (int4 in groups of 64, uniform routing), one product streamed / on tiles of 32 / of 64 / of 128 rows while the other is on tiles
// of 64, at so many rows per expert; in brackets the busy experts' tiles:
//   gate and up                          1                   12                  40                  64                  128
//    8 experts of 1024 x 512 (32)     16 / 20 / 20 / 23   17 / 21 / 21 / 23   23 / 25 / 27 / 29   25 / 25 / 29 / 33   29 / 26 / 29 / 36
//   16 of 2048 x 768 (96)             22 / 28 / 29 / 33   25 / 31 / 31 / 34   34 / 34 / 38 / 42   44 / 36 / 41 / 47   68 / 53 / 48 / 60
//    8 of 7168 x 2048 (128)           50 / 68 / 76 / 81   54 / 69 / 78 / 82   82 / 80 / 91 / 103 138 / 125 / 112 / 131 211 / 222 / 182 / 182
//   20 of 2112 x 1344 (220)           35 / 35 / 36 / 40   44 / 40 / 42 / 43   61 / 54 / 47 / 51   91 / 85 / 72 / 66  123 / 96 / 102 / 113
//   64 of 2048 x 768 (384)            42 / 40 / 41 / 49   56 / 53 / 51 / 61   84 / 87 / 68 / 84  129 / 102 / 110 / 106 201 / 170 / 140 / 169
//   64 of 4096 x 1408 (704)          101 / 90 / 90 / 113 149 / 152 / 150 / 156 226 / 220 / 197 / 209 334 / 295 / 246 / 254 572 / 499 / 428 / 424
//   32 of 7168 x 2048, groups of 128 (512): 2 rows 152 / 142 / 139 / 166, 16 rows 184 / 162 / 158 / 174, 24 rows 205 / 198 / 171 / 194, 64 rows
//   396 / 351 / 325 / 288, 96 rows 534 / 459 / 373 / 356, 128 rows 683 / 576 / 510 / 489, 256 rows 1227 / 1012 / 880 / 814.
//   down
//    8 of 1024 x 512 (32)             15 / 20 / 20 / 21   16 / 20 / 21 / 21   22 / 25 / 27 / 27   24 / 26 / 29 / 30   28 / 26 / 29 / 31
//   16 of 2048 x 768 (128)            24 / 27 / 29 / 29   26 / 29 / 31 / 31   35 / 35 / 38 / 38   48 / 41 / 41 / 42   59 / 53 / 48 / 45
//   20 of 2112 x 1344 (180)           28 / 33 / 36 / 36   38 / 38 / 42 / 40   55 / 49 / 47 / 48   78 / 65 / 72 / 66  125 / 108 / 102 / 108
//    8 of 7168 x 2048 (224)           70 / 71 / 76 / 76   77 / 74 / 78 / 78  103 / 95 / 91 / 93  126 / 118 / 112 / 103 206 / 169 / 182 / 178
//   64 of 2048 x 768 (512)            41 / 38 / 41 / 43   56 / 47 / 51 / 50   86 / 71 / 68 / 69  136 / 109 / 110 / 102 186 / 142 / 140 / 131
//   64 of 4096 x 1408 (1024)          82 / 80 / 90 / 87  163 / 142 / 150 / 154 260 / 217 / 197 / 211 315 / 250 / 246 / 240 576 / 458 / 428 / 422
//   32 of 7168 x 2048, groups of 128 (896): 2 rows 134 / 130 / 139 / 148, 16 rows 167 / 154 / 158 / 169, 24 rows 193 / 166 / 171 / 182, 64 rows
//   401 / 335 / 325 / 321, 128 rows 657 / 528 / 510 / 498, 256 rows 1175 / 945 / 880 / 844.
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
