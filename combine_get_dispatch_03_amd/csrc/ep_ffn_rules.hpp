// ep_ffn_rules.hpp -- which kernels a call of the expert block takes: plain host code on the call's sizes, so that a test can
// ask it too.
#pragma once

#include <cmath>
#include <cstdint>

namespace ep {

struct FfnSizes {
    int T, K, E, El;
    int hidden, inter;
    bool fp8;
};

// Rows an expert gets on average.  The host knows sizes only, not the routing: of T * K entries, an expert's share.
inline double mean_rows(const FfnSizes& s) { return (double)s.T * s.K / s.E; }

// Local experts that get a row, at most.
inline int busy_experts(const FfnSizes& s) { return (int64_t)s.T * s.K < s.El ? s.T * s.K : s.El; }

// Whether the gate and up projection's weights are worth marking as read once (copy16_to_lds): one row tile per expert, whole
// lines, and more of them than the 256 MB memory-side cache keeps beside the rest of a layer.
//   Rows, us of the product with the mark and without: 32 experts of 7168 x 2048, bf16, 16 rows each 302 and 319, 64 rows 319 and
// 332, 128 rows 354 and 373, 900 rows (four row tiles) 1409 and 1262; 256 experts, e4m3, 4 rows 1103 and 1209.  Of the whole
// call: 128 experts, bf16, 96 rows 2107 and 2165, 128 to 200 rows within 1%, 256 rows (some with two tiles) 3279 and 3158; 256
// experts, e4m3, 48 rows 2080 and 2144, 64 rows 2123 and 2194, 80 rows 2308 and 2298, 96 rows 2431 and 2413.
//   Size: 20 experts of 2112 x 1352 (228 MB), 117 rows 68 and 85; of 1344 x 512 (55 MB), 80 rows 28 and 23, of 1352 x 512 (rows of
// 2704 bytes) 39 and 27.  Of the whole call, 16 experts of 4096 channels, 8 rows, the same weights call after call, bf16 and e4m3: 128
// MiB 80 and 64, 57 and 49; 160 MiB 83 and 71, 61 and 53; 192 MiB 86 and 90, 71 and 73; 256 MiB 99 and 105, 95 and 104.  Four sets
// of weights in turn, as layers are: 64 MiB 73 and 75, 46 and 47; 128 MiB 82 and 85, 58 and 61; 160 MiB 88 and 91, 65 and 69.  So the
// limit, between what one set in the cache and what several want, gives up a few percent on either side of it.
inline bool weights_once(const FfnSizes& s) {
    const int64_t row = (int64_t)s.hidden * (s.fp8 ? 1 : 2);
    return mean_rows(s) <= (s.fp8 ? 64 : 128) && row % 128 == 0 && row * 2 * s.inter * s.El > (128ll << 20);
}

// Weights streamed past the rows (ep_ffn_stream.hip) rather than tiles of both through LDS: where an expert has so few rows
// that its weights' bytes decide, or where the tiles would leave most CUs idle.  Measured, 32 experts of 7168 x 2048, us of the
// product, streamed / tiled, at so many rows per expert (gate and up with its weights marked as read once; in brackets tiled
// without the mark):
//              gate, up, bf16       down, bf16    gate, up, e4m3       down, e4m3
//    2 rows    296 / 279 (303)      154 / 206     155 / 143 (154)       81 / 105
//    8         312 / 294 (318)      170 / 215     165 / 154 (164)       93 / 108
//   16         326 / 298 (320)      179 / 219     186 / 158 (167)      109 / 111
//   32         366 / 304 (323)      203 / 224     225 / 166 (169)      154 / 118
//   64         584 / 317 (333)      299 / 235     366 / 187 (182)      272 / 142
// (512 and 896 tiles: a tiled product takes a round of 256 for as long with fewer, a streamed one gets shorter.)
// Down, us of the whole call at other sizes and tiles, bf16 at 24, 32 and 47 or 48 rows and e4m3 at 16, 24 and 32:
//   4 experts of 7168 x 2048, 112 tiles     98 /  93  116 / 100  144 / 113       49 /  57   50 /  56   63 /  62
//   8 of 4096 x 1408, 128                   73 /  79   80 /  85   90 /  94       46 /  51   48 /  53   55 /  56
//   32 of 2048 x 1408, 256                 128 / 126  135 / 130  150 / 140       76 /  74   75 /  65   81 /  67
//   64 of 4096 x 1408, 1024                466 / 447  479 / 454  501 / 464      257 / 256  270 / 261  305 / 268
//   8 of  256 x  512,    8                  10 /  14   10 /  16   11 /  17       12 /  15   12 /  15   12 /  16
//   8 of 1024 x  512,   32                  16 /  19   18 /  20   21 /  21       14 /  17   14 /  18   16 /  20
//  16 of 1024 x  512,   64                  23 /  22   25 /  24   33 /  29       15 /  18   16 /  19   19 /  21
// With few tiles it is the rows times the tiles, the work that streaming spreads over idle CUs; 8 tiles and 80 rows 15 / 20 and 13 / 18,
// 32 tiles 30 / 28 and 21 / 23.
inline bool few_rows_down(const FfnSizes& s) {
    const double rows = mean_rows(s);
    const int64_t tiles = (int64_t)busy_experts(s) * ((s.hidden + 255) / 256);
    return rows < (s.fp8 ? 16 : 28) || (rows <= 80 && rows * tiles < (s.fp8 ? 3600 : 2100));
}

// The same for the gate and up projection.  Without the mark the weights are few and mostly come from the caches.  Streaming
// wins where its finer grid is what fills the chip: the fewer 128-channel tiles and, in e4m3, rows there are, and past one
// row tile of its own (64 rows) by its pieces of 64 rows x 32 channels.  us of the whole call, streamed / tiled, at so many rows:
//                                   bf16: 2          16         32         64        e4m3: 2         16         32         64
//    8 experts of 2048 x 768, 48 tiles    22 / 33    28 / 36    36 / 42    53 / 45      16 / 23    19 / 25    25 / 30    40 / 36
//   16 of 2048 x 768, 96                  34 / 46    41 / 50    48 / 53    78 / 57      23 / 26    28 / 28    35 / 34    46 / 37
//   64 of 2048 x 256, 128                 47 / 59    62 / 70    69 / 76    88 / 70      31 / 33    35 / 34    40 / 38    63 / 44
//   20 of 1280 x 1024, 160                36 / 38    47 / 48    60 / 58    71 / 55      26 / 23    32 / 26    37 / 32    48 / 34
//   32 of 1024 x 768, 192                 36 / 33    43 / 38    48 / 41    67 / 46      25 / 22    31 / 25    38 / 30    47 / 31
//  256 of  256 x 512, 1024                63 / 54    79 / 61    90 / 65   125 / 67      48 / 35    57 / 37    65 / 41    97 / 48
// us of the product: 4 experts of 3328 x 384 with 70, 128 and 256 rows (99, 143 and 239 pieces) 23 / 45 and 21 / 32, 23 / 50 and 21 /
// 37, 41 / 60 and 21 / 38; 8 of 2048 x 512, 100 rows (326) 28 / 33 and 18 / 24; 4 of 2048 x 1024, 256 rows (638) 50 / 42 and 27 / 25.
//   With weights marked as read once both forms run at the memory's rate with a few rows per expert, and what decides is how
// much of its last round the tiles fill, of those experts that uniform routing gives a row.  Streaming reads the rows again
// for every 32 channels, so it falls behind as rows come on, in e4m3, with half the weights' bytes, twice as fast.  us of the
// whole call, streamed / tiled, 32 experts of 7168 channels (a test holds these and some 900 more sizes):
//   rounds            4 or 8 rows   16          32          47         e4m3: 4 or 8 rows   16          32          47
//   0.25, 0.375        79 / 139      97 / 149   118 / 164   139 / 173         81 /  97      91 /  97   106 / 105   119 / 110
//   0.5               134 / 168     151 / 182   172 / 197   209 / 206        102 / 109     108 / 113   121 / 123   131 / 131
//   0.75              222 / 205     238 / 217   237 / 232   284 / 245        126 / 107     147 / 110   163 / 120   165 / 128
//   1.125             297 / 363     326 / 372   350 / 387   387 / 400        177 / 185     198 / 198   216 / 212   240 / 218
//   1.375             352 / 390     376 / 400   421 / 419   466 / 435        192 / 206     221 / 222   256 / 231   280 / 238
//   1.625             425 / 428     429 / 436   490 / 459   539 / 477        236 / 226     261 / 243   294 / 255   326 / 263
//   1.75              448 / 436     463 / 442   502 / 469   564 / 491        244 / 231     276 / 250   309 / 261   354 / 272
// One round, however full, is spread over all XCDs; of several the last one is not, so it costs more of a whole one.
inline bool few_rows_up(const FfnSizes& s) {
    const double rows = mean_rows(s);
    const int cols = (s.inter + 127) / 128;
    if (!weights_once(s)) {
        const int64_t tiles = (int64_t)busy_experts(s) * cols;
        if (rows > 52) return (rows * s.El + 63.0 * busy_experts(s)) / 64 * ((s.inter + 31) / 32) < 340;
        if (s.fp8) return tiles < 130 && rows * tiles < 3100;
        return rows < 12 ? tiles < 165 : tiles < 135 && rows * tiles < 4200;
    }
    if (rows >= 48) return false;
    const double idle = std::pow(1.0 - (s.K < s.E ? (double)s.K / s.E : 1.0), s.T), rounds = s.El * (1.0 - idle) * cols / 256;
    const double more = rows > 16 ? rows - 16 : 0;
    const double fill = rounds <= 1 ? 0.58 - (s.fp8 ? 0.008 : 0.004) * more : s.fp8 ? 0.76 - 0.010 * more : 0.95 - 0.008 * more;
    return rounds < fill * std::ceil(rounds);
}

}  // namespace ep
