// ep_few_rules.hpp -- which kernels the layer for a few tokens takes: plain host code on the call's sizes.  (The host does not know the
// routing, so the rules go by what a uniform one gives.)
#pragma once

namespace ep {

constexpr int kFewWaves = 16;      // of a workgroup of the second kernel: as many entries of several tokens can stand by themselves

// Each entry by itself, or an expert's entries together.  An entry by itself has its weights under way at once, but reads them
// itself; together, an expert's are read once, after its entries are found.  us of the whole call, by themselves / together, experts of
// 7168 x 2048, entries spread evenly over that many experts:
//                            int4, groups of 128      e4m3                     bf16
//    1 token of top-8 (16)       42 /  45               68 /  74               132 / 132
//    2 tokens of top-4 (8)       41 /  44               67 /  74               132 / 130
//    2 tokens of top-4 (4)       36 /  35               53 /  42               119 /  70
//    2 tokens of top-8 (16)      75 /  77              126 / 134               260 / 254
//    2 tokens of top-8 (8)       62 /  45              112 /  75               242 / 131
//    4 tokens of top-4 (4)       58 /  35               94 /  43               212 /  71
// Routed at random, 16 entries: of 16 experts (int4) 64 / 58, of 24 68 / 73, of 32 68 / 73, of 64 69 / 73; e4m3 110 / 96, 116 / 120, 113 / 121,
// 116 / 124; 8 entries of 8 experts 41 / 43 and 72 / 78.  Small experts, 256 x 512 in bf16: 8 entries of 8 11.6 / 15.6, of 4 11.6 / 13.0, 16
// of 8 16.0 / 16.3.  One token's entries have an expert each (and its workspace room for no other form of
// h); of several tokens enough experts for few to be shared.
inline bool few_by_entry(int T, int K, int E) {
    const int n = T * K;
    return T == 1 || (n <= kFewWaves && (n <= 8 ? n : 2 * n) <= E);
}

// 16 output channels a workgroup of the second kernel, or 32, which have half as many loads of rows per byte of weights.  A CU has room for
// one workgroup: 16 as long as they are one round on the 256 CUs, otherwise 32.  us of the whole call, 16 / 32 channels, 64 experts of H x
// 1024, top-8:
//                     H = 2048     3584      4096       4224       4608      5632       7168       12288
//    int4, 1 token    15 / 16    18 / 19    18 / 20    24 / 21    24 / 21    28 / 25    32 / 29    52 / 51
//         32 tokens   74 / 86    92 / 103   97 / 108  138 / 112  141 / 115  154 / 128  172 / 147  273 / 256
//        128 tokens  126 / 135  148 / 157  152 / 162  235 / 167  242 / 172  257 / 189  280 / 213  439 / 381
//    bf16, 32 tokens 197 / 254  254 / 310  281 / 336  370 / 338  388 / 355  432 / 400  501 / 471  826 / 856
// The limit is the same with e4m3 and e2m1.
constexpr int kFewCus = 256;
inline bool few_narrow(int H) { return H <= 16 * kFewCus; }

// Steps of 16 rows that a workgroup takes past the weights at a time, by the rows that an expert has on average.  us of the whole call, 32
// experts of 7168 x 2048, top-8, one / two / four steps in the first kernel (one in the second):
//   rows an expert    int4, groups of 128     e2m1, groups of 32      e4m3                 bf16
//        8             161 / 162 / 196         179 / 174 / 211        278 / 275 / 282      515 / 520 / 511
//       12             186 / 185 / 215         200 / 197 / 228        316 / 303 / 311      563 / 561 / 547
//       16             228 / 222 / 246         249 / 239 / 262        403 / 360 / 368      711 / 636 / 625
//       24             293 / 278 / 287         321 / 301 / 307        537 / 456 / 449      928 / 771 / 752
//       32             358 / 346 / 342         393 / 373 / 367        663 / 574 / 527     1146 / 972 / 886
//   32 (16 experts)    189 / 188 / 175         210 / 203 / 186        356 / 312 / 274      607 / 518 / 450
// Two instead of one in the second kernel: 8 rows +1, +1, -3, +11 us, 12 rows -1, 0, -6, 0, 16 rows -8, -13, -20, -40, 32 rows -12, -21, -58,
// -97.  Popular experts (popularity (i + 1)^-1.1) move the limits down a little: at 12 rows +4, +2, -10, -7.
inline double few_rows(int T, int K, int E) { return (double)T * K / E; }
inline int few_up_steps(double rows) { return rows <= 12 ? 1 : rows <= 24 ? 2 : 4; }
inline int few_down_steps(double rows) { return rows <= 12 ? 1 : 2; }

}  // namespace ep
