// ep_few_rules.hpp -- which kernels the layer for a few tokens takes: plain host code on the call's sizes.  (The host does not know the
// routing, so the rules go by what a uniform one gives.)
#pragma once

namespace ep {

constexpr int kFewWaves = 16;      // of a workgroup of the second kernel: as many entries can stand by themselves

// Each entry by itself, or an expert's entries together.  An entry by itself has its weights under way at once, but reads them
// itself; together, an expert's are read once, after its entries are found.  us of the whole call, by themselves / together, experts of
// 7168 x 2048, entries spread evenly over that many experts:
//                            int4, groups of 128      e4m3                     bf16
//    1 token of top-8 (16)       41 /  43               67 /  72               132 / 131
//    2 tokens of top-4 (8)       40 /  43               67 /  71               130 / 129
//    2 tokens of top-4 (4)       35 /  33               53 /  40               114 /  69
//    2 tokens of top-8 (16)      73 /  76              126 / 129               253 / 248
//    2 tokens of top-8 (8)       60 /  44              110 /  72               235 / 130
//    4 tokens of top-4 (4)       56 /  33               93 /  41               206 /  69
// Routed at random, 16 entries: of 16 experts (int4) 62 / 57, of 24 65 / 71, of 32 66 / 71, of 64 68 / 72; e4m3 109 / 95, 115 / 119, 111 / 119,
// 116 / 122; 8 entries of 8 experts 40 / 42 and 71 / 76.  Small experts, 256 x 512 in bf16: 8 entries of 8 11.3 / 13.8, of 4 11.0 / 11.7, 16
// of 8 15.7 / 15.3.  One token's entries have an expert each; of several tokens enough experts for few to be shared.
inline bool few_by_entry(int T, int K, int E) {
    const int n = T * K;
    return T == 1 || (n <= kFewWaves && (n <= 8 ? n : 2 * n) <= E);
}

// 16 output channels a workgroup of the second kernel, or 32, which have half as many loads of rows per byte of weights.  A CU has room for
// one workgroup: 16 as long as they are one round on the 256 CUs, otherwise 32.  us of the whole call, 16 / 32 channels, 64 experts of H x
// 1024, top-8:
//                     H = 2048     3584      4096       4224       4608      5632       7168       12288
//    int4, 1 token    14 / 16    17 / 19    18 / 20    22 / 20    23 / 21    27 / 25    31 / 29    51 / 47
//         32 tokens   68 / 80    86 / 98    91 / 102  130 / 107  132 / 110  145 / 123  163 / 141  255 / 244
//        128 tokens  121 / 130  143 / 152  147 / 156  224 / 161  231 / 167  247 / 183  270 / 207  418 / 362
//    bf16, 32 tokens 190 / 244  246 / 300  273 / 324  352 / 328  370 / 344  412 / 389  480 / 458  787 / 835
// The limit is the same with e4m3 and e2m1.
constexpr int kFewCus = 256;
inline bool few_narrow(int H) { return H <= 16 * kFewCus; }

// Steps of 16 rows that a workgroup takes past the weights at a time, by the rows that an expert has on average.  us of the whole call, 32
// experts of 7168 x 2048, top-8, one / two / four steps in the first kernel (one in the second):
//   rows an expert    int4, groups of 128     e2m1, groups of 32      e4m3                 bf16
//        8             157 / 159 / 193         177 / 171 / 209        271 / 270 / 279      504 / 508 / 500
//       12             182 / 181 / 210         195 / 192 / 224        313 / 300 / 309      545 / 543 / 528
//       16             224 / 217 / 241         244 / 234 / 257        396 / 355 / 363      694 / 619 / 607
//       24             286 / 273 / 281         315 / 295 / 300        528 / 446 / 438      911 / 752 / 731
//       32             350 / 337 / 335         383 / 364 / 357        652 / 564 / 517     1121 / 948 / 861
//   32 (16 experts)    184 / 184 / 170         204 / 198 / 182        349 / 307 / 268      595 / 506 / 438
// Two instead of one in the second kernel: 12 rows 0, 0, -5, -6 us, 16 rows -10, -15, -28, -49, 32 rows -13, -22, -54, -109.  Popular experts
// (popularity (i + 1)^-1.1) move the limits down a little: at 12 rows +3, +1, -7, -18.
inline double few_rows(int T, int K, int E) { return (double)T * K / E; }
inline int few_up_steps(double rows) { return rows <= 12 ? 1 : rows <= 24 ? 2 : 4; }
inline int few_down_steps(double rows) { return rows <= 12 ? 1 : 2; }

}  // namespace ep
