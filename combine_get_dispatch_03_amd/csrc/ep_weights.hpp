// ep_weights.hpp -- rows of weights in their formats on the way from memory into the fragments of the matrix instruction, for the
// kernels that stream them (ep_stream.hpp, ep_w4_tile.hip).
//
// A piece is 16 rows (output channels) by 128 k.  A lane (r = lane & 15, g = lane >> 4) holds row r's terms of four 16x16x32
// instructions, 8 k each; which k these are is the format's choice (k_of), as long as the other operand agrees.
//
//   bf16   rows [N, K] as they are.  K may end inside a piece: what does not exist is zero.
//   e4m3   rows [N, K] of bytes, an fp32 scale per 128 x 128 block; widened to bf16 (exact); the scale goes to the piece's sums.
//   4-bit  laid out once (pack): a piece is 1024 bytes in a row, 16 a lane, so a wave's load is whole lines of one place; a group
//          of 32, 64 or 128 k has a bf16 scale per row, which goes to the group's sums in fp32.  Codes are widened to bf16
//          (exact): e2m1 by the conversion instruction, integers (-8 .. 7, two's complement) by way of one that gives a sixteenth
//          of them as fp32 (kUnit).  K is filled up with zeros to whole pieces.  A piece's scales are [16 rows][groups].
//
// e4m3 and 4-bit codes are exact in fp16, too (kFitsF16).
//
// The rows that meet the weights are the instruction's first operand, so lane (r, g) ends up with weight row r's sums of rows
// 4 g .. 4 g + 3: one scale per group is all that it needs.
#pragma once

#include "ep_device.hpp"
#include "ep_gemm_core.hpp"
#include "ep_h_rows.hpp"
#include "ep_internal.hpp"

namespace ep {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kPieceK = 128, kPieceRows = 16, kPieceBytes = 1024;
inline __host__ __device__ int pieces_of(int K) { return (K + kPieceK - 1) / kPieceK; }

// A weight tensor of a launch: [matrices, N, K].
struct WeightArgs {
    const char* values;
    const char* scales;
    int N, K;
};

// Memory read through a buffer resource: base and what is added to it for a whole wave stand in scalar registers, and what lies
// at kNoElement or beyond the size is zero without a branch or any traffic.
struct Buffer {
    uint64_t base;

    __device__ __forceinline__ void init(const void* at) { base = uniform64((uint64_t)at); }
    // `there`: whether anything is read at all (the same in the whole wave, and said so: a resource that the compiler takes to differ
    // between lanes costs a loop per load)
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(bool there) const {
        return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, __builtin_amdgcn_readfirstlane(there ? (int)kNoElement : 0), 0x00020000);
    }
};
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t wave) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)lane, (int)wave, 0));
}

// Eight codes, widened pair by pair.
template <bool INT4>
struct Codes;
// Integers: a sixteenth of each.  The odd ones are shifted down once, and every byte of the two words is an operand of its own
// (left alone, the compiler shifts each nibble by itself).
template <>
struct Codes<true> {
    uint32_t even, odd;
    __device__ __forceinline__ explicit Codes(uint32_t q) : even(q), odd(q >> 4) { asm("" : "+v"(odd)); }
    static __device__ __forceinline__ float sixteenth(uint32_t q, int i) {
        return __builtin_amdgcn_cvt_off_f32_i4((int)(i == 0 ? q : i == 3 ? q >> 24 : q >> (i * 8) & 0xffu));
    }
    __device__ __forceinline__ int pair(int i) const { return upper_halves(sixteenth(even, i), sixteenth(odd, i)); }
    __device__ __forceinline__ int pair16(int i) const { return __builtin_bit_cast(int, __builtin_amdgcn_cvt_pkrtz(sixteenth(even, i), sixteenth(odd, i))); }
};
template <>
struct Codes<false> {
    uint32_t q;
    __device__ __forceinline__ explicit Codes(uint32_t v) : q(v) {}
    __device__ __forceinline__ int pair(int i) const {
        const bf16x2 v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 0)
                         : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 1)
                         : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 2)
                                  : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 3);
        return __builtin_bit_cast(int, v);
    }
    __device__ __forceinline__ int pair16(int i) const {
        const f16x2 v = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0)
                        : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1)
                        : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3);
        return __builtin_bit_cast(int, v);
    }
};
template <bool INT4>
__device__ __forceinline__ bf16x8 widen_codes(uint32_t q) {
    const Codes<INT4> c(q);
    return __builtin_bit_cast(bf16x8, i32x4{c.pair(0), c.pair(1), c.pair(2), c.pair(3)});
}
template <bool INT4>
__device__ __forceinline__ f16x8 widen_codes16(uint32_t q) {
    const Codes<INT4> c(q);
    return __builtin_bit_cast(f16x8, i32x4{c.pair16(0), c.pair16(1), c.pair16(2), c.pair16(3)});
}

// The bf16 scales of a row's S groups.
template <int S>
struct GroupScales {
    uint32_t v[S == 4 ? 2 : 1];

    __device__ __forceinline__ void load(const char* at) {
        if constexpr (S == 1) {
            v[0] = *reinterpret_cast<const uint16_t*>(at);
        } else if constexpr (S == 2) {
            v[0] = *reinterpret_cast<const uint32_t*>(at);
        } else {
            const i32x2 q = *reinterpret_cast<const i32x2*>(at);
            v[0] = (uint32_t)q[0], v[1] = (uint32_t)q[1];
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, uint32_t lane, uint32_t wave) {
        if constexpr (S == 1) {
            v[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, (int)lane, (int)wave, 0);
        } else if constexpr (S == 2) {
            v[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(b, (int)lane, (int)wave, 0);
        } else {
            const i32x2 q = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(b, (int)lane, (int)wave, 0));
            v[0] = (uint32_t)q[0], v[1] = (uint32_t)q[1];
        }
    }
    __device__ __forceinline__ float get(int group) const { return group & 1 ? bf16hi(v[group / 2]) : bf16lo(v[group / 2]); }
};

// of_block(): of the numbers of a piece's eight blocks (ep_h_rows.hpp), the one whose block the lane's terms of instruction j are in; here for
// k_of(j, g) = 32 j + 8 g.
__device__ __forceinline__ uint32_t of_block_32(i32x4 e, int j, int g) { return __builtin_amdgcn_ubfe((uint32_t)e[j], (g >> 1) * 16, 16); }

// NF rows of pieces of one matrix; S: groups of a piece (4-bit).  init(): the first row of the workgroup (uniform), and of each
// row of pieces how many weight rows behind it stands (a multiple of 16) and how many rows exist from there on.
template <WeightFormat F, int S>
struct Weights;

template <>
struct Weights<kWeightsBf16, 0> {
    static constexpr int kGroups = 1;
    static constexpr bool kScaled = false, kTail = true, kFitsF16 = false;
    static constexpr float kUnit = 1.0f;
    struct Raw {
        i32x4 v[4];
    };
    static __device__ __forceinline__ int k_of(int j, int g) { return j * 32 + g * 8; }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) { return __builtin_bit_cast(bf16x8, raw.v[j]); }
    static __device__ __forceinline__ uint32_t of_block(i32x4 e, int j, int g) { return of_block_32(e, j, g); }

    template <int NF>
    struct Rows {
        Buffer values;
        uint32_t at[NF];
        int K;
        __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0) {
            values.init(w.values + ((int64_t)matrix * w.N + row0) * w.K * 2);
            K = w.K;
        }
        __device__ __forceinline__ void place(int b, int behind, int exist) {
            const int r = lane_id() & 15;
            at[b] = r < exist ? (uint32_t)(behind + r) * (uint32_t)K * 2 + (lane_id() >> 4) * 16 : kNoElement;
        }
        __device__ __forceinline__ Raw load(int b, int piece, bool there) const {
            const __amdgpu_buffer_rsrc_t buffer = values.resource(there);
            Raw raw;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                raw.v[j] = load16(buffer, piece * kPieceK + k_of(j, lane_id() >> 4) < K ? at[b] + j * 64 : kNoElement, (uint32_t)piece * kPieceK * 2);
            return raw;
        }
    };
};

template <>
struct Weights<kWeightsE4m3, 0> {
    static constexpr int kGroups = 1;
    static constexpr bool kScaled = true, kTail = false, kFitsF16 = true;
    static constexpr float kUnit = 1.0f;
    struct Raw {
        i32x4 v[2];
        float scale;
    };
    static __device__ __forceinline__ int k_of(int j, int g) { return (j >> 1) * 64 + g * 16 + (j & 1) * 8; }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) {
        const i32x4 q = raw.v[j >> 1];
        return widen_e4m3x8(j & 1 ? i32x2{q[2], q[3]} : i32x2{q[0], q[1]});
    }
    static __device__ __forceinline__ f16x8 fragment16(const Raw& raw, int j) {
        const i32x4 q = raw.v[j >> 1];
        const int a = q[j & 1 ? 2 : 0], b = q[j & 1 ? 3 : 1];
        const f16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false), v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
        const f16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false), v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
        return f16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
    }
    static __device__ __forceinline__ uint32_t of_block(i32x4 e, int j, int g) {
        int lower = e[(j >> 1) * 2], upper = e[(j >> 1) * 2 + 1];
        asm("" : "+v"(lower), "+v"(upper));      // (as an index that differs between lanes they would go to memory)
        return __builtin_amdgcn_ubfe((uint32_t)(g >> 1 ? upper : lower), (g & 1) * 16, 16);
    }
    static __device__ __forceinline__ float scale_of(const Raw& raw, int) { return raw.scale; }

    template <int NF>
    struct Rows {
        Buffer values, scales;
        uint32_t at, row[NF], scale_row[NF];
        int K, in_block;
        __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0) {
            values.init(w.values + ((int64_t)matrix * w.N + row0) * w.K);
            scales.init(w.scales + ((int64_t)matrix * (w.N / 128) + row0 / 128) * (w.K / 128) * 4);
            at = (uint32_t)(lane_id() & 15) * (uint32_t)w.K + (lane_id() >> 4) * 16;
            K = w.K;
            in_block = row0 % 128;
        }
        __device__ __forceinline__ void place(int b, int behind, int) {
            row[b] = (uint32_t)behind * (uint32_t)K;
            scale_row[b] = (uint32_t)((in_block + behind) / 128 * (K / 128) * 4);
        }
        __device__ __forceinline__ Raw load(int b, int piece, bool there) const {
            const __amdgpu_buffer_rsrc_t buffer = values.resource(there);
            Raw raw;
#pragma unroll
            for (int j = 0; j < 2; ++j) raw.v[j] = load16(buffer, at + j * 64, row[b] + (uint32_t)piece * kPieceK);
            raw.scale = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(scales.resource(there), 0, (int)(scale_row[b] + piece * 4), 0));
            return raw;
        }
    };
};

template <WeightFormat F, int S>
struct Weights {
    static constexpr int kGroups = S;
    static constexpr bool kScaled = true, kTail = true, kFitsF16 = true;
    static constexpr float kUnit = F == kWeightsInt4 ? 16.0f : 1.0f;
    struct Raw {
        i32x4 v;
        GroupScales<S> s;
    };
    static __device__ __forceinline__ int k_of(int j, int g) { return j * 32 + g * 8; }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) {
        return widen_codes<F == kWeightsInt4>((uint32_t)raw.v[j]);
    }
    static __device__ __forceinline__ f16x8 fragment16(const Raw& raw, int j) {
        return widen_codes16<F == kWeightsInt4>((uint32_t)raw.v[j]);
    }
    static __device__ __forceinline__ uint32_t of_block(i32x4 e, int j, int g) { return of_block_32(e, j, g); }
    static __device__ __forceinline__ float scale_of(const Raw& raw, int group) { return raw.s.get(group); }

    template <int NF>
    struct Rows {
        Buffer values, scales;
        uint32_t first[NF];
        int pieces;
        __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0) {
            pieces = pieces_of(w.K);
            const int64_t piece = ((int64_t)matrix * (w.N / kPieceRows) + row0 / kPieceRows) * pieces;
            values.init(w.values + piece * kPieceBytes);
            scales.init(w.scales + piece * (32 * S));
        }
        __device__ __forceinline__ void place(int b, int behind, int) { first[b] = (uint32_t)(behind / kPieceRows * pieces); }
        __device__ __forceinline__ Raw load(int b, int piece, bool there) const {
            Raw raw;
            raw.v = load16(values.resource(there), lane_id() * 16, (first[b] + piece) * kPieceBytes);
            raw.s.load(scales.resource(there), (lane_id() & 15) * (2 * S), (first[b] + piece) * (32 * S));
            return raw;
        }
    };
};

// acc[NF][MT] += NF pieces' products with 16 * MT rows (x: a fragment per row tile and instruction).  H: the rows are h's, in fp16.
template <class W, bool H, int MT, int NF>
__device__ __forceinline__ void add_pieces(const typename W::Raw (&raw)[NF], const i32x4 (&x)[MT][4], f32x4 (&acc)[NF][MT]) {
    if constexpr (H && !W::kFitsF16) {
        static_assert(!W::kScaled);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            i32x4 first[MT], second[MT];
#pragma unroll
            for (int a = 0; a < MT; ++a) two_bf16(x[a][j], &first[a], &second[a]);
#pragma unroll
            for (int b = 0; b < NF; ++b)
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const bf16x8 f = W::fragment(raw[b], j);
                    acc[b][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, first[a]), f, acc[b][a], 0, 0, 0);
                    acc[b][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, second[a]), f, acc[b][a], 0, 0, 0);
                }
        }
    } else {
        constexpr int kPer = 4 / W::kGroups;
#pragma unroll
        for (int b = 0; b < NF; ++b)
#pragma unroll
            for (int s = 0; s < W::kGroups; ++s) {
                f32x4 part[MT];
#pragma unroll
                for (int a = 0; a < MT; ++a) part[a] = W::kScaled ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[b][a];
#pragma unroll
                for (int j = s * kPer; j < (s + 1) * kPer; ++j) {
                    if constexpr (H) {
                        const f16x8 f = W::fragment16(raw[b], j);
#pragma unroll
                        for (int a = 0; a < MT; ++a) part[a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x[a][j]), f, part[a], 0, 0, 0);
                    } else {
                        const bf16x8 f = W::fragment(raw[b], j);
#pragma unroll
                        for (int a = 0; a < MT; ++a) part[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[a][j]), f, part[a], 0, 0, 0);
                    }
                }
                if constexpr (W::kScaled) {
                    const float scale = W::scale_of(raw[b], s);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][a][i] = fmaf(part[a][i], scale, acc[b][a][i]);
                        // here, not wherever acc is used next: the compiler would sink it past the next loads' branch and keep all parts
                        asm volatile("" : "+v"(acc[b][a]));
                    }
                } else {
#pragma unroll
                    for (int a = 0; a < MT; ++a) acc[b][a] = part[a];
                }
            }
    }
}

}  // namespace ep
