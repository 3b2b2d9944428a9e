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
//          (exact): e2m1 by the conversion instruction, integers (-8 .. 7, two's complement) by way of v_cvt_off_f32_i4, which
//          gives a sixteenth of them (kUnit).  K is filled up with zeros to whole pieces.
#pragma once

#include "ep_device.hpp"
#include "ep_gemm_core.hpp"
#include "ep_internal.hpp"

namespace ep {

constexpr int kPieceK = 128, kPieceRows = 16, kPieceBytes = 1024;
inline __host__ __device__ int pieces_of(int K) { return (K + kPieceK - 1) / kPieceK; }

// A weight tensor of a launch: [matrices, N, K].
struct WeightArgs {
    const char* values;
    const char* scales;
    int N, K;
};

// Integers of four bits, bytes 0..3 of q: a sixteenth of each, low and high nibbles.
template <int BYTE>
__device__ __forceinline__ float sixteenth(uint32_t q) {
    float f;
    if constexpr (BYTE == 0) asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(q));
    if constexpr (BYTE == 1) asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(q));
    if constexpr (BYTE == 2) asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(q));
    if constexpr (BYTE == 3) asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(q));
    return f;
}
// The upper halves of two floats that bf16 holds exactly.
__device__ __forceinline__ int upper_halves(float lo, float hi) {
    return (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
__device__ __forceinline__ bf16x8 widen_int4x8(uint32_t q) {
    const uint32_t h = q >> 4;
    return __builtin_bit_cast(bf16x8, i32x4{upper_halves(sixteenth<0>(q), sixteenth<0>(h)), upper_halves(sixteenth<1>(q), sixteenth<1>(h)),
                                            upper_halves(sixteenth<2>(q), sixteenth<2>(h)), upper_halves(sixteenth<3>(q), sixteenth<3>(h))});
}
__device__ __forceinline__ bf16x8 widen_e2m1x8(uint32_t q) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// S: groups of a piece (4-bit).
template <WeightFormat F, int S>
struct Weights;

template <>
struct Weights<kWeightsBf16, 0> {
    static constexpr int kGroups = 1;
    static constexpr bool kScaled = false;
    static constexpr float kUnit = 1.0f;
    struct Raw {
        i32x4 v[4];
    };
    const char* at;
    int left;      // k of the lane's first fragment on
    static __device__ __forceinline__ int k_of(int j, int g) { return j * 32 + g * 8; }

    // Rows row0 .. row0 + 15 of a matrix; those from `end` on are taken as its last one (nobody uses their sums).
    __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0, int end) {
        const int r = row0 + (lane_id() & 15), g = lane_id() >> 4;
        at = w.values + (((int64_t)matrix * w.N + (r < end ? r : end - 1)) * w.K + g * 8) * 2;
        left = w.K - g * 8;
    }
    __device__ __forceinline__ Raw load(int piece) const {
        Raw raw;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            raw.v[j] = i32x4{0, 0, 0, 0};
            if (piece * kPieceK + j * 32 < left) raw.v[j] = *reinterpret_cast<const i32x4*>(at + (int64_t)piece * kPieceK * 2 + j * 64);
        }
        return raw;
    }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) { return __builtin_bit_cast(bf16x8, raw.v[j]); }
};

template <>
struct Weights<kWeightsE4m3, 0> {
    static constexpr int kGroups = 1;
    static constexpr bool kScaled = true;
    static constexpr float kUnit = 1.0f;
    struct Raw {
        i32x4 v[2];
        float scale;
    };
    const char* at;
    const float* scale;
    static __device__ __forceinline__ int k_of(int j, int g) { return (j >> 1) * 64 + g * 16 + (j & 1) * 8; }

    __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0, int) {
        at = w.values + ((int64_t)matrix * w.N + row0 + (lane_id() & 15)) * w.K + (lane_id() >> 4) * 16;
        scale = reinterpret_cast<const float*>(w.scales) + ((int64_t)matrix * (w.N / 128) + row0 / 128) * (w.K / 128);
    }
    __device__ __forceinline__ Raw load(int piece) const {
        Raw raw;
#pragma unroll
        for (int j = 0; j < 2; ++j) raw.v[j] = *reinterpret_cast<const i32x4*>(at + (int64_t)piece * kPieceK + j * 64);
        raw.scale = scale[piece];
        return raw;
    }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) {
        const i32x4 q = raw.v[j >> 1];
        return widen_e4m3x8(j & 1 ? i32x2{q[2], q[3]} : i32x2{q[0], q[1]});
    }
    static __device__ __forceinline__ f32x4 scales(const Raw& raw, int) { return f32x4{raw.scale, raw.scale, raw.scale, raw.scale}; }
};

template <WeightFormat F, int S>
struct Weights {
    static constexpr int kGroups = S;
    static constexpr bool kScaled = true;
    static constexpr float kUnit = F == kWeightsInt4 ? 16.0f : 1.0f;
    typedef int scale_regs __attribute__((ext_vector_type(2 * S)));
    struct Raw {
        i32x4 v;
        scale_regs s;      // 4 rows of each group, as bf16
    };
    const char* at;
    const char* scale;
    static __device__ __forceinline__ int k_of(int j, int g) { return j * 32 + g * 8; }

    __device__ __forceinline__ void init(const WeightArgs& w, int matrix, int row0, int) {
        const int64_t piece = ((int64_t)matrix * (w.N / kPieceRows) + row0 / kPieceRows) * pieces_of(w.K);
        at = w.values + piece * kPieceBytes + lane_id() * 16;
        scale = w.scales + piece * (32 * S) + (lane_id() >> 4) * (8 * S);
    }
    __device__ __forceinline__ Raw load(int piece) const {
        Raw raw;
        raw.v = *reinterpret_cast<const i32x4*>(at + (int64_t)piece * kPieceBytes);
        raw.s = *reinterpret_cast<const scale_regs*>(scale + (int64_t)piece * (32 * S));
        return raw;
    }
    static __device__ __forceinline__ bf16x8 fragment(const Raw& raw, int j) {
        return F == kWeightsInt4 ? widen_int4x8((uint32_t)raw.v[j]) : widen_e2m1x8((uint32_t)raw.v[j]);
    }
    static __device__ __forceinline__ f32x4 scales(const Raw& raw, int group) {
        const uint32_t a = (uint32_t)raw.s[2 * group], b = (uint32_t)raw.s[2 * group + 1];
        return f32x4{bf16lo(a), bf16hi(a), bf16lo(b), bf16hi(b)};
    }
};

// acc[MT] += the piece's products with 16 * MT rows (x: a fragment per row tile and instruction).
template <class W, int MT>
__device__ __forceinline__ void add_piece(const typename W::Raw& raw, const i32x4 (&x)[MT][4], f32x4 (&acc)[MT]) {
    constexpr int kPer = 4 / W::kGroups;
#pragma unroll
    for (int s = 0; s < W::kGroups; ++s) {
        f32x4 part[MT];
#pragma unroll
        for (int a = 0; a < MT; ++a) part[a] = W::kScaled ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[a];
#pragma unroll
        for (int j = s * kPer; j < (s + 1) * kPer; ++j) {
            const bf16x8 f = W::fragment(raw, j);
#pragma unroll
            for (int a = 0; a < MT; ++a) part[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, __builtin_bit_cast(bf16x8, x[a][j]), part[a], 0, 0, 0);
        }
        if constexpr (W::kScaled) {
            const f32x4 scale = W::scales(raw, s);
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[a][i] = fmaf(part[a][i], scale[i], acc[a][i]);
        } else {
#pragma unroll
            for (int a = 0; a < MT; ++a) acc[a] = part[a];
        }
    }
}

}  // namespace ep
