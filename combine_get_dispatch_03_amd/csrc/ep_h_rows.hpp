// ep_h_rows.hpp -- h, the experts' input of the second product, as it stands in the workspace between the two kernels.
//
// As one bf16 it would put the result 0.0023 to 0.0025 from the one in 64 bits (relative, Euclidean), where the result's own rounding to
// bf16 leaves 0.0016 to 0.0017.  So it keeps three bits more, as fp16, whose range is made up for by numbers beside it: a row is [I channels in
// fp16][numbers], h_pitch(I) elements in whole lines.  16 channels share a number E and are h 2^(154 - E), the largest below 2^14: E - 140 is
// the exponent of 2 above it among -8, 8, 24 and so on, or E is 0 for zeros.  In such wide steps the blocks of a row nearly always
// have the same number, and what the product does is to multiply a row's sums by 2^(E - 154).  Blocks with smaller numbers than the
// row's largest are brought to it first.  2^-11 of a value at most is lost, or 2^-23 of the row's largest: an eighth of a bf16 rounding,
// which with the result's own is 1.008 times that alone.  Infinities and NaN stay.  Numbers have 16 bits and room for whole eights; behind
// them is room for the row's unit in fp32.
//
// e4m3 and 4-bit weights are exact in fp16, which is what their products with h are in.  bf16 weights are not: there fp16 values are taken
// apart into two bf16 (exactly), and the second product takes its instructions twice.
#pragma once

#include "ep_device.hpp"
#include "ep_ffn.hpp"
#include "ep_internal.hpp"

namespace ep {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kShared = 16;      // channels of a block
inline __host__ __device__ constexpr int numbers_of(int I) { return (I + 8 * kShared - 1) / (8 * kShared) * 8; }

// Max of the bits of values without their signs (which is theirs, NaN above all) over 4, 8 or 16 neighbouring lanes.
template <int LANES>
__device__ __forceinline__ uint32_t max_bits(uint32_t v) {
    const auto with = [](uint32_t x, float y) { return max(x, __builtin_bit_cast(uint32_t, y)); };
    const auto f = [](uint32_t x) { return __builtin_bit_cast(float, x); };
    v = with(v, dpp_f<0xB1>(f(v)));                              // quad_perm [1,0,3,2]
    v = with(v, dpp_f<0x4E>(f(v)));                              // quad_perm [2,3,0,1]
    if constexpr (LANES >= 8) v = with(v, dpp_f<0x141>(f(v)));   // row_half_mirror
    if constexpr (LANES >= 16) v = with(v, dpp_f<0x128>(f(v)));  // row_ror:8
    return v;
}
__device__ __forceinline__ uint32_t size_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

// The upper halves of two floats, and what they leave of one (nothing of infinities and NaN).
__device__ __forceinline__ int upper_halves(float lo, float hi) {
    return (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
__device__ __forceinline__ float upper_half(float v) { return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v) & 0xffff0000u); }
__device__ __forceinline__ float rest_of(float v) {
    const float rest = v - upper_half(v);
    return size_bits(v) >= 0x7f800000u ? 0.0f : rest;
}

// From the bits of the largest: 118 + 16 n < exponent field <= 134 + 16 n gives 148 + 16 n.
__device__ __forceinline__ int block_number(uint32_t most) { return most ? (int)((((most >> 23) + 9u) & ~15u) + 20u) : 0; }
__device__ __forceinline__ float shared_value(float v, int e) { return ldexpf(v, 154 - e); }
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) { return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b}); }
// Channels c .. c + 3 of a row, zeros behind its end; the four lanes of a block's 16 call it together.
template <class V4>
__device__ __forceinline__ void store4_h(uint16_t* row, int I, int c, V4 v) {
    const int e = block_number(max_bits<4>(max(max(size_bits(v[0]), size_bits(v[1])), max(size_bits(v[2]), size_bits(v[3])))));
    if (c >= I) return;
    *reinterpret_cast<u32x2*>(row + c) = u32x2{pack_f16x2(shared_value(v[0], e), shared_value(v[1], e)), pack_f16x2(shared_value(v[2], e), shared_value(v[3], e))};
    if (c % kShared == 0) row[I + c / kShared] = (uint16_t)e;
}
// Eight fp16 as two bf16 each.
template <class V>
__device__ __forceinline__ void two_bf16(V x, V* first, V* second) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const f16x2 v = __builtin_bit_cast(f16x2, (int)x[d]);
        const float a = (float)v[0], b = (float)v[1];
        (*first)[d] = upper_halves(a, b);
        (*second)[d] = upper_halves(rest_of(a), rest_of(b));
    }
}
// Eight values of a block with number e, brought to `top`.  (Where there is no block the values are zeros and e is anything.)
template <class V>
__device__ __forceinline__ V bring_to(V x, int e, int top) {
    const _Float16 f = __builtin_amdgcn_ldexph((_Float16)1.0f, min(e - top, 0));
#pragma unroll
    for (int d = 0; d < 4; ++d) x[d] = __builtin_bit_cast(int, __builtin_bit_cast(f16x2, (int)x[d]) * f16x2{f, f});
    return x;
}
// Largest and smallest number of blocks, two at a time (of those that there are); zeros' count for neither.
struct NumberRange {
    u16x2 most{0, 0}, least{0xffff, 0xffff};      // least: less one
    __device__ __forceinline__ void add(uint32_t two, int there) {
        const u16x2 e = __builtin_bit_cast(u16x2, there <= 0 ? 0u : there == 1 ? two & 0xffffu : two);
        most = __builtin_elementwise_max(most, e);
        least = __builtin_elementwise_min(least, (u16x2)(e - u16x2{1, 1}));
    }
    __device__ __forceinline__ int top() const { return max((int)most[0], (int)most[1]); }
    __device__ __forceinline__ int low() const { return min((int)least[0], (int)least[1]) + 1; }
};
// What sums of a row's values are to be multiplied by.
__device__ __forceinline__ float shared_unit(int top) { return ldexpf(1.0f, top - 154); }

}  // namespace ep
