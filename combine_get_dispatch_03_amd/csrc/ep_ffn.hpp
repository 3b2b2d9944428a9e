// ep_ffn.hpp -- the expert block's launchers (ep_ffn_rules.hpp chooses between them).
#pragma once

#include "ep_device.hpp"
#include "ep_ffn_rules.hpp"
#include "ep_internal.hpp"

namespace ep {

inline FfnSizes sizes(const Handle& h, const FfnArgs& a) { return FfnSizes{h.T, h.K, h.E, h.El, a.hidden, a.inter, a.fp8}; }

hipError_t launch_tile_up(const Handle& h, const FfnArgs& a, hipStream_t stream);           // bf16
hipError_t launch_tile_down(const Handle& h, const FfnArgs& a, hipStream_t stream);
hipError_t launch_tile_fp8_up(const Handle& h, const FfnArgs& a, hipStream_t stream);       // e4m3
hipError_t launch_tile_fp8_down(const Handle& h, const FfnArgs& a, hipStream_t stream);
hipError_t launch_stream_up(const Handle& h, const FfnArgs& a, hipStream_t stream);         // either
hipError_t launch_stream_down(const Handle& h, const FfnArgs& a, hipStream_t stream);

// The order in which workgroups take the tiles of a rows x cols grid.  Consecutive tiles run down kGroup rows, then on to
// the next column; 32 of them (4 x 8) are what the 32 CUs of an XCD work on at a time, few rows and few weights from its
// own L2.  Such batches go to the XCDs (workgroup number mod 8) in turn, so that experts with many rows are spread.  With
// fewer tiles than CUs the batches shrink, to keep every XCD at work.
constexpr int kXcds = 8, kGroup = 4, kBatch = 32;

struct TileAt {
    int row, col;
};
// Tile number `round` of workgroup `block` of kXcds * kBatch; false: there is none, nor in later rounds.
__device__ __forceinline__ bool tile_at(int block, int round, int rows, int cols, TileAt* t) {
    const int total = rows * cols, batch = total >= kXcds * kBatch ? kBatch : (total + kXcds - 1) / kXcds;
    const int in_batch = block / kXcds;
    const int i = (round * kXcds + block % kXcds) * batch + in_batch;
    if (in_batch >= batch || i >= total) return false;
    const int group = i / (kGroup * cols), first = group * kGroup;
    const int height = rows - first < kGroup ? rows - first : kGroup, in = i - group * kGroup * cols;
    t->row = first + in % height;
    t->col = in / height;
    return true;
}
// Workgroups to launch for at most `tiles` tiles: each walks through its rounds.
inline unsigned walking_blocks(int64_t tiles) { return (unsigned)(tiles < kXcds * kBatch ? (tiles + kXcds - 1) / kXcds * kXcds : kXcds * kBatch); }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(a, b), pack_bf16x2(c, d)};
}
template <class V4>
__device__ __forceinline__ void store8(uint16_t* p, V4 a, V4 b) {
    *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

}  // namespace ep
