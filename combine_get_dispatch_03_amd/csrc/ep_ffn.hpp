// ep_ffn.hpp -- the expert block's launchers and the rules that choose between them.
#pragma once

#include "ep_device.hpp"
#include "ep_internal.hpp"

namespace ep {

// Rows an expert gets on average.  The host knows sizes only, not the routing: of T * K entries, an expert's share.
inline double mean_rows(const Handle& h) { return (double)h.T * h.K / h.E; }

// Weights streamed past the rows rather than tiles of both through LDS.
inline bool few_rows(const Handle& h) { return mean_rows(h) < 48; }

hipError_t launch_ffn_tile(const Handle& h, const FfnArgs& a, hipStream_t stream);       // bf16
hipError_t launch_ffn_tile_fp8(const Handle& h, const FfnArgs& a, hipStream_t stream);   // e4m3
hipError_t launch_ffn_stream(const Handle& h, const FfnArgs& a, hipStream_t stream);     // either, few rows per expert

// Workgroups of one XCD (every eighth) take consecutive tiles, and a run of consecutive tiles is kGroup row tiles by
// as many channel tiles as fit, so that what an XCD's 32 CUs read at a time is few rows and few weights, from its own L2.
constexpr int kXcds = 8, kGroup = 4;

struct TileAt {
    int row, col;
};
__device__ __forceinline__ bool tile_at(int block, int rows, int cols, TileAt* t) {
    const int total = rows * cols, share = (total + kXcds - 1) / kXcds;
    const int at = block / kXcds, i = block % kXcds * share + at;
    if (at >= share || i >= total) return false;
    const int group = i / (kGroup * cols), first = group * kGroup;
    const int height = rows - first < kGroup ? rows - first : kGroup, in = i - group * kGroup * cols;
    t->row = first + in % height;
    t->col = in / height;
    return true;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(a, b), pack_bf16x2(c, d)};
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + __expf(-g)); }

// Workgroups for `tiles` tiles, as tile_at() deals them out.
inline unsigned tile_blocks(int64_t tiles) { return (unsigned)((tiles + kXcds - 1) / kXcds * kXcds); }

}  // namespace ep
