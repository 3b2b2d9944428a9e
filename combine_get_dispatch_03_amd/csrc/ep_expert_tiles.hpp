// ep_expert_tiles.hpp -- which rows of which expert a workgroup works on, from the device counts of a layout.
#pragma once

#include "ep_device.hpp"

namespace ep {

struct RowTile {
    int expert;   // local expert
    int row0;     // first row of the tile
    int rows;     // valid rows of the tile (1..BM)
};

// The tiles of all experts, in the experts' order: ceil(count / BM) each, as even in height as multiples of `unit` rows
// allow (1050 rows are five tiles of 224 and 154 rather than four of 256 and one of 26).  Every wave of a workgroup works
// them out for itself (no LDS, no barrier): lane l takes experts [l * per, l * per + per), a wave scan places their tiles,
// and of the first KEPT experts of each lane (4: of up to 256) counts and starts stay in registers for find().
template <int BM, int KEPT = 4>
struct RowTiles {
    static constexpr int kKept = KEPT;
    const int32_t* cnt;
    const int32_t* psum;
    int per, sum, incl, total;
    int count[kKept > 0 ? kKept : 1], start[kKept > 0 ? kKept : 1];

    __device__ __forceinline__ RowTiles(const int32_t* counts, const int32_t* starts, int El) : cnt(counts), psum(starts) {
        per = (El + kWave - 1) / kWave;
        sum = 0;
        const int e0 = lane_id() * per;
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            const bool in = i < per && e0 + i < El;
            count[i] = in ? cnt[e0 + i] : 0;
            start[i] = in ? psum[e0 + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kKept; ++i) sum += (count[i] + BM - 1) / BM;
        for (int i = kKept; i < per; ++i)
            if (e0 + i < El) sum += (cnt[e0 + i] + BM - 1) / BM;
        incl = wave_inclusive_scan(sum);
        total = readlane(incl, kWave - 1);
    }

    static __device__ __forceinline__ RowTile split(int e, int first, int c, int n, int i, int unit) {
        const int height = ((c + n - 1) / n + unit - 1) / unit * unit, m0 = i * height;
        return RowTile{e, first + m0, c - m0 < height ? c - m0 : height};
    }

    __device__ __forceinline__ RowTile find(int t, int unit = BM) const {   // 0 <= t < total
        const int src = __builtin_ctzll(ballot(incl > t));
        int left = t - (readlane(incl, src) - readlane(sum, src));
#pragma unroll
        for (int i = 0; i < kKept; ++i) {
            const int c = readlane(count[i], src), n = (c + BM - 1) / BM;
            if (left < n) return split(src * per + i, readlane(start[i], src), c, n, left, unit);
            left -= n;
        }
        for (int e = src * per + kKept;; ++e) {
            const int c = __builtin_amdgcn_readfirstlane(cnt[e]), n = (c + BM - 1) / BM;
            if (left < n) return split(e, __builtin_amdgcn_readfirstlane(psum[e]), c, n, left, unit);
            left -= n;
        }
    }
};

// Counts and starts of up to 256 experts in a wave's registers, of more in memory.
struct ExpertRows {
    const int32_t* cnt;
    const int32_t* psum;
    int count[4], start[4];

    __device__ __forceinline__ ExpertRows(const int32_t* counts, const int32_t* starts, int El) : cnt(counts), psum(starts) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = i * kWave + lane_id();
            count[i] = e < El ? cnt[e] : 0;
            start[i] = e < El ? psum[e] : 0;
        }
    }
    __device__ __forceinline__ RowTile get(int e) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e < (i + 1) * kWave) return RowTile{e, readlane(start[i], e & 63), readlane(count[i], e & 63)};
        return RowTile{e, __builtin_amdgcn_readfirstlane(psum[e]), __builtin_amdgcn_readfirstlane(cnt[e])};
    }
};

}  // namespace ep
