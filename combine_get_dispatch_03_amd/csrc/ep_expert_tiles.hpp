// ep_expert_tiles.hpp -- which rows of which expert a workgroup works on, from the device counts of a layout.
#pragma once

#include "ep_device.hpp"

namespace ep {

struct RowTile {
    int expert;   // local expert
    int m0;       // first row of the tile inside the expert's segment
    int rows;     // valid rows of the tile (1..BM)
    int total;    // tiles of all experts
};

// The `t`-th tile of BM rows, experts in order, ceil(count / BM) tiles each.  Every wave of the workgroup works it
// out for itself (no LDS, no barrier): lane l sums the tiles of experts [l * per, l * per + per), a wave scan finds the
// lane, and at most `per` (16 for 1024 experts) uniform steps find the expert.  expert = -1: t is past the last tile.
template <int BM>
__device__ __forceinline__ RowTile find_row_tile(const int32_t* cnt, int El, int t) {
    const int lane = lane_id();
    const int per = (El + kWave - 1) / kWave;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e < El) sum += (cnt[e] + BM - 1) / BM;
    }
    const int incl = wave_inclusive_scan(sum);
    RowTile r;
    r.total = readlane(incl, kWave - 1);
    r.expert = -1;
    r.m0 = r.rows = 0;
    if (t >= r.total) return r;
    const int src = __builtin_ctzll(ballot(incl > t));
    int left = t - (readlane(incl, src) - readlane(sum, src));
    for (int e = src * per;; ++e) {
        const int c = __builtin_amdgcn_readfirstlane(cnt[e]);
        const int n = (c + BM - 1) / BM;
        if (left < n) {
            r.expert = e;
            r.m0 = left * BM;
            r.rows = c - r.m0 < BM ? c - r.m0 : BM;
            return r;
        }
        left -= n;
    }
}

}  // namespace ep
