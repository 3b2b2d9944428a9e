// ep_expert_tiles.hpp -- which rows of which expert a workgroup works on, from the device counts of a layout.
#pragma once

#include "ep_device.hpp"

namespace ep {

struct RowTile {
    int expert;   // local expert
    int m0;       // first row of the tile inside the expert's segment
    int rows;     // valid rows of the tile (1..BM)
};

// The tiles of all experts, in the experts' order: ceil(count / BM) each, as even in height as multiples of `unit` rows
// allow (1050 rows are five tiles of 224 and 154 rather than four of 256 and one of 26).  Every wave of a workgroup works
// them out for itself (no LDS, no barrier): lane l sums the tiles of experts [l * per, l * per + per) and a wave scan
// places them; find() then needs at most `per` (16 for 1024 experts) uniform steps.
template <int BM>
struct RowTiles {
    const int32_t* cnt;
    int El, per, sum, incl, total;

    __device__ __forceinline__ RowTiles(const int32_t* counts, int num_experts) : cnt(counts), El(num_experts) {
        per = (El + kWave - 1) / kWave;
        sum = 0;
        for (int i = 0; i < per; ++i) {
            const int e = lane_id() * per + i;
            if (e < El) sum += (cnt[e] + BM - 1) / BM;
        }
        incl = wave_inclusive_scan(sum);
        total = readlane(incl, kWave - 1);
    }

    __device__ __forceinline__ RowTile find(int t, int unit = BM) const {   // 0 <= t < total
        const int src = __builtin_ctzll(ballot(incl > t));
        int left = t - (readlane(incl, src) - readlane(sum, src));
        for (int e = src * per;; ++e) {
            const int c = __builtin_amdgcn_readfirstlane(cnt[e]);
            const int n = (c + BM - 1) / BM;
            if (left < n) {
                const int height = ((c + n - 1) / n + unit - 1) / unit * unit, m0 = left * height;
                return RowTile{e, m0, c - m0 < height ? c - m0 : height};
            }
            left -= n;
        }
    }
};

}  // namespace ep
