// ep_w4.hpp -- the launchers of the expert block with 4-bit weights (ep_w4_rules.hpp chooses between them).
#pragma once

#include "ep_internal.hpp"
#include "ep_w4_rules.hpp"

namespace ep {

hipError_t launch_w4_tile_up(const Handle& h, const W4Args& a, W4Kernel kernel, hipStream_t stream);
hipError_t launch_w4_tile_down(const Handle& h, const W4Args& a, W4Kernel kernel, hipStream_t stream);

}  // namespace ep
