// ep_ffn.hpp -- the expert block's launchers and the rules that choose between them.
#pragma once

#include "ep_internal.hpp"

namespace ep {

// Rows an expert gets on average.  The host knows sizes only, not the routing: of T * K entries, an expert's share.
inline double mean_rows(const Handle& h) { return (double)h.T * h.K / h.E; }

// Row tiles of 256 rather than 128.
inline bool many_rows(const Handle& h) { return mean_rows(h) >= 192; }

hipError_t launch_ffn_tile(const Handle& h, const FfnArgs& a, hipStream_t stream);   // bf16

}  // namespace ep
