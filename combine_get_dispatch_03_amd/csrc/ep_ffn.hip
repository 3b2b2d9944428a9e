// ep_ffn.hip -- the experts' gated feed-forward block: which kernels a call takes.
#include "ep_ffn.hpp"

namespace ep {

hipError_t launch_expert_ffn(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    if (few_rows(h)) return launch_ffn_stream(h, a, stream);
    return a.fp8 ? launch_ffn_tile_fp8(h, a, stream) : launch_ffn_tile(h, a, stream);
}

}  // namespace ep
