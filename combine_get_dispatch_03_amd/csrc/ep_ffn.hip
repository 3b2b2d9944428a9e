// ep_ffn.hip -- the experts' gated feed-forward block: which kernels a call takes.
#include "ep_ffn.hpp"

namespace ep {

hipError_t launch_expert_ffn(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const FfnSizes s = sizes(h, a);
    const hipError_t e = few_rows_up(s) ? launch_stream_up(h, a, stream)
                         : a.fp8        ? launch_tile_fp8_up(h, a, stream)
                                        : launch_tile_up(h, a, stream);
    if (e != hipSuccess) return e;
    return few_rows_down(s) ? launch_stream_down(h, a, stream)
           : a.fp8          ? launch_tile_fp8_down(h, a, stream)
                            : launch_tile_down(h, a, stream);
}

}  // namespace ep
