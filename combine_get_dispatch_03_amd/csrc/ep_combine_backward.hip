// ep_combine_backward.hip -- gradient of the weighted combine.
//
//   out[t] = sum_k w[t,k] y[slot(t,k)]   =>   grad_y[slot(t,k)] = w[t,k] g[t],   grad_w[t,k] = <g[t], y[slot(t,k)]>
//
// One workgroup per token: its gradient row is read once into registers (a thread holds every kThreads-th 16-byte
// chunk), then for each entry the row of y is read and the row of grad_y written.  A slot belongs to one entry, so
// nothing is summed across workgroups.
#include "ep_device.hpp"
#include "ep_internal.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct Params {
    const uint16_t* g;
    const uint16_t* y;
    const float* w;
    uint16_t* gy;
    float* gw;
    const int32_t* slot;
    int H, K;
};

__device__ __forceinline__ float wave_sum(float v) {
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

__global__ __launch_bounds__(kThreads) void k_combine_backward(Params p) {
    __shared__ float part[kMaxTopk][kWaves];
    const int t = blockIdx.x, nchunk = p.H / 8;
    const u32x4* g = reinterpret_cast<const u32x4*>(p.g + (int64_t)t * p.H);
    for (int k = 0; k < p.K; ++k) {
        const int s = p.slot[(int64_t)t * p.K + k];
        float dot = 0.0f;
        if (s >= 0) {
            const float w = p.w ? p.w[(int64_t)t * p.K + k] : 1.0f;
            for (int c = threadIdx.x; c < nchunk; c += kThreads) {
                const u32x4 gv = g[c];
                if (p.gy) {
                    u32x4 o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(w * bf16lo(gv[i]), w * bf16hi(gv[i]));
                    st_nt(reinterpret_cast<u32x4*>(p.gy + (int64_t)s * p.H) + c, o);
                }
                if (p.gw) {
                    const u32x4 yv = ld_nt(reinterpret_cast<const u32x4*>(p.y + (int64_t)s * p.H) + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dot = fmaf(bf16lo(gv[i]), bf16lo(yv[i]), dot);
                        dot = fmaf(bf16hi(gv[i]), bf16hi(yv[i]), dot);
                    }
                }
            }
        }
        dot = wave_sum(dot);
        if (lane_id() == 0) part[k][threadIdx.x / kWave] = dot;
    }
    __syncthreads();
    if (p.gw && (int)threadIdx.x < p.K) {
        float sum = 0.0f;
        for (int i = 0; i < kWaves; ++i) sum += part[threadIdx.x][i];
        p.gw[(int64_t)t * p.K + threadIdx.x] = sum;
    }
}

}  // namespace

hipError_t launch_combine_backward(const Handle& h, const CombineBackwardArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const Params p{(const uint16_t*)a.grad_out, (const uint16_t*)a.y, a.topk_weights, (uint16_t*)a.grad_y, a.grad_w,
                   h.ws.slot, a.hidden, h.K};
    hipLaunchKernelGGL(k_combine_backward, dim3((unsigned)h.T), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace ep
