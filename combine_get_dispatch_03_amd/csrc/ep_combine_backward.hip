// ep_combine_backward.hip -- gradient of the weighted combine.
//
//   out[t] = sum_k w[t,k] y[slot(t,k)]   =>   grad_y[slot(t,k)] = w[t,k] g[t],   grad_w[t,k] = <g[t], y[slot(t,k)]>
//
// One workgroup per token: bound by reading y's rows and writing grad_y's (2 * 2H bytes per routed entry).  The token's
// slots and weights are one load, in lanes; its gradient row stays in registers (kChunks 16-byte chunks a thread) while
// the token's valid entries go by, kBatch at a time: their rows of y are all requested before the first is used, so a
// thread has kBatch * kChunks loads in flight.  A slot belongs to one entry, so nothing is summed across workgroups; a
// thread's products, then the wave's (by lane exchange), then the waves' are added in a fixed order.
// Measured at 4096 tokens, top-8, 7168 channels (1.0 GB): 192 us, 5.2 TB/s, what this chip takes of scattered row stores
// beside as many reads (201 us one entry after the other; 2, 4 or 8 entries at a time and 2 or 4 chunks a thread within
// 1%; plain loads of y 203 us).  61 tokens, top-6, 1032 channels: 4.6 us with 2 chunks, 5.6 with 4.
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
    int T, H, K;
};

constexpr int kChunks = 2, kBatch = 4;

// Sum over the 64 lanes, the same in every lane: within each 16 lanes by row rotations, then the four rows' sums.
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp_f<0x128>(v);     // row_ror:8
    v += dpp_f<0x124>(v);     // row_ror:4
    v += dpp_f<0x122>(v);     // row_ror:2
    v += dpp_f<0x121>(v);     // row_ror:1
    return (readlane_f(v, 0) + readlane_f(v, 16)) + (readlane_f(v, 32) + readlane_f(v, 48));
}

__device__ __forceinline__ float dot8(u32x4 a, u32x4 b, float sum) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = fmaf(bf16lo(a[i]), bf16lo(b[i]), sum);
        sum = fmaf(bf16hi(a[i]), bf16hi(b[i]), sum);
    }
    return sum;
}

__global__ __launch_bounds__(kThreads) void k_combine_backward(Params p) {
    __shared__ float part[kWaves][kMaxTopk];
    const int64_t token = block_id();
    if (token >= p.T) return;
    const int t = (int)token, nchunk = p.H / 8, lane = lane_id(), wave = threadIdx.x / kWave;
    const int64_t entry = (int64_t)t * p.K + (lane < p.K ? lane : 0);
    const int slot = lane < p.K ? p.slot[entry] : -1;
    const float weight = p.w ? p.w[entry] : 1.0f;
    const u32x4* g = reinterpret_cast<const u32x4*>(p.g + (int64_t)t * p.H);
    const uint64_t valid = ballot(slot >= 0);
    float mine = 0.0f;      // lane k: this wave's part of entry k's dot product
    for (int c0 = 0; c0 < nchunk; c0 += kChunks * kThreads) {      // the same for every lane: sums cross lanes
        u32x4 gv[kChunks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int c = c0 + j * kThreads + (int)threadIdx.x;
            gv[j] = c < nchunk ? g[c] : u32x4{0, 0, 0, 0};
        }
        for (uint64_t left = valid; left != 0;) {
            int k[kBatch], row[kBatch];
            bool there[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                there[b] = left != 0;
                k[b] = there[b] ? __builtin_ctzll(left) : k[0];
                left &= left - 1;
                row[b] = readlane(slot, k[b]);
            }
            u32x4 yv[kBatch][kChunks];
            if (p.gw) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) {
                        const int c = c0 + j * kThreads + (int)threadIdx.x;
                        yv[b][j] = u32x4{0, 0, 0, 0};
                        if (there[b] && c < nchunk) yv[b][j] = ld_nt(reinterpret_cast<const u32x4*>(p.y + (int64_t)row[b] * p.H) + c);
                    }
            }
            if (p.gy) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    const float w = readlane_f(weight, k[b]);
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) {
                        const int c = c0 + j * kThreads + (int)threadIdx.x;
                        u32x4 o;
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(w * bf16lo(gv[j][i]), w * bf16hi(gv[j][i]));
                        if (there[b] && c < nchunk) st_nt(reinterpret_cast<u32x4*>(p.gy + (int64_t)row[b] * p.H) + c, o);
                    }
                }
            }
            if (p.gw) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (!there[b]) break;
                    float dot = 0.0f;
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) dot = dot8(gv[j], yv[b][j], dot);
                    dot = wave_sum(dot);
                    mine += lane == k[b] ? dot : 0.0f;
                }
            }
        }
    }
    if (!p.gw) return;
    if (lane < p.K) part[wave][lane] = mine;
    __syncthreads();
    if ((int)threadIdx.x < p.K) {
        float sum = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) sum += part[i][threadIdx.x];
        p.gw[(int64_t)t * p.K + threadIdx.x] = sum;
    }
}

}  // namespace

hipError_t launch_combine_backward(const Handle& h, const CombineBackwardArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const Params p{(const uint16_t*)a.grad_out, (const uint16_t*)a.y, a.topk_weights, (uint16_t*)a.grad_y, a.grad_w,
                   h.ws.slot, h.T, a.hidden, h.K};
    hipLaunchKernelGGL(k_combine_backward, grid_of(h.T), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace ep
