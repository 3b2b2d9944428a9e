// ep_adapter.hip -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + s_a B_a (A_a x[t])      a = the token's adapter
//
// This first form gives a workgroup to each token: its rank inner products, then the output row.
#include "ep_device.hpp"
#include "ep_internal.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;

struct Params {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scales;
    const uint16_t* base;
    uint16_t* out;
    const int64_t* ids;
    int H, r, N, lo, El;
};

__device__ __forceinline__ float widen(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

__global__ __launch_bounds__(kThreads) void k_adapter(Params p) {
    __shared__ float v[kMaxAdapterRank];
    const int t = blockIdx.x;
    const int64_t id = p.ids[t] - p.lo;
    const bool has = p.ids[t] >= 0 && id >= 0 && id < p.El;
    if (has) {
        for (int j = threadIdx.x / kWave; j < p.r; j += kThreads / kWave) {
            float sum = 0.0f;
            const uint16_t* a = p.a + (id * p.r + j) * p.H;
            for (int k = lane_id(); k < p.H; k += kWave) sum = fmaf(widen(a[k]), widen(p.x[(int64_t)t * p.H + k]), sum);
            for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
            if (lane_id() == 0) v[j] = (float)(__bf16)(sum * (p.scales ? p.scales[id] : 1.0f));
        }
    }
    __syncthreads();
    for (int n = threadIdx.x; n < p.N; n += kThreads) {
        float sum = 0.0f;
        if (has)
            for (int j = 0; j < p.r; ++j) sum = fmaf(v[j], widen(p.b[(id * p.N + n) * p.r + j]), sum);
        const float base = p.base ? widen(p.base[(int64_t)t * p.N + n]) : 0.0f;
        p.out[(int64_t)t * p.N + n] = __builtin_bit_cast(uint16_t, (__bf16)(base + sum));
    }
}

}  // namespace

size_t adapter_workspace_bytes(int, int, int, int) { return 256; }

hipError_t launch_adapter(const Handle& h, const AdapterArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const Params p{(const uint16_t*)a.x, (const uint16_t*)a.a, (const uint16_t*)a.b, a.scales, (const uint16_t*)a.base,
                   (uint16_t*)a.out, h.topk_idx, a.hidden, a.rank, a.n_out, h.lo, h.El};
    hipLaunchKernelGGL(k_adapter, dim3((unsigned)h.T), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

}  // namespace ep
