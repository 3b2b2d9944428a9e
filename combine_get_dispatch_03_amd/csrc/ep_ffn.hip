// ep_ffn.hip -- the experts' gated feed-forward block over expert-major rows, and its gradients.
//
//   forward    g|u = x W13^T,  h = silu(g) u,  y = h W2^T
//   backward   dh = dy W2,  du = dh silu(g),  dg = dh u s (1 + g (1 - s)),  dx = (dg|du) W13,
//              dW13 = (dg|du)^T x,  dW2 = dy^T h                               (s = 1 / (1 + exp(-g)))
//
// Six products over ragged segments.  This first form is one kernel template: 64 x 64 outputs per workgroup, operands
// widened to fp32 in LDS, fp32 FMA; a product is a functor that says how an element is read and what is done with
// the sums.
#include "ep_device.hpp"
#include "ep_expert_tiles.hpp"
#include "ep_ffn.hpp"

namespace ep {
namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;

__device__ __forceinline__ float widen(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
__device__ __forceinline__ float widen8(uint8_t b) { return __builtin_amdgcn_cvt_f32_fp8((int)b, 0); }
__device__ __forceinline__ uint16_t narrow(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

struct Segments {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
};

struct GateUp {   // S = x rows, F = gate rows and up rows of W13
    static constexpr int kSums = 2;
    Segments seg;
    const void* x; const float* xs; const void* w; const float* ws;
    float* pre; uint16_t* h;
    int H, I; bool fp8;
    __device__ int N() const { return I; }
    __device__ int K() const { return H; }
    __device__ float s(int64_t row, int k) const {
        const int64_t i = row * H + k;
        return fp8 ? widen8(((const uint8_t*)x)[i]) * xs[row * (H / 128) + k / 128] : widen(((const uint16_t*)x)[i]);
    }
    __device__ float f(int j, int e, int n, int k) const {
        const int64_t r = (int64_t)e * 2 * I + j * I + n, i = r * H + k;
        return fp8 ? widen8(((const uint8_t*)w)[i]) * ws[r / 128 * (H / 128) + k / 128] : widen(((const uint16_t*)w)[i]);
    }
    __device__ void put(int64_t row, int, int n, const float* v) const {
        if (pre) pre[row * 2 * I + n] = v[0], pre[row * 2 * I + I + n] = v[1];
        h[row * I + n] = narrow(v[0] / (1.0f + __expf(-v[0])) * v[1]);
    }
};

struct Down {   // S = h rows, F = W2 rows
    static constexpr int kSums = 1;
    Segments seg;
    const uint16_t* h; const void* w; const float* ws; uint16_t* y;
    int H, I; bool fp8;
    __device__ int N() const { return H; }
    __device__ int K() const { return I; }
    __device__ float s(int64_t row, int k) const { return widen(h[row * I + k]); }
    __device__ float f(int, int e, int n, int k) const {
        const int64_t r = (int64_t)e * H + n, i = r * I + k;
        return fp8 ? widen8(((const uint8_t*)w)[i]) * ws[r / 128 * (I / 128) + k / 128] : widen(((const uint16_t*)w)[i]);
    }
    __device__ void put(int64_t row, int, int n, const float* v) const { y[row * H + n] = narrow(v[0]); }
};

template <class Get>
__device__ __forceinline__ void load_tile(float (*dst)[kTile + 1], int rows, int cols_k, Get get) {
    for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
        const int r = i / kStep, k = i % kStep;
        dst[k][r] = r < rows && k < cols_k ? get(r, k) : 0.0f;
    }
}

// Rows of one expert against the expert's weights.
template <class Op>
__global__ __launch_bounds__(kThreads) void k_rows(Op op) {
    __shared__ float S[kStep][kTile + 1], F[Op::kSums][kStep][kTile + 1];
    const RowTiles<kTile> tiles(op.seg.cnt, op.seg.El);
    if ((int)blockIdx.y >= tiles.total) return;
    const RowTile t = tiles.find((int)blockIdx.y);
    const int64_t row0 = (int64_t)op.seg.psum[t.expert] + t.m0;
    const int n0 = blockIdx.x * kTile, nn = min(kTile, op.N() - n0);
    const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
    float acc[Op::kSums][4][4] = {};
    for (int k0 = 0; k0 < op.K(); k0 += kStep) {
        const int kk = min(kStep, op.K() - k0);
        load_tile(S, t.rows, kk, [&](int r, int k) { return op.s(row0 + r, k0 + k); });
        for (int j = 0; j < Op::kSums; ++j)
            load_tile(F[j], nn, kk, [&](int r, int k) { return op.f(j, t.expert, n0 + r, k0 + k); });
        __syncthreads();
        for (int k = 0; k < kStep; ++k)
            for (int j = 0; j < Op::kSums; ++j)
                for (int a = 0; a < 4; ++a)
                    for (int b = 0; b < 4; ++b)
                        acc[j][a][b] = fmaf(S[k][tm + 16 * a], F[j][k][tn + 16 * b], acc[j][a][b]);
        __syncthreads();
    }
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const int m = tm + 16 * a, n = tn + 16 * b;
            if (m >= t.rows || n >= nn) continue;
            float v[Op::kSums];
            for (int j = 0; j < Op::kSums; ++j) v[j] = acc[j][a][b];
            op.put(row0 + m, t.expert, n0 + n, v);
        }
}

int tiles(int64_t n) { return (int)((n + kTile - 1) / kTile); }

// Row tiles any routing of the handle can give: every expert may end in a short one.
int row_tiles(const Handle& h) { return (int)((int64_t)h.T * h.K / kTile) + h.El; }

template <class Op>
hipError_t rows_launch(const Handle& h, const Op& op, int N, hipStream_t stream) {
    hipLaunchKernelGGL(k_rows<Op>, dim3((unsigned)tiles(N), (unsigned)row_tiles(h)), dim3(kThreads), 0, stream, op);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_ffn(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    if (!a.fp8) return launch_ffn_tile(h, a, stream);
    const Segments seg{h.ws.cnt_local, h.ws.psum, h.El};
    hipError_t e = rows_launch(h, GateUp{seg, a.x, a.x_scales, a.w13, a.w13_scales, a.pre, a.h, a.hidden, a.inter, a.fp8},
                               a.inter, stream);
    if (e != hipSuccess) return e;
    return rows_launch(h, Down{seg, a.h, a.w2, a.w2_scales, (uint16_t*)a.y, a.hidden, a.inter, a.fp8}, a.hidden, stream);
}

}  // namespace ep
