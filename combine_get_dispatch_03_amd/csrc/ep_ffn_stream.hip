// ep_ffn_stream.hip -- the expert block's forward pass for few rows per expert (decode): bound by reading the weights.
//
// A workgroup takes up to 16, 32 or 64 rows of an expert and 32 or 64 rows of its weights: half gate and the same up
// channels, or output channels.  Its four waves split k: each streams its part of the weight rows from memory straight into the
// fragments of the matrix instruction, the next step's loads in flight while the current one is multiplied; nothing is
// shared, so no barrier stands in the loop.  The rows' fragments come from the caches.  At the end the waves' sums meet
// in LDS.
// Measured, 7168 x 2048: one token of 8 experts, bf16, gate and up 80 us (5.9 TB/s), down 46 us (5.1); 256 experts, e4m3, 4
// rows each, down 0.65 ms (5.7 TB/s).  Experts of 256 x 512 with 32 rows: 6.0 and 5.0 us, launch and latency.
// h is rounded to bf16, as on tiles.
#include "ep_expert_tiles.hpp"
#include "ep_ffn.hpp"
#include "ep_gemm_core.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
    const void* s;
    const float* s_scales;
    const void* f;
    const float* f_scales;
    uint16_t* out;
    float* pre;
    int N, K;      // channels of a projection's output, of its input
    int sp, op;    // elements between rows of s and of out
};

enum Format { kBf16, kFp8 };

// 128 bytes of each of a wave's weight rows: the lane's two 16-byte pieces per fragment.
template <int NF>
struct Weights {
    i32x4 v[NF][2];
};
template <Format F, bool UP>
struct RowsOf;
template <bool UP>
struct RowsOf<kBf16, UP> { static constexpr int kPieces = 2; };     // 64 k of bf16
template <>
struct RowsOf<kFp8, true> { static constexpr int kPieces = 2; };    // 128 k of e4m3
template <>
struct RowsOf<kFp8, false> { static constexpr int kPieces = 4; };   // 128 k of bf16 beside e4m3 weights

template <Format F, bool UP, int COLS, int MT>
__device__ __forceinline__ void product(const Params& p, const RowTile& t, int n0, char* smem) {
    constexpr int kCols = COLS, kNF = kCols / 16, kSumPitch = kCols + 4;
    const int64_t row0 = t.row0;
    constexpr int kPieces = RowsOf<F, UP>::kPieces;
    constexpr int kWide = F == kFp8 ? 1 : 2;                   // bytes of a weight
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    const int f_bytes = p.K * kWide;                           // of a weight row
    const int steps = (f_bytes + 127) / 128;

    const char* f[kNF];
    bool f_there[kNF];
#pragma unroll
    for (int b = 0; b < kNF; ++b) {
        const int c = UP ? n0 + b % (kNF / 2) * 16 + r : n0 + b * 16 + r;
        f_there[b] = c < p.N;
        const int64_t row = (int64_t)t.expert * (UP ? 2 : 1) * p.N + (UP && b >= kNF / 2 ? p.N : 0) + (f_there[b] ? c : n0);
        f[b] = (const char*)p.f + row * f_bytes + g * 16;
    }
    const char* s[MT];
    bool s_there[MT];
    const int s_bytes = UP ? f_bytes : p.K * 2, s_pitch = p.sp * (UP ? kWide : 2);
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        s_there[a] = a * 16 + r < t.rows;
        s[a] = (const char*)p.s + (row0 + (s_there[a] ? a * 16 + r : 0)) * s_pitch + (F == kFp8 && !UP ? g * 32 : g * 16);
    }

    auto load_f = [&](int st) {
        Weights<kNF> w;
        const int at = st * 128;
#pragma unroll
        for (int b = 0; b < kNF; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                w.v[b][j] = i32x4{0, 0, 0, 0};
                if (at + j * 64 + g * 16 < f_bytes) w.v[b][j] = *(const i32x4*)(f[b] + at + j * 64);
            }
        return w;
    };

    f32x4 acc[MT][kNF];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < kNF; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const f32x4 zero{0.0f, 0.0f, 0.0f, 0.0f};

    Weights<kNF> next = load_f(wave < steps ? wave : 0);
    for (int st = wave; st < steps; st += kWaves) {
        // the rows' pieces of this step, then the weights of the next: the wait for the first leaves the second in flight
        i32x4 sv[MT][kPieces];
        float s_scale[MT], f_scale[2];
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                sv[a][j] = i32x4{0, 0, 0, 0};
                // where the pieces of 16 bytes stand: j * 64 beside weights of the rows' own format; beside e4m3 weights
                // the lane's 16 k are 32 bytes of bf16
                const int at = F == kFp8 && !UP ? st * 256 + (j >> 1) * 128 + (j & 1) * 16 : st * 128 + j * 64;
                if (s_there[a] && at + (F == kFp8 && !UP ? g * 32 : g * 16) < s_bytes) sv[a][j] = *(const i32x4*)(s[a] + at);
            }
        if constexpr (F == kFp8) {
            const int blocks = p.K / 128;
            if constexpr (UP) {
#pragma unroll
                for (int a = 0; a < MT; ++a) s_scale[a] = s_there[a] ? p.s_scales[(row0 + a * 16 + r) * blocks + st] : 0.0f;
                const float* fs = p.f_scales + ((int64_t)t.expert * 2 * p.N + n0) / 128 * blocks + st;
                f_scale[0] = fs[0];
                f_scale[1] = fs[(int64_t)p.N / 128 * blocks];
            } else {
                f_scale[0] = p.f_scales[((int64_t)t.expert * p.N + n0) / 128 * blocks + st];
            }
        }
        const Weights<kNF> cur = next;
        next = load_f(st + kWaves < steps ? st + kWaves : st);
        if constexpr (F == kBf16) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < kNF; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cur.v[b][j]),
                                                                            __builtin_bit_cast(bf16x8, sv[a][j]), acc[a][b], 0, 0, 0);
        } else if constexpr (UP) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const i32x8 sa = __builtin_shufflevector(sv[a][0], sv[a][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int b = 0; b < kNF; ++b) {
                    const i32x8 fb = __builtin_shufflevector(cur.v[b][0], cur.v[b][1], 0, 1, 2, 3, 4, 5, 6, 7);
                    const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, sa, zero, 0, 0, 0, 0, 0, 0);
                    const float scale = s_scale[a] * f_scale[b / (kNF / 2)];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(part[i], scale, acc[a][b][i]);
                }
            }
        } else {
#pragma unroll
            for (int b = 0; b < kNF; ++b) {
                f32x4 part[MT];
#pragma unroll
                for (int a = 0; a < MT; ++a) part[a] = zero;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const i32x4 q = cur.v[b][j >> 1];
                    const bf16x8 fv = widen_e4m3x8(j & 1 ? i32x2{q[2], q[3]} : i32x2{q[0], q[1]});
#pragma unroll
                    for (int a = 0; a < MT; ++a)
                        part[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, __builtin_bit_cast(bf16x8, sv[a][j]), part[a], 0, 0, 0);
                }
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(part[a][i], f_scale[0], acc[a][b][i]);
            }
        }
    }

    // sums of the waves: [wave][16 rows][64 channels], 16 rows at a time
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kNF; ++b)
            *reinterpret_cast<f32x4*>(sums + (wave * 16 + r) * kSumPitch + b * 16 + g * 4) = acc[a][b];
        __syncthreads();
        constexpr int kOut = UP ? kCols / 2 : kCols;      // 16 rows x kOut channels, 4 per thread
        for (int i = threadIdx.x; i < 16 * kOut / 4; i += kThreads) {
            const int m = i / (kOut / 4), n4 = i % (kOut / 4) * 4;
            if (a * 16 + m >= t.rows || n0 + n4 >= p.N) continue;
            const int64_t row = row0 + a * 16 + m;
            f32x4 v = zero;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(sums + (w * 16 + m) * kSumPitch + n4);
            if constexpr (UP) {
                f32x4 u = zero, h;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) u += *reinterpret_cast<const f32x4*>(sums + (w * 16 + m) * kSumPitch + kOut + n4);
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = v[i] * sigmoid(v[i]) * u[i];
                if (p.pre) {
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.N + n0 + n4) = v;
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.N + p.N + n0 + n4) = u;
                }
                store4(p.out + row * p.op + n0 + n4, h[0], h[1], h[2], h[3]);
            } else {
                store4(p.out + row * p.op + n0 + n4, v[0], v[1], v[2], v[3]);
            }
        }
    }
}

// Rows in steps of 16, up to MAX; half as many registers with one or two leave room for twice the waves, and their loads.
template <Format F, bool UP, int COLS, int MAX>
__global__ __launch_bounds__(kThreads) void k_stream(Params p) {
    __shared__ __align__(16) char smem[kWaves * 16 * (COLS + 4) * 4];
    const RowTiles<MAX * 16> tiles(p.cnt, p.psum, p.El);
    constexpr int kChannels = UP ? COLS / 2 : COLS;
    const int cols = (p.N + kChannels - 1) / kChannels, tile = blockIdx.x / cols;
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    const int n0 = blockIdx.x % cols * kChannels;
    const int steps = (t.rows + 15) / 16;
    if (MAX == 1 || steps == 1) product<F, UP, COLS, 1>(p, t, n0, smem);
    else if (MAX == 2 || steps == 2) product<F, UP, COLS, 2>(p, t, n0, smem);
    else if (steps == 3) product<F, UP, COLS, 3>(p, t, n0, smem);
    else product<F, UP, COLS, 4>(p, t, n0, smem);
}

template <Format F, bool UP, int COLS, int MAX>
hipError_t stream_launch(const Handle& h, int busy, const Params& p, hipStream_t stream) {
    constexpr int kChannels = UP ? COLS / 2 : COLS, kRows = MAX * 16;
    // tiles that any routing can give: every expert with rows may end in a short one
    const int64_t tiles = ((int64_t)h.T * h.K + (int64_t)(kRows - 1) * busy) / kRows;
    hipLaunchKernelGGL((k_stream<F, UP, COLS, MAX>), dim3((unsigned)(tiles * ((p.N + kChannels - 1) / kChannels))), dim3(kThreads), 0, stream, p);
    return hipGetLastError();
}

// 64 weight rows per workgroup, or 32 (bf16) where that leaves the chip short of workgroups or, in the down projection, a
// few rows per expert make more and smaller ones the better stream; then it takes 16 rows.  Measured, 32 experts of 7168 x
// 2048: down projection at 2 rows per expert 171 us with 64 weight rows, 162 with 32, 153 with 16 rows too; at 8 rows 178,
// 167 and 170; at 16 rows 180 and 196; gate and up 297 and 295, 327 and 388.  8 experts of 256 x 512, 32 rows each: 7.0 and
// 6.0 us, down 7.2, 6.4 and 5.0.
// e4m3, down: 32 rows, not 64, at 4 rows per expert 651 and 712 us (256 experts; with 16 rows 668), at 8 94 and 100 (32).
bool narrow(const FfnSizes& s, int N, bool up) {
    const int64_t blocks = (int64_t)busy_experts(s) * ((N + (up ? 31 : 63)) / (up ? 32 : 64));
    return blocks < 512 || (!up && mean_rows(s) <= 8);
}

}  // namespace

hipError_t launch_stream_up(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.x, a.x_scales, a.w13, a.w13_scales, a.h, a.pre, a.inter, a.hidden,
                   a.hidden, row_pitch(a.inter)};
    const FfnSizes s = sizes(h, a);
    const int busy = busy_experts(s);
    if (a.fp8) return stream_launch<kFp8, true, 64, 4>(h, busy, p, stream);
    return narrow(s, a.inter, true) ? stream_launch<kBf16, true, 32, 4>(h, busy, p, stream)
                                    : stream_launch<kBf16, true, 64, 4>(h, busy, p, stream);
}

hipError_t launch_stream_down(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.h, nullptr, a.w2, a.w2_scales, (uint16_t*)a.y, nullptr, a.hidden, a.inter,
                   row_pitch(a.inter), a.hidden};
    const FfnSizes s = sizes(h, a);
    const int busy = busy_experts(s);
    if (a.fp8) return stream_launch<kFp8, false, 64, 2>(h, busy, p, stream);
    return narrow(s, a.hidden, false) ? stream_launch<kBf16, false, 32, 1>(h, busy, p, stream)
                                      : stream_launch<kBf16, false, 64, 4>(h, busy, p, stream);
}

}  // namespace ep
