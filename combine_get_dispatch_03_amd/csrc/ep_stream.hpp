// ep_stream.hpp -- products of few rows with many weights: the weights stream from memory into the matrix instruction's
// registers, past nothing (see ep_weights.hpp for what a piece of them is); the rows' fragments come from the caches.
#pragma once

#include "ep_ffn.hpp"
#include "ep_weights.hpp"

namespace ep {

// 16 * MT rows' fragments beside a piece: lane (r, g) holds row r of each 16.  A row that does not exist is kNoElement.
template <class W, int MT>
struct RowFragments {
    Buffer rows;
    uint32_t at[MT];
    int K;

    __device__ __forceinline__ void init(const void* base, int k) {
        rows.init(base);
        K = k;
    }
    __device__ __forceinline__ void place(int a, bool there, uint32_t offset) {
        at[a] = there ? offset + W::k_of(0, lane_id() >> 4) * 2 : kNoElement;
    }
    __device__ __forceinline__ void load(i32x4 (&x)[MT][4], int piece, bool there) const {
        const __amdgpu_buffer_rsrc_t buffer = rows.resource(there);
        // lanes of rows that do not exist stay out (and keep what they hold: nobody uses their sums); as zeros they would cost
        // the address and data paths as much as rows
#pragma unroll
        for (int a = 0; a < MT; ++a)
            if (at[a] != kNoElement)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = !W::kTail || piece * kPieceK + W::k_of(j, lane_id() >> 4) < K;
                    x[a][j] = load16(buffer, in ? at[a] + W::k_of(j, 0) * 2 : kNoElement, (uint32_t)piece * kPieceK * 2);
                }
    }
};

// acc[NF][MT] += pieces first, first + step, ... below `end` of NF rows of pieces, by the rows.  A wave's next piece is under way
// while others multiply; more per wave only lengthens the queue.  Measured, 8 tokens of 64 bf16 experts of 7168 x 2048, asked for
// when needed 801 us, one piece ahead 668; one token's down projection (int4) one ahead 15.1 us, two 15.7, eight 17.5; 32
// tokens, e4m3, down one ahead 440, two 453, four 595 (16 channels a workgroup).
template <class W, int MT, int NF>
__device__ __forceinline__ void stream_pieces(const typename W::template Rows<NF>& w, const RowFragments<W, MT>& rows, int first, int step,
                                              int end, f32x4 (&acc)[NF][MT]) {
    typename W::Raw raw[NF];
    i32x4 x[MT][4];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[a][j] = i32x4{0, 0, 0, 0};
    auto load = [&](int piece) {
        rows.load(x, piece, piece < end);
#pragma unroll
        for (int b = 0; b < NF; ++b) raw[b] = w.load(b, piece, piece < end);
    };
    load(first);
    for (int piece = first; piece < end; piece += step) {
#pragma unroll
        for (int b = 0; b < NF; ++b) add_piece<W, MT>(raw[b], x, acc[b]);
        load(piece + step);
    }
}

// One workgroup's product: `count` rows (up to 16 * MT) by NF rows of pieces of an expert's weights, k split over the waves, whose
// sums meet in LDS.  UP: half of the pieces are gate channels from n0 on, half the same up channels, N of each, and h = silu(g) u is
// stored; otherwise output channels from n0 on.  out_row(m): where row m goes.
//   h is rounded to bf16, one of two roundings on the way to y (the other is y's own): it is an operand of the second product, whose
// instruction takes 16 bits.  That puts the result 0.0023 to 0.0025 from the one in 64 bits (relative, Euclidean) instead of the 0.0016 to
// 0.0017 that y's rounding leaves; a second bf16 part of h would take twice the instructions of the second product and twice the workspace.
constexpr int kStreamThreads = 256, kStreamWaves = kStreamThreads / kWave;
template <int NF>
constexpr int stream_lds() { return kStreamWaves * 16 * (NF * 16 + 4) * 4; }

template <class W, bool UP, int MT, int NF, class OutRow>
__device__ __forceinline__ void stream_product(const WeightArgs& weights, int expert, int N, int K, int n0, const RowFragments<W, MT>& rows,
                                               int count, float* sums, OutRow out_row) {
    constexpr int kCols = NF * 16, kOut = UP ? kCols / 2 : kCols, kPitch = kCols + 4;
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    typename W::template Rows<NF> w;
    w.init(weights, expert, n0);
#pragma unroll
    for (int b = 0; b < NF; ++b) {
        const int n = (UP ? b % (NF / 2) : b) * 16, exist = N - n0 - n;
        w.place(b, (exist > 0 ? n : 0) + (UP ? b / (NF / 2) * N : 0), exist);
    }
    f32x4 acc[NF][MT];
#pragma unroll
    for (int b = 0; b < NF; ++b)
#pragma unroll
        for (int a = 0; a < MT; ++a) acc[b][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    stream_pieces<W, MT, NF>(w, rows, wave, kStreamWaves, pieces_of(K), acc);

    // [wave][16 rows][channels], 16 rows at a time
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        if (a * 16 >= count) break;
        __syncthreads();
#pragma unroll
        for (int b = 0; b < NF; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[(wave * 16 + g * 4 + j) * kPitch + b * 16 + r] = acc[b][a][j];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * kOut / 4; i += kStreamThreads) {
            const int m = i / (kOut / 4), n4 = i % (kOut / 4) * 4;
            if (a * 16 + m >= count || n0 + n4 >= N) continue;
            f32x4 v{0.0f, 0.0f, 0.0f, 0.0f}, u = v;
#pragma unroll
            for (int q = 0; q < kStreamWaves; ++q) {
                v += *reinterpret_cast<const f32x4*>(sums + (q * 16 + m) * kPitch + n4);
                if constexpr (UP) u += *reinterpret_cast<const f32x4*>(sums + (q * 16 + m) * kPitch + kOut + n4);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] *= W::kUnit;
                if constexpr (UP) v[j] = v[j] * sigmoid(v[j]) * (u[j] * W::kUnit);
            }
            store4(out_row(a * 16 + m) + n0 + n4, v[0], v[1], v[2], v[3]);
        }
    }
}

}  // namespace ep
