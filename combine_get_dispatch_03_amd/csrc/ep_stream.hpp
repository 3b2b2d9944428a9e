// ep_stream.hpp -- products of few rows with many weights: the weights stream from memory into the matrix instruction's
// registers, past nothing (see ep_weights.hpp for what a piece of them is); the rows' fragments come from the caches.
#pragma once

#include "ep_ffn.hpp"
#include "ep_h_rows.hpp"
#include "ep_weights.hpp"

namespace ep {

// 16 * MT rows' fragments beside a piece: lane (r, g) holds row r of each 16.  A row that does not exist is kNoElement.
// H: of h (ep_h_rows.hpp), otherwise of bf16.
template <class W, int MT, bool H>
struct RowFragments {
    typedef i32x4 Held[MT][4];
    Buffer rows;
    uint32_t at[MT];
    int K, top[H ? MT : 1];                         // largest number of a row
    bool mixed;                                     // some row has others

    __device__ __forceinline__ void init(const void* base, int k) {
        rows.init(base);
        K = k;
    }
    __device__ __forceinline__ void place(int a, bool there, uint32_t offset) {
        at[a] = there ? offset + W::k_of(0, lane_id() >> 4) * 2 : kNoElement;
    }
    // The numbers of a piece's eight blocks, of a row that exists.
    __device__ __forceinline__ i32x4 numbers(int a, int piece) const {
        return load16(rows.resource(true), at[a] - W::k_of(0, lane_id() >> 4) * 2 + (uint32_t)piece * 16, (uint32_t)K * 2);
    }
    __device__ __forceinline__ void load(Held& x, int piece, bool there) const {
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
    // The rows' numbers, by the four lanes of a row together, kAsked pieces' a lane at a time.  The first are asked for before the rows,
    // and looked at once those are under way: after them they would be waited for apart (1.8 us of a small call's 14).
    static constexpr int kAsked = MT == 1 ? 4 : 2;
    typedef i32x4 Numbers[MT][kAsked];
    __device__ __forceinline__ void ask(Numbers& e, int piece) const {
        if constexpr (H)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int i = 0; i < kAsked; ++i) {
                    const int p = piece + i * 4 + (lane_id() >> 4);
                    const uint32_t from = at[a] - W::k_of(0, lane_id() >> 4) * 2 + (uint32_t)(K * 2 + p * 16);
                    e[a][i] = load16(rows.resource(true), at[a] != kNoElement && p < pieces_of(K) ? from : kNoElement, 0);
                }
    }
    __device__ __forceinline__ void find_tops(Numbers& e) {
        mixed = false;
        if constexpr (H) {
            NumberRange range[MT];
            const int blocks = (K + kShared - 1) / kShared;
            for (int piece = 0;;) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int i = 0; i < kAsked; ++i)
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            range[a].add((uint32_t)e[a][i][d], blocks - ((piece + i * 4 + (lane_id() >> 4)) * 8 + d * 2));
                piece += kAsked * 4;
                if (piece >= pieces_of(K)) break;
                ask(e, piece);
            }
            bool differ = false;
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                int t = range[a].top();
                t = max(t, __shfl_xor(t, 16));
                top[a] = max(t, __shfl_xor(t, 32));
                differ |= range[a].low() < top[a];
            }
            mixed = ballot(differ) != 0;
        }
    }
    // A piece of rows with more than one, brought to the largest.
    __device__ __forceinline__ void settle(Held& x, int piece) const {
        if constexpr (H) {
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                if (at[a] == kNoElement) continue;
                const i32x4 e = numbers(a, piece);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[a][j] = bring_to(x[a][j], (int)W::of_block(e, j, lane_id() >> 4), top[a]);
            }
        }
    }
    // What sums of row a * 16 + 4 * (lane / 16) + i are to be multiplied by.
    __device__ __forceinline__ float unit(int a, int i) const {
        if constexpr (H) return shared_unit(__shfl(top[a], (lane_id() >> 4) * 4 + i));
        else return 1.0f;
    }
};

// acc[NF][MT] += pieces first, first + step, ... below `end` of NF rows of pieces, by the rows.  A wave's next piece is under way
// while others multiply; more per wave only lengthens the queue.  Measured, 8 tokens of 64 bf16 experts of 7168 x 2048, asked for
// when needed 801 us, one piece ahead 668; one token's down projection (int4) one ahead 15.1 us, two 15.7, eight 17.5; 32
// tokens, e4m3, down one ahead 440, two 453, four 595 (16 channels a workgroup).
template <class W, bool H, int MT, int NF>
__device__ __forceinline__ void stream_pieces(const typename W::template Rows<NF>& w, RowFragments<W, MT, H>& rows, int first, int step,
                                              int end, f32x4 (&acc)[NF][MT]) {
    typedef RowFragments<W, MT, H> R;
    typename W::Raw raw[NF];
    typename R::Held x;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[a][j] = i32x4{0, 0, 0, 0};
    auto load = [&](int piece) {
        rows.load(x, piece, piece < end);
#pragma unroll
        for (int b = 0; b < NF; ++b) raw[b] = w.load(b, piece, piece < end);
    };
    typename R::Numbers numbers;
    rows.ask(numbers, 0);
    load(first);
    rows.find_tops(numbers);
    for (int piece = first; piece < end; piece += step) {
        if (rows.mixed) rows.settle(x, piece);
        add_pieces<W, H>(raw, x, acc);
        load(piece + step);
    }
}

// One workgroup's product: `count` rows (up to 16 * MT) by NF rows of pieces of an expert's weights, k split over the waves, whose
// sums meet in LDS.  UP: half of the pieces are gate channels from n0 on, half the same up channels, N of each, and h = silu(g) u is
// stored; otherwise output channels from n0 on, and the rows are h's.  out_row(m): where row m goes.
constexpr int kStreamThreads = 256, kStreamWaves = kStreamThreads / kWave;
template <int NF>
constexpr int stream_lds() { return kStreamWaves * 16 * (NF * 16 + 4) * 4; }

template <class W, bool UP, int MT, int NF, class OutRow>
__device__ __forceinline__ void stream_product(const WeightArgs& weights, int expert, int N, int K, int n0,
                                               RowFragments<W, MT, !UP>& rows, int count, float* sums, OutRow out_row) {
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
    stream_pieces(w, rows, wave, kStreamWaves, pieces_of(K), acc);

    // [wave][16 rows][channels], 16 rows at a time
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        if (a * 16 >= count) break;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float unit = rows.unit(a, j);
#pragma unroll
            for (int b = 0; b < NF; ++b) sums[(wave * 16 + g * 4 + j) * kPitch + b * 16 + r] = acc[b][a][j] * unit;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * kOut / 4; i += kStreamThreads) {
            const int m = i / (kOut / 4), n4 = i % (kOut / 4) * 4;
            if (a * 16 + m >= count || (!UP && n0 + n4 >= N)) continue;
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
            uint16_t* out = out_row(a * 16 + m);
            if constexpr (UP) store4_h(out, N, n0 + n4, v);      // (a block's 16 channels are four neighbouring lanes')
            else store4(out + n0 + n4, v[0], v[1], v[2], v[3]);
        }
    }
}

}  // namespace ep
