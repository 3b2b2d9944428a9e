// ep_ffn_tile.hip -- the products of the expert block on large tiles (see ep_gemm_core.hpp).
#include "ep_expert_tiles.hpp"
#include "ep_ffn.hpp"
#include "ep_gemm_core.hpp"

namespace ep {
namespace {

enum Product { kGateUp, kDown, kDownGrad, kInGrad };

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
    const uint16_t* s;    // rows of the segments
    const uint16_t* f;    // the weights
    uint16_t* out;        // kGateUp: h   kDown: y   kDownGrad: dp   kInGrad: dx
    uint16_t* out2;       // kDownGrad: h
    float* pre;           // kGateUp: written when given   kDownGrad: read
    int H, I;
};

template <Product P, int MT, class Tile>
__device__ __forceinline__ void rows_tile(const Params& p, Tile& g, char* smem, int K, int rows, int64_t row0, int n0, int N) {
    g.template run<MT>(smem, K);
    const int wave = wave_id(), m_at = (wave >> 2) * MT * 16 + (lane_id() & 15), n_in = (lane_id() >> 4) * 4;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const int m = m_at + a * 16;
        if (m >= rows) continue;
        const int64_t row = row0 + m;
        if constexpr (P == kGateUp) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int n = n0 + (wave & 3) * 32 + b * 16 + n_in;
                if (n >= N) continue;
                const f32x4 gate = g.acc[a][b], up = g.acc[a][b + 2];
                if (p.pre) {
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.I + n) = gate;
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.I + p.I + n) = up;
                }
                f32x4 h;
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = gate[i] * sigmoid(gate[i]) * up[i];
                store4(p.out + row * p.I + n, h[0], h[1], h[2], h[3]);
            }
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int n = n0 + (wave & 3) * 64 + b * 16 + n_in;
                if (n >= N) continue;
                const f32x4 v = g.acc[a][b];
                if constexpr (P == kDownGrad) {
                    const f32x4 gate = *reinterpret_cast<const f32x4*>(p.pre + row * 2 * p.I + n);
                    const f32x4 up = *reinterpret_cast<const f32x4*>(p.pre + row * 2 * p.I + p.I + n);
                    f32x4 dg, du, h;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float sg = sigmoid(gate[i]), act = gate[i] * sg;
                        dg[i] = v[i] * up[i] * sg * (1.0f + gate[i] * (1.0f - sg));
                        du[i] = v[i] * act;
                        h[i] = act * up[i];
                    }
                    store4(p.out + row * 2 * p.I + n, dg[0], dg[1], dg[2], dg[3]);
                    store4(p.out + row * 2 * p.I + p.I + n, du[0], du[1], du[2], du[3]);
                    store4(p.out2 + row * p.I + n, h[0], h[1], h[2], h[3]);
                } else {
                    store4(p.out + row * N + n, v[0], v[1], v[2], v[3]);
                }
            }
        }
    }
}

template <Product P>
__global__ __launch_bounds__(kGemmThreads, 2) void k_rows(Params p) {
    constexpr bool kFks = P == kDownGrad || P == kInGrad;
    typedef Bf16Tile<false, kFks> Tile;
    extern __shared__ __align__(1024) char smem[];
    const RowTiles<Tile::kBM> tiles(p.cnt, p.El);
    constexpr int kCols = P == kGateUp ? kBN / 2 : kBN;     // channels of N per tile
    const int N = P == kGateUp || P == kDownGrad ? p.I : p.H;
    const int K = P == kGateUp || P == kDownGrad ? p.H : P == kDown ? p.I : 2 * p.I;
    TileAt at;
    if (!tile_at((int)blockIdx.x, tiles.total, (N + kCols - 1) / kCols, &at)) return;
    const RowTile t = tiles.find(at.row, 32);
    const int64_t row0 = (int64_t)__builtin_amdgcn_readfirstlane(p.psum[t.expert]) + t.m0;
    const int n0 = at.col * kCols;

    Tile g;
    const uint32_t lds_s = 2u * K;
    g.s.init(p.s + row0 * K, [&](int r) { return r < t.rows ? r * lds_s : kNoElement; });
    if constexpr (P == kGateUp) {
        // a wave's 64 rows of F: 32 gate channels, then the same 32 up channels
        const uint64_t up = (uint64_t)p.I * p.H * 2;
        g.f.init(p.f + ((int64_t)t.expert * 2 * p.I + n0) * p.H, [&](int r) {
            const int c = r / 64 * 32 + r % 32;
            return n0 + c < N ? (uint32_t)((r % 64 >= 32 ? up : 0) + (uint64_t)c * p.H * 2) : kNoElement;
        });
    } else if constexpr (P == kDown) {
        g.f.init(p.f + ((int64_t)t.expert * p.H + n0) * p.I, [&](int r) { return n0 + r < N ? (uint32_t)r * p.I * 2 : kNoElement; });
    } else if constexpr (P == kDownGrad) {
        g.f.init(p.f + (int64_t)t.expert * p.H * p.I + n0, (int64_t)p.I * 2, N - n0);
    } else {
        g.f.init(p.f + (int64_t)t.expert * 2 * p.I * p.H + n0, (int64_t)p.H * 2, N - n0);
    }
    // as many 16-row steps per wave as the tile is high
    switch ((t.rows + 31) / 32) {
        case 1: rows_tile<P, 1>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 2: rows_tile<P, 2>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 3: rows_tile<P, 3>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 4: rows_tile<P, 4>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 5: rows_tile<P, 5>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 6: rows_tile<P, 6>(p, g, smem, K, t.rows, row0, n0, N); break;
        case 7: rows_tile<P, 7>(p, g, smem, K, t.rows, row0, n0, N); break;
        default: rows_tile<P, 8>(p, g, smem, K, t.rows, row0, n0, N); break;
    }
}

// out[e] [M, N] = sum over the expert's rows of s[row, m] f[row, n]
__global__ __launch_bounds__(kGemmThreads, 2) void k_weights(const int32_t* cnt, const int32_t* psum, int El, const uint16_t* s,
                                                    const uint16_t* f, uint16_t* out, int M, int N) {
    typedef Bf16Tile<true, true> Tile;
    extern __shared__ __align__(1024) char smem[];
    const int mt = (M + Tile::kBM - 1) / Tile::kBM, nt = (N + kBN - 1) / kBN;
    TileAt at;
    if (!tile_at((int)blockIdx.x, El * mt, nt, &at)) return;
    const int e = at.row / mt, m0 = at.row % mt * Tile::kBM, n0 = at.col * kBN;
    const int rows = __builtin_amdgcn_readfirstlane(cnt[e]);
    const int64_t row0 = __builtin_amdgcn_readfirstlane(psum[e]);
    Tile g;
    g.s.init(s + row0 * M + m0, (int64_t)M * 2, M - m0);
    g.f.init(f + row0 * N + n0, (int64_t)N * 2, N - n0);
    g.run<8>(smem, rows);
    const int wave = wave_id(), m_at = m0 + (wave >> 2) * 128 + (lane_id() & 15);
    const int n_at = n0 + (wave & 3) * 64 + (lane_id() >> 4) * 4;
#pragma unroll
    for (int a = 0; a < 8; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int m = m_at + a * 16, n = n_at + b * 16;
            const f32x4 v = g.acc[a][b];
            if (m < M && n < N) store4(out + ((int64_t)e * M + m) * N + n, v[0], v[1], v[2], v[3]);
        }
}

template <Product P>
hipError_t rows_launch(const Handle& h, const Params& p, hipStream_t stream) {
    typedef Bf16Tile<false, P == kDownGrad || P == kInGrad> Tile;
    const int N = P == kGateUp || P == kDownGrad ? p.I : p.H, cols = P == kGateUp ? kBN / 2 : kBN;
    // row tiles that any routing can give: every expert may end in a short one
    const int64_t rows = (int64_t)h.T * h.K / Tile::kBM + h.El;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_rows<P>), Tile::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_rows<P>), dim3(tile_blocks(rows * ((N + cols - 1) / cols))), dim3(kGemmThreads), Tile::kLds, stream, p);
    return hipGetLastError();
}

hipError_t weights_launch(const Handle& h, const uint16_t* s, const uint16_t* f, uint16_t* out, int M, int N, hipStream_t stream) {
    typedef Bf16Tile<true, true> Tile;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_weights), Tile::kLds);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t)h.El * ((M + Tile::kBM - 1) / Tile::kBM) * ((N + kBN - 1) / kBN);
    hipLaunchKernelGGL(k_weights, dim3(tile_blocks(tiles)), dim3(kGemmThreads), Tile::kLds, stream, h.ws.cnt_local, h.ws.psum,
                       h.El, s, f, out, M, N);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_tile(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const Params up{h.ws.cnt_local, h.ws.psum, h.El, (const uint16_t*)a.x, (const uint16_t*)a.w13, a.h, nullptr, a.pre, a.hidden, a.inter};
    const hipError_t e = rows_launch<kGateUp>(h, up, stream);
    if (e != hipSuccess) return e;
    const Params down{h.ws.cnt_local, h.ws.psum, h.El, a.h, (const uint16_t*)a.w2, (uint16_t*)a.y, nullptr, nullptr, a.hidden, a.inter};
    return rows_launch<kDown>(h, down, stream);
}

hipError_t launch_expert_ffn_backward(const Handle& h, const FfnBackwardArgs& a, hipStream_t stream) {
    const uint16_t* dy = (const uint16_t*)a.dy;
    hipError_t e = hipSuccess;
    if (h.T > 0) {
        const Params dg{h.ws.cnt_local, h.ws.psum, h.El, dy, (const uint16_t*)a.w2, a.dp, a.h, const_cast<float*>(a.pre), a.hidden, a.inter};
        e = rows_launch<kDownGrad>(h, dg, stream);
        if (e == hipSuccess && a.dx) {
            const Params ig{h.ws.cnt_local, h.ws.psum, h.El, a.dp, (const uint16_t*)a.w13, (uint16_t*)a.dx, nullptr, nullptr, a.hidden, a.inter};
            e = rows_launch<kInGrad>(h, ig, stream);
        }
    }
    if (e == hipSuccess && a.dw2) e = weights_launch(h, dy, a.h, (uint16_t*)a.dw2, a.hidden, a.inter, stream);
    if (e == hipSuccess && a.dw13)
        e = weights_launch(h, a.dp, (const uint16_t*)a.x, (uint16_t*)a.dw13, 2 * a.inter, a.hidden, stream);
    return e;
}

}  // namespace ep
