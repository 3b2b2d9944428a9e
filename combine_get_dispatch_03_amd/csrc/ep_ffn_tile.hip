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

// Where a finished tile goes.
struct Target {
    int64_t row0;
    int rows, n0;
};

template <Product P, int MT>
__device__ __forceinline__ void store_rows(const Params& p, const f32x4 (&acc)[MT][4], const Target& t, int N) {
    const int wave = wave_id(), m_at = (wave >> 2) * MT * 16 + (lane_id() & 15), n_in = (lane_id() >> 4) * 4;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const int m = m_at + a * 16;
        if (m >= t.rows) continue;
        const int64_t row = t.row0 + m;
        if constexpr (P == kGateUp) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int n = t.n0 + (wave & 3) * 32 + b * 16 + n_in;
                if (n >= N) continue;
                const f32x4 gate = acc[a][b], up = acc[a][b + 2];
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
                const int n = t.n0 + (wave & 3) * 64 + b * 16 + n_in;
                if (n >= N) continue;
                const f32x4 v = acc[a][b];
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
struct RowsKernel {
    typedef Bf16Tile<false, P == kDownGrad || P == kInGrad> Tile;
    static constexpr int kCols = P == kGateUp ? kBN / 2 : kBN;     // channels of N per tile

    const Params& p;
    char* smem;
    RowTiles<Tile::kBM> tiles;
    int N, K;
    Tile g;
    int round = 0;

    __device__ __forceinline__ RowsKernel(const Params& params, char* lds)
        : p(params), smem(lds), tiles(params.cnt, params.psum, params.El) {
        N = P == kGateUp || P == kDownGrad ? p.I : p.H;
        K = P == kGateUp || P == kDownGrad ? p.H : P == kDown ? p.I : 2 * p.I;
    }

    // The workgroup's next tile: its first copies are issued.
    __device__ __forceinline__ bool begin(Target* next) {
        TileAt at;
        if (!tile_at((int)blockIdx.x, round++, tiles.total, (N + kCols - 1) / kCols, &at)) return false;
        const RowTile t = tiles.find(at.row, 32);
        const int n0 = at.col * kCols;
        *next = Target{t.row0, t.rows, n0};
        g.s.init(p.s + (int64_t)t.row0 * K, [&](int r) { return r < t.rows ? r * (2u * K) : kNoElement; });
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
        g.begin(smem, K);
        return true;
    }

    template <int MT>
    __device__ __forceinline__ bool tile(Target* t) {
        f32x4 acc[MT][4];
        g.template run<MT>(smem, K, acc);
        const Target done = *t;
        const bool more = begin(t);
        store_rows<P, MT>(p, acc, done, N);
        return more;
    }
};

// A workgroup stays on its CU and walks through its tiles: a tile's first copies are under way while the tile before is
// stored.  Waves take as many 16-row steps as the tile is high.
template <Product P>
__global__ __launch_bounds__(kGemmThreads, 2) void k_rows(Params p) {
    extern __shared__ __align__(1024) char smem[];
    RowsKernel<P> k(p, smem);
    Target t;
    bool more = k.begin(&t);
    while (more) {
        switch ((t.rows + 31) / 32) {
            case 1: more = k.template tile<1>(&t); break;
            case 2: more = k.template tile<2>(&t); break;
            case 3: more = k.template tile<3>(&t); break;
            case 4: more = k.template tile<4>(&t); break;
            case 5: more = k.template tile<5>(&t); break;
            case 6: more = k.template tile<6>(&t); break;
            case 7: more = k.template tile<7>(&t); break;
            default: more = k.template tile<8>(&t); break;
        }
    }
}

// out[e] [M, N] = sum over the expert's rows of s[row, m] f[row, n]
__global__ __launch_bounds__(kGemmThreads, 2) void k_weights(const int32_t* cnt, const int32_t* psum, int El, const uint16_t* s,
                                                             const uint16_t* f, uint16_t* out, int M, int N) {
    typedef Bf16Tile<true, true> Tile;
    extern __shared__ __align__(1024) char smem[];
    const int mt = (M + Tile::kBM - 1) / Tile::kBM, nt = (N + kBN - 1) / kBN;
    Tile g;
    f32x4 acc[8][4];
    int64_t last_out = 0;
    int last_m = 0, last_n = 0;
    for (int round = 0;; ++round) {
        TileAt at;
        const bool more = tile_at((int)blockIdx.x, round, El * mt, nt, &at);
        int rows = 0, m0 = 0, n0 = 0;
        int64_t to = 0;
        if (more) {
            const int e = at.row / mt;
            m0 = at.row % mt * Tile::kBM, n0 = at.col * kBN;
            rows = __builtin_amdgcn_readfirstlane(cnt[e]);
            const int64_t row0 = __builtin_amdgcn_readfirstlane(psum[e]);
            to = (int64_t)e * M * N;
            g.s.init(s + row0 * M + m0, (int64_t)M * 2, M - m0);
            g.f.init(f + row0 * N + n0, (int64_t)N * 2, N - n0);
            g.begin(smem, rows);
        }
        if (round > 0) {
            const int wave = wave_id(), m_at = last_m + (wave >> 2) * 128 + (lane_id() & 15);
            const int n_at = last_n + (wave & 3) * 64 + (lane_id() >> 4) * 4;
#pragma unroll
            for (int a = 0; a < 8; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int m = m_at + a * 16, n = n_at + b * 16;
                    const f32x4 v = acc[a][b];
                    if (m < M && n < N) store4(out + last_out + (int64_t)m * N + n, v[0], v[1], v[2], v[3]);
                }
        }
        if (!more) break;
        g.run<8>(smem, rows, acc);
        last_out = to, last_m = m0, last_n = n0;
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
    hipLaunchKernelGGL((k_rows<P>), dim3(walking_blocks(rows * ((N + cols - 1) / cols))), dim3(kGemmThreads), Tile::kLds, stream, p);
    return hipGetLastError();
}

hipError_t weights_launch(const Handle& h, const uint16_t* s, const uint16_t* f, uint16_t* out, int M, int N, hipStream_t stream) {
    typedef Bf16Tile<true, true> Tile;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_weights), Tile::kLds);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t)h.El * ((M + Tile::kBM - 1) / Tile::kBM) * ((N + kBN - 1) / kBN);
    hipLaunchKernelGGL(k_weights, dim3(walking_blocks(tiles)), dim3(kGemmThreads), Tile::kLds, stream, h.ws.cnt_local, h.ws.psum,
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
