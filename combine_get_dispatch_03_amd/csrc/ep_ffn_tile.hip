// ep_ffn_tile.hip -- the products of the expert block in bf16 on large tiles (see ep_gemm_core.hpp).
//
//   k_rows     a segment's rows by an expert's weights, 256 x 256 tiles, with the activation in the epilogue:
//                gate and up   pre = x W13^T (a tile holds 128 gate channels and the same 128 up channels), h = silu(g) u
//                down          y = h W2^T
//                down's grad   dh = dy W2 and, from pre, dp = (dg, du) and h once more: no pass over them of its own
//                input's grad  dx = dp W13
//   k_weights  out_e = s^T f over the expert's rows (dW2 = dy^T h, dW13 = dp^T x), sums in fp32, each written once
//
// With hundreds of rows per expert they are bound by the matrix units at the clock the power limit leaves (1.73 to 1.89
// GHz here): they are busy 60 to 71% of the cycles, 56% at 1.96 GHz in k_weights, whose sums are short and stores many (without
// the stores 1.59 instead of 1.83 ms).  No bank conflicts in LDS.  With few rows, by the weights' bytes.
// Measured, 32 experts of 7168 x 2048, 32768 rows, medians (TFLOP/s): gate and up 1.54 ms (1248), down 0.83 (1153), down's grad
// 0.99 (971), input's grad 1.52 (1270), dW13 1.77 (1086), dW2 0.97 (996).  20 experts of 2112 x 1352, 2211
// rows, 33 to 540 each: 54, 46, 67, 87, 90 and 51 us.
//
// h and dp are rounded to bf16 (2^-8 of an element at most, 2^-9 on average): it is the type the next product's matrix instruction takes, and in
// two parts each would double that product.
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

// Where a tile's sums go.
struct Target {
    int64_t row0;
    int rows, n0;
};

// A lane holds 8 consecutive channels of a row in acc[a][0], acc[a][1] and, 32 channels on (kGateUp: the up projection's), 8 in
// acc[a][2], acc[a][3].
template <Product P, int MT>
__device__ __forceinline__ void store_rows(const Params& p, const f32x4 (&acc)[MT][4], const Target& t, int N) {
    const int wave = wave_id(), m_at = (wave >> 2) * MT * 16 + (lane_id() & 15), n_in = (lane_id() >> 4) * 8;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const int m = m_at + a * 16;
        if (m >= t.rows) continue;
        const int64_t row = t.row0 + m;
        if constexpr (P == kGateUp) {
            const int n = t.n0 + (wave & 3) * 32 + n_in;
            if (n >= N) continue;
            f32x4 h[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const f32x4 gate = acc[a][b], up = acc[a][b + 2];
                if (p.pre) {
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.I + n + b * 4) = gate;
                    *reinterpret_cast<f32x4*>(p.pre + row * 2 * p.I + p.I + n + b * 4) = up;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) h[b][i] = gate[i] * sigmoid(gate[i]) * up[i];
            }
            store8(p.out + row * row_pitch(p.I) + n, h[0], h[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = t.n0 + (wave & 3) * 64 + j * 32 + n_in;
                if (n >= N) continue;
                if constexpr (P == kDownGrad) {
                    f32x4 dg[2], du[2], h[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const f32x4 v = acc[a][j * 2 + b];
                        const f32x4 gate = *reinterpret_cast<const f32x4*>(p.pre + row * 2 * p.I + n + b * 4);
                        const f32x4 up = *reinterpret_cast<const f32x4*>(p.pre + row * 2 * p.I + p.I + n + b * 4);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float sg = sigmoid(gate[i]), act = gate[i] * sg;
                            dg[b][i] = v[i] * up[i] * sg * (1.0f + gate[i] * (1.0f - sg));
                            du[b][i] = v[i] * act;
                            h[b][i] = act * up[i];
                        }
                    }
                    store8(p.out + row * row_pitch(2 * p.I) + n, dg[0], dg[1]);
                    store8(p.out + row * row_pitch(2 * p.I) + p.I + n, du[0], du[1]);
                    store8(p.out2 + row * row_pitch(p.I) + n, h[0], h[1]);
                } else {
                    store8(p.out + row * N + n, acc[a][j * 2], acc[a][j * 2 + 1]);
                }
            }
        }
    }
}

template <Product P, bool ONCE>
struct RowsKernel {
    typedef Bf16Tiles<false, P == kDownGrad || P == kInGrad, ONCE> Tiles;
    static constexpr int kCols = P == kGateUp ? kBN / 2 : kBN;     // channels of N per tile

    const Params& p;
    RowTiles<Tiles::kBM, 0> rows;      // the registers are needed: find() reads the counts again
    int N, K;
    Tiles g;
    int round = 0;
    Target now, next;

    __device__ __forceinline__ explicit RowsKernel(const Params& params)
        : p(params), rows(params.cnt, params.psum, params.El) {
        N = P == kGateUp || P == kDownGrad ? p.I : p.H;
        K = P == kGateUp || P == kDownGrad ? p.H : P == kDown ? p.I : 2 * p.I;
    }

    // The workgroup's next tile: where it goes and its operands.  next.rows = 0: there is none.
    __device__ __forceinline__ void look_ahead() {
        TileAt at;
        next.rows = g.next_k = 0;
        if (!tile_at((int)blockIdx.x, round++, rows.total, (N + kCols - 1) / kCols, &at)) return;
        const RowTile t = rows.find(at.row, 32);
        const int n0 = at.col * kCols;
        next = Target{t.row0, t.rows, n0};
        g.next_k = K;
        const uint32_t pitch = P == kDown || P == kInGrad ? row_pitch(K) : K;
        g.next_s.init(p.s + (int64_t)t.row0 * pitch, [&](int r) { return r < t.rows ? r * (2u * pitch) : kNoElement; });
        if constexpr (P == kGateUp) {
            // a wave's 64 rows of F: 32 gate channels (fragments 0, 1), then the same 32 up channels
            const uint64_t up = (uint64_t)p.I * p.H * 2;
            g.next_f.init(p.f + ((int64_t)t.expert * 2 * p.I + n0) * p.H, [&](int r) {
                const int c = r / 64 * 32 + channel_of(r / 16 & 1, r & 15);
                return n0 + c < N ? (uint32_t)((r & 32 ? up : 0) + (uint64_t)c * p.H * 2) : kNoElement;
            });
        } else if constexpr (P == kDown) {
            g.next_f.init(p.f + ((int64_t)t.expert * p.H + n0) * p.I, [&](int r) {
                const int c = r / 64 * 64 + channel_of(r / 16 & 3, r & 15);
                return n0 + c < N ? (uint32_t)c * p.I * 2 : kNoElement;
            });
        } else if constexpr (P == kDownGrad) {
            g.next_f.init(p.f + (int64_t)t.expert * p.H * p.I + n0, (int64_t)p.I * 2, N - n0);
        } else {
            g.next_f.init(p.f + (int64_t)t.expert * 2 * p.I * p.H + n0, (int64_t)p.H * 2, N - n0);
        }
    }

    template <int MT>
    __device__ __forceinline__ void tile() {
        f32x4 acc[MT][4];
        g.template run<MT>(acc);
        store_rows<P, MT>(p, acc, now, N);
    }
};

// A workgroup stays on its CU and walks through its tiles.  Waves take as many 16-row steps as the tile is high.
template <Product P, bool ONCE>
__global__ __launch_bounds__(kGemmThreads, 2) void k_rows(Params p) {
    extern __shared__ __align__(1024) char smem[];
    RowsKernel<P, ONCE> k(p);
    k.look_ahead();
    if (k.next.rows == 0) return;
    k.g.s = k.g.next_s, k.g.f = k.g.next_f;
    k.g.begin(smem, k.K);
    do {
        k.now = k.next;
        k.look_ahead();
        switch ((k.now.rows + 31) / 32) {
            case 1: k.template tile<1>(); break;
            case 2: k.template tile<2>(); break;
            case 3: k.template tile<3>(); break;
            case 4: k.template tile<4>(); break;
            case 5: k.template tile<5>(); break;
            case 6: k.template tile<6>(); break;
            case 7: k.template tile<7>(); break;
            default: k.template tile<8>(); break;
        }
    } while (k.next.rows > 0);
    k.g.end();
}

// out[e] [M, N] = sum over the expert's rows of s[row, m] f[row, n]; rows of s and f are sp and fp elements apart.
__global__ __launch_bounds__(kGemmThreads, 2) void k_weights(const int32_t* cnt, const int32_t* psum, int El, const uint16_t* s,
                                                             const uint16_t* f, uint16_t* out, int M, int N, int sp, int fp) {
    typedef Bf16Tiles<true, true> Tiles;
    extern __shared__ __align__(1024) char smem[];
    const ExpertRows experts(cnt, psum, El);
    const int mt = (M + Tiles::kBM - 1) / Tiles::kBM, nt = (N + kBN - 1) / kBN;
    Tiles g;
    struct Out {
        int64_t at;
        int m0, n0, k;
    } next, now;
    int round = 0;
    bool more;
    auto look_ahead = [&]() {
        TileAt at;
        g.next_k = 0;
        more = tile_at((int)blockIdx.x, round++, El * mt, nt, &at);
        if (!more) return;
        const RowTile e = experts.get(at.row / mt);
        next = Out{(int64_t)e.expert * M * N, at.row % mt * Tiles::kBM, at.col * kBN, e.rows};
        g.next_k = e.rows;
        g.next_s.init(s + (int64_t)e.row0 * sp + next.m0, (int64_t)sp * 2, M - next.m0);
        g.next_f.init(f + (int64_t)e.row0 * fp + next.n0, (int64_t)fp * 2, N - next.n0);
    };
    look_ahead();
    if (!more) return;
    g.s = g.next_s, g.f = g.next_f;
    g.begin(smem, next.k);
    do {
        now = next;
        look_ahead();
        f32x4 acc[8][4];
        g.run<8>(acc);
        const int wave = wave_id(), m_at = now.m0 + (wave >> 2) * 128 + (lane_id() & 15);
        const int n_at = now.n0 + (wave & 3) * 64 + (lane_id() >> 4) * 8;
#pragma unroll
        for (int a = 0; a < 8; ++a)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int m = m_at + a * 16, n = n_at + j * 32;
                if (m < M && n < N) store8(out + now.at + (int64_t)m * N + n, acc[a][j * 2], acc[a][j * 2 + 1]);
            }
    } while (more);
    g.end();
}

template <Product P, bool ONCE = false>
hipError_t rows_launch(const Handle& h, const Params& p, hipStream_t stream) {
    typedef Bf16Tiles<false, P == kDownGrad || P == kInGrad> Tile;
    const int N = P == kGateUp || P == kDownGrad ? p.I : p.H, cols = P == kGateUp ? kBN / 2 : kBN;
    // row tiles that any routing can give: every expert may end in a short one
    const int64_t rows = (int64_t)h.T * h.K / Tile::kBM + h.El;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_rows<P, ONCE>), Tile::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_rows<P, ONCE>), dim3(walking_blocks(rows * ((N + cols - 1) / cols))), dim3(kGemmThreads), Tile::kLds, stream, p);
    return hipGetLastError();
}

hipError_t weights_launch(const Handle& h, const uint16_t* s, const uint16_t* f, uint16_t* out, int M, int N, int sp, int fp,
                          hipStream_t stream) {
    typedef Bf16Tiles<true, true> Tile;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_weights), Tile::kLds);
    if (e != hipSuccess) return e;
    const int64_t tiles = (int64_t)h.El * ((M + Tile::kBM - 1) / Tile::kBM) * ((N + kBN - 1) / kBN);
    hipLaunchKernelGGL(k_weights, dim3(walking_blocks(tiles)), dim3(kGemmThreads), Tile::kLds, stream, h.ws.cnt_local, h.ws.psum,
                       h.El, s, f, out, M, N, sp, fp);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tile_up(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, (const uint16_t*)a.x, (const uint16_t*)a.w13, a.h, nullptr, a.pre, a.hidden, a.inter};
    return weights_once(sizes(h, a)) ? rows_launch<kGateUp, true>(h, p, stream) : rows_launch<kGateUp>(h, p, stream);
}

hipError_t launch_tile_down(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.h, (const uint16_t*)a.w2, (uint16_t*)a.y, nullptr, nullptr, a.hidden, a.inter};
    return rows_launch<kDown>(h, p, stream);
}

hipError_t launch_expert_ffn_backward(const Handle& h, const FfnBackwardArgs& a, hipStream_t stream) {
    const uint16_t* dy = (const uint16_t*)a.dy;
    hipError_t e = hipSuccess;
    if (h.T > 0) {
        const Params dg{h.ws.cnt_local, h.ws.psum, h.El, dy, (const uint16_t*)a.w2, a.dp, a.h, const_cast<float*>(a.pre), a.hidden, a.inter};
        e = rows_launch<kDownGrad>(h, dg, stream);
    }
    if (e == hipSuccess && a.dw2) e = weights_launch(h, dy, a.h, (uint16_t*)a.dw2, a.hidden, a.inter, a.hidden, row_pitch(a.inter), stream);
    if (e == hipSuccess && a.dw13)
        e = weights_launch(h, a.dp, (const uint16_t*)a.x, (uint16_t*)a.dw13, 2 * a.inter, a.hidden,
                           row_pitch(2 * a.inter), a.hidden, stream);
    if (e == hipSuccess && a.dx && h.T > 0) {
        const Params ig{h.ws.cnt_local, h.ws.psum, h.El, a.dp, (const uint16_t*)a.w13, (uint16_t*)a.dx, nullptr, nullptr, a.hidden, a.inter};
        e = rows_launch<kInGrad>(h, ig, stream);
    }
    return e;
}

}  // namespace ep
