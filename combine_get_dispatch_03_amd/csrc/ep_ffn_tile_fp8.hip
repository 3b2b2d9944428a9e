// ep_ffn_tile_fp8.hip -- the expert block's forward pass with e4m3 rows and weights on large tiles.
//
// Gate and up projection: e4m3 by e4m3, twice the rate of bf16.  h stays bf16 (e4m3 would cost it 2^-4 of an element), so
// the down projection is bf16 by e4m3 weights widened on the way to the matrix unit.
//
// An expert's rows rarely fill a tile in serving: the weights pass by once, and both kernels lie between the bytes and the
// products.  Measured, 256 experts of 7168 x 2048, 128 rows each, medians: gate and up 1.57 ms (8.1 GB read, 5.2 TB/s; the matrix
// units are busy 38% of the cycles), down 1.20 ms (4.7 GB read and 0.5 written, 4.4 TB/s; 52%).  With data of zeros, which leave
// the clock higher, 1.49 and 1.00 ms.  4 rows each, weights marked as read once: gate and up 1.10 ms, 6.7 TB/s.
#include "ep_expert_tiles.hpp"
#include "ep_ffn.hpp"
#include "ep_gemm_core.hpp"

namespace ep {
namespace {

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
    const void* s;
    const float* s_scales;    // gate and up: [rows, H / 128]
    const uint8_t* f;
    const float* f_scales;
    uint16_t* out;
    int H, I;
};

template <bool ONCE>
struct GateUp {
    typedef Fp8Tiles<ONCE> Tiles;
    const Params& p;
    RowTiles<Tiles::kBM, 0> rows;      // the registers are needed: find() reads the counts again
    Tiles g;
    int round = 0;
    RowTile now, next;
    int now_n0, next_n0;

    __device__ __forceinline__ explicit GateUp(const Params& params) : p(params), rows(params.cnt, params.psum, params.El) {}

    // The workgroup's next tile; next.rows = 0: there is none.
    __device__ __forceinline__ void look_ahead() {
        TileAt at;
        next.rows = g.next_k = 0;
        if (!tile_at((int)blockIdx.x, round++, rows.total, p.I / 128, &at)) return;
        next = rows.find(at.row, 32);
        const int n0 = next_n0 = at.col * 128, blocks = p.H / 128;
        g.next_k = p.H;
        g.next_s.init((const uint8_t*)p.s + (int64_t)next.row0 * p.H, [&](int r) { return r < next.rows ? (uint32_t)(r * p.H) : kNoElement; });
        // a wave's 64 rows of F: 32 gate channels (fragments 0, 1), then the same 32 up channels
        const uint32_t up = (uint32_t)p.I * p.H;
        g.next_f.init(p.f + ((int64_t)next.expert * 2 * p.I + n0) * p.H,
                      [&](int r) { return (r & 32 ? up : 0u) + (uint32_t)((r / 64 * 32 + channel_of(r / 16 & 1, r & 15)) * p.H); });
        g.next_row_scales(p.s_scales + (int64_t)next.row0 * blocks, blocks, next.rows);
        g.copy_next_f_scales(p.f_scales + ((int64_t)next.expert * 2 * p.I + n0) / 128 * blocks, (uint32_t)(p.I / 128 * blocks) * 4, blocks,
                             round & 1 ? 0 : 1);
    }

    template <int MT>
    __device__ __forceinline__ void tile() {
        f32x4 acc[MT][4];
        g.template run<MT>(acc);
        const int m_at = (wave_id() >> 2) * MT * 16 + (lane_id() & 15), n = now_n0 + (wave_id() & 3) * 32 + (lane_id() >> 4) * 8;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const int m = m_at + a * 16;
            if (m >= now.rows) continue;
            f32x4 h[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) h[b][i] = acc[a][b][i] * sigmoid(acc[a][b][i]) * acc[a][b + 2][i];
            store8(p.out + (int64_t)(now.row0 + m) * p.I + n, h[0], h[1]);
        }
    }
};

// A workgroup stays on its CU and walks through its tiles.  Waves take as many 16-row steps as the tile is high.
template <bool ONCE>
__global__ __launch_bounds__(kGemmThreads, 2) void k_gate_up(Params p) {
    extern __shared__ __align__(1024) char smem[];
    GateUp<ONCE> k(p);
    k.g.smem = smem;
    k.look_ahead();
    if (k.next.rows == 0) return;
    k.g.begin(p.H);
    do {
        k.now = k.next, k.now_n0 = k.next_n0;
        k.look_ahead();
        switch ((k.now.rows + 31) / 32) {
            case 1: k.template tile<1>(); break;
            case 2: k.template tile<2>(); break;
            case 3: k.template tile<3>(); break;
            case 4: k.template tile<4>(); break;
            case 5: k.template tile<5>(); break;
            default: k.template tile<6>(); break;
        }
    } while (k.next.rows > 0);
    k.g.end();
}

struct Down {
    const Params& p;
    RowTiles<Bf16ByFp8Tiles::kBM, 0> rows;
    Bf16ByFp8Tiles g;
    int round = 0;
    RowTile now, next;
    int now_n0, next_n0;

    __device__ __forceinline__ explicit Down(const Params& params) : p(params), rows(params.cnt, params.psum, params.El) {}

    // The workgroup's next tile; next.rows = 0: there is none.
    __device__ __forceinline__ void look_ahead() {
        TileAt at;
        next.rows = g.next_k = 0;
        if (!tile_at((int)blockIdx.x, round++, rows.total, (p.H + kBN - 1) / kBN, &at)) return;
        next = rows.find(at.row, 32);
        const int n0 = next_n0 = at.col * kBN, blocks = p.I / 128;
        g.next_k = p.I;
        g.next_s.init((const uint16_t*)p.s + (int64_t)next.row0 * p.I, [&](int r) { return r < next.rows ? (uint32_t)r * p.I * 2 : kNoElement; });
        g.init_next_f(p.f + ((int64_t)next.expert * p.H + n0) * p.I, [&](int r) {
            const int c = r / 64 * 64 + channel_of(r / 16 & 3, r & 15);
            return n0 + c < p.H ? (uint32_t)(c * p.I) : kNoElement;
        });
        // (a last tile of 128 channels has no second row of scales: its first stands in for channels that do not exist)
        g.copy_next_f_scales(p.f_scales + ((int64_t)next.expert * p.H + n0) / 128 * blocks, n0 + 128 < p.H ? blocks * 4u : 0u, blocks,
                             round & 1 ? 0 : 1);
    }

    template <int MT>
    __device__ __forceinline__ void tile() {
        f32x4 acc[MT][4];
        g.run<MT>(acc);
        const int m_at = (wave_id() >> 2) * MT * 16 + (lane_id() & 15), n_at = now_n0 + (wave_id() & 3) * 64 + (lane_id() >> 4) * 8;
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const int m = m_at + a * 16;
            if (m >= now.rows) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (n_at + j * 32 < p.H) store8(p.out + (int64_t)(now.row0 + m) * p.H + n_at + j * 32, acc[a][j * 2], acc[a][j * 2 + 1]);
        }
    }
};

__global__ __launch_bounds__(kGemmThreads, 2) void k_down(Params p) {
    extern __shared__ __align__(1024) char smem[];
    Down k(p);
    k.g.smem = smem;
    k.look_ahead();
    if (k.next.rows == 0) return;
    k.g.begin(p.I);
    do {
        k.now = k.next, k.now_n0 = k.next_n0;
        k.look_ahead();
        switch ((k.now.rows + 31) / 32) {
            case 1: k.tile<1>(); break;
            case 2: k.tile<2>(); break;
            case 3: k.tile<3>(); break;
            case 4: k.tile<4>(); break;
            default: k.tile<5>(); break;
        }
    } while (k.next.rows > 0);
    k.g.end();
}

}  // namespace

template <bool ONCE>
hipError_t up_launch(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    typedef Fp8Tiles<ONCE> Tiles;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_gate_up<ONCE>), Tiles::kLds);
    if (e != hipSuccess) return e;
    // row tiles that any routing can give: every expert may end in a short one
    const int64_t rows = (int64_t)h.T * h.K / Tiles::kBM + h.El;
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.x, a.x_scales, (const uint8_t*)a.w13, a.w13_scales, a.h, a.hidden, a.inter};
    hipLaunchKernelGGL(k_gate_up<ONCE>, dim3(walking_blocks(rows * (a.inter / 128))), dim3(kGemmThreads), Tiles::kLds, stream, p);
    return hipGetLastError();
}

hipError_t launch_tile_fp8_up(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    return weights_once(sizes(h, a)) ? up_launch<true>(h, a, stream) : up_launch<false>(h, a, stream);
}

hipError_t launch_tile_fp8_down(const Handle& h, const FfnArgs& a, hipStream_t stream) {
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_down), Bf16ByFp8Tiles::kLds);
    if (e != hipSuccess) return e;
    const int64_t rows = (int64_t)h.T * h.K / Bf16ByFp8Tiles::kBM + h.El;
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.h, nullptr, (const uint8_t*)a.w2, a.w2_scales, (uint16_t*)a.y, a.hidden, a.inter};
    hipLaunchKernelGGL(k_down, dim3(walking_blocks(rows * ((a.hidden + kBN - 1) / kBN))), dim3(kGemmThreads), Bf16ByFp8Tiles::kLds, stream, p);
    return hipGetLastError();
}

}  // namespace ep
