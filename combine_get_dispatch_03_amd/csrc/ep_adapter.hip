// ep_adapter.hip -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + B_a v[t],   v[t] = bf16(s_a A_a x[t])      a = the token's adapter
//
// Two kernels, both over tiles of up to 64 tokens of one adapter (the layout's segments), so an adapter's matrices are
// read once per 64 of its tokens and not once per token:
//   shrink   v: the tile's tokens against A_a's rows.  hidden is split over workgroups until the grid fills the chip (a
//            decode batch has few tiles), and over a workgroup's four waves; each workgroup leaves its partial sums per
//            token in the workspace.
//   expand   the partial sums are added in order, scaled and rounded to bf16 in LDS; then B_a's rows times v, added to
//            base and stored, 256 output channels per workgroup.  More workgroups copy base where a token has no adapter.
// Both are bound by memory (x and A; base, out and B): matrix instructions only keep the arithmetic out of the way.
// The layout maps tokens to rows; a tile finds its tokens by going over that map once (4 bytes a token, from L2).
#include "ep_expert_tiles.hpp"
#include "ep_gemm_core.hpp"
#include "ep_internal.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave, kRows = 64;
constexpr int kChunkUnit = kWaves * 64;      // hidden channels of a workgroup: a multiple of this
constexpr int kTargetBlocks = 512;           // two workgroups per CU
constexpr int kOut = 256;                    // output channels of an expand workgroup

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    const int32_t* slot;
    int T, El;
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scales;
    const uint16_t* base;
    uint16_t* out;
    float* part;          // [chunks][T][r]
    int H, r, N;
    int chunk, chunks;    // hidden channels per chunk
};

// Tokens of a tile, in the layout's order, to LDS.  Ends with a barrier.
__device__ __forceinline__ void find_tokens(const Params& p, const RowTile& t, int* tok) {
    const int quads = p.T / 4;
    const i32x4* q = reinterpret_cast<const i32x4*>(p.slot);
    auto put = [&](int s, int token) {
        const uint32_t m = (uint32_t)(s - t.row0);
        if (m < (uint32_t)t.rows) tok[m] = token;
    };
    for (int i = threadIdx.x; i < quads; i += kThreads) {
        const i32x4 s = q[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) put(s[j], i * 4 + j);
    }
    const int rest = quads * 4 + (int)threadIdx.x;
    if (rest < p.T) put(p.slot[rest], rest);
    __syncthreads();
}

template <int NF, int MT>
__device__ __forceinline__ void shrink(const Params& p, const RowTile& t, int chunk, const int* tok, float* sums) {
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    const uint16_t* f[NF];
    bool f_there[NF];
#pragma unroll
    for (int b = 0; b < NF; ++b) {
        f_there[b] = b * 16 + r < p.r;
        f[b] = p.a + ((int64_t)t.expert * p.r + (f_there[b] ? b * 16 + r : 0)) * p.H + g * 8;
    }
    const uint16_t* s[MT];
    bool s_there[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        s_there[a] = a * 16 + r < t.rows;
        s[a] = p.x + (int64_t)tok[s_there[a] ? a * 16 + r : 0] * p.H + g * 8;
    }
    f32x4 acc[MT][NF];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NF; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int end = min(p.H, (chunk + 1) * p.chunk);
    for (int k = chunk * p.chunk + wave * 64; k < end; k += kChunkUnit) {
        i32x4 sv[MT][2], fv[NF][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bool in = k + j * 32 + g * 8 < end;
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                sv[a][j] = i32x4{0, 0, 0, 0};
                if (in && s_there[a]) sv[a][j] = *(const i32x4*)(s[a] + k + j * 32);
            }
#pragma unroll
            for (int b = 0; b < NF; ++b) {
                fv[b][j] = i32x4{0, 0, 0, 0};
                if (in && f_there[b]) fv[b][j] = *(const i32x4*)(f[b] + k + j * 32);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < NF; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fv[b][j]),
                                                                        __builtin_bit_cast(bf16x8, sv[a][j]), acc[a][b], 0, 0, 0);
    }
    constexpr int kPitch = NF * 16 + 4;
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        __syncthreads();
#pragma unroll
        for (int b = 0; b < NF; ++b) *reinterpret_cast<f32x4*>(sums + (wave * 16 + r) * kPitch + b * 16 + g * 4) = acc[a][b];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * NF * 4; i += kThreads) {
            const int m = i / (NF * 4), n4 = i % (NF * 4) * 4;
            if (a * 16 + m >= t.rows || n4 >= p.r) continue;
            f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += *reinterpret_cast<const f32x4*>(sums + (w * 16 + m) * kPitch + n4);
            *reinterpret_cast<f32x4*>(p.part + ((int64_t)chunk * p.T + tok[a * 16 + m]) * p.r + n4) = v;
        }
    }
}

template <int NF>
__global__ __launch_bounds__(kThreads) void k_shrink(Params p) {
    __shared__ __align__(16) float sums[kWaves * 16 * (NF * 16 + 4)];
    __shared__ int tok[kRows];
    const RowTiles<kRows> tiles(p.cnt, p.psum, p.El);
    const int tile = blockIdx.x / p.chunks;
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    find_tokens(p, t, tok);
    const int chunk = blockIdx.x % p.chunks;
    if (t.rows <= 16) shrink<NF, 1>(p, t, chunk, tok, sums);
    else if (t.rows <= 32) shrink<NF, 2>(p, t, chunk, tok, sums);
    else shrink<NF, 4>(p, t, chunk, tok, sums);
}

// NK: steps of 32 over the rank.
template <int NK>
__global__ __launch_bounds__(kThreads) void k_expand(Params p, int max_tiles) {
    constexpr int kPitch = NK * 32 + 8;
    __shared__ __align__(16) uint16_t v[kRows * kPitch];
    __shared__ int tok[kRows];
    const RowTiles<kRows> tiles(p.cnt, p.psum, p.El);
    const int cols = (p.N + kOut - 1) / kOut, tile = blockIdx.x / cols, n0 = blockIdx.x % cols * kOut;
    if (tile >= max_tiles) {      // tokens without an adapter: base as it is
        const int t0 = (tile - max_tiles) * kRows;
        for (int i = threadIdx.x; i < kRows * (kOut / 8); i += kThreads) {
            const int t = t0 + i / (kOut / 8), n = n0 + i % (kOut / 8) * 8;
            if (t >= p.T || n >= p.N || p.slot[t] >= 0) continue;
            const int64_t at = (int64_t)t * p.N + n;
            *reinterpret_cast<i32x4*>(p.out + at) = p.base ? *reinterpret_cast<const i32x4*>(p.base + at) : i32x4{0, 0, 0, 0};
        }
        return;
    }
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    // 64 channels per wave.  Fragment b takes channels 16 g + 4 b + i as its rows 4 g + i, so that a lane ends up with 16
    // consecutive channels of a token.
    const int nw = n0 + wave * 64;
    i32x4 fv[4][NK];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int n = nw + (r >> 2) * 16 + b * 4 + (r & 3);
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            fv[b][j] = i32x4{0, 0, 0, 0};
            if (n < p.N && j * 32 + g * 8 < p.r)
                fv[b][j] = *(const i32x4*)(p.b + ((int64_t)t.expert * p.N + n) * p.r + j * 32 + g * 8);
        }
    }
    find_tokens(p, t, tok);
    const float scale = p.scales ? p.scales[t.expert] : 1.0f;
    for (int i = threadIdx.x; i < kRows * NK * 8; i += kThreads) {
        const int m = i / (NK * 8), k4 = i % (NK * 8) * 4;
        f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
        if (m < t.rows && k4 < p.r) {
            const float* from = p.part + (int64_t)tok[m] * p.r + k4;
            for (int c = 0; c < p.chunks; ++c) sum += *reinterpret_cast<const f32x4*>(from + (int64_t)c * p.T * p.r);
        }
        *reinterpret_cast<i32x2*>(v + m * kPitch + k4) =
            i32x2{(int)pack_bf16x2(sum[0] * scale, sum[1] * scale), (int)pack_bf16x2(sum[2] * scale, sum[3] * scale)};
    }
    __syncthreads();
    for (int a = 0; a * 16 < t.rows; ++a) {
        const int m = a * 16 + r, n = nw + g * 16;
        const bool in[2] = {m < t.rows && n < p.N, m < t.rows && n + 8 < p.N};
        const int64_t at = in[0] ? (int64_t)tok[m] * p.N + n : 0;
        i32x4 base[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            base[j] = i32x4{0, 0, 0, 0};
            if (in[j] && p.base) base[j] = *reinterpret_cast<const i32x4*>(p.base + at + j * 8);
        }
        f32x4 acc[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const bf16x8 sv = *reinterpret_cast<const bf16x8*>(v + m * kPitch + j * 32 + g * 8);
#pragma unroll
            for (int b = 0; b < 4; ++b)
                acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fv[b][j]), sv, acc[b], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            i32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 d = acc[j * 2 + i / 2];
                o[i] = (int)pack_bf16x2(bf16lo((uint32_t)base[j][i]) + d[i % 2 * 2], bf16hi((uint32_t)base[j][i]) + d[i % 2 * 2 + 1]);
            }
            if (in[j]) *reinterpret_cast<i32x4*>(p.out + at + j * 8) = o;
        }
    }
}

// Tiles that any routing can give: no more than tokens, and every adapter may end in a short one.
int max_tiles(int T, int El) {
    const int64_t n = (int64_t)T / kRows + El;
    return (int)(n < T ? n : T);
}

// Hidden channels per workgroup: enough workgroups to fill the chip, as few partial sums as that allows.
int chunk_of(int T, int El, int H) {
    const int units = (H + kChunkUnit - 1) / kChunkUnit, tiles = max_tiles(T, El) > 0 ? max_tiles(T, El) : 1;
    int chunks = kTargetBlocks / tiles;
    if (chunks < 1) chunks = 1;
    if (chunks > units) chunks = units;
    return (units + chunks - 1) / chunks * kChunkUnit;
}

}  // namespace

size_t adapter_workspace_bytes(int T, int El, int hidden, int rank) {
    const int chunk = chunk_of(T, El, hidden), chunks = (hidden + chunk - 1) / chunk;
    const size_t bytes = (size_t)chunks * (size_t)T * (size_t)rank * sizeof(float);
    return bytes > 256 ? bytes : 256;
}

hipError_t launch_adapter(const Handle& h, const AdapterArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const int chunk = chunk_of(h.T, h.El, a.hidden), chunks = (a.hidden + chunk - 1) / chunk, tiles = max_tiles(h.T, h.El);
    const Params p{h.ws.cnt_local, h.ws.psum, h.ws.slot, h.T, h.El, (const uint16_t*)a.x, (const uint16_t*)a.a,
                   (const uint16_t*)a.b, a.scales, (const uint16_t*)a.base, (uint16_t*)a.out, (float*)a.ws,
                   a.hidden, a.rank, a.n_out, chunk, chunks};
    const dim3 shrink_grid((unsigned)(tiles * chunks)), block(kThreads);
    if (a.rank <= 16) hipLaunchKernelGGL(k_shrink<1>, shrink_grid, block, 0, stream, p);
    else if (a.rank <= 32) hipLaunchKernelGGL(k_shrink<2>, shrink_grid, block, 0, stream, p);
    else if (a.rank <= 64) hipLaunchKernelGGL(k_shrink<4>, shrink_grid, block, 0, stream, p);
    else hipLaunchKernelGGL(k_shrink<8>, shrink_grid, block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // in place, the tokens without an adapter already hold their base
    const int bare = a.out == a.base ? 0 : (h.T + kRows - 1) / kRows;
    const dim3 expand_grid((unsigned)((int64_t)(tiles + bare) * ((a.n_out + kOut - 1) / kOut)));
    if (a.rank <= 32) hipLaunchKernelGGL(k_expand<1>, expand_grid, block, 0, stream, p, tiles);
    else if (a.rank <= 64) hipLaunchKernelGGL(k_expand<2>, expand_grid, block, 0, stream, p, tiles);
    else hipLaunchKernelGGL(k_expand<4>, expand_grid, block, 0, stream, p, tiles);
    return hipGetLastError();
}

}  // namespace ep
