// ep_adapter.hip -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = base[t] + B_a v[t],   v[t] = bf16(s_a A_a x[t])      a = the token's adapter
//
// Two kernels, both over tiles of up to 64 tokens of one adapter (the layout's segments), so an adapter's matrices are
// read once per 64 of its tokens and not once per token:
//   shrink   v: the tile's tokens against A_a's rows.  hidden is split over workgroups until the grid fills the chip (a
//            decode batch has few tiles), and over a workgroup's four waves; each workgroup leaves its partial sums
//            in the workspace, tile by tile, and the first of a tile which tokens they are.
//   expand   the partial sums are added in order, scaled and rounded to bf16 in LDS; then B_a's rows times v, added to
//            base and stored.  More workgroups copy base where a token has no adapter.
// v is rounded to bf16, the type the second product's matrix instruction takes.  That is 2^-8 of an element at most, 2^-9 on
// average, beside the same of the output: 0.0019 to 0.0022 of the result in all, where the output's rounding alone leaves 0.0016.  Two bf16 parts
// would keep 16 bits for twice the instructions and LDS.
// Both are bound by memory (x and A; base, out and B): matrix instructions only keep the arithmetic out of the way.
// Measured, 7168 channels in and out: 4096 tokens, 8 adapters of rank 64, shrink 26 us (2.3 TB/s), expand 32 us (3.7 TB/s);
// 128 tokens, 32 adapters of rank 16, 5.2 and 6.8 us; one token, rank 64, 2112 out, 4.7 and 5.8 us: latency, with each
// kernel's chain of dependent loads (segment, token, row).
// The layout maps tokens to rows; a tile finds its tokens by going over that map once (4 bytes a token, from L2), or, where
// there are many tokens, a kernel before turns the map round for all tiles.
#include "ep_expert_tiles.hpp"
#include "ep_gemm_core.hpp"
#include "ep_internal.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave, kRows = 64;
constexpr int kChunkUnit = kWaves * 64;      // hidden channels of a workgroup: a multiple of this
constexpr int kTargetBlocks = 256;           // of shrink: more of them shorten it less than their partial sums lengthen expand
constexpr int kExpandBlocks = 512;
constexpr int kMaxChunks = 32;               // partial sums per token
constexpr int kOut = 256;                    // output channels of an expand workgroup at a time

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
    float* part;          // [chunks][tiles][64][r]
    int32_t* tokens;      // [tiles][64], a tile's tokens in the layout's order
    int tiles;            // that any routing can give
    int bare;             // groups of kRows tokens to look through for those without an adapter
    bool listed;          // tokens come from k_tokens (many tokens), not from shrink
    int H, r, N;
    int chunk, chunks;    // hidden channels per chunk
};

// From so many tokens on their tiles are worked out once, by a kernel of its own (3 us, and a launch): a tile's own search
// is 4 bytes a token, and all searches together go with the square of the tokens.
constexpr int kManyTokens = 8192;

// The thread's part of the layout's map, all of it requested at the start of the kernel, before the tile is known (4096
// tokens: shrink 25.0 us, 25.8 with one piece at the start and the others one by one).
struct Slots {
    i32x4 quad[kManyTokens / 4 / kThreads];
    int rest;
};
__device__ __forceinline__ Slots load_slots(const Params& p) {
    Slots s;
    const int quads = p.T / 4;
#pragma unroll
    for (int u = 0; u < kManyTokens / 4 / kThreads; ++u) {
        const int i = u * kThreads + (int)threadIdx.x;
        s.quad[u] = !p.listed && i < quads ? reinterpret_cast<const i32x4*>(p.slot)[i] : i32x4{-1, -1, -1, -1};
    }
    const int i = quads * 4 + (int)threadIdx.x;
    s.rest = !p.listed && i < p.T ? p.slot[i] : -1;
    return s;
}
// Tokens of a tile, in the layout's order, to LDS.  Ends with a barrier.
__device__ __forceinline__ void find_tokens(const Params& p, const RowTile& t, int tile, const Slots& slots, int* tok) {
    if (p.listed) {
        if ((int)threadIdx.x < t.rows) tok[threadIdx.x] = p.tokens[(int64_t)tile * kRows + threadIdx.x];
        __syncthreads();
        return;
    }
    auto put = [&](int s, int token) {
        const uint32_t m = (uint32_t)(s - t.row0);
        if (m < (uint32_t)t.rows) tok[m] = token;
    };
#pragma unroll
    for (int u = 0; u < kManyTokens / 4 / kThreads; ++u) {
        if (u * kThreads * 4 >= p.T) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) put(slots.quad[u][j], (u * kThreads + (int)threadIdx.x) * 4 + j);
    }
    put(slots.rest, p.T / 4 * 4 + (int)threadIdx.x);
    __syncthreads();
}

// tokens[tile][m] for every token with an adapter.
__global__ __launch_bounds__(kThreads) void k_tokens(Params p) {
    __shared__ int before[kMaxExperts];      // tiles of the adapters before each
    __shared__ int start[kMaxExperts];       // their first rows
    for (int e = threadIdx.x; e < p.El; e += kThreads) start[e] = p.psum[e];
    if (threadIdx.x < kWave) {
        const RowTiles<kRows, 0> tiles(p.cnt, p.psum, p.El);
        int at = tiles.incl - tiles.sum;
        for (int i = 0; i < tiles.per; ++i) {
            const int e = lane_id() * tiles.per + i;
            if (e >= p.El) break;
            before[e] = at;
            at += (p.cnt[e] + kRows - 1) / kRows;
        }
    }
    __syncthreads();
    const int t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= p.T) return;
    const int slot = p.slot[t];
    if (slot < 0) return;
    int e = 0;                               // the last adapter that starts at or before the row: the others there are empty
    for (int n = p.El; n > 1;) {
        const int half = n / 2;
        if (start[e + half] <= slot) e += half;
        n -= half;
    }
    p.tokens[(int64_t)before[e] * kRows + (slot - start[e])] = t;      // a tile's rows are consecutive, and so are tiles
}

template <int NF, int MT>
__device__ __forceinline__ void shrink(const Params& p, const RowTile& t, int tile, int chunk, const Slots& slots, int* tok, float* sums) {
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    // Up to 32 tokens: four lanes beside each other load 64 bytes of a row, and the fragments are put right by an exchange
    // of lanes; 128 tokens of 32 adapters of rank 16 5.4 us, 5.9 without; 64 tokens a tile 25.6 and 24.9 us.
    constexpr bool kTurn = MT <= 2;
    const int lr = kTurn ? lane >> 2 : r, lg = kTurn ? lane & 3 : g;
    auto turn = [&](i32x4 v) {
        if constexpr (kTurn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_ds_bpermute((r * 4 + g) * 4, v[i]);
        }
        return v;
    };
    const uint16_t* f[NF];
    bool f_there[NF];
#pragma unroll
    for (int b = 0; b < NF; ++b) {
        f_there[b] = b * 16 + lr < p.r;
        f[b] = p.a + ((int64_t)t.expert * p.r + (f_there[b] ? b * 16 + lr : 0)) * p.H + lg * 8;
    }
    f32x4 acc[MT][NF];
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NF; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int end = min(p.H, (chunk + 1) * p.chunk);
    struct Step {
        i32x4 s[MT][2], f[NF][2];
    };
    const int first = chunk * p.chunk + wave * 64;
    Step next;
    auto load_f = [&](Step& v, int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int b = 0; b < NF; ++b) {
                v.f[b][j] = i32x4{0, 0, 0, 0};
                if (k + j * 32 + lg * 8 < end && f_there[b]) v.f[b][j] = *(const i32x4*)(f[b] + k + j * 32);
            }
    };
    load_f(next, first);       // A's rows do not depend on the tokens
    find_tokens(p, t, tile, slots, tok);
    if (chunk == 0 && !p.listed && (int)threadIdx.x < t.rows) p.tokens[(int64_t)tile * kRows + threadIdx.x] = tok[threadIdx.x];
    const uint16_t* s[MT];
    bool s_there[MT];
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        s_there[a] = a * 16 + lr < t.rows;
        s[a] = p.x + (int64_t)tok[s_there[a] ? a * 16 + lr : 0] * p.H + lg * 8;
    }
    auto load_s = [&](Step& v, int k) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                v.s[a][j] = i32x4{0, 0, 0, 0};
                if (k + j * 32 + lg * 8 < end && s_there[a]) v.s[a][j] = *(const i32x4*)(s[a] + k + j * 32);
            }
    };
    load_s(next, first);
    for (int k = first; k < end; k += kChunkUnit) {
        Step cur;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int b = 0; b < NF; ++b) cur.f[b][j] = turn(next.f[b][j]);
#pragma unroll
            for (int a = 0; a < MT; ++a) cur.s[a][j] = turn(next.s[a][j]);
        }
        load_f(next, k + kChunkUnit);     // past the end: nothing is read
        load_s(next, k + kChunkUnit);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < NF; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cur.f[b][j]),
                                                                        __builtin_bit_cast(bf16x8, cur.s[a][j]), acc[a][b], 0, 0, 0);
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
            *reinterpret_cast<f32x4*>(p.part + (((int64_t)chunk * p.tiles + tile) * kRows + a * 16 + m) * p.r + n4) = v;
        }
    }
}

template <int NF>
__global__ __launch_bounds__(kThreads) void k_shrink(Params p) {
    __shared__ __align__(16) float sums[kWaves * 16 * (NF * 16 + 4)];
    __shared__ int tok[kRows];
    const Slots slots = load_slots(p);
    const RowTiles<kRows> tiles(p.cnt, p.psum, p.El);
    const int tile = blockIdx.x / p.chunks;
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    const int chunk = blockIdx.x % p.chunks;
    if (t.rows <= 16) shrink<NF, 1>(p, t, tile, chunk, slots, tok, sums);
    else if (t.rows <= 32) shrink<NF, 2>(p, t, tile, chunk, slots, tok, sums);
    else shrink<NF, 4>(p, t, tile, chunk, slots, tok, sums);
}

// What the lanes of a wave wrote to LDS is there for all of them, and what they read has been read.
__device__ __forceinline__ void wave_meets() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// NK: steps of 32 over the rank.  A workgroup takes `steps` times 256 channels.
template <int NK>
__global__ __launch_bounds__(kThreads) void k_expand(Params p, int steps) {
    constexpr int kPitch = NK * 32 + 8;
    __shared__ __align__(16) uint16_t v[kRows * kPitch];
    __shared__ __align__(16) f32x4 shared_sums[kThreads];
    constexpr int kTurnPitch = 64 + 4;
    __shared__ __align__(16) float turn[kWaves][16 * kTurnPitch];
    const int cols = (p.N + kOut * steps - 1) / (kOut * steps), block = (int)block_id(), tile = block / cols, first = block % cols * kOut * steps;
    const int last = min(p.N, first + kOut * steps);
    if (tile >= p.tiles) {      // tokens without an adapter: base as it is
        if (tile - p.tiles >= p.bare) return;
        const int t0 = (tile - p.tiles) * kRows, width = (last - first) / 8;
        uint64_t bare = ballot(t0 + lane_id() < p.T && p.slot[min(t0 + lane_id(), p.T - 1)] < 0);
        for (int i = 0; bare != 0; ++i, bare &= bare - 1) {
            if (i % kWaves != wave_id()) continue;
            const int64_t at = (int64_t)(t0 + __builtin_ctzll(bare)) * p.N + first;
            for (int c = lane_id(); c < width; c += kWave)
                *reinterpret_cast<i32x4*>(p.out + at + c * 8) = p.base ? *reinterpret_cast<const i32x4*>(p.base + at + c * 8) : i32x4{0, 0, 0, 0};
        }
        return;
    }
    const RowTiles<kRows> tiles(p.cnt, p.psum, p.El);
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4;
    // A wave's product is 64 channels of 16 tokens at a time, a lane's share of it four channels of a token 16 lanes from the
    // next.  It goes round by LDS: base is read and out written with eight lanes on a token's 128 bytes, which the address
    // unit takes at four lanes a cycle; lane by lane from as many rows it takes one.
    int tok[kRows / 8];       // of the rows that the lane stores
#pragma unroll
    for (int a = 0; a < kRows / 8; ++a) tok[a] = a * 8 + (lane >> 3) < t.rows ? p.tokens[(int64_t)tile * kRows + a * 8 + (lane >> 3)] : 0;
    struct Rows {
        i32x4 v[4][NK];
    };
    auto load_b = [&](int nw) {
        Rows f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int n = nw + b * 16 + r;
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                f.v[b][j] = i32x4{0, 0, 0, 0};
                if (n < last && j * 32 + g * 8 < p.r)
                    f.v[b][j] = *(const i32x4*)(p.b + ((int64_t)t.expert * p.N + n) * p.r + j * 32 + g * 8);
            }
        }
        return f;
    };
    struct Base {
        i32x4 v[kRows / 8];
    };
    const int n_in = (lane & 7) * 8;
    auto load_base = [&](int nw) {
        Base o;
#pragma unroll
        for (int a = 0; a < kRows / 8; ++a) {
            o.v[a] = i32x4{0, 0, 0, 0};
            if (p.base && a * 8 + (lane >> 3) < t.rows && nw + n_in < last)
                o.v[a] = *reinterpret_cast<const i32x4*>(p.base + (int64_t)tok[a] * p.N + nw + n_in);
        }
        return o;
    };
    int nw = first + wave * 64;
    Rows next = load_b(nw);
    Base next_base = load_base(nw);
    const float scale = p.scales ? p.scales[t.expert] : 1.0f;
    // v of the tile's tokens, zeros past the last token and past the rank, 4 ranks per item; the chunks are added in a fixed
    // order.  A few tokens: the workgroup's threads share an item's chunks and meet in LDS.  Many: two items a thread,
    // eight chunks of each in flight.
    const int items = ((t.rows + 15) & ~15) * NK * 8;
    auto item = [&](int i, const float** from) {
        const int m = i / (NK * 8), k4 = i % (NK * 8) * 4;
        *from = m < t.rows && k4 < p.r ? p.part + ((int64_t)tile * kRows + m) * p.r + k4 : nullptr;
        return m * kPitch + k4;
    };
    auto put = [&](int at, f32x4 sum) {
        *reinterpret_cast<i32x2*>(v + at) = i32x2{(int)pack_bf16x2(sum[0] * scale, sum[1] * scale), (int)pack_bf16x2(sum[2] * scale, sum[3] * scale)};
    };
    const int64_t stride = (int64_t)p.tiles * kRows * p.r;
    if (t.rows <= 16) {
        // only rows that exist are shared out; the others' v is zero
        constexpr int kPerRow = NK * 8;
        int rows = 1;
        while (rows < t.rows) rows *= 2;
        const int live = rows * kPerRow, shares = live < kThreads ? kThreads / live : 1;
        for (int i = threadIdx.x; i < items; i += kThreads)
            if (i >= live) put(i / kPerRow * kPitch + i % kPerRow * 4, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        for (int i0 = 0; i0 < live; i0 += kThreads) {
            const int i = i0 + (int)threadIdx.x % (kThreads / shares), share = (int)threadIdx.x / (kThreads / shares);
            const float* from;
            const int at = item(i, &from);
            f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
            for (int c0 = share; c0 < p.chunks; c0 += 4 * shares) {
                f32x4 part[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    part[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    if (from && c0 + u * shares < p.chunks) part[u] = *reinterpret_cast<const f32x4*>(from + (c0 + u * shares) * stride);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) sum += part[u];
            }
            if (shares > 1) {
                __syncthreads();
                shared_sums[threadIdx.x] = sum;
                __syncthreads();
                if (share == 0)
                    for (int q = 1; q < shares; ++q) sum += shared_sums[threadIdx.x + q * (kThreads / shares)];
            }
            if (share == 0) put(at, sum);
        }
    } else {
        constexpr int kAt = 2, kDeep = 8;
        for (int i0 = threadIdx.x; i0 < items; i0 += kAt * kThreads) {
            const float* from[kAt];
            int at[kAt];
            f32x4 sum[kAt];
#pragma unroll
            for (int q = 0; q < kAt; ++q) {
                at[q] = i0 + q * kThreads < items ? item(i0 + q * kThreads, &from[q]) : -1;
                if (at[q] < 0) from[q] = nullptr;
                sum[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
            for (int c = 0; c < p.chunks; c += kDeep) {
                f32x4 part[kDeep][kAt];
#pragma unroll
                for (int u = 0; u < kDeep; ++u)
#pragma unroll
                    for (int q = 0; q < kAt; ++q) {
                        part[u][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                        if (from[q] && c + u < p.chunks) part[u][q] = *reinterpret_cast<const f32x4*>(from[q] + (c + u) * stride);
                    }
#pragma unroll
                for (int u = 0; u < kDeep; ++u)
#pragma unroll
                    for (int q = 0; q < kAt; ++q) sum[q] += part[u][q];
            }
#pragma unroll
            for (int q = 0; q < kAt; ++q)
                if (at[q] >= 0) put(at[q], sum[q]);
        }
    }
    __syncthreads();
    for (; nw < last; nw += kOut) {
        const Rows cur = next;
        const Base base = next_base;
        if (nw + kOut < last) {
            next = load_b(nw + kOut);
            next_base = load_base(nw + kOut);
        }
#pragma unroll
        for (int a = 0; a < kRows / 16; ++a) {
            if (a * 16 >= t.rows) break;
            f32x4 acc[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const bf16x8 sv = *reinterpret_cast<const bf16x8*>(v + (a * 16 + r) * kPitch + j * 32 + g * 8);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cur.v[b][j]), sv, acc[b], 0, 0, 0);
            }
            wave_meets();
#pragma unroll
            for (int b = 0; b < 4; ++b) *reinterpret_cast<f32x4*>(turn[wave] + r * kTurnPitch + b * 16 + g * 4) = acc[b];
            wave_meets();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int m8 = a * 2 + h;
                const float* at = turn[wave] + (h * 8 + (lane >> 3)) * kTurnPitch + n_in;
                const f32x4 d[2] = {*reinterpret_cast<const f32x4*>(at), *reinterpret_cast<const f32x4*>(at + 4)};
                i32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t two = (uint32_t)base.v[m8][i];
                    o[i] = (int)pack_bf16x2(bf16lo(two) + d[i / 2][i % 2 * 2], bf16hi(two) + d[i / 2][i % 2 * 2 + 1]);
                }
                if (m8 * 8 + (lane >> 3) < t.rows && nw + n_in < last) *reinterpret_cast<i32x4*>(p.out + (int64_t)tok[m8] * p.N + nw + n_in) = o;
            }
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
    if (chunks > kMaxChunks) chunks = kMaxChunks;
    return (units + chunks - 1) / chunks * kChunkUnit;
}

}  // namespace

// The workspace: partial sums, then the tiles' tokens.
static size_t part_bytes(int chunks, int tiles, int rank) {
    return ((size_t)chunks * (size_t)tiles * kRows * (size_t)rank * sizeof(float) + 255) / 256 * 256;
}

size_t adapter_workspace_bytes(int T, int El, int hidden, int rank) {
    const int chunk = chunk_of(T, El, hidden), chunks = (hidden + chunk - 1) / chunk, tiles = max_tiles(T, El);
    return part_bytes(chunks, tiles, rank) + (size_t)(tiles > 0 ? tiles : 1) * kRows * sizeof(int32_t);
}

hipError_t launch_adapter(const Handle& h, const AdapterArgs& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    const int chunk = chunk_of(h.T, h.El, a.hidden), chunks = (a.hidden + chunk - 1) / chunk, tiles = max_tiles(h.T, h.El);
    int32_t* tokens = reinterpret_cast<int32_t*>(static_cast<char*>(a.ws) + part_bytes(chunks, tiles, a.rank));
    const bool listed = h.T >= kManyTokens;
    // in place, the tokens without an adapter already hold their base
    const int bare = a.out == a.base ? 0 : (int)(((int64_t)h.T + kRows - 1) / kRows);
    const Params p{h.ws.cnt_local, h.ws.psum, h.ws.slot, h.T, h.El, (const uint16_t*)a.x, (const uint16_t*)a.a,
                   (const uint16_t*)a.b, a.scales, (const uint16_t*)a.base, (uint16_t*)a.out, (float*)a.ws, tokens, tiles, bare, listed,
                   a.hidden, a.rank, a.n_out, chunk, chunks};
    if (listed) {
        hipLaunchKernelGGL(k_tokens, dim3((unsigned)((h.T + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 shrink_grid((unsigned)((int64_t)tiles * chunks)), block(kThreads);
    if (a.rank <= 16) hipLaunchKernelGGL(k_shrink<1>, shrink_grid, block, 0, stream, p);
    else if (a.rank <= 32) hipLaunchKernelGGL(k_shrink<2>, shrink_grid, block, 0, stream, p);
    else if (a.rank <= 64) hipLaunchKernelGGL(k_shrink<4>, shrink_grid, block, 0, stream, p);
    else hipLaunchKernelGGL(k_shrink<8>, shrink_grid, block, 0, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // as many channels per workgroup as leave the chip full: a workgroup adds up v before it starts
    const int columns = (a.n_out + kOut - 1) / kOut, want = (kExpandBlocks + tiles - 1) / tiles, steps = columns > want ? (columns + want - 1) / want : 1;
    const dim3 expand_grid = grid_of((int64_t)(tiles + bare) * ((columns + steps - 1) / steps));
    if (a.rank <= 32) hipLaunchKernelGGL(k_expand<1>, expand_grid, block, 0, stream, p, steps);
    else if (a.rank <= 64) hipLaunchKernelGGL(k_expand<2>, expand_grid, block, 0, stream, p, steps);
    else hipLaunchKernelGGL(k_expand<4>, expand_grid, block, 0, stream, p, steps);
    return hipGetLastError();
}

}  // namespace ep
