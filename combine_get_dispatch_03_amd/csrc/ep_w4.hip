// ep_w4.hip -- experts with weights of four bits: laying the weights out (once, when they are loaded) and the gated feed-forward
// block over the rows that a dispatch placed.
//
//   w[n][k] = s[n][k / group] * v(code[n][k])        v = code - 8, or the e2m1 value of the code
#include "ep_expert_tiles.hpp"
#include "ep_stream.hpp"
#include "ep_w4.hpp"

namespace ep {
namespace {

// Laying out is a copy: 3.8 GB of codes (256 experts' gate and up of 7168 x 2048) take 2.3 ms (3.3 TB/s, reads and writes).
//
// A thread writes 16 bytes of codes, one lane's part of a piece: k j * 32 + g * 8 .. + 7 for j = 0..3 (see ep_weights.hpp).
__global__ __launch_bounds__(256) void k_pack_codes(const uint8_t* codes, char* packed, uint32_t flip, int N, int K, int64_t parts) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= parts) return;
    const int pieces = pieces_of(K), lane = (int)(i & 63), r = lane & 15, g = lane >> 4;
    const int64_t piece = i >> 6, row = piece / pieces * kPieceRows + r;       // of all matrices' rows: N is a multiple of 16
    const int k0 = (int)(piece % pieces) * kPieceK;
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * 32 + g * 8;
        v[j] = k < K ? *reinterpret_cast<const uint32_t*>(codes + (row * K + k) / 2) ^ flip : 0u;
    }
    reinterpret_cast<u32x4*>(packed)[i] = v;
}

// Scales of a piece: [16 rows][groups], bf16; a thread writes one.
__global__ __launch_bounds__(256) void k_pack_scales(const uint16_t* scales, uint16_t* packed, int K, int group, int64_t count) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= count) return;
    const int pieces = pieces_of(K), groups = kPieceK / group, per = 16 * groups;
    const int64_t piece = i / per;
    const int at = (int)(i % per), k = (int)(piece % pieces) * groups + at % groups;
    const int64_t row = piece / pieces * kPieceRows + at / groups;
    packed[i] = k < K / group ? scales[row * (K / group) + k] : (uint16_t)0;
}

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
    const uint16_t* s;     // rows
    WeightArgs w;
    uint16_t* out;
    int N, K;              // channels of a projection's output, of its input
    int sp, op;            // elements between rows of s and of out
};

constexpr int kStreamRows = 64, kStreamPieces = 4;      // of a workgroup: rows, and rows of pieces
template <bool UP>
constexpr int kStreamChannels = kStreamPieces * (UP ? 8 : 16);

template <class W, bool UP, int MT>
__device__ __forceinline__ void rows_product(const Params& p, const RowTile& t, int n0, float* sums) {
    const int r = lane_id() & 15;
    RowFragments<W, MT, !UP> rows;
    rows.init(p.s + (int64_t)t.row0 * p.sp, p.K);
#pragma unroll
    for (int a = 0; a < MT; ++a) rows.place(a, a * 16 + r < t.rows, (uint32_t)(a * 16 + r) * (uint32_t)(p.sp * 2));
    stream_product<W, UP, MT, kStreamPieces>(p.w, t.expert, p.N, p.K, n0, rows, t.rows, sums,
                                             [&](int m) { return p.out + (int64_t)(t.row0 + m) * p.op; });
}

// Up to 64 rows of an expert by four rows of pieces of its weights.  Few tiles spread over idle CUs, and a short sum's latency is what
// they cost: 128 tokens, 8 experts of 256 x 512 take 6.3 us a product.  64 rows' sums and fragments (192 to 217 registers) leave a CU
// room for two workgroups, also where there are fewer rows.
template <class W, bool UP>
__global__ __launch_bounds__(kStreamThreads, 2) void k_w4_stream(Params p) {
    __shared__ __align__(16) float sums[stream_lds<kStreamPieces>() / 4];
    const RowTiles<kStreamRows> tiles(p.cnt, p.psum, p.El);
    const int cols = (p.N + kStreamChannels<UP> - 1) / kStreamChannels<UP>, tile = blockIdx.x / cols;
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find(tile);
    const int n0 = blockIdx.x % cols * kStreamChannels<UP>;
    if (t.rows <= 16) rows_product<W, UP, 1>(p, t, n0, sums);
    else if (t.rows <= 32) rows_product<W, UP, 2>(p, t, n0, sums);
    else rows_product<W, UP, 4>(p, t, n0, sums);
}

template <class W, bool UP>
hipError_t stream_launch(const Handle& h, const Params& p, hipStream_t stream) {
    const int64_t entries = (int64_t)h.T * h.K, busy = entries < h.El ? entries : h.El;
    // tiles that any routing can give: every expert with rows may end in a short one
    const int64_t tiles = (entries + (kStreamRows - 1) * busy) / kStreamRows;
    const int cols = (p.N + kStreamChannels<UP> - 1) / kStreamChannels<UP>;
    hipLaunchKernelGGL((k_w4_stream<W, UP>), dim3((unsigned)(tiles * cols)), dim3(kStreamThreads), 0, stream, p);
    return hipGetLastError();
}

template <class W>
hipError_t ffn(const Handle& h, const W4Args& a, hipStream_t stream) {
    const Params up{h.ws.cnt_local, h.ws.psum, h.El, (const uint16_t*)a.x, WeightArgs{(const char*)a.w13.values, (const char*)a.w13.scales, 2 * a.inter, a.hidden},
                    a.h, a.inter, a.hidden, a.hidden, h_pitch(a.inter)};
    const Params down{h.ws.cnt_local, h.ws.psum, h.El, a.h, WeightArgs{(const char*)a.w2.values, (const char*)a.w2.scales, a.hidden, a.inter},
                      (uint16_t*)a.y, a.hidden, a.inter, h_pitch(a.inter), a.hidden};
    W4Kernel kernel = w4_kernel(W4Sizes{h.T, h.K, h.E, h.El, a.inter, true});
    const hipError_t e = kernel == kW4Stream ? stream_launch<W, true>(h, up, stream) : launch_w4_tile_up(h, a, kernel, stream);
    if (e != hipSuccess) return e;
    kernel = w4_kernel(W4Sizes{h.T, h.K, h.E, h.El, a.hidden, false});
    return kernel == kW4Stream ? stream_launch<W, false>(h, down, stream) : launch_w4_tile_down(h, a, kernel, stream);
}

template <WeightFormat F>
hipError_t by_group(const Handle& h, const W4Args& a, hipStream_t stream) {
    if (a.group == 128) return ffn<Weights<F, 1>>(h, a, stream);
    if (a.group == 64) return ffn<Weights<F, 2>>(h, a, stream);
    return ffn<Weights<F, 4>>(h, a, stream);
}

}  // namespace

size_t w4_packed_bytes(int64_t matrices, int N, int K) { return (size_t)(matrices * (N / kPieceRows) * pieces_of(K)) * kPieceBytes; }
size_t w4_packed_scale_bytes(int64_t matrices, int N, int K, int group) {
    return (size_t)(matrices * (N / kPieceRows) * pieces_of(K)) * (32 * (kPieceK / group));
}

hipError_t launch_w4_pack(const W4PackArgs& a, hipStream_t stream) {
    const int64_t parts = (int64_t)(w4_packed_bytes(a.matrices, a.N, a.K) / 16);
    hipLaunchKernelGGL(k_pack_codes, grid_of((parts + 255) / 256), dim3(256), 0, stream, a.codes, (char*)a.packed, a.int4 ? 0x88888888u : 0u, a.N, a.K, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t count = (int64_t)(w4_packed_scale_bytes(a.matrices, a.N, a.K, a.group) / 2);
    hipLaunchKernelGGL(k_pack_scales, grid_of((count + 255) / 256), dim3(256), 0, stream, a.scales, (uint16_t*)a.packed_scales, a.K, a.group, count);
    return hipGetLastError();
}

hipError_t launch_expert_ffn_w4(const Handle& h, const W4Args& a, hipStream_t stream) {
    if (h.T == 0) return hipSuccess;
    return a.int4 ? by_group<kWeightsInt4>(h, a, stream) : by_group<kWeightsE2m1>(h, a, stream);
}

}  // namespace ep
