// ep_w4_tile.hip -- the expert block with 4-bit weights on tiles: up to 32, 64 or 128 rows by 256 channels.
//
// Rows, codes and scales of 128 k (a stage) are copied to LDS without passing registers, one or two stages ahead; a piece of
// codes is 1024 bytes in a row in memory and in LDS, so copying and reading it take whole lines and no two lanes meet in a
// bank.  A wave widens its codes (exactly) on their way from LDS to the matrix instruction; a group's sums are kept apart and take
// their scale in fp32 on the way into acc.  Those second sums are what limits a tile to 128 rows.  All eight waves stand along the
// channels, so that every code is widened once (with two rows of waves, int4: 4096 tokens 2.97 and 2.75 ms).  A tile of 128 rows
// has a CU to itself; of 32 and 64 rows there are two, each of which works while the other waits (16 tokens, 32 experts of 7168 x
// 2048, int4: 148 us, one workgroup of six stages 158).  A workgroup stays on its CU and its tiles form one stream of stages, as in
// Bf16Tiles.
//
// h goes out in fp16 beside numbers (ep_h_rows.hpp) and comes back to the down product in fp16, a row in one unit.
//
// What bounds them: with 32 rows an expert (128 tokens, 32 such experts, int4 in groups of 128) bytes, widening and products together,
// gate and up 110 us (4.5 TB/s), down 68 (3.6 TB/s). With 1024 rows (4096 tokens, 2.89 TFLOP) the sum of the matrix unit's time and the
// vector unit's: the whole call with e2m1 in groups of 128 takes 2.65 ms (1.09 PFLOP/s), in groups of 32, four times the scalings, 3.2, with
// int4 in groups of 128, three times the widening, 2.85. Tiles of 64 rows have 128 registers and spill up to 14 of them in the down product
// of groups of 64 and 128 (and one for gate and up); tiles of 32 and 128 rows none.
#include "ep_expert_tiles.hpp"
#include "ep_ffn.hpp"
#include "ep_w4.hpp"
#include "ep_weights.hpp"

namespace ep {
namespace {

struct Params {
    const int32_t* cnt;
    const int32_t* psum;
    int El;
    const uint16_t* s;     // rows: x, or h with one number a row
    WeightArgs w;
    uint16_t* out;         // h, or y
    int N, K;              // channels of a projection's output, of its input
    int sp, op;            // elements between rows of s and of out
};

// h's rows go to LDS as they are, so a row needs one number for all of its blocks before: a wave looks at a row's numbers, brings
// blocks with others to the largest where there are any, and leaves the row's unit, which the tiles multiply their sums by.  1024 rows 4.6
// us, 32768 rows of 2048 channels 11.5 us (looking at all rows of the workspace, without finding those that experts have: 8.0 and 14).
__device__ __forceinline__ float* row_unit(uint16_t* row, int I) { return reinterpret_cast<float*>(row + I + numbers_of(I)); }
constexpr int kUnitRows = 4;
__global__ __launch_bounds__(kUnitRows * kWave) void k_one_number(const int32_t* cnt, const int32_t* psum, int El, uint16_t* h, int I) {
    const RowTiles<kUnitRows> tiles(cnt, psum, El);
    const int64_t tile = block_id();
    if (tile >= tiles.total) return;
    const RowTile t = tiles.find((int)tile);
    if (wave_id() >= t.rows) return;
    uint16_t* row = h + (int64_t)(t.row0 + wave_id()) * h_pitch(I);
    const uint32_t* numbers = reinterpret_cast<const uint32_t*>(row + I);      // two each: I is a multiple of 32
    NumberRange range;
    for (int i = lane_id(); i < I / (2 * kShared); i += kWave) range.add(numbers[i], 2);
    const uint32_t most = max_bits<16>((uint32_t)range.top());
    const int top = max(max(readlane((int)most, 0), readlane((int)most, 16)), max(readlane((int)most, 32), readlane((int)most, 48)));
    if (ballot(range.low() < top))
        for (int c = lane_id(); c < I / 8; c += kWave) {
            u32x4* at = reinterpret_cast<u32x4*>(row) + c;
            *at = bring_to(*at, (int)row[I + c / (kShared / 8)], top);
        }
    if (lane_id() == 0) *row_unit(row, I) = shared_unit(top);
}

// Rows with 128 k of each per stage, ROWS of them: 256 bytes, whose 16-byte chunks are permuted by the row number so that a
// fragment read (16 rows, 16 bytes at one place of each) is spread over all banks.
template <int ROWS>
struct WideRows {
    static constexpr int kCopies = ROWS / 4 / kGemmWaves, kBytes = ROWS * 256;
    uint64_t base;
    uint32_t offset[kCopies];

    static __device__ __forceinline__ int row(int i) { return (i * kGemmWaves + wave_id()) * 4 + (lane_id() >> 4); }
    static __device__ __forceinline__ int chunk(int i) { return (lane_id() & 15) ^ (row(i) & 15); }
    __device__ __forceinline__ void settle() {
        base = uniform64(base);
        asm volatile("s_nop 4" : "+s"(base));
    }
    // row_offset(r): byte offset of row r from `start`, or kNoElement.
    template <class RowOffset>
    __device__ __forceinline__ void init(const void* start, RowOffset row_offset) {
        base = uniform64((uint64_t)start);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t o = row_offset(row(i));
            offset[i] = o == kNoElement ? kNoElement : o + chunk(i) * 16;
        }
    }
    // As KcOperand::copy: `left` bytes of each row to go.
    __device__ __forceinline__ void copy(uint32_t lds, int left) {
        if (left < 256) {
            stay_branch();
#pragma unroll
            for (int i = 0; i < kCopies; ++i) offset[i] = chunk(i) * 16 < left ? offset[i] : kNoElement;
        }
        const i32x4 res = ep::resource(base);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds + threadIdx.x / kWave * 1024);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) copy16_to_lds(to + i * kGemmWaves * 1024, offset[i], res);
        base += 256;
    }
    // LDS offset of the lane's 16 bytes of the rows from row0 (a multiple of 16) for the first instruction; ^ 64 j for the j-th.
    static __device__ __forceinline__ uint32_t fragment(int row0) {
        const int r = lane_id() & 15, g = lane_id() >> 4;
        return (row0 + r) * 256 + ((g ^ (r & 3)) << 4 | (r & 12) << 4);
    }
};

// F16: the rows are fp16, otherwise bf16.
template <WeightFormat F, int S, int BM, bool F16>
struct W4Tiles {
    static constexpr int kBM = BM, kCodes = 16;                                      // 16 rows of pieces: 256 channels
    static constexpr int NT = kCodes / kGemmWaves, kSteps = BM / 16;                 // of a wave: rows of pieces, 16-row steps
    typedef WideRows<BM> SOp;
    static constexpr int kW = SOp::kBytes, kScales = kW + kCodes * kPieceBytes, kStage = kScales + kGemmWaves * 256;
    static constexpr int kPerCu = BM == 128 ? 1 : 2;                                 // workgroups
    static constexpr int kBuffers = BM == 64 ? 2 : 3, kAhead = kBuffers - 1, kLds = kStage * kBuffers;
    static constexpr int kWCopies = kCodes / kGemmWaves, kCopies = SOp::kCopies + kWCopies + 1;      // of a stage per wave
    static constexpr int kPieceScales = 32 * S;                                      // bytes

    char* smem;
    SOp s, next_s;
    uint64_t w, next_w, scales, next_scales;
    uint32_t w_offset[kWCopies], next_w_offset[kWCopies], scale_offset, next_scale_offset;
    int next_k, k, left, buf;

    // The next tile's weights: row_piece(i) is the number of its i-th row of pieces (of 16), from `start` and `scale` on, or -1.
    template <class RowPiece>
    __device__ __forceinline__ void init_next_w(const char* start, const char* scale, int pieces, RowPiece row_piece) {
        next_w = uniform64((uint64_t)start);
        next_scales = uniform64((uint64_t)scale);
#pragma unroll
        for (int i = 0; i < kWCopies; ++i) {
            const int at = row_piece(i * kGemmWaves + wave_id());
            next_w_offset[i] = at < 0 ? kNoElement : (uint32_t)at * (uint32_t)(pieces * kPieceBytes) + lane_id() * 16;
        }
        const int byte = (int)threadIdx.x * 4, i = byte / kPieceScales, at = i < kCodes ? row_piece(i) : -1;
        next_scale_offset = at < 0 ? kNoElement : (uint32_t)at * (uint32_t)(pieces * kPieceScales) + byte % kPieceScales;
    }
    __device__ __forceinline__ void copy(int to) {
        const uint32_t lds = lds_address(smem) + to * kStage;
        s.copy(lds, left * 2);
        const uint32_t size = left > 0 ? kNoElement : 0u;
        const i32x4 rw = resource(w, size), rs = resource(scales, size);
        const uint32_t lw = __builtin_amdgcn_readfirstlane(lds + kW + threadIdx.x / kWave * kPieceBytes);
#pragma unroll
        for (int i = 0; i < kWCopies; ++i) copy16_to_lds(lw + i * kGemmWaves * kPieceBytes, w_offset[i], rw);
        copy4_to_lds(__builtin_amdgcn_readfirstlane(lds + kScales + threadIdx.x / kWave * 256), scale_offset, rs);
        w += kPieceBytes;
        scales += kPieceScales;
        left -= kPieceK;
    }
    __device__ __forceinline__ void settle() {
        s.settle();
        next_s.settle();
        w = uniform64(w);
        next_w = uniform64(next_w);
        scales = uniform64(scales);
        next_scales = uniform64(next_scales);
        asm volatile("s_nop 4" : "+s"(w), "+s"(next_w), "+s"(scales), "+s"(next_scales));
    }
    __device__ __forceinline__ void take_next() {
        s = next_s, w = next_w, scales = next_scales, left = next_k;
        scale_offset = next_scale_offset;
#pragma unroll
        for (int i = 0; i < kWCopies; ++i) w_offset[i] = next_w_offset[i];
    }
    // The workgroup's first tile, which next_* describe.
    __device__ __forceinline__ void begin(char* lds) {
        smem = lds;
        w = scales = 0;
        s = next_s;
        settle();
        take_next();
        k = next_k;
        buf = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) copy(i);
    }

    // The sums of the tile under way; afterwards the next one is.
    template <int MT>
    __device__ __forceinline__ void run(f32x4 (&acc)[NT][MT]) {
        const int wave = wave_id(), lane = lane_id();
        const int stages = __builtin_amdgcn_readfirstlane(k > kAhead * kPieceK ? pieces_of(k) : kAhead);      // enough that one tile ahead will do
        left = __builtin_amdgcn_readfirstlane(left);
        next_k = __builtin_amdgcn_readfirstlane(next_k);
        buf = __builtin_amdgcn_readfirstlane(buf);
        settle();
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
            for (int a = 0; a < MT; ++a) acc[b][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t s_at = SOp::fragment(0);
        for (int st = 0; st < stages; ++st) {
            if (st == stages - kAhead) {
                stay_branch();
                take_next();
            }
            // this stage has landed, and every wave has left the one before, whose buffer the copies go to
            wait_and_meet<(kBuffers - 2) * kCopies>();
            copy(buf == 0 ? kBuffers - 1 : buf - 1);
            const char* ls = smem + buf * kStage;
            const char* lw = ls + kW + wave * NT * kPieceBytes + lane * 16;
            const char* lc = ls + kScales + wave * NT * kPieceScales + (lane & 15) * (2 * S);
            i32x4 code[NT];
            GroupScales<S> scale[NT];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                code[b] = *reinterpret_cast<const i32x4*>(lw + b * kPieceBytes);
                scale[b].load(lc + b * kPieceScales);
            }
            constexpr int kPer = 4 / S;
#pragma unroll
            for (int grp = 0; grp < S; ++grp) {
                f32x4 part[NT][MT];
                // the wave that multiplies goes first, while another of its SIMD scales: 2 to 3% (4096 tokens 3.38 and 3.28 ms)
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int j = grp * kPer; j < (grp + 1) * kPer; ++j) {
                    bf16x8 sv[MT];
#pragma unroll
                    for (int a = 0; a < MT; ++a) sv[a] = read_kc(ls, (s_at ^ (j * 64)) + a * 4096);
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        if constexpr (F16) {
                            const f16x8 fv = widen_codes16<F == kWeightsInt4>((uint32_t)code[b][j]);
#pragma unroll
                            for (int a = 0; a < MT; ++a)
                                part[b][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, sv[a]), fv, j == grp * kPer ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : part[b][a], 0, 0, 0);
                        } else {
                            const bf16x8 fv = widen_codes<F == kWeightsInt4>((uint32_t)code[b][j]);
#pragma unroll
                            for (int a = 0; a < MT; ++a)
                                part[b][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(sv[a], fv, j == grp * kPer ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : part[b][a], 0, 0, 0);
                        }
                    }
                }
                __builtin_amdgcn_s_setprio(0);
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    const float by = scale[b].get(grp);
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][a][i] = fmaf(part[b][a][i], by, acc[b][a][i]);
                }
            }
            buf = buf == kBuffers - 1 ? 0 : buf + 1;
        }
        k = next_k;
    }

    // No copy may land after the workgroup has left its LDS.
    static __device__ __forceinline__ void end() { wait_and_meet<0>(); }
};

// UP: half of a wave's rows of pieces are gate channels, half the same up channels, and h = silu(g) u is stored.
template <WeightFormat F, int S, int BM, bool UP>
struct Kernel {
    typedef W4Tiles<F, S, BM, !UP> Tiles;
    static constexpr int NT = Tiles::NT, kOut = UP ? NT / 2 : NT;            // rows of pieces that a wave stores
    static constexpr int kCols = kGemmWaves * kOut * 16;
    static constexpr float kValue = Weights<F, S>::kUnit;

    const Params& p;
    RowTiles<BM, 0> rows;
    Tiles g;
    int round = 0;
    struct Target {
        int64_t row0;
        int rows, n0;
    } now, next;

    __device__ __forceinline__ explicit Kernel(const Params& params) : p(params), rows(params.cnt, params.psum, params.El) {}

    __device__ __forceinline__ void look_ahead() {
        TileAt at;
        next.rows = g.next_k = 0;
        if (!tile_at<kBatch * Tiles::kPerCu>((int)blockIdx.x, round++, rows.total, (p.N + kCols - 1) / kCols, &at)) return;
        const RowTile t = rows.find(at.row, 16);
        const int n0 = at.col * kCols, pieces = pieces_of(p.K);
        next = Target{t.row0, t.rows, n0};
        g.next_k = p.K;
        g.next_s.init(p.s + (int64_t)t.row0 * p.sp, [&](int r) { return r < t.rows ? r * (2u * p.sp) : kNoElement; });
        const int64_t piece = ((int64_t)t.expert * (p.w.N / kPieceRows) + n0 / kPieceRows) * pieces;
        g.init_next_w(p.w.values + piece * kPieceBytes, p.w.scales + piece * (32 * S), pieces, [&](int i) {
            const int b = i % NT, c = (i / NT * kOut + b % kOut) * 16;
            return n0 + c < p.N ? (c + b / kOut * p.N) / kPieceRows : -1;
        });
    }

    // A lane has 4 rows of one channel; two neighbours swap, so that each has 2 rows of 2 channels: the even one the first two.
    static __device__ __forceinline__ void swap_rows(const float (&v)[4], int odd, float (&x)[4]) {
        const float x0 = dpp_f<0xB1>(odd ? v[0] : v[2]), x1 = dpp_f<0xB1>(odd ? v[1] : v[3]);
        x[0] = odd ? x0 : v[0], x[1] = odd ? v[2] : x0;
        x[2] = odd ? x1 : v[1], x[3] = odd ? v[3] : x1;
    }

    template <int MT>
    __device__ __forceinline__ void tile() {
        f32x4 acc[NT][MT];
        g.template run<MT>(acc);
        // the units of the rows of h, one or two a lane
        constexpr int kUnits = UP ? 1 : (MT * 16 + kWave - 1) / kWave;
        float units[kUnits];
        if constexpr (!UP)
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int m = i * kWave + lane_id();
                units[i] = m < now.rows ? *row_unit(const_cast<uint16_t*>(p.s) + (now.row0 + m) * p.sp, p.K) : 0.0f;
            }
        const int wave = wave_id(), r = lane_id() & 15, odd = r & 1;
        int m_at = (lane_id() >> 4) * 4 + odd * 2;
        asm("" : "+v"(m_at));      // not to be looked into: all rows' addresses in registers (20 more) would slow the tile down by 2%
#pragma unroll
        for (int b = 0; b < kOut; ++b) {
            const int n = now.n0 + (wave * kOut + b) * 16 + (r & ~1);
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = acc[b][a][i] * kValue;
                    if constexpr (UP) v[i] = v[i] * sigmoid(v[i]) * (acc[b + kOut][a][i] * kValue);
                }
                const int m = m_at + a * 16;
                uint16_t* out = p.out + (now.row0 + m) * p.op;
                float x[4];
                uint32_t first, second;
                if constexpr (UP) {
                    // a wave's 16 channels are a block, which 16 neighbouring lanes have; one of them for each row stores its number
                    int e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        e[i] = block_number(max_bits<16>(size_bits(v[i])));
                        v[i] = shared_value(v[i], e[i]);
                    }
                    const int row = m_at - odd * 2 + a * 16 + r;
                    if (r < 4 && row < now.rows && n < p.N)
                        p.out[(now.row0 + row) * p.op + p.N + now.n0 / kShared + wave] = (uint16_t)(r == 0 ? e[0] : r == 1 ? e[1] : r == 2 ? e[2] : e[3]);
                    swap_rows(v, odd, x);
                    first = pack_f16x2(x[0], x[1]);
                    second = pack_f16x2(x[2], x[3]);
                } else {
                    const float u0 = __shfl(units[a / 4], m & 63), u1 = __shfl(units[a / 4], (m + 1) & 63);
                    swap_rows(v, odd, x);
                    first = pack_bf16x2(x[0] * u0, x[1] * u0);
                    second = pack_bf16x2(x[2] * u1, x[3] * u1);
                }
                if (n < p.N && m < now.rows) *reinterpret_cast<uint32_t*>(out + n) = first;
                if (n < p.N && m + 1 < now.rows) *reinterpret_cast<uint32_t*>(out + p.op + n) = second;
                __builtin_amdgcn_sched_barrier(0);      // one step's after another's, for the registers
            }
        }
    }
};

template <WeightFormat F, int S, int BM, bool UP>
__global__ __launch_bounds__(kGemmThreads, BM == 128 ? 2 : 4) void k_w4_tiles(Params p) {
    typedef Kernel<F, S, BM, UP> K;
    extern __shared__ __align__(1024) char smem[];
    K k(p);
    k.look_ahead();
    if (k.next.rows == 0) return;
    k.g.begin(smem);
    do {
        k.now = k.next;
        k.look_ahead();
        const int steps = (k.now.rows + 15) / 16;
        constexpr int kSteps = K::Tiles::kSteps;
        if constexpr (kSteps == 8) {
            if (steps <= 2) k.template tile<2>();
            else if (steps <= 4) k.template tile<4>();
            else if (steps <= 6) k.template tile<6>();
            else k.template tile<8>();
        } else {
            if (steps == 1) k.template tile<1>();
            else if (kSteps == 2 || steps == 2) k.template tile<2>();
            else if (steps == 3) k.template tile<(kSteps < 3 ? 2 : 3)>();
            else k.template tile<(kSteps < 4 ? 2 : 4)>();
        }
    } while (k.next.rows > 0);
    k.g.end();
}

template <WeightFormat F, int S, int BM, bool UP>
hipError_t tiles_launch(const Handle& h, const Params& p, hipStream_t stream) {
    typedef Kernel<F, S, BM, UP> K;
    // row tiles that any routing can give: every expert may end in a short one
    const int64_t rows = (int64_t)h.T * h.K / BM + h.El;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_w4_tiles<F, S, BM, UP>), K::Tiles::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_w4_tiles<F, S, BM, UP>), dim3(walking_blocks(rows * ((p.N + K::kCols - 1) / K::kCols), kBatch * K::Tiles::kPerCu)), dim3(kGemmThreads), K::Tiles::kLds,
                       stream, p);
    return hipGetLastError();
}

template <WeightFormat F, int S, bool UP>
hipError_t by_height(const Handle& h, const Params& p, W4Kernel kernel, hipStream_t stream) {
    if (kernel == kW4Tile32) return tiles_launch<F, S, 32, UP>(h, p, stream);
    if (kernel == kW4Tile64) return tiles_launch<F, S, 64, UP>(h, p, stream);
    return tiles_launch<F, S, 128, UP>(h, p, stream);
}

template <WeightFormat F, bool UP>
hipError_t by_group(const Handle& h, const Params& p, int group, W4Kernel kernel, hipStream_t stream) {
    if (group == 128) return by_height<F, 1, UP>(h, p, kernel, stream);
    if (group == 64) return by_height<F, 2, UP>(h, p, kernel, stream);
    return by_height<F, 4, UP>(h, p, kernel, stream);
}

}  // namespace

hipError_t launch_w4_tile_up(const Handle& h, const W4Args& a, W4Kernel kernel, hipStream_t stream) {
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, (const uint16_t*)a.x, WeightArgs{(const char*)a.w13.values, (const char*)a.w13.scales, 2 * a.inter, a.hidden},
                   a.h, a.inter, a.hidden, a.hidden, h_pitch(a.inter)};
    return a.int4 ? by_group<kWeightsInt4, true>(h, p, a.group, kernel, stream) : by_group<kWeightsE2m1, true>(h, p, a.group, kernel, stream);
}

hipError_t launch_w4_tile_down(const Handle& h, const W4Args& a, W4Kernel kernel, hipStream_t stream) {
    // row tiles that any routing can give
    const int64_t entries = (int64_t)h.T * h.K, busy = entries < h.El ? entries : h.El;
    hipLaunchKernelGGL(k_one_number, grid_of((entries + (kUnitRows - 1) * busy) / kUnitRows), dim3(kUnitRows * kWave), 0, stream, h.ws.cnt_local, h.ws.psum,
                       h.El, a.h, a.inter);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const Params p{h.ws.cnt_local, h.ws.psum, h.El, a.h, WeightArgs{(const char*)a.w2.values, (const char*)a.w2.scales, a.hidden, a.inter},
                   (uint16_t*)a.y, a.hidden, a.inter, h_pitch(a.inter), a.hidden};
    return a.int4 ? by_group<kWeightsInt4, false>(h, p, a.group, kernel, stream) : by_group<kWeightsE2m1, false>(h, p, a.group, kernel, stream);
}

}  // namespace ep
