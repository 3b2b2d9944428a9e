// ep_few.hip -- a whole mixture-of-experts layer for a few tokens, in two kernels: from tokens and routing to tokens.
//
//   k_few_up     h[t,k] = silu(g) u,  g | u = x[t] W13_e^T           one workgroup: rows of one expert x 16 * NF / 2 channels of I
//   k_few_down   out[t] = sum_k w[t,k] h[t,k] W2_e^T + bias[t]       one workgroup: all experts in use x 16 or 32 channels of H
//
// No layout, dispatch or combine runs before or between: every workgroup finds the experts in use and their entries from the
// routing table itself (items: up to 16 * MT entries of one expert).  Both are bound by reading the weights of the experts in
// use, once each.  In the second the waves take items in turn, and each entry's values of the channels stand in LDS until they
// are weighted and summed in ascending k, so that nothing depends on the order in which waves finish.
//
// Measured: 32 tokens, 256 e4m3 experts of 7168 x 2048, top-8 (7.2 GB): 808 us (6.0 TB/s) and 465 (5.2 TB/s; 224 workgroups on 256
// CUs).  One token, int4: 24 and 16.5 us (5.0 and 3.7 TB/s).  61 tokens on 32 e2m1 experts in groups of 32, uneven: 128 and 98 us
// (4.1 and 2.7 TB/s): with some 16 rows beside a piece of 1 KiB the rows' 4 KiB from L2 bound it, not the weights.
// Splitting all items' pieces evenly over the waves of the second kernel gained nothing (227 and 231 us in all, 1262 and 1271).
#include "ep_few_rules.hpp"
#include "ep_ffn.hpp"
#include "ep_stream.hpp"

namespace ep {
namespace {

constexpr int kDownWaves = kFewWaves, kDownThreads = kDownWaves * kWave;

struct Params {
    const uint16_t* x;        // [T, H]
    const int64_t* idx;       // [T, K]
    const float* topk_w;      // [T, K] or nullptr
    const uint16_t* bias;
    WeightArgs w13, w2;       // [El, 2 I, H], [El, H, I]
    uint16_t* h;              // workspace [T * K, h_pitch(I)] (ep_h_rows.hpp), or [T * K, row_pitch(I)] where entries stand by themselves
    uint16_t* out;            // [T, H]
    int T, K, H, I, lo, El;
};

// The local expert of an entry, or -1.
__device__ __forceinline__ int local_expert(const Params& p, int entry) {
    const int64_t id = p.idx[entry];
    return id >= p.lo && id < (int64_t)p.lo + p.El ? (int)(id - p.lo) : -1;
}

// The items of a call, in LDS.  Of entries t * K + k with a local expert, those of one expert in groups of up to GROUP.
struct Items {
    int* expert;          // [items]
    int* first;           // [items] place of its first entry in `order` (ALL, or up to one wave's entries), or among its expert's
    int* count;           // [items]
    int* cursor;          // [El] (many entries)
    uint16_t* order;
    int total;
    float* weight;        // [entries] (ALL): the routing weights, and which entries there are, a bit each
    uint64_t* valid;
};
struct ItemsLayout {
    int items, order, cursor, weights;      // sizes
    int bytes() const { return (3 * items + cursor + 4) * 4 + (weights + 63) / 64 * (64 * 4 + 8) + order * 2; }
};
// Up to one wave's entries: every item has GROUP places in order.  Of more, all entries stand there, or one item's.
inline ItemsLayout items_layout(int entries, int El, int group, bool all) {
    const int busy = entries < El ? entries : El;
    const int items = (int)((entries + (int64_t)(group - 1) * busy) / group);
    const int weights = all ? entries : 0;
    if (entries <= kWave) return ItemsLayout{items, items * group, 0, weights};
    return ItemsLayout{items, all ? entries : group, El, weights};
}

// Items are the same in every workgroup.  ALL: all of them are wanted, and the order of an expert's entries is whatever it is: a
// row's values do not depend on the rows beside it.  Otherwise item `wanted` is, and as other workgroups take its other channels,
// its entries are the same everywhere: by their place among the expert's in the routing table.
template <int GROUP, int THREADS, bool ALL>
__device__ __forceinline__ Items find_items(const Params& p, char* lds, int max_items, int cursors, int wanted) {
    Items it;
    int* at = reinterpret_cast<int*>(lds);
    int* total = at;
    const int n = p.T * p.K, lane = lane_id(), chunks = ALL ? (n + kWave - 1) / kWave : 0;
    it.valid = reinterpret_cast<uint64_t*>(at + 4);
    it.weight = reinterpret_cast<float*>(it.valid + chunks);
    it.expert = reinterpret_cast<int*>(it.weight + chunks * kWave);
    it.first = it.expert + max_items;
    it.count = it.first + max_items;
    it.cursor = it.count + max_items;
    it.order = reinterpret_cast<uint16_t*>(it.cursor + cursors);
    if constexpr (ALL)
        for (int i = threadIdx.x; i < n; i += THREADS) it.weight[i] = p.topk_w ? p.topk_w[i] : 1.0f;
    if (n <= kWave) {
        // every wave works it out in its registers; the first leaves it in LDS
        const int id = lane < n ? local_expert(p, lane) : -1, e = id < 0 ? 0 : id;
        const bool in = id >= 0;
        const uint64_t peers = match_peers(e, in, 10);
        const int rank = popc64(peers & lanemask_lt());
        const uint64_t heads = ballot(in && rank % GROUP == 0);
        // an entry's item is that of the last head among its peers up to itself
        const uint64_t mine = peers & heads & (lanemask_lt() | (1ull << lane));
        const int head = mine ? 63 - __builtin_clzll(mine) : 0, item = popc64(heads & ((1ull << head) - 1));
        const uint64_t valid = ballot(in);
        if (ALL && threadIdx.x == 0) it.valid[0] = valid;
        if ((int)threadIdx.x < kWave && in) {
            if (head == lane) {
                const int after = popc64(peers) - rank;
                it.expert[item] = e;
                it.first[item] = item * GROUP;
                it.count[item] = after < GROUP ? after : GROUP;
            }
            it.order[item * GROUP + rank % GROUP] = (uint16_t)lane;
        }
        it.total = popc64(heads);      // (uniform, a ballot)
        __syncthreads();
        return it;
    }
    for (int e = threadIdx.x; e < p.El; e += THREADS) it.cursor[e] = 0;
    __syncthreads();
    constexpr int kPer = (kFewEntries + THREADS - 1) / THREADS;
    __shared__ int chunk[ALL ? 1 : kFewEntries / kWave];
    int mine[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int entry = i * THREADS + threadIdx.x;
        mine[i] = entry < n ? local_expert(p, entry) : -1;
        if (mine[i] >= 0) atomicAdd(&it.cursor[mine[i]], 1);
        const uint64_t valid = ballot(mine[i] >= 0);
        if (ALL && lane == 0 && entry < n) it.valid[entry / kWave] = valid;
    }
    __syncthreads();
    if (threadIdx.x < kWave) {
        int items = 0, entries = 0;
        for (int e0 = 0; e0 < p.El; e0 += kWave) {
            const int e = e0 + lane, c = e < p.El ? it.cursor[e] : 0, groups = (c + GROUP - 1) / GROUP;
            const int place = entries + wave_inclusive_scan(c) - c, item = items + wave_inclusive_scan(groups) - groups;
            for (int i = 0; i < groups; ++i) {
                it.expert[item + i] = e;
                it.first[item + i] = (ALL ? place : 0) + i * GROUP;
                it.count[item + i] = c - i * GROUP < GROUP ? c - i * GROUP : GROUP;
            }
            if (e < p.El) it.cursor[e] = place;
            entries = readlane(place + c, kWave - 1);
            items = readlane(item + groups, kWave - 1);
        }
        if (lane == 0) *total = items;
    }
    __syncthreads();
    if constexpr (ALL) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (mine[i] >= 0) it.order[atomicAdd(&it.cursor[mine[i]], 1)] = (uint16_t)(i * THREADS + threadIdx.x);
        __syncthreads();
    } else if (wanted < *total) {
        // entries of the expert in each 64, then an entry's place among them (the cursors are not needed any more)
        const int e = it.expert[wanted], first = it.first[wanted], wave = wave_id();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint64_t there = ballot(mine[i] == e);
            if (lane == 0) chunk[i * (THREADS / kWave) + wave] = popc64(there);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint64_t there = ballot(mine[i] == e);
            if (!there) continue;
            int place = popc64(there & lanemask_lt()) - first;
            for (int c = 0; c < i * (THREADS / kWave) + wave; ++c) place += chunk[c];
            if (mine[i] == e && place >= 0 && place < GROUP) it.order[place] = (uint16_t)(i * THREADS + threadIdx.x);
        }
        __syncthreads();
        it.first[wanted] = 0;      // every thread, after all have read it
    }
    it.total = __builtin_amdgcn_readfirstlane(*total);
    return it;
}

// A workgroup's rows are an item's entries, its channels 16 * NF / 2 of I.
template <class W, int MT, int NF>
__global__ __launch_bounds__(kStreamThreads, MT == 4 ? 2 : 4) void k_few_up(Params p, int max_items, int cursors, int lists, int cols) {
    extern __shared__ __align__(16) char smem[];
    const int item = blockIdx.x / cols, n0 = blockIdx.x % cols * (NF * 8);
    const Items it = find_items<16 * MT, kStreamThreads, false>(p, smem, max_items, cursors, item);
    if (item >= it.total) return;
    const int first = it.first[item], count = it.count[item], r = lane_id() & 15;
    RowFragments<W, MT, false> rows;
    rows.init(p.x, p.H);
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const bool there = a * 16 + r < count;
        rows.place(a, there, (uint32_t)(it.order[first + (there ? a * 16 + r : 0)] / p.K) * (uint32_t)(p.H * 2));
    }
    stream_product<W, true, MT, NF>(p.w13, __builtin_amdgcn_readfirstlane(it.expert[item]), p.I, p.H, n0, rows, count, reinterpret_cast<float*>(smem + lists),
                                       [&](int m) { return p.h + (int64_t)it.order[first + m] * h_pitch(p.I); });
}

// Items (and, of few items, parts of their k) go to the waves in turn; parts is a power of two.
template <class W, int MT, int NF>
__global__ __launch_bounds__(kDownThreads) void k_few_down(Params p, int max_items, int cursors, int lists, int max_values) {
    extern __shared__ __align__(16) char smem[];
    const Items it = find_items<16 * MT, kDownThreads, true>(p, smem, max_items, cursors, 0);
    constexpr int kCols = NF * 16;
    float* values = reinterpret_cast<float*>(smem + lists);       // [parts][T * K][kCols]
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4, n0 = blockIdx.x * kCols, n = p.T * p.K;
    const int pieces = pieces_of(p.I);
    int log_parts = 0;
    while ((it.total << (log_parts + 1)) <= kDownWaves && (2 << log_parts) <= pieces && (n << (log_parts + 1)) <= max_values) ++log_parts;
    const int parts = 1 << log_parts, work = it.total << log_parts;
    for (int i = wave; i < work; i += kDownWaves) {
        const int item = i >> log_parts, part = i & (parts - 1);
        const int expert = __builtin_amdgcn_readfirstlane(it.expert[item]), first = it.first[item], count = it.count[item];
        RowFragments<W, MT, true> rows;
        rows.init(p.h, p.I);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const bool there = a * 16 + r < count;
            rows.place(a, there, (uint32_t)it.order[first + (there ? a * 16 + r : 0)] * (uint32_t)(h_pitch(p.I) * 2));
        }
        typename W::template Rows<NF> w;
        w.init(p.w2, expert, n0);
        f32x4 acc[NF][MT];
#pragma unroll
        for (int b = 0; b < NF; ++b) {
            const int exist = p.H - n0 - b * 16;
            w.place(b, exist > 0 ? b * 16 : 0, exist);
#pragma unroll
            for (int a = 0; a < MT; ++a) acc[b][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        stream_pieces(w, rows, part, parts, pieces, acc);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = a * 16 + g * 4 + j;
                const float unit = rows.unit(a, j);
                if (m >= count) continue;
                float* to = values + (part * n + it.order[first + m]) * kCols + r;
#pragma unroll
                for (int b = 0; b < NF; ++b) to[b * 16] = acc[b][a][j] * unit;
            }
    }
    __syncthreads();
    constexpr int kQuads = kCols / 4;
    for (int i = threadIdx.x; i < p.T * kQuads; i += kDownThreads) {
        const int t = i / kQuads, in = i % kQuads * 4, c = n0 + in;
        if (c >= p.H) continue;
        f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < p.K; ++k) {
            const int e = t * p.K + k;
            if (!(it.valid[e / kWave] >> (e % kWave) & 1)) continue;
            f32x4 v = *reinterpret_cast<const f32x4*>(values + e * kCols + in);
            for (int q = 1; q < parts; ++q) v += *reinterpret_cast<const f32x4*>(values + (q * n + e) * kCols + in);
            const float weight = W::kUnit * it.weight[e];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = fmaf(weight, v[j], sum[j]);
        }
        if (p.bias) {
            const uint16_t* b = p.bias + (int64_t)t * p.H + c;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += __builtin_bit_cast(float, (uint32_t)b[j] << 16);
        }
        store4(p.out + (int64_t)t * p.H + c, sum[0], sum[1], sum[2], sum[3]);
    }
}

template <class W, int MT, int NF>
hipError_t launch_up(const Params& p, hipStream_t stream) {
    const ItemsLayout l = items_layout(p.T * p.K, p.El, 16 * MT, false);
    const int lists = (l.bytes() + 15) & ~15, lds = lists + stream_lds<NF>(), cols = (p.I + NF * 8 - 1) / (NF * 8);
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_few_up<W, MT, NF>), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_up<W, MT, NF>), dim3((unsigned)(l.items * cols)), dim3(kStreamThreads), lds, stream, p, l.items, l.cursor, lists, cols);
    return hipGetLastError();
}

template <class W, int MT, int NF>
hipError_t launch_down(const Params& p, hipStream_t stream) {
    const int n = p.T * p.K;
    const ItemsLayout l = items_layout(n, p.El, 16 * MT, true);
    // room for the parts of few items' entries
    const int lists = (l.bytes() + 15) & ~15, values = n > 8 * 16 ? n : 8 * (n < 16 ? n : 16), lds = lists + values * NF * 64;
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_few_down<W, MT, NF>), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_down<W, MT, NF>), dim3((p.H + NF * 16 - 1) / (NF * 16)), dim3(kDownThreads), lds, stream, p, l.items, l.cursor, lists, values);
    return hipGetLastError();
}

// ---- one token, or up to 16 entries on enough experts ---------------------------------------------------------------
//
// An entry is an item of its own: its expert is one load away, so the weights are under way a microsecond into the kernel, and
// most of a wave's share of them at once.  (An expert that two entries share is read twice, the second time from a cache;
// few_by_entry says when that pays.)
//
// Every row of the instruction's first operand is the entry's, so half of them can be second parts, at no cost.  h takes 16 bits in
// the workspace: fp16 as in ep_h_rows.hpp, but of eight channels, whose number E = 16 n + 4 (or 0, and n = 0) stands in the lowest bits of
// the first five, bit i of n in the i-th; these keep a bit less (all but 2^-10 of a value, or 2^-22 of the largest of the eight).  The eight are
// taken to fp32 and apart into two bf16, each by its number.
constexpr int kNumberBits = 5;

// Channel c of the lanes' eight; all of them call it.
__device__ __forceinline__ uint16_t value_and_bit(float v, int c) {
    const int e = block_number(max_bits<8>(size_bits(v)));
    uint32_t q = __builtin_bit_cast(uint16_t, (_Float16)shared_value(v, e));
    if ((c & 7) < kNumberBits) {
        q += q & q >> 1 & 1u;      // to the nearest without the last bit, or from the middle to the even one (an infinity's is 0)
        q = (q & ~1u) | ((uint32_t)e >> (4 + (c & 7)) & 1u);
    }
    return (uint16_t)q;
}
// Eight channels' two parts.
__device__ __forceinline__ void two_parts(i32x4 q, i32x4* first, i32x4* second) {
    const uint32_t n = (uint32_t)((q[0] & 1) | (q[0] >> 15 & 2) | (q[1] & 1) << 2 | (q[1] >> 13 & 8) | (q[2] & 1) << 4);
    q[0] &= ~0x10001, q[1] &= ~0x10001, q[2] &= ~1;
    const int by = (int)n * 16 + 4 - 154;
    const bool large = ballot(n == 17) != 0;      // an infinity or NaN among them, perhaps
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const f16x2 v = __builtin_bit_cast(f16x2, (int)q[d]);
        const float a = ldexpf((float)v[0], by), b = ldexpf((float)v[1], by);
        (*first)[d] = upper_halves(a, b);
        // (11 bits: what the first part leaves is exact in its upper half)
        (*second)[d] = large ? upper_halves(rest_of(a), rest_of(b)) : upper_halves(a - upper_half(a), b - upper_half(b));
    }
}

// acc[NF] += pieces first, first + step, ... below `end` of NF rows of pieces by one row x of K channels; the wave's part of it stands
// in LDS, up to `room` pieces at a time.  PARTS 1: bf16, and every row of the instruction's first operand is x.  PARTS 2: as
// value_and_bit leaves them, and even rows are first parts, odd ones second.
template <class W, int PARTS, int NF>
__device__ __forceinline__ void one_row(const typename W::template Rows<NF>& w, const uint16_t* x, int K, int first, int step, int end,
                                        char* lds, int room, f32x4 (&acc)[NF][1]) {
    Buffer row;
    row.init(x);
    const int count = (end - first + step - 1) / step, lane = lane_id();
    typename W::Raw raw[NF];
    auto load = [&](int i) {
#pragma unroll
        for (int b = 0; b < NF; ++b) raw[b] = w.load(b, first + i * step, i < count);
    };
    for (int i0 = 0; i0 < count; i0 += room) {
        const int n = count - i0 < room ? count - i0 : room;
        for (int c = lane; c < n * 16; c += kWave) {      // 16 bytes
            const int k = (first + (i0 + c / 16) * step) * kPieceK + c % 16 * 8;
            const i32x4 q = load16(row.resource(true), k < K ? (uint32_t)k * 2 : kNoElement, 0);
            i32x4* to = reinterpret_cast<i32x4*>(lds + c * 16);
            if constexpr (PARTS == 1) *to = q;
            else two_parts(q, to, to + room * 16);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (i0 == 0) load(0);
        const char* at = lds + W::k_of(0, lane >> 4) * 2 + (PARTS == 2 && (lane & 1) ? room * (kPieceK * 2) : 0);
        for (int i = i0; i < i0 + n; ++i, at += kPieceK * 2) {
            i32x4 v[1][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[0][j] = *reinterpret_cast<const i32x4*>(at + W::k_of(j, 0) * 2);
            add_pieces<W, false>(raw, v, acc);
            load(i + 1);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");      // before the next of them come
        __builtin_amdgcn_wave_barrier();
    }
}

template <class W, int NF>
__global__ __launch_bounds__(kStreamThreads, 4) void k_one_up(Params p, int cols, int per_wave) {
    constexpr int kHalf = NF * 8;
    extern __shared__ __align__(16) char smem[];      // [waves][NF * 16] sums, then each wave's part of x
    const int entry = blockIdx.x / cols, n0 = blockIdx.x % cols * kHalf, wave = wave_id();
    const int expert = __builtin_amdgcn_readfirstlane(local_expert(p, entry));
    if (expert < 0) return;
    typename W::template Rows<NF> w;
    w.init(p.w13, expert, n0);
    f32x4 acc[NF][1];
#pragma unroll
    for (int b = 0; b < NF; ++b) {
        const int n = b % (NF / 2) * 16, exist = p.I - n0 - n;
        w.place(b, (exist > 0 ? n : 0) + b / (NF / 2) * p.I, exist);
        acc[b][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    float* sums = reinterpret_cast<float*>(smem);
    char* mine = smem + kStreamWaves * NF * 64 + wave * per_wave * (kPieceK * 2);
    if (wave < pieces_of(p.H)) one_row<W, 1, NF>(w, p.x + (int64_t)(entry / p.K) * p.H, p.H, wave, kStreamWaves, pieces_of(p.H), mine, per_wave, acc);
    if (lane_id() < 16) {
#pragma unroll
        for (int b = 0; b < NF; ++b) sums[wave * NF * 16 + b * 16 + lane_id()] = acc[b][0][0];
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= kHalf || n0 + c >= p.I) return;
    float gate = 0.0f, up = 0.0f;
#pragma unroll
    for (int v = 0; v < kStreamWaves; ++v) {
        gate += sums[v * NF * 16 + c];
        up += sums[v * NF * 16 + kHalf + c];
    }
    gate *= W::kUnit;
    p.h[(int64_t)entry * row_pitch(p.I) + n0 + c] = value_and_bit(gate * sigmoid(gate) * (up * W::kUnit), c);
}

// Waves take parts of entries in turn, i % parts of i / parts, `room` pieces of them at a time.
template <class W, int NF>
__global__ __launch_bounds__(kDownThreads) void k_one_down(Params p, int parts, int room) {
    constexpr int kCols = NF * 16;
    extern __shared__ __align__(16) char smem[];      // [entries][parts][kCols] sums, then each wave's part of h
    __shared__ float weight[kMaxTopk];
    __shared__ int valid[kMaxTopk];
    const int n0 = blockIdx.x * kCols, wave = wave_id(), n = p.T * p.K;
    float* sums = reinterpret_cast<float*>(smem);
    // what the sum over k needs, asked for before the weights
    const int t = threadIdx.x / kCols, c = threadIdx.x % kCols;
    const bool mine_out = t < p.T && n0 + c < p.H;
    const int64_t at = (int64_t)t * p.H + n0 + c;
    const float bias = mine_out && p.bias ? __builtin_bit_cast(float, (uint32_t)p.bias[at] << 16) : 0.0f;
    if ((int)threadIdx.x < n) {
        valid[threadIdx.x] = local_expert(p, threadIdx.x) >= 0;
        weight[threadIdx.x] = W::kUnit * (p.topk_w ? p.topk_w[threadIdx.x] : 1.0f);
    }
    for (int i = wave; i < n * parts; i += kDownWaves) {
        const int entry = i / parts, part = i % parts, expert = __builtin_amdgcn_readfirstlane(local_expert(p, entry));
        if (expert < 0) continue;
        typename W::template Rows<NF> w;
        w.init(p.w2, expert, n0);
        f32x4 acc[NF][1];
#pragma unroll
        for (int b = 0; b < NF; ++b) {
            const int exist = p.H - n0 - b * 16;
            w.place(b, exist > 0 ? b * 16 : 0, exist);
            acc[b][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        char* mine = smem + n * parts * kCols * 4 + wave * room * (kPieceK * 4);
        one_row<W, 2, NF>(w, p.h + (int64_t)entry * row_pitch(p.I), p.I, part, parts, pieces_of(p.I), mine, room, acc);
        if (lane_id() < 16) {
#pragma unroll
            for (int b = 0; b < NF; ++b) sums[i * kCols + b * 16 + lane_id()] = acc[b][0][0] + acc[b][0][1];
        }
    }
    __syncthreads();
    if (!mine_out) return;
    float y = 0.0f;
    for (int k = 0; k < p.K; ++k) {
        const int e = t * p.K + k;
        if (!valid[e]) continue;
        float v = 0.0f;
        for (int q = 0; q < parts; ++q) v += sums[(e * parts + q) * kCols + c];
        y = fmaf(weight[e], v, y);
    }
    p.out[at] = __builtin_bit_cast(uint16_t, (__bf16)(y + bias));
}

// Parts of an entry's pieces, one at least, and how many of them a wave has in LDS: up to 16, 128 KB of a workgroup's.
struct OneParts {
    int parts, room;
    OneParts(int entries, int I) {
        const int pieces = pieces_of(I), most = entries < kDownWaves ? kDownWaves / entries : 1;
        parts = most < pieces ? most : pieces;
        room = (pieces + parts - 1) / parts;
        room = room < 16 ? room : 16;
    }
    int lds(int entries, int NF) const { return entries * parts * NF * 64 + kDownWaves * room * (kPieceK * 4); }
};

template <class W, int NF>
hipError_t launch_one_down(const Params& p, hipStream_t stream) {
    const int n = p.T * p.K;
    const OneParts o(n, p.I);
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_one_down<W, NF>), o.lds(n, NF));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_one_down<W, NF>), dim3((p.H + NF * 16 - 1) / (NF * 16)), dim3(kDownThreads), o.lds(n, NF), stream, p, o.parts, o.room);
    return hipGetLastError();
}

template <class W, int NF>
hipError_t launch_one(const Params& p, hipStream_t stream) {
    const int n = p.T * p.K, cols = (p.I + NF * 8 - 1) / (NF * 8), per_wave = (pieces_of(p.H) + kStreamWaves - 1) / kStreamWaves;
    const int up_lds = kStreamWaves * (NF * 64 + per_wave * (kPieceK * 2));
    hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_one_up<W, NF>), up_lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_one_up<W, NF>), dim3((unsigned)(n * cols)), dim3(kStreamThreads), up_lds, stream, p, cols, per_wave);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return few_narrow(p.H) ? launch_one_down<W, 1>(p, stream) : launch_one_down<W, 2>(p, stream);
}

template <class W, int NF>
hipError_t by_rows(const Params& p, int E, hipStream_t stream) {
    if (few_by_entry(p.T, p.K, E)) return launch_one<W, NF>(p, stream);
    const double rows = few_rows(p.T, p.K, E);
    const int up = few_up_steps(rows), down = few_down_steps(rows);
    const hipError_t e = up == 1 ? launch_up<W, 1, NF>(p, stream) : up == 2 ? launch_up<W, 2, NF>(p, stream) : launch_up<W, 4, NF>(p, stream);
    if (e != hipSuccess) return e;
    if (few_narrow(p.H)) return down == 1 ? launch_down<W, 1, 1>(p, stream) : launch_down<W, 2, 1>(p, stream);
    return down == 1 ? launch_down<W, 1, 2>(p, stream) : launch_down<W, 2, 2>(p, stream);
}

template <WeightFormat F>
hipError_t by_group(const Params& p, int E, int group, hipStream_t stream) {
    if (group == 128) return by_rows<Weights<F, 1>, 4>(p, E, stream);
    if (group == 64) return by_rows<Weights<F, 2>, 4>(p, E, stream);
    return by_rows<Weights<F, 4>, 4>(p, E, stream);
}

}  // namespace

// (one token's entries stand by themselves)
size_t few_workspace_bytes(int T, int K, int inter) {
    return (size_t)(T * K > 0 ? T * K : 1) * (T > 1 ? h_pitch(inter) : row_pitch(inter)) * sizeof(uint16_t);
}

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int El = a.E / a.R;
    const Params p{(const uint16_t*)a.x, a.topk_idx, a.topk_weights, (const uint16_t*)a.bias,
                   WeightArgs{(const char*)a.w13.values, (const char*)a.w13.scales, 2 * a.inter, a.hidden},
                   WeightArgs{(const char*)a.w2.values, (const char*)a.w2.scales, a.hidden, a.inter},
                   (uint16_t*)a.workspace, (uint16_t*)a.out, a.T, a.K, a.hidden, a.inter, a.rank * El, El};
    switch (a.format) {
        case kWeightsBf16: return by_rows<Weights<kWeightsBf16, 0>, 2>(p, a.E, stream);
        case kWeightsE4m3: return by_rows<Weights<kWeightsE4m3, 0>, 4>(p, a.E, stream);
        case kWeightsInt4: return by_group<kWeightsInt4>(p, a.E, a.group, stream);
        default: return by_group<kWeightsE2m1>(p, a.E, a.group, stream);
    }
}

}  // namespace ep
