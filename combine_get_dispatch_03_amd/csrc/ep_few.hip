// ep_few.hip -- a whole mixture-of-experts layer for a few tokens, in two kernels: from tokens and routing to tokens.
//
//   k_few_up     h[t,k] = silu(g) u,  g | u = x[t] W13_e^T           one workgroup: rows of one expert x 16 * NF / 2 channels of I
//   k_few_down   out[t] = sum_k w[t,k] h[t,k] W2_e^T + bias[t]       one workgroup: all experts in use x 16 channels of H
//
// No layout, dispatch or combine runs before or between: every workgroup finds the experts in use and their entries from the
// routing table itself (items: up to 16 * MT entries of one expert).  Both are bound by reading the weights of the experts in
// use, once each.  In the second the waves take items in turn, and each entry's 16 values stand in LDS until they are
// weighted and summed in ascending k, so that nothing depends on the order in which waves finish.
#include "ep_ffn.hpp"
#include "ep_stream.hpp"

namespace ep {
namespace {

constexpr int kDownThreads = 512, kDownWaves = kDownThreads / kWave;

struct Params {
    const uint16_t* x;        // [T, H]
    const int64_t* idx;       // [T, K]
    const float* topk_w;      // [T, K] or nullptr
    const uint16_t* bias;
    WeightArgs w13, w2;       // [El, 2 I, H], [El, H, I]
    uint16_t* h;              // workspace [T * K, row_pitch(I)]
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
};
struct ItemsLayout {
    int items, order, cursor;      // sizes
    int bytes() const { return (3 * items + cursor + 4) * 4 + order * 2; }
};
// Up to one wave's entries: every item has GROUP places in order.  Of more, all entries stand there, or one item's.
inline ItemsLayout items_layout(int entries, int El, int group, bool all) {
    const int busy = entries < El ? entries : El;
    const int items = (int)((entries + (int64_t)(group - 1) * busy) / group);
    if (entries <= kWave) return ItemsLayout{items, items * group, 0};
    return ItemsLayout{items, all ? entries : group, El};
}

// Items are the same in every workgroup.  ALL: all of them are wanted, and the order of an expert's entries is whatever it is: a
// row's values do not depend on the rows beside it.  Otherwise item `wanted` is, and as other workgroups take its other channels,
// its entries are the same everywhere: by their place among the expert's in the routing table.
template <int GROUP, int THREADS, bool ALL>
__device__ __forceinline__ Items find_items(const Params& p, char* lds, int max_items, int cursors, int wanted) {
    Items it;
    int* at = reinterpret_cast<int*>(lds);
    int* total = at;
    it.expert = at + 4;
    it.first = it.expert + max_items;
    it.count = it.first + max_items;
    it.cursor = it.count + max_items;
    it.order = reinterpret_cast<uint16_t*>(it.cursor + cursors);
    const int n = p.T * p.K, lane = lane_id();
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
        if ((int)threadIdx.x < kWave && in) {
            if (head == lane) {
                const int after = popc64(peers) - rank;
                it.expert[item] = e;
                it.first[item] = item * GROUP;
                it.count[item] = after < GROUP ? after : GROUP;
            }
            it.order[item * GROUP + rank % GROUP] = (uint16_t)lane;
        }
        it.total = popc64(heads);
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
    it.total = *total;
    return it;
}

// A workgroup's rows are an item's entries, its channels 16 * NF / 2 of I.
template <class W, int MT, int NF, int D>
__global__ __launch_bounds__(kStreamThreads, MT == 1 ? 4 : MT == 2 ? 3 : 2) void k_few_up(Params p, int max_items, int cursors, int lists, int cols) {
    extern __shared__ __align__(16) char smem[];
    const int item = blockIdx.x / cols, n0 = blockIdx.x % cols * (NF * 8);
    const Items it = find_items<16 * MT, kStreamThreads, false>(p, smem, max_items, cursors, item);
    if (item >= it.total) return;
    const int first = it.first[item], count = it.count[item], r = lane_id() & 15;
    RowFragments<W, MT> rows;
    rows.init(p.x, p.H);
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        const bool there = a * 16 + r < count;
        rows.place(a, there, (uint32_t)(it.order[first + (there ? a * 16 + r : 0)] / p.K) * (uint32_t)(p.H * 2));
    }
    stream_product<W, true, MT, NF, D>(p.w13, __builtin_amdgcn_readfirstlane(it.expert[item]), p.I, p.H, n0, rows, count, reinterpret_cast<float*>(smem + lists),
                                       [&](int m) { return p.h + (int64_t)it.order[first + m] * row_pitch(p.I); });
}

// Items (and, of few items, parts of their k) go to the waves in turn; parts = 1, 2, 4 or 8.
template <class W, int MT, int D>
__global__ __launch_bounds__(kDownThreads, MT == 4 ? 2 : 4) void k_few_down(Params p, int max_items, int cursors, int lists, int max_values) {
    extern __shared__ __align__(16) char smem[];
    const Items it = find_items<16 * MT, kDownThreads, true>(p, smem, max_items, cursors, 0);
    float* values = reinterpret_cast<float*>(smem + lists);       // [parts][T * K][16]
    const int lane = lane_id(), wave = wave_id(), r = lane & 15, g = lane >> 4, n0 = blockIdx.x * 16, n = p.T * p.K;
    const int pieces = pieces_of(p.I);
    int log_parts = 0;
    while (log_parts < 3 && (it.total << (log_parts + 1)) <= kDownWaves && (n << (log_parts + 1)) <= max_values) ++log_parts;
    const int parts = 1 << log_parts, work = it.total << log_parts;
    for (int i = wave; i < work; i += kDownWaves) {
        const int item = i >> log_parts, part = i & (parts - 1);
        const int expert = __builtin_amdgcn_readfirstlane(it.expert[item]), first = it.first[item], count = it.count[item];
        RowFragments<W, MT> rows;
        rows.init(p.h, p.I);
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            const bool there = a * 16 + r < count;
            rows.place(a, there, (uint32_t)it.order[first + (there ? a * 16 + r : 0)] * (uint32_t)(row_pitch(p.I) * 2));
        }
        typename W::template Rows<1> w;
        w.init(p.w2, expert, n0);
        w.place(0, 0, p.H - n0);
        f32x4 acc[1][MT];
#pragma unroll
        for (int a = 0; a < MT; ++a) acc[0][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        stream_pieces<W, MT, 1, D>(w, rows, part, parts, pieces, acc);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = a * 16 + g * 4 + j;
                if (m < count) values[(part * n + it.order[first + m]) * 16 + r] = acc[0][a][j];
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * 4; i += kDownThreads) {
        const int t = i / 4, c = n0 + i % 4 * 4;
        if (c >= p.H) continue;
        f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < p.K; ++k) {
            if (local_expert(p, t * p.K + k) < 0) continue;
            f32x4 v = *reinterpret_cast<const f32x4*>(values + (t * p.K + k) * 16 + i % 4 * 4);
            for (int q = 1; q < parts; ++q) v += *reinterpret_cast<const f32x4*>(values + (q * n + t * p.K + k) * 16 + i % 4 * 4);
            const float weight = W::kUnit * (p.topk_w ? p.topk_w[(int64_t)t * p.K + k] : 1.0f);
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

template <class W, int MT, int UP_NF, int UP_D, int DOWN_D>
hipError_t launch(const Params& p, hipStream_t stream) {
    const int n = p.T * p.K;
    ItemsLayout l = items_layout(n, p.El, 16 * MT, false);
    int lists = (l.bytes() + 15) & ~15;
    const int up_lds = lists + stream_lds<UP_NF>(), cols = (p.I + UP_NF * 8 - 1) / (UP_NF * 8);
    hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_few_up<W, MT, UP_NF, UP_D>), up_lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_up<W, MT, UP_NF, UP_D>), dim3((unsigned)(l.items * cols)), dim3(kStreamThreads), up_lds, stream, p, l.items,
                       l.cursor, lists, cols);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    l = items_layout(n, p.El, 16 * MT, true);
    lists = (l.bytes() + 15) & ~15;
    // room for the parts of few items' entries
    const int values = n > kDownWaves * 16 * MT ? n : kDownWaves * (n < 16 * MT ? n : 16 * MT), down_lds = lists + values * 64;
    e = allow_dynamic_lds(reinterpret_cast<const void*>(&k_few_down<W, MT, DOWN_D>), down_lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_few_down<W, MT, DOWN_D>), dim3((p.H + 15) / 16), dim3(kDownThreads), down_lds, stream, p, l.items, l.cursor, lists, values);
    return hipGetLastError();
}

// Rows an expert has on average decide how many steps of 16 a workgroup takes past the weights at a time.
template <class W, int UP_NF, int UP_D, int DOWN_D>
hipError_t by_rows(const Params& p, int E, hipStream_t stream) {
    const double rows = (double)p.T * p.K / E;
    if (rows <= 12) return launch<W, 1, UP_NF, UP_D, DOWN_D>(p, stream);
    if (rows <= 24) return launch<W, 2, UP_NF, 1, 2>(p, stream);
    return launch<W, 4, UP_NF, 1, 1>(p, stream);
}

template <WeightFormat F>
hipError_t by_group(const Params& p, int E, int group, hipStream_t stream) {
    if (group == 128) return by_rows<Weights<F, 1>, 4, 2, 4>(p, E, stream);
    if (group == 64) return by_rows<Weights<F, 2>, 4, 2, 4>(p, E, stream);
    return by_rows<Weights<F, 4>, 4, 2, 4>(p, E, stream);
}

}  // namespace

size_t few_workspace_bytes(int T, int K, int inter) { return (size_t)(T * K > 0 ? T * K : 1) * row_pitch(inter) * sizeof(uint16_t); }

hipError_t launch_few(const FewArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int El = a.E / a.R;
    const Params p{(const uint16_t*)a.x, a.topk_idx, a.topk_weights, (const uint16_t*)a.bias,
                   WeightArgs{(const char*)a.w13.values, (const char*)a.w13.scales, 2 * a.inter, a.hidden},
                   WeightArgs{(const char*)a.w2.values, (const char*)a.w2.scales, a.hidden, a.inter},
                   (uint16_t*)a.workspace, (uint16_t*)a.out, a.T, a.K, a.hidden, a.inter, a.rank * El, El};
    switch (a.format) {
        case kWeightsBf16: return by_rows<Weights<kWeightsBf16, 0>, 2, 2, 2>(p, a.E, stream);
        case kWeightsE4m3: return by_rows<Weights<kWeightsE4m3, 0>, 4, 2, 3>(p, a.E, stream);
        case kWeightsInt4: return by_group<kWeightsInt4>(p, a.E, a.group, stream);
        default: return by_group<kWeightsE2m1>(p, a.E, a.group, stream);
    }
}

}  // namespace ep
