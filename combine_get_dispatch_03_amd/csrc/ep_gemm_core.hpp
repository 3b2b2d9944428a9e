// ep_gemm_core.hpp -- the matrix product inside the expert kernels: one workgroup, one output tile.
//
//   acc[m][n] = sum_k S[m][k] F[n][k]        m: rows of the segment (or of a weight gradient), n: output channels
//
// Eight waves, 2 along m by 4 along n; 16x16x32 bf16 matrix instructions with fp32 sums.  The instruction's first operand is F, so a lane ends up with 4
// consecutive n of one m and stores them with one instruction.
//
// Operands travel global -> LDS by the buffer loads that write LDS directly (no registers, no ds_write), a few
// stages deep.  An element that does not exist (a row past the segment, a channel past N, a k past
// the end) is loaded from an offset past the resource's end, which the hardware answers with zero: no branch, and
// nothing outside the tensors (or in padding rows, whose NaNs would spread) is read.
//
// Two LDS forms, by the operand's layout in memory:
//   k contiguous (KC): 128 bytes a row, 16-byte chunks permuted by the row number so that a fragment read (16 rows, 16
//     bytes at one place of each) is spread over all banks.
//   k strided (KS): a k-row of all columns; fragments come from the transposing LDS read (four k of a column per
//     lane), chunks permuted by the k-row for the same reason.
#pragma once

#include "ep_device.hpp"

namespace ep {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kGemmThreads = 512;
constexpr int kGemmWaves = kGemmThreads / kWave;
constexpr int kBN = 256;                       // output channels of a tile (rows of F)
constexpr uint32_t kNoElement = 0xC0000000u;   // resource size and the offset of an element that does not exist

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave); }

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32;
}

// What happens once per tile stays behind a branch (the compiler would make it selects in every step of the loop).
__device__ __forceinline__ void stay_branch() { asm volatile(""); }

__device__ __forceinline__ i32x4 resource(uint64_t base, uint32_t bytes = kNoElement) {
    i32x4 r;
    r[0] = (int)(uint32_t)base;
    r[1] = (int)((uint32_t)(base >> 32) & 0xFFFFu);
    r[2] = (int)bytes;
    r[3] = 0x00020000;
    return r;
}

// 64 lanes x 16 bytes from resource + offset into LDS at `lds` + lane * 16.  Counted
// by vmcnt; the compiler does not see it, so whoever reads the LDS waits for it.  ONCE: marked non-temporal, for whole
// lines that no other workgroup reads.
template <bool ONCE = false>
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, uint32_t offset, i32x4 res) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(lds), "v"(offset), "s"(res) : "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(res) : "m0");
}
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, uint32_t offset, i32x4 res) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(res) : "m0");
}

// All LDS reads of this wave are back, and of its copies to LDS all but the newest `LEFT`; then the workgroup meets.
template <int LEFT>
__device__ __forceinline__ void wait_and_meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Which of a wave's 64 rows of F stands at row `i` (0 .. 15) of its fragment `b`.  The matrix instruction leaves lane group
// g with its rows 4g .. 4g + 3, so fragments 2j and 2j + 1 together give it channels 32 j + 8 g .. + 7: 16 bytes of
// bf16 to store at once, 64 bytes in a row over the four groups.
__device__ __forceinline__ int channel_of(int b, int i) { return (b >> 1) * 32 + (i >> 2) * 8 + (b & 1) * 4 + (i & 3); }

// An operand whose k is contiguous: ROWS rows, 128 bytes of each per stage (64 bf16, or 128 e4m3).  A row is a line of LDS,
// its 16-byte chunks permuted by the row number.
// SPREAD: fragment() and fragment() ^ 64 give lane group g the row's chunks 2g and 2g + 1 (otherwise g and g + 4), the 16
// terms for which one read fetches the other operand's e4m3.
template <int ROWS, bool SPREAD = false>
struct KcOperand {
    static constexpr int kCopies = ROWS / 8 / kGemmWaves;     // copies of a stage per wave
    static constexpr int kBytes = ROWS * 128;
    uint64_t base;
    uint32_t offset[kCopies];

    // The base comes out of vector registers: five wait states before a memory instruction reads it.  Back into scalar registers, wherever the compiler kept it between begin() and the loop.
    __device__ __forceinline__ void settle() {
        base = uniform64(base);
        asm volatile("s_nop 4" : "+s"(base));
    }

    static __device__ __forceinline__ int chunk() {      // the lane's, of 8
        const int at = (lane_id() & 7) ^ (lane_id() >> 3);
        return SPREAD ? (at & 3) << 1 | at >> 2 : at;
    }

    // row_offset(r): byte offset of tile row r from `start`, or kNoElement.
    template <class RowOffset>
    __device__ __forceinline__ void init(const void* start, RowOffset row_offset) {
        base = uniform64((uint64_t)start);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t o = row_offset((i * kGemmWaves + wave_id()) * 8 + (lane_id() >> 3));
            offset[i] = o == kNoElement ? kNoElement : o + chunk() * 16;
        }
    }
    // The next stage, with `left` bytes of each row to go (none or fewer: nothing is read, LDS is zeroed).  What the last
    // stage lacks is taken out of the offsets for good; the operand of another tile follows.
    template <bool ONCE = false>
    __device__ __forceinline__ void copy(uint32_t lds, int left) {
        if (left < 128) {
            stay_branch();
#pragma unroll
            for (int i = 0; i < kCopies; ++i) offset[i] = chunk() * 16 < left ? offset[i] : kNoElement;
        }
        const i32x4 res = resource(base);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds + threadIdx.x / kWave * 1024);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) copy16_to_lds<ONCE>(to + i * kGemmWaves * 1024, offset[i], res);
        base += 128;
    }
    // LDS offset of the lane's 16 bytes of the rows from row0, first half of the line; the second half is at ^ 64, the
    // next 16 rows at + 2048.
    static __device__ __forceinline__ uint32_t fragment(int row0) {
        const int r = lane_id() & 15, g = lane_id() >> 4;
        return (row0 + r) * 128 + ((g ^ (r & 7)) << 4);
    }
};

// An operand whose k is strided: 64 k-rows per stage, COLS columns of bf16.  Its fragments are read transposed, half a wave
// at a time: two lane groups, 8 k-rows apart, of 8 bytes from each of four k-rows.  permute() spreads these 256 bytes over
// the 64 banks.  A read then takes 2.7 cycles, 4.0 where the two groups met in the same banks.
template <int COLS, bool IS_F>
struct KsOperand {
    static constexpr int kRowBytes = COLS * 2, kChunks = kRowBytes / 16;
    static constexpr int kCopies = 64 * kRowBytes / 1024 / kGemmWaves;
    static constexpr int kBytes = 64 * kRowBytes;
    uint64_t base;
    uint64_t step;     // bytes of 64 k-rows
    uint32_t offset[kCopies];

    __device__ __forceinline__ void settle() {
        base = uniform64(base);
        step = uniform64(step);
        asm volatile("s_nop 4" : "+s"(base), "+s"(step));
    }

    static __device__ __forceinline__ int permute(int k) { return (k & 3) << 2 | (k >> 3 & 1) << (IS_F ? 0 : 1); }
    static __device__ __forceinline__ int row(int i) { return (i * kGemmWaves + wave_id()) * (kWave / kChunks) + lane_id() / kChunks; }

    // cols: columns that exist, counted from the tile's first.
    __device__ __forceinline__ void init(const void* start, int64_t stride_bytes, int cols) {
        base = uniform64((uint64_t)start);
        step = uniform64((uint64_t)stride_bytes * 64);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int c = (lane_id() % kChunks) ^ permute(row(i));
            offset[i] = c * 8 < cols ? (uint32_t)(row(i) * stride_bytes) + c * 16 : kNoElement;
        }
    }
    // The next stage, with `left` k-rows to go (as KcOperand).
    template <bool ONCE = false>
    __device__ __forceinline__ void copy(uint32_t lds, int left) {
        if (left < 64) {
            stay_branch();
#pragma unroll
            for (int i = 0; i < kCopies; ++i) offset[i] = row(i) < left ? offset[i] : kNoElement;
        }
        const i32x4 res = resource(base);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds + threadIdx.x / kWave * 1024);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) copy16_to_lds<ONCE>(to + i * kGemmWaves * 1024, offset[i], res);
        base += step;
    }
    // LDS offset of the lane's part of 16 columns: k-rows 8g .. 8g + 3; + 4 * kRowBytes for 8g + 4 .. 8g + 7,
    // + 32 * kRowBytes for the second 32 k.  S's fragment: the columns from col0 on.  F's fragment b of a wave's 64
    // columns: four columns for every g, placed as channel_of() says, but for odd g changed with those of fragment b ^ 1: a
    // fragment then has halves of chunks of both kinds, and restore_channels() sets the sums right.
    static __device__ __forceinline__ uint32_t fragment(int col0) {
        const int lane = lane_id(), k = (lane >> 4) * 8 + ((lane & 15) >> 2), q = lane & 3;
        return k * kRowBytes + (((col0 / 8 + (q >> 1)) ^ permute(k)) << 4) + (q & 1) * 8;
    }
    static __device__ __forceinline__ uint32_t fragment_f(int col0, int b) {
        const int lane = lane_id(), k = (lane >> 4) * 8 + ((lane & 15) >> 2), col = col0 + channel_of(b ^ (lane & 1), (lane & 3) * 4);
        return k * kRowBytes + (((col / 8) ^ permute(k)) << 4) + (col & 4) * 2;
    }
};

__device__ __forceinline__ bf16x8 read_kc(const char* lds, uint32_t at) { return *reinterpret_cast<const bf16x8*>(lds + at); }

template <int ROW_BYTES>
__device__ __forceinline__ bf16x8 read_ks(const char* lds, uint32_t at) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at + 4 * ROW_BYTES));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Eight e4m3 -> eight bf16, exact.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bf16x8 widen_e4m3x8(i32x2 q) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[0], 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[0], 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[1], 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[1], 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Sums of a k-strided F (KsOperand::fragment_f): back in channel_of()'s order.
template <int MT, int NT>
__device__ __forceinline__ void restore_channels(f32x4 (&acc)[MT][NT]) {
    const bool odd = lane_id() >> 4 & 1;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; b += 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = acc[a][b][i], hi = acc[a][b + 1][i];
                acc[a][b][i] = odd ? hi : lo;
                acc[a][b + 1][i] = odd ? lo : hi;
            }
}

template <int ROWS, bool KS, bool IS_F>
struct OperandOf { typedef KcOperand<ROWS> type; };
template <int ROWS, bool IS_F>
struct OperandOf<ROWS, true, IS_F> { typedef KsOperand<ROWS, IS_F> type; };

// The bf16 tiles of a workgroup, one after the other: up to 256 rows of S against 256 rows of F, 64 k per stage.  A wave
// owns 16 * MT rows (MT of run(), up to 8) by 64 channels.
//
// Waves 0-3 (the upper rows) run half a step ahead of waves 4-7, so that on every SIMD one wave feeds the matrix unit
// while the other reads its next fragments; two barriers per 32 k keep them in step.  The copies of a step are issued
// before its reads.  S is two stages deep in LDS and F three: all 160 KiB.  F's stage st + 2 and S's stage st + 1 are
// under way while stage st is multiplied; weights come from HBM and need the longer lead, rows are read again and
// again from L2.  Measured on 8192 x 8192 x 4096 (dense, everything in reach of L2): 1.43 PFLOP/s; 32 k per stage, four stages
// deep, 1.39; with the copies left out 1.70, the reads too 1.86.
//
// The stages of a workgroup's tiles form one stream: the last two stages of a tile copy the first of the next one
// (next_s, next_f, next_k), which then starts on data that has landed, while its predecessor is being stored.
//
// ONCE: F is read by this tile only (see copy16_to_lds).
template <bool SKS, bool FKS, bool ONCE = false>
struct Bf16Tiles {
    static constexpr int kBM = 256, NT = 4;
    typedef typename OperandOf<kBM, SKS, false>::type SOp;
    typedef typename OperandOf<kBN, FKS, true>::type FOp;
    static constexpr int kSBuffers = 2, kFBuffers = 3, kF = SOp::kBytes * kSBuffers;
    static constexpr int kLds = kF + FOp::kBytes * kFBuffers;
    static constexpr int kSUnit = SKS ? 1 : 2, kFUnit = FKS ? 1 : 2;      // what copy() counts in: k-rows, or bytes of a row

    char* smem;
    SOp s, next_s;
    FOp f, next_f;
    int next_k;                // terms of the next tile's sums; 0: no next tile (next_s and next_f then only need a value)
    int k, s_left, f_left;     // of the tile under way; k that its operands have yet to copy
    int sbuf, fbuf;            // buffers of the stage to be multiplied next

    __device__ __forceinline__ void copy_s(int buf) {
        s.copy(lds_address(smem) + buf * SOp::kBytes, s_left * kSUnit);
        s_left -= 64;
    }
    __device__ __forceinline__ void copy_f(int buf) {
        f.template copy<ONCE>(lds_address(smem) + kF + buf * FOp::kBytes, f_left * kFUnit);
        f_left -= 64;
    }
    // s, f and k_terms are the workgroup's first tile.
    __device__ __forceinline__ void begin(char* lds, int k_terms) {
        smem = lds;
        k = s_left = f_left = k_terms;
        sbuf = fbuf = 0;
        s.settle();
        f.settle();
        copy_f(0);
        copy_s(0);
        copy_f(1);
        wait_and_meet<FOp::kCopies>();
    }

    // The sums of the tile under way; afterwards the next one is.  Global loads and stores may stand between two run()s: the
    // waits below count copies, which land in order.
    template <int MT>
    __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT]) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
        // at least two, so that only one tile has to be known ahead
        const int stages = __builtin_amdgcn_readfirstlane(k > 64 ? (k + 63) / 64 : 2);
        s_left = __builtin_amdgcn_readfirstlane(s_left);
        f_left = __builtin_amdgcn_readfirstlane(f_left);
        next_k = __builtin_amdgcn_readfirstlane(next_k);
        sbuf = __builtin_amdgcn_readfirstlane(sbuf);
        fbuf = __builtin_amdgcn_readfirstlane(fbuf);
        s.settle();
        f.settle();
        next_s.settle();
        next_f.settle();
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        uint32_t s_at[SKS ? MT : 1], f_at[FKS ? NT : 1];
#pragma unroll
        for (int a = 0; a < (SKS ? MT : 1); ++a) s_at[a] = SOp::fragment((wm * MT + a) * 16);
        if constexpr (FKS) {
#pragma unroll
            for (int b = 0; b < NT; ++b) f_at[b] = FOp::fragment_f(wn * 64, b);
        } else {
            f_at[0] = FOp::fragment(wn * 64);
        }

        meet();
        if (wm == 1) meet();
        for (int st = 0; st < stages; ++st) {
            const char* ls = smem + sbuf * SOp::kBytes;
            const char* lf = smem + kF + fbuf * FOp::kBytes;
            if (st == stages - 1) {
                stay_branch();
                s = next_s, s_left = next_k;
            }
            if (st == stages - 2) {
                stay_branch();
                f = next_f, f_left = next_k;
            }
            sbuf ^= 1;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // both targets were last read in the stage before, which every wave had left before the last barrier
                if (half == 0) copy_s(sbuf);
                else copy_f(fbuf == 0 ? 2 : fbuf - 1);
                bf16x8 sv[MT], fv[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    if constexpr (FKS) fv[b] = read_ks<FOp::kRowBytes>(lf, f_at[b] + half * 32 * FOp::kRowBytes);
                    else fv[b] = read_kc(lf, (f_at[0] ^ (half * 64)) + b * 2048);
                }
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    if constexpr (SKS) sv[a] = read_ks<SOp::kRowBytes>(ls, s_at[a] + half * 32 * SOp::kRowBytes);
                    else sv[a] = read_kc(ls, (s_at[0] ^ (half * 64)) + a * 2048);
                }
                // before a wave goes on to the next stage all but the newest copies, F's of the stage after it, have landed
                if (half == 0) wait_and_meet<63>();
                else wait_and_meet<FOp::kCopies>();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < NT; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv[b], sv[a], acc[a][b], 0, 0, 0);
                __builtin_amdgcn_s_setprio(0);
                meet();
            }
            fbuf = fbuf == 2 ? 0 : fbuf + 1;
        }
        if (wm == 0) meet();
        if constexpr (FKS) restore_channels(acc);
        k = next_k;
    }

    // No copy may land after the workgroup has left its LDS.
    static __device__ __forceinline__ void end() { wait_and_meet<0>(); }
};

// ---- e4m3 operands ----------------------------------------------------------------------------------------------

// 32 bytes of a lane: which k they are does not matter as long as both operands agree.
__device__ __forceinline__ i32x8 read_line(const char* lds, uint32_t at) {
    const i32x4 a = *reinterpret_cast<const i32x4*>(lds + at), b = *reinterpret_cast<const i32x4*>(lds + (at ^ 64));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The e4m3 tiles of a workgroup, one after the other (as Bf16Tiles): up to 192 rows of S with a scale per row and 128 k,
// against 256 rows of F with a scale per half of each wave's rows and 128 k.  One 16x16x128 matrix instruction gives a block's sums, which
// take the product of the two scales on their way into acc: products and scales are exact, sums are fp32.
//
// 128 k per stage, in two half steps of two fragments of F each; S's fragments stay for both.
template <bool ONCE>
struct Fp8Tiles {
    static constexpr int kBM = 192, NT = 4;
    typedef KcOperand<kBM> SOp;
    typedef KcOperand<kBN> FOp;
    static constexpr int kSBuffers = 2, kFBuffers = 3, kF = SOp::kBytes * kSBuffers;
    // [2][64 * waves] scales of a stage's rows.  Each is a cache line of its own in memory, so no two waves fetch the same.
    static constexpr int kRowScales = kF + FOp::kBytes * kFBuffers, kRowScaleBytes = kGemmWaves * 256;
    static constexpr int kFScales = kRowScales + 2 * kRowScaleBytes;             // [2 tiles][2 rows of up to 256 fp32]
    static constexpr int kLds = kFScales + 2 * 2048;
    static constexpr int kAhead = FOp::kCopies + SOp::kCopies + 1;               // copies under way past the next stage

    char* smem;
    SOp s, next_s;
    FOp f, next_f;
    uint64_t scales, next_scales;              // of the tile's rows; 4 bytes further each stage
    uint32_t scale_offset, next_scale_offset;
    int next_k, k, s_left, f_left, sbuf, fbuf, tile;

    __device__ __forceinline__ void next_row_scales(const float* at, int blocks, int rows) {
        next_scales = uniform64((uint64_t)at);
        const int r = (int)threadIdx.x;
        next_scale_offset = r < rows ? (uint32_t)(r * blocks) * 4 : kNoElement;
    }
    // The next tile's F scales: two rows of `blocks`, the second `second` bytes behind the first; zeros up to the 256th.
    __device__ __forceinline__ void copy_next_f_scales(const float* at, uint32_t second, int blocks, int which) {
        const int i = (wave_id() & 3) * 64 + lane_id();
        uint64_t base = uniform64((uint64_t)at);
        asm volatile("s_nop 4" : "+s"(base));
        copy4_to_lds(lds_address(smem) + kFScales + which * 2048 + wave_id() * 256,
                     i < blocks ? (wave_id() >> 2) * second + i * 4 : kNoElement, resource(base));
    }
    __device__ __forceinline__ void copy_s(int buf) {
        const uint32_t lds0 = lds_address(smem);
        s.copy(lds0 + buf * SOp::kBytes, s_left);
        copy4_to_lds(__builtin_amdgcn_readfirstlane(lds0 + kRowScales + buf * kRowScaleBytes + threadIdx.x / kWave * 256), scale_offset, resource(scales, s_left > 0 ? kNoElement : 0u));
        scales += 4;
        s_left -= 128;
    }
    __device__ __forceinline__ void copy_f(int buf) {
        f.template copy<ONCE>(lds_address(smem) + kF + buf * FOp::kBytes, f_left);
        f_left -= 128;
    }
    __device__ __forceinline__ void settle() {
        s.settle();
        f.settle();
        next_s.settle();
        next_f.settle();
        scales = uniform64(scales);
        next_scales = uniform64(next_scales);
        asm volatile("s_nop 4" : "+s"(scales), "+s"(next_scales));
    }
    __device__ __forceinline__ void take_next_s() {
        s = next_s, scales = next_scales, s_left = next_k;
        scale_offset = next_scale_offset;
    }
    // The workgroup's first tile, which next_* describe (and its F scales are on their way to buffer 0).
    __device__ __forceinline__ void begin(int k_terms) {
        next_k = k_terms;
        settle();
        f = next_f, f_left = next_k;
        take_next_s();
        k = next_k;
        sbuf = fbuf = tile = 0;
        copy_f(0);
        copy_s(0);
        copy_f(1);
        copy_s(1);
        wait_and_meet<kAhead>();
    }

    template <int MT>
    __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT]) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
        const int stages = __builtin_amdgcn_readfirstlane(k > 128 ? k / 128 : 2);
        s_left = __builtin_amdgcn_readfirstlane(s_left);
        f_left = __builtin_amdgcn_readfirstlane(f_left);
        next_k = __builtin_amdgcn_readfirstlane(next_k);
        sbuf = __builtin_amdgcn_readfirstlane(sbuf);
        fbuf = __builtin_amdgcn_readfirstlane(fbuf);
        settle();
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t s_at = SOp::fragment(wm * MT * 16), f_at = FOp::fragment(wn * 64);
        const float* fs = reinterpret_cast<const float*>(smem + kFScales + tile * 2048);
        meet();
        if (wm == 1) meet();
        for (int st = 0; st < stages; ++st) {
            const char* ls = smem + sbuf * SOp::kBytes;
            const char* lf = smem + kF + fbuf * FOp::kBytes;
            const float* rs = reinterpret_cast<const float*>(smem + kRowScales + sbuf * kRowScaleBytes) + wm * MT * 16 + (lane_id() & 15);
            if (st == stages - 2) {
                stay_branch();
                take_next_s();
                f = next_f, f_left = next_k;
            }
            i32x8 sv[MT];
            float row_scale[MT];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // stage st + 2: F where stage st - 1 was, S where stage st is, whose fragments every wave took in the
                // first half step
                if (half == 0) copy_f(fbuf == 0 ? 2 : fbuf - 1);
                else copy_s(sbuf);
                i32x8 fv[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) fv[b] = read_line(lf, f_at + (half * 2 + b) * 2048);
                if (half == 0) {
#pragma unroll
                    for (int a = 0; a < MT; ++a) sv[a] = read_line(ls, s_at + a * 2048);
#pragma unroll
                    for (int a = 0; a < MT; ++a) row_scale[a] = rs[a * 16];
                }
                const float f_scale = fs[half * 256 + st];      // zero in a stage past k, as all behind the last block
                if (half == 0) wait_and_meet<63>();
                else wait_and_meet<kAhead>();
                __builtin_amdgcn_s_setprio(1);
                f32x4 part[MT][2];
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        part[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fv[b], sv[a], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const float scale = row_scale[a] * f_scale;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[a][half * 2 + b][i] = fmaf(part[a][b][i], scale, acc[a][half * 2 + b][i]);
                }
                __builtin_amdgcn_s_setprio(0);
                meet();
            }
            sbuf ^= 1;
            fbuf = fbuf == 2 ? 0 : fbuf + 1;
        }
        if (wm == 0) meet();
        k = next_k;
        tile ^= 1;
    }

    static __device__ __forceinline__ void end() { wait_and_meet<0>(); }
};

// The tiles of bf16 rows by e4m3 weights, one after the other (as Bf16Tiles): up to 160 rows of S against 256 rows of F
// with a scale per wave and 128 k.  F is widened to bf16 (exact) on its way from LDS; a block's sums are kept apart and
// take the scale in fp32 on their way into acc.  (Those two sets of sums are what limits the rows: 5 steps of 16 per wave.)
// 64 k per stage: 128 bytes of a row of S, 64 of F (two rows a line of LDS).  S is three stages deep and F four.
struct Bf16ByFp8Tiles {
    static constexpr int kBM = 160, NT = 4;
    typedef KcOperand<192, true> SOp;                // whole copies per wave; rows from 160 on do not exist
    static constexpr int kFBytes = kBN * 64, kFCopies = 2;
    static constexpr int kSBuffers = 3, kFBuffers = 4, kF = SOp::kBytes * kSBuffers;
    static constexpr int kFScales = kF + kFBytes * kFBuffers;     // [2 tiles][2 rows of up to 256 fp32]: channels 0..127, 128..255
    static constexpr int kLds = kFScales + 2 * 2048;
    static constexpr int kAhead = kFCopies + SOp::kCopies + kFCopies;    // copies under way past the next stage

    char* smem;
    SOp s, next_s;
    uint64_t f, next_f;
    uint32_t f_offset[kFCopies], next_f_offset[kFCopies];
    int next_k, k, s_left, f_left, sbuf, fbuf, tile;      // sbuf, fbuf: of the stage to be multiplied next

    // A copy of F is 16 rows of 64 bytes; a row's four chunks are permuted by the pair of rows it stands in.
    template <class RowOffset>
    __device__ __forceinline__ void init_next_f(const void* start, RowOffset row_offset) {
        next_f = uniform64((uint64_t)start);
        const int x = (lane_id() & 7) ^ (lane_id() >> 3);
#pragma unroll
        for (int i = 0; i < kFCopies; ++i) {
            const uint32_t o = row_offset((i * kGemmWaves + wave_id()) * 16 + (lane_id() >> 3) * 2 + (x >> 2));
            next_f_offset[i] = o == kNoElement ? kNoElement : o + (x & 3) * 16;
        }
    }
    // The next tile's F scales: two rows of `blocks`, the second `second` bytes behind the first; zeros up to the 256th.
    __device__ __forceinline__ void copy_next_f_scales(const float* at, uint32_t second, int blocks, int which) {
        const int i = (wave_id() & 3) * 64 + lane_id();
        uint64_t base = uniform64((uint64_t)at);
        asm volatile("s_nop 4" : "+s"(base));
        copy4_to_lds(lds_address(smem) + kFScales + which * 2048 + wave_id() * 256,
                     i < blocks ? (wave_id() >> 2) * second + i * 4 : kNoElement, resource(base));
    }
    __device__ __forceinline__ void copy_s(int buf) {
        s.copy(lds_address(smem) + buf * SOp::kBytes, s_left * 2);
        s_left -= 64;
    }
    __device__ __forceinline__ void copy_f(int buf) {
        const i32x4 res = resource(f, f_left > 0 ? kNoElement : 0u);
        const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(smem) + kF + buf * kFBytes + threadIdx.x / kWave * 1024);
#pragma unroll
        for (int i = 0; i < kFCopies; ++i) copy16_to_lds(to + i * kGemmWaves * 1024, f_offset[i], res);
        f += 64;
        f_left -= 64;
    }
    __device__ __forceinline__ void settle() {
        s.settle();
        next_s.settle();
        f = uniform64(f);
        next_f = uniform64(next_f);
        asm volatile("s_nop 4" : "+s"(f), "+s"(next_f));
    }
    __device__ __forceinline__ void take_next_s() { s = next_s, s_left = next_k; }
    __device__ __forceinline__ void take_next_f() {
        f = next_f, f_left = next_k;
#pragma unroll
        for (int i = 0; i < kFCopies; ++i) f_offset[i] = next_f_offset[i];
    }
    // The workgroup's first tile, which next_* describe (and its F scales are on their way to buffer 0).
    __device__ __forceinline__ void begin(int k_terms) {
        next_k = k_terms;
        settle();
        take_next_s();
        take_next_f();
        k = next_k;
        sbuf = fbuf = tile = 0;
        copy_f(0);
        copy_s(0);
        copy_f(1);
        copy_s(1);
        copy_f(2);
        wait_and_meet<kAhead>();
    }

    template <int MT>
    __device__ __forceinline__ void run(f32x4 (&acc)[MT][NT]) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
        const int stages = __builtin_amdgcn_readfirstlane(k > 256 ? k / 64 : 4);     // enough that one tile ahead will do
        s_left = __builtin_amdgcn_readfirstlane(s_left);
        f_left = __builtin_amdgcn_readfirstlane(f_left);
        next_k = __builtin_amdgcn_readfirstlane(next_k);
        sbuf = __builtin_amdgcn_readfirstlane(sbuf);
        fbuf = __builtin_amdgcn_readfirstlane(fbuf);
        settle();
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // a lane reads the 16 e4m3 of k 16g .. 16g + 15; half h of them goes with the bf16 at SOp's half h
        const int r = lane_id() & 15, g = lane_id() >> 4;
        const uint32_t s_at = SOp::fragment(wm * MT * 16);
        const uint32_t f_at = (wn * 64 + (r & ~1)) * 64 + (((((r & 1) << 2) | g) ^ (r >> 1)) << 4);
        const float* fs = reinterpret_cast<const float*>(smem + kFScales + tile * 2048) + (wn >> 1) * 256;
        meet();
        if (wm == 1) meet();
        for (int st = 0; st < stages; st += 2) {
            f32x4 part[MT][NT];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const char* ls = smem + sbuf * SOp::kBytes;
                const char* lf = smem + kF + fbuf * kFBytes;
                if (st + q == stages - 2) {
                    stay_branch();
                    take_next_s();
                }
                if (st + q == stages - 3) {
                    stay_branch();
                    take_next_f();
                }
                // the buffers of the stage before, which every wave had left before the last barrier
                copy_s(sbuf == 0 ? kSBuffers - 1 : sbuf - 1);
                copy_f((fbuf + kFBuffers - 1) % kFBuffers);
                bf16x8 sv[MT][2];
                i32x4 fq[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b) fq[b] = *reinterpret_cast<const i32x4*>(lf + f_at + b * 1024);
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    sv[a][0] = read_kc(ls, s_at + a * 2048);
                    sv[a][1] = read_kc(ls, (s_at ^ 64) + a * 2048);
                }
                const float scale = q == 1 ? fs[st / 2] : 0.0f;      // zero past k, as in Fp8Tiles
                wait_and_meet<kAhead>();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        const bf16x8 fv = widen_e4m3x8(i32x2{fq[b][2 * h], fq[b][2 * h + 1]});
#pragma unroll
                        for (int a = 0; a < MT; ++a)
                            part[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, sv[a][h], q + h == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : part[a][b], 0, 0, 0);
                    }
                if (q == 1) {
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(part[a][b][i], scale, acc[a][b][i]);
                }
                __builtin_amdgcn_s_setprio(0);
                meet();
                sbuf = sbuf == kSBuffers - 1 ? 0 : sbuf + 1;
                fbuf = (fbuf + 1) % kFBuffers;
            }
        }
        if (wm == 0) meet();
        k = next_k;
        tile ^= 1;
    }

    static __device__ __forceinline__ void end() { wait_and_meet<0>(); }
};

}  // namespace ep
