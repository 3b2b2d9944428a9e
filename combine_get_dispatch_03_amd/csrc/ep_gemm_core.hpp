// ep_gemm_core.hpp -- the matrix product inside the expert kernels: one workgroup, one output tile.
//
//   acc[m][n] = sum_k S[m][k] F[n][k]        m: rows of the segment (or of a weight gradient), n: output channels
//
// Workgroup: 8 waves, 2 along m by 4 along n, 16x16x32 bf16 matrix instructions with fp32 sums.  The instruction's first
// operand is F, so a lane ends up with 4 consecutive n of one m and stores them with one instruction.
//
// Operands travel global -> LDS by the buffer loads that write LDS directly (no registers, no ds_write), 32 k per
// stage, kBuffers stages deep.  An element that does not exist (a row past the segment, a channel past N, a k past
// the end) is loaded from an offset past the resource's end, which the hardware answers with zero: no branch, and
// nothing outside the tensors (or in padding rows, whose NaNs would spread) is read.
//
// Two LDS forms, by the operand's layout in memory:
//   k contiguous (KC): 64 bytes a row, two rows a 128-byte line, 16-byte chunks permuted by the line number so that the
//     16 lanes x 16 bytes of a fragment read hit every bank once.
//   k strided (KS): a k-row of all columns; fragments come from the transposing LDS read (four k of a column per
//     lane), chunk pairs permuted by the k-row for the same reason.
//
// Schedule: the waves of the lower m half run half a step ahead of the others, so that on every SIMD one wave feeds the
// matrix unit while the other reads its next fragments; barriers keep the two in step.
#pragma once

#include "ep_device.hpp"

namespace ep {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

__device__ __forceinline__ i32x4 resource(uint64_t base, uint32_t bytes) {
    i32x4 r;
    r[0] = (int)(uint32_t)base;
    r[1] = (int)((uint32_t)(base >> 32) & 0xFFFFu);
    r[2] = (int)bytes;
    r[3] = 0x00020000;
    return r;
}

// 64 lanes x 16 bytes from resource + offset into LDS at `lds` + lane * 16.  Counted by vmcnt; the compiler does not see
// it, so whoever reads the LDS waits for it (wait_stage).
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, uint32_t offset, i32x4 res) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(res)
                 : "m0");
}
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, uint32_t offset, i32x4 res) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(res)
                 : "m0");
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

// An operand whose k is contiguous: ROWS rows, 64 bytes of each per stage (32 bf16, or 64 e4m3).
template <int ROWS>
struct KcOperand {
    static constexpr int kCopies = ROWS / 16 / kGemmWaves;   // copies of a stage per wave
    static constexpr int kBytes = ROWS * 64;
    uint64_t base;
    uint32_t offset[kCopies];
    int chunk;     // the lane's 16-byte chunk of its rows

    // row_offset(r): byte offset of tile row r from `start`, or kNoElement.
    template <class RowOffset>
    __device__ __forceinline__ void init(const void* start, RowOffset row_offset) {
        const int lane = lane_id(), wave = wave_id();
        base = uniform64((uint64_t)start);
        const int x = (lane & 7) ^ (lane >> 3);
        chunk = x & 3;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int line = (i * kGemmWaves + wave) * 8 + (lane >> 3);
            const uint32_t o = row_offset(2 * line + (x >> 2));
            offset[i] = o == kNoElement ? kNoElement : o + chunk * 16;
        }
    }
    // Stage with `left` bytes of each row to go (<= 0: nothing is read, LDS is zeroed).
    __device__ __forceinline__ void copy(uint32_t lds, int left) {
        const i32x4 res = resource(base, left > 0 ? kNoElement : 0u);
        const uint32_t to = lds + wave_id() * 1024;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t o = left >= 64 || chunk * 16 < left ? offset[i] : kNoElement;
            copy16_to_lds(to + i * kGemmWaves * 1024, o, res);
        }
        base += 64;
    }
    // LDS offset of the lane's 16 bytes (8 bf16) of fragment row 0; fragment j is at + j * 1024.
    static __device__ __forceinline__ uint32_t fragment(int row0) {
        const int r = lane_id() & 15, g = lane_id() >> 4, line = r >> 1;
        return row0 * 64 + line * 128 + (((((r & 1) << 2) | g) ^ line) << 4);
    }
};

// An operand whose k is strided: 32 k-rows per stage, COLS columns of bf16.
template <int COLS>
struct KsOperand {
    static constexpr int kRowBytes = COLS * 2, kChunks = kRowBytes / 16;
    static constexpr int kCopies = 32 * kRowBytes / 1024 / kGemmWaves;
    static constexpr int kBytes = 32 * kRowBytes;
    uint64_t base;
    uint64_t step;     // bytes of 32 k-rows
    uint32_t offset[kCopies];
    int row[kCopies];

    static __device__ __forceinline__ int permute(int k) { return ((k & 3) | ((k >> 3) & 1) << 2) << 1; }

    // cols: columns that exist, counted from the tile's first.
    __device__ __forceinline__ void init(const void* start, int64_t stride_bytes, int cols) {
        const int lane = lane_id(), wave = wave_id();
        base = uniform64((uint64_t)start);
        step = uniform64((uint64_t)stride_bytes * 32);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            row[i] = (i * kGemmWaves + wave) * (kWave / kChunks) + lane / kChunks;
            const int c = (lane % kChunks) ^ permute(row[i]);
            offset[i] = c * 8 < cols ? (uint32_t)(row[i] * stride_bytes) + c * 16 : kNoElement;
        }
    }
    // Stage with `left` k-rows to go.
    __device__ __forceinline__ void copy(uint32_t lds, int left) {
        const i32x4 res = resource(base, left > 0 ? kNoElement : 0u);
        const uint32_t to = lds + wave_id() * 1024;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t o = left >= 32 || row[i] < left ? offset[i] : kNoElement;
            copy16_to_lds(to + i * kGemmWaves * 1024, o, res);
        }
        base += step;
    }
    // LDS offset of the lane's part of the 16 columns from col0: k-rows 8g .. 8g + 3, and + 4 * kRowBytes for the rest.
    static __device__ __forceinline__ uint32_t fragment(int col0) {
        const int lane = lane_id(), k = (lane >> 4) * 8 + ((lane & 15) >> 2), q = lane & 3;
        return k * kRowBytes + (((col0 / 8 + (q >> 1)) ^ permute(k)) << 4) + (q & 1) * 8;
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

template <int ROWS, bool KS>
struct OperandOf { typedef KcOperand<ROWS> type; };
template <int ROWS>
struct OperandOf<ROWS, true> { typedef KsOperand<ROWS> type; };

// The tile: 2 * MT * 16 rows of S against 256 rows of F.
template <int MT, bool SKS, bool FKS>
struct Bf16Tile {
    static constexpr int kBM = 2 * MT * 16, NT = 4;
    typedef typename OperandOf<kBM, SKS>::type SOp;
    typedef typename OperandOf<kBN, FKS>::type FOp;
    static constexpr int kStage = SOp::kBytes + FOp::kBytes;
    static constexpr int kBuffers = MT == 8 ? 4 : 3;     // the smaller tile: two workgroups on a CU
    static constexpr int kLds = kStage * kBuffers;
    static constexpr int kCopies = SOp::kCopies + FOp::kCopies;

    SOp s;
    FOp f;
    f32x4 acc[MT][NT];

    // `k` elements of the sum; k_unit: what the operands' copy() counts `left` in (bytes of a row, or k-rows)
    __device__ __forceinline__ void copy_stage(uint32_t lds, int stage, int k) {
        const int left = k - stage * 32;
        s.copy(lds, SKS ? left : 2 * left);
        f.copy(lds + SOp::kBytes, FKS ? left : 2 * left);
    }

    __device__ __forceinline__ void run(char* smem, int k) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
        const int stages = (k + 31) / 32;
        const uint32_t lds0 = lds_address(smem);
        // the bases come out of vector registers: five wait states before a memory instruction reads them
        asm volatile("s_nop 4" : "+s"(s.base), "+s"(f.base));
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        uint32_t s_at[SKS ? MT : 1], f_at[FKS ? NT : 1];
        if constexpr (SKS) {
#pragma unroll
            for (int a = 0; a < MT; ++a) s_at[a] = SOp::fragment(wm * MT * 16 + a * 16);
        } else {
            s_at[0] = SOp::fragment(wm * MT * 16);
        }
        if constexpr (FKS) {
#pragma unroll
            for (int b = 0; b < NT; ++b) f_at[b] = SOp::kBytes + FOp::fragment(wn * 64 + b * 16);
        } else {
            f_at[0] = SOp::kBytes + FOp::fragment(wn * 64);
        }

#pragma unroll
        for (int i = 0; i < kBuffers - 1; ++i) copy_stage(lds0 + i * kStage, i, k);
        wait_and_meet<(kBuffers - 2) * kCopies>();
        if (wm == 1) meet();
        int buf = 0;
        for (int st = 0; st < stages; ++st) {
            const char* l = smem + buf * kStage;
            bf16x8 sv[MT], fv[NT];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                if constexpr (FKS) fv[b] = read_ks<FOp::kRowBytes>(l, f_at[b]);
                else fv[b] = read_kc(l, f_at[0] + b * 1024);
            }
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                if constexpr (SKS) sv[a] = read_ks<SOp::kRowBytes>(l, s_at[a]);
                else sv[a] = read_kc(l, s_at[0] + a * 1024);
            }
            const int nbuf = buf == 0 ? kBuffers - 1 : buf - 1;      // the buffer read in the step before
            copy_stage(lds0 + nbuf * kStage, st + kBuffers - 1, k);
            wait_and_meet<(kBuffers - 2) * kCopies>();
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int b = 0; b < NT; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv[b], sv[a], acc[a][b], 0, 0, 0);
            __builtin_amdgcn_s_setprio(0);
            meet();
            buf = buf == kBuffers - 1 ? 0 : buf + 1;
        }
        if (wm == 0) meet();
        wait_and_meet<0>();      // no copy may land after the workgroup has left its LDS
    }
};

// ---- e4m3 operands ----------------------------------------------------------------------------------------------

// ROWS rows of e4m3, 128 k (one scale group) per stage: a row is a 128-byte line, chunks permuted by the row number.
template <int ROWS>
struct Kc128Operand {
    static constexpr int kCopies = ROWS / 8 / kGemmWaves;
    static constexpr int kBytes = ROWS * 128;
    uint64_t base;
    uint32_t offset[kCopies];

    template <class RowOffset>
    __device__ __forceinline__ void init(const void* start, RowOffset row_offset) {
        const int lane = lane_id();
        base = uniform64((uint64_t)start);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int row = (i * kGemmWaves + wave_id()) * 8 + (lane >> 3);
            const uint32_t o = row_offset(row);
            offset[i] = o == kNoElement ? kNoElement : o + (((lane & 7) ^ (row & 7)) << 4);
        }
    }
    __device__ __forceinline__ void copy(uint32_t lds, bool more) {
        const i32x4 res = resource(base, more ? kNoElement : 0u);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) copy16_to_lds(lds + wave_id() * 1024 + i * kGemmWaves * 1024, offset[i], res);
        base += 128;
    }
    // LDS offset of the first 16 of the lane's 32 bytes; the other 16 are at ^ 64; fragment j is at + j * 2048.  (Which k a
    // lane holds does not matter as long as both operands agree.)
    static __device__ __forceinline__ uint32_t fragment(int row0) {
        const int r = lane_id() & 15, g = lane_id() >> 4;
        return (row0 + r) * 128 + ((g ^ (r & 7)) << 4);
    }
    static __device__ __forceinline__ i32x8 read(const char* lds, uint32_t at) {
        const i32x4 a = *reinterpret_cast<const i32x4*>(lds + at), b = *reinterpret_cast<const i32x4*>(lds + (at ^ 64));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// 128 rows of e4m3 with a scale per row and 128 k, against 256 rows of e4m3 F with a scale per half of each wave's rows
// and 128 k: 16x16x128 matrix instructions, whose sums over one 128-block are exact products in fp32, then one FMA with the
// product of the two scales.
struct Fp8Tile {
    static constexpr int MT = 4, NT = 4, kBM = 128;
    typedef Kc128Operand<kBM> SOp;
    typedef Kc128Operand<kBN> FOp;
    static constexpr int kStage = SOp::kBytes + FOp::kBytes, kBuffers = 3;
    static constexpr int kCopies = SOp::kCopies + FOp::kCopies + 1;
    static constexpr int kRowScales = kStage * kBuffers;                          // per wave and stage 64 fp32
    static constexpr int kFScales = kRowScales + kGemmWaves * kBuffers * 256;     // two rows of up to 256 fp32
    static constexpr int kLds = kFScales + 2048;

    SOp s;
    FOp f;
    uint64_t scales;         // of the wave's 64 rows; 4 bytes further each stage
    uint32_t scale_offset;
    f32x4 acc[MT][NT];

    __device__ __forceinline__ void copy_stage(uint32_t lds0, int buf, bool more) {
        s.copy(lds0 + buf * kStage, more);
        f.copy(lds0 + buf * kStage + SOp::kBytes, more);
        copy4_to_lds(lds0 + kRowScales + (buf * kGemmWaves + wave_id()) * 256, scale_offset, resource(scales, more ? kNoElement : 0u));
        scales += 4;
    }

    // blocks of 128 k.  The F scales are in LDS at kFScales (written before the call): fragments 0, 1 of a wave take
    // the first row, 2, 3 the second.
    __device__ __forceinline__ void run(char* smem, int blocks) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
        const uint32_t lds0 = lds_address(smem);
        asm volatile("s_nop 4" : "+s"(s.base), "+s"(f.base), "+s"(scales));
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t s_at = SOp::fragment(wm * 64), f_at = SOp::kBytes + FOp::fragment(wn * 64);
        const float* fs = reinterpret_cast<const float*>(smem + kFScales);
#pragma unroll
        for (int i = 0; i < kBuffers - 1; ++i) copy_stage(lds0, i, i < blocks);
        wait_and_meet<(kBuffers - 2) * kCopies>();
        if (wm == 1) meet();
        int buf = 0;
        for (int st = 0; st < blocks; ++st) {
            const char* l = smem + buf * kStage;
            i32x8 sv[MT], fv[NT];
            float row_scale[MT];
#pragma unroll
            for (int b = 0; b < NT; ++b) fv[b] = FOp::read(l, f_at + b * 2048);
#pragma unroll
            for (int a = 0; a < MT; ++a) sv[a] = SOp::read(l, s_at + a * 2048);
#pragma unroll
            for (int a = 0; a < MT; ++a)
                row_scale[a] = *reinterpret_cast<const float*>(smem + kRowScales + (buf * kGemmWaves + wave) * 256 + (a * 16 + (lane_id() & 15)) * 4);
            const float f0 = fs[st], f1 = fs[256 + st];
            const int nbuf = buf == 0 ? kBuffers - 1 : buf - 1;
            copy_stage(lds0, nbuf, st + kBuffers - 1 < blocks);
            wait_and_meet<(kBuffers - 2) * kCopies>();
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                f32x4 part[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b)
                    part[b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fv[b], sv[a], f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                const float g0 = row_scale[a] * f0, g1 = row_scale[a] * f1;
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(part[b][i], b < 2 ? g0 : g1, acc[a][b][i]);
            }
            __builtin_amdgcn_s_setprio(0);
            meet();
            buf = buf == kBuffers - 1 ? 0 : buf + 1;
        }
        if (wm == 0) meet();
        wait_and_meet<0>();
    }
};

// 128 rows of bf16 against 256 rows of e4m3 F with a scale per wave and 128 k: F is widened to bf16 (exact) on its way from
// LDS, a block's sums get the scale in fp32.
struct Bf16ByFp8Tile {
    static constexpr int MT = 4, NT = 4, kBM = 128;
    typedef KcOperand<kBM> SOp;
    static constexpr int kFBytes = kBN * 32;
    static constexpr int kStage = SOp::kBytes + kFBytes, kBuffers = 4;
    static constexpr int kCopies = SOp::kCopies + 1;
    static constexpr int kFScales = kStage * kBuffers;     // two rows of up to 256 fp32: channels 0..127, 128..255
    static constexpr int kLds = kFScales + 2048;

    SOp s;
    uint64_t f;
    uint32_t f_offset;
    f32x4 acc[MT][NT];

    template <class RowOffset>
    __device__ __forceinline__ void init_f(const void* start, RowOffset row_offset) {
        f = uniform64((uint64_t)start);
        const uint32_t o = row_offset(wave_id() * 32 + lane_id() / 2);
        f_offset = o == kNoElement ? kNoElement : o + (lane_id() & 1) * 16;
    }
    __device__ __forceinline__ void copy_stage(uint32_t lds, int left) {
        s.copy(lds, 2 * left);
        copy16_to_lds(lds + SOp::kBytes + wave_id() * 1024, f_offset, resource(f, left > 0 ? kNoElement : 0u));
        f += 32;
    }

    __device__ __forceinline__ void run(char* smem, int k) {
        const int wave = wave_id(), wm = wave >> 2, wn = wave & 3, stages = k / 32;
        const uint32_t lds0 = lds_address(smem);
        asm volatile("s_nop 4" : "+s"(s.base), "+s"(f));
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t s_at = SOp::fragment(wm * 64);
        const uint32_t f_at = SOp::kBytes + (wn * 64 + (lane_id() & 15)) * 32 + (lane_id() >> 4) * 8;
        const float* fs = reinterpret_cast<const float*>(smem + kFScales) + (wn >> 1) * 256;
#pragma unroll
        for (int i = 0; i < kBuffers - 1; ++i) copy_stage(lds0 + i * kStage, k - i * 32);
        wait_and_meet<(kBuffers - 2) * kCopies>();
        if (wm == 1) meet();
        for (int st = 0; st < stages; st += 4) {
            f32x4 part[MT][NT];
            const float scale = fs[st / 4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {     // kBuffers = 4: the buffer is q
                const char* l = smem + q * kStage;
                bf16x8 sv[MT];
                i32x2 fq[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b) fq[b] = *reinterpret_cast<const i32x2*>(l + f_at + b * 512);
#pragma unroll
                for (int a = 0; a < MT; ++a) sv[a] = read_kc(l, s_at + a * 1024);
                copy_stage(lds0 + (q + 3) % 4 * kStage, k - (st + q + 3) * 32);
                wait_and_meet<(kBuffers - 2) * kCopies>();
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    const bf16x8 fv = widen_e4m3x8(fq[b]);
#pragma unroll
                    for (int a = 0; a < MT; ++a)
                        part[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, sv[a], q == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : part[a][b], 0, 0, 0);
                }
                if (q == 3) {
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int b = 0; b < NT; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[a][b][i] = fmaf(part[a][b][i], scale, acc[a][b][i]);
                }
                __builtin_amdgcn_s_setprio(0);
                meet();
            }
        }
        if (wm == 0) meet();
        wait_and_meet<0>();
    }
};

}  // namespace ep
