// ep_norm.hip -- the combine with the norms around a block, and its gradient.
//
//   f = sum_k w[t,k] y[slot(t,k)] + bias[t]      or the block's output itself
//   a = f rf post,  rf = 1 / sqrt(mean f^2 + eps)
//   r = rs residual + gate a                     -> out
//   n = r rr pre,   rr = 1 / sqrt(mean r^2 + eps)   -> normed
//
// One workgroup per token, a thread holds V 16-byte chunks of the row in registers from the first load to the last store:
// every row of y is read once, out and normed are written once, and what a norm needs of the whole row is one sum over
// the workgroup (lanes by register exchange, waves through LDS, in a fixed order).  Memory bounds it: 4096 tokens of 7168 through a
// handle with top-8 bf16 rows, bias, residual and two outputs 118 us (704 MB, 6.0 TB/s); without a handle, with residual (8 bytes a
// channel), 4096 rows of 7168 50 us (4.7 TB/s), 38 where y and residual are still in the memory-side cache.  Rows of more than 8192
// channels (four chunks a thread, 12 of its 128 registers spilled, room for 16 such waves a CU): 4096 of 8200 98 us (2.7 TB/s), of 16384
// 124 us (4.3 TB/s), of 32768 252 us (4.3 TB/s).
#include "ep_device.hpp"
#include "ep_internal.hpp"

namespace ep {
namespace {

constexpr int kMaxWaves = 16;

struct Params {
    const uint16_t* y;
    const float* w;          // [T, K] or nullptr (weights of 1)
    const int32_t* slot;     // [T, K]; nullptr: y holds a row per token
    const uint16_t* bias;
    NormVectors v;
    uint16_t* out;
    uint16_t* normed;
    float* kept;
    int T, H, K;
};

// Eight elements of a row (bf16 or fp32), chunk c.
__device__ __forceinline__ void load8(const void* row, bool bf16, int c, float* v) {
    if (bf16) {
        const u32x4 q = reinterpret_cast<const u32x4*>(row)[c];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(q[i]), v[2 * i + 1] = bf16hi(q[i]);
    } else {
        const f32x4* q = reinterpret_cast<const f32x4*>(row) + 2 * c;
        const f32x4 a = q[0], b = q[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    }
}
__device__ __forceinline__ void fill8(float* v, float x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x;
}
__device__ __forceinline__ u32x4 round8(const float* v) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// Sums over the workgroup of N values a thread, the same in every thread.  Whoever calls it again with the same LDS has
// passed another barrier in between.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*lds)[N]) {
    const int waves = blockDim.x / kWave;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = wave_sum(v[j]);
    if (waves == 1) return;
    if (lane_id() == 0) {
#pragma unroll
        for (int j = 0; j < N; ++j) lds[threadIdx.x / kWave][j] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        v[j] = lds[0][j];
        for (int i = 1; i < waves; ++i) v[j] += lds[i][j];
    }
}

__device__ __forceinline__ float inverse_rms(float squares, int H, float eps) { return 1.0f / sqrtf(squares / (float)H + eps); }

// f += the next N valid entries' rows by their weights, all N * V loads under way before the first is used.
template <int N, int V>
__device__ __forceinline__ void gather(float (&f)[V][8], const Params& p, uint64_t& left, int slot, float weight, const int (&c)[V]) {
    u32x4 q[N][V];
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = __builtin_ctzll(left);
        left &= left - 1;
        const u32x4* row = reinterpret_cast<const u32x4*>(p.y + (int64_t)readlane(slot, k) * p.H);
        w[i] = readlane_f(weight, k);
#pragma unroll
        for (int j = 0; j < V; ++j) q[i][j] = ld_nt(row + c[j]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[j][2 * e] = fmaf(w[i], bf16lo(q[i][j][e]), f[j][2 * e]);
                f[j][2 * e + 1] = fmaf(w[i], bf16hi(q[i][j][e]), f[j][2 * e + 1]);
            }
}

// Chunks past the row's end are read as its chunk 0 and neither summed nor stored.
template <int V, int THREADS>
__global__ __launch_bounds__(THREADS) void k_combine_norm(Params p) {
    __shared__ float sums[2][kMaxWaves][1];
    const int64_t token = block_id();
    if (token >= p.T) return;
    const int t = (int)token, chunks = p.H / 8;
    int c[V];
    bool there[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        c[j] = j * (int)blockDim.x + (int)threadIdx.x;
        there[j] = c[j] < chunks;
        c[j] = there[j] ? c[j] : 0;
    }
    float f[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) fill8(f[j], 0.0f);
    if (p.slot) {
        const int lane = lane_id();
        const int64_t entry = (int64_t)t * p.K + (lane < p.K ? lane : 0);
        const int slot = lane < p.K ? p.slot[entry] : -1;
        const float weight = p.w ? p.w[entry] : 1.0f;
        uint64_t left = ballot(slot >= 0);
        while (popc64(left) >= 8) gather<8, V>(f, p, left, slot, weight, c);
        if (popc64(left) >= 4) gather<4, V>(f, p, left, slot, weight, c);
        if (popc64(left) >= 2) gather<2, V>(f, p, left, slot, weight, c);
        if (left) gather<1, V>(f, p, left, slot, weight, c);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) load8(p.y + (int64_t)t * p.H, true, c[j], f[j]);
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (p.bias) {
            float b[8];
            load8(p.bias + (int64_t)t * p.H, true, c[j], b);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[j][i] += b[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[j][i] = there[j] ? f[j][i] : 0.0f;
            sum[0] = fmaf(f[j][i], f[j][i], sum[0]);
        }
        if (p.kept && there[j]) {
            f32x4* k = reinterpret_cast<f32x4*>(p.kept + (int64_t)t * p.H) + 2 * c[j];
            k[0] = f32x4{f[j][0], f[j][1], f[j][2], f[j][3]};
            k[1] = f32x4{f[j][4], f[j][5], f[j][6], f[j][7]};
        }
    }
    float rf = 1.0f;
    if (p.v.post) {
        block_sum<1>(sum, sums[0]);
        rf = inverse_rms(sum[0], p.H, p.v.eps);
    }
    sum[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float m[8];
        fill8(m, rf);
        if (p.v.post) {
            float v[8];
            load8(p.v.post, p.v.bf16, c[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] *= v[i];
        }
        if (p.v.gate) {
            float v[8];
            if (p.v.gate_per_token) load8((const uint16_t*)p.v.gate + (int64_t)t * p.H, true, c[j], v);
            else load8(p.v.gate, p.v.bf16, c[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] *= v[i];
        }
        float r[8];
        fill8(r, 0.0f);
        if (p.v.residual) {
            load8(p.v.residual + (int64_t)t * p.H, true, c[j], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] *= p.v.residual_scale;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[j][i] = there[j] ? fmaf(m[i], f[j][i], r[i]) : 0.0f;
            sum[0] = fmaf(f[j][i], f[j][i], sum[0]);
        }
        if (p.out && there[j]) reinterpret_cast<u32x4*>(p.out + (int64_t)t * p.H)[c[j]] = round8(f[j]);
    }
    if (!p.normed) return;
    block_sum<1>(sum, sums[1]);
    const float rr = inverse_rms(sum[0], p.H, p.v.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float v[8];
        load8(p.v.pre, p.v.bf16, c[j], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f[j][i] * rr;
        if (there[j]) reinterpret_cast<u32x4*>(p.normed + (int64_t)t * p.H)[c[j]] = round8(v);
    }
}

// ---- gradient -------------------------------------------------------------------------------------------------------
//
//   dr = dout + rr (dn pre - rhat mean(dn pre rhat)),  rhat = r rr        dpre = sum_t dn rhat
//   dres = rs dr        dgate = dr a (a gate per channel: summed over t)  da = gate dr
//   df = rf (da post - fhat mean(da post fhat)),       fhat = f rf        dpost = sum_t da fhat
//
// Workgroups walk over the tokens, each thread with the sums over t of its own channels; a second kernel adds the
// workgroups' sums up in their order.

struct GradParams {
    const uint16_t* dout;
    const uint16_t* dn;
    const void* f;
    bool f_bf16;
    NormVectors v;
    uint16_t* df;
    uint16_t* dres;
    uint16_t* dgate;     // per token; the sums over t go to part
    float* part;         // [blocks, 3, H]: post, pre, gate
    bool sum_post, sum_pre, sum_gate;
    int T, H;
};

// Rows of up to 8192 channels: one chunk a thread.  The vectors and their sums stay in registers for all of a workgroup's tokens (with
// fp32 f four of the 128 are spilled), and the next token's rows are under way while one is worked on.  With fp32 f, residual, both
// gradients and both outputs (14 bytes a channel) and a gate per channel 4096 rows of 7168 take 110 us (3.7 TB/s), 4096 of 4096 59 us, 4096
// of 2048 34 us (53 and 32 where the rows are still in the memory-side cache), with the sums over workgroups: three sums over a row,
// one after the other, leave memory idle in between, and a CU's registers hold one workgroup of 8192 channels.
// Taking the next token's first sum together with this one's last was slower (135 us: its rows are waited for earlier).
template <bool F_BF16>
__global__ __launch_bounds__(1024) void k_combine_norm_backward(GradParams p) {
    __shared__ float sums1[2][kMaxWaves][1], sums2[2][kMaxWaves][2], sums3[2][kMaxWaves][1];
    const int chunks = p.H / 8, c = (int)threadIdx.x < chunks ? (int)threadIdx.x : 0;
    const bool there = (int)threadIdx.x < chunks;
    const bool row_gate = p.v.gate && p.v.gate_per_token;
    float post[8], pre[8], gate[8], spost[8], spre[8], sgate[8];
    fill8(spost, 0.0f), fill8(spre, 0.0f), fill8(sgate, 0.0f);
    if (p.v.post) load8(p.v.post, p.v.bf16, c, post);
    else fill8(post, 1.0f);
    if (p.dn) load8(p.v.pre, p.v.bf16, c, pre);
    if (p.v.gate && !row_gate) load8(p.v.gate, p.v.bf16, c, gate);
    else fill8(gate, 1.0f);

    struct Rows {
        u32x4 f[F_BF16 ? 1 : 2], residual, dn, dout, gate;
    };
    auto load = [&](Rows& r, int64_t t) {
        const int64_t at = t * chunks + c;
#pragma unroll
        for (int i = 0; i < (F_BF16 ? 1 : 2); ++i) r.f[i] = reinterpret_cast<const u32x4*>(p.f)[F_BF16 ? at : at * 2 + i];
        if (p.v.residual) r.residual = reinterpret_cast<const u32x4*>(p.v.residual)[at];
        if (p.dn) r.dn = reinterpret_cast<const u32x4*>(p.dn)[at];
        if (p.dout) r.dout = reinterpret_cast<const u32x4*>(p.dout)[at];
        if (row_gate) r.gate = reinterpret_cast<const u32x4*>(p.v.gate)[at];
    };
    auto unpack = [](u32x4 q, float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(q[i]), v[2 * i + 1] = bf16hi(q[i]);
    };
    Rows next{};
    load(next, blockIdx.x);
    bool odd = false;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, odd = !odd) {
        const Rows row = next;
        if (t + gridDim.x < p.T) load(next, t + gridDim.x);
        const int64_t at = t * chunks + c;
        float f[8], r[8], d[8], dn[8], v[8];
        if constexpr (F_BF16) {
            unpack(row.f[0], f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = row.f[i / 4][i % 4];
                f[i] = __builtin_bit_cast(float, bits);
            }
        }
        float s1[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = there ? f[i] : 0.0f;
            s1[0] = fmaf(f[i], f[i], s1[0]);
        }
        float rf = 1.0f;
        if (p.v.post) {
            block_sum<1>(s1, sums1[odd]);
            rf = inverse_rms(s1[0], p.H, p.v.eps);
        }
        if (row_gate) unpack(row.gate, gate);
        fill8(r, 0.0f);
        if (p.v.residual) unpack(row.residual, r);
        fill8(d, 0.0f);
        if (p.dn) unpack(row.dn, dn);
        float s2[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r[i] = there ? fmaf(gate[i] * post[i] * rf, f[i], p.v.residual_scale * r[i]) : 0.0f;
            s2[0] = fmaf(r[i], r[i], s2[0]);
            if (p.dn) {
                d[i] = dn[i] * pre[i];
                s2[1] = fmaf(d[i], r[i], s2[1]);
            }
        }
        if (p.dn) {
            if (!there) s2[1] = 0.0f;
            block_sum<2>(s2, sums2[odd]);
            const float rr = inverse_rms(s2[0], p.H, p.v.eps), mean = rr * (s2[1] / (float)p.H);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float hat = r[i] * rr;
                spre[i] = fmaf(dn[i], hat, spre[i]);
                d[i] = rr * (d[i] - hat * mean);
            }
        }
        if (p.dout) {
            unpack(row.dout, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += v[i];
        }
        if (p.dres && there) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p.v.residual_scale * d[i];
            reinterpret_cast<u32x4*>(p.dres)[at] = round8(v);
        }
        float s3[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float hat = f[i] * rf;
            v[i] = d[i] * hat * post[i];
            sgate[i] += v[i];
            d[i] *= gate[i];      // da
            spost[i] = fmaf(d[i], hat, spost[i]);
            d[i] *= post[i];
            s3[0] = fmaf(d[i], f[i], s3[0]);
        }
        if (p.dgate && there) reinterpret_cast<u32x4*>(p.dgate)[at] = round8(v);
        if (!p.df) continue;
        if (p.v.post) {
            if (!there) s3[0] = 0.0f;
            block_sum<1>(s3, sums3[odd]);
            const float mean = rf * (s3[0] / (float)p.H);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rf * (d[i] - f[i] * rf * mean);
        }
        if (there) reinterpret_cast<u32x4*>(p.df)[at] = round8(d);
    }
    if (!there) return;
    f32x4* part = reinterpret_cast<f32x4*>(p.part + (int64_t)blockIdx.x * 3 * p.H) + 2 * c;
    auto put = [&](int which, const float (&v)[8]) {
        part[which * (p.H / 4)] = f32x4{v[0], v[1], v[2], v[3]};
        part[which * (p.H / 4) + 1] = f32x4{v[4], v[5], v[6], v[7]};
    };
    if (p.sum_post) put(0, spost);
    if (p.sum_pre) put(1, spre);
    if (p.sum_gate) put(2, sgate);
}

// Rows of more: a thread's chunks do not fit its registers, so each of the three sums over the row reads the chunks again (from L2) and
// works out what the one before it has.  The vectors' sums are added up in the workgroup's own place in memory.  1024 rows of 32768
// take 277 us (with a gate per channel 340), with eight chunks a thread in (spilled) registers 602; 1000 rows of 8200 74 and 84.
__global__ __launch_bounds__(1024) void k_combine_norm_backward_long(GradParams p) {
    __shared__ float sums1[kMaxWaves][1], sums2[kMaxWaves][2], sums3[kMaxWaves][1];
    const int chunks = p.H / 8;
    float* part = p.part + (int64_t)blockIdx.x * 3 * p.H;
    auto add = [&](int which, int c, const float* v, bool first) {
        f32x4* at = reinterpret_cast<f32x4*>(part + (int64_t)which * p.H) + 2 * c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 x{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            at[h] = first ? x : at[h] + x;
        }
    };
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const bool first = t == (int64_t)blockIdx.x;
        const int64_t row = t * p.H;
        float rf = 1.0f, rr = 1.0f, mean2 = 0.0f;
        auto load_f = [&](int c, float (&f)[8]) {
            load8(p.f_bf16 ? (const void*)((const uint16_t*)p.f + row) : (const void*)((const float*)p.f + row), p.f_bf16, c, f);
        };
        struct Chunk {
            float f[8], r[8], dn[8], post[8], gate[8], pre[8];
        };
        auto load = [&](int c, Chunk& x) {
            load_f(c, x.f);
            fill8(x.post, 1.0f), fill8(x.gate, 1.0f), fill8(x.r, 0.0f), fill8(x.dn, 0.0f), fill8(x.pre, 0.0f);
            if (p.v.post) load8(p.v.post, p.v.bf16, c, x.post);
            if (p.v.gate) {
                if (p.v.gate_per_token) load8((const uint16_t*)p.v.gate + row, true, c, x.gate);
                else load8(p.v.gate, p.v.bf16, c, x.gate);
            }
            if (p.v.residual) load8(p.v.residual + row, true, c, x.r);
            if (p.dn) {
                load8(p.v.pre, p.v.bf16, c, x.pre);
                load8(p.dn + row, true, c, x.dn);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x.r[i] = fmaf(x.gate[i] * x.post[i] * rf, x.f[i], p.v.residual_scale * x.r[i]);
        };
        // the gradient with respect to r
        auto grad = [&](int c, const Chunk& x, float (&d)[8]) {
            float dout[8];
            fill8(dout, 0.0f);
            if (p.dout) load8(p.dout + row, true, c, dout);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = p.dn ? fmaf(rr, x.dn[i] * x.pre[i] - x.r[i] * rr * mean2, dout[i]) : dout[i];
        };
        if (p.v.post) {
            float s1[1] = {0.0f};
            for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
                float f[8];
                load_f(c, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) s1[0] = fmaf(f[i], f[i], s1[0]);
            }
            block_sum<1>(s1, sums1);
            rf = inverse_rms(s1[0], p.H, p.v.eps);
        }
        if (p.dn) {
            float s2[2] = {0.0f, 0.0f};
            for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
                Chunk x;
                load(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s2[0] = fmaf(x.r[i], x.r[i], s2[0]);
                    s2[1] = fmaf(x.dn[i] * x.pre[i], x.r[i], s2[1]);
                }
            }
            block_sum<2>(s2, sums2);
            rr = inverse_rms(s2[0], p.H, p.v.eps), mean2 = rr * (s2[1] / (float)p.H);
        }
        float s3[1] = {0.0f};
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            Chunk x;
            float d[8], v[8];
            load(c, x);
            grad(c, x, d);
            if (p.sum_pre) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = x.dn[i] * (x.r[i] * rr);
                add(1, c, v, first);
            }
            if (p.dres) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = p.v.residual_scale * d[i];
                reinterpret_cast<u32x4*>(p.dres + row)[c] = round8(v);
            }
            if (p.dgate || p.sum_gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = d[i] * x.f[i] * rf * x.post[i];
                if (p.sum_gate) add(2, c, v, first);
                else reinterpret_cast<u32x4*>(p.dgate + row)[c] = round8(v);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float da = d[i] * x.gate[i];
                v[i] = da * x.f[i] * rf;
                s3[0] = fmaf(da * x.post[i], x.f[i], s3[0]);
            }
            if (p.sum_post) add(0, c, v, first);
        }
        if (!p.df) {
            __syncthreads();      // the sums' places are written again
            continue;
        }
        float mean3 = 0.0f;
        if (p.v.post) {
            block_sum<1>(s3, sums3);
            mean3 = rf * (s3[0] / (float)p.H);
        }
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            Chunk x;
            float d[8];
            load(c, x);
            grad(c, x, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] *= x.gate[i] * x.post[i];
                if (p.v.post) d[i] = rf * (d[i] - x.f[i] * rf * mean3);
            }
            reinterpret_cast<u32x4*>(p.df + row)[c] = round8(d);
        }
        __syncthreads();
    }
}

// out[which][h] = sum over the workgroups, 64 channels a workgroup, its waves a part of the rows each.
struct SumParams {
    const float* part;
    float* out[3];
    int blocks, H;
};
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * kWave) void k_sum_blocks(SumParams p) {
    __shared__ float sums[kSumWaves][kWave];
    float* out = p.out[blockIdx.y];
    if (!out) return;
    const int h = blockIdx.x * kWave + lane_id(), q = threadIdx.x / kWave, per = (p.blocks + kSumWaves - 1) / kSumWaves;
    const int b1 = (q + 1) * per < p.blocks ? (q + 1) * per : p.blocks;
    float sum = 0.0f;
    if (h < p.H) {
        const float* at = p.part + (int64_t)blockIdx.y * p.H + h;
#pragma unroll 16
        for (int b = q * per; b < b1; ++b) sum += at[(int64_t)b * 3 * p.H];
    }
    sums[q][lane_id()] = sum;
    __syncthreads();
    if (q > 0 || h >= p.H) return;
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i) sum += sums[i][lane_id()];
    out[h] = sum;
}

// Workgroups of the gradient, and rows of sums: a CU has room for one of 1024 threads, of more with fewer.
constexpr int kGradBlocks = 512;
int grad_blocks(int T, int hidden) {
    const int most = hidden > 4096 ? 256 : kGradBlocks;
    return T < most ? T : most;
}

int whole_waves(int threads) { return (threads + kWave - 1) / kWave * kWave; }

}  // namespace

hipError_t launch_combine_norm(const CombineNormArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const Params p{(const uint16_t*)a.y, a.topk_weights, a.slot, (const uint16_t*)a.bias, a.v, (uint16_t*)a.out, (uint16_t*)a.normed,
                   a.kept, a.T, a.hidden, a.K};
    const int chunks = a.hidden / 8;
    if (chunks <= 512) hipLaunchKernelGGL((k_combine_norm<1, 512>), grid_of(a.T), dim3(whole_waves(chunks)), 0, stream, p);
    else if (chunks <= 1024) hipLaunchKernelGGL((k_combine_norm<2, 512>), grid_of(a.T), dim3(whole_waves((chunks + 1) / 2)), 0, stream, p);
    else hipLaunchKernelGGL((k_combine_norm<4, 1024>), grid_of(a.T), dim3(whole_waves((chunks + 3) / 4)), 0, stream, p);
    return hipGetLastError();
}

size_t combine_norm_workspace_bytes(int T, int hidden) {
    const int blocks = grad_blocks(T, hidden);
    return (size_t)(blocks > 0 ? blocks : 1) * 3 * hidden * sizeof(float);
}

hipError_t launch_combine_norm_backward(const CombineNormBackwardArgs& a, hipStream_t stream) {
    const int blocks = grad_blocks(a.T, a.hidden);
    if (a.T > 0) {
        const bool gate_sum = a.grad_gate && !a.v.gate_per_token;
        const GradParams p{(const uint16_t*)a.grad_out, (const uint16_t*)a.grad_normed, a.f, a.f_bf16, a.v, (uint16_t*)a.grad_f,
                           (uint16_t*)a.grad_residual, gate_sum ? nullptr : (uint16_t*)a.grad_gate, (float*)a.workspace,
                           a.grad_post != nullptr, a.grad_pre != nullptr, gate_sum, a.T, a.hidden};
        const int chunks = a.hidden / 8;
        if (chunks > 1024) hipLaunchKernelGGL(k_combine_norm_backward_long, dim3(blocks), dim3(1024), 0, stream, p);
        else if (a.f_bf16)
            hipLaunchKernelGGL((k_combine_norm_backward<true>), dim3(blocks), dim3(whole_waves(chunks)), 0, stream, p);
        else
            hipLaunchKernelGGL((k_combine_norm_backward<false>), dim3(blocks), dim3(whole_waves(chunks)), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    float* gate = a.v.gate_per_token ? nullptr : (float*)a.grad_gate;
    if (!a.grad_post && !a.grad_pre && !gate) return hipSuccess;
    const SumParams s{(const float*)a.workspace, {a.grad_post, a.grad_pre, gate}, blocks, a.hidden};
    hipLaunchKernelGGL(k_sum_blocks, dim3((a.hidden + kWave - 1) / kWave, 3), dim3(kSumWaves * kWave), 0, stream, s);
    return hipGetLastError();
}

}  // namespace ep
