// ep_norm.hip -- the combine with the norms around a block, and its gradient.
//
//   f = sum_k w[t,k] y[slot(t,k)] + bias[t]      or the block's output itself
//   a = f rf post,  rf = 1 / sqrt(mean f^2 + eps)
//   r = rs residual + gate a                     -> out
//   n = r rr pre,   rr = 1 / sqrt(mean r^2 + eps)   -> normed
//
// One workgroup per token, a thread holds V 16-byte chunks of the row in registers from the first load to the last store:
// every row of y is read once, out and normed are written once, and what a norm needs of the whole row is one sum over
// the workgroup (lanes by register exchange, waves through LDS, in a fixed order).
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

template <int V, int THREADS, bool IN_MEMORY>
__global__ __launch_bounds__(THREADS) void k_combine_norm_backward(GradParams p) {
    __shared__ float sums1[2][kMaxWaves][1], sums2[2][kMaxWaves][2], sums3[2][kMaxWaves][1];
    const int chunks = p.H / 8;
    int c[V];
    bool there[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        c[j] = j * (int)blockDim.x + (int)threadIdx.x;
        there[j] = c[j] < chunks;
        c[j] = there[j] ? c[j] : 0;
    }
    constexpr int kHeld = IN_MEMORY ? 1 : V;
    float spost[kHeld][8], spre[kHeld][8], sgate[kHeld][8];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) fill8(spost[j], 0.0f), fill8(spre[j], 0.0f), fill8(sgate[j], 0.0f);
    float* part = p.part + (int64_t)blockIdx.x * 3 * p.H;
    // adds v to this thread's sums of chunk j
    auto add = [&](float (&held)[kHeld][8], int which, int j, const float* v, bool first) {
        if constexpr (IN_MEMORY) {
            if (!there[j]) return;
            f32x4* at = reinterpret_cast<f32x4*>(part + (int64_t)which * p.H) + 2 * c[j];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 x{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
                at[h] = first ? x : at[h] + x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) held[j][i] += v[i];
        }
    };
    bool odd = false;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, odd = !odd) {
        const bool first = t == (int64_t)blockIdx.x;
        const int64_t row = t * p.H;
        float f[V][8], r[V][8], d[V][8];
        float s1[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            load8(p.f_bf16 ? (const void*)((const uint16_t*)p.f + row) : (const void*)((const float*)p.f + row), p.f_bf16, c[j], f[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[j][i] = there[j] ? f[j][i] : 0.0f;
                s1[0] = fmaf(f[j][i], f[j][i], s1[0]);
            }
        }
        float rf = 1.0f;
        if (p.v.post) {
            block_sum<1>(s1, sums1[odd]);
            rf = inverse_rms(s1[0], p.H, p.v.eps);
        }
        auto load_gate = [&](int j, float* v) {
            if (!p.v.gate) fill8(v, 1.0f);
            else if (p.v.gate_per_token) load8((const uint16_t*)p.v.gate + row, true, c[j], v);
            else load8(p.v.gate, p.v.bf16, c[j], v);
        };
        float s2[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float post[8], gate[8], pre[8], dn[8];
            if (p.v.post) load8(p.v.post, p.v.bf16, c[j], post);
            else fill8(post, 1.0f);
            load_gate(j, gate);
            fill8(r[j], 0.0f);
            if (p.v.residual) load8(p.v.residual + row, true, c[j], r[j]);
            fill8(d[j], 0.0f);
            if (p.dn) {
                load8(p.v.pre, p.v.bf16, c[j], pre);
                load8(p.dn + row, true, c[j], dn);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                r[j][i] = there[j] ? fmaf(gate[i] * post[i] * rf, f[j][i], p.v.residual_scale * r[j][i]) : 0.0f;
                s2[0] = fmaf(r[j][i], r[j][i], s2[0]);
                if (p.dn) {
                    d[j][i] = dn[i] * pre[i];
                    s2[1] = fmaf(d[j][i], r[j][i], s2[1]);
                }
            }
        }
        if (p.dn) {
            block_sum<2>(s2, sums2[odd]);
            const float rr = inverse_rms(s2[0], p.H, p.v.eps), mean = rr * (s2[1] / (float)p.H);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (p.sum_pre) {
                    float dn[8];
                    load8(p.dn + row, true, c[j], dn);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dn[i] *= r[j][i] * rr;
                    add(spre, 1, j, dn, first);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] = rr * (d[j][i] - r[j][i] * rr * mean);
            }
        }
        float s3[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float dout[8], post[8], gate[8], v[8];
            if (p.dout) {
                load8(p.dout + row, true, c[j], dout);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] += dout[i];
            }
            if (p.dres && there[j]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = p.v.residual_scale * d[j][i];
                reinterpret_cast<u32x4*>(p.dres + row)[c[j]] = round8(v);
            }
            if (p.v.post) load8(p.v.post, p.v.bf16, c[j], post);
            else fill8(post, 1.0f);
            load_gate(j, gate);
            if (p.dgate || p.sum_gate) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = d[j][i] * f[j][i] * rf * post[i];
                if (p.sum_gate) add(sgate, 2, j, v, first);
                else if (there[j]) reinterpret_cast<u32x4*>(p.dgate + row)[c[j]] = round8(v);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) d[j][i] *= gate[i];      // da
            if (p.sum_post) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = d[j][i] * f[j][i] * rf;
                add(spost, 0, j, v, first);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[j][i] *= post[i];
                s3[0] = fmaf(d[j][i], f[j][i], s3[0]);
            }
        }
        if (!p.df) continue;
        if (p.v.post) {
            block_sum<1>(s3, sums3[odd]);
            const float mean = rf * (s3[0] / (float)p.H);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) d[j][i] = rf * (d[j][i] - f[j][i] * rf * mean);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (there[j]) reinterpret_cast<u32x4*>(p.df + row)[c[j]] = round8(d[j]);
    }
    if constexpr (!IN_MEMORY) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!there[j]) continue;
#pragma unroll
            for (int which = 0; which < 3; ++which) {
                if (!(which == 0 ? p.sum_post : which == 1 ? p.sum_pre : p.sum_gate)) continue;
                const float* v = which == 0 ? spost[j] : which == 1 ? spre[j] : sgate[j];
                f32x4* at = reinterpret_cast<f32x4*>(part + (int64_t)which * p.H) + 2 * c[j];
                at[0] = f32x4{v[0], v[1], v[2], v[3]};
                at[1] = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
    }
}

// out[which][h] = sum over the workgroups, 64 channels a workgroup, its four waves a quarter of the rows each.
struct SumParams {
    const float* part;
    float* out[3];
    int blocks, H;
};
__global__ __launch_bounds__(256) void k_sum_blocks(SumParams p) {
    __shared__ float quarter[4][kWave];
    float* out = p.out[blockIdx.y];
    if (!out) return;
    const int h = blockIdx.x * kWave + lane_id(), q = threadIdx.x / kWave, per = (p.blocks + 3) / 4;
    const int b1 = (q + 1) * per < p.blocks ? (q + 1) * per : p.blocks;
    float sum = 0.0f;
    if (h < p.H) {
        const float* at = p.part + (int64_t)blockIdx.y * p.H + h;
#pragma unroll 8
        for (int b = q * per; b < b1; ++b) sum += at[(int64_t)b * 3 * p.H];
    }
    quarter[q][lane_id()] = sum;
    __syncthreads();
    if (q == 0 && h < p.H) out[h] = (quarter[0][lane_id()] + quarter[1][lane_id()]) + (quarter[2][lane_id()] + quarter[3][lane_id()]);
}

constexpr int kGradBlocks = 512;

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
    return (size_t)(T < kGradBlocks ? (T > 0 ? T : 1) : kGradBlocks) * 3 * hidden * sizeof(float);
}

hipError_t launch_combine_norm_backward(const CombineNormBackwardArgs& a, hipStream_t stream) {
    const int blocks = a.T < kGradBlocks ? a.T : kGradBlocks;
    if (a.T > 0) {
        const bool gate_sum = a.grad_gate && !a.v.gate_per_token;
        const GradParams p{(const uint16_t*)a.grad_out, (const uint16_t*)a.grad_normed, a.f, a.f_bf16, a.v, (uint16_t*)a.grad_f,
                           (uint16_t*)a.grad_residual, gate_sum ? nullptr : (uint16_t*)a.grad_gate, (float*)a.workspace,
                           a.grad_post != nullptr, a.grad_pre != nullptr, gate_sum, a.T, a.hidden};
        const int chunks = a.hidden / 8;
        if (chunks <= 512)
            hipLaunchKernelGGL((k_combine_norm_backward<1, 512, false>), dim3(blocks), dim3(whole_waves(chunks)), 0, stream, p);
        else if (chunks <= 1024)
            hipLaunchKernelGGL((k_combine_norm_backward<2, 512, false>), dim3(blocks), dim3(whole_waves((chunks + 1) / 2)), 0, stream, p);
        else
            hipLaunchKernelGGL((k_combine_norm_backward<4, 1024, true>), dim3(blocks), dim3(whole_waves((chunks + 3) / 4)), 0, stream, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    float* gate = a.v.gate_per_token ? nullptr : (float*)a.grad_gate;
    if (!a.grad_post && !a.grad_pre && !gate) return hipSuccess;
    const SumParams s{(const float*)a.workspace, {a.grad_post, a.grad_pre, gate}, blocks, a.hidden};
    hipLaunchKernelGGL(k_sum_blocks, dim3((a.hidden + kWave - 1) / kWave, 3), dim3(256), 0, stream, s);
    return hipGetLastError();
}

}  // namespace ep
