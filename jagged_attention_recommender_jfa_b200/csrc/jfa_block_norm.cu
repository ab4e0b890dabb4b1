// The norms before and after a block of a transformer, fused with the block's
// gate and residual scale, forward and backward.  For a row of D elements of
// the residual stream x, the block's output b and the gate u:
//   p = N_post(b)                      (RMS norm, LayerNorm or none)
//   y = x + s * act(u) * p             (the residual stream behind the block)
//   n = N_pre(y)                       (the next block's input)
// with N(v) = (v - mu) * r * gamma + beta, r = 1 / sqrt(mean((v - mu)^2) + eps),
// mu the mean for LayerNorm and 0 for the RMS norm.
//
// Backward, from dy and dn (gradients of y and n), with hat = (v - mu) * r:
//   through a norm: dv = r * (g - hat * mean(g * hat) - [LayerNorm] mean(g)), g = dN * gamma
//   d  = dy + (dn through N_pre)       = dx
//   dp = d * s * act(u);  db = dp through N_post
//   du = d * s * p * act'(u)
//   ds = sum_rows d * act(u) * p;  dgamma = sum_rows dN * hat;  dbeta = sum_rows dN
// The forward's values are recomputed from its inputs, so nothing has to be
// kept between the passes.  All arithmetic and sums are fp32; each result is
// rounded once.
//
// Bound: HBM.  Forward 3 tensors read and 2 written, backward 5 read and 3
// written.  A row is read once into the registers of a group of threads
// (eight elements per thread and tensor), and all statistics are taken from
// there; centred sums, so that a large mean costs no digits.  The parameter
// gradients are summed per thread over the rows a CTA takes, written as one
// partial row per CTA and summed in a fixed order by a second small kernel:
// no atomics, the same result every time.
#include "jfa_common.cuh"

namespace jfa {

namespace {

constexpr int kE = 8;              // elements per thread, chunk and tensor
constexpr int kMaxDim = 8192;
constexpr int kMaxParts = 1184;    // partial rows of the backward: 8 CTAs on each of 148 SMs

struct NormArgs {
    const void *x, *block, *gate;
    const float *scale, *post_gamma, *post_beta, *pre_gamma, *pre_beta;
    const void *dy, *dn;
    void *y, *n;                   // forward results
    void *dx, *dblock, *dgate;     // backward results
    float* parts;                  // [grid][5][D]
    int64_t rows;
    int D, post, pre, gate_kind;
    float eps;
};

// Group of threads that shares a row: G lanes of a warp (several rows per
// warp) or whole warps, then one row per CTA.
struct Group {
    int G, t;          // size, index in the group
    int warps;         // 1: within a warp
    float2* buf;       // [2][32]
    int turn;
    // sums of a and b over the group, in every thread
    __device__ __forceinline__ float2 sum(float a, float b) {
        const int width = G < 32 ? G : 32;
        for (int o = width >> 1; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (warps == 1) return make_float2(a, b);
        // alternating buffers: one barrier per sum
        float2* const p = buf + (turn & 1) * 32;
        ++turn;
        if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        float2 s = make_float2(0.f, 0.f);
        for (int w = 0; w < warps; ++w) {
            s.x += p[w].x;
            s.y += p[w].y;
        }
        return s;
    }
};

// Column of element u of chunk ch: eight consecutive columns per thread when
// rows are 16-byte aligned (VEC), else columns G apart, so that a warp's
// access is 32 consecutive elements.
template <bool VEC>
__device__ __forceinline__ int column(const Group& g, int ch, int u) {
    return VEC ? (ch * g.G + g.t) * kE + u : (ch * kE + u) * g.G + g.t;
}

template <bool VEC>
__device__ __forceinline__ void load_row(const float* p, const Group& g, int ch, int D, float (&f)[kE]) {
    if (VEC) {
        const int c = column<VEC>(g, ch, 0);
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (c < D) {
            a = __ldg(reinterpret_cast<const float4*>(p + c));
            b = __ldg(reinterpret_cast<const float4*>(p + c) + 1);
        }
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int c = column<VEC>(g, ch, u);
            f[u] = c < D ? __ldg(p + c) : 0.f;
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, const Group& g, int ch, int D, float (&f)[kE]) {
    if (VEC) {
        const int c = column<VEC>(g, ch, 0);
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (c < D) raw = __ldg(reinterpret_cast<const uint4*>(p + c));
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            f[2 * u] = __uint_as_float(w[u] << 16);
            f[2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int c = column<VEC>(g, ch, u);
            f[u] = c < D ? __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p + c)) << 16) : 0.f;
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void store_row(float* p, const Group& g, int ch, int D, const float (&f)[kE]) {
    if (VEC) {
        const int c = column<VEC>(g, ch, 0);
        if (c < D) {
            reinterpret_cast<float4*>(p + c)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4*>(p + c)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int c = column<VEC>(g, ch, u);
            if (c < D) p[c] = f[u];
        }
    }
}
template <bool VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const Group& g, int ch, int D, const float (&f)[kE]) {
    if (VEC) {
        const int c = column<VEC>(g, ch, 0);
        if (c < D) {
            uint4 o;
            __nv_bfloat162* w = reinterpret_cast<__nv_bfloat162*>(&o);
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = __floats2bfloat162_rn(f[2 * u], f[2 * u + 1]);
            *reinterpret_cast<uint4*>(p + c) = o;
        }
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) {
            const int c = column<VEC>(g, ch, u);
            if (c < D) p[c] = __float2bfloat16_rn(f[u]);
        }
    }
}
// A parameter vector's values (a constant where it is absent).
template <bool VEC>
__device__ __forceinline__ void load_param(const float* p, float absent, const Group& g, int ch, int D, float (&f)[kE]) {
    if (p) {
        load_row<VEC>(p, g, ch, D, f);
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) f[u] = absent;
    }
}

// 1 / (1 + e^-u): a large negative u gives 0.
__device__ __forceinline__ float sigmoid(float u) { return __fdividef(1.0f, 1.0f + expf(-u)); }

__device__ __forceinline__ float gate_value(int kind, float u) {
    if (kind == JFA_GATE_NONE) return 1.0f;
    if (kind == JFA_GATE_IDENTITY) return u;
    const float s = sigmoid(u);
    return kind == JFA_GATE_SILU ? u * s : s;
}

// Turns v into (v - mu) * r in place and returns r.
template <bool VEC, int NCH>
__device__ __forceinline__ float normalise(float (&v)[NCH][kE], int kind, Group& g, int D, float eps) {
    if (kind == JFA_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
            for (int u = 0; u < kE; ++u) s += v[ch][u];
        const float mu = g.sum(s, 0.f).x / (float)D;   // exact for a constant row of exact sum
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
            for (int u = 0; u < kE; ++u) v[ch][u] = column<VEC>(g, ch, u) < D ? v[ch][u] - mu : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
        for (int u = 0; u < kE; ++u) q = fmaf(v[ch][u], v[ch][u], q);
    const float r = 1.0f / sqrtf(g.sum(q, 0.f).x / (float)D + eps);
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
        for (int u = 0; u < kE; ++u) v[ch][u] *= r;
    return r;
}

__device__ __forceinline__ Group make_group(int G, float2* buf) {
    Group g;
    g.G = G;
    g.t = threadIdx.x % G;
    g.warps = G <= 32 ? 1 : G / 32;
    g.buf = buf;
    g.turn = 0;
    return g;
}

// One row per group.  Threads of rows behind the last take part in the
// shuffles with zeros and store nothing.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) block_norm_fwd(const NormArgs a, int G) {
    __shared__ float2 buf[64];
    Group g = make_group(G, buf);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
    const bool live = row < a.rows;
    const int D = live ? a.D : 0;   // a dead row reads and writes no column
    const int64_t at = row * a.D;
    float x[1][kE], b[1][kE], u[kE], w[kE], v[kE];
    load_row<VEC>(reinterpret_cast<const T*>(a.block) + at, g, 0, D, b[0]);
    load_row<VEC>(reinterpret_cast<const T*>(a.x) + at, g, 0, D, x[0]);
    if (a.gate_kind != JFA_GATE_NONE) load_row<VEC>(reinterpret_cast<const T*>(a.gate) + at, g, 0, D, u);
    if (a.post != JFA_NORM_NONE) {
        normalise<VEC, 1>(b, a.post, g, a.D, a.eps);
        load_param<VEC>(a.post_gamma, 1.f, g, 0, a.D, w);
        load_param<VEC>(a.post_beta, 0.f, g, 0, a.D, v);
#pragma unroll
        for (int i = 0; i < kE; ++i) b[0][i] = fmaf(b[0][i], w[i], v[i]);
    }
    load_param<VEC>(a.scale, 1.f, g, 0, a.D, w);
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const float k = a.gate_kind != JFA_GATE_NONE ? w[i] * gate_value(a.gate_kind, u[i]) : w[i];
        x[0][i] = fmaf(k, b[0][i], x[0][i]);
    }
    store_row<VEC>(reinterpret_cast<T*>(a.y) + at, g, 0, D, x[0]);
    if (a.pre == JFA_NORM_NONE) return;
    normalise<VEC, 1>(x, a.pre, g, a.D, a.eps);
    load_param<VEC>(a.pre_gamma, 1.f, g, 0, a.D, w);
    load_param<VEC>(a.pre_beta, 0.f, g, 0, a.D, v);
#pragma unroll
    for (int i = 0; i < kE; ++i) x[0][i] = fmaf(x[0][i], w[i], v[i]);
    store_row<VEC>(reinterpret_cast<T*>(a.n) + at, g, 0, D, x[0]);
}

enum { Q_SCALE = 0, Q_POST_GAMMA, Q_POST_BETA, Q_PRE_GAMMA, Q_PRE_BETA, Q_COUNT };

// The sums over rows: in registers for one chunk, in shared memory (each
// thread its own columns) for two, where registers run out.
template <int NCH>
struct Sums;
template <>
struct Sums<1> {
    float v[Q_COUNT][kE];
    __device__ void init(float*, const Group&, int) {
#pragma unroll
        for (int q = 0; q < Q_COUNT; ++q)
#pragma unroll
            for (int u = 0; u < kE; ++u) v[q][u] = 0.f;
    }
    __device__ __forceinline__ void add(int q, int, int u, float x) { v[q][u] += x; }
    __device__ __forceinline__ float get(int q, int, int u) const { return v[q][u]; }
};
template <>
struct Sums<2> {
    float* mine;
    int stride;
    __device__ void init(float* smem, const Group& g, int) {
        mine = smem + g.t;
        stride = g.G;
        for (int i = 0; i < Q_COUNT * 2 * kE; ++i) mine[i * stride] = 0.f;
    }
    __device__ __forceinline__ void add(int q, int ch, int u, float x) { mine[((q * 2 + ch) * kE + u) * stride] += x; }
    __device__ __forceinline__ float get(int q, int ch, int u) const { return mine[((q * 2 + ch) * kE + u) * stride]; }
};

// A CTA takes rows blockIdx, blockIdx + gridDim, ... (in units of its groups).
template <typename T, bool VEC, int NCH>
__global__ void __launch_bounds__(512) block_norm_bwd(const NormArgs a, int G) {
    extern __shared__ float smem[];   // NCH == 2: the sums; small groups: the CTA's reduction
    __shared__ float2 buf[64];
    Group g = make_group(G, buf);
    Sums<NCH> sums;
    sums.init(smem, g, a.D);
    const int groups = blockDim.x / G;
    const float inv_d = 1.0f / (float)a.D;
    for (int64_t base = (int64_t)blockIdx.x * groups; base < a.rows; base += (int64_t)gridDim.x * groups) {
        const int64_t row = base + threadIdx.x / G;
        const int D = row < a.rows ? a.D : 0;
        const int64_t at = row * a.D;
        float b[NCH][kE], y[NCH][kE], u[NCH][kE], d[NCH][kE], dn[NCH][kE];
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            load_row<VEC>(reinterpret_cast<const T*>(a.block) + at, g, ch, D, b[ch]);
            load_row<VEC>(reinterpret_cast<const T*>(a.x) + at, g, ch, D, y[ch]);
            if (a.gate_kind != JFA_GATE_NONE) load_row<VEC>(reinterpret_cast<const T*>(a.gate) + at, g, ch, D, u[ch]);
            load_row<VEC>(reinterpret_cast<const T*>(a.dy) + at, g, ch, D, d[ch]);
            if (a.pre != JFA_NORM_NONE) load_row<VEC>(reinterpret_cast<const T*>(a.dn) + at, g, ch, D, dn[ch]);
        }
        float rb = 1.f;
        if (a.post != JFA_NORM_NONE) rb = normalise<VEC, NCH>(b, a.post, g, a.D, a.eps);   // b: hat of the block
        float gate[NCH][kE];   // act(u)
        if (a.pre != JFA_NORM_NONE) {
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
                float s[kE], pg[kE], pb[kE];
                load_param<VEC>(a.scale, 1.f, g, ch, a.D, s);
                load_param<VEC>(a.post_gamma, 1.f, g, ch, a.D, pg);
                load_param<VEC>(a.post_beta, 0.f, g, ch, a.D, pb);
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    gate[ch][i] = a.gate_kind != JFA_GATE_NONE ? gate_value(a.gate_kind, u[ch][i]) : 1.f;
                    y[ch][i] = fmaf(s[i] * gate[ch][i], fmaf(b[ch][i], pg[i], pb[i]), y[ch][i]);
                }
            }
            const float ry = normalise<VEC, NCH>(y, a.pre, g, a.D, a.eps);   // y: hat of y
            float c1 = 0.f, c2 = 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch) {
                float w[kE];
                load_param<VEC>(a.pre_gamma, 1.f, g, ch, a.D, w);
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    sums.add(Q_PRE_GAMMA, ch, i, dn[ch][i] * y[ch][i]);
                    sums.add(Q_PRE_BETA, ch, i, dn[ch][i]);
                    dn[ch][i] *= w[i];
                    c1 = fmaf(dn[ch][i], y[ch][i], c1);
                    c2 += dn[ch][i];
                }
            }
            const float2 c = g.sum(c1, c2);
            c1 = c.x * inv_d;
            c2 = a.pre == JFA_NORM_LAYER ? c.y * inv_d : 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int i = 0; i < kE; ++i) d[ch][i] = fmaf(ry, dn[ch][i] - fmaf(y[ch][i], c1, c2), d[ch][i]);
        } else {
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int i = 0; i < kE; ++i) gate[ch][i] = a.gate_kind != JFA_GATE_NONE ? gate_value(a.gate_kind, u[ch][i]) : 1.f;
        }
        // d is dx; with the block: dp, the gate's gradient and the sums
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            store_row<VEC>(reinterpret_cast<T*>(a.dx) + at, g, ch, D, d[ch]);
            float s[kE], pg[kE], pb[kE];
            load_param<VEC>(a.scale, 1.f, g, ch, a.D, s);
            load_param<VEC>(a.post_gamma, 1.f, g, ch, a.D, pg);
            load_param<VEC>(a.post_beta, 0.f, g, ch, a.D, pb);
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                if (column<VEC>(g, ch, i) >= D) {   // columns behind the row: no part in any sum
                    d[ch][i] = 0.f;
                    b[ch][i] = 0.f;
                }
                const float p = fmaf(b[ch][i], pg[i], pb[i]);
                sums.add(Q_SCALE, ch, i, d[ch][i] * gate[ch][i] * p);
                const float ds = d[ch][i] * s[i];
                const float dp = ds * gate[ch][i];
                if (a.gate_kind == JFA_GATE_IDENTITY) {
                    u[ch][i] = ds * p;
                } else if (a.gate_kind != JFA_GATE_NONE) {
                    const float v = u[ch][i], q = sigmoid(v);
                    u[ch][i] = ds * p * (a.gate_kind == JFA_GATE_SILU ? q * fmaf(v, 1.0f - q, 1.0f) : q * (1.0f - q));
                }
                sums.add(Q_POST_GAMMA, ch, i, dp * b[ch][i]);
                sums.add(Q_POST_BETA, ch, i, dp);
                d[ch][i] = dp * pg[i];
                c1 = fmaf(d[ch][i], b[ch][i], c1);
                c2 += d[ch][i];
            }
            if (a.gate_kind != JFA_GATE_NONE) store_row<VEC>(reinterpret_cast<T*>(a.dgate) + at, g, ch, D, u[ch]);
        }
        if (a.post != JFA_NORM_NONE) {
            const float2 c = g.sum(c1, c2);
            c1 = c.x * inv_d;
            c2 = a.post == JFA_NORM_LAYER ? c.y * inv_d : 0.f;
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int i = 0; i < kE; ++i) d[ch][i] = rb * (d[ch][i] - fmaf(b[ch][i], c1, c2));
        }
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) store_row<VEC>(reinterpret_cast<T*>(a.dblock) + at, g, ch, D, d[ch]);
    }
    // this CTA's partial row of each sum
    float* const part = a.parts + (int64_t)blockIdx.x * Q_COUNT * a.D;
    if (groups == 1) {
#pragma unroll
        for (int q = 0; q < Q_COUNT; ++q)
#pragma unroll
            for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const int c = column<VEC>(g, ch, i);
                    if (c < a.D) part[q * a.D + c] = sums.get(q, ch, i);
                }
    } else if (NCH == 1) {
        // the groups' sums in group order, through shared memory [groups][G * 8]
        const int width = G * kE;
#pragma unroll
        for (int q = 0; q < Q_COUNT; ++q) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kE; ++i) smem[(threadIdx.x / G) * width + column<VEC>(g, 0, i)] = sums.get(q, 0, i);
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
                float s = 0.f;
                for (int k = 0; k < groups; ++k) s += smem[k * width + c];
                part[q * a.D + c] = s;
            }
        }
    }
}

struct SumOut {
    float* out[Q_COUNT];
};

// out[q][c] = sum over the partial rows, in order within eight interleaved
// strands that are then added in order.
__global__ void __launch_bounds__(256) block_norm_sum(const float* __restrict__ parts, int n, int D, SumOut o) {
    __shared__ float s_part[8][33];
    float* const out = o.out[blockIdx.y];
    if (!out) return;
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < D)
        for (int p = strand; p < n; p += 8) s += parts[((int64_t)p * Q_COUNT + blockIdx.y) * D + c];
    s_part[strand][lane] = s;
    __syncthreads();
    if (strand == 0 && c < D) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += s_part[k][lane];
        out[c] = s;
    }
}

// Threads per row: one per eight elements, a power of two within a warp,
// whole warps above.
int group_size(int D) {
    const int need = (D + kE - 1) / kE;
    if (need > 32) return (need + 31) / 32 * 32;
    int G = 1;
    while (G < need) G *= 2;
    return G;
}
constexpr int kSmallThreads = 128;   // CTA size for rows within a warp

struct BwdShape {
    int G, threads, nch, grid;
    size_t smem;
};
BwdShape bwd_shape(int64_t rows, int D) {
    BwdShape s{};
    s.nch = D > 512 * kE ? 2 : 1;
    s.G = group_size((D + s.nch - 1) / s.nch);
    s.threads = s.G <= 32 ? kSmallThreads : s.G;
    const int groups = s.threads / s.G;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // about 112 registers a thread: 512 threads fill an SM
    int64_t cap = (int64_t)sms * (512 / s.threads > 0 ? 512 / s.threads : 1);
    if (cap > kMaxParts) cap = kMaxParts;
    const int64_t need = (rows + groups - 1) / groups;
    s.grid = (int)(need < cap ? need : cap);
    s.smem = s.nch == 2 ? sizeof(float) * Q_COUNT * 2 * kE * s.G : (groups > 1 ? sizeof(float) * s.threads * kE : 0);
    return s;
}

jfa_status check_desc(const jfa_block_norm* d, const char* who) {
    if (!d) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: descriptor is NULL", who);
    if (d->rows < 0 || d->rows >= (int64_t)1 << 31 || d->dim < 1)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: rows in [0, 2^31) and dim >= 1", who);
    if (d->dim > kMaxDim) return set_last_error(JFA_ERR_UNSUPPORTED, "%s: dim %d > %d", who, d->dim, kMaxDim);
    if (d->dtype != JFA_F32 && d->dtype != JFA_BF16)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: dtype must be JFA_F32 or JFA_BF16", who);
    for (int k : {(int)d->post_norm, (int)d->pre_norm})
        if (k != JFA_NORM_NONE && k != JFA_NORM_RMS && k != JFA_NORM_LAYER)
            return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: bad norm kind %d", who, k);
    if (d->gate != JFA_GATE_NONE && d->gate != JFA_GATE_IDENTITY && d->gate != JFA_GATE_SILU && d->gate != JFA_GATE_SIGMOID)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: bad gate kind %d", who, (int)d->gate);
    if (!(d->eps > 0.f) || !(d->eps <= 3.4e38f))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: eps must be positive and finite", who);
    return JFA_OK;
}

// Parameters that the descriptor's norms do not have are refused rather than
// ignored.
jfa_status check_params(const jfa_block_norm* d, const void* gate, const float* scale, const float* post_gamma,
                        const float* post_beta, const float* pre_gamma, const float* pre_beta, const char* who) {
    if ((d->post_norm == JFA_NORM_NONE && post_gamma) || (d->post_norm != JFA_NORM_LAYER && post_beta) ||
        (d->pre_norm == JFA_NORM_NONE && pre_gamma) || (d->pre_norm != JFA_NORM_LAYER && pre_beta))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: a gamma needs a norm, a beta a LayerNorm", who);
    if (d->gate == JFA_GATE_NONE && gate)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: gate given for JFA_GATE_NONE", who);
    if (((uintptr_t)scale | (uintptr_t)post_gamma | (uintptr_t)post_beta | (uintptr_t)pre_gamma | (uintptr_t)pre_beta) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: parameters must be 16-byte aligned", who);
    return JFA_OK;
}

template <typename T>
cudaError_t fwd_launch(const NormArgs& a, cudaStream_t st) {
    const int G = group_size(a.D), threads = G <= 32 ? kSmallThreads : G;
    const int64_t grid = (a.rows + threads / G - 1) / (threads / G);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    prof_begin(st);
    if (a.D % kE == 0) block_norm_fwd<T, true><<<(unsigned)grid, threads, 0, st>>>(a, G);
    else block_norm_fwd<T, false><<<(unsigned)grid, threads, 0, st>>>(a, G);
    prof_end(st, K_BLOCK_NORM_FWD);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_launch(const NormArgs& a, const BwdShape& s, cudaStream_t st) {
    const bool vec = a.D % kE == 0;
    void (*kern)(NormArgs, int) =
        s.nch == 2 ? (vec ? block_norm_bwd<T, true, 2> : block_norm_bwd<T, false, 2>)
                   : (vec ? block_norm_bwd<T, true, 1> : block_norm_bwd<T, false, 1>);
    if (s.smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.smem);
        if (e != cudaSuccess) return e;
    }
    prof_begin(st);
    kern<<<s.grid, s.threads, s.smem, st>>>(a, s.G);
    prof_end(st, K_BLOCK_NORM_BWD);
    return cudaGetLastError();
}

}  // namespace
}  // namespace jfa

extern "C" {

size_t jfa_block_norm_workspace_bytes(const jfa_block_norm* desc) {
    if (jfa::check_desc(desc, "block_norm_workspace_bytes") != JFA_OK) return 0;
    const int64_t rows = desc->rows < jfa::kMaxParts ? desc->rows : jfa::kMaxParts;
    return jfa::align256(sizeof(float) * jfa::Q_COUNT * (size_t)(rows > 0 ? rows : 1) * (size_t)desc->dim);
}

jfa_status jfa_block_norm_forward(const jfa_block_norm* desc, const void* x, const void* block, const void* gate,
                                  const float* scale, const float* post_gamma, const float* post_beta,
                                  const float* pre_gamma, const float* pre_beta, void* y, void* n,
                                  jfa_stream_t stream) {
    using namespace jfa;
    const char* who = "block_norm_forward";
    jfa_status s = check_desc(desc, who);
    if (s != JFA_OK) return s;
    if (desc->rows == 0) return JFA_OK;
    if (!x || !block || !y || (desc->gate != JFA_GATE_NONE && !gate) || (desc->pre_norm != JFA_NORM_NONE && !n))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: NULL tensor", who);
    if (((uintptr_t)x | (uintptr_t)block | (uintptr_t)gate | (uintptr_t)y | (uintptr_t)n) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: tensors must be 16-byte aligned", who);
    if ((s = check_params(desc, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, who)) != JFA_OK) return s;
    NormArgs a{};
    a.x = x; a.block = block; a.gate = gate; a.scale = scale;
    a.post_gamma = post_gamma; a.post_beta = post_beta; a.pre_gamma = pre_gamma; a.pre_beta = pre_beta;
    a.y = y; a.n = n; a.rows = desc->rows; a.D = desc->dim;
    a.post = desc->post_norm; a.pre = desc->pre_norm; a.gate_kind = desc->gate; a.eps = desc->eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = desc->dtype == JFA_F32 ? fwd_launch<float>(a, st) : fwd_launch<__nv_bfloat16>(a, st);
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return JFA_OK;
}

jfa_status jfa_block_norm_backward(const jfa_block_norm* desc, const void* x, const void* block, const void* gate,
                                   const float* scale, const float* post_gamma, const float* post_beta,
                                   const float* pre_gamma, const float* pre_beta, const void* dy, const void* dn,
                                   void* dx, void* dblock, void* dgate, float* dscale, float* dpost_gamma,
                                   float* dpost_beta, float* dpre_gamma, float* dpre_beta, void* workspace,
                                   size_t ws_bytes, jfa_stream_t stream) {
    using namespace jfa;
    const char* who = "block_norm_backward";
    jfa_status s = check_desc(desc, who);
    if (s != JFA_OK) return s;
    if ((s = check_params(desc, gate, scale, post_gamma, post_beta, pre_gamma, pre_beta, who)) != JFA_OK) return s;
    if ((s = check_params(desc, nullptr, dscale, dpost_gamma, dpost_beta, dpre_gamma, dpre_beta, who)) != JFA_OK) return s;
    if (!workspace || ((uintptr_t)workspace & 15))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: workspace must be non-NULL and 16-byte aligned", who);
    const size_t need = jfa_block_norm_workspace_bytes(desc);
    if (ws_bytes < need) return set_last_error(JFA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
    const bool gated = desc->gate != JFA_GATE_NONE, pre = desc->pre_norm != JFA_NORM_NONE;
    if (desc->rows > 0 && (!x || !block || !dy || !dx || !dblock || (gated && (!gate || !dgate)) || (pre && !dn)))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: NULL tensor", who);
    if (((uintptr_t)x | (uintptr_t)block | (uintptr_t)gate | (uintptr_t)dy | (uintptr_t)dn | (uintptr_t)dx |
         (uintptr_t)dblock | (uintptr_t)dgate) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: tensors must be 16-byte aligned", who);
    NormArgs a{};
    a.x = x; a.block = block; a.gate = gate; a.scale = scale;
    a.post_gamma = post_gamma; a.post_beta = post_beta; a.pre_gamma = pre_gamma; a.pre_beta = pre_beta;
    a.dy = dy; a.dn = dn; a.dx = dx; a.dblock = dblock; a.dgate = dgate;
    a.parts = reinterpret_cast<float*>(workspace);
    a.rows = desc->rows; a.D = desc->dim;
    a.post = desc->post_norm; a.pre = desc->pre_norm; a.gate_kind = desc->gate; a.eps = desc->eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const BwdShape shape = bwd_shape(a.rows, a.D);
    cudaError_t e = cudaSuccess;
    if (a.rows > 0) e = desc->dtype == JFA_F32 ? bwd_launch<float>(a, shape, st) : bwd_launch<__nv_bfloat16>(a, shape, st);
    if (e == cudaSuccess && (dscale || dpost_gamma || dpost_beta || dpre_gamma || dpre_beta)) {
        SumOut o{{dscale, dpost_gamma, dpost_beta, dpre_gamma, dpre_beta}};
        prof_begin(st);
        block_norm_sum<<<dim3((a.D + 31) / 32, Q_COUNT), 256, 0, st>>>(a.parts, a.rows > 0 ? shape.grid : 0, a.D, o);
        prof_end(st, K_BLOCK_NORM_SUM);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return JFA_OK;
}

}  // extern "C"
