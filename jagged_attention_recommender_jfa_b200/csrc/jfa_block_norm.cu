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
// With S1 = sum_rows d * act(u) * hat and S2 = sum_rows d * act(u) of the
// block's norm the parameter gradients are dgamma_post = s S1, dbeta_post = s S2
// and ds = gamma S1 + beta S2, so two sums (one without a LayerNorm) serve all
// three; the same pair without the gate serves N_pre's.
//
// Bound: HBM.  Forward 3 tensors read and 2 written, backward 5 read and 3
// written.  Persistent groups of threads take rows in turn, a row's values in
// registers, one 16-byte vector per thread, tensor and chunk; the next row's
// vectors are loaded before the current row is worked on (in the backward where
// a thread has one vector per tensor: more leave no registers for it), and the
// parameters wait in shared memory where they fit (Params, kBwdParamsInSmem).
// Statistics are taken from the registers: centred sums, so
// that a large mean costs no digits.  Parameter gradients are summed per thread
// over the group's rows, written as one partial row per CTA and summed in a
// fixed order by a second small kernel: no atomics, the same result every time.
//
// Rows of any width go in aligned vectors: a row that starts s elements behind
// a 16-byte boundary is taken from that boundary on, the elements of its
// neighbours masked.  s repeats every 16 / sizeof(element) rows, and a group's
// rows are a multiple of that apart, so that a thread keeps the same columns
// (and its parameters and sums) for all its rows.
#include "jfa_common.cuh"
#include "jfa_sm100.cuh"

namespace jfa {

namespace {

constexpr int kMaxDim = 8192;
constexpr int kMaxThreads = 512;   // per row; wider rows take several vectors per thread
constexpr int kSmallThreads = 128; // CTA size for rows within a warp
constexpr int kMaxParts = 1184;    // partial rows of the backward: 8 CTAs on each of 148 SMs

struct NormArgs {
    const void *x, *block, *gate;
    const float *scale, *post_gamma, *post_beta, *pre_gamma, *pre_beta;
    const void *dy, *dn;
    void *y, *n;                   // forward results
    void *dx, *dblock, *dgate;     // backward results
    float* parts;                  // [grid][Q_COUNT][D]
    int64_t rows;
    int D, post, pre, gate_kind;
    float eps;
};

// Group of threads that shares a row: G lanes of a warp (several rows per
// warp) or whole warps, then one row per CTA.
constexpr int kMostSums = 3;
struct GroupBuf {
    float4 v[2][kMostSums][kMaxThreads / 128];   // [turn][which sum], a float per warp
};
struct Group {
    int G, t;          // size, index in the group
    int warps;         // 1: within a warp
    GroupBuf* buf;
    int turn;
    __device__ __forceinline__ Group(int G_, GroupBuf* b) : G(G_), t(threadIdx.x % G_), warps(G_ <= 32 ? 1 : G_ / 32), buf(b), turn(0) {
        if (warps == 1) return;
        // entries of warps that do not exist stay zero
        for (int i = threadIdx.x; i < (int)(sizeof(GroupBuf) / 4); i += blockDim.x) reinterpret_cast<float*>(buf)[i] = 0.f;
        __syncthreads();
    }
    __device__ __forceinline__ float total(const float4* p) const {
        float4 s = p[0];
#pragma unroll
        for (int i = 1; i < kMaxThreads / 128; ++i)
            if (warps > 4 * i) {
                const float4 q = p[i];
                s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
            }
        return (s.x + s.y) + (s.z + s.w);
    }
    // sums of N values over the group, in every thread
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
        static_assert(N <= kMostSums, "buffer");
        if (G >= 32) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
            if (warps == 1) return;
            // alternating buffers: one barrier per turn
            const int k = turn & 1;
            ++turn;
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int n = 0; n < N; ++n) reinterpret_cast<float*>(buf->v[k][n])[threadIdx.x >> 5] = v[n];
            __syncthreads();
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = total(buf->v[k][n]);
            return;
        }
        for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    }
};

// Values are kept in pairs: the paired fp32 instructions do two elements at
// once, and these kernels are close to being bound by issue.
using sm100::add2;
using sm100::fma2;
using sm100::mul2;
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(const uint4& r, float2* f) {
        f[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
        f[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ static __forceinline__ uint4 pack(const float2* f) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(const uint4& r, float2* f) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) f[u] = make_float2(__uint_as_float(w[u] << 16), __uint_as_float(w[u] & 0xFFFF0000u));
    }
    __device__ static __forceinline__ uint4 pack(const float2* f) {
        return make_uint4(sm100::pack_bf16(f[0].x, f[0].y), sm100::pack_bf16(f[1].x, f[1].y),
                          sm100::pack_bf16(f[2].x, f[2].y), sm100::pack_bf16(f[3].x, f[3].y));
    }
};

// A thread's columns of its group's rows: vector (ch * G + t) from the aligned
// start, `shift` elements before column 0.
template <typename T, int NCH>
struct Cols {
    static constexpr int V = Vec<T>::N;
    static constexpr int P = NCH * V / 2;   // pairs
    int D, c0, step;   // c0: column of the first element of chunk 0; chunks are `step` apart
    bool clean;        // every element of every chunk lies in the row
    int64_t total;
    __device__ __forceinline__ Cols(int D_, int64_t rows, int64_t row, const Group& g)
        : D(D_), c0(g.t * V - (int)((row * D_) % V)), step(g.G * V), total(rows * D_) {
        clean = true;
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) clean = clean && full(ch);
    }
    __device__ __forceinline__ int first(int ch) const { return c0 + ch * step; }
    __device__ __forceinline__ bool any(int ch) const { return first(ch) < D && first(ch) + V > 0; }
    __device__ __forceinline__ bool full(int ch) const { return first(ch) >= 0 && first(ch) + V <= D; }
    __device__ __forceinline__ bool in(int ch, int u) const { return (unsigned)(first(ch) + u) < (unsigned)D; }

    // the thread's vectors of N tensors (absent ones NULL: zero) for the row
    // whose column 0 is at offset `at`
    template <int N>
    __device__ __forceinline__ void load(const void* const (&base)[N], int64_t at, bool live, uint4 (&r)[N][NCH]) const {
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            const int64_t off = at + first(ch);
            const bool here = live && any(ch);
            if (!here || off + V > total) {
#pragma unroll
                for (int n = 0; n < N; ++n) r[n][ch] = make_uint4(0u, 0u, 0u, 0u);
                if (!here) continue;
                // the tensor ends inside this vector
#pragma unroll
                for (int n = 0; n < N; ++n)
                    if (base[n])
#pragma unroll
                        for (int u = 0; u < V; ++u)
                            if (in(ch, u)) reinterpret_cast<T*>(&r[n][ch])[u] = reinterpret_cast<const T*>(base[n])[off + u];
                continue;
            }
#pragma unroll
            for (int n = 0; n < N; ++n)
                r[n][ch] = base[n] ? __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(base[n]) + off))
                                   : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // elements outside the row (a neighbour's, or nothing) to zero
    __device__ __forceinline__ void mask(float2 (&f)[P]) const {
        if (clean) return;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!in(2 * i / V, 2 * i % V)) f[i].x = 0.f;
            if (!in(2 * i / V, 2 * i % V + 1)) f[i].y = 0.f;
        }
    }
    __device__ __forceinline__ void get(const uint4 (&r)[NCH], float2 (&f)[P]) const {
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) Vec<T>::unpack(r[ch], f + ch * V / 2);
        mask(f);
    }
    __device__ __forceinline__ void store(void* base, int64_t at, const float2 (&f)[P]) const {
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            T* p = reinterpret_cast<T*>(base) + (at + first(ch));
            if (full(ch)) {
                *reinterpret_cast<uint4*>(p) = Vec<T>::pack(f + ch * V / 2);
            } else if (any(ch)) {
#pragma unroll
                for (int u = 0; u < V; ++u)
                    if (in(ch, u)) p[u] = from_f<T>(u & 1 ? f[(ch * V + u) / 2].y : f[(ch * V + u) / 2].x);
            }
        }
    }
    // a parameter vector's values (`absent` where there is none, 0 outside the row)
    __device__ __forceinline__ float param(const float* p, float absent, int i) const {
        const int ch = i / V, u = i % V;
        return in(ch, u) ? (p ? __ldg(p + first(ch) + u) : absent) : 0.f;
    }
};

// A thread's parameters, K vectors of P pairs.  Where they fit beside the sums
// (MEM) they wait in shared memory, each thread its own: registers are what
// limits the warps of an SM with up to eight elements per thread and tensor, and
// those hide the latencies of the row sums; and what spills in wide rows (us in
// registers / in shared memory: 10000 x 8192 fp32 RMS forward 356 / 320,
// backward 733 / 671, 15000 x 6000 bf16 LayerNorm forward 402 / 355).
template <int K, int P, bool MEM>
struct Params {
    float2 v[K][P];
    __device__ __forceinline__ Params(float*) {}
    __device__ __forceinline__ void set(int k, int i, float2 x) { v[k][i] = x; }
    __device__ __forceinline__ void get(int k, float2 (&f)[P]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) f[i] = v[k][i];
    }
};
template <int K, int P>
struct Params<K, P, true> {
    float4* mine;
    __device__ __forceinline__ Params(float* smem) : mine(reinterpret_cast<float4*>(smem) + threadIdx.x) {}
    __device__ __forceinline__ void set(int k, int i, float2 x) {
        reinterpret_cast<float2*>(mine + (k * (P / 2) + i / 2) * blockDim.x)[i & 1] = x;
    }
    __device__ __forceinline__ void get(int k, float2 (&f)[P]) const {
#pragma unroll
        for (int i = 0; i < P; i += 2) {
            const float4 q = mine[(k * (P / 2) + i / 2) * blockDim.x];
            f[i] = make_float2(q.x, q.y);
            f[i + 1] = make_float2(q.z, q.w);
        }
    }
};

// 1 / (1 + e^-u) with the hardware's base-2 exponential and reciprocal (a few
// units in the last place, times 1 + |u| / 16 for the rounding of the scaled
// argument); a large negative u gives 0.
__device__ __forceinline__ float sigmoid(float u) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + sm100::ex2(u * -1.4426950408889634f)));
    return r;
}

// act(u) in place and, SLOPE, act'(u).
template <int P, bool SLOPE>
__device__ __forceinline__ void gate_values(int kind, float2 (&u)[P], float2 (&slope)[SLOPE ? P : 1]) {
    if (kind == JFA_GATE_SILU) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 q = make_float2(sigmoid(u[i].x), sigmoid(u[i].y)), v = u[i];
            u[i] = mul2(v, q);
            // q (1 + v (1 - q)) = q + v q - (v q) q
            if (SLOPE) slope[SLOPE ? i : 0] = mul2(q, fma2(v, fma2(q, both(-1.f), both(1.f)), both(1.f)));
        }
    } else if (kind == JFA_GATE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            u[i] = make_float2(sigmoid(u[i].x), sigmoid(u[i].y));
            if (SLOPE) slope[SLOPE ? i : 0] = mul2(u[i], fma2(u[i], both(-1.f), both(1.f)));
        }
    } else if (kind == JFA_GATE_IDENTITY) {
        if (SLOPE) {
#pragma unroll
            for (int i = 0; i < P; ++i) slope[SLOPE ? i : 0] = both(1.f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) u[i] = both(1.f);
    }
}

template <int P>
__device__ __forceinline__ float dot(const float2 (&a)[P], const float2 (&b)[P]) {
    float2 q = mul2(a[0], b[0]);
#pragma unroll
    for (int i = 1; i < P; ++i) q = fma2(a[i], b[i], q);
    return q.x + q.y;
}
template <int P>
__device__ __forceinline__ float plain_sum(const float2 (&a)[P]) {
    float2 q = a[0];
#pragma unroll
    for (int i = 1; i < P; ++i) q = add2(q, a[i]);
    return q.x + q.y;
}
template <int P>
__device__ __forceinline__ void scale_by(float2 (&a)[P], float r) {
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = mul2(a[i], both(r));
}
template <int P>
__device__ __forceinline__ void shift_by(float2 (&a)[P], float r) {
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = add2(a[i], both(r));
}

// v * (vector k1) (+ vector k0) in place.
template <int P, bool LN, typename Par>
__device__ __forceinline__ void scale_shift(const Par& par, int k1, int k0, float2 (&v)[P]) {
    float2 w[P];
    par.get(k1, w);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], w[i]);
    if (LN) {
        par.get(k0, w);
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = add2(v[i], w[i]);
    }
}

// sum / D, corrected to the last place: exact for a row of one number whose sum
// is exact (the rounding of 1 / D alone left 6e-8 of the number, which 1 /
// sqrt(eps) makes 0.02 at 1000).
__device__ __forceinline__ float mean_of(float sum, int D, float inv_d) {
    const float mu = sum * inv_d;
    return fmaf(fmaf(-mu, (float)D, sum), inv_d, mu);
}

// The block's norm and the way to y.  In: b, x, k = act(u) (ones without a
// gate).  Out: b = hat of the block, x = y - mu_y with mu_y the mean for a
// LayerNorm next and 0 otherwise; returns the block's r.  The mean of
//   y = x + k (w0 + w1 hat) = (x + k w0) + r (k w1 c),  c = b - mu
// comes from two sums taken together with the sum of c^2, so that it needs no
// turn of its own; y is the sum of its parts either way.
template <typename T, int NCH, bool LN, typename Par>
__device__ __forceinline__ float to_y(const Par& par, int W1, int W0, int post, int pre, const Cols<T, NCH>& cols, Group& g,
                                      float inv_d, float eps, float2 (&b)[Cols<T, NCH>::P], float2 (&x)[Cols<T, NCH>::P],
                                      const float2 (&k)[Cols<T, NCH>::P], float& mu_y) {
    constexpr int P = Cols<T, NCH>::P;
    if (LN && post == JFA_NORM_LAYER) {
        float s[1] = {plain_sum<P>(b)};
        g.template sum<1>(s);
        shift_by<P>(b, -mean_of(s[0], cols.D, inv_d));
        cols.mask(b);
    }
    float2 w[P];
    if (LN) {
        par.get(W0, w);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = fma2(k[i], w[i], x[i]);
    }
    par.get(W1, w);
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = mul2(mul2(w[i], k[i]), b[i]);
    float r = 1.f;
    mu_y = 0.f;
    if (LN && pre == JFA_NORM_LAYER) {
        float s[3] = {dot<P>(b, b), plain_sum<P>(x), plain_sum<P>(w)};
        g.template sum<3>(s);
        if (post != JFA_NORM_NONE) r = rsqrtf(fmaf(s[0], inv_d, eps));
        mu_y = mean_of(fmaf(r, s[2], s[1]), cols.D, inv_d);
    } else if (post != JFA_NORM_NONE) {
        float s[1] = {dot<P>(b, b)};
        g.template sum<1>(s);
        r = rsqrtf(fmaf(s[0], inv_d, eps));
    }
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = fma2(both(r), w[i], x[i]);
    if (post != JFA_NORM_NONE) scale_by<P>(b, r);
    return r;
}

// Whether so many vectors of a thread's pairs fit into shared memory.
template <typename T, int NCH, int VECTORS, int BOUND>
constexpr bool kFits = VECTORS * (NCH * Vec<T>::N / 2) * (int)sizeof(float2) * BOUND <= 220 * 1024;

// Registers per thread through the launch bound: 80 for the forward (64 fp32,
// 96 with two vectors)
// and 80 for the fp32 backward with one vector per thread, 128 otherwise.
// 60000 x 1024 fp32 backward at 128 / 96 / 80 / 64 registers: 451 / 383 / 331 /
// 350 us; 222283 x 1024 bf16 backward at 128 / 96 / 80: 769 / 1228 / 1670 us
// (spills), forward at 80 / 64: 393 / 431 us.
template <typename T, int NCH>
constexpr int kFwdBound = NCH > 1 ? (sizeof(T) == 4 && NCH == 2 ? 640 : kMaxThreads) : (sizeof(T) == 4 ? 1024 : 768);
template <typename T, int NCH>
constexpr int kBwdBound = NCH == 1 && sizeof(T) == 4 ? 768 : kMaxThreads;

// bf16 rows of two and three vectors per thread spill at 128 registers; up to
// 384 threads there are 168.  Two vectors need no more up to 6144 columns, three
// never do (352; 10000 x 8191, us at 512 / 384: RMS forward 308 / 250, backward
// 817 / 587, LayerNorm 517 / 408 and 1110 / 821).  fp32 rows of five vectors
// have 416 threads, for which there are 128 again: the registers are dealt to
// the SM's four schedulers, and 13 warps are four on one of them.
constexpr int kFewThreads = 384;
template <typename T, int BOUND>
constexpr int kFewBound = sizeof(T) == 2 ? kFewThreads : BOUND;

// LN: a norm is a LayerNorm, so that there may be betas.
template <typename T, int NCH, bool LN, int BOUND = kFwdBound<T, NCH>>
__global__ void __launch_bounds__(BOUND, 1) block_norm_fwd(const NormArgs a, int G) {
    constexpr int P = Cols<T, NCH>::P;
    extern __shared__ float4 smem4[];
    __shared__ GroupBuf buf;
    Group g(G, &buf);
    Params<LN ? 4 : 2, P, kFits<T, NCH, LN ? 4 : 2, BOUND>> par(reinterpret_cast<float*>(smem4));
    const int groups = blockDim.x / G;
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t base = (int64_t)blockIdx.x * groups, row = base + threadIdx.x / G;
    const Cols<T, NCH> cols(a.D, a.rows, row, g);
    const bool gated = a.gate_kind != JFA_GATE_NONE, pre = a.pre != JFA_NORM_NONE;
    const float inv_d = 1.0f / (float)a.D;
    const void* const in[3] = {a.block, a.x, gated ? a.gate : nullptr};
    uint4 raw[3][NCH];
    int64_t at = row * a.D, at_next = at;
    cols.load(in, at, row < a.rows, raw);
    // y = x + act(u) * (w1 * hat + w0), n = hat_y * q1 + q0
    enum { W1 = 0, Q1, W0, Q0 };
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 s = make_float2(cols.param(a.scale, 1.f, 2 * i), cols.param(a.scale, 1.f, 2 * i + 1));
        par.set(W1, i, mul2(s, make_float2(cols.param(a.post_gamma, 1.f, 2 * i), cols.param(a.post_gamma, 1.f, 2 * i + 1))));
        par.set(Q1, i, make_float2(cols.param(a.pre_gamma, 1.f, 2 * i), cols.param(a.pre_gamma, 1.f, 2 * i + 1)));
        if (LN) {
            par.set(LN ? W0 : 0, i, mul2(s, make_float2(cols.param(a.post_beta, 0.f, 2 * i), cols.param(a.post_beta, 0.f, 2 * i + 1))));
            par.set(LN ? Q0 : 0, i, make_float2(cols.param(a.pre_beta, 0.f, 2 * i), cols.param(a.pre_beta, 0.f, 2 * i + 1)));
        }
    }
    for (; base < a.rows; base += stride, row += stride, at = at_next) {
        float2 b[P], x[P], k[P], none[1];
        cols.get(raw[0], b);
        cols.get(raw[1], x);
        cols.get(raw[2], k);
        at_next = at + stride * a.D;
        cols.load(in, at_next, row + stride < a.rows, raw);
        gate_values<P, false>(a.gate_kind, k, none);
        float mu;
        to_y<T, NCH, LN>(par, W1, LN ? W0 : 0, a.post, a.pre, cols, g, inv_d, a.eps, b, x, k, mu);
        const bool live = row < a.rows;
        if (live) cols.store(a.y, at, x);
        if (!pre) continue;
        if (LN && a.pre == JFA_NORM_LAYER) {
            shift_by<P>(x, -mu);
            cols.mask(x);
        }
        float s[1] = {dot<P>(x, x)};
        g.template sum<1>(s);
        scale_by<P>(x, rsqrtf(fmaf(s[0], inv_d, a.eps)));
        scale_shift<P, LN>(par, Q1, LN ? Q0 : 0, x);
        if (live) cols.store(a.n, at, x);
    }
}

enum { Q_POST1 = 0, Q_PRE1, Q_POST0, Q_PRE0, Q_COUNT };   // S1 of the two norms, S2 of the two

// The sums over rows, in pairs: in registers, or in shared memory (each thread
// its own) where registers run out: several vectors per thread, and the four
// sums of a LayerNorm (222283 x 1024 bf16: 1366 us in registers, with spills,
// 1189 us in shared memory; 9001 x 1003 fp32: 103 and 89 us).
template <typename T, int NCH, bool LN>
constexpr bool kSumsInSmem = NCH * Vec<T>::N > 8 || LN;
template <bool LN>
constexpr int kBwdParams = LN ? 3 : 2;
// Except beside the four sums of bf16 LayerNorms with two vectors per thread,
// where the 168 registers of up to 384 threads hold the parameters (us in
// registers / in shared memory: 15000 x 6000 769 / 804, 6144 746 / 795, 4200
// 695 / 699, 5003 805 / 806; beside the sums of 512 threads they do not fit).
template <typename T, int NCH, bool LN, int BOUND>
constexpr bool kBwdParamsInSmem = !(LN && sizeof(T) == 2 && NCH == 2) &&
                                  kFits<T, NCH, kBwdParams<LN> + (kSumsInSmem<T, NCH, LN> ? (LN ? 4 : 2) : 0), BOUND>;
template <int P, int Q, bool SMEM>
struct Sums {
    float2 v[Q][P];
    __device__ __forceinline__ Sums(float*) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < P; ++i) v[q][i] = both(0.f);
    }
    __device__ __forceinline__ void add(int q, int i, float2 x) { v[q][i] = add2(v[q][i], x); }
    __device__ __forceinline__ void fma(int q, int i, float2 x, float2 y) { v[q][i] = fma2(x, y, v[q][i]); }
    __device__ __forceinline__ float2 get(int q, int i) const { return v[q][i]; }
};
template <int P, int Q>
struct Sums<P, Q, true> {
    float2* mine;
    int stride;
    __device__ __forceinline__ Sums(float* smem) : mine(reinterpret_cast<float2*>(smem) + threadIdx.x), stride(blockDim.x) {
        for (int i = 0; i < Q * P; ++i) mine[i * stride] = both(0.f);
    }
    __device__ __forceinline__ void add(int q, int i, float2 x) {
        float2& m = mine[(q * P + i) * stride];
        m = add2(m, x);
    }
    __device__ __forceinline__ void fma(int q, int i, float2 x, float2 y) {
        float2& m = mine[(q * P + i) * stride];
        m = fma2(x, y, m);
    }
    __device__ __forceinline__ float2 get(int q, int i) const { return mine[(q * P + i) * stride]; }
};

template <typename T, int NCH, bool LN, int BOUND = kBwdBound<T, NCH>>
__global__ void __launch_bounds__(BOUND, 1) block_norm_bwd(const NormArgs a, int G) {
    constexpr int V = Vec<T>::N, P = Cols<T, NCH>::P, Q = LN ? 4 : 2;
    constexpr bool kSmem = kSumsInSmem<T, NCH, LN>, kAhead = NCH == 1;
    extern __shared__ float4 smem4[];   // parameters, sums, each where they are kept here; at the end the small groups' reduction
    float* const smem = reinterpret_cast<float*>(smem4);
    __shared__ GroupBuf buf;
    Group g(G, &buf);
    constexpr bool kPar = kBwdParamsInSmem<T, NCH, LN, BOUND>;
    Params<kBwdParams<LN>, P, kPar> par(smem);
    Sums<P, Q, kSmem> sums(smem + (kPar ? kBwdParams<LN> * 2 * P * blockDim.x : 0));
    const int groups = blockDim.x / G;
    const int64_t stride = (int64_t)gridDim.x * groups;
    int64_t base = (int64_t)blockIdx.x * groups, row = base + threadIdx.x / G;
    const Cols<T, NCH> cols(a.D, a.rows, row, g);
    const bool gated = a.gate_kind != JFA_GATE_NONE, pre = a.pre != JFA_NORM_NONE;
    const float inv_d = 1.0f / (float)a.D;
    const void* const in[5] = {a.block, a.x, gated ? a.gate : nullptr, pre ? a.dn : nullptr, a.dy};
    uint4 raw[5][NCH];
    int64_t at = row * a.D, at_next = at;
    if (kAhead) cols.load(in, at, row < a.rows, raw);
    enum { W1 = 0, Q1, W0 };   // s * gamma of the block's norm, gamma of the next one's, s * beta
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 s = make_float2(cols.param(a.scale, 1.f, 2 * i), cols.param(a.scale, 1.f, 2 * i + 1));
        par.set(W1, i, mul2(s, make_float2(cols.param(a.post_gamma, 1.f, 2 * i), cols.param(a.post_gamma, 1.f, 2 * i + 1))));
        par.set(Q1, i, make_float2(cols.param(a.pre_gamma, 1.f, 2 * i), cols.param(a.pre_gamma, 1.f, 2 * i + 1)));
        if (LN)
            par.set(LN ? W0 : 0, i, mul2(s, make_float2(cols.param(a.post_beta, 0.f, 2 * i), cols.param(a.post_beta, 0.f, 2 * i + 1))));
    }
    for (; base < a.rows; base += stride, row += stride, at = at_next) {
        const bool live = row < a.rows;
        if (!kAhead) cols.load(in, at, live, raw);
        float2 b[P], y[P], u[P], d[P], dn[P], slope[P];
        cols.get(raw[0], b);
        cols.get(raw[1], y);
        cols.get(raw[2], u);
        // dn and dy wait as they came (half the registers in bf16)
        uint4 later[2][NCH];
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
            later[0][ch] = raw[3][ch];
            later[1][ch] = raw[4][ch];
        }
        at_next = at + stride * a.D;
        if (kAhead) cols.load(in, at_next, row + stride < a.rows, raw);
        gate_values<P, true>(a.gate_kind, u, slope);   // u: act(u)
        float mu;
        const float r_b = to_y<T, NCH, LN>(par, W1, LN ? W0 : 0, a.post, a.pre, cols, g, inv_d, a.eps, b, y, u, mu);
        float2 w[P];
        if (pre) {
            const bool layer = LN && a.pre == JFA_NORM_LAYER;
            if (layer) {
                shift_by<P>(y, -mu);
                cols.mask(y);
            }
            cols.get(later[0], dn);
            if (LN)
#pragma unroll
                for (int i = 0; i < P; ++i) sums.add(LN ? Q_PRE0 : 0, i, dn[i]);
            // g = dn * gamma; with y = c of the norm, hat = r c:
            //   d += r (g - hat mean(g hat) - mean(g)), the two sums with that of c^2
            par.get(Q1, w);
#pragma unroll
            for (int i = 0; i < P; ++i) w[i] = mul2(dn[i], w[i]);
            float s[LN ? 3 : 2] = {dot<P>(y, y), dot<P>(w, y)};
            if (LN) s[LN ? 2 : 0] = plain_sum<P>(w);
            g.template sum<LN ? 3 : 2>(s);
            const float r_y = rsqrtf(fmaf(s[0], inv_d, a.eps));
            scale_by<P>(y, r_y);
            const float2 c1 = both(-r_y * s[1] * inv_d);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sums.fma(Q_PRE1, i, dn[i], y[i]);
                w[i] = fma2(y[i], c1, w[i]);
            }
            if (layer) {
                shift_by<P>(w, -s[LN ? 2 : 0] * inv_d);
                cols.mask(w);   // no part in the sums below
            }
            cols.get(later[1], d);
#pragma unroll
            for (int i = 0; i < P; ++i) d[i] = fma2(both(r_y), w[i], d[i]);
        } else {
            cols.get(later[1], d);
        }
        // d is dx; on to the block: dp, the gate's gradient and the sums
        if (live) cols.store(a.dx, at, d);
        if (gated) {
#pragma unroll
            for (int i = 0; i < P; ++i) w[i] = b[i];
            scale_shift<P, LN>(par, W1, LN ? W0 : 0, w);
#pragma unroll
            for (int i = 0; i < P; ++i) slope[i] = mul2(mul2(d[i], slope[i]), w[i]);
            if (live) cols.store(a.dgate, at, slope);
        }
        par.get(W1, w);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            d[i] = mul2(d[i], u[i]);
            sums.fma(Q_POST1, i, d[i], b[i]);
            if (LN) sums.add(LN ? Q_POST0 : 0, i, d[i]);
            d[i] = mul2(d[i], w[i]);
        }
        if (a.post != JFA_NORM_NONE) {
            float s[LN ? 2 : 1] = {dot<P>(d, b)};
            if (LN) s[LN ? 1 : 0] = plain_sum<P>(d);
            g.template sum<LN ? 2 : 1>(s);
            const float2 c1 = both(-s[0] * inv_d);
#pragma unroll
            for (int i = 0; i < P; ++i) d[i] = fma2(b[i], c1, d[i]);
            if (LN && a.post == JFA_NORM_LAYER) shift_by<P>(d, -s[LN ? 1 : 0] * inv_d);
            scale_by<P>(d, r_b);
        }
        if (live) cols.store(a.dblock, at, d);
    }
    // this CTA's partial row of each sum
    float* const part = a.parts + (int64_t)blockIdx.x * Q_COUNT * a.D;
    auto put = [&](float* to, int q) {
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) {
            const float2 v = sums.get(q, i / 2);
            if (cols.in(i / V, i % V)) to[cols.first(i / V) + i % V] = i & 1 ? v.y : v.x;
        }
    };
    if (groups == 1) {
#pragma unroll
        for (int q = 0; q < Q; ++q) put(part + q * a.D, q);
    } else {
        // the groups' sums in group order, through shared memory [groups][D]
        // behind the parameters and sums
        float* const area = smem + ((kPar ? kBwdParams<LN> : 0) + (kSmem ? Q : 0)) * 2 * P * blockDim.x;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            __syncthreads();
            put(area + (threadIdx.x / G) * a.D, q);
            __syncthreads();
            for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
                float s = 0.f;
                for (int k = 0; k < groups; ++k) s += area[k * a.D + c];
                part[q * a.D + c] = s;
            }
        }
    }
}

// Adds the partial rows (in order within 32 interleaved strands, which
// are then added in order) and forms the parameter gradients: blockIdx.y 0 the
// block's norm and the scale, 1 the next norm.
constexpr int kStrands = 32;
__global__ void __launch_bounds__(32 * kStrands) block_norm_sum(const NormArgs a, int n, float* dscale, float* dpost_gamma,
                                                                float* dpost_beta, float* dpre_gamma, float* dpre_beta) {
    __shared__ float2 s_part[kStrands][32];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, which = blockIdx.y;
    const bool two = (which == 0 ? a.post : a.pre) == JFA_NORM_LAYER;
    const int64_t pitch = (int64_t)Q_COUNT * a.D;
    float2 s = make_float2(0.f, 0.f);
    if (c < a.D) {
        const float* p1 = a.parts + (int64_t)(which == 0 ? Q_POST1 : Q_PRE1) * a.D + c;
        const float* p0 = a.parts + (int64_t)(which == 0 ? Q_POST0 : Q_PRE0) * a.D + c;
#pragma unroll 4
        for (int p = strand; p < n; p += kStrands) {
            s.x += p1[p * pitch];
            if (two) s.y += p0[p * pitch];
        }
    }
    s_part[strand][lane] = s;
    __syncthreads();
    if (strand != 0 || c >= a.D) return;
#pragma unroll
    for (int k = 1; k < kStrands; ++k) {
        s.x += s_part[k][lane].x;
        s.y += s_part[k][lane].y;
    }
    if (which == 0) {
        const float sc = a.scale ? a.scale[c] : 1.f;
        if (dscale) {
            float v = s.x * (a.post_gamma ? a.post_gamma[c] : 1.f);
            if (a.post_beta) v = fmaf(s.y, a.post_beta[c], v);
            dscale[c] = v;
        }
        if (dpost_gamma) dpost_gamma[c] = sc * s.x;
        if (dpost_beta) dpost_beta[c] = sc * s.y;
    } else {
        if (dpre_gamma) dpre_gamma[c] = s.x;
        if (dpre_beta) dpre_beta[c] = s.y;
    }
}

// How a row width is cut up: vectors per thread and threads per row, a power
// of two within a warp, whole warps above.  Widths that are no multiple of a
// vector need one more vector.  In fp32 a vector is four elements, and two of
// them per thread halve the row sums' share of the work: LayerNorm 60000 x
// 1024 with one / two: forward 258 / 196 us, backward 505 / 410, 100000 x 300
// backward 307 / 333; RMS 60000 x 1024 forward 187 / 209, backward 336 / 324,
// 30000 x 2048 (where one per thread leaves one CTA on an SM) backward 437 /
// 342.  In bf16 one vector of eight is best up to 512 threads.
struct RowShape {
    int G, threads, nch, groups;
    int period;   // rows after which the alignment repeats
};
// Vectors per thread of the widest rows: 8191 columns that start off a
// boundary take 1025 vectors of bf16 and 2049 of fp32.  Above 2 x 512 vectors
// each count has its kernels (10000 x 6731 fp32 RMS backward: 1617 us with five
// vectors, for which the compiler took 64 registers, 689 with four).
template <typename T>
constexpr int kMostChunks = sizeof(T) == 4 ? 5 : 3;
static_assert(kMostChunks<float> * kMaxThreads * 4 >= kMaxDim + 4 && kMostChunks<__nv_bfloat16> * kMaxThreads * 8 >= kMaxDim + 8,
              "the widest rows fit");

template <typename T, bool LN>
RowShape row_shape(int D) {
    constexpr int V = Vec<T>::N;
    RowShape s{};
    const int vecs = D % V == 0 ? D / V : (D + V - 2) / V + 1;
    const int one = sizeof(T) == 2 ? kMaxThreads : (LN ? 128 : 384);   // most vectors of a row with one per thread
    s.nch = vecs <= one ? 1 : (vecs <= 2 * kMaxThreads ? 2 : (vecs + kMaxThreads - 1) / kMaxThreads);
    const int need = (vecs + s.nch - 1) / s.nch;
    if (need > 32) {
        s.G = (need + 31) / 32 * 32;
    } else {
        s.G = 1;
        while (s.G < need) s.G *= 2;
    }
    s.threads = s.G <= 32 ? kSmallThreads : s.G;
    s.groups = s.threads / s.G;
    s.period = V;
    while (s.period > 1 && (int64_t)D * (s.period / 2) % V == 0) s.period /= 2;
    return s;
}

// CTAs for `rows` rows: one round if an SM's worth each is enough, else as many
// as are resident at a time, with the rows of a group gridDim * groups apart,
// which has to be a multiple of the period.
template <typename K>
cudaError_t row_grid(K kern, const RowShape& s, int64_t rows, size_t smem, int64_t limit, int* grid) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t need = (rows + s.groups - 1) / s.groups;
    *grid = (int)need;
    if (need <= sms) return cudaSuccess;
    int per_sm = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, s.threads, smem);
    if (e != cudaSuccess) return e;
    int64_t cap = (int64_t)sms * (per_sm > 0 ? per_sm : 1);
    if (cap > limit) cap = limit;
    if (need <= cap) return cudaSuccess;
    while (cap > 1 && cap * s.groups % s.period != 0) --cap;
    *grid = (int)cap;
    return cudaSuccess;
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

// A kernel, the vectors of its threads' pairs that it keeps in shared memory and
// the most shared memory that a call of any of its widths asks for.  That
// constant, and not the call's own need, is the limit that is set: the limit
// belongs to the device, so that a narrow call of another host thread would
// otherwise lower it between a wide call's setting and its launch.
struct Kernel {
    void (*kern)(NormArgs, int);
    int vectors;
    size_t most;
};
// `vectors` of up to BOUND threads, or of the CTAs of several rows with the
// area that these sum their groups in (at most their threads' columns).
template <typename T, int NCH, int BOUND>
constexpr size_t most_smem(int vectors) {
    const size_t each = sizeof(float2) * (NCH * Vec<T>::N / 2) * vectors;
    const size_t wide = each * (BOUND < kMaxThreads ? BOUND : kMaxThreads);
    const size_t small = (each + sizeof(float) * NCH * Vec<T>::N) * kSmallThreads;
    return wide > small ? wide : small;
}
constexpr size_t kSmemOfSm = 227 * 1024;

cudaError_t allow_smem(const Kernel& k, size_t smem) {
    // 48 KB, static shared memory included, need no permission
    return smem > 40 * 1024 ? cudaFuncSetAttribute(k.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.most) : cudaSuccess;
}

template <typename T, int NCH, bool LN, int BOUND = kFwdBound<T, NCH>>
Kernel fwd_kernel() {
    constexpr int vectors = kFits<T, NCH, LN ? 4 : 2, BOUND> ? (LN ? 4 : 2) : 0;
    constexpr size_t most = most_smem<T, NCH, BOUND>(vectors);
    static_assert(most + sizeof(GroupBuf) <= kSmemOfSm, "shared memory");
    return {block_norm_fwd<T, NCH, LN, BOUND>, vectors, most};
}
template <typename T, int NCH, bool LN, int BOUND = kBwdBound<T, NCH>>
Kernel bwd_kernel() {
    constexpr int vectors = (kBwdParamsInSmem<T, NCH, LN, BOUND> ? kBwdParams<LN> : 0) + (kSumsInSmem<T, NCH, LN> ? (LN ? 4 : 2) : 0);
    constexpr size_t most = most_smem<T, NCH, BOUND>(vectors);
    static_assert(most + sizeof(GroupBuf) <= kSmemOfSm, "shared memory");
    return {block_norm_bwd<T, NCH, LN, BOUND>, vectors, most};
}
// bf16 rows have at most three vectors per thread.
template <typename T, bool LN>
Kernel fwd_kernel_of(const RowShape& s) {
    constexpr int M = kMostChunks<T>;
    switch (s.nch) {
        case 1: return fwd_kernel<T, 1, LN>();
        case 2: return s.threads <= kFewThreads ? fwd_kernel<T, 2, LN, kFewBound<T, kFwdBound<T, 2>>>() : fwd_kernel<T, 2, LN>();
        case 3: return fwd_kernel<T, 3, LN, kFewBound<T, kFwdBound<T, 3>>>();
        case 4: return fwd_kernel<T, M < 4 ? M : 4, LN, kFewBound<T, kFwdBound<T, 4>>>();
        default: return fwd_kernel<T, M, LN, kFewBound<T, kFwdBound<T, M>>>();
    }
}
template <typename T, bool LN>
Kernel bwd_kernel_of(const RowShape& s) {
    constexpr int M = kMostChunks<T>;
    switch (s.nch) {
        case 1: return bwd_kernel<T, 1, LN>();
        case 2: return s.threads <= kFewThreads ? bwd_kernel<T, 2, LN, kFewBound<T, kBwdBound<T, 2>>>() : bwd_kernel<T, 2, LN>();
        case 3: return bwd_kernel<T, 3, LN, kFewBound<T, kBwdBound<T, 3>>>();
        case 4: return bwd_kernel<T, M < 4 ? M : 4, LN, kFewBound<T, kBwdBound<T, 4>>>();
        default: return bwd_kernel<T, M, LN, kFewBound<T, kBwdBound<T, M>>>();
    }
}

template <typename T, bool LN>
cudaError_t fwd_launch(const NormArgs& a, cudaStream_t st) {
    const RowShape s = row_shape<T, LN>(a.D);
    const Kernel k = fwd_kernel_of<T, LN>(s);
    const size_t smem = sizeof(float2) * (s.nch * Vec<T>::N / 2) * s.threads * k.vectors;
    int grid = 0;
    cudaError_t e = allow_smem(k, smem);
    if (e == cudaSuccess) e = row_grid(k.kern, s, a.rows, smem, 0x7fffffff, &grid);
    if (e != cudaSuccess) return e;
    prof_begin(st);
    k.kern<<<grid, s.threads, smem, st>>>(a, s.G);
    prof_end(st, K_BLOCK_NORM_FWD);
    return cudaGetLastError();
}

// Returns the number of partial rows in *parts.
template <typename T, bool LN>
cudaError_t bwd_launch(const NormArgs& a, int* parts, cudaStream_t st) {
    const RowShape s = row_shape<T, LN>(a.D);
    const Kernel k = bwd_kernel_of<T, LN>(s);
    const size_t smem = sizeof(float2) * (s.nch * Vec<T>::N / 2) * s.threads * k.vectors +
                        (s.groups > 1 ? sizeof(float) * s.groups * a.D : 0);
    cudaError_t e = allow_smem(k, smem);
    if (e == cudaSuccess) e = row_grid(k.kern, s, a.rows, smem, kMaxParts, parts);
    if (e != cudaSuccess) return e;
    prof_begin(st);
    k.kern<<<*parts, s.threads, smem, st>>>(a, s.G);
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
    const bool ln = desc->post_norm == JFA_NORM_LAYER || desc->pre_norm == JFA_NORM_LAYER;
    const cudaError_t e = desc->dtype == JFA_F32 ? (ln ? fwd_launch<float, true>(a, st) : fwd_launch<float, false>(a, st))
                                                 : (ln ? fwd_launch<__nv_bfloat16, true>(a, st)
                                                       : fwd_launch<__nv_bfloat16, false>(a, st));
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
    const bool ln = desc->post_norm == JFA_NORM_LAYER || desc->pre_norm == JFA_NORM_LAYER;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0)
        e = desc->dtype == JFA_F32 ? (ln ? bwd_launch<float, true>(a, &parts, st) : bwd_launch<float, false>(a, &parts, st))
                                   : (ln ? bwd_launch<__nv_bfloat16, true>(a, &parts, st)
                                         : bwd_launch<__nv_bfloat16, false>(a, &parts, st));
    if (e == cudaSuccess && (dscale || dpost_gamma || dpost_beta || dpre_gamma || dpre_beta)) {
        prof_begin(st);
        block_norm_sum<<<dim3((a.D + 31) / 32, 2), 32 * kStrands, 0, st>>>(a, parts, dscale, dpost_gamma, dpost_beta,
                                                                           dpre_gamma, dpre_beta);
        prof_end(st, K_BLOCK_NORM_SUM);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return JFA_OK;
}

}  // extern "C"
