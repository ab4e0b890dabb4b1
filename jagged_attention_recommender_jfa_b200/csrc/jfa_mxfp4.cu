// MXFP4 quantisation (OCP Microscaling v1.0, E2M1 elements with one E8M0
// power-of-two scale per 32) of the operands of jfa_matmul_mxfp4
// ("Meta Enhances GEM Training Efficiency with Advanced LLM-Scale
// Innovations", "Implementing Ultra-Low-Precision Methods").
//
//   X     = floor(log2(amax)) - 2   (2 = largest E2M1 exponent), in [-127, 127]
//   code  = E2M1_rne_satfinite(x * 2^-X), scale byte = X + 127
// A block that holds an infinity or a NaN has the scale byte 255 (E8M0 NaN)
// and zero codes.  x * 2^-X is a power-of-two scaling, exact unless the result
// is below 2^-126, far under half the smallest code: the conversion is the
// only rounding.
//
// Bound: HBM.  2 (bf16) or 4 bytes read and 1/2 + 1/32 written per element,
// plus 2 or 4 with the dequantised copy.
#include "jfa_common.cuh"
#include "jfa_mx4.cuh"

namespace jfa {

namespace {

using mx4::absmax3;
using mx4::absmax_bf16x2;
using mx4::cvt8;
using mx4::pack8;
using mx4::scale_value;
using mx4::scaled;
using mx4::Shared;
using mx4::unpack8;

// Eight consecutive elements as they lie in memory; the bits of their largest
// magnitude as an fp32 number (infinities and NaN compare above every finite
// number, so an exponent field of 255 survives the maximum); their codes under
// a shared exponent; and, for rows that end inside them, zeros from element n on.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void words(const uint32_t (&w)[4]) { r = make_uint4(w[0], w[1], w[2], w[3]); }
    __device__ __forceinline__ static uint32_t first(uint32_t w, int n) { return n >= 2 ? w : n == 1 ? w & 0xFFFFu : 0u; }
    __device__ __forceinline__ void clip(int n) {
        r = make_uint4(first(r.x, n), first(r.y, n - 2), first(r.z, n - 4), first(r.w, n - 6));
    }
    __device__ __forceinline__ uint32_t max_bits() const {
        const uint32_t m = absmax_bf16x2(absmax_bf16x2(r.x, r.y), absmax_bf16x2(r.z, r.w));
        return max(m << 16, m & 0xFFFF0000u);   // bits of magnitudes order like the magnitudes
    }
    __device__ __forceinline__ uint32_t codes(const Shared& sh) const {
        const uint32_t s = sh.inv_bf16x2();
        float f[8];
        scaled(r.x, s, f[0], f[1]);
        scaled(r.y, s, f[2], f[3]);
        scaled(r.z, s, f[4], f[5]);
        scaled(r.w, s, f[6], f[7]);
        return sh.nan ? 0u : cvt8(f);
    }
    // to shared memory: the eight, the first vector of them, and into the tile of mx4_both
    __device__ __forceinline__ void put_vectors(uint8_t* s) const { *reinterpret_cast<uint4*>(s) = r; }
    __device__ __forceinline__ void put_vector(uint8_t* s) const { *reinterpret_cast<uint4*>(s) = r; }
    __device__ __forceinline__ void put(uint8_t* s, int row, int lane) const;
};
template <>
struct Raw8<float> {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void words(const uint32_t (&w)[8]) {
        a = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        b = make_float4(__uint_as_float(w[4]), __uint_as_float(w[5]), __uint_as_float(w[6]), __uint_as_float(w[7]));
    }
    __device__ __forceinline__ void clip(int n) {
        a = make_float4(n > 0 ? a.x : 0.f, n > 1 ? a.y : 0.f, n > 2 ? a.z : 0.f, n > 3 ? a.w : 0.f);
        b = make_float4(n > 4 ? b.x : 0.f, n > 5 ? b.y : 0.f, n > 6 ? b.z : 0.f, n > 7 ? b.w : 0.f);
    }
    __device__ __forceinline__ uint32_t max_bits() const {
        return __float_as_uint(absmax3(absmax3(a.x, a.y, a.z), absmax3(a.w, b.x, b.y), absmax3(b.z, b.w, 0.f)));
    }
    __device__ __forceinline__ uint32_t codes(const Shared& sh) const {
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        return sh.nan ? 0u : pack8(f, sh.inv());
    }
    __device__ __forceinline__ void put_vectors(uint8_t* s) const {
        reinterpret_cast<float4*>(s)[0] = a;
        reinterpret_cast<float4*>(s)[1] = b;
    }
    __device__ __forceinline__ void put_vector(uint8_t* s) const { *reinterpret_cast<float4*>(s) = a; }
    __device__ __forceinline__ void put(uint8_t* s, int row, int lane) const;
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    uint4 o;
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * u], f[2 * u + 1]);
        w[u] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// A CTA of the row kernels takes 128 rows x 128 columns: one scale tile, whose
// 512 bytes leave together (those of rows and blocks behind the tensor as
// zeros).  Sixteen lanes take a segment (the tile's part of a row), eight
// elements each; the loads of all of a half warp's segments are in flight
// before the first conversion.  The first version walked the segments in
// memory order and stored each scale byte by itself: 12% of its time.
//
// Next to HBM these kernels are bound by instructions (75 a warp for its eight
// elements a lane, 70% of the issue slots at 5.3 TB/s), so a thread takes many
// segments to share its addresses.  bf16, us, 512 threads and 3 CTAs an SM / 256
// and 4 / 256 and 5: 65537 x 4096 107 / 103 / 109, both ways 183 / 171 / 205.
// fp32 (twice the bytes per segment), 512 and 2 / 256 and 2: 65537 x 1003 64 /
// 68, both ways of 65537 x 1024 70 / 76.
template <typename T>
constexpr int kRowThreads = sizeof(T) == 2 ? 256 : 512;
template <typename T>
constexpr int kHalvesOf = kRowThreads<T> / 16;
template <typename T>
constexpr int kRowCtas = sizeof(T) == 2 ? 4 : 2;
// mx4_any, 222283 x 1023 bf16 without / with the copy: 146 / 255 us at 3,
// 140 / 261 at 4 (spills with the copy).
template <typename T>
constexpr int kAnyCtas = sizeof(T) == 2 ? 3 : 2;

struct Tile {
    int64_t rt, r0;   // row tile and its first row
    int kt;           // column tile
    __device__ __forceinline__ explicit Tile(int tiles_k) {
        rt = blockIdx.x / (unsigned)tiles_k;
        r0 = rt * 128;
        kt = (int)(blockIdx.x - (unsigned)rt * (unsigned)tiles_k);
    }
};
// Rows of the tensor from the tile's row i on.
__device__ __forceinline__ int rows_left(int64_t r0, int64_t rows, int i) {
    return (int)(rows - r0 < 128 ? rows - r0 : 128) - i;
}
// The scale byte of block j of row i of the tile, staged as it is stored.
__device__ __forceinline__ int staged_scale(int i, int j) { return (i & 31) * 16 + (i >> 5) * 4 + j; }
__device__ __forceinline__ void store_scale_tile(const uint8_t* staged, uint8_t* scales) {
    __syncthreads();
    if (threadIdx.x < 32)
        reinterpret_cast<uint4*>(scales + (int64_t)blockIdx.x * 512)[threadIdx.x] = reinterpret_cast<const uint4*>(staged)[threadIdx.x];
}

// cols % 8 == 0: a lane's eight elements are 16 or 32 aligned bytes.
template <typename T, bool DEQ>
__global__ void __launch_bounds__(kRowThreads<T>, kRowCtas<T>) mx4_rows_vec(const T* __restrict__ x, int64_t rows, int cols, int tiles_k,
                                                                         uint8_t* __restrict__ codes, int code_pitch,
                                                                         uint8_t* __restrict__ scales, T* __restrict__ y) {
    constexpr int kHalves = kHalvesOf<T>, kSegs = 128 / kHalves;
    __shared__ __align__(16) uint8_t staged[512];
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const Tile tile(tiles_k);
    const int c = tile.kt * 128 + lane * 8;
    const int left = rows_left(tile.r0, rows, half);
    const int in = c < cols ? left : 0, out = c / 2 < code_pitch ? left : 0;   // rows to read, to write codes of
    const int64_t at = (tile.r0 + half) * cols + c, step = (int64_t)kHalves * cols;
    const T* p = x + at;
    T* o = y + at;
    uint8_t* q = codes + (tile.r0 + half) * code_pitch + c / 2;
    Raw8<T> raw[kSegs];
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
        if (i * kHalves < in) raw[i].load(p);
        p += step;
    }
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
        uint32_t m = raw[i].max_bits();
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const Shared sh(m);
        const int b = sh.byte();
        const uint32_t code = raw[i].codes(sh);
        if ((lane & 3) == 0) staged[staged_scale(i * kHalves + half, lane >> 2)] = (uint8_t)b;
        if (i * kHalves < out) *reinterpret_cast<uint32_t*>(q) = code;
        q += (int64_t)kHalves * code_pitch;
        if (DEQ) {
            if (i * kHalves < in) {
                float d[8];
                unpack8(code, scale_value(b), d);
                store8(o, d);
            }
            o += step;
        }
    }
    store_scale_tile(staged, scales);
}

// Any width.  A row of the tile starts `shift` elements behind a 16-byte
// boundary, the same for all rows of a thread (they are a multiple of eight
// apart).  Lane l takes the aligned vectors from 8 l - shift on and works on
// them in place: of lanes 0, 4, 8 and 12 the first `shift` elements (lo) belong
// to the block before, so these lanes have two maxima and two scales.  Only the
// codes are shifted, by a funnel shift of a lane's and the next lane's.  The
// last `shift` elements of a tile's row lie in one vector more: those a half
// warp needs are held by its first lanes and finished together, after the rows.
// A first version shifted the elements themselves, and the dequantised ones
// back: 222283 x 1023 bf16 174 us, 340 with the copy, now 146 and 255; 65537 x
// 1003 fp32 76 and 127, now 64 and 109.  Bound by the ALU pipe (80% busy).

// Which elements of eight are the first n: masks of packed pairs, or n itself.
template <typename T>
struct Lo;
template <>
struct Lo<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ explicit Lo(int n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = Raw8<__nv_bfloat16>::first(0xFFFFFFFFu, n - 2 * k);
    }
    __device__ __forceinline__ uint32_t pick(int k, uint32_t lo, uint32_t hi) const { return (w[k] & lo) | (~w[k] & hi); }
};
template <>
struct Lo<float> {
    int n;   // below 4
    __device__ __forceinline__ explicit Lo(int n_) : n(n_) {}
    __device__ __forceinline__ float pick(int u, float lo, float hi) const { return u < 3 && u < n ? lo : hi; }
};

__device__ __forceinline__ void max_split(const Raw8<__nv_bfloat16>& e, const Lo<__nv_bfloat16>& l, uint32_t& lo, uint32_t& hi) {
    const uint32_t x[4] = {e.r.x, e.r.y, e.r.z, e.r.w};
    uint32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        a[k] = x[k] & l.w[k];
        b[k] = x[k] & ~l.w[k];
    }
    const uint32_t m = absmax_bf16x2(absmax_bf16x2(a[0], a[1]), absmax_bf16x2(a[2], a[3]));
    const uint32_t n = absmax_bf16x2(absmax_bf16x2(b[0], b[1]), absmax_bf16x2(b[2], b[3]));
    lo = max(m << 16, m & 0xFFFF0000u);
    hi = max(n << 16, n & 0xFFFF0000u);
}
__device__ __forceinline__ void max_split(const Raw8<float>& e, const Lo<float>& l, uint32_t& lo, uint32_t& hi) {
    lo = __float_as_uint(absmax3(l.pick(0, e.a.x, 0.f), l.pick(1, e.a.y, 0.f), l.pick(2, e.a.z, 0.f)));
    hi = __float_as_uint(absmax3(absmax3(l.pick(0, 0.f, e.a.x), l.pick(1, 0.f, e.a.y), l.pick(2, 0.f, e.a.z)),
                                 absmax3(e.a.w, e.b.x, e.b.y), absmax3(e.b.z, e.b.w, 0.f)));
}

// Eight elements as codes, the lo ones scaled by one power of two (packed bf16;
// fp32 takes the upper half).
__device__ __forceinline__ uint32_t split_codes(const Raw8<__nv_bfloat16>& e, const Lo<__nv_bfloat16>& l, uint32_t p, uint32_t q) {
    float f[8];
    scaled(e.r.x, l.pick(0, p, q), f[0], f[1]);
    scaled(e.r.y, l.pick(1, p, q), f[2], f[3]);
    scaled(e.r.z, l.pick(2, p, q), f[4], f[5]);
    scaled(e.r.w, l.pick(3, p, q), f[6], f[7]);
    return cvt8(f);
}
__device__ __forceinline__ uint32_t split_codes(const Raw8<float>& e, const Lo<float>& l, uint32_t p2, uint32_t q2) {
    const float p = __uint_as_float(p2 & 0xFFFF0000u), q = __uint_as_float(q2 & 0xFFFF0000u);
    const float f[8] = {e.a.x * l.pick(0, p, q), e.a.y * l.pick(1, p, q), e.a.z * l.pick(2, p, q), e.a.w * q,
                        e.b.x * q, e.b.y * q, e.b.z * q, e.b.w * q};
    return cvt8(f);
}

// The values of eight codes as they are stored.
__device__ __forceinline__ void split_values(uint32_t code, const Lo<__nv_bfloat16>& l, int b_lo, int b_hi, uint32_t (&w)[4]) {
    const uint32_t p = mx4::scale_bf16x2(b_lo), q = mx4::scale_bf16x2(b_hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = mx4::value_bf16x2(code >> (8 * k), l.pick(k, p, q));
}
__device__ __forceinline__ void split_values(uint32_t code, const Lo<float>& l, int b_lo, int b_hi, uint32_t (&w)[8]) {
    const float p = scale_value(b_lo), q = scale_value(b_hi);
    float f[8];
    unpack8(code, 1.f, f);
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = __float_as_uint(f[u] * l.pick(u, p, q));
}

// The half words of an aligned vector (four words) from s on, and before s, in
// at most three stores.
__device__ __forceinline__ void store_from(uint16_t* p, const uint32_t* w, int s) {
    if (s & 1) p[s] = (uint16_t)((s & 4 ? (s & 2 ? w[3] : w[2]) : (s & 2 ? w[1] : w[0])) >> 16);
    const int a = (s + 1) >> 1;   // first whole word
    if (a & 1) reinterpret_cast<uint32_t*>(p)[a] = a & 2 ? w[3] : w[1];
    if (a > 0 && a < 3) reinterpret_cast<uint2*>(p)[1] = make_uint2(w[2], w[3]);
}
__device__ __forceinline__ void store_before(uint16_t* p, const uint32_t* w, int s) {
    if (s & 4) reinterpret_cast<uint2*>(p)[0] = make_uint2(w[0], w[1]);
    if (s & 2) reinterpret_cast<uint32_t*>(p)[s & 4 ? 2 : 0] = s & 4 ? w[2] : w[0];
    if (s & 1) p[s - 1] = (uint16_t)(s & 4 ? (s & 2 ? w[3] : w[2]) : (s & 2 ? w[1] : w[0]));
}

// The operand of the transpose: blocks are 32 consecutive rows of a column.
// A CTA takes 128 rows x 128 columns, which is one 512-byte scale tile of the
// result; a thread holds 32 rows of CPT adjacent columns (all 32 loads in
// flight, a warp's load 64 to 128 contiguous bytes), and the codes go through
// shared memory so that each column's 64 bytes leave together.
constexpr int kTile = 128;
constexpr int kStagePitch = 80;   // bytes per column: 64 of codes, padded to spread the banks

// The staged codes ([column][64 bytes]) and scales ([column][block]) of a tile
// to the operand of the transpose.
__device__ __forceinline__ void store_col_tile(const uint8_t* s_codes, const uint8_t* s_scale, int64_t rt, int ct, int cols,
                                               int64_t blocks_k, int64_t tiles_k, uint8_t* codes, uint8_t* scales) {
    __syncthreads();
    // 16 bytes of codes per step: four consecutive threads write a column's 64
    for (int i = threadIdx.x; i < kTile * 4; i += blockDim.x) {
        const int col = i >> 2, part = i & 3;
        if (ct * kTile + col < cols && rt * 4 + part < blocks_k)
            *reinterpret_cast<uint4*>(codes + ((int64_t)(ct * kTile + col) * blocks_k + rt * 4 + part) * 16) =
                *reinterpret_cast<const uint4*>(s_codes + col * kStagePitch + part * 16);
    }
    // the scale tile: word w holds column (w % 4) * 32 + w / 4
    if (threadIdx.x < kTile) {
        const int w = threadIdx.x;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(s_scale + ((w & 3) * 32 + (w >> 2)) * 4);
        *reinterpret_cast<uint32_t*>(scales + ((int64_t)ct * tiles_k + rt) * 512 + w * 4) = word;
    }
}

// A row's elements of a lane's columns; of R rows the scale bytes (PAIRED: of
// the block's rows that this lane and lane ^ 16 hold) and the codes.
template <typename T, int CPT>
struct Cols;
template <int CPT>
struct Cols<__nv_bfloat16, CPT> {
    uint32_t raw = 0;   // CPT == 1: in the lower half
    __device__ void load(const __nv_bfloat16* p) {
        raw = CPT == 2 ? __ldg(reinterpret_cast<const unsigned int*>(p)) : __ldg(reinterpret_cast<const unsigned short*>(p));
    }
    __device__ void take(const uint8_t* s) {   // from shared memory
        raw = CPT == 2 ? *reinterpret_cast<const uint32_t*>(s) : *reinterpret_cast<const uint16_t*>(s);
    }
    template <int R, bool PAIRED>
    __device__ static void quantize(const Cols (&v)[R], int (&b)[CPT], uint32_t (&code)[CPT][R / 8]) {
        uint32_t k = 0;
#pragma unroll
        for (int t = 0; t < R; ++t) k = absmax_bf16x2(k, v[t].raw);
        if (PAIRED) k = absmax_bf16x2(k, __shfl_xor_sync(0xffffffffu, k, 16));
        const int lo = Shared(k << 16).byte(), hi = Shared(k & 0xFFFF0000u).byte();
        const uint32_t s = ((uint32_t)(254 - min(lo, 253)) << 7) | ((uint32_t)(254 - min(hi, 253)) << 23);
        b[0] = lo;
        b[CPT - 1] = CPT == 2 ? hi : lo;
#pragma unroll
        for (int w = 0; w < R / 8; ++w) {
            float f[8], g[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) scaled(v[8 * w + u].raw, s, f[u], g[u]);
            code[0][w] = lo == mx4::kNanScale ? 0u : cvt8(f);
            if (CPT == 2) code[CPT - 1][w] = hi == mx4::kNanScale ? 0u : cvt8(g);
        }
    }
    __device__ static void store(__nv_bfloat16* p, float a, float b) {
        if (CPT == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
        else *p = __float2bfloat16_rn(a);
    }
};
template <>
struct Cols<float, 1> {
    float raw = 0.f;
    __device__ void load(const float* p) { raw = __ldg(p); }
    __device__ void take(const uint8_t* s) { raw = *reinterpret_cast<const float*>(s); }
    template <int R, bool PAIRED>
    __device__ static void quantize(const Cols (&v)[R], int (&b)[1], uint32_t (&code)[1][R / 8]) {
        static_assert(!PAIRED, "a lane holds whole blocks");
        float k = 0.f;
#pragma unroll
        for (int t = 0; t < R; t += 2) k = absmax3(k, v[t].raw, v[t + 1].raw);
        const Shared sh(__float_as_uint(k));
        const float s = sh.inv();
        b[0] = sh.byte();
#pragma unroll
        for (int w = 0; w < R / 8; ++w) {
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = v[8 * w + u].raw;
            code[0][w] = sh.nan ? 0u : pack8(f, s);
        }
    }
    __device__ static void store(float* p, float a, float) { *p = a; }
};

// CTAs an SM should hold, us: fp32 2 / 3 (65537 x 1003) 54 / 58, with the copy
// 99 / 113 (three spill); bf16, one column per thread, 2 / 3 (222283 x 1023, with
// the copy) 252 / 246; two columns 3 / 4 / 5 (222283 x 1024) 103 / 93 / 93, with
// the copy 166 / 167 / 170, a million rows of 100 with it 84 / 78 / 76.
template <typename T, int CPT>
constexpr int kColCtas = sizeof(T) == 4 ? 2 : CPT == 2 ? 4 : 3;

template <typename T, int CPT, bool DEQ>
__global__ void __launch_bounds__(512 / CPT, kColCtas<T, CPT>) mx4_cols(const T* __restrict__ x, int64_t rows, int cols,
                                                      int col_tiles, int64_t blocks_k, int64_t tiles_k,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, T* __restrict__ y) {
    __shared__ __align__(16) uint8_t s_codes[kTile * kStagePitch];
    __shared__ __align__(4) uint8_t s_scale[4 * kTile];   // [column][block]
    constexpr int kLanes = kTile / CPT;      // threads across the columns
    const Tile tile(col_tiles);   // the row tile is the operand's k tile
    const int64_t rt = tile.rt;
    const int ct = tile.kt;
    const int cl = (threadIdx.x % kLanes) * CPT, blk = threadIdx.x / kLanes;
    const int c = ct * kTile + cl;
    const int64_t r0 = rt * kTile + blk * 32;
    const int n = (int)(rows - r0 < 32 ? rows - r0 : 32);   // may be negative
    Cols<T, CPT> v[32];
    if (c < cols) {
        const T* p = x + r0 * cols + c;
#pragma unroll
        for (int t = 0; t < 32; ++t) {
            if (t < n) v[t].load(p);
            p += cols;
        }
    }
    uint32_t code[CPT][4];
    int b[CPT];
    Cols<T, CPT>::template quantize<32, false>(v, b, code);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        *reinterpret_cast<uint4*>(s_codes + (cl + i) * kStagePitch + blk * 16) =
            make_uint4(code[i][0], code[i][1], code[i][2], code[i][3]);
        s_scale[(cl + i) * 4 + blk] = (uint8_t)b[i];
    }
    if (DEQ && c < cols) {
        T* p = y + r0 * cols + c;
        const float k0 = scale_value(b[0]), k1 = scale_value(b[CPT - 1]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float d0[8], d1[8];
            unpack8(code[0][w], k0, d0);
            unpack8(code[CPT - 1][w], k1, d1);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (8 * w + u < n) Cols<T, CPT>::store(p, d0[u], d1[u]);
                p += cols;
            }
        }
    }
    store_col_tile(s_codes, s_scale, rt, ct, cols, blocks_k, tiles_k, codes, scales);
}

// COLS: the operand of the transpose, alone or as well; the elements go through
// shared memory as the vectors hold them, a row of the tile 16 bytes longer than
// its 128 elements, and a lane then takes 32 rows of a column.  Both operands in
// one pass instead of two: 65537 x 1003 bf16 97 -> 68 us, fp32 122 -> 91, 65537
// x 4093 bf16 337 -> 240.  Alone, 222283 x 1023 bf16: 123 us, 146 by columns
// from global memory (mx4_cols, whose fp32 keeps up: 5.5 TB/s).
template <typename T>
constexpr int kAnyPitch = kTile * (int)sizeof(T) + 16;
template <typename T>
constexpr int kAnySmem = kTile * (kAnyPitch<T> + kStagePitch + 4);

template <typename T, bool ROWS, bool DEQ, bool COLS>
__global__ void __launch_bounds__(kRowThreads<T>, kAnyCtas<T>) mx4_any(const T* __restrict__ x, int64_t rows, int cols, int tiles_k,
                                                                         uint8_t* __restrict__ codes, int code_pitch,
                                                                         uint8_t* __restrict__ scales, T* __restrict__ y,
                                                                         int64_t t_blocks, int64_t t_tiles,
                                                                         uint8_t* __restrict__ t_codes,
                                                                         uint8_t* __restrict__ t_scales) {
    extern __shared__ __align__(16) uint8_t smem[];   // COLS: elements, codes and scales of the columns
    constexpr int kHalves = kHalvesOf<T>, kSegs = 128 / kHalves;
    constexpr int V = 16 / sizeof(T), N = 8 / V, H = sizeof(T) / 2;   // elements of a vector, vectors of eight, half words
    __shared__ __align__(16) uint8_t staged[512];
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const Tile tile(tiles_k);
    const int left = rows_left(tile.r0, rows, half);
    const int c0 = tile.kt * 128, lim = min(cols, c0 + 128);
    const int64_t row = (tile.r0 + half) * cols, step = (int64_t)kHalves * cols;
    const int shift = (int)(row & (V - 1)), c = c0 + lane * 8 - shift;   // the lane's first column
    const T* const end = x + rows * cols;
    const T* p = x + row + c;
    // eight elements' worth of vectors, or one vector
    auto load = [&](Raw8<T>& e, const T* from, int col, bool one) {
        uint32_t w[4 * N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if ((n == 0 || !one) && col + n * V < cols) {
                if (from + (n + 1) * V <= end) {
                    v = __ldg(reinterpret_cast<const uint4*>(from + n * V));
                } else {
                    T* t = reinterpret_cast<T*>(&v);   // the tensor ends inside this vector
#pragma unroll
                    for (int u = 0; u < V; ++u)
                        if (from + n * V + u < end) t[u] = from[n * V + u];
                }
            }
            w[4 * n] = v.x;
            w[4 * n + 1] = v.y;
            w[4 * n + 2] = v.z;
            w[4 * n + 3] = v.w;
        }
        e.words(w);
    };
    Raw8<T> raw[kSegs], ext;
    if (tile.r0 + 128 + 8 <= rows) {   // eight rows more are at least a vector
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
            uint32_t w[4 * N] = {};
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (c + n * V < cols) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + n * V));
                    w[4 * n] = v.x;
                    w[4 * n + 1] = v.y;
                    w[4 * n + 2] = v.z;
                    w[4 * n + 3] = v.w;
                }
            raw[i].words(w);
            p += step;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
            if (i * kHalves < left) load(raw[i], p, c, false);
            p += step;
        }
    }
    // lane i < kSegs: the vector behind row i's last lane
    const int ext_col = c0 + 128 - shift, ext_n = min(max(cols - ext_col, 0), shift);
    if (lane < kSegs && lane * kHalves < left && ext_n > 0) load(ext, x + row + lane * step + ext_col, ext_col, true);
    ext.clip(ext_n);
    const uint32_t ext_max = ext.max_bits();

    const int lo_n = lane & 3 ? 0 : shift;
    const Lo<T> lo(lo_n);
    const uint32_t lo_codes = (1u << (4 * lo_n)) - 1u;
    uint8_t* q = codes + (tile.r0 + half) * code_pitch + c0 / 2 + lane * 4;
    const int out = c0 + lane * 8 < 2 * code_pitch ? left : 0;
    T* o = y + row + c;
    uint32_t ext_m = 0u, ext_code = 0u;
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
        if (c + 8 > cols) raw[i].clip(cols - c);   // the rest is the next row's
        if (COLS) raw[i].put_vectors(smem + (i * kHalves + half) * kAnyPitch<T> + lane * 8 * (int)sizeof(T));
        if (!ROWS) continue;
        uint32_t m_lo, m;
        max_split(raw[i], lo, m_lo, m);
        const uint32_t behind = __shfl_down_sync(0xffffffffu, m_lo, 1, 16), last = __shfl_sync(0xffffffffu, ext_max, i, 16);
        m = max(m, lane == 15 ? last : behind);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const Shared sh(m);
        const uint32_t inv = sh.inv_bf16x2();
        const int b = sh.byte();
        uint32_t code = split_codes(raw[i], lo, __shfl_up_sync(0xffffffffu, inv, 1, 16), inv);
        if (__any_sync(0xffffffffu, sh.nan)) {
            const bool nan_lo = __shfl_up_sync(0xffffffffu, b, 1, 16) == mx4::kNanScale;
            code &= (nan_lo ? 0u : lo_codes) | (sh.nan ? 0u : ~lo_codes);
        }
        const uint32_t next = __shfl_down_sync(0xffffffffu, code, 1, 16);
        const uint32_t m15 = __shfl_sync(0xffffffffu, m, 15, 16), c15 = __shfl_sync(0xffffffffu, code, 15, 16);
        if (lane == i) {
            ext_m = m15;
            ext_code = c15;
        }
        if ((lane & 3) == 0) staged[staged_scale(i * kHalves + half, lane >> 2)] = (uint8_t)b;
        if (lane < 15 && i * kHalves < out) *reinterpret_cast<uint32_t*>(q) = __funnelshift_r(code, next, 4 * shift);
        q += (int64_t)kHalves * code_pitch;
        if (DEQ) {
            const int b_lo = __shfl_up_sync(0xffffffffu, b, 1, 16);
            if (i * kHalves < left) {
                uint32_t w[4 * N];
                split_values(code, lo, b_lo, b, w);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int at = c + n * V;
                    uint16_t* const to = reinterpret_cast<uint16_t*>(o + n * V);
                    if (at >= c0 && at + V <= lim) {
                        *reinterpret_cast<uint4*>(to) = make_uint4(w[4 * n], w[4 * n + 1], w[4 * n + 2], w[4 * n + 3]);
                    } else if (at >= c0) {
                        if (at < lim) store_before(to, w + 4 * n, (lim - at) * H);
                    } else if (at + V <= lim) {
                        store_from(to, w + 4 * n, shift * H);
                    } else {   // a row within one vector
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (u >= shift * H && u < (lim - at) * H) to[u] = (uint16_t)(w[4 * n + u / 2] >> (16 * (u & 1)));
                    }
                }
            }
            o += step;
        }
    }
    if (COLS && lane < kSegs) ext.put_vector(smem + (lane * kHalves + half) * kAnyPitch<T> + kTile * (int)sizeof(T));
    // the rows' last lanes: their codes with the ones behind, and the values of those
    if (ROWS && lane < kSegs && lane * kHalves < left) {
        const Shared sh(ext_m);
        const uint32_t code = ext.codes(sh);
        if (c0 + 120 < 2 * code_pitch)
            *reinterpret_cast<uint32_t*>(codes + (tile.r0 + half + lane * kHalves) * code_pitch + c0 / 2 + 60) =
                __funnelshift_r(ext_code, code, 4 * shift);
        if (DEQ && ext_n > 0) {
            uint32_t w[4 * N];
            split_values(code, Lo<T>(0), sh.byte(), sh.byte(), w);
            store_before(reinterpret_cast<uint16_t*>(y + row + lane * step + ext_col), w, ext_n * H);
        }
    }
    if (ROWS) store_scale_tile(staged, scales);
    if (COLS) {
        __syncthreads();   // the elements are complete
        uint8_t* const s_codes = smem + kTile * kAnyPitch<T>;
        uint8_t* const s_scale = s_codes + kTile * kStagePitch;
        const int warp = threadIdx.x >> 5, blk = warp & 3;
#pragma unroll 1
        for (int h = 0; h < 4 * 128 / kRowThreads<T>; ++h) {
            const int cl = ((warp >> 2) + h * (kRowThreads<T> / 128)) * 32 + (threadIdx.x & 31);
            Cols<T, 1> v[32];
            const uint8_t* const from = smem + blk * 32 * kAnyPitch<T> + cl * (int)sizeof(T);
#pragma unroll
            for (int t = 0; t < 32; ++t)   // row t of the block starts t * cols elements, modulo a vector, behind a boundary
                v[t].take(from + t * kAnyPitch<T> + ((t * (cols & (V - 1))) & (V - 1)) * (int)sizeof(T));
            uint32_t code[1][4];
            int b[1];
            Cols<T, 1>::template quantize<32, false>(v, b, code);
            *reinterpret_cast<uint4*>(s_codes + cl * kStagePitch + blk * 16) = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
            s_scale[cl * 4 + blk] = (uint8_t)b[0];
        }
        store_col_tile(s_codes, s_scale, tile.rt, tile.kt, cols, t_blocks, t_tiles, t_codes, t_scales);
    }
}

// Both operands of x in one pass over it: rows as mx4_rows_vec, and the tile
// through shared memory for the columns, as raw elements in 16-byte chunks.
// Chunk j of row i lies at j ^ (i & 7) ^ (i & 16 ? 4 : 0): a half warp writes a
// row's chunks, and in bf16 reads two rows 16 apart, without bank conflicts.
// bf16: a lane takes two columns x 16 rows, two lanes a block; fp32: a column
// x 32 rows.
template <typename T>
constexpr int kBothSmem = kTile * kTile * (int)sizeof(T) + kTile * kStagePitch + 4 * kTile + 512;

template <typename T>
__device__ __forceinline__ int chunk_at(int i, int j) {
    return i * (kTile * (int)sizeof(T)) + ((j ^ (i & 7) ^ (i & 16 ? 4 : 0)) << 4);
}

__device__ __forceinline__ void Raw8<__nv_bfloat16>::put(uint8_t* s, int row, int lane) const {
    *reinterpret_cast<uint4*>(s + chunk_at<__nv_bfloat16>(row, lane)) = r;
}
__device__ __forceinline__ void Raw8<float>::put(uint8_t* s, int row, int lane) const {
    *reinterpret_cast<float4*>(s + chunk_at<float>(row, 2 * lane)) = a;
    *reinterpret_cast<float4*>(s + chunk_at<float>(row, 2 * lane + 1)) = b;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads<T>, kRowCtas<T>) mx4_both(const T* __restrict__ x, int64_t rows, int cols, int tiles_k,
                                                                     uint8_t* __restrict__ codes, int code_pitch,
                                                                     uint8_t* __restrict__ scales, int64_t t_blocks,
                                                                     int64_t t_tiles, uint8_t* __restrict__ t_codes,
                                                                     uint8_t* __restrict__ t_scales) {
    constexpr int kHalves = kHalvesOf<T>, kSegs = 128 / kHalves;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* const s_x = smem;
    uint8_t* const s_codes = s_x + kTile * kTile * sizeof(T);
    uint8_t* const s_scale = s_codes + kTile * kStagePitch;
    uint8_t* const staged = s_scale + 4 * kTile;
    const Tile tile(tiles_k);
    {
        const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
        const int c = tile.kt * 128 + lane * 8;
        const int left = rows_left(tile.r0, rows, half);
        const int in = c < cols ? left : 0, out = c / 2 < code_pitch ? left : 0;
        const T* p = x + (tile.r0 + half) * cols + c;
        uint8_t* q = codes + (tile.r0 + half) * code_pitch + c / 2;
        Raw8<T> raw[kSegs];
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
            if (i * kHalves < in) raw[i].load(p);
            p += (int64_t)kHalves * cols;
        }
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
            const int row = i * kHalves + half;
            raw[i].put(s_x, row, lane);
            uint32_t m = raw[i].max_bits();
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const Shared sh(m);
            const uint32_t code = raw[i].codes(sh);
            if ((lane & 3) == 0) staged[staged_scale(row, lane >> 2)] = (uint8_t)sh.byte();
            if (i * kHalves < out) *reinterpret_cast<uint32_t*>(q) = code;
            q += (int64_t)kHalves * code_pitch;
        }
    }
    store_scale_tile(staged, scales);   // and the tile is complete
    {
        constexpr int CPT = sizeof(T) == 2 ? 2 : 1, R = 32 / CPT, kCols = 32;   // columns and rows a lane, columns a warp
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int blk = warp & 3;
        const int row0 = blk * 32 + (CPT == 2 ? (lane >> 4) * 16 : 0);
#pragma unroll 1
        for (int h = 0; h < kTile / kCols * 128 / kRowThreads<T>; ++h) {
            const int cl = ((warp >> 2) + h * (kRowThreads<T> / 128)) * kCols + (CPT == 2 ? (lane & 15) * 2 : lane);
            Cols<T, CPT> v[R];
#pragma unroll
            for (int t = 0; t < R; ++t)
                v[t].take(s_x + chunk_at<T>(row0 + t, cl * (int)sizeof(T) / 16) + cl * sizeof(T) % 16);
            uint32_t code[CPT][R / 8];
            int b[CPT];
            Cols<T, CPT>::template quantize<R, CPT == 2>(v, b, code);
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                uint8_t* const to = s_codes + (cl + i) * kStagePitch + row0 / 2;
#pragma unroll
                for (int w = 0; w < R / 8; w += 2) *reinterpret_cast<uint2*>(to + 4 * w) = make_uint2(code[i][w], code[i][w + 1]);
                if (CPT == 1 || lane < 16) s_scale[(cl + i) * 4 + blk] = (uint8_t)b[i];
            }
        }
    }
    store_col_tile(s_codes, s_scale, tile.rt, tile.kt, cols, t_blocks, t_tiles, t_codes, t_scales);
}

template <typename T, bool DEQ>
cudaError_t launch_rows(const T* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales, T* y, cudaStream_t st) {
    const int tiles_k = (int)mx4::scale_tiles_k(cols);
    const int64_t grid = mx4::scale_tiles_r(rows) * tiles_k;
    const int pitch = (int)(mx4::padded_cols(cols) / 2);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    prof_begin(st);
    if (cols % 8 == 0) mx4_rows_vec<T, DEQ><<<(unsigned)grid, kRowThreads<T>, 0, st>>>(x, rows, cols, tiles_k, codes, pitch, scales, y);
    else
        mx4_any<T, true, DEQ, false><<<(unsigned)grid, kRowThreads<T>, 0, st>>>(x, rows, cols, tiles_k, codes, pitch, scales, y, 0, 0,
                                                                                nullptr, nullptr);
    prof_end(st, K_MX4_ROWS);
    return cudaGetLastError();
}

template <typename T, int CPT, bool DEQ>
cudaError_t launch_cols(const T* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales, T* y, cudaStream_t st) {
    const int col_tiles = (int)mx4::scale_tiles_r(cols);
    const int64_t grid = mx4::scale_tiles_k(rows) * col_tiles;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    prof_begin(st);
    mx4_cols<T, CPT, DEQ><<<(unsigned)grid, 512 / CPT, 0, st>>>(x, rows, cols, col_tiles, (rows + 31) / 32,
                                                                 mx4::scale_tiles_k(rows), codes, scales, y);
    prof_end(st, K_MX4_COLS);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_both(const T* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales, uint8_t* t_codes,
                        uint8_t* t_scales, cudaStream_t st) {
    const int tiles_k = (int)mx4::scale_tiles_k(cols), pitch = (int)(mx4::padded_cols(cols) / 2);
    const int64_t grid = mx4::scale_tiles_r(rows) * tiles_k, t_blocks = (rows + 31) / 32, t_tiles = mx4::scale_tiles_k(rows);
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const bool vec = cols % 8 == 0;
    const cudaError_t e = vec ? cudaFuncSetAttribute(mx4_both<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBothSmem<T>)
                              : cudaFuncSetAttribute(mx4_any<T, true, false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     kAnySmem<T>);
    if (e != cudaSuccess) return e;
    prof_begin(st);
    if (vec)
        mx4_both<T><<<(unsigned)grid, kRowThreads<T>, kBothSmem<T>, st>>>(x, rows, cols, tiles_k, codes, pitch, scales, t_blocks,
                                                                          t_tiles, t_codes, t_scales);
    else
        mx4_any<T, true, false, true><<<(unsigned)grid, kRowThreads<T>, kAnySmem<T>, st>>>(
            x, rows, cols, tiles_k, codes, pitch, scales, nullptr, t_blocks, t_tiles, t_codes, t_scales);
    prof_end(st, K_MX4_BOTH);
    return cudaGetLastError();
}

// The operand of the transpose of a bf16 x of odd width, without the copy.
cudaError_t launch_cols_odd(const __nv_bfloat16* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
    using T = __nv_bfloat16;
    const int tiles_k = (int)mx4::scale_tiles_k(cols);
    const int64_t grid = mx4::scale_tiles_r(rows) * tiles_k;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const cudaError_t e = cudaFuncSetAttribute(mx4_any<T, false, false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAnySmem<T>);
    if (e != cudaSuccess) return e;
    prof_begin(st);
    mx4_any<T, false, false, true><<<(unsigned)grid, kRowThreads<T>, kAnySmem<T>, st>>>(
        x, rows, cols, tiles_k, nullptr, 0, nullptr, nullptr, (rows + 31) / 32, mx4::scale_tiles_k(rows), codes, scales);
    prof_end(st, K_MX4_COLS);
    return cudaGetLastError();
}

// A bf16 row of an even width is 4-byte aligned, so its columns can be taken
// in pairs; an odd width's go through shared memory or, with the copy, which is
// written by columns too, one by one.
template <bool DEQ>
cudaError_t dispatch(const void* x, int dtype, int64_t rows, int cols, int along_rows, uint8_t* codes,
                     uint8_t* scales, void* y, cudaStream_t st) {
    if (dtype == JFA_F32) {
        const float* p = reinterpret_cast<const float*>(x);
        float* o = reinterpret_cast<float*>(y);
        return along_rows ? launch_cols<float, 1, DEQ>(p, rows, cols, codes, scales, o, st)
                          : launch_rows<float, DEQ>(p, rows, cols, codes, scales, o, st);
    }
    const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(x);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(y);
    if (!along_rows) return launch_rows<__nv_bfloat16, DEQ>(p, rows, cols, codes, scales, o, st);
    if (cols % 2 == 0) return launch_cols<__nv_bfloat16, 2, DEQ>(p, rows, cols, codes, scales, o, st);
    if constexpr (DEQ) return launch_cols<__nv_bfloat16, 1, true>(p, rows, cols, codes, scales, o, st);
    else return launch_cols_odd(p, rows, cols, codes, scales, st);
}

jfa_status check_quantize(const char* who, const void* x, int dtype, int64_t rows, int64_t cols, const uint8_t* codes,
                          const uint8_t* scales, const void* other, const void* other2) {
    if (dtype != JFA_F32 && dtype != JFA_BF16)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: dtype must be JFA_F32 or JFA_BF16", who);
    if (rows < 0 || cols < 0 || rows > kMx4MaxDim || cols > kMx4MaxDim)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: rows and cols in [0, 2^30]", who);
    if (rows == 0 || cols == 0) return JFA_OK;
    if (!x || !codes || !scales) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: NULL tensor", who);
    if (((uintptr_t)x | (uintptr_t)codes | (uintptr_t)scales | (uintptr_t)other | (uintptr_t)other2) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: tensors must be 16-byte aligned", who);
    return JFA_OK;
}

jfa_status quantize_entry(const char* who, const void* x, int dtype, int64_t rows, int64_t cols, int along_rows,
                          uint8_t* codes, uint8_t* scales, void* dequant, jfa_stream_t stream) {
    const jfa_status s = check_quantize(who, x, dtype, rows, cols, codes, scales, dequant, nullptr);
    if (s != JFA_OK || rows == 0 || cols == 0) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dequant ? dispatch<true>(x, dtype, rows, (int)cols, along_rows, codes, scales, dequant, st)
                                  : dispatch<false>(x, dtype, rows, (int)cols, along_rows, codes, scales, nullptr, st);
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return JFA_OK;
}

jfa_status quantize_both(const char* who, const void* x, int dtype, int64_t rows, int64_t cols, uint8_t* codes,
                         uint8_t* scales, uint8_t* t_codes, uint8_t* t_scales, jfa_stream_t stream) {
    const jfa_status s = check_quantize(who, x, dtype, rows, cols, codes, scales, t_codes, t_scales);
    if (s != JFA_OK || rows == 0 || cols == 0) return s;
    if (!t_codes || !t_scales) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "%s: NULL tensor", who);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == JFA_F32 ? launch_both(reinterpret_cast<const float*>(x), rows, (int)cols, codes, scales, t_codes, t_scales, st)
                         : launch_both(reinterpret_cast<const __nv_bfloat16*>(x), rows, (int)cols, codes, scales, t_codes, t_scales, st);
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return JFA_OK;
}

}  // namespace
}  // namespace jfa

extern "C" {

size_t jfa_mxfp4_code_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > jfa::kMx4MaxDim || cols > jfa::kMx4MaxDim) return 0;
    return (size_t)rows * (size_t)(jfa::mx4::padded_cols(cols) / 2);
}

size_t jfa_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > jfa::kMx4MaxDim || cols > jfa::kMx4MaxDim) return 0;
    return (size_t)jfa::mx4::scale_tiles_r(rows) * (size_t)jfa::mx4::scale_tiles_k(cols) * 512;
}

jfa_status jfa_quantize_mxfp4(const void* x, jfa_dtype dtype, int64_t rows, int64_t cols, int along_rows,
                              uint8_t* codes, uint8_t* scales, jfa_stream_t stream) {
    return jfa::quantize_entry("quantize_mxfp4", x, dtype, rows, cols, along_rows, codes, scales, nullptr, stream);
}

jfa_status jfa_quantize_mxfp4_dequant(const void* x, jfa_dtype dtype, int64_t rows, int64_t cols, int along_rows,
                                      uint8_t* codes, uint8_t* scales, void* dequant, jfa_stream_t stream) {
    if (rows > 0 && cols > 0 && !dequant)
        return jfa::set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4_dequant: NULL dequant");
    return jfa::quantize_entry("quantize_mxfp4_dequant", x, dtype, rows, cols, along_rows, codes, scales, dequant, stream);
}

jfa_status jfa_quantize_mxfp4_both(const void* x, jfa_dtype dtype, int64_t rows, int64_t cols, uint8_t* codes,
                                   uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t, jfa_stream_t stream) {
    return jfa::quantize_both("quantize_mxfp4_both", x, dtype, rows, cols, codes, scales, codes_t, scales_t, stream);
}

}  // extern "C"
