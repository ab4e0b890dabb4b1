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

using mx4::inv_scale;
using mx4::pack2;
using mx4::scale_byte;
using mx4::scale_value;
using mx4::scale_word;
using mx4::unpack2;

// Eight consecutive elements as floats, and the bits of their largest
// magnitude as an fp32 number (infinities and NaN compare above every finite
// number, so an exponent field of 255 survives the maximum).
__device__ __forceinline__ uint32_t load8(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(p));
    const __nv_bfloat162* p2 = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const float2 v = __bfloat1622float2(p2[u]);
        f[2 * u] = v.x;
        f[2 * u + 1] = v.y;
    }
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(f[u]) & 0x7FFFFFFFu);
    return m;
}
__device__ __forceinline__ uint32_t load8(const float* p, float (&f)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(f[u]) & 0x7FFFFFFFu);
    return m;
}
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

// Work unit of the row kernels: a segment, 128 columns (four blocks, one
// scale word) of one row.  Segments of rows up to the next multiple of 128
// are visited too: those behind the last row only write their zero scale
// word, so that every byte of the scale tiles is defined.
constexpr int kSegsPerHalfWarp = 4;
constexpr int kRowThreads = 256;
constexpr int kSegsVec = kRowThreads / 16 * kSegsPerHalfWarp;   // segments per CTA

// cols % 8 == 0: sixteen lanes take a segment, eight elements (16 or 32 bytes)
// each; the loads of a half warp's four segments are all in flight before the
// first conversion.
template <typename T, bool DEQ>
__global__ void __launch_bounds__(kRowThreads) mx4_rows_vec(const T* __restrict__ x, int64_t rows, int cols,
                                                            int64_t segs, int tiles_k,
                                                            uint8_t* __restrict__ codes, int code_pitch,
                                                            uint8_t* __restrict__ scales, T* __restrict__ y) {
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int64_t seg0 = (int64_t)blockIdx.x * kSegsVec;
    const int64_t row0 = seg0 / tiles_k;
    const int kt0 = (int)(seg0 - row0 * tiles_k);
    float f[kSegsPerHalfWarp][8];
    uint32_t m[kSegsPerHalfWarp];
#pragma unroll
    for (int i = 0; i < kSegsPerHalfWarp; ++i) {
        const unsigned at = (unsigned)(kt0 + i * (kRowThreads / 16) + half);
        const int64_t r = row0 + at / (unsigned)tiles_k;
        const int c = (int)(at % (unsigned)tiles_k) * 128 + lane * 8;
        m[i] = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) f[i][u] = 0.f;
        if (r < rows && c < cols) m[i] = load8(x + r * cols + c, f[i]);
    }
#pragma unroll
    for (int i = 0; i < kSegsPerHalfWarp; ++i) {
        const int local = i * (kRowThreads / 16) + half;
        const unsigned at = (unsigned)(kt0 + local);
        const int64_t r = row0 + at / (unsigned)tiles_k;
        const int kt = (int)(at % (unsigned)tiles_k), c = kt * 128 + lane * 8;
        uint32_t mx = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int b = scale_byte(mx);
        const float s = inv_scale(b);
        uint32_t code = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) code |= pack2(f[i][2 * u] * s, f[i][2 * u + 1] * s) << (8 * u);
        if (b == mx4::kNanScale) code = 0;
        // the word of the segment's four scale bytes, in every fourth lane's byte
        uint32_t word = (uint32_t)b << (8 * (lane >> 2));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if (seg0 + local >= segs) continue;
        if (lane == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(r, kt, tiles_k)) = word;
        if (r >= rows) continue;
        if (c / 2 < code_pitch) *reinterpret_cast<uint32_t*>(codes + r * code_pitch + c / 2) = code;
        if (DEQ && c < cols) {
            const float back = scale_value(b);
            float d[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 v = unpack2((code >> (8 * u)) & 0xFF);
                d[2 * u] = v.x * back;
                d[2 * u + 1] = v.y * back;
            }
            store8(y + r * cols + c, d);
        }
    }
}

// Any width: a warp takes a segment, lane l the element l of each of its four
// blocks (rows need not be aligned; a warp's load is 32 consecutive elements).
// The block maximum is one warp reduction; codes are packed by a shuffle with
// the neighbour (two codes to a byte) and a 4 x 4 byte transpose among the
// even lanes of eight, after which each holds four bytes of one block.
constexpr int kSegsPerWarp = 4;
constexpr int kSegsAny = kRowThreads / 32 * kSegsPerWarp;

__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) {
    return __bfloat162float(__ushort_as_bfloat16(__ldg(reinterpret_cast<const unsigned short*>(p))));
}

template <typename T, bool DEQ>
__global__ void __launch_bounds__(kRowThreads) mx4_rows_any(const T* __restrict__ x, int64_t rows, int cols,
                                                            int64_t segs, int tiles_k,
                                                            uint8_t* __restrict__ codes, int code_pitch,
                                                            uint8_t* __restrict__ scales, T* __restrict__ y) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t seg0 = (int64_t)blockIdx.x * kSegsAny;
    const int64_t row0 = seg0 / tiles_k;
    const int kt0 = (int)(seg0 - row0 * tiles_k);
    float f[kSegsPerWarp][4];
#pragma unroll
    for (int i = 0; i < kSegsPerWarp; ++i) {
        const unsigned at = (unsigned)(kt0 + i * (kRowThreads / 32) + warp);
        const int64_t r = row0 + at / (unsigned)tiles_k;
        const int c = (int)(at % (unsigned)tiles_k) * 128 + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i][j] = (r < rows && c + 32 * j < cols) ? load1(x + r * cols + c + 32 * j) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kSegsPerWarp; ++i) {
        const int local = i * (kRowThreads / 32) + warp;
        if (seg0 + local >= segs) return;   // whole warps leave together
        const unsigned at = (unsigned)(kt0 + local);
        const int64_t r = row0 + at / (unsigned)tiles_k;
        const int kt = (int)(at % (unsigned)tiles_k);
        uint32_t word = 0, four = 0;   // scale bytes; this lane's four codes, a byte each
        int b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            b[j] = scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(f[i][j]) & 0x7FFFFFFFu));
            word |= (uint32_t)b[j] << (8 * j);
            const uint32_t code = b[j] == mx4::kNanScale ? 0u : pack2(f[i][j] * inv_scale(b[j]), 0.f);
            four |= code << (8 * j);
        }
        if (lane == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(r, kt, tiles_k)) = word;
        if (r >= rows) continue;
        // even lanes: byte j = codes (2i, 2i + 1) of block j
        const uint32_t pair = four | (__shfl_down_sync(0xffffffffu, four, 1) << 4);
        // transpose among lanes 0, 2, 4, 6 of eight: lane 2q ends with block q's
        // bytes.  First the 2 x 2 blocks of bytes (lanes 4 apart), then within
        // them (lanes 2 apart).
        const int q = (lane >> 1) & 3;
        uint32_t o = __shfl_xor_sync(0xffffffffu, pair, 4);
        uint32_t t = (q & 2) ? __byte_perm(o, pair, 0x7632) : __byte_perm(pair, o, 0x5410);
        o = __shfl_xor_sync(0xffffffffu, t, 2);
        t = (q & 1) ? __byte_perm(o, t, 0x7351) : __byte_perm(t, o, 0x6240);
        const int byte = kt * 64 + q * 16 + (lane >> 3) * 4;
        if ((lane & 1) == 0 && byte < code_pitch) *reinterpret_cast<uint32_t*>(codes + r * code_pitch + byte) = t;
        if (DEQ) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = kt * 128 + 32 * j + lane;
                if (c < cols) y[r * cols + c] = from_f<T>(unpack2((four >> (8 * j)) & 0xF).x * scale_value(b[j]));
            }
        }
    }
}

// The operand of the transpose: blocks are 32 consecutive rows of a column.
// A CTA takes 128 rows x 128 columns, which is one 512-byte scale tile of the
// result; a thread holds 32 rows of CPT adjacent columns (all 32 loads in
// flight, a warp's load 64 to 128 contiguous bytes), and the codes go through
// shared memory so that each column's 64 bytes leave together.
constexpr int kTile = 128;
constexpr int kStagePitch = 80;   // bytes per column: 64 of codes, padded to spread the banks

template <typename T, int CPT>
struct Cols;
template <>
struct Cols<__nv_bfloat16, 2> {
    uint32_t raw = 0;
    __device__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const unsigned int*>(p)); }
    __device__ float get(int i) const { return __uint_as_float(i ? (raw & 0xFFFF0000u) : (raw << 16)); }
    __device__ static void store(__nv_bfloat16* p, float a, float b) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
    }
};
template <>
struct Cols<__nv_bfloat16, 1> {
    uint32_t raw = 0;
    __device__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const unsigned short*>(p)); }
    __device__ float get(int) const { return __uint_as_float(raw << 16); }
    __device__ static void store(__nv_bfloat16* p, float a, float) { *p = __float2bfloat16_rn(a); }
};
template <>
struct Cols<float, 1> {
    float raw = 0.f;
    __device__ void load(const float* p) { raw = __ldg(p); }
    __device__ float get(int) const { return raw; }
    __device__ static void store(float* p, float a, float) { *p = a; }
};

template <typename T, int CPT, bool DEQ>
__global__ void __launch_bounds__(512 / CPT) mx4_cols(const T* __restrict__ x, int64_t rows, int cols,
                                                      int col_tiles, int64_t blocks_k, int64_t tiles_k,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, T* __restrict__ y) {
    __shared__ __align__(16) uint8_t s_codes[kTile * kStagePitch];
    __shared__ uint8_t s_scale[4 * kTile];   // [column][block]
    constexpr int kLanes = kTile / CPT;      // threads across the columns
    const int64_t rt = blockIdx.x / (unsigned)col_tiles;   // row tile = k tile of the operand
    const int ct = (int)(blockIdx.x - rt * col_tiles);
    const int cl = (threadIdx.x % kLanes) * CPT, blk = threadIdx.x / kLanes;
    const int c = ct * kTile + cl;
    const int64_t r0 = rt * kTile + blk * 32;
    const int n = (int)(rows - r0 < 32 ? rows - r0 : 32);   // may be negative
    Cols<T, CPT> v[32];
    if (c < cols) {
        const T* p = x + r0 * cols + c;
#pragma unroll
        for (int t = 0; t < 32; ++t)
            if (t < n) v[t].load(p + (int64_t)t * cols);
    }
    uint32_t code[CPT][4];
    int b[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int t = 0; t < 32; ++t) m = max(m, __float_as_uint(v[t].get(i)) & 0x7FFFFFFFu);
        b[i] = scale_byte(m);
        const float s = inv_scale(b[i]);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t o = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) o |= pack2(v[8 * w + 2 * u].get(i) * s, v[8 * w + 2 * u + 1].get(i) * s) << (8 * u);
            code[i][w] = b[i] == mx4::kNanScale ? 0u : o;
        }
        *reinterpret_cast<uint4*>(s_codes + (cl + i) * kStagePitch + blk * 16) =
            make_uint4(code[i][0], code[i][1], code[i][2], code[i][3]);
        s_scale[(cl + i) * 4 + blk] = (uint8_t)b[i];
    }
    if (DEQ && c < cols) {
        T* p = y + r0 * cols + c;
        const float k0 = scale_value(b[0]), k1 = scale_value(b[CPT - 1]);
#pragma unroll
        for (int t = 0; t < 32; t += 2) {
            const float2 a0 = unpack2((code[0][t >> 3] >> (4 * (t & 7))) & 0xFF);
            const float2 a1 = unpack2((code[CPT - 1][t >> 3] >> (4 * (t & 7))) & 0xFF);
            if (t < n) Cols<T, CPT>::store(p + (int64_t)t * cols, a0.x * k0, a1.x * k1);
            if (t + 1 < n) Cols<T, CPT>::store(p + (int64_t)(t + 1) * cols, a0.y * k0, a1.y * k1);
        }
    }
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

template <typename T, bool DEQ>
cudaError_t launch_rows(const T* x, int64_t rows, int cols, uint8_t* codes, uint8_t* scales, T* y, cudaStream_t st) {
    const int tiles_k = (int)mx4::scale_tiles_k(cols);
    const int64_t segs = mx4::scale_tiles_r(rows) * 128 * tiles_k;
    const int pitch = (int)(mx4::padded_cols(cols) / 2);
    const bool vec = cols % 8 == 0;
    const int64_t per = vec ? kSegsVec : kSegsAny;
    const int64_t grid = (segs + per - 1) / per;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    prof_begin(st);
    if (vec) mx4_rows_vec<T, DEQ><<<(unsigned)grid, kRowThreads, 0, st>>>(x, rows, cols, segs, tiles_k, codes, pitch, scales, y);
    else mx4_rows_any<T, DEQ><<<(unsigned)grid, kRowThreads, 0, st>>>(x, rows, cols, segs, tiles_k, codes, pitch, scales, y);
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

// A bf16 row of an even width is 4-byte aligned, so its columns can be taken
// in pairs; other widths take one column per thread.
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
    return cols % 2 == 0 ? launch_cols<__nv_bfloat16, 2, DEQ>(p, rows, cols, codes, scales, o, st)
                         : launch_cols<__nv_bfloat16, 1, DEQ>(p, rows, cols, codes, scales, o, st);
}

jfa_status quantize_entry(const void* x, int dtype, int64_t rows, int64_t cols, int along_rows, uint8_t* codes,
                          uint8_t* scales, void* dequant, jfa_stream_t stream) {
    if (dtype != JFA_F32 && dtype != JFA_BF16)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4: dtype must be JFA_F32 or JFA_BF16");
    if (rows < 0 || cols < 0 || rows > kMx4MaxDim || cols > kMx4MaxDim)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4: rows and cols in [0, 2^30]");
    if (rows == 0 || cols == 0) return JFA_OK;
    if (!x || !codes || !scales) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4: NULL tensor");
    if (((uintptr_t)x | (uintptr_t)codes | (uintptr_t)scales | (uintptr_t)dequant) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4: tensors must be 16-byte aligned");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = dequant ? dispatch<true>(x, dtype, rows, (int)cols, along_rows, codes, scales, dequant, st)
                                  : dispatch<false>(x, dtype, rows, (int)cols, along_rows, codes, scales, nullptr, st);
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "quantize_mxfp4: %s", cudaGetErrorString(e));
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
    return jfa::quantize_entry(x, dtype, rows, cols, along_rows, codes, scales, nullptr, stream);
}

jfa_status jfa_quantize_mxfp4_dequant(const void* x, jfa_dtype dtype, int64_t rows, int64_t cols, int along_rows,
                                      uint8_t* codes, uint8_t* scales, void* dequant, jfa_stream_t stream) {
    if (rows > 0 && cols > 0 && !dequant)
        return jfa::set_last_error(JFA_ERR_INVALID_ARGUMENT, "quantize_mxfp4_dequant: NULL dequant");
    return jfa::quantize_entry(x, dtype, rows, cols, along_rows, codes, scales, dequant, stream);
}

}  // extern "C"
