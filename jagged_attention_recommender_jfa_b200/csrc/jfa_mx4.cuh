// MXFP4 (OCP Microscaling v1.0: E2M1 elements, one E8M0 scale per 32) helpers
// shared by the quantisers, the norms and the product: shared exponents, the
// hardware E2M1 conversions and the layout of the scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace jfa {

constexpr int64_t kMx4MaxDim = (int64_t)1 << 30;   // rows and columns of an operand

namespace mx4 {

constexpr int kNanScale = 255;   // E8M0 NaN: a block that holds an infinity or a NaN

inline int64_t padded_cols(int64_t cols) { return (cols + 31) / 32 * 32; }
__host__ __device__ inline int64_t scale_tiles_k(int64_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline int64_t scale_tiles_r(int64_t rows) { return (rows + 127) / 128; }

// Byte offset of the 4-byte word that holds the scales of row r, columns
// [128 kt, 128 kt + 128): tiles of 128 rows x 4 scales, 512 contiguous bytes
// each, in the order tcgen05.cp spreads over 32 lanes x 16 bytes.
__host__ __device__ inline int64_t scale_word(int64_t r, int64_t kt, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + kt) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Scale byte of a block from the bits of its largest magnitude:
// X = floor(log2(amax)) - 2 (2 = the largest E2M1 exponent) clamped to
// [-127, 127], byte X + 127.  The biased fp32 exponent e of a normal amax is
// floor(log2) + 127, so the byte is e - 2, and 0 (X = -127) where that is
// negative or amax is zero or subnormal.  e = 255: infinity or NaN.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);
    return e == 255 ? kNanScale : max(e - 2, 0);
}

// 2^-X and 2^X of a scale byte (X = byte - 127).  Bytes of finite blocks are
// at most 252, so 2^-X is a normal number (2^-125 .. 2^127); 2^-127 is an
// fp32 subnormal.
__device__ __forceinline__ float inv_scale(int byte) {
    return __uint_as_float((uint32_t)(254 - min(byte, 253)) << 23);
}
__device__ __forceinline__ float scale_value(int byte) {
    if (byte == kNanScale) return __uint_as_float(0x7FFFFFFFu);
    return byte > 0 ? __uint_as_float((uint32_t)byte << 23) : __uint_as_float(1u << 22);
}

// Two E2M1 codes in a byte, `lo` in the low four bits: round to nearest even,
// saturating at 6.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
__device__ __forceinline__ float2 unpack2(uint32_t byte) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)byte, __NV_E2M1);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace mx4
}  // namespace jfa
