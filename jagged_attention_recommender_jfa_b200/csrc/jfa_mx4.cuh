// MXFP4 (OCP Microscaling v1.0: E2M1 elements, one E8M0 scale per 32) helpers
// shared by the quantisers and the product: shared exponents, the hardware E2M1
// conversions and the layout of the scales.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "jfa_sm100.cuh"

namespace jfa {

constexpr int64_t kMx4MaxDim = (int64_t)1 << 30;   // rows and columns of an operand

namespace mx4 {

constexpr int kNanScale = 255;   // E8M0 NaN: a block that holds an infinity or a NaN

inline int64_t padded_cols(int64_t cols) { return (cols + 31) / 32 * 32; }
__host__ __device__ inline int64_t scale_tiles_k(int64_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline int64_t scale_tiles_r(int64_t rows) { return (rows + 127) / 128; }

// Largest magnitude, a NaN if there is one: exponent field 255 then, as for an
// infinity.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// The shared exponent of a block from the bits of its largest magnitude:
// X = floor(log2(amax)) - 2 (2 = the largest E2M1 exponent) clamped to
// [-127, 127].  The biased fp32 exponent e of a normal amax is floor(log2) + 127,
// so X + 127 is e - 2, and 0 where that is negative or amax is zero or subnormal.
// e = 255: an infinity or NaN.  x is at most 252 for finite blocks, so 2^-X is a
// normal number (2^-125 .. 2^127) in fp32 and bf16; it is 2^-126 for the others.
struct Shared {
    int x;
    bool nan;
    __device__ __forceinline__ explicit Shared(uint32_t amax_bits) {
        const int e = (int)(amax_bits >> 23);
        x = max(e - 2, 0);
        nan = e == 255;
    }
    __device__ __forceinline__ int byte() const { return nan ? kNanScale : x; }
    __device__ __forceinline__ float inv() const { return __uint_as_float((uint32_t)(254 - x) << 23); }
    __device__ __forceinline__ uint32_t inv_bf16x2() const { return (uint32_t)(254 - x) * 0x00800080u; }
};
// The byte X + 127's 2^X; 2^-127 is a subnormal.
__device__ __forceinline__ float scale_value(int byte) {
    if (byte == kNanScale) return __uint_as_float(0x7FFFFFFFu);
    return byte > 0 ? __uint_as_float((uint32_t)byte << 23) : __uint_as_float(1u << 22);
}

// Eight scaled values as E2M1 codes, four bits each, value 0 lowest: round to
// nearest even, saturating at 6.
__device__ __forceinline__ uint32_t cvt8(const float (&f)[8]) {
    uint32_t o;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(o)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return o;
}
// Eight values times s as codes.
__device__ __forceinline__ uint32_t pack8(const float (&g)[8], float s) {
    float f[8];
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        const float2 v = sm100::mul2(make_float2(g[u], g[u + 1]), make_float2(s, s));
        f[u] = v.x;
        f[u + 1] = v.y;
    }
    return cvt8(f);
}
// A packed pair of bf16 widened and scaled by a packed pair of powers of two
// (exactly; -0 added keeps the sign of a zero).
__device__ __forceinline__ void scaled(uint32_t pair, uint32_t s, float& lo, float& hi) {
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "mov.b32 {c, d}, %3;\n\t"
        "fma.rn.f32.bf16 %0, a, c, %4;\n\t"
        "fma.rn.f32.bf16 %1, b, d, %4;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(pair), "r"(s), "f"(-0.0f));
}
// The eight values of codes, times s (exact).
__device__ __forceinline__ void unpack8(uint32_t codes, float s, float (&f)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        const float2 p = sm100::mul2(v, make_float2(s, s));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
// Of two codes (the lowest byte) the values as packed bf16, times packed scales:
// shifted by three bits, the fp16 pattern of an E2M1 value is that of the value
// times 2^-112 in bf16.  Both products are exact.
__device__ __forceinline__ uint32_t scale_bf16x2(int byte) {
    return byte == kNanScale ? 0x7FFF7FFFu : byte > 0 ? (uint32_t)byte * 0x00800080u : 0x00400040u;
}
__device__ __forceinline__ uint32_t value_bf16x2(uint32_t codes, uint32_t s) {
    uint32_t h, o;
    asm("{\n\t.reg .b8 a;\n\t"
        "cvt.u8.u32 a, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
        : "=r"(h)
        : "r"(codes));
    h = (h & 0x80008000u) | ((h >> 3) & 0x0FFF0FFFu);
    asm("{\n\t.reg .b32 t;\n\t"
        "mul.rn.bf16x2 t, %1, %2;\n\t"
        "mul.rn.bf16x2 %0, t, %3;\n\t}"
        : "=r"(o)
        : "r"(h), "r"(0x77807780u), "r"(s));
    return o;
}
}  // namespace mx4
}  // namespace jfa
