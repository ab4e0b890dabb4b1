// What the MXFP4 product kernels share: the parameter block and the
// tcgen05 kind::mxf4 building blocks.
#pragma once

#include "jfa_mx4.cuh"
#include "jfa_sm100.cuh"

namespace jfa {

struct Mx4Params {
    CUtensorMap ta, tb;     // codes: bytes [rows][Kp / 2], boxes of 128 bytes (256 columns)
    CUtensorMap tsa, tsb;   // scales: 32-bit words [row tiles][tiles_k * 128], boxes of 256 words
    int m, n;
    int k_stages;           // 256-column steps; 0: an empty sum
    int last_steps;         // 64-column MMA steps of the last one
    const float* bias;
    void* out;              // [m][n]
    int out_bf16, accumulate;
    WsHeader* hdr;
};

namespace mx4 {

constexpr uint32_t kSfTile = 512;     // bytes of a 128-row x 4-scale tile
constexpr uint32_t kDescHi = sm100::sw128_desc_hi(1024);

// Operand of 128-byte swizzled rows, K-major: a K step of 64 codes is 32 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, int k) {
    return sm100::sw128_desc(sm100::sw128_desc_lo(addr, 16) + (uint32_t)k * 2u, kDescHi);
}

// Unswizzled K-major descriptor of a scale tile (32 rows of 16 bytes, core
// matrices of 8 rows 128 bytes apart) for tcgen05.cp.
__device__ __forceinline__ uint64_t sf_desc(uint32_t addr) {
    return sm100::sw128_desc(((addr & 0x3FFFF) >> 4) | (1u << 16), (128u >> 4) | (1u << 14));
}

// Instruction descriptor, kind::mxf4: E2M1 A and B (format 1), both K-major,
// E8M0 scales; `id` (0 or 2) selects which two of the four scale bytes of a
// column serve this K step.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int id) {
    return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 7) << 27) | ((uint32_t)id << 29);
}

template <int CTAS>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa, uint32_t sfb,
                                    uint32_t accumulate) {
    if constexpr (CTAS == 1) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    }
}

// A scale tile from shared memory to TMEM columns taddr .. taddr + 3: column j
// of lane l holds the four scales of row 32 j + l, in all four lane quarters.
template <int CTAS>
__device__ __forceinline__ void cp_sf(uint32_t taddr, uint64_t desc) {
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();   // the barrier takes whole warps
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ int ld_cluster_i32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

}  // namespace mx4
}  // namespace jfa
