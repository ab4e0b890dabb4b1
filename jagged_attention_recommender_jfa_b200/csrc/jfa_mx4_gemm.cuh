// What the MXFP4 product kernels share: the parameter block and the
// tcgen05 kind::mxf4 building blocks.
#pragma once

#include "jfa_mx4.cuh"
#include "jfa_sm100.cuh"

namespace jfa {

struct Mx4Params {
    CUtensorMap ta, tb;     // codes: bytes [rows][Kp / 2], boxes of 128 bytes (256 columns)
    CUtensorMap tsa, tsb;   // scales: 32-bit words [row tiles][tiles_k * 128], boxes of 256 words
    CUtensorMap tout;       // result, boxes of 128 bytes x 32 rows (pair kernel, aligned rows)
    int m, n;
    int k_stages;           // 256-column steps; 0: an empty sum
    int last_steps;         // 64-column MMA steps of the last one
    const float* bias;
    void* out;              // [m][n]
    int out_bf16, accumulate;
    int test_skip_load;     // test hook: CTA 0 leaves out its first load, so that the bounded waits run out
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

// The issuing loops run on a whole warp, with warp-uniform values and control
// flow, and only the instruction itself is predicated to one lane (`one`): so
// descriptors and addresses stay in uniform registers.  Issued from inside an
// `if (lane == 0)` every operand of every instruction first had to be moved
// there, and the issue, not the tensor core, set the pace.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// Warp index as a warp-uniform value.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

// mbar_wait by a whole warp with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, WsHeader* hdr) {
    if (__all_sync(0xffffffffu, sm100::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, sm100::mbar_wait(bar, parity, abort_flag, hdr)) != 0;
}

template <int CTAS>
__device__ __forceinline__ void mma(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t sfa,
                                    uint32_t sfb, uint32_t accumulate) {
    if constexpr (CTAS == 1) {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "setp.ne.b32 q, %7, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(one)
            : "memory");
    }
}

// A scale tile from shared memory to TMEM columns taddr .. taddr + 3: column j
// of lane l holds the four scales of row 32 j + l, in all four lane quarters.
template <int CTAS>
__device__ __forceinline__ void cp_sf(uint32_t one, uint32_t taddr, uint64_t desc) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
            "l"(desc), "r"(one)
            : "memory");
}

// Arrives on `bar` once the tcgen05 operations issued so far have completed.
__device__ __forceinline__ void commit_one(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(sm100::smem_u32(bar)),
        "r"(one)
        : "memory");
}

__device__ __forceinline__ void expect_tx_one(uint32_t one, uint64_t* bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(sm100::smem_u32(bar)),
        "r"(bytes), "r"(one)
        : "memory");
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

// An arrival on the same barrier of CTA `rank` of the cluster.  What it hands
// over is TMEM, ordered by the tcgen05 fences around it; no generic memory
// access crosses, so the arrival needs no cluster-wide release.
__device__ __forceinline__ void mbar_arrive_rank(uint64_t* bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(map_rank(sm100::smem_u32(bar), rank)) : "memory");
}

// TMA load into this CTA's shared memory that signals a barrier of either CTA
// of the pair (`bar` is a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t one, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                                 int y) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(one)
        : "memory");
}

// Arrives on this barrier in both CTAs of the pair once the pair's tcgen05
// operations issued so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t one, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            sm100::smem_u32(bar)),
        "h"((uint16_t)3), "r"(one)
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm100::smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// TMA store (or fp32 sum into the tensor) of a staged box, by one lane.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// the staged boxes of all committed stores have been read / written out
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void tma_load_2d(uint32_t one, uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(one)
        : "memory");
}

// Four consecutive columns of the result.
__device__ __forceinline__ void store4_out(const Mx4Params& P, int64_t at, float4 v) {
    if (P.out_bf16) {
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(P.out) + at;
        if (P.accumulate) {
            const float4 p = load4(o);
            v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
        }
        store4(o, v);
    } else {
        float* o = reinterpret_cast<float*>(P.out) + at;
        if (P.accumulate) {
            const float4 p = load4(o);
            v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
        }
        store4(o, v);
    }
}
__device__ __forceinline__ void store1_out(const Mx4Params& P, int64_t at, float v) {
    if (P.out_bf16) {
        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(P.out) + at;
        *o = __float2bfloat16_rn(P.accumulate ? v + __bfloat162float(*o) : v);
    } else {
        float* o = reinterpret_cast<float*>(P.out) + at;
        *o = P.accumulate ? v + *o : v;
    }
}

// Thread `t` of `threads` stores its share of a tile at (m0, n0) whose partial
// sums lie in the shared memory of the cluster's `split` CTAs, added in rank
// order.  Rows of a multiple of four
// columns go in pieces of four, others one by one; four pieces of a thread
// are under way at a time (a remote read takes some hundred cycles).
template <int BN, int PITCH, int VEC>
__device__ __forceinline__ void store_by(const Mx4Params& P, const float* part, int m0, int n0, int rows, int t,
                                         int threads, int split) {
    constexpr int kRow = BN / VEC, kAhead = 4;
    const int cols = min(BN, P.n - n0), total = rows * kRow;
    const uint32_t base = sm100::smem_u32(part);
    for (int u0 = t; u0 < total; u0 += kAhead * threads) {
        float4 v[kAhead];
        uint32_t at[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int u = min(u0 + i * threads, total - 1);
            at[i] = base + (uint32_t)((u / kRow) * PITCH + ((u % kRow) * VEC & ~3)) * 4;
            v[i] = ld_cluster4(map_rank(at[i], 0));
        }
        for (int q = 1; q < split; ++q) {
            float4 p[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) p[i] = ld_cluster4(map_rank(at[i], q));
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                v[i].x += p[i].x; v[i].y += p[i].y; v[i].z += p[i].z; v[i].w += p[i].w;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int u = u0 + i * threads;
            const int r = u / kRow, c = (u % kRow) * VEC;
            if (u >= total || c >= cols) continue;
            const int64_t o = (int64_t)(m0 + r) * P.n + n0 + c;
            if (VEC == 4) {
                if (P.bias) {
                    const float* b = P.bias + n0 + c;
                    v[i].x += __ldg(b); v[i].y += __ldg(b + 1); v[i].z += __ldg(b + 2); v[i].w += __ldg(b + 3);
                }
                store4_out(P, o, v[i]);
            } else {
                const int j = c & 3;
                float e = j == 0 ? v[i].x : (j == 1 ? v[i].y : (j == 2 ? v[i].z : v[i].w));
                if (P.bias) e += __ldg(P.bias + n0 + c);
                store1_out(P, o, e);
            }
        }
    }
}
template <int BN, int PITCH>
__device__ __forceinline__ void store_partials(const Mx4Params& P, const float* part, int m0, int n0, int rows, int t,
                                               int threads, int split) {
    if (rows <= 0) return;
    if ((P.n & 3) == 0) store_by<BN, PITCH, 4>(P, part, m0, n0, rows, t, threads, split);
    else store_by<BN, PITCH, 1>(P, part, m0, n0, rows, t, threads, split);
}

}  // namespace mx4
}  // namespace jfa
