// MXFP4 product for large results: a pair of CTAs (two SMs) per 256 x BN tile,
// tcgen05.mma.cta_group::2 with M = 256, persistent over the tiles.
//
// Each CTA of the pair holds its own 128 rows of A and half of B's rows (the
// tensor cores read both halves), so a 256-column step of the contraction
// brings 32 KB of codes into each SM for 4 MMAs of 128 cycles: half the
// operand traffic of two independent 128 x 256 tiles.  Per SM and 256 columns:
// A 16 KB, B BN / 2 rows, the scales of its 128 rows of A and of all BN rows
// of B (the scales live in each SM's TMEM whole).
//
// Warps: one for TMA (both CTAs load their own halves and signal the first
// CTA's barrier), one for the MMAs (the first CTA's issues for the pair), 8 that
// read the accumulator out (32 lanes x half of the columns each).  Two accumulators
// alternate, so the read-out of a tile runs under the MMAs of the next one.
// With BN = 256 they share 128 columns (384 in all): the warps that read those
// let the next tile's MMAs start as soon as they have them in registers.  The
// remaining columns hold the scale factors, one slot per stage of the ring.
#include "jfa_mx4_gemm.cuh"

namespace jfa {

bool mx4_operand_maps(CUtensorMap* codes_map, CUtensorMap* scales_map, const uint8_t* codes, const uint8_t* scales,
                      int64_t rows, int64_t cols, int box_rows, int sf_tiles);
bool mx4_out_map(CUtensorMap* map, void* out, int64_t m, int64_t n, int bf16);

namespace {

using namespace sm100;

constexpr uint32_t kStageBytes = 4096;   // staging per read-out warp: a box of 32 rows x 128 bytes, 1024-byte aligned

template <int BN>
struct Shape {
    static constexpr int kWarpCols = BN / 2;                       // columns a read-out warp takes
    static constexpr int kEpiWarps = 8;
    static constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
    static constexpr int kThreads = (kEpiWarps + 2) * 32;
    static constexpr int kBTiles = BN / 128;                       // 128-row scale tiles that hold BN rows of B
    static constexpr uint32_t kA = 128 * 128;
    static constexpr uint32_t kB = BN / 2 * 128;
    static constexpr uint32_t kSfA = 2 * mx4::kSfTile;             // 128 rows, 256 columns
    static constexpr uint32_t kSfB = kBTiles * 2 * mx4::kSfTile;
    static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = BN == 128 ? 7 : 5;
    static constexpr uint32_t kRing = kStages * kStage;
    static constexpr uint32_t kSmem = kRing + kEpiWarps * (kStageBytes + kWarpCols * 4) + 1024;
    static constexpr bool kShared = BN == 256;                     // the accumulators share columns
    static constexpr uint32_t kAccStride = 128;                   // TMEM columns from one accumulator to the other
    static constexpr uint32_t kSfCol = kAccStride + BN;            // a slot of scale columns per ring stage
    static constexpr uint32_t kSfSlot = 8 + 8 * kBTiles;
    static_assert(kSfCol + kStages * kSfSlot <= 512, "TMEM columns");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(kStage % 1024 == 0 && kB % 1024 == 0, "swizzle atoms");
};

struct Bars {
    uint64_t full[8];      // first CTA: both CTAs' copies of a stage have landed
    uint64_t empty[8];     // each CTA: the MMAs that read the stage have completed
    uint64_t acc_full[2];  // each CTA: the tile's MMAs have completed
    uint64_t acc_free[2];  // first CTA: every read-out warp of both CTAs has read the accumulator (BN = 256: its shared columns)
    uint64_t done;         // each CTA: every MMA of the pair has completed
    uint32_t tmem;
    int abort;
};

// How a read-out warp stores its 32 rows (lane = row) from registers.
enum { OUT_ANY = 0, OUT_BF16 = 1, OUT_F32 = 2, OUT_F32_ADD = 3 };

// Rows that start on 16 bytes: a 128-byte wide box (64 bf16 or 32 fp32
// columns) is staged with the 128-byte swizzle (a row's 16-byte pieces in
// different banks for consecutive lanes) and leaves as one TMA store, which
// also cuts off what lies behind the last row and column; fp32 sums into the
// result are TMA reductions (one addition per element).  `bias`: the box's
// columns' in shared memory, or NULL.  Stored straight from registers, each
// lane its row's piece (32 rows an instruction), the read-out of a 256 x 192
// tile took 4,900 cycles, more than twice its MMAs at k = 1024.
template <int OUT>
__device__ __forceinline__ void store_box(const Mx4Params& P, const uint32_t* r, int row0, int col0, int lane,
                                          uint32_t stage, const float* bias) {
    if (row0 >= P.m || col0 >= P.n) return;   // nothing of the box lies inside
    if (lane == 0) mx4::bulk_wait_read();
    __syncwarp();
    constexpr int kParts = OUT == OUT_BF16 ? 2 : 1;
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
        float v[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) v[t] = __uint_as_float(r[32 * h + t]);
        if (bias) {
#pragma unroll
            for (int t = 0; t < 32; t += 4) {
                const float4 b = *reinterpret_cast<const float4*>(bias + 32 * h + t);   // the same for all lanes
                v[t] += b.x; v[t + 1] += b.y; v[t + 2] += b.z; v[t + 3] += b.w;
            }
        }
#pragma unroll
        for (int q = 0; q < (OUT == OUT_BF16 ? 4 : 8); ++q) {
            uint4 w;
            if (OUT == OUT_BF16)
                w = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                               pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
            else
                w = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                               __float_as_uint(v[4 * q + 3]));
            const uint32_t at = stage + lane * 128 + ((uint32_t)((h * 4 + q) ^ (lane & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                         : "memory");
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (OUT == OUT_F32_ADD) mx4::tma_add_2d(&P.tout, stage, col0, row0);
        else mx4::tma_store_2d(&P.tout, stage, col0, row0);
        mx4::bulk_commit();
    }
}

// Any row start, and bf16 sums: 32 columns through the staging tile, lane =
// column, eight rows under way at a time.
template <typename T, bool ADD>
__device__ __forceinline__ void store_rows(const Mx4Params& P, const float* stage, int row0, int col0, int lane, int rows,
                                           int cols, float b) {
    constexpr int kAhead = 8;
    const bool in = lane < cols;
    T* o = reinterpret_cast<T*>(P.out) + (int64_t)row0 * P.n + col0 + (in ? lane : 0);
#pragma unroll 1
    for (int i0 = 0; i0 < rows; i0 += kAhead, o += (int64_t)kAhead * P.n) {
        float v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            v[i] = stage[(i0 + i) * 32 + (lane ^ (i0 + i))] + b;
            if (ADD && i0 + i < rows) v[i] += to_f(o[(int64_t)i * P.n]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (in && i0 + i < rows) o[(int64_t)i * P.n] = from_f<T>(v[i]);
    }
}

__device__ __forceinline__ void store_any(const Mx4Params& P, const uint32_t* r, int row0, int col0, int lane,
                                          float* stage) {
    const int rows = min(32, P.m - row0), cols = min(32, P.n - col0);
    if (cols <= 0 || rows <= 0) return;
    // column t of row i at t ^ i: distinct banks both ways
#pragma unroll
    for (int t = 0; t < 32; ++t) stage[lane * 32 + (t ^ lane)] = __uint_as_float(r[t]);
    __syncwarp();
    const float b = (P.bias && lane < cols) ? __ldg(P.bias + col0 + lane) : 0.f;
    if (P.out_bf16) {
        if (P.accumulate) store_rows<__nv_bfloat16, true>(P, stage, row0, col0, lane, rows, cols, b);
        else store_rows<__nv_bfloat16, false>(P, stage, row0, col0, lane, rows, cols, b);
    } else {
        if (P.accumulate) store_rows<float, true>(P, stage, row0, col0, lane, rows, cols, b);
        else store_rows<float, false>(P, stage, row0, col0, lane, rows, cols, b);
    }
    __syncwarp();
}

template <int BN, int OUT>
__global__ void __launch_bounds__(Shape<BN>::kThreads, 1) mx4_gemm_pair(const __grid_constant__ Mx4Params P, int n_tiles, int tiles) {
    using S = Shape<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - smem_u32(smem_raw));
    const int warp = mx4::uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = mx4::cluster_rank();
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
    volatile int* const abort_flag = &bars.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.acc_full[0], 1);
        mbar_init(&bars.acc_full[1], 1);
        mbar_init(&bars.acc_free[0], 2 * S::kEpiWarps);
        mbar_init(&bars.acc_free[1], 2 * S::kEpiWarps);
        mbar_init(&bars.done, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == S::kMmaWarp) {
        mx4::tmem_alloc_pair(&bars.tmem, 512);
        tc_fence_before();
    }
    __syncthreads();
    mx4::cluster_sync();   // both CTAs' barriers exist before any remote arrival
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == S::kTmaWarp) {
        const uint32_t one = mx4::elect_one();
        const uint32_t arm = rank == 0 ? one : 0u;
        const uint32_t full0 = mx4::map_rank(smem_u32(&bars.full[0]), 0);
        int it = 0, s = 0, ph = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += step) {
            const int m0 = (tile / n_tiles) * 256 + (int)rank * 128, n0 = (tile % n_tiles) * BN;
            for (int kk = 0; kk < P.k_stages; ++kk, ++it) {
                if (it >= S::kStages && !mx4::warp_wait(&bars.empty[s], ph ^ 1, abort_flag, P.hdr)) {
                    ok = false;
                    break;
                }
                const uint32_t st = base + s * S::kStage, bar = full0 + s * 8;
                mx4::expect_tx_one(arm, &bars.full[s], 2 * S::kStage);
                const uint32_t skip = P.test_skip_load && blockIdx.x == 0 && it == 0;
                mx4::tma_load_2d_pair(skip ? 0u : one, st, &P.ta, bar, kk * 128, m0);
                mx4::tma_load_2d_pair(one, st + S::kA, &P.tb, bar, kk * 128, n0 + (int)rank * (BN / 2));
                mx4::tma_load_2d_pair(one, st + S::kA + S::kB, &P.tsa, bar, kk * 256, m0 >> 7);
                mx4::tma_load_2d_pair(one, st + S::kA + S::kB + S::kSfA, &P.tsb, bar, kk * 256, n0 >> 7);
                if (++s == S::kStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        // copies and arrivals still under way end before the CTA leaves
        if (ok) {
            for (int i = max(0, it - S::kStages); i < it; ++i)
                mbar_wait_drain(&bars.empty[i % S::kStages], (i / S::kStages) & 1, P.hdr);
        } else if (rank == 0) {
            for (int i = max(0, it - S::kStages); i < it; ++i)
                mbar_wait_drain(&bars.full[i % S::kStages], (i / S::kStages) & 1, P.hdr);
        } else {
            // given up after a second of waiting: the copies issued before
            // that signal the other CTA, so they get a fixed time to land
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 1000000ull) {
            }
        }
        mbar_wait_drain(&bars.done, 0, P.hdr);
    } else if (warp == S::kMmaWarp) {
        if (rank == 0) {
            const uint32_t one = mx4::elect_one();
            const int my = first < tiles ? (tiles - first + step - 1) / step : 0;
            const int64_t total = (int64_t)my * P.k_stages;
            int kk = 0, turn = 0;
            uint32_t ph = 0, acc = tmem;
            int64_t it = 0;
            bool ok = true;
            // unrolled over the ring: every address is a constant away from a base
            while (ok && it < total) {
#pragma unroll
                for (int s = 0; s < S::kStages; ++s) {
                    if (!ok || it == total) break;
                    if (kk == 0) {
                        // the previous tile has left the shared columns (and so the
                        // tile before it all of its); BN = 128: the tile before it
                        // has left this accumulator
                        const int prev = turn - (S::kShared ? 1 : 2);
                        if (prev >= 0 && !mx4::warp_wait(&bars.acc_free[prev & 1], (prev >> 1) & 1, abort_flag, P.hdr)) {
                            ok = false;
                            break;
                        }
                        acc = tmem + (turn & 1) * S::kAccStride;
                    }
                    // a full stage also says that the MMAs of its last use, and so
                    // the last readers of its scale slot, have completed
                    if (!mx4::warp_wait(&bars.full[s], ph, abort_flag, P.hdr)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = base + s * S::kStage;
                    const uint32_t sfa = tmem + S::kSfCol + s * S::kSfSlot, sfb = sfa + 8;
                    const uint32_t sf_a = st + S::kA + S::kB, sf_b = sf_a + S::kSfA;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx4::cp_sf<2>(one, sfa + 4 * h, mx4::sf_desc(sf_a + h * mx4::kSfTile));
#pragma unroll
                        for (int q = 0; q < S::kBTiles; ++q)
                            mx4::cp_sf<2>(one, sfb + (h * S::kBTiles + q) * 4, mx4::sf_desc(sf_b + (q * 2 + h) * mx4::kSfTile));
                    }
                    const bool last = kk == P.k_stages - 1;
                    const int steps = last ? P.last_steps : 4;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (k >= steps) break;
                        const uint32_t id = (k & 1) * 2;
                        mx4::mma<2>(one, acc, mx4::operand_desc(st, k), mx4::operand_desc(st + S::kA, k),
                                    mx4::idesc(256, BN, (k & 1) * 2), (sfa + (k >> 1) * 4) | (id << 30),
                                    (sfb + (k >> 1) * (S::kBTiles * 4)) | (id << 30), (kk | k) != 0);
                    }
                    mx4::commit_pair(one, &bars.empty[s]);
                    if (last) mx4::commit_pair(one, &bars.acc_full[turn & 1]);
                    kk = last ? 0 : kk + 1;
                    turn += last ? 1 : 0;
                    ++it;
                }
                ph ^= 1;
            }
            mx4::commit_pair(one, &bars.done);
            mbar_wait_drain(&bars.done, 0, P.hdr);
        }
    } else {
        const int quarter = warp & 3, group = warp >> 2;   // TMEM lanes; columns
        uint8_t* const stage = smem + S::kRing + warp * kStageBytes;
        float* const bias = reinterpret_cast<float*>(smem + S::kRing + S::kEpiWarps * kStageBytes) + warp * S::kWarpCols;
        int turn = 0;
        for (int tile = first; tile < tiles; tile += step, ++turn) {
            const int row0 = (tile / n_tiles) * 256 + (int)rank * 128 + quarter * 32;
            const int col0 = (tile % n_tiles) * BN + group * S::kWarpCols;
            if (OUT != OUT_ANY && P.bias) {
                // while the tile is computed: this warp's columns of the bias
                __syncwarp();
#pragma unroll
                for (int t = lane; t < S::kWarpCols; t += 32) bias[t] = col0 + t < P.n ? __ldg(P.bias + col0 + t) : 0.f;
                __syncwarp();
            }
            // lane 0 waits for the warp
            int up = 0;
            if (lane == 0) up = mbar_wait(&bars.acc_full[turn & 1], (turn >> 1) & 1, abort_flag, P.hdr) ? 1 : 0;
            if (!__shfl_sync(0xffffffffu, up, 0)) break;
            tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + (turn & 1) * S::kAccStride + group * S::kWarpCols;
            // all of this warp's columns to registers, then the accumulator is
            // free.  BN = 256: the columns shared with the next tile's are the
            // upper half of an even tile and the lower half of an odd one; the
            // other half's warps, done with the tile before, hold nothing the next
            // tile's MMAs could overwrite
            constexpr int kChunks = S::kWarpCols / 32;
            const bool early = S::kShared && group == (turn & 1);
            uint32_t r[kChunks][32];
            if (early) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mx4::mbar_arrive_rank(&bars.acc_free[turn & 1], 0);
            }
#pragma unroll
            for (int i = 0; i < kChunks; ++i) tmem_ld32(src + i * 32, r[i]);
            tmem_wait_ld();
            if (!early) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mx4::mbar_arrive_rank(&bars.acc_free[turn & 1], 0);
            }
#pragma unroll
            for (int i = 0; i < kChunks; i += OUT == OUT_BF16 ? 2 : 1) {
                if (OUT == OUT_ANY) store_any(P, r[i], row0, col0 + i * 32, lane, reinterpret_cast<float*>(stage));
                else store_box<OUT>(P, r[i], row0, col0 + i * 32, lane, smem_u32(stage), P.bias ? bias + i * 32 : nullptr);
            }
        }
        if (OUT != OUT_ANY && lane == 0) mx4::bulk_wait();
    }
    // both CTAs' work, remote arrivals included, has ended
    __syncthreads();
    mx4::cluster_sync();
    if (warp == S::kMmaWarp) {
        tc_fence_after();
        mx4::tmem_dealloc_pair(tmem, 512);
    }
}

template <int BN>
cudaError_t launch(Mx4Params& P, int64_t m, int64_t n, int64_t k, const uint8_t* ac, const uint8_t* as,
                   const uint8_t* bc, const uint8_t* bs, int sms, cudaStream_t st) {
    using S = Shape<BN>;
    if (!mx4_operand_maps(&P.ta, &P.tsa, ac, as, m, k, 128, 1) ||
        !mx4_operand_maps(&P.tb, &P.tsb, bc, bs, n, k, BN / 2, S::kBTiles))
        return cudaErrorInvalidValue;
    const int64_t n_tiles = (n + BN - 1) / BN, tiles = (m + 255) / 256 * n_tiles;
    if (tiles > 0x3fffffff) return cudaErrorInvalidConfiguration;
    const int elem = P.out_bf16 ? 2 : 4;
    int kind = OUT_ANY;
    if ((n * elem) % 16 == 0 && !(P.out_bf16 && P.accumulate))
        kind = P.out_bf16 ? OUT_BF16 : (P.accumulate ? OUT_F32_ADD : OUT_F32);
    if (kind != OUT_ANY && !mx4_out_map(&P.tout, P.out, m, n, P.out_bf16)) return cudaErrorInvalidValue;
    void (*kern)(Mx4Params, int, int) = kind == OUT_BF16  ? mx4_gemm_pair<BN, OUT_BF16>
                                        : kind == OUT_F32 ? mx4_gemm_pair<BN, OUT_F32>
                                        : kind == OUT_ANY ? mx4_gemm_pair<BN, OUT_ANY>
                                                          : mx4_gemm_pair<BN, OUT_F32_ADD>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    const int64_t pairs = sms / 2;
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    prof_begin(st);
    e = cudaLaunchKernelEx(&cfg, kern, P, (int)n_tiles, (int)tiles);
    prof_end(st, K_MX4_GEMM_PAIR);
    return e;
}

}  // namespace

cudaError_t mx4_product_pair(Mx4Params& P, int64_t m, int64_t n, int64_t k, const uint8_t* ac, const uint8_t* as,
                             const uint8_t* bc, const uint8_t* bs, int bn, int sms, cudaStream_t st) {
    return bn == 256 ? launch<256>(P, m, n, k, ac, as, bc, bs, sms, st)
                     : launch<128>(P, m, n, k, ac, as, bc, bs, sms, st);
}

}  // namespace jfa
