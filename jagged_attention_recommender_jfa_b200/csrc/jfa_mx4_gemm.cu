// MXFP4 product on the 5th-generation tensor cores:
//   out[i][j] = sum_k A[i][k] B[j][k] (+ bias[j]) (+ out[i][j])
// A [m][k] and B [n][k] are MXFP4 operands (E2M1 codes, one E8M0 scale per 32
// along k), the products and sums are tcgen05.mma.kind::mxf4.block_scale with
// fp32 accumulation in TMEM; the result is rounded once, to bf16 or fp32.
//
// This kernel: one CTA per 128 x BN tile and share of k.  Warp 4 brings the
// codes (TMA, 128-byte swizzle) and the scale tiles of 256 columns a step into
// a ring of shared-memory stages, warp 5 copies the scales to TMEM and issues
// the MMAs (K = 64 each, four a step), warps 0..3 read the accumulator out.
// With few tiles the k range is split over a cluster of S CTAs; the partial
// tiles are summed through distributed shared memory in rank order, so the
// result does not depend on timing and no workspace or second launch is
// needed.  Rows and columns behind the tensors' ends are read as zero and not
// stored.
//
// Each stage of the ring has its own TMEM columns for its scale factors.
#include "jfa_mx4_gemm.cuh"

namespace jfa {

cudaError_t mx4_product_pair(Mx4Params& P, int64_t m, int64_t n, int64_t k, const uint8_t* ac, const uint8_t* as,
                             const uint8_t* bc, const uint8_t* bs, int bn, int sms, cudaStream_t st);

namespace {

using namespace sm100;

constexpr int kBM = 128;
constexpr int kThreads = 192;
constexpr int kTmaWarp = 4, kMmaWarp = 5;

template <int BN>
struct Shape {
    static constexpr uint32_t kA = kBM * 128;             // bytes of codes per stage
    static constexpr uint32_t kB = BN * 128;
    static constexpr uint32_t kSf = 2 * mx4::kSfTile;     // scales of 128 rows, 256 columns
    static constexpr uint32_t kStage = kA + kB + 2 * kSf;
    static constexpr int kStages = BN == 64 ? 7 : 6;
    static constexpr uint32_t kPitch = BN + 4;            // floats per staged output row
    static constexpr uint32_t kSmem = kStages * kStage + 1024;
    static constexpr uint32_t kTmem = 256;                // BN accumulator columns, 16 of scales per stage
    static_assert(kBM * kPitch * 4 <= kStages * kStage, "output staging reuses the ring");
    static_assert(kSmem <= 232448, "shared memory");
    static_assert(BN + 16 * kStages <= (int)kTmem, "TMEM columns");
};

struct Bars {
    uint64_t full[8], empty[8], acc;
    uint32_t tmem;
    int abort;
};

template <int BN>
__global__ void __launch_bounds__(kThreads) mx4_gemm(const __grid_constant__ Mx4Params P, int n_tiles, int split,
                                                     uint32_t stage_bytes) {
    using S = Shape<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars bars;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;   // swizzle atoms are 1024-byte aligned
    uint8_t* const smem = smem_raw + (base - smem_u32(smem_raw));
    const int warp = mx4::uniform_warp(), lane = threadIdx.x & 31;
    const int tile = blockIdx.x / split, rank = blockIdx.x - tile * split;
    const int m0 = (tile / n_tiles) * kBM, n0 = (tile % n_tiles) * BN;
    const int per = (P.k_stages + split - 1) / split;
    const int k0 = rank * per;
    const int nk = max(0, min(P.k_stages, k0 + per) - k0);
    volatile int* const abort_flag = &bars.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.acc, 1);
        bars.abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&bars.tmem, S::kTmem);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == kTmaWarp) {
        const uint32_t one = mx4::elect_one();
        int issued = 0;
        for (; issued < nk; ++issued) {
            const int s = issued % S::kStages, ph = (issued / S::kStages) & 1;
            if (issued >= S::kStages && !mx4::warp_wait(&bars.empty[s], ph ^ 1, abort_flag, P.hdr)) break;
            const uint32_t st = base + s * S::kStage, bar = smem_u32(&bars.full[s]);
            const int kk = k0 + issued;
            mx4::expect_tx_one(one, &bars.full[s], stage_bytes);
            const uint32_t skip = P.test_skip_load && blockIdx.x == 0 && issued == 0;
            mx4::tma_load_2d(skip ? 0u : one, st, &P.ta, bar, kk * 128, m0);
            mx4::tma_load_2d(one, st + S::kA, &P.tb, bar, kk * 128, n0);
            mx4::tma_load_2d(one, st + S::kA + S::kB, &P.tsa, bar, kk * 256, m0 >> 7);
            mx4::tma_load_2d(one, st + S::kA + S::kB + S::kSf, &P.tsb, bar, kk * 256, n0 >> 7);
        }
        // copies in flight end before the CTA leaves, whatever happened
        for (int i = max(0, issued - S::kStages); i < issued; ++i)
            mbar_wait_drain(&bars.full[i % S::kStages], (i / S::kStages) & 1, P.hdr);
    } else if (warp == kMmaWarp) {
        const uint32_t one = mx4::elect_one();
        // the second 64 rows of a scale tile are its columns 2 and 3
        const uint32_t sfb_half = BN == 64 ? (uint32_t)((n0 >> 6) & 1) * 2u : 0u;
        int done = 0;
        uint32_t ph = 0;
        bool ok = true;
        // unrolled over the ring: every address is a constant away from a base
        while (ok && done < nk) {
#pragma unroll
            for (int s = 0; s < S::kStages; ++s) {
                if (!ok || done == nk) break;
                // a full stage also says that the MMAs of its last use, and so the
                // last readers of its scale slot, have completed
                if (!mx4::warp_wait(&bars.full[s], ph, abort_flag, P.hdr)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = base + s * S::kStage;
                const uint32_t sfa = tmem + BN + s * 16, sfb = sfa + 8;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx4::cp_sf<1>(one, sfa + 4 * h, mx4::sf_desc(st + S::kA + S::kB + h * mx4::kSfTile));
                    mx4::cp_sf<1>(one, sfb + 4 * h, mx4::sf_desc(st + S::kA + S::kB + S::kSf + h * mx4::kSfTile));
                }
                const int steps = k0 + done == P.k_stages - 1 ? P.last_steps : 4;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k >= steps) break;
                    const uint32_t id = (k & 1) * 2;
                    const uint32_t col = (uint32_t)(k >> 1) * 4;
                    mx4::mma<1>(one, tmem, mx4::operand_desc(st, k), mx4::operand_desc(st + S::kA, k),
                                mx4::idesc(kBM, BN, (k & 1) * 2), (sfa + col) | (id << 30),
                                (sfb + sfb_half + col) | (id << 30), (done | k) != 0);
                }
                mx4::commit_one(one, &bars.empty[s]);
                ++done;
            }
            ph ^= 1;
        }
        mx4::commit_one(one, &bars.acc);
        mbar_wait_drain(&bars.acc, 0, P.hdr);
        tc_fence_before();
    }
    __syncwarp();
    // every MMA and copy of this CTA has ended (or its bounded wait has):
    // the ring is free for the partial tile
    __syncthreads();
    const bool bad = *abort_flag != 0;
    float* const part = reinterpret_cast<float*>(smem);
    if (warp < 4) {
        tc_fence_after();
        float* row = part + (warp * 32 + lane) * S::kPitch;
#pragma unroll
        for (int c = 0; c < BN; c += 32) {
            uint32_t r[32];
            if (nk > 0) {
                tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + c, r);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int t = 0; t < 32; ++t) r[t] = 0;
            }
#pragma unroll
            for (int t = 0; t < 32; t += 4)
                *reinterpret_cast<uint4*>(row + c + t) = make_uint4(r[t], r[t + 1], r[t + 2], r[t + 3]);
        }
        tc_fence_before();
    }
    const int rows = min(kBM, P.m - m0);
    bool skip = bad;
    if (split > 1) {
        mx4::cluster_sync();
        for (int r = 0; r < split; ++r) skip |= mx4::ld_cluster_i32(mx4::map_rank(smem_u32(&bars.abort), r)) != 0;
    } else {
        __syncthreads();
    }
    // every rank stores its share of the tile
    if (!skip)
        mx4::store_partials<BN, S::kPitch>(P, part, m0, n0, rows, rank * kThreads + threadIdx.x, split * kThreads, split);
    // no CTA leaves while another reads its partial tile
    if (split > 1) mx4::cluster_sync();
    else __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmem);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t inner, uint64_t rows,
               uint64_t pitch_bytes, uint32_t box_x, uint32_t box_y, CUtensorMapSwizzle swizzle) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {pitch_bytes};
    const cuuint32_t box[2] = {box_x, box_y}, step[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Tensor maps of one operand: codes in boxes of `box_rows` rows x 256 columns,
// scales in boxes of `sf_tiles` row tiles x 256 columns.
bool mx4_operand_maps(CUtensorMap* codes_map, CUtensorMap* scales_map, const uint8_t* codes, const uint8_t* scales,
                      int64_t rows, int64_t cols, int box_rows, int sf_tiles) {
    const uint64_t pitch = (uint64_t)mx4::padded_cols(cols) / 2;
    const uint64_t words = (uint64_t)mx4::scale_tiles_k(cols) * 128;
    return encode_2d(codes_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, pitch, (uint64_t)rows, pitch, 128,
                     (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
           encode_2d(scales_map, CU_TENSOR_MAP_DATA_TYPE_INT32, scales, words, (uint64_t)mx4::scale_tiles_r(rows),
                     words * 4, 256, (uint32_t)sf_tiles, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The result in boxes of 128 bytes x 32 rows.
bool mx4_out_map(CUtensorMap* map, void* out, int64_t m, int64_t n, int bf16) {
    const uint64_t elem = bf16 ? 2 : 4;
    return encode_2d(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, out, (uint64_t)n,
                     (uint64_t)m, (uint64_t)n * elem, (uint32_t)(128 / elem), 32, CU_TENSOR_MAP_SWIZZLE_128B);
}

namespace {

template <int BN>
cudaError_t launch(Mx4Params& P, int64_t m, int64_t n, int64_t k, const uint8_t* ac, const uint8_t* as,
                   const uint8_t* bc, const uint8_t* bs, int split, cudaStream_t st) {
    using S = Shape<BN>;
    // fewer rows than a tile: only those (in eights) are brought in; the other
    // rows of the stage hold anything, and so do their unused sums
    const int box = m < kBM ? (int)(m + 7) / 8 * 8 : kBM;
    const uint32_t stage_bytes = S::kStage - (uint32_t)(kBM - box) * 128;
    if (k > 0 && (!mx4_operand_maps(&P.ta, &P.tsa, ac, as, m, k, box, 1) ||
                  !mx4_operand_maps(&P.tb, &P.tsb, bc, bs, n, k, BN, 1)))
        return cudaErrorInvalidValue;
    const int64_t n_tiles = (n + BN - 1) / BN, tiles = (m + kBM - 1) / kBM * n_tiles;
    if (tiles * split > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(mx4_gemm<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    prof_begin(st);
    e = cudaLaunchKernelEx(&cfg, mx4_gemm<BN>, P, (int)n_tiles, split, stage_bytes);
    prof_end(st, K_MX4_GEMM);
    return e;
}

}  // namespace

namespace {

struct Plan {
    bool pair;
    int bn, split;
};

// The kernel, tile width and split of the contraction with the least
// estimated time: rounds of the tiles over the device x (steps of 256 columns
// x time of one + time of a tile's end), with times measured on a B200:
//   pair, 256 x 256     0.27 us a step, 1.0 us between tiles
//   pair, 256 x 128     0.21, 0.7
//   one CTA, 128 x 128  0.20, 2.5   (its end is not overlapped with a next tile)
//   one CTA, 128 x 64   0.20, 1.5;  a split adds 0.6
// and 148, 74, 33 and 15 clusters of 1, 2, 4 and 8 CTAs resident at a time (16:
// 7, slower wherever it was tried).  Measured, in us (pair 256 / pair 128 /
// best one-CTA form):
//   8192 x 8192 x 8192    177 / 212 / 441     2048 x 1024 x 1024   6.6 / 5.9 / 7.7
//   222283 x 4096 x 1024  457 / 514 / 3200    4999 x 1032 x 2008  13.8 / 14.0 / 27
//   512 x 512 x 65536     76 / 52 / 19 (64 wide, split 4)
//   1024 x 1024 x 65536   77 / 55 / 35 (128 wide, split 2)
// Up to 128 rows the one-CTA form always wins (1 x 4096 x 1024: 5.5 / 5.4 /
// 4.2, 1 x 8192 x 8192: 18 / 17 / 7.9): it fetches only the rows there are.
Plan choose(int64_t m, int64_t n, int64_t steps, int sms) {
    Plan best{false, 64, 1};
    double least = 1e300;
    auto consider = [&](bool pair, int bn, int split, double step, double end) {
        const int bm = pair ? 256 : kBM;
        const int64_t tiles = ((m + bm - 1) / bm) * ((n + bn - 1) / bn);
        const int64_t slots = pair ? sms / 2 : (split <= 2 ? sms / split : (split == 4 ? sms * 33 / 148 : sms * 15 / 148));
        const int64_t rounds = (tiles + slots - 1) / slots;
        const double t = (double)rounds * ((double)((steps + split - 1) / split) * step + end);
        if (t < least) {
            least = t;
            best = Plan{pair, bn, split};
        }
    };
    if (m > kBM && steps > 0) {
        consider(true, 256, 1, 0.27, 1.0);
        consider(true, 128, 1, 0.21, 0.7);
    }
    for (int split = 1; split <= 8 && (split == 1 || split <= steps); split *= 2) {
        consider(false, 64, split, 0.20, split > 1 ? 2.1 : 1.5);
        consider(false, 128, split, 0.20, split > 1 ? 3.1 : 2.5);
    }
    return best;
}

}  // namespace

cudaError_t mx4_product(int64_t m, int64_t n, int64_t k, const uint8_t* ac, const uint8_t* as, const uint8_t* bc,
                        const uint8_t* bs, const float* bias, void* out, int out_bf16, int accumulate, WsHeader* hdr,
                        cudaStream_t st) {
    Mx4Params P{};
    P.m = (int)m;
    P.n = (int)n;
    const int64_t kp = mx4::padded_cols(k);
    P.k_stages = (int)((kp + 255) / 256);
    P.last_steps = P.k_stages ? (int)((kp - (int64_t)(P.k_stages - 1) * 256 + 63) / 64) : 0;
    P.bias = bias;
    P.out = out;
    P.out_bf16 = out_bf16;
    P.accumulate = accumulate;
    P.hdr = hdr;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const Plan plan = choose(m, n, P.k_stages, sms);
    P.test_skip_load = k > 0 ? take_test_hook(JFA_TEST_MATMUL_SKIP_LOAD) : 0;
    cudaError_t e = cudaSuccess;
    if (P.test_skip_load) {
        static const int32_t limit = kTestWaitLimitUs;
        e = cudaMemcpyAsync(&hdr->wait_limit_us, &limit, sizeof(limit), cudaMemcpyHostToDevice, st);
        if (e != cudaSuccess) return e;
    }
    if (plan.pair) e = mx4_product_pair(P, m, n, k, ac, as, bc, bs, plan.bn, sms, st);
    else if (plan.bn == 64) e = launch<64>(P, m, n, k, ac, as, bc, bs, plan.split, st);
    else e = launch<128>(P, m, n, k, ac, as, bc, bs, plan.split, st);
    if (P.test_skip_load && e == cudaSuccess) e = cudaMemsetAsync(&hdr->wait_limit_us, 0, sizeof(int32_t), st);
    return e;
}

}  // namespace jfa

extern "C" {

size_t jfa_mxfp4_workspace_bytes(void) { return sizeof(jfa::WsHeader); }

jfa_status jfa_matmul_mxfp4(int64_t m, int64_t n, int64_t k, const uint8_t* a_codes, const uint8_t* a_scales,
                            const uint8_t* b_codes, const uint8_t* b_scales, const float* bias, void* out,
                            jfa_dtype out_dtype, int accumulate, void* workspace, size_t ws_bytes,
                            jfa_stream_t stream) {
    using namespace jfa;
    if (out_dtype != JFA_F32 && out_dtype != JFA_BF16)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: out_dtype must be JFA_F32 or JFA_BF16");
    if (m < 0 || n < 0 || k < 0 || m > kMx4MaxDim || n > kMx4MaxDim || k > kMx4MaxDim)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: m, n and k in [0, 2^30]");
    if (!workspace) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: NULL workspace");
    if (ws_bytes < sizeof(WsHeader))
        return set_last_error(JFA_ERR_WORKSPACE, "matmul_mxfp4: workspace %zu < %zu bytes", ws_bytes, sizeof(WsHeader));
    if (m == 0 || n == 0) return JFA_OK;
    if (!out || (k > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)))
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: NULL tensor");
    if (((uintptr_t)a_codes | (uintptr_t)a_scales | (uintptr_t)b_codes | (uintptr_t)b_scales | (uintptr_t)out |
         (uintptr_t)workspace) & 15)
        return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: tensors and workspace must be 16-byte aligned");
    if ((uintptr_t)bias & 3) return set_last_error(JFA_ERR_INVALID_ARGUMENT, "matmul_mxfp4: bias must be 4-byte aligned");
    const cudaError_t e = mx4_product(m, n, k, a_codes, a_scales, b_codes, b_scales, bias, out, out_dtype == JFA_BF16,
                                      accumulate ? 1 : 0, reinterpret_cast<WsHeader*>(workspace),
                                      reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_last_error(JFA_ERR_CUDA, "matmul_mxfp4: %s", cudaGetErrorString(e));
    return JFA_OK;
}

}  // extern "C"
