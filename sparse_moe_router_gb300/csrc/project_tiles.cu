// project_tiles.cu -- moe_project for many rows and outputs on the 5th-generation tensor cores.
//
// A pair of blocks (two SMs, cta_group::2) computes 256 rows of x by BN outputs with one stream of MMAs: each block
// holds its own 128 rows of x and half of the outputs' rows of w, and its 128 rows of the sums in TMEM, twice, so
// that the epilogue of one tile runs under the products of the next.  Pairs walk the tiles in turn, rows first, so that
// what runs at once shares rows of w.
//
// Roles: warps 0-7 epilogue (two for each quarter of the lanes, half of the columns each), 8 copies, 9 the MMAs.  A lane of
// TMEM is a row: 32 columns at a time go through the warp's own buffer, in 32 bits, so that rows leave in 64-byte pieces
// and bias, activation and residual are taken there, before the only rounding.
#include <mutex>

#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;  // of x a block
constexpr int kEpiWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kThreads = 320;
constexpr int kXBytes = kRows * 128;
constexpr int kTurnLd = 36;  // floats of a row of 32 columns, padded for the banks
constexpr int kTurnBytes = kEpiWarps * 32 * kTurnLd * 4;

template <int BN>
struct Shape {
    static constexpr int kWBytes = BN / 2 * 128;
    static constexpr int kStageBytes = kXBytes + kWBytes;
    static constexpr int kStages = 186 * 1024 / kStageBytes < 8 ? 186 * 1024 / kStageBytes : 8;
    static constexpr int kSmem = 1024 + kStages * kStageBytes + kTurnBytes + (2 * kStages + 5) * 8 + 16;
    static constexpr uint32_t kCols = 2 * BN < 32 ? 32 : 2 * BN;
    static_assert(kSmem <= 227 * 1024, "shared memory over the per-block limit");
};

struct Maps {
    CUtensorMap x, w;
};

template <int BN, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    project_tiles_kernel(const __grid_constant__ ProjectArgs p, const __grid_constant__ Maps maps) {
    using C = Shape<BN>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    float *turn = reinterpret_cast<float *>(smem + kStages * C::kStageBytes);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * C::kStageBytes + kTurnBytes), *empty = full + kStages;
    uint64_t *sums_full = empty + kStages, *sums_empty = sums_full + 2, *drain = sums_empty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile int *fills = abort_flag + 1;  // stages filled and used, read when a wait ran out
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = (int)ptx::cluster_ctarank();
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sums_full[i], 1), ptx::mbar_init(&sums_empty[i], 2 * kEpiWarps);
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        fills[0] = fills[1] = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) ptx::tmem_alloc_pair(tmem_holder, C::kCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the other block's barriers are ready before anyone signals them
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int tiles_t = (p.T + 2 * kRows - 1) / (2 * kRows), tiles = tiles_t * ((p.N + BN - 1) / BN);
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1, blocks = (p.K + 63) / 64;
    bool ok = true;
    if (warp == kLoadWarp) {
        if (lane == 0) {
            ptx::tma_prefetch_desc(&maps.x);
            ptx::tma_prefetch_desc(&maps.w);
            const uint32_t full_even = ptx::mapa_shared(ptx::smem_u32(full), 0);  // both blocks' copies are counted there
            int it = 0, s = 0;
            uint32_t phase = 1;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                const int t0 = tile % tiles_t * (2 * kRows) + rank * kRows, n0 = tile / tiles_t * BN + rank * (BN / 2);
                for (int k = 0; k < blocks; ++k, ++it) {
                    if (!(ok = ptx::mbar_sleep_wait(&empty[s], phase, abort_flag))) break;
                    uint8_t *stage = smem + s * C::kStageBytes;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
                    ptx::tma_load_2d_pair(stage, &maps.x, k * 64, t0, full_even + s * 8);
                    ptx::tma_load_2d_pair(stage + kXBytes, &maps.w, k * 64, n0, full_even + s * 8);
                    if (++s == kStages) s = 0, phase ^= 1;
                }
            }
            fills[0] = it;
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = ptx::idesc_16_f32(F16, 2 * kRows, BN, false, false);
            const uint64_t desc0 = ptx::sw128_desc(ptx::smem_u32(smem));
            int it = 0, s = 0, n = 0;
            uint32_t phase = 0;
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++n) {
                const int buf = n & 1;
                if (!(ok = ptx::mbar_wait_cluster(&sums_empty[buf], ((n >> 1) & 1) ^ 1, 2000000000ull, abort_flag))) break;
                ptx::tc_fence_after();
                for (int k = 0; k < blocks; ++k, ++it) {
                    if (!(ok = ptx::mbar_wait_cluster(&full[s], phase, 2000000000ull, abort_flag))) break;
                    ptx::tc_fence_after();
                    const uint64_t da = desc0 + (uint64_t)(s * C::kStageBytes >> 4), db = da + (kXBytes >> 4);
                    ptx::mma_bf16_pair(tmem + buf * BN, da, db, idesc, k > 0);
#pragma unroll
                    for (int j = 1; j < 4; ++j) ptx::mma_bf16_pair(tmem + buf * BN, da + 2 * j, db + 2 * j, idesc, 1);
                    ptx::mma_commit_pair(&empty[s], 3);
                    if (++s == kStages) s = 0, phase ^= 1;
                }
                if (ok) ptx::mma_commit_pair(&sums_full[buf], 3);
            }
            fills[1] = it;
            ptx::mma_commit_pair(drain, 1);  // nothing of the pair may run on when TMEM is freed
            int zero = 0;
            if (!ptx::mbar_sleep_wait(drain, 0, &zero)) ok = false;
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, c0 = (warp >> 2) * (BN / 2);
        constexpr int kEach = BN / 2 < 32 ? 32 : BN / 2;  // columns of a warp
        float *mine = turn + warp * (32 * kTurnLd);
        const uint32_t empty_even = ptx::mapa_shared(ptx::smem_u32(sums_empty), 0);
        int n = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++n) {
            const int buf = n & 1;
            ok = __all_sync(0xffffffffu, ptx::mbar_sleep_wait(&sums_full[buf], (n >> 1) & 1, abort_flag)) != 0;
            if (!ok) break;
            ptx::tc_fence_after();
            const int t0 = tile % tiles_t * (2 * kRows) + rank * kRows + quarter * 32, n0 = tile / tiles_t * BN + c0;
            const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + c0;
#pragma unroll 1
            for (int c = 0; c < kEach; c += 32) {
                uint32_t r[32];
                __syncwarp();
                ptx::tmem_ld_32(lanes + c, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(r[j]));
                if (c + 32 >= kEach) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0) ptx::mbar_arrive(&sums_empty[buf]);
                        else ptx::mbar_arrive_remote(empty_even + buf * 8);
                    }
                }
                if (t0 >= p.T || n0 + c >= p.N) continue;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4 *>(mine + lane * kTurnLd + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                __syncwarp();
                const int col = n0 + c + (lane & 3) * 8;
                if (col >= p.N) continue;
                float bias[8];
                load_bias<8, F16>(p, col, bias);
#pragma unroll 1
                for (int i = lane >> 2; i < 32 && t0 + i < p.T; i += 8) {
                    const float4 u = *reinterpret_cast<const float4 *>(mine + i * kTurnLd + (lane & 3) * 8);
                    const float4 v = *reinterpret_cast<const float4 *>(mine + i * kTurnLd + (lane & 3) * 8 + 4);
                    float z[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
                    finish<8, F16>(p, t0 + i, col, z, bias);
                }
            }
        }
    }
    if (!ok) {
        atomicCAS(p.status, 0, (int)MOE_ERR_TIMEOUT);
        *abort_flag = 1;
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // Copies under way land before the pair's shared memory is given up: the even block's barriers count both blocks';
        // the odd one cannot wait on them and gives its own a fixed 100 us.
        if (tid == kLoadWarp * 32) {
            int zero = 0;
            if (rank == 0) {
                for (int i = fills[1]; i < fills[0]; ++i) ptx::mbar_sleep_wait(&full[i % kStages], i / kStages & 1, &zero);
            } else {
                const uint64_t begun = ptx::globaltimer();
                while (ptx::globaltimer() - begun < 100000ull) {}
            }
        }
        __syncthreads();
    }
    ptx::cluster_sync();  // neither block leaves, or frees TMEM, while the other may still signal it
    if (warp == kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem, C::kCols);
    }
}

// Pairs of blocks that the device holds at once.
template <int BN, bool F16>
cudaError_t resident_pairs(int *pairs) {
    static int most[64] = {0};
    static std::mutex mu;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (most[dev] == 0) {
        auto *kernel = project_tiles_kernel<BN, F16>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<BN>::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(device_info().sm_count & ~1);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Shape<BN>::kSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        most[dev] = n;
    }
    *pairs = most[dev];
    return cudaSuccess;
}

template <int BN, bool F16>
cudaError_t launch_shape(const ProjectArgs &a, cudaStream_t s) {
    int pairs = 0;
    cudaError_t e = resident_pairs<BN, F16>(&pairs);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)((a.T + 2 * kRows - 1) / (2 * kRows)) * ((a.N + BN - 1) / BN);
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
    if (tiles < pairs) pairs = (int)tiles;
    Maps m;
    if (!encode_tmap_rows(&m.x, a.x, a.T, a.K, a.x_ld, kRows) || !encode_tmap_rows(&m.w, a.w, a.N, a.K, a.w_ld, BN / 2))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<BN>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    LaunchScope scope(KC_PROJECT_TILES, s);
    e = cudaLaunchKernelEx(&cfg, project_tiles_kernel<BN, F16>, a, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool F16>
cudaError_t launch(const ProjectArgs &a, cudaStream_t s) {
    // The tile that ends soonest: rounds of all pairs times a tile's time, in columns; a narrow tile's products wait for
    // their operands (128 columns: about 1.15 of its share), and its start and end count as 24.
    const int pairs = device_info().sm_count / 2;
    const int64_t rows = (a.T + 2 * kRows - 1) / (2 * kRows);
    auto cost = [&](int bn, double slow) {
        const int64_t tiles = rows * ((a.N + bn - 1) / bn);
        return (double)((tiles + pairs - 1) / pairs) * (bn * slow + 24);
    };
    const double c256 = cost(256, 1.0), c128 = cost(128, 1.15), c64 = cost(64, 1.6);
    if (c256 <= c128 && c256 <= c64) return launch_shape<256, F16>(a, s);
    return c128 <= c64 ? launch_shape<128, F16>(a, s) : launch_shape<64, F16>(a, s);
}

}  // namespace

cudaError_t launch_project_tiles(const ProjectArgs &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
