// project_tiles.cu -- moe_project for many rows and outputs on the 5th-generation tensor cores.
//
// A pair of blocks (two SMs, cta_group::2) computes 256 rows of x by bn outputs with one stream of MMAs: each block
// holds its own 128 rows of x and half of the outputs' rows of w, and its 128 rows of the sums in TMEM, twice, so
// that the epilogue of one tile runs under the products of the next.  Pairs walk the tiles in turn, rows first, so that
// what runs at once shares rows of w.
//
// Bound: the tensor cores (95% of the cycles busy) where tiles fill the rounds.  Measured: 8192 rows of 2048 and 12,288
// outputs 209 to 220 us (1870 to 1970 TFLOP/s; cuBLAS's burst rate here is 1887), 243 to 251 when the power cap holds the clock
// at 1.55 GHz (1640 to 1700; cuBLAS's sustained rate is 1694); 1031 rows of 1032, 4104 outputs, bias and GELU
// in fp16 20.3 us, where 5 row tiles and tiles of 144 outputs make 145 for 76 pairs (128 outputs: 27; two rounds of
// 17 steps take 8, the epilogue of the last round, start and end the rest).  The MMAs are issued by an elected lane
// of a warp that waits as a whole: a lane chosen by comparison takes 610 cycles a step of K whatever the tile, this
// 335, as operands stay in uniform registers (245 us for the first case).
//
// Roles: warps 0-7 epilogue (two for each quarter of the lanes, half of the columns each), 8 copies, 9 the MMAs.  A lane of
// TMEM is a row: 32 columns at a time go through the warp's own buffer, in 32 bits, so that rows leave in 64-byte pieces
// and bias, activation and residual are taken there, before the only rounding.
#include <atomic>
#include <cmath>

#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 128;  // of x a block
constexpr int kEpiWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kThreads = 320;
constexpr int kXBytes = kRows * 128;
constexpr int kTurnLd = 36;  // floats of a row of 32 columns, padded for the banks
constexpr int kTurnBytes = kEpiWarps * 32 * kTurnLd * 4;

constexpr int kMostStages = 8, kStageRoom = 186 * 1024;
constexpr int kBarBytes = (2 * kMostStages + 5) * 8 + 16;
constexpr int kSmem = 1024 + kStageRoom + kTurnBytes + kBarBytes;
static_assert(kSmem <= 227 * 1024, "shared memory over the per-block limit");
constexpr int kBuf = 256;  // TMEM columns of a tile's sums
struct Shape {
    int bn, stage_bytes, stages;  // outputs a tile (a multiple of 16, at most 256)
};

struct Maps {
    CUtensorMap x, w;
};

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    project_tiles_kernel(const __grid_constant__ ProjectArgs p, const __grid_constant__ Maps maps, const Shape sh) {
    const int stages = sh.stages, bn = sh.bn;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    float *turn = reinterpret_cast<float *>(smem + kStageRoom);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStageRoom + kTurnBytes), *empty = full + kMostStages;
    uint64_t *sums_full = empty + kMostStages, *sums_empty = sums_full + 2, *drain = sums_empty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile int *fills = abort_flag + 1;  // stages filled and used, read when a wait ran out
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = (int)ptx::cluster_ctarank();
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sums_full[i], 1), ptx::mbar_init(&sums_empty[i], 2 * kEpiWarps);
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        fills[0] = fills[1] = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) ptx::tmem_alloc_pair(tmem_holder, 2 * kBuf);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::cluster_sync();  // the other block's barriers are ready before anyone signals them
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    ptx::launch_dependents();
    ptx::wait_prior_grid();
    const int tiles_t = (p.T + 2 * kRows - 1) / (2 * kRows), tiles = tiles_t * ((p.N + bn - 1) / bn);
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
                const int t0 = tile % tiles_t * (2 * kRows) + rank * kRows, n0 = tile / tiles_t * bn + rank * (bn / 2);
                for (int k = 0; k < blocks; ++k, ++it) {
                    if (!(ok = ptx::mbar_sleep_wait(&empty[s], phase, abort_flag))) break;
                    uint8_t *stage = smem + s * sh.stage_bytes;
                    if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * sh.stage_bytes);
                    ptx::tma_load_2d_pair(stage, &maps.x, k * 64, t0, full_even + s * 8);
                    ptx::tma_load_2d_pair(stage + kXBytes, &maps.w, k * 64, n0, full_even + s * 8);
                    if (++s == stages) s = 0, phase ^= 1;
                }
            }
            fills[0] = it;
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0) {  // the whole warp waits, one lane of it issues (its operands then stay in uniform registers)
            const uint32_t idesc = ptx::idesc_16_f32(F16, 2 * kRows, bn, false, false);
            const uint64_t desc0 = ptx::sw128_desc(ptx::smem_u32(smem));
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return __all_sync(0xffffffffu, ptx::mbar_sleep_wait<true>(bar, parity, abort_flag)) != 0;
            };
            int it = 0, s = 0, n = 0;
            uint32_t phase = 0;
            for (int tile = pair; tile < tiles && ok; tile += pairs, ++n) {
                const int buf = n & 1;
                if (!(ok = wait(&sums_empty[buf], ((n >> 1) & 1) ^ 1))) break;
                ptx::tc_fence_after();
                for (int k = 0; k < blocks; ++k, ++it) {
                    if (!(ok = wait(&full[s], phase))) break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint64_t da = desc0 + (uint64_t)(s * sh.stage_bytes >> 4), db = da + (kXBytes >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) ptx::mma_bf16_pair(tmem + buf * kBuf, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
                        ptx::mma_commit_pair(&empty[s], 3);
                        if (k + 1 == blocks) ptx::mma_commit_pair(&sums_full[buf], 3);
                    }
                    __syncwarp();
                    if (++s == stages) s = 0, phase ^= 1;
                }
            }
            fills[1] = it;
            if (ptx::elect_one()) ptx::mma_commit_pair(drain, 1);  // nothing of the pair may run on when TMEM is freed
            int zero = 0;
            if (!__all_sync(0xffffffffu, ptx::mbar_sleep_wait(drain, 0, &zero))) ok = false;
        }
        __syncwarp();
    } else {
        // the two warps of a quarter take turns of 32 columns
        const int quarter = warp & 3, half = warp >> 2;
        float *mine = turn + warp * (32 * kTurnLd);
        const uint32_t empty_even = ptx::mapa_shared(ptx::smem_u32(sums_empty), 0);
        int n = 0;
        for (int tile = pair; tile < tiles; tile += pairs, ++n) {
            const int buf = n & 1;
            ok = __all_sync(0xffffffffu, ptx::mbar_sleep_wait(&sums_full[buf], (n >> 1) & 1, abort_flag)) != 0;
            if (!ok) break;
            ptx::tc_fence_after();
            const int t0 = tile % tiles_t * (2 * kRows) + rank * kRows + quarter * 32, n0 = tile / tiles_t * bn, n1 = min(n0 + bn, p.N);
            const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + buf * kBuf;
            auto done = [&]() {  // the sums are in registers
                ptx::tc_fence_before();
                __syncwarp();
                if (lane != 0) return;
                if (rank == 0) ptx::mbar_arrive(&sums_empty[buf]);
                else ptx::mbar_arrive_remote(empty_even + buf * 8);
            };
            if (half * 32 >= bn) done();
#pragma unroll 1
            for (int c = half * 32; c < bn; c += 64) {
                uint32_t r[32];
                __syncwarp();
                ptx::tmem_ld_32(lanes + c, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(r[j]));
                if (c + 64 >= bn) done();
                if (t0 >= p.T || n0 + c >= n1) continue;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4 *>(mine + lane * kTurnLd + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                __syncwarp();
                const int col = n0 + c + (lane & 3) * 8;
                if (col >= n1) continue;
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
                for (int i = fills[1]; i < fills[0]; ++i) ptx::mbar_sleep_wait(&full[i % stages], i / stages & 1, &zero);
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
        ptx::tmem_dealloc_pair(tmem, 2 * kBuf);
    }
}

cudaLaunchConfig_t config(cudaLaunchAttribute *attr, int blocks, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    overlap_prior(attr[1]);
    cfg.numAttrs = 2;
    return cfg;
}

// Pairs of blocks that the device holds at once.
template <bool F16>
cudaError_t resident_pairs(int *pairs) {
    static std::atomic<int> most[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int n = most[dev].load(std::memory_order_acquire);
    if (n == 0) {
        auto *kernel = project_tiles_kernel<F16>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(attr, device_info().sm_count & ~1, nullptr);
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        most[dev].store(n, std::memory_order_release);
    }
    *pairs = n;
    return cudaSuccess;
}

template <bool F16>
cudaError_t launch(const ProjectArgs &a, cudaStream_t s) {
    int pairs = 0;
    cudaError_t e = resident_pairs<F16>(&pairs);
    if (e != cudaSuccess) return e;
    // The tile that ends soonest, in cycles: rounds of all pairs, each of K / 64 steps and about 800 for its start and end.  A
    // step's MMAs take 2 cycles a column; its operands, (128 + bn / 2) rows of 128 bytes, come at about 66 bytes a cycle
    // from L2, which is more below 256 columns (and narrower tiles have to gain 3%); a step alone takes 340.
    const int64_t rows = (a.T + 2 * kRows - 1) / (2 * kRows), steps = (a.K + 63) / 64;
    int bn = 256;
    double least = 1e30;
    for (int n = 256; n >= 48; n -= 16) {
        const int64_t rounds = (rows * ((a.N + n - 1) / n) + pairs - 1) / pairs;
        const double cost = (double)rounds * (steps * fmax(2.0 * n, fmax(340, 248 + 0.97 * n)) + 800) * (n == 256 ? 1.0 : 1.03);
        if (cost < least) least = cost, bn = n;
    }
    Shape sh;
    sh.bn = bn;
    sh.stage_bytes = kXBytes + bn / 2 * 128;
    sh.stages = min(kStageRoom / sh.stage_bytes, kMostStages);
    const int64_t tiles = rows * ((a.N + bn - 1) / bn);
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
    if (tiles < pairs) pairs = (int)tiles;
    Maps m;
    if (!encode_tmap_rows(&m.x, a.x, a.T, a.K, a.x_ld, kRows) || !encode_tmap_rows(&m.w, a.w, a.N, a.K, a.w_ld, bn / 2))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(attr, 2 * pairs, s);
    LaunchScope scope(KC_PROJECT_TILES, s);
    e = cudaLaunchKernelEx(&cfg, project_tiles_kernel<F16>, a, m, sh);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// About how long it takes with a short side of at most 256: steps of K, or the bytes at 85% of 6.5 TB/s, and a start and end.
double project_tiles_time(const ProjectArgs &a) {
    const int64_t tiles = (int64_t)((a.T + 255) / 256) * ((a.N + 255) / 256), pairs = max(device_info().sm_count / 2, 1);
    const double steps = (double)((tiles + pairs - 1) / pairs) * ((a.K + 63) / 64);
    return fmax(0.21 * steps, 2e-6 * a.K * ((double)a.T + a.N) / 5.6) + 5;
}

cudaError_t launch_project_tiles(const ProjectArgs &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
