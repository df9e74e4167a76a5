// project_batch.cu -- moe_project on the 5th-generation tensor cores where one side is short: up to 256 rows (a decode
// step), or up to 256 outputs.
//
// The long side's rows (w, or x) are what there is to read, and go by once: 128 of them on the M side of a tile, all rows of
// the short side on its N side.  There are fewer such tiles than SMs, so a cluster of blocks shares K, each with its
// own part, and joins the parts through distributed shared memory, each block a share of the outputs, in the order
// of the blocks.
//
// Bound: its start and end, then the long side's bytes.  Measured: 48 rows of 4096, 2048 outputs and a residual 7.4 us (16
// tiles in 8 parts; the weights alone would take 2.6), 8192 rows of 2048 and 32 outputs 9.6 (the rows 5.2).  The setup runs
// under the end of the kernel before.  More warps that read the sums (8 or 16 for 4) gained nothing: 7.6 and 7.7, 8.9 and 9.4.
#include <atomic>
#include <cmath>
#include <mutex>

#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 192;  // a warp for copies, one for the MMAs, four that read the sums
constexpr int kLong = 128;     // rows of the long side
constexpr int kLongBytes = kLong * 128;
constexpr int kMaxStages = 8, kMaxSplit = 8, kMostSmem = 221 * 1024;

struct Maps {
    CUtensorMap a, b;  // long side, short side
};
struct Shape {
    int nb, stages, stage_bytes, sums_at, cols;  // short side's rows, rounded up to 16; TMEM columns
};

// SWAP: the long side is w, so that the sums are [output][row]; else it is x.
template <bool SWAP, bool F16>
__global__ void __launch_bounds__(kThreads)
    project_batch_kernel(const __grid_constant__ ProjectArgs p, const __grid_constant__ Maps maps, const Shape sh, int split) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], sums_full;
    __shared__ uint32_t tmem_holder;
    __shared__ int abort_word;
    volatile int *abort_flag = &abort_word;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = split > 1 ? (int)ptx::cluster_ctarank() : 0, a0 = (int)blockIdx.x / split * kLong;
    const int blocks = (p.K + 63) / 64, k0 = blocks * rank / split, k1 = blocks * (rank + 1) / split;
    if (tid == 0) {
        for (int s = 0; s < sh.stages; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
        ptx::mbar_init(&sums_full, 1);
        abort_word = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) ptx::tmem_alloc(&tmem_holder, sh.cols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_holder;
    ptx::launch_dependents();
    ptx::wait_prior_grid();
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            ptx::tma_prefetch_desc(&maps.a);
            ptx::tma_prefetch_desc(&maps.b);
            int issued = 0;
            for (int k = k0; k < k1; ++k, ++issued) {
                const int s = issued % sh.stages;
                if (issued >= sh.stages && !(ok = ptx::mbar_sleep_wait(&empty[s], (issued / sh.stages - 1) & 1, abort_flag))) break;
                uint8_t *stage = smem + s * sh.stage_bytes;
                ptx::mbar_arrive_expect_tx(&full[s], (uint32_t)sh.stage_bytes);
                ptx::tma_load_2d(stage, &maps.a, k * 64, a0, &full[s]);
                ptx::tma_load_2d(stage + kLongBytes, &maps.b, k * 64, 0, &full[s]);
            }
            if (!ok) {  // copies under way land before the shared memory is used for anything else
                int zero = 0;
                for (int i = max(issued - sh.stages, 0); i < issued; ++i)
                    ptx::mbar_sleep_wait(&full[i % sh.stages], i / sh.stages & 1, &zero);
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = ptx::idesc_16_f32(F16, kLong, sh.nb, false, false);
        const uint64_t desc0 = ptx::sw128_desc(ptx::smem_u32(smem));
        for (int i = 0; i < k1 - k0; ++i) {
            const int s = i % sh.stages;
            ok = __all_sync(0xffffffffu, ptx::mbar_sleep_wait(&full[s], i / sh.stages & 1, abort_flag)) != 0;
            if (!ok) break;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                const uint64_t da = desc0 + (uint64_t)(s * sh.stage_bytes >> 4), db = da + (kLongBytes >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) ptx::mma_f16_ss(tmem, da + 2 * k, db + 2 * k, idesc, i > 0 || k > 0);
                ptx::mma_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (ptx::elect_one()) ptx::mma_commit(&sums_full);  // (also when a wait ran out: nothing may run on when TMEM is freed)
        __syncwarp();
    }
    // every warp: the products are done, and with them all reads of the stages
    __syncwarp();
    int zero = 0;
    if (!(__all_sync(0xffffffffu, ptx::mbar_sleep_wait(&sums_full, 0, &zero)))) ok = false;
    if (!ok) {
        *abort_flag = 1;
        atomicCAS(p.status, 0, (int)MOE_ERR_TIMEOUT);
    }
    __syncthreads();
    ptx::tc_fence_after();
    // The block's sums in shared memory, [row of x][128 outputs] or [row of x][outputs], padded for the banks.
    const int rows = SWAP ? p.T : p.N;  // of the short side
    float *sums = reinterpret_cast<float *>(smem);
    const int ld = SWAP ? kLong : sh.nb + 4;
    if (warp >= 2) {
        const int quarter = warp & 3, a = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < sh.nb; c += 16) {
            uint32_t r[16];
            ptx::tmem_ld_16(lanes + c, r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(r[j]));
            if (SWAP) {
#pragma unroll
                for (int j = 0; j < 16; ++j) sums[(c + j) * ld + a] = __uint_as_float(r[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<uint4 *>(sums + a * ld + c + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
            }
        }
        ptx::tc_fence_before();
    }
    if (split > 1) ptx::cluster_sync(); else __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, sh.cols);
    }
    // The block's share of the outputs: rows of x, 4 outputs a thread.
    const int all = SWAP ? rows : min(kLong, p.T - a0), r0 = all * rank / split, r1 = all * (rank + 1) / split;
    const int pieces = SWAP ? kLong / 4 : (rows + 3) / 4, n0 = SWAP ? a0 : 0;
    const uint32_t base = ptx::smem_u32(sums);
    for (int i = tid; i < (r1 - r0) * pieces; i += kThreads) {
        const int r = r0 + i / pieces, c = i % pieces * 4;
        if (n0 + c >= p.N) continue;
        float z[4] = {0.f, 0.f, 0.f, 0.f}, bias[4];
        load_bias<4, F16>(p, n0 + c, bias);
        if (split > 1) {
#pragma unroll 4
            for (int s = 0; s < split; ++s) {
                const float4 v = ptx::ld_cluster_f4(ptx::mapa_shared(base + (uint32_t)(r * ld + c) * 4, s));
                z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
            }
        } else {
            const float4 v = *reinterpret_cast<const float4 *>(sums + r * ld + c);
            z[0] = v.x, z[1] = v.y, z[2] = v.z, z[3] = v.w;
        }
        finish<4, F16>(p, SWAP ? r : a0 + r, n0 + c, z, bias);
    }
    if (split > 1) ptx::cluster_sync();  // nobody leaves while others read its sums
}

// Rows of the long and the short side; blocks whose shared memory goes twice on an SM where the short side leaves room.
struct Sides {
    int64_t a;
    int b, nb, room, per_sm;
    explicit Sides(const ProjectArgs &p) {
        a = p.T <= p.N ? p.N : p.T, b = p.T <= p.N ? p.T : p.N;
        nb = (b + 15) / 16 * 16;
        per_sm = nb <= 128 ? 2 : 1;
        room = per_sm == 2 ? 108 * 1024 : 220 * 1024;
    }
};

template <bool SWAP, bool F16>
cudaLaunchConfig_t config(cudaLaunchAttribute (&attr)[2], int64_t blocks, int split, int smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    overlap_prior(attr[0]);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cfg;
}

// Clusters of each size that the device holds at once with one block an SM: fewer than SMs / size, as a cluster stays within
// a group of SMs (76 clusters of 2, 36 of 4, 23 of 6, 15 of 8).
struct Held {
    std::atomic<bool> ready;
    int clusters[kMaxSplit + 1];
};
template <bool SWAP, bool F16>
cudaError_t held(const Held **out) {
    static Held all[64];
    static std::mutex lock;
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    Held &h = all[dev];
    if (!h.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> hold(lock);
        if (!h.ready.load(std::memory_order_relaxed)) {  // (another thread may have filled it, and others read it, meanwhile)
            auto *kernel = project_batch_kernel<SWAP, F16>;
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
            if (e != cudaSuccess) return e;
            h.clusters[1] = device_info().sm_count;
            for (int n = 2; n <= kMaxSplit; ++n) {
                cudaLaunchAttribute attr[2];
                const cudaLaunchConfig_t cfg = config<SWAP, F16>(attr, (int64_t)n * device_info().sm_count, n, kMostSmem, nullptr);
                if ((e = cudaOccupancyMaxActiveClusters(&h.clusters[n], kernel, &cfg)) != cudaSuccess) return e;
            }
            h.ready.store(true, std::memory_order_release);
        }
    }
    *out = &h;
    return cudaSuccess;
}

// How many blocks share a tile's K, and about how long the whole takes (us): rounds of as many clusters as the device holds,
// each of K / 64 steps (0.26 us of 16 columns, 0.39 of 256) or of its share of the bytes at 6.5 TB/s, if that is longer, and of
// a start and end of 2.8 and more for each column that is laid down and joined.  Measured, us, with 1, 2, 4 and 8 blocks a tile:
// 48 rows of 4096 and 2048 outputs 23, 14, 9, 7.3; 8192 of 2048 and 32 14.4, 10.3, 9.0, 14.3; 256 of 4096 and 2048 33.5,
// 23.3, 15.3, 23.9 (6: 14.8).
template <bool SWAP, bool F16>
cudaError_t plan(const ProjectArgs &p, int *split, double *us) {
    const Held *h = nullptr;
    const cudaError_t e = held<SWAP, F16>(&h);
    if (e != cudaSuccess) return e;
    const Sides d(p);
    const int blocks = (p.K + 63) / 64;
    const int64_t tiles = (d.a + kLong - 1) / kLong;
    const double step = 0.252 + 0.00054 * d.nb, move = 2e-6 * p.K * (d.a + d.b) / 6.5;
    *us = 1e30;
    for (int n = 1; n <= min(kMaxSplit, blocks); ++n) {
        const int64_t most = max(h->clusters[n] * d.per_sm, 1), rounds = (tiles + most - 1) / most;
        const double t = fmax(rounds * step * ((blocks + n - 1) / n), move) + rounds * (2.8 + d.nb * (0.023 + 0.022 / n));
        if (t < *us) *us = t, *split = n;
    }
    return cudaSuccess;
}

template <bool SWAP, bool F16>
cudaError_t launch(const ProjectArgs &a, cudaStream_t s) {
    int split = 1;
    double us = 0;
    cudaError_t e = plan<SWAP, F16>(a, &split, &us);
    if (e != cudaSuccess) return e;
    const Sides d(a);
    Shape sh;
    sh.nb = d.nb;
    sh.stage_bytes = kLongBytes + sh.nb * 128;
    sh.cols = sh.nb <= 32 ? 32 : sh.nb <= 64 ? 64 : sh.nb <= 128 ? 128 : 256;
    const int sums = kLong * (SWAP ? sh.nb : sh.nb + 4) * 4;
    sh.stages = min(d.room / sh.stage_bytes, kMaxStages);
    const int smem = 1024 + max(sh.stages * sh.stage_bytes, sums);
    Maps m;
    if (!encode_tmap_rows(&m.a, SWAP ? a.w : a.x, d.a, a.K, SWAP ? a.w_ld : a.x_ld, kLong) ||
        !encode_tmap_rows(&m.b, SWAP ? a.x : a.w, d.b, a.K, SWAP ? a.x_ld : a.w_ld, sh.nb))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config<SWAP, F16>(attr, (d.a + kLong - 1) / kLong * split, split, smem, s);
    LaunchScope scope(KC_PROJECT_BATCH, s);
    e = cudaLaunchKernelEx(&cfg, project_batch_kernel<SWAP, F16>, a, m, sh, split);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t project_batch_time(const ProjectArgs &a, int dtype, double *us) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    int split;
    if (a.T <= a.N) return f16 ? plan<true, true>(a, &split, us) : plan<true, false>(a, &split, us);
    return f16 ? plan<false, true>(a, &split, us) : plan<false, false>(a, &split, us);
}

cudaError_t launch_project_batch(const ProjectArgs &a, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    // the shorter side on the N side
    if (a.T <= a.N) return f16 ? launch<true, true>(a, s) : launch<true, false>(a, s);
    return f16 ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace moe
