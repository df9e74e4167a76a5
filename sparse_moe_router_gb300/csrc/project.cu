// project.cu -- moe_project row by row: y = resid + alpha act(x w^T + bias) for a few rows of x.
//
// With few rows the weights are all there is to move.  A warp takes 4 rows of w and up to 4 rows of x; its lanes
// walk K in 16-byte pieces (8 weights), so that every piece of x serves 4 weights and every weight all rows of x.  Where
// N gives too few warps, the warps of a block share K.
//
// Bound: HBM, the weights.  Measured, one row of 2048 and 12,288 outputs: 10.0 us (5.0 TB/s, 74% of the measured copy; the
// rest is its start and end); with 2 rows of w a warp 9.9, so no gain.  One row of 4096 and 2048 outputs 3.4, of 2048 and 256 1.7.
#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kWRows = 4;  // rows of w a warp

// X rows of x; S warps share K.
template <int X, int S, bool F16>
__global__ void __launch_bounds__(kThreads) project_rows_kernel(const __grid_constant__ ProjectArgs p) {
    __shared__ float part[kWarps][kWRows * X];
    ptx::launch_dependents();
    ptx::wait_prior_grid();
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int group = warp / S, share = warp % S;
    const int n0 = ((int)blockIdx.x * (kWarps / S) + group) * kWRows, t0 = (int)blockIdx.y * X;
    float acc[kWRows][X];
#pragma unroll
    for (int i = 0; i < kWRows; ++i)
#pragma unroll
        for (int j = 0; j < X; ++j) acc[i][j] = 0.f;
    const uint16_t *w[kWRows], *x[X];
#pragma unroll
    for (int i = 0; i < kWRows; ++i) w[i] = p.w + (int64_t)min(n0 + i, p.N - 1) * p.w_ld;
#pragma unroll
    for (int j = 0; j < X; ++j) x[j] = p.x + (int64_t)min(t0 + j, p.T - 1) * p.x_ld;
    if (n0 < p.N) {
#pragma unroll 2
        for (int k = (share * 32 + lane) * 8; k < p.K; k += S * 256) {
            uint4 wv[kWRows], xv[X];
#pragma unroll
            for (int i = 0; i < kWRows; ++i) wv[i] = load_codes16(reinterpret_cast<const uint8_t *>(w[i] + k));
#pragma unroll
            for (int j = 0; j < X; ++j) xv[j] = __ldg(reinterpret_cast<const uint4 *>(x[j] + k));
#pragma unroll
            for (int i = 0; i < kWRows; ++i) {
                float a[8];
                unpack8<F16>(wv[i], a);
#pragma unroll
                for (int j = 0; j < X; ++j) {
                    float b[8];
                    unpack8<F16>(xv[j], b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i][j] = fmaf(a[e], b[e], acc[i][j]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kWRows; ++i)
#pragma unroll
        for (int j = 0; j < X; ++j) {
            float v = acc[i][j];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) part[warp][i * X + j] = v;
        }
    __syncthreads();
    for (int e = (int)threadIdx.x; e < kWarps / S * kWRows * X; e += kThreads) {
        const int g = e / (kWRows * X), i = e / X % kWRows, j = e % X;
        const int n = ((int)blockIdx.x * (kWarps / S) + g) * kWRows + i, t = t0 + j;
        if (n >= p.N || t >= p.T) continue;
        float z = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) z += part[g * S + s][i * X + j];
        if (p.bias) z += load1<F16>(p.bias + n);
        float v[1] = {z};
        activate(v, p.act);
        z = p.scale * v[0];
        if (p.out_f32) {
            if (p.resid) z += static_cast<const float *>(p.resid)[t * p.resid_ld + n];
            static_cast<float *>(p.y)[t * p.y_ld + n] = z;
        } else {
            if (p.resid) z += load1<F16>(static_cast<const uint16_t *>(p.resid) + t * p.resid_ld + n);
            static_cast<uint16_t *>(p.y)[t * p.y_ld + n] = (uint16_t)pack2<F16>(z, 0.f);
        }
    }
}

template <int X, int S, bool F16>
cudaError_t launch_shape(const ProjectArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_PROJECT_ROWS, s);
    const int rows = kWarps / S * kWRows;
    cudaLaunchAttribute attr[1];
    overlap_prior(attr[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + rows - 1) / rows, (a.T + X - 1) / X);  // (2^20 outputs are more blocks than y has places)
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, project_rows_kernel<X, S, F16>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int X, bool F16>
cudaError_t launch(const ProjectArgs &a, cudaStream_t s) {
    const int64_t warps = (int64_t)(a.N + kWRows - 1) / kWRows * ((a.T + X - 1) / X);
    // Warps that share K, the fewer the more there are: us with 1, 2, 4 and 8, one row of 2048: 2048 outputs 3.5, 2.9, 2.7, 2.4;
    // 4096 6.3, 5.1, 3.4, 4.1; 8192 7.7, 6.6, 6.8, 7.7; 12,288 10.0, 11.8, 10.3, 10.9.  Long rows want several all the same:
    // of 4096, 12,288 outputs 17.9, 20.7, 17.2, 17.5; 24,576 34.6, 33.4, 31.5, 31.7.
    const int sms = device_info().sm_count;
    if (warps <= 4 * sms) return launch_shape<X, 8, F16>(a, s);
    if (warps <= 8 * sms || a.K >= 4096) return launch_shape<X, 4, F16>(a, s);
    return warps <= 16 * sms ? launch_shape<X, 2, F16>(a, s) : launch_shape<X, 1, F16>(a, s);
}

}  // namespace

cudaError_t launch_project_rows(const ProjectArgs &a, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (a.T == 1) return f16 ? launch<1, true>(a, s) : launch<1, false>(a, s);
    return f16 ? launch<4, true>(a, s) : launch<4, false>(a, s);
}

}  // namespace moe
