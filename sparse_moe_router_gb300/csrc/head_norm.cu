// head_norm.cu -- moe_head_norm: the norm of each head of each row, with its weight and gate.
//
//   y = (x - m) w / sqrt(mean((x - m)^2) + eps) act(gate)
// A head's values meet in two sums at most, so a few lanes of one warp hold it in registers: x and the gate are read
// once, y written once.  The mean comes first and the squares are taken of what is left (the difference
// of the two sums would lose a head whose mean is large).
//
// Bound: instructions (issue slots 83% used; one head of 128 takes 16 lanes some 110 of them, with a gate 150), then HBM.
// Measured: 8192 x 32 heads of 128 with a SiLU gate 35.2 us (5.7 TB/s, 84% of the measured copy), without 27.6; one row of 32
// heads 1.4 (5.3 for a call from Python).  On the way: 64-bit places and an IEEE root and division 45.6; two, three and four heads a thread 38.0, 37.8 and
// 40.9 where one took 36.7 (registers); paired fp32 arithmetic 36.4 against 35.2.
#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// L lanes a head, C 16-byte chunks (8 values) a lane: chunk i of lane l is chunk l + i L.
template <int L, int C, bool F16>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const __grid_constant__ HeadNormArgs p) {
    ptx::launch_dependents();
    // (32 bits: a launch has fewer than 2^30 heads)
    const uint32_t item = blockIdx.x * (kThreads / L) + threadIdx.x / L;
    const bool live = item < (uint32_t)p.T * p.heads;
    const uint32_t row = live ? item / (uint32_t)p.heads : 0;
    const int lane = (int)threadIdx.x & (L - 1), chunks = p.dim >> 3, at = live ? (int)(item - row * p.heads) * p.dim : 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 xv[C], gv[C], wv[C];
    ptx::wait_prior_grid();
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + i * L;
        const bool in = live && c < chunks;
        xv[i] = in ? *reinterpret_cast<const uint4 *>(p.x + row * p.x_ld + at + c * 8) : zero;
        gv[i] = in && p.gate ? *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_ld + at + c * 8) : zero;
        wv[i] = in && p.weight ? __ldg(reinterpret_cast<const uint4 *>(p.weight + (p.weight_each ? at : 0) + c * 8)) : zero;
    }
    float x[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) unpack8<F16>(xv[i], x[i]);
    const float inv_d = 1.0f / (float)p.dim, unit = p.unit_offset ? 1.0f : 0.0f;
    if (p.center) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += x[i][j];
        const float mean = lanes_sum<L>(sum) * inv_d;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] = lane + i * L < chunks ? x[i][j] - mean : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
    const float inv = rsqrtf(lanes_sum<L>(ss) * inv_d + p.eps);  // (2 ulp; the root and the division were a fifth of the instructions)
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + i * L;
        if (!live || c >= chunks) continue;
        float w[8], g[8];
        unpack8<F16>(wv[i], w);
        unpack8<F16>(gv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] *= p.weight ? inv * (w[j] + unit) : inv;
        if (p.gate_kind == MOE_HEAD_GATE_SIGMOID) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= sigmoid_fast(g[j]);
        } else if (p.gate_kind == MOE_HEAD_GATE_SILU) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i][j] *= silu_fast(g[j]);
        }
        *reinterpret_cast<uint4 *>(p.y + row * p.y_ld + at + c * 8) = pack8<F16>(x[i]);
    }
}

template <int L, int C, bool F16>
cudaError_t launch_lanes(const HeadNormArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_HEAD_NORM, s);
    const int each = kThreads / L;
    cudaLaunchAttribute attr[1];
    overlap_prior(attr[0]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.T * a.heads + each - 1) / each));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, head_norm_kernel<L, C, F16>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool F16>
cudaError_t launch(const HeadNormArgs &a, cudaStream_t s) {
    const int chunks = a.dim / 8;
    if (chunks <= 8) return launch_lanes<8, 1, F16>(a, s);
    if (chunks <= 16) return launch_lanes<16, 1, F16>(a, s);
    if (chunks <= 32) return launch_lanes<32, 1, F16>(a, s);
    if (chunks <= 64) return launch_lanes<32, 2, F16>(a, s);
    return launch_lanes<32, 4, F16>(a, s);
}

}  // namespace

cudaError_t launch_head_norm(const HeadNormArgs &a, int dtype, cudaStream_t s) {
    const int most = (1 << 30) / a.heads;  // rows a launch
    for (int t = 0; t < a.T; t += most < a.T - t ? most : a.T - t) {
        HeadNormArgs b = a;
        b.x += t * a.x_ld;
        b.y += t * a.y_ld;
        if (b.gate) b.gate += t * a.gate_ld;
        b.T = most < a.T - t ? most : a.T - t;
        const cudaError_t e = dtype == MOE_DTYPE_F16 ? launch<true>(b, s) : launch<false>(b, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace moe
