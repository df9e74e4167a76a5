// head_norm.cu -- moe_head_norm: the norm of each head of each row, with its weight and gate.
//
//   y = (x - m) w / sqrt(mean((x - m)^2) + eps) act(gate)
// A head's values meet in two sums at most, so a few lanes of one warp hold it in registers: x and the gate are read
// once, y written once.  The mean comes first and the squares are taken of what is left (the difference
// of the two sums would lose a head whose mean is large).
#include "mixer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// L lanes a head, C 16-byte chunks (8 values) a lane: chunk i of lane l is chunk l + i L.
template <int L, int C, bool F16>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const __grid_constant__ HeadNormArgs p) {
    const int lane = (int)threadIdx.x & (L - 1), chunks = p.dim >> 3;
    const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L, items = (int64_t)p.T * p.heads;
    const bool live = item < items;
    const int64_t row = live ? item / p.heads : 0;
    const int head = live ? (int)(item - row * p.heads) : 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 xv[C], gv[C], wv[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + i * L;
        const bool in = live && c < chunks;
        xv[i] = in ? *reinterpret_cast<const uint4 *>(p.x + row * p.x_ld + head * p.dim + c * 8) : zero;
        gv[i] = in && p.gate ? *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_ld + head * p.dim + c * 8) : zero;
        wv[i] = in && p.weight ? __ldg(reinterpret_cast<const uint4 *>(p.weight + (p.weight_each ? head * p.dim : 0) + c * 8)) : zero;
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
    const float inv = 1.0f / sqrtf(lanes_sum<L>(ss) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = lane + i * L;
        if (!live || c >= chunks) continue;
        float w[8], g[8];
        unpack8<F16>(wv[i], w);
        unpack8<F16>(gv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[i][j] *= inv * (p.weight ? w[j] + unit : 1.0f);
            if (p.gate_kind == MOE_HEAD_GATE_SIGMOID) x[i][j] *= sigmoid_fast(g[j]);
            else if (p.gate_kind == MOE_HEAD_GATE_SILU) x[i][j] *= silu_fast(g[j]);
        }
        *reinterpret_cast<uint4 *>(p.y + row * p.y_ld + head * p.dim + c * 8) = pack8<F16>(x[i]);
    }
}

template <int L, int C, bool F16>
cudaError_t launch_lanes(const HeadNormArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_HEAD_NORM, s);
    const int64_t threads = (int64_t)a.T * a.heads * L, blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    head_norm_kernel<L, C, F16><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
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
    return dtype == MOE_DTYPE_F16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
