// norm.cu -- moe_block_norm: the norm after a block, its gate and residual scale, the residual
// update, and the norm before the next block, in one pass over the row.
//
// Per row:  n = x w_post / sqrt(mean(x^2) + eps);  r' = resid + alpha g n;
//           y = r' w_pre / sqrt(mean(r'^2) + eps).
// The two means are the only places where a row's values meet, so a block keeps its row in
// registers between them: x, resid and the gate are read once, r' and y written once, and nothing
// else touches memory.  Both sums of squares are fp32.
#include "layer.h"

namespace moe {
namespace {

// Sum over the block, returned to every thread.  `buf` holds a float per warp and is not used
// for another sum of the same call.
__device__ __forceinline__ float block_sum(float v, float *buf, int warps) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = (int)(threadIdx.x & 31) < warps ? buf[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

// C 16-byte chunks (8 values) a thread; chunk i of thread t is chunk t + i * blockDim of the row.
template <int C, bool F16>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ float buf[2][32];
    const int warps = (int)blockDim.x >> 5, chunks = p.H >> 3;
    const int64_t row = blockIdx.x;
    const float inv_h = 1.0f / (float)p.H;
    float r[C][8];
    uint4 xv[C], rv[C], gv[C];
    bool in[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        in[i] = c < chunks;
        xv[i] = rv[i] = gv[i] = make_uint4(0, 0, 0, 0);
        if (!in[i]) continue;
        if (p.x) xv[i] = *reinterpret_cast<const uint4 *>(p.x + row * p.x_ld + c * 8);
        if (p.resid) rv[i] = *reinterpret_cast<const uint4 *>(p.resid + row * p.resid_ld + c * 8);
        if (p.gate_kind == MOE_GATE_ELEMENT) gv[i] = *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_ld + c * 8);
        if (p.gate_kind == MOE_GATE_CHANNEL) gv[i] = *reinterpret_cast<const uint4 *>(p.gate + c * 8);
    }
    const float unit = p.unit_offset ? 1.0f : 0.0f;
    float g_row = 1.0f;
    if (p.gate_kind == MOE_GATE_TOKEN) {
        g_row = load1<F16>(p.gate + row * p.gate_ld);
        if (p.sigmoid) g_row = 1.0f / (1.0f + __expf(-g_row));
    }
    float inv = 1.0f;
    if (p.x && p.w_post) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float x[8];
            unpack8<F16>(xv[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        }
        inv = 1.0f / sqrtf(block_sum(ss, buf[0], warps) * inv_h + p.eps);
    }
    inv *= p.alpha * g_row;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        float x[8], w[8], g[8];
        unpack8<F16>(rv[i], r[i]);
        if (p.x && in[i]) {
            unpack8<F16>(xv[i], x);
            if (p.w_post) unpack8<F16>(*reinterpret_cast<const uint4 *>(p.w_post + c * 8), w);
            if (p.gate_kind & MOE_GATE_CHANNEL) unpack8<F16>(gv[i], g);  // per channel or per element
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float n = x[j] * inv;
                if (p.w_post) n *= w[j] + unit;
                if (p.gate_kind & MOE_GATE_CHANNEL) n *= p.sigmoid ? 1.0f / (1.0f + __expf(-g[j])) : g[j];
                r[i][j] += n;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
        if (p.resid_out && in[i]) *reinterpret_cast<uint4 *>(p.resid_out + row * p.resid_out_ld + c * 8) = pack8<F16>(r[i]);
    }
    if (!p.y) return;
    const float inv2 = 1.0f / sqrtf(block_sum(ss, buf[1], warps) * inv_h + p.eps);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        if (!in[i]) continue;
        float w[8];
        unpack8<F16>(*reinterpret_cast<const uint4 *>(p.w_pre + c * 8), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= inv2 * (w[j] + unit);
        *reinterpret_cast<uint4 *>(p.y + row * p.y_ld + c * 8) = pack8<F16>(r[i]);
    }
}

template <bool F16>
cudaError_t launch(const NormArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_BLOCK_NORM, s);
    const int chunks = a.H / 8;
    if (chunks <= 1024) {
        block_norm_kernel<1, F16><<<a.T, (chunks + 31) / 32 * 32, 0, s>>>(a);
    } else {
        block_norm_kernel<2, F16><<<a.T, ((chunks + 1) / 2 + 31) / 32 * 32, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
