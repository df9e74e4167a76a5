// norm.cu -- moe_block_norm: the norm after a block, its gate and residual scale, the residual
// update, and the norm before the next block, in one pass over the row.
//
// Per row:  n = x w_post / sqrt(mean(x^2) + eps);  r' = resid + alpha g n;
//           y = r' w_pre / sqrt(mean(r'^2) + eps).
// The two means are the only places where a row's values meet, so a block keeps its row in
// registers between them: x, resid and the gate are read once, r' and y written once, and nothing
// else touches memory.  Both sums of squares are fp32.
//
// Bound: HBM from a few hundred rows on, below that the launch and two dependent sums.  Measured: one
// row of 2048 2.7 us; 1031 rows of 4096 with a channel gate 10.1 us (3.3 TB/s: 16 warps an SM, each with
// one row of its seven ahead); 8192 rows of 2048 with a gate on each element 32.6 us (5.1 TB/s,
// 77% of the measured copy; before a block kept its weights and had its next row under way, 45).
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

// 1 / (1 + e^-x) to about 2 ulp (the fast exponential and reciprocal): 2 of 4 instructions on the
// special-function pipe, against 12 with an IEEE division; x -> -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
    return r;
}

// C 16-byte chunks (8 values) a thread; chunk i of thread t is chunk t + i * blockDim of the row.  A block walks
// rows blockIdx.x, + gridDim.x, ...: it keeps the weights, and the next row is under way while the two
// sums of this one are taken.
template <int C, bool F16>
__global__ void __launch_bounds__(C == 1 ? 1024 : 512) block_norm_kernel(const __grid_constant__ NormArgs p) {
    __shared__ float buf[2][2][32];
    const int warps = (int)blockDim.x >> 5, chunks = p.H >> 3;
    const float inv_h = 1.0f / (float)p.H, unit = p.unit_offset ? 1.0f : 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool by_element = p.gate_kind == MOE_GATE_ELEMENT;
    uint4 xv[C], rv[C], gv[C], post[C], pre[C];
    bool in[C];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = (int)threadIdx.x + i * (int)blockDim.x;
            xv[i] = rv[i] = zero;
            if (!in[i]) continue;
            if (p.x) xv[i] = *reinterpret_cast<const uint4 *>(p.x + row * p.x_ld + c * 8);
            if (p.resid) rv[i] = *reinterpret_cast<const uint4 *>(p.resid + row * p.resid_ld + c * 8);
            if (by_element) gv[i] = *reinterpret_cast<const uint4 *>(p.gate + row * p.gate_ld + c * 8);
        }
    };
    int64_t row = blockIdx.x;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        in[i] = c < chunks;
        gv[i] = post[i] = pre[i] = zero;
    }
    load(row);
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        if (!in[i]) continue;
        if (p.gate_kind == MOE_GATE_CHANNEL) gv[i] = *reinterpret_cast<const uint4 *>(p.gate + c * 8);
        if (p.w_post) post[i] = *reinterpret_cast<const uint4 *>(p.w_post + c * 8);
        if (p.y) pre[i] = *reinterpret_cast<const uint4 *>(p.w_pre + c * 8);
    }
    for (int turn = 0; row < p.T; turn ^= 1) {
        float g_row = p.alpha, r[C][8];
        if (p.gate_kind == MOE_GATE_TOKEN) {
            const float g = load1<F16>(p.gate + row * p.gate_ld);
            g_row *= p.sigmoid ? sigmoid(g) : g;
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
            inv = 1.0f / sqrtf(block_sum(ss, buf[turn][0], warps) * inv_h + p.eps);
        }
        inv *= g_row;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            unpack8<F16>(rv[i], r[i]);
            if (p.x) {
                float x[8], w[8], g[8];
                unpack8<F16>(xv[i], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= inv;
                if (p.w_post) {
                    unpack8<F16>(post[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= w[j] + unit;
                }
                if (p.gate_kind & MOE_GATE_CHANNEL) {  // per channel or per element
                    unpack8<F16>(gv[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= p.sigmoid ? sigmoid(g[j]) : g[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[i][j] += x[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(r[i][j], r[i][j], ss);
        }
        const int64_t next = row + gridDim.x;
        if (next < p.T) load(next);
        if (p.resid_out) {
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (in[i])
                    *reinterpret_cast<uint4 *>(p.resid_out + row * p.resid_out_ld + ((int)threadIdx.x + i * (int)blockDim.x) * 8) =
                        pack8<F16>(r[i]);
        }
        if (p.y) {
            const float inv2 = 1.0f / sqrtf(block_sum(ss, buf[turn][1], warps) * inv_h + p.eps);
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (!in[i]) continue;
                float w[8];
                unpack8<F16>(pre[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) r[i][j] *= inv2 * (w[j] + unit);
                *reinterpret_cast<uint4 *>(p.y + row * p.y_ld + ((int)threadIdx.x + i * (int)blockDim.x) * 8) = pack8<F16>(r[i]);
            }
        }
        row = next;
    }
}

template <int C, bool F16>
void launch_rows(const NormArgs &a, cudaStream_t s) {
    const int threads = ((a.H / 8 + C - 1) / C + 31) / 32 * 32;
    // as many blocks as are resident together (by registers, 1024 or 512 threads an SM)
    const int resident = device_info().sm_count * max((C == 1 ? 1024 : 512) / threads, 1);
    block_norm_kernel<C, F16><<<min(a.T, resident), threads, 0, s>>>(a);
}

template <bool F16>
cudaError_t launch(const NormArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_BLOCK_NORM, s);
    // One chunk a thread has a row soonest and the most warps an SM; two, in blocks that fit an SM twice, are
    // ahead where an SM has a few rows, so that their start and end count.  us with one and two: 500 rows of
    // 4096 6.1 and 6.1, 1000 of 2048 6.1 and 5.6, 1031 of 4096 10.5 and 10.1, 2048 of 2048 9.6 and 9.5, 4096 of 4096
    // 29.7 and 30.1, 8192 of 2048, gated, 32.6 and 33.1 (four: 51.9).
    const int chunks = a.H / 8, sms = device_info().sm_count;
    if (chunks > 1024) launch_rows<4, F16>(a, s);
    else if (chunks >= 128 && chunks <= 512 && a.T >= 4 * sms && a.T < 16 * sms) launch_rows<2, F16>(a, s);
    else launch_rows<1, F16>(a, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs &a, int dtype, cudaStream_t s) {
    return dtype == MOE_DTYPE_F16 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moe
