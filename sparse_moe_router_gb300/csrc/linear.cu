// linear.cu -- moe_linear_attention token by token: S = e^g S + k v^T, out = scale S^T q.
//
// Columns of a state (value channels) do not meet, so a block takes some of them with all DK rows in registers, from the
// first new token to the last: the state is read once and written once, however many tokens there are.  Eight tokens
// at a time share two barriers: their queries and keys go to shared memory together, and the warps' parts of their
// outputs are joined together.
//
// Bound: HBM, 2 x 4 DK DV bytes a head and sequence; for a few heads the launch and three dependent reads (the sequence, its
// state, the joined sums).  Measured, 32 heads of 128 and 128: one sequence 2.8 us, 48 sequences 35.6 to 38 (5.3 to 5.7 TB/s,
// 78 to 84% of the measured copy), 200 130 (95%); 8 sequences of 4 tokens, 8 heads of 64 and 64, 3.1.  (A call from Python
// takes 4 to 5 us of the host beside that.)
#include "mixer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;     // tokens

// kCols value channels a block, 4 a thread.
template <int DK, int kCols, bool F16>
__global__ void __launch_bounds__(kThreads, 2) linear_tokens_kernel(const __grid_constant__ LinearArgs p) {
    constexpr int kRowsAtOnce = kThreads / (kCols / 4), R = DK / kRowsAtOnce;
    __shared__ float ks[kAtOnce][DK], qs[kAtOnce][DK], fs[kAtOnce];
    __shared__ float4 part[kAtOnce][kThreads / 32][kCols / 4];
    const int tid = (int)threadIdx.x, c = tid & (kCols / 4 - 1), r = tid / (kCols / 4);
    const int tiles = p.DV / kCols, b = (int)blockIdx.x / tiles, h = (int)blockIdx.y;
    const int col0 = ((int)blockIdx.x - b * tiles) * kCols, col = col0 + c * 4;
    const Run run = load_run(p, b);
    if (run.n < p.chunk_tokens) {  // (the others are the chunk kernel's)
        for (int i = tid; i < run.pad * kCols; i += kThreads)
            p.out[(int64_t)(run.q0 - run.pad + i / kCols) * p.out_ld + (int64_t)h * p.DV + col0 + i % kCols] = 0;
        float4 S[R];
        float *state = p.states + ((int64_t)max(run.slot, 0) * p.VH + h) * DK * p.DV + col;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!run.fresh && run.n > 0) S[i] = *reinterpret_cast<const float4 *>(state + (int64_t)(r + i * kRowsAtOnce) * p.DV);
        }
        const int kh = h / p.G;
        for (int t0 = 0; t0 < run.n; t0 += kAtOnce) {
            const int m = min(run.n - t0, kAtOnce);
            const int64_t row0 = run.q0 + t0;
            if (t0 > 0) __syncthreads();
            for (int i = tid; i < m * DK; i += kThreads) {
                const int64_t row = row0 + i / DK;
                const int d = kh * DK + i % DK;
                ks[i / DK][i % DK] = load1<F16>(p.k + row * p.k_ld + d);
                qs[i / DK][i % DK] = load1<F16>(p.q + row * p.q_ld + d);
            }
            if (tid < m) fs[tid] = expf(checked_decay(p, raw_decay(p, row0 + tid, h)));
            const uint16_t *v = p.v + row0 * p.v_ld + (int64_t)h * p.DV + col;
            uint2 vw = *reinterpret_cast<const uint2 *>(v);
            __syncthreads();
            for (int t = 0; t < m; ++t) {
                const float2 v0 = unpack2<F16>(vw.x), v1 = unpack2<F16>(vw.y);
                if (t + 1 < m) vw = *reinterpret_cast<const uint2 *>(v + (t + 1) * p.v_ld);
                const float f = fs[t];
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float k = ks[t][r + i * kRowsAtOnce], q = qs[t][r + i * kRowsAtOnce];
                    S[i].x = fmaf(S[i].x, f, k * v0.x), S[i].y = fmaf(S[i].y, f, k * v0.y);
                    S[i].z = fmaf(S[i].z, f, k * v1.x), S[i].w = fmaf(S[i].w, f, k * v1.y);
                    acc.x = fmaf(q, S[i].x, acc.x), acc.y = fmaf(q, S[i].y, acc.y);
                    acc.z = fmaf(q, S[i].z, acc.z), acc.w = fmaf(q, S[i].w, acc.w);
                }
#pragma unroll
                for (int o = kCols / 4; o < 32; o <<= 1) {
                    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o), acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
                    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o), acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
                }
                if ((tid & 31) < kCols / 4) part[t][tid >> 5][c] = acc;
            }
            if (t0 + m >= run.n && run.slot >= 0) {
#pragma unroll
                for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(state + (int64_t)(r + i * kRowsAtOnce) * p.DV) = S[i];
            }
            __syncthreads();
            for (int y = tid; y < m * (kCols / 2); y += kThreads) {  // two channels a thread
                const int t = y / (kCols / 2), e = y % (kCols / 2);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kThreads / 32; ++w) {
                    const float2 a = reinterpret_cast<const float2 *>(part[t][w])[e];
                    sum.x += a.x, sum.y += a.y;
                }
                *reinterpret_cast<uint32_t *>(p.out + (row0 + t) * p.out_ld + (int64_t)h * p.DV + col0 + e * 2) =
                    pack2<F16>(sum.x * p.scale, sum.y * p.scale);
            }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the chunk kernel's end: what follows this grid follows both
}

template <int DK, int kCols, bool F16>
cudaError_t launch_cols(const LinearArgs &a, bool after_chunks, cudaStream_t s) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(a.DV / kCols) * a.n_seqs, a.VH);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = after_chunks ? 1 : 0;
    LaunchScope scope(KC_LINEAR_TOKENS, s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_tokens_kernel<DK, kCols, F16>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DK, bool F16>
cudaError_t launch(const LinearArgs &a, bool after_chunks, cudaStream_t s) {
    // Whole heads (of up to 128 channels) a block, with 64 KB under way in it, where they give every SM one; else 32 channels,
    // so that few heads reach all SMs.  us with 32 and 128 channels, 32 heads of 128 and 128: 1 sequence 2.9 and 4.1, 8 6.7
    // and 5.8, 48 41.5 and 35.5, 200 160 and 130 (64 channels: 3.1, 6.9, 44.7, 173).
    const bool many = (int64_t)a.n_seqs * a.VH >= device_info().sm_count;
    if (!many) return launch_cols<DK, 32, F16>(a, after_chunks, s);
    return a.DV == 64 ? launch_cols<DK, 64, F16>(a, after_chunks, s) : launch_cols<DK, 128, F16>(a, after_chunks, s);
}

}  // namespace

// after_chunks: the launch just before, on the same stream, is the same call's chunk kernel, beside which this one may run.
cudaError_t launch_linear_tokens(const LinearArgs &a, int dtype, bool after_chunks, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (a.DK == 64) return f16 ? launch<64, true>(a, after_chunks, s) : launch<64, false>(a, after_chunks, s);
    return f16 ? launch<128, true>(a, after_chunks, s) : launch<128, false>(a, after_chunks, s);
}

}  // namespace moe
