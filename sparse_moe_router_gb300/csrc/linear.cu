// linear.cu -- moe_linear_attention token by token: S = e^g S + k v^T, out = scale S^T q.
//
// Columns of a state (value channels) do not meet, so a block takes 32 of them with all DK rows in registers, from the
// first new token to the last: the state is read once and written once, however many tokens there are.
#include "mixer.h"

namespace moe {
namespace {

constexpr int kCols = 32;      // value channels a block: 8 threads of 4
constexpr int kThreads = 256;  // 32 rows at once
constexpr int kRowsAtOnce = kThreads / (kCols / 4);

template <int DK, bool F16>
__global__ void __launch_bounds__(kThreads) linear_tokens_kernel(const __grid_constant__ LinearArgs p) {
    constexpr int R = DK / kRowsAtOnce;
    __shared__ float qk[2][2][DK];
    __shared__ float4 part[2][kThreads / 32][kCols / 4];
    const int tid = (int)threadIdx.x, c = tid & 7, r = tid >> 3;
    const int tiles = p.DV / kCols, b = (int)blockIdx.x / tiles, h = (int)blockIdx.y;
    const int col0 = ((int)blockIdx.x - b * tiles) * kCols, col = col0 + c * 4;
    const Run run = load_run(p, b);
    if (run.n >= p.chunk_tokens) return;  // the chunk kernel's
    for (int i = tid; i < run.pad * kCols; i += kThreads)
        p.out[(int64_t)(run.q0 - run.pad + i / kCols) * p.out_ld + (int64_t)h * p.DV + col0 + i % kCols] = 0;
    if (run.n <= 0) return;
    float4 S[R];
    float *state = p.states + ((int64_t)max(run.slot, 0) * p.VH + h) * DK * p.DV + col;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!run.fresh) S[i] = *reinterpret_cast<const float4 *>(state + (int64_t)(r + i * kRowsAtOnce) * p.DV);
    }
    const int kh = h / p.G;
    auto load = [&](int t) -> float {  // a key or query value of token t for shared memory
        const int64_t row = run.q0 + t;
        if (tid < DK) return load1<F16>(p.k + row * p.k_ld + kh * DK + tid);
        if (tid >= kThreads - DK) return load1<F16>(p.q + row * p.q_ld + kh * DK + tid - (kThreads - DK));
        return 0.f;
    };
    float next = load(0);
    for (int t = 0; t < run.n; ++t) {
        const int buf = t & 1;
        if (tid < DK) qk[buf][0][tid] = next;
        if (tid >= kThreads - DK) qk[buf][1][tid - (kThreads - DK)] = next;
        const int64_t row = run.q0 + t;
        const uint2 vw = *reinterpret_cast<const uint2 *>(p.v + row * p.v_ld + (int64_t)h * p.DV + col);
        const float f = expf(checked_decay(p, raw_decay(p, row, h)));
        const float2 v0 = unpack2<F16>(vw.x), v1 = unpack2<F16>(vw.y);
        if (t + 1 < run.n) next = load(t + 1);
        __syncthreads();
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float k = qk[buf][0][r + i * kRowsAtOnce], q = qk[buf][1][r + i * kRowsAtOnce];
            S[i].x = fmaf(S[i].x, f, k * v0.x), S[i].y = fmaf(S[i].y, f, k * v0.y);
            S[i].z = fmaf(S[i].z, f, k * v1.x), S[i].w = fmaf(S[i].w, f, k * v1.y);
            acc.x = fmaf(q, S[i].x, acc.x), acc.y = fmaf(q, S[i].y, acc.y);
            acc.z = fmaf(q, S[i].z, acc.z), acc.w = fmaf(q, S[i].w, acc.w);
        }
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o), acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o), acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
        if ((tid & 31) < 8) part[buf][tid >> 5][c] = acc;
        __syncthreads();
        if (tid < kCols / 2) {  // two channels a thread
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                const float2 a = reinterpret_cast<const float2 *>(part[buf][w])[tid];
                sum.x += a.x, sum.y += a.y;
            }
            *reinterpret_cast<uint32_t *>(p.out + row * p.out_ld + (int64_t)h * p.DV + col0 + tid * 2) =
                pack2<F16>(sum.x * p.scale, sum.y * p.scale);
        }
    }
    if (run.slot >= 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(state + (int64_t)(r + i * kRowsAtOnce) * p.DV) = S[i];
    }
}

template <int DK, bool F16>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_LINEAR_TOKENS, s);
    linear_tokens_kernel<DK, F16><<<dim3((unsigned)(a.DV / kCols) * a.n_seqs, a.VH), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_tokens(const LinearArgs &a, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (a.DK == 64) return f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace moe
