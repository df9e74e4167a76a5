// mixer.h -- declarations shared by the kernels of the recurrent token mixer: linear attention over a state,
// the heads' norm, products with an epilogue.
#pragma once

#include "layer.h"

namespace moe {

struct LinearArgs {
    const int32_t *q_start, *kv_len, *slots;
    float *states;
    const uint16_t *q, *k, *v;
    const float *decay;
    uint16_t *out;
    int64_t q_ld, k_ld, v_ld, out_ld, decay_ld;
    int n_seqs, n_tokens, n_slots;
    int KH, VH, G, DK, DV;
    float scale;
    int *status;
    // sequences with at least this many new tokens are the chunk kernel's, the others the token kernel's
    int chunk_tokens;
    // chunk kernel: a run's chunks in segments of so many; with several, the state that each adds and its decay
    int segment_chunks, place_tokens;
    float *seg_states, *seg_decay;
};
constexpr int kChunk = 64;  // tokens a chunk
// Places of a batch's segments.  Sequence b owns the places base(q_start[b], b) .. base(q_start[b+1], b+1)-1: at least as many
// as its run of n has segments of W tokens.  With place_tokens 0 one more than n / W for each sequence, else for each
// place_tokens tokens (runs of fewer are not the chunk kernel's): of many sequences with few tokens, that is fewer.
__host__ __device__ __forceinline__ int segment_base(int q_start, int b, int segment_chunks, int place_tokens) {
    return q_start / (segment_chunks * kChunk) + (place_tokens > 0 ? q_start / place_tokens : b);
}
cudaError_t launch_linear_chunks(const LinearArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_linear_tokens(const LinearArgs &a, int dtype, bool after_chunks, cudaStream_t s);

struct HeadNormArgs {
    const uint16_t *x, *weight, *gate;
    uint16_t *y;
    int64_t x_ld, gate_ld, y_ld;
    int T, heads, dim, center, gate_kind, weight_each, unit_offset;
    float eps;
};
cudaError_t launch_head_norm(const HeadNormArgs &a, int dtype, cudaStream_t s);

// Activations of fp32 outputs that have a form of their own (ProjectArgs::act, beside moe_act).
constexpr int kSilu32 = MOE_ACT_LOG_SIGMOID + 1, kSigmoid32 = kSilu32 + 1;
struct ProjectArgs {
    const uint16_t *x, *w, *bias;
    const void *resid;
    void *y;
    int64_t x_ld, w_ld, resid_ld, y_ld;
    int T, K, N, act, out_f32;
    float scale;
    int *status;
};
cudaError_t launch_project_rows(const ProjectArgs &a, int dtype, cudaStream_t s);   // a few rows
cudaError_t launch_project_batch(const ProjectArgs &a, int dtype, cudaStream_t s);  // at most 256 rows or outputs
cudaError_t launch_project_tiles(const ProjectArgs &a, int dtype, cudaStream_t s);  // any
// Estimates, us, of the last two, for at most 256 rows or outputs.
cudaError_t project_batch_time(const ProjectArgs &a, int dtype, double *us);
double project_tiles_time(const ProjectArgs &a);

// Lets a kernel's setup run under the end of the one before it on the stream (it then waits before its first access).
inline void overlap_prior(cudaLaunchAttribute &attr) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
}

// A log decay below this counts as this: its factor is 0 in fp32, and sums of 64 stay finite.
constexpr float kLeastDecay = -10000.f;

#ifdef __CUDACC__
// 1 / (1 + e^-x) for what is rounded to 16 bits: to 2 ulp above 0, to 2 + 1.2 |x| ulp below (__expf's error; 2^-16 at its end),
// and 0 below -87.3, where the result is less than 2^-126.
__device__ __forceinline__ float sigmoid_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
    return r;
}
__device__ __forceinline__ float silu_fast(float x) { return x * sigmoid_fast(x); }
// The same to a few ulp everywhere, for outputs in 32 bits: e^x / (1 + e^x) below 0, down to fp32's least value.  (For all outputs
// it would cost 22% where the epilogue bounds: 8192 rows of 512, 8192 bf16 outputs with SiLU 88 and 108 us.)
__device__ __forceinline__ float sigmoid(float x) {
    const float u = expf(-fabsf(x)), s = __fdividef(1.f, 1.f + u);
    return x < 0.f ? u * s : s;
}

// z Phi(z), Phi(-x) = erfc(x / sqrt(2)) / 2, by the Chebyshev fit of erfc whose error is below 1.2e-7 of the value
// everywhere (Press et al., Numerical Recipes, "erfcc"), beside which far below 0 the rounding of x^2 and __expf leave some 4 x^2
// half steps: with erff and its branches a product of 1031 rows and 4104 outputs took 36.7 us, with this 26.5.
__device__ __forceinline__ float gelu(float z) {
    const float x = fabsf(z) * 0.70710678118654752f, t = __fdividef(1.f, fmaf(0.5f, x, 1.f));
    float e = fmaf(t, 0.17087277f, -0.82215223f);
    e = fmaf(t, e, 1.48851587f);
    e = fmaf(t, e, -1.13520398f);
    e = fmaf(t, e, 0.27886807f);
    e = fmaf(t, e, -0.18628806f);
    e = fmaf(t, e, 0.09678418f);
    e = fmaf(t, e, 0.37409196f);
    e = fmaf(t, e, 1.00002368f);
    e = fmaf(t, e, -1.26551223f);
    const float half = 0.5f * t * __expf(fmaf(-x, x, e));
    return z * (z < 0.f ? half : 1.f - half);
}
// -log(1 + e^-z) = min(z, 0) - log(1 + u), u = e^-|z|, with log(1 + u) = 2 artanh(s), s = u / (2 + u) <= 1/3, by its series:
// exact to the last bits of values near 0 too, as long sums of log decays need.
__device__ __forceinline__ float log_sigmoid(float z) {
    const float u = expf(-fabsf(z)), s = __fdividef(u, 2.f + u), q = s * s;
    float r = fmaf(q, 1.f / 15.f, 1.f / 13.f);
    r = fmaf(q, r, 1.f / 11.f);
    r = fmaf(q, r, 1.f / 9.f);
    r = fmaf(q, r, 1.f / 7.f);
    r = fmaf(q, r, 1.f / 5.f);
    r = fmaf(q, r, 1.f / 3.f);
    return fminf(z, 0.f) - 2.f * fmaf(s * q, r, s);
}
template <int V>
__device__ __forceinline__ void activate(float (&z)[V], int act) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = z[j] < 0.f ? 0.f : z[j];
            break;
        case MOE_ACT_GELU:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = gelu(z[j]);
            break;
        case MOE_ACT_SILU:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = silu_fast(z[j]);
            break;
        case MOE_ACT_SIGMOID:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = sigmoid_fast(z[j]);
            break;
        case kSilu32:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] *= sigmoid(z[j]);
            break;
        case kSigmoid32:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = sigmoid(z[j]);
            break;
        case MOE_ACT_LOG_SIGMOID:
#pragma unroll
            for (int j = 0; j < V; ++j) z[j] = log_sigmoid(z[j]);
            break;
        default: break;
    }
}

// The epilogue of V outputs of one row from output n on: z + bias, activation, scale, residual, one rounding, one store.
template <int V, bool F16>
__device__ __forceinline__ void finish(const ProjectArgs &p, int64_t t, int n, float (&z)[V], const float (&bias)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] += bias[j];
    activate(z, p.act);
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] *= p.scale;
    if (p.out_f32) {
        if (p.resid) {
            const float4 *r = reinterpret_cast<const float4 *>(static_cast<const float *>(p.resid) + t * p.resid_ld + n);
#pragma unroll
            for (int j = 0; j < V / 4; ++j) z[4 * j] += r[j].x, z[4 * j + 1] += r[j].y, z[4 * j + 2] += r[j].z, z[4 * j + 3] += r[j].w;
        }
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(p.y) + t * p.y_ld + n);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) y[j] = make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
    } else {
        if (p.resid) {
            const uint2 *r = reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.resid) + t * p.resid_ld + n);
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                const uint2 w = r[j];
                const float2 a = unpack2<F16>(w.x), b = unpack2<F16>(w.y);
                z[4 * j] += a.x, z[4 * j + 1] += a.y, z[4 * j + 2] += b.x, z[4 * j + 3] += b.y;
            }
        }
        uint32_t w[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) w[j] = pack2<F16>(z[2 * j], z[2 * j + 1]);
        uint16_t *y = static_cast<uint16_t *>(p.y) + t * p.y_ld + n;
        if constexpr (V == 8) *reinterpret_cast<uint4 *>(y) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(y) = make_uint2(w[0], w[1]);
    }
}
// (0 without a bias)
template <int V, bool F16>
__device__ __forceinline__ void load_bias(const ProjectArgs &p, int n, float (&bias)[V]) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        uint2 w = make_uint2(0, 0);
        if (p.bias) w = __ldg(reinterpret_cast<const uint2 *>(p.bias + n + j));
        const float2 a = unpack2<F16>(w.x), b = unpack2<F16>(w.y);
        bias[j] = a.x, bias[j + 1] = a.y, bias[j + 2] = b.x, bias[j + 3] = b.y;
    }
}

// One sequence of the batch: rows q0 .. q0+n-1 count (padding in front left out), its state's slot or -1, and whether
// it begins with an empty state.  What the device arrays say is checked before it is used.
struct Run {
    int q0, n, pad, slot;
    bool fresh;
};
__device__ __forceinline__ Run load_run(const LinearArgs &a, int b) {
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], kv = a.kv_len[b], slot = a.slots[b];
    Run r;
    r.q0 = q0;
    r.n = q1 - q0;
    r.slot = slot;
    bool bad = false;
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens) {
        r.q0 = r.n = 0;
        bad = true;
    }
    if (slot < 0 || slot >= a.n_slots) {
        r.slot = -1;
        bad = bad || r.n > 0;
    }
    r.fresh = kv <= r.n || r.slot < 0;
    r.pad = max(r.n - max(kv, 0), 0);
    r.q0 += r.pad;
    r.n -= r.pad;
    if (bad) layer_error(a.status);
    return r;
}

// Log decay of row t (of value head h) as it is given, and checked.
__device__ __forceinline__ float raw_decay(const LinearArgs &a, int64_t t, int h) {
    return a.decay ? __ldg(a.decay + (a.decay_ld ? t * a.decay_ld : 0) + h) : 0.f;
}
__device__ __forceinline__ float checked_decay(const LinearArgs &a, float g) {
    if (!(g <= 0.f)) layer_error(a.status);
    return g <= 0.f ? fmaxf(g, kLeastDecay) : 0.f;
}
#endif

}  // namespace moe
