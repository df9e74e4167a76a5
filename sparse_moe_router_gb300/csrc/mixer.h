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
    int segment_chunks;
    float *seg_states, *seg_decay;
};
constexpr int kChunk = 64;  // tokens a chunk
// Segments of a batch, at most (sequence b owns the places base(b) .. base(b+1)-1, base(b) = q_start[b] / tokens + b).
inline int64_t linear_segments(int64_t n_tokens, int64_t n_seqs, int64_t segment_chunks) {
    return n_tokens / (segment_chunks * kChunk) + n_seqs;
}
cudaError_t launch_linear_chunks(const LinearArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_linear_tokens(const LinearArgs &a, int dtype, cudaStream_t s);

struct HeadNormArgs {
    const uint16_t *x, *weight, *gate;
    uint16_t *y;
    int64_t x_ld, gate_ld, y_ld;
    int T, heads, dim, center, gate_kind, weight_each, unit_offset;
    float eps;
};
cudaError_t launch_head_norm(const HeadNormArgs &a, int dtype, cudaStream_t s);

struct ProjectArgs {
    const uint16_t *x, *w, *bias;
    const void *resid;
    void *y;
    int64_t x_ld, w_ld, resid_ld, y_ld;
    int T, K, N, act, out_f32;
    float scale;
    int *status;
};
cudaError_t launch_project_rows(const ProjectArgs &a, int dtype, cudaStream_t s);

// A log decay below this counts as this: its factor is 0 in fp32, and sums of 64 stay finite.
constexpr float kLeastDecay = -10000.f;

#ifdef __CUDACC__
// 1 / (1 + e^-x) to about 2 ulp; x -> -inf gives 1 / inf = 0.
__device__ __forceinline__ float sigmoid_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
    return r;
}
// x / (1 + e^-x): at x -> -inf the product would be -inf * 0.
__device__ __forceinline__ float silu_fast(float x) { return x < -88.f ? x * __expf(x) : x * sigmoid_fast(x); }

__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case MOE_ACT_RELU: return z > 0.f ? z : z != z ? z : 0.f;
        case MOE_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        case MOE_ACT_SILU: return silu_fast(z);
        case MOE_ACT_SIGMOID: return sigmoid_fast(z);
        case MOE_ACT_LOG_SIGMOID: return fminf(z, 0.f) - log1pf(expf(-fabsf(z)));
        default: return z;
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
    r.pad = min(max(r.n - kv, 0), r.n);
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
