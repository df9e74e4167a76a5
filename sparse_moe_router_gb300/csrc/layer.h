// layer.h -- declarations shared by the kernels of the decoder layer's other half: block norms,
// append into the paged 8-bit cache, attention over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace moe {

// The cache and the batch as the kernels see them (include/moe.h: moe_kv_cache, moe_kv_batch).
struct KvView {
    const int32_t *q_start, *kv_len, *table;
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    int n_seqs, n_tokens, max_pages, n_pages;
    int QH, KH, G, P, log_p;
    int *status;
};

// Exponents of a cache scale (a power of two): amax <= 448 * 2^e, and 448 = 1.75 * 2^8.
constexpr int kScaleMinExp = -60;

struct AppendArgs {
    KvView kv;
    const uint16_t *q, *k, *v;
    int64_t q_ld, k_ld, v_ld, q_out_ld;
    const float *rope;
    int rope_rows, rot, interleaved;
    uint16_t *q_out;
    int q_tokens;    // tokens a block of the q part handles
    int page_items;  // (page slots) x 2 x kv heads
    int page_blocks; // blocks that they take (set by the launch)
};
cudaError_t launch_kv_append(const AppendArgs &a, int D, int dtype, cudaStream_t s);

struct SplitDesc {
    int parts, rows, q0, row0, head;  // parts 0: none
};

struct AttnArgs {
    KvView kv;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t q_ld, out_ld;
    float scale_log2;  // softmax_scale * log2(e)
    int causal, window;
    // split kernel: partial results, two slots a block, and where the segment is that begins in a block and
    // goes on in others
    float *part;
    SplitDesc *desc;
    // sequences with at least this many query rows a kv head (new tokens x G) are the prompt
    // kernel's, the others the split kernel's
    int prompt_rows;
    // prompt kernel: the keys of a block in so many parts at most, and with more than one each part's rows, [parts, T, QH, D]
    // normalised and [parts, T, QH] the log2 of their sums: -infinity where a part has nothing, and in the first
    // +infinity where it has all and its block has written the output
    int parts;
    float *part_out, *part_lse;
};
// The workspace is sized for so many SMs; the split kernel has one or two blocks on each.
constexpr int kSplitMaxSms = 160, kSplitMaxBlocks = 2 * kSplitMaxSms;
// Floats of workspace the split kernel needs for partial results.
size_t split_part_floats(int D);
cudaError_t launch_attn_split(const AttnArgs &a, int D, int dtype, bool shared, bool after_prompt, cudaStream_t s);
cudaError_t launch_attn_prompt(const AttnArgs &a, int D, int dtype, cudaStream_t s);
inline int prompt_block_rows(int D) { return D == 256 ? 128 : 256; }  // query rows a block of the prompt kernel
constexpr int kPromptParts = 16;  // at most

// Softmax weights 2^(z - m) are rounded to fp16 for the product with the values: 11 bits from 2^-14 on, an absolute 2^-25
// below, 0 below that, while their sum keeps them in fp32.  So that keys far below a row's largest one still count
// (together they may be most of its output, where that key's value is near 0), the reference m lies 2^9 under
// the largest z when it is set: 11 bits down to 2^-23 of the largest weight, something down to 2^-34.
constexpr float kBelowTop = 9.f;

struct NormArgs {
    const uint16_t *x, *resid, *gate, *w_post, *w_pre;
    uint16_t *resid_out, *y;
    int64_t x_ld, resid_ld, gate_ld, resid_out_ld, y_ld;
    int T, H, gate_kind, sigmoid, unit_offset;
    float eps, alpha;
};
cudaError_t launch_block_norm(const NormArgs &a, int dtype, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ void layer_error(int *status) { atomicCAS(status, 0, (int)MOE_ERR_INVALID_ARG); }

// 16-bit activations <-> fp32, by the call's dtype.
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (F16) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <bool F16>
__device__ __forceinline__ float load1(const uint16_t *p) {
    const uint32_t v = *p;
    return F16 ? __half2float(__ushort_as_half((unsigned short)v)) : __uint_as_float(v << 16);
}
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = unpack2<F16>(w[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
}

// Four E4M3 codes as two pairs of fp16 values (exact: every E4M3 value is an fp16 value).
__device__ __forceinline__ void widen4(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}

// 16 codes, read once by this block: not kept in L1.
__device__ __forceinline__ uint4 load_codes16(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// One sequence of the batch.  What the device arrays say is checked before it is used: a range
// outside the batch's tokens counts as no tokens, a length outside the table as the nearest end.
struct Seq {
    int q0, n, kv;
};
__device__ __forceinline__ Seq checked_seq(const KvView &v, int q0, int q1, int kv) {
    Seq s;
    s.q0 = q0;
    s.n = q1 - q0;
    s.kv = kv;
    const long long most = (long long)v.max_pages << v.log_p;
    bool bad = false;
    if (q0 < 0 || q1 < q0 || q1 > v.n_tokens) {
        s.q0 = s.n = 0;
        bad = true;
    }
    if (s.kv < 0 || s.kv > most) {
        s.kv = s.kv < 0 ? 0 : (int)most;
        bad = true;
    }
    if (bad) layer_error(v.status);
    return s;
}
__device__ __forceinline__ Seq load_seq(const KvView &v, int b) {
    return checked_seq(v, v.q_start[b], v.q_start[b + 1], v.kv_len[b]);
}
#endif

}  // namespace moe
