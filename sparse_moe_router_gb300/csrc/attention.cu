// attention.cu -- attention over the paged 8-bit cache, split along the keys: the form for single
// tokens and short query runs.
//
// Per row (token, q head): o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j), with k_j = 2^ek code
// and v_j = 2^ev code under the page's exponents.  In base 2 and with the value's scale drawn into
// the weight:  z_j = S_j 2^ek c + ev,  w_j = 2^(z_j - m),  o = sum_j w_j code_j / sum_j w_j 2^-ev:
// the products then run on the codes alone, which are exact in fp16, and pages of any scales mix.
//
// Bound: every code byte is read once and takes part in 2 x (rows of its head) products, so a
// decode step is bound by HBM.  The kernel streams the codes straight from global memory into the
// register fragments of mma.sync.m16n8k16: with keys (or value dims) on the 16-row side and up to
// 8 query rows on the 8-wide side no product is wasted for a group of 8 heads, the contraction
// index is free to be permuted, so each thread reads its fragment as 16-byte runs of a row, and
// nothing passes through shared memory.  (tcgen05 would need 128 rows on one side and the codes
// widened in shared memory first: with 8 rows a head the tensor cores are nearly idle either way.)
//
// Split: the batch's work is laid out as one line of 64-key steps (sequence by sequence, kv
// head by kv head, 8-row tile by tile) and cut into equal runs, one a block, whatever the
// lengths.  A run that ends inside a segment leaves partial sums; the block that finishes a
// segment last joins them in order, so the result does not depend on which one that is.
#include "layer.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16 * kWarps;  // keys a block takes at once, 16 a warp

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8x8 matrix of 16-bit values held two a thread.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ int exponent_of(float s) { return (int)((__float_as_uint(s) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// The keys that rows of tokens [t0, t1) (of a sequence's n) see at least one of: [lo, hi).
__device__ __forceinline__ void key_range(const AttnArgs &p, const Seq &q, int t0, int t1, int &lo, int &hi) {
    const int pos0 = q.kv - q.n + t0, pos1 = q.kv - q.n + t1 - 1;
    hi = p.causal ? min(q.kv, pos1 + 1) : q.kv;
    lo = p.window > 0 ? max(0, pos0 + 1 - p.window) : 0;
    if (hi < lo) hi = lo;
}

// Rows a tile holds: 8 query rows (token, head) of one kv head.
constexpr int kRows = 8;

// A sequence's share of the line of steps: tiles * steps * kv heads.
struct SeqWork {
    Seq q;
    int tiles, step0, steps;
};
__device__ __forceinline__ SeqWork seq_work(const AttnArgs &p, int b) {
    SeqWork w;
    w.q = load_seq(p.kv, b);
    if ((int64_t)w.q.n * p.kv.G >= p.prompt_rows) w.q.n = 0;  // the prompt kernel's
    w.tiles = (int)(((int64_t)w.q.n * p.kv.G + kRows - 1) / kRows);
    int lo, hi;
    key_range(p, w.q, 0, max(w.q.n, 1), lo, hi);
    w.step0 = lo / kStep;
    w.steps = max((hi + kStep - 1) / kStep - w.step0, 1);  // one at least: it writes the empty rows
    return w;
}
__device__ __forceinline__ int64_t line_steps(const AttnArgs &p, const SeqWork &w) {
    return (int64_t)w.tiles * w.steps * p.kv.KH;
}

template <int D, bool F16>
struct Split {
    static constexpr int kKLoads = D / 64;     // 16-byte runs of a key row a thread reads
    static constexpr int kVRun = D / 8;        // value dims a thread owns (of every 4th..: 4 tokens)
    static constexpr int kMT = D / 16;         // 16-dim output tiles
    static constexpr int kPart = kRows * D + 2 * kRows;  // floats of a partial result: sums, m, l
};

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, D <= 128 ? 3 : 2) attn_split_kernel(const __grid_constant__ AttnArgs p) {
    using C = Split<D, F16>;
    constexpr int kMT = C::kMT;
    const KvView &v = p.kv;
    __shared__ int64_t scan[kWarps + 1];
    __shared__ int64_t found_at;
    __shared__ int found_b;
    __shared__ float merge_m[kWarps][kRows], merge_l[kWarps][kRows];
    __shared__ __align__(16) float merge_o[kWarps][kRows][D];  // read and written as float4
    __shared__ int last_flag;

    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;

    // ------------------------------------------------- this block's run of the line --
    // total steps, then the sequence that holds the run's first step
    int64_t total = 0;
    for (int b = tid; b < v.n_seqs; b += kThreads) total += line_steps(p, seq_work(p, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += scan[w];
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    const int64_t begin = per * blockIdx.x, end = min(total, begin + per);
    if (begin >= end) return;
    int64_t before = 0;  // steps of the sequences before the chunk
    for (int b0 = 0;; b0 += kThreads) {
        __syncthreads();
        const int b = b0 + tid;
        const int64_t own = b < v.n_seqs ? line_steps(p, seq_work(p, b)) : 0;
        int64_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) scan[warp] = inc;
        if (tid == 0) found_b = -1;
        __syncthreads();
        int64_t base = before, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += scan[w];
            all += scan[w];
        }
        if (begin >= base + inc - own && begin < base + inc) {
            found_b = b;
            found_at = base + inc - own;
        }
        __syncthreads();
        if (found_b >= 0) break;
        before += all;
    }
    int b = found_b;
    int64_t seq_at = found_at;  // where sequence b begins on the line
    SeqWork sw = seq_work(p, b);

    for (int64_t at = begin; at < end;) {
        while (at >= seq_at + line_steps(p, sw)) {
            seq_at += line_steps(p, sw);
            sw = seq_work(p, ++b);
        }
        // ---------------------------------------------------------------- a segment --
        const int64_t seg = (at - seq_at) / sw.steps;  // (head, tile) of the sequence
        const int64_t seg_at = seq_at + seg * sw.steps, seg_end = seg_at + sw.steps;
        const int head = (int)(seg / sw.tiles), tile = (int)(seg % sw.tiles);
        const int s0 = (int)(at - seg_at), s1 = (int)(min(end, seg_end) - seg_at);
        at = seg_at + s1;
        const int row0 = tile * kRows, rows = min(kRows, sw.q.n * v.G - row0);
        const int first_pos = sw.q.kv - sw.q.n;

        // q rows: fragment rows are n = g, dims i*64 + t*16 + 4s of the four k-steps of run i
        uint32_t qf[C::kKLoads][4][2];
        int q_exp = 0;
        {
            float amax = 0.f;
            float qv[C::kKLoads][16];
            const int r = row0 + g;
            const uint16_t *row = p.q + (int64_t)(sw.q.q0 + r / v.G) * p.q_ld + (int64_t)(head * v.G + r % v.G) * D + t * 16;
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i) {
                uint4 a = make_uint4(0, 0, 0, 0), c = a;
                if (g < rows) {
                    a = *reinterpret_cast<const uint4 *>(row + i * 64);
                    c = *reinterpret_cast<const uint4 *>(row + i * 64 + 8);
                }
                float x[8], y[8];
                unpack8<F16>(a, x);
                unpack8<F16>(c, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    qv[i][j] = x[j];
                    qv[i][8 + j] = y[j];
                    amax = fmaxf(amax, fmaxf(fabsf(x[j]), fabsf(y[j])));
                }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // largest magnitude into [1, 2): fp16 then holds every bf16 digit down to 2^-17 of it
            q_exp = amax > 0.f ? max(min((int)(__float_as_uint(amax) >> 23) - 127, 126), -126) : 0;
            const float inv = pow2f(-q_exp);
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    qf[i][s][0] = pack2<true>(qv[i][4 * s] * inv, qv[i][4 * s + 1] * inv);
                    qf[i][s][1] = pack2<true>(qv[i][4 * s + 2] * inv, qv[i][4 * s + 3] * inv);
                }
        }
        // the two rows whose logits and sums this thread holds: n = 2t, 2t + 1
        float mul[2];
        int lo[2], hi[2];
        int all_lo = 0, all_hi = 0x7fffffff;  // keys in [all_lo, all_hi) are seen by every row
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int e = __shfl_sync(0xffffffffu, q_exp, (2 * t + c) * 4);
            mul[c] = p.scale_log2 * pow2f(e);
            const int pos = first_pos + (row0 + 2 * t + c) / v.G;
            hi[c] = p.causal ? min(sw.q.kv, pos + 1) : sw.q.kv;
            lo[c] = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
            if (2 * t + c < rows) {
                all_lo = max(all_lo, lo[c]);
                all_hi = min(all_hi, hi[c]);
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
            all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        }

        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        float o[kMT][4];
#pragma unroll
        for (int i = 0; i < kMT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        // tiles of 16 keys: [key0, key0 + 16), key0 = (step0 + s) * 64 + warp * 16, up to the last
        // key that a row of this tile sees
        int klo, khi;
        key_range(p, sw.q, row0 / v.G, (row0 + rows - 1) / v.G + 1, klo, khi);
        const int32_t *table = v.table + (int64_t)b * v.max_pages;
        int ks = max((sw.step0 + s0) * kStep, klo / kStep * kStep) + warp * 16;
        const int ke = min((sw.step0 + s1) * kStep, khi);
        auto page_of = [&](int key) {
            int page = 0;
            if (key < ke) {
                page = __ldg(table + (key >> v.log_p));
                if (page < 0 || page >= v.n_pages) {
                    layer_error(v.status);
                    page = 0;
                }
            }
            return page;
        };
        uint4 kr[2][C::kKLoads];
        uint32_t vr[4][C::kVRun / 4];
        auto load_k = [&](int key, int page) {
            const uint8_t *base = v.k_codes + (((int64_t)page * v.KH + head) * v.P + (key & (v.P - 1))) * D + t * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < C::kKLoads; ++i) kr[h][i] = load_codes16(base + (h * 8 + g) * D + i * 64);
        };
        auto load_v = [&](int key, int page) {
            const uint8_t *base = v.v_codes + (((int64_t)page * v.KH + head) * v.P + (key & (v.P - 1))) * D;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int tok = 2 * t + (j & 1) + (j >> 1) * 8;
                const bool live = key + tok < sw.q.kv;  // slots past the end hold anything
                if (D == 64) {
                    const uint2 x = load_codes8(base + tok * D + g * 8);
                    vr[j][0] = live ? x.x : 0u;
                    vr[j][1] = live ? x.y : 0u;
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        const uint4 x = load_codes16(base + tok * D + i * 128 + g * 16);
                        vr[j][4 * i] = live ? x.x : 0u;
                        vr[j][4 * i + 1] = live ? x.y : 0u;
                        vr[j][4 * i + 2] = live ? x.z : 0u;
                        vr[j][4 * i + 3] = live ? x.w : 0u;
                    }
                }
            }
        };
        int page = page_of(ks), page1 = page_of(ks + kStep);
        float sk = 1.f, sv = 1.f;
        if (ks < ke) {
            load_k(ks, page);
            load_v(ks, page);
            sk = __ldg(v.k_scale + (int64_t)page * v.KH + head);
            sv = __ldg(v.v_scale + (int64_t)page * v.KH + head);
        }
        for (; ks < ke; ks += kStep) {
            const int next = ks + kStep;
            const int page2 = page_of(next + kStep);
            // ------------------------------------------------------------ S = K q --
            float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i) {
                const uint32_t w0[4] = {kr[0][i].x, kr[0][i].y, kr[0][i].z, kr[0][i].w};
                const uint32_t w1[4] = {kr[1][i].x, kr[1][i].y, kr[1][i].z, kr[1][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a0, a1, a2, a3;
                    widen4(w0[j], a0, a2);
                    widen4(w1[j], a1, a3);
                    mma_f16(j & 1 ? s2 : s, a0, a1, a2, a3, qf[i][j][0], qf[i][j][1]);
                }
            }
            const float ev = (float)exponent_of(sv), inv_sv = 1.0f / sv;
            const float mk[2] = {mul[0] * sk, mul[1] * sk};
            if (next < ke) {
                load_k(next, page1);
                sk = __ldg(v.k_scale + (int64_t)page1 * v.KH + head);
                sv = __ldg(v.v_scale + (int64_t)page1 * v.KH + head);
            }
            // ------------------------------------------------------------- softmax --
            float z[4];  // keys g, g, g + 8, g + 8 of rows 2t, 2t + 1
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = fmaf(s[i] + s2[i], mk[i & 1], ev);
            if (ks < all_lo || ks + 16 > all_hi) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = ks + g + (i >> 1) * 8;
                    if (key < lo[i & 1] || key >= hi[i & 1]) z[i] = -INFINITY;
                }
            }
            // The reference m of a row moves only when a logit passes it by more than 2^8 (the
            // weights then stay below 256, well inside fp16); most steps change nothing.
            const bool up = fmaxf(z[0], z[2]) > m[0] + 8.f || fmaxf(z[1], z[3]) > m[1] + 8.f;
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(m[c], fmaxf(z[c], z[2 + c]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float f = mx == -INFINITY ? 1.f : exp2_fast(m[c] - mx);
                    m[c] = mx;
                    l[c] *= f;
#pragma unroll
                    for (int i = 0; i < kMT; ++i) {
                        o[i][c] *= f;
                        o[i][2 + c] *= f;
                    }
                }
            }
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = exp2_fast(z[i] - (m[i & 1] == -INFINITY ? 0.f : m[i & 1]));
            l[0] = fmaf(w[0] + w[2], inv_sv, l[0]);
            l[1] = fmaf(w[1] + w[3], inv_sv, l[1]);
            // -------------------------------------------------------- O += V^T w --
            // w as [key][row] pairs of rows; transposed into [row][key] pairs of keys
            const uint32_t b0 = transpose8(pack2<true>(w[0], w[1]));
            const uint32_t b1 = transpose8(pack2<true>(w[2], w[3]));
#pragma unroll
            for (int j = 0; j < C::kVRun / 4; ++j) {
                // four dims of keys 2t, 2t+1 (and 2t+8, 2t+9): pairs of keys a dim
                const uint32_t x = __byte_perm(vr[0][j], vr[1][j], 0x5140), y = __byte_perm(vr[0][j], vr[1][j], 0x7362);
                const uint32_t x8 = __byte_perm(vr[2][j], vr[3][j], 0x5140), y8 = __byte_perm(vr[2][j], vr[3][j], 0x7362);
                uint32_t a0, a1, a2, a3;
                widen4(x, a0, a1);
                widen4(x8, a2, a3);
                mma_f16(o[2 * j], a0, a1, a2, a3, b0, b1);
                widen4(y, a0, a1);
                widen4(y8, a2, a3);
                mma_f16(o[2 * j + 1], a0, a1, a2, a3, b0, b1);
            }
            if (next < ke) load_v(next, page1);
            page = page1;
            page1 = page2;
        }

        // ------------------------------------------------- join the block's four warps --
        // o[2j][0], o[2j][2], o[2j+1][0], o[2j+1][2] of thread (g, t): four dims of row 2t
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            if (g == 0) {
                merge_m[warp][2 * t + c] = m[c];
                merge_l[warp][2 * t + c] = l[c];
            }
#pragma unroll
            for (int j = 0; j < C::kVRun / 4; ++j) {
                const int dim = (D == 64) ? g * 8 + 4 * j : (j / 4) * 128 + g * 16 + (j % 4) * 4;
                *reinterpret_cast<float4 *>(&merge_o[warp][2 * t + c][dim]) =
                    make_float4(o[2 * j][c], o[2 * j][2 + c], o[2 * j + 1][c], o[2 * j + 1][2 + c]);
            }
        }
        __syncthreads();
        const bool whole = s0 == 0 && s1 == sw.steps;
        // a block has at most two unfinished segments: the one it begins inside, and its last
        float *slot = p.part + ((int64_t)blockIdx.x * 2 + (s0 > 0 ? 0 : 1)) * C::kPart;
        for (int i = tid; i < rows * D / 4; i += kThreads) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float top = merge_m[0][r];
            for (int k = 1; k < kWarps; ++k) top = fmaxf(top, merge_m[k][r]);
            const float ref = top == -INFINITY ? 0.f : top;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
            for (int k = 0; k < kWarps; ++k) {
                const float f = exp2_fast(merge_m[k][r] - ref);
                const float4 x = *reinterpret_cast<const float4 *>(&merge_o[k][r][d]);
                acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
                acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
                sum = fmaf(merge_l[k][r], f, sum);
            }
            if (whole) {
                const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
                const int64_t tok = sw.q.q0 + (row0 + r) / v.G;
                const int qh = head * v.G + (row0 + r) % v.G;
                *reinterpret_cast<uint2 *>(p.out + tok * p.out_ld + (int64_t)qh * D + d) =
                    make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
                if (p.lse && d == 0) p.lse[tok * v.QH + qh] = (top + log2f(sum)) * 0.6931471805599453f;
            } else {
                __stcg(reinterpret_cast<float4 *>(slot + r * D + d), acc);
                if (d == 0) {
                    __stcg(slot + kRows * D + r, top);
                    __stcg(slot + kRows * D + kRows + r, sum);
                }
            }
        }
        if (!whole) {
            // ------------------------------- the last block of the segment joins its parts --
            const int64_t c0 = seg_at / per, c1 = (seg_end - 1) / per;  // blocks that hold a part
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                // the segment's ticket: only one segment can begin inside block c0 and leave it
                const unsigned n = (unsigned)(c1 - c0 + 1);
                const unsigned got = atomicAdd(p.ticket + c0, 1u);
                last_flag = got + 1 == n;
                if (got + 1 == n) p.ticket[c0] = 0;
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                auto part = [&](int64_t c) {
                    const bool inside = seg_at < c * per;  // block c begins inside the segment
                    return p.part + (c * 2 + (inside ? 0 : 1)) * C::kPart;
                };
                for (int i = tid; i < rows * D / 4; i += kThreads) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4;
                    float top = -INFINITY;
                    for (int64_t c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(part(c) + kRows * D + r));
                    const float ref = top == -INFINITY ? 0.f : top;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float *x = part(c);
                        const float f = exp2_fast(__ldcg(x + kRows * D + r) - ref);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(x + r * D + d));
                        acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y);
                        acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
                        sum = fmaf(__ldcg(x + kRows * D + kRows + r), f, sum);
                    }
                    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
                    const int64_t tok = sw.q.q0 + (row0 + r) / v.G;
                    const int qh = head * v.G + (row0 + r) % v.G;
                    *reinterpret_cast<uint2 *>(p.out + tok * p.out_ld + (int64_t)qh * D + d) =
                        make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
                    if (p.lse && d == 0) p.lse[tok * v.QH + qh] = (top + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }
        __syncthreads();  // merge buffers are free again
    }
}

template <int D, bool F16>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_ATTN_SPLIT, s);
    int grid = device_info().sm_count * (D <= 128 ? 3 : 2);
    if (grid > kSplitMaxBlocks) grid = kSplitMaxBlocks;
    attn_split_kernel<D, F16><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t split_part_floats(int D) { return (size_t)kSplitMaxBlocks * 2 * (kRows * D + 2 * kRows); }

cudaError_t launch_attn_split(const AttnArgs &a, int D, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (D == 64) return f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (D == 128) return f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace moe
