// append.cu -- moe_kv_append: position rotation of q and k, and k and v written into the paged
// cache as E4M3 codes with one power-of-two scale a (page, kv head).
//
// One launch.  Its first blocks own one (page, kv head, k or v) each: such a block holds all of the
// page's new values of that head in registers, reduces their largest magnitude, settles the
// page's scale, re-rounds the codes that the page held before if the scale grew, and writes the
// new codes -- no other block touches that page and head, so no scale is ever contended.  The
// blocks after them rotate q: a thread takes the same 16 dims of two heads of a token, so that it reads
// their cosines and sines once.
//
// Bound: every value is read and written once (HBM) for prompts; a decode step is two or three
// dependent reads (sequence, page, values) and the launch.  Measured: one token of each of 48 sequences
// 5.7 us; 8192 tokens of 16 q and 2 kv heads 21.0 us (4.0 TB/s, of which the rotation of q, with its reads of
// the table, is the longer part; issue slots are 58% used, DRAM 27%: it is the latency of the warps that 64 registers
// leave room for); 11 sequences of up to 700 tokens, 24 and 8 heads of 64 dims, pages of 16, 11.1 us
// (23.9 with a block for each small page, 12.8 with q's heads one by one).
//
// Exact codes.  The rotation a cos - b sin of 16-bit a, b with an fp32 table is carried as an
// unevaluated fp32 pair (products and the sum with their rounding errors, error-free
// transformations after Dekker and Knuth) and rounded to odd: the low bit of the fp32 result is
// set when anything was lost.  Rounding that once more to 4 or 8 bits (or comparing it with a scale's
// border) then gives what the exact value would give, so codes and scales do not depend on how
// the rotation was summed.
#include "layer.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSeqCache = 1024;  // sequences whose places a block stages in shared memory

// a*c - b*s rounded to odd (see above); not finite, as the plain formula gives it (the errors of infinite products and
// sums are NaN).  Explicit _rn operations: none may be contracted.
__device__ __forceinline__ float rotate_odd(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), q = -__fmul_rn(b, s);
    const float ep = __fmaf_rn(a, c, -p), eq = __fmaf_rn(-b, s, -q);
    const float r = __fadd_rn(p, q);
    const float z = __fsub_rn(r, p);
    const float er = __fadd_rn(__fsub_rn(p, __fsub_rn(r, z)), __fsub_rn(q, z));
    const float err = __fadd_rn(er, __fadd_rn(ep, eq));
    const float r2 = __fadd_rn(r, err);
    const float lost = __fsub_rn(err, __fsub_rn(r2, r));
    int bits = __float_as_int(r2);
    if (lost != 0.f && !(bits & 1)) bits += ((lost > 0.f) == (r2 > 0.f)) ? 1 : -1;
    return fabsf(r) <= 3.402823466e38f ? __int_as_float(bits) : r;
}

// The same to nearest, and whether that is so near the middle between two 16-bit values that rounding it
// again might go wrong.  Its error is half an ulp for each of two additions (the products are exact), 1.5 ulp
// where the second leaves the binade, and the middle lies on the fp32 grid too: one ulp to either side.
// For q, where it costs 5 operations an element against 20 and the second look is rare.
template <bool F16>
__device__ __forceinline__ float2 rotate_near(float2 a, float2 c, float2 b, float2 minus_s, bool &near) {
    const float2 q = __fmul2_rn(b, minus_s);
    const float2 r = __fadd2_rn(__ffma2_rn(a, c, q), __ffma2_rn(b, minus_s, make_float2(-q.x, -q.y)));
    const uint32_t u = __float_as_uint(r.x), v = __float_as_uint(r.y);
    if (F16) {  // (subnormal results: coarser)
        near |= (((u + 1u) ^ 0x1000u) & 0x1ffcu) == 0u | (((v + 1u) ^ 0x1000u) & 0x1ffcu) == 0u;
        near |= fminf(fabsf(r.x), fabsf(r.y)) < 0x1p-13f;
    } else {
        near |= (((u + 1u) ^ 0x8000u) & 0xfffcu) == 0u | (((v + 1u) ^ 0x8000u) & 0xfffcu) == 0u;
    }
    return r;
}

// The exponent e of the smallest 2^e with amax <= 448 * 2^e (448 = 1.75 * 2^8), not below the floor.
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(fminf(amax, 3.402823466e38f));
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, kScaleMinExp);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    uint32_t lo, hi;
    widen4(w, lo, hi);
    const float2 a = unpack2<true>(lo), b = unpack2<true>(hi);
    return codes4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// A unit is 16 values of a row in two 8-value chunks that the rotation needs together: chunks
// (8u, 8u + rot/2) of half-split pairs, (16u, 16u + 8) of interleaved ones and of the dims past rot.
__device__ __forceinline__ void unit_dims(int u, int rot, bool interleaved, int &d0, int &d1) {
    const bool half_split = !interleaved && u < (rot >> 4);
    d0 = half_split ? 8 * u : 16 * u;
    d1 = half_split ? 8 * u + (rot >> 1) : 16 * u + 8;
}

// The 8 cosines and sines of unit u.  Rows of the table are rot floats, a multiple of 16: every 8 of them
// start on 16 bytes.
struct Angles {
    float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const float *rope_row, int u, int rot, Angles &g) {
    const float4 *cp = reinterpret_cast<const float4 *>(rope_row + 8 * u);
    const float4 *sp = reinterpret_cast<const float4 *>(rope_row + (rot >> 1) + 8 * u);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    g.c[0] = c0.x, g.c[1] = c0.y, g.c[2] = c0.z, g.c[3] = c0.w, g.c[4] = c1.x, g.c[5] = c1.y, g.c[6] = c1.z, g.c[7] = c1.w;
    g.s[0] = s0.x, g.s[1] = s0.y, g.s[2] = s0.z, g.s[3] = s0.w, g.s[4] = s1.x, g.s[5] = s1.y, g.s[6] = s1.z, g.s[7] = s1.w;
}

// Turns the unit's 8 pairs: (a[j], b[j]), or interleaved (a[2j], a[2j+1]) and (b[2j], b[2j+1]).  turn(x, c, y, s)
// is x c - y s.
template <typename F>
__device__ __forceinline__ void turn_unit(float (&a)[8], float (&b)[8], const Angles &g, bool interleaved, F turn) {
    if (!interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = a[j], y = b[j];
            a[j] = turn(x, g.c[j], y, g.s[j]);
            b[j] = turn(y, g.c[j], x, -g.s[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x = a[2 * j], y = a[2 * j + 1];
            a[2 * j] = turn(x, g.c[j], y, g.s[j]);
            a[2 * j + 1] = turn(y, g.c[j], x, -g.s[j]);
            x = b[2 * j], y = b[2 * j + 1];
            b[2 * j] = turn(x, g.c[4 + j], y, g.s[4 + j]);
            b[2 * j + 1] = turn(y, g.c[4 + j], x, -g.s[4 + j]);
        }
    }
}

// The last sequence b with f(b) <= i, f not descending, f(0) <= i.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int i, F f) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (f(mid) <= i) lo = mid; else hi = mid - 1;
    }
    return lo;
}

constexpr int kHeads = 2;  // heads a thread of the q part turns with one set of angles

// U: units a thread of a page block holds (P * D / 16 / blockDim)
template <int D, int U, bool F16>
__global__ void __launch_bounds__(kThreads, U <= 2 ? 4 : U == 4 ? 2 : 1) kv_append_kernel(const __grid_constant__ AppendArgs p) {
    constexpr int kUnits = D / 16;  // of a row
    const KvView &v = p.kv;
    __shared__ int starts[kSeqCache + 1], lens[kSeqCache];
    __shared__ float red[kThreads / 32];
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
    const int P = 1 << v.log_p;
    const bool staged = v.n_seqs <= kSeqCache;
    auto stage = [&]() {
        if (staged) {
            for (int i = tid; i <= v.n_seqs; i += nt) {
                starts[i] = v.q_start[i];
                if (i < v.n_seqs) lens[i] = v.kv_len[i];
            }
            __syncthreads();
        }
    };
    auto start_of = [&](int b) { return staged ? starts[b] : v.q_start[b]; };
    auto seq_of = [&](int b) { return staged ? checked_seq(v, starts[b], starts[b + 1], lens[b]) : load_seq(v, b); };

    // (Page blocks spread among the q blocks instead of before them: 25.1 against 21.2 us for an 8192-token prompt.)
    if ((int)blockIdx.x >= p.page_blocks) {
        // ---------------------------------------------------------------- rotation of q --
        const int t0 = ((int)blockIdx.x - p.page_blocks) * p.q_tokens;
        const int t1 = min(t0 + p.q_tokens, v.n_tokens);
        const int groups = (v.QH + kHeads - 1) / kHeads;
        const int u = tid % kUnits;
        int d0, d1;
        unit_dims(u, p.rot, p.interleaved, d0, d1);
        uint4 lo[kHeads], hi[kHeads];
        auto load = [&](int item) {
            const int tok = t0 + item / groups, h0 = item % groups * kHeads;
            const uint16_t *src = p.q + tok * p.q_ld + h0 * D;
#pragma unroll
            for (int i = 0; i < kHeads; ++i)
                if (h0 + i < v.QH) {
                    lo[i] = *reinterpret_cast<const uint4 *>(src + i * D + d0);
                    hi[i] = *reinterpret_cast<const uint4 *>(src + i * D + d1);
                }
        };
        const int first_item = tid / kUnits, items = (t1 - t0) * groups;
        if (first_item < items) load(first_item);  // under way while the sequences are read
        stage();
        for (int item = first_item; item < items; item += nt / kUnits) {
            const int tok = t0 + item / groups, h0 = item % groups * kHeads;
            if (item != first_item) load(item);
            const Seq q = seq_of(last_at_most(v.n_seqs, tok, start_of));
            const int pos = q.kv - q.n + tok - q.q0;
            const bool held = tok - q.q0 < q.n;  // else a row behind the last sequence's
            const bool ok = held && pos >= 0 && (pos < p.rope_rows || p.rot == 0);
            if (!ok && held && pos >= 0) layer_error(v.status);
            const bool turned = ok && u < (p.rot >> 4);
            Angles g;
            if (turned) load_angles(p.rope + (int64_t)pos * p.rot, u, p.rot, g);
            uint16_t *dst = p.q_out + tok * p.q_out_ld + h0 * D;
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                if (h0 + i >= v.QH) break;
                if (!ok) lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
                if (turned) {
                    float x[8], y[8];
                    unpack8<F16>(lo[i], x);
                    unpack8<F16>(hi[i], y);
                    bool near = false;
                    if (!p.interleaved) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const float2 c = make_float2(g.c[j], g.c[j + 1]), s = make_float2(g.s[j], g.s[j + 1]);
                            const float2 a = make_float2(x[j], x[j + 1]), b = make_float2(y[j], y[j + 1]);
                            const float2 a2 = rotate_near<F16>(a, c, b, make_float2(-s.x, -s.y), near);
                            const float2 b2 = rotate_near<F16>(b, c, a, s, near);
                            x[j] = a2.x, x[j + 1] = a2.y, y[j] = b2.x, y[j + 1] = b2.y;
                        }
                    } else {
                        auto pair = [&](float &a, float &b, float c, float s) {  // (a, b) (c, c) - (b, a) (s, -s)
                            const float2 r = rotate_near<F16>(make_float2(a, b), make_float2(c, c), make_float2(b, a), make_float2(-s, s), near);
                            a = r.x, b = r.y;
                        };
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            pair(x[2 * j], x[2 * j + 1], g.c[j], g.s[j]);
                            pair(y[2 * j], y[2 * j + 1], g.c[4 + j], g.s[4 + j]);
                        }
                    }
                    if (near) {
                        unpack8<F16>(lo[i], x);
                        unpack8<F16>(hi[i], y);
                        turn_unit(x, y, g, p.interleaved, rotate_odd);
                    }
                    lo[i] = pack8<F16>(x);
                    hi[i] = pack8<F16>(y);
                }
                *reinterpret_cast<uint4 *>(dst + i * D + d0) = lo[i];
                *reinterpret_cast<uint4 *>(dst + i * D + d1) = hi[i];
            }
        }
        return;
    }

    // ------------------------------------------------------------- one page of one head --
    // Pages of fewer than 256 units share a block: each takes the threads it needs.
    // Sequence b has the page slots base(b) .. base(b+1)-1: its n new tokens touch at most n/P + 2 pages.
    stage();
    const int team = min(P * kUnits, kThreads), item = (int)blockIdx.x * (kThreads / team) + tid / team;
    const int k0 = tid % team;  // the thread's first unit
    const bool any = item < p.page_items;
    const int slot = item / (2 * v.KH), which = item / v.KH & 1, head = item % v.KH;
    const int b = any ? last_at_most(v.n_seqs, slot, [&](int i) { return (start_of(i) >> v.log_p) + 2 * i; }) : 0;
    const Seq q = seq_of(b);
    const int first = q.kv - q.n;  // position of the first new token
    const int col = (max(first, 0) >> v.log_p) + slot - ((q.q0 >> v.log_p) + 2 * b);
    const int pos0 = col << v.log_p;
    // (col < 0: a descending q_start)
    bool here = any && col >= 0 && q.n > 0 && pos0 < q.kv;
    const int page = here ? v.table[(int64_t)b * v.max_pages + col] : 0;
    const uint16_t *src = which ? p.v : p.k;
    const int64_t ld = which ? p.v_ld : p.k_ld;
    const int rot = which ? 0 : p.rot;  // values are not rotated

    float x[U][8], y[U][8];
    float amax = 0.f;
    bool odd = false;
    uint4 lo[U], hi[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int k = i * team + k0, pos = pos0 + k / kUnits;
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        if (!here || pos < max(first, 0) || pos >= q.kv) continue;
        int d0, d1;
        unit_dims(k % kUnits, rot, p.interleaved, d0, d1);
        const uint16_t *row = src + (int64_t)(q.q0 + pos - first) * ld + head * D;
        lo[i] = *reinterpret_cast<const uint4 *>(row + d0);
        hi[i] = *reinterpret_cast<const uint4 *>(row + d1);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int k = i * team + k0, pos = pos0 + k / kUnits;
        const bool live = here && pos >= max(first, 0) && pos < q.kv;
        if (live && rot && pos >= p.rope_rows) {  // no angle: stored as zeros, reported
            odd = true;
            lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        }
        unpack8<F16>(lo[i], x[i]);
        unpack8<F16>(hi[i], y[i]);
        if (live && k % kUnits < (rot >> 4) && pos < p.rope_rows) {
            Angles g;
            load_angles(p.rope + (int64_t)pos * rot, k % kUnits, rot, g);
            turn_unit(x[i], y[i], g, p.interleaved, rotate_odd);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            odd |= !(fabsf(x[i][j]) <= 3.402823466e38f) || !(fabsf(y[i][j]) <= 3.402823466e38f);
            if (x[i][j] != x[i][j]) x[i][j] = 0.f;
            if (y[i][j] != y[i][j]) y[i][j] = 0.f;
            amax = fmaxf(amax, fmaxf(fabsf(x[i][j]), fabsf(y[i][j])));
        }
    }
    if (here && (page < 0 || page >= v.n_pages)) {
        odd = true;
        here = false;
    }
    if (odd) layer_error(v.status);
    const int64_t ph = (int64_t)(here ? page : 0) * v.KH + head;
    uint8_t *codes = (which ? v.v_codes : v.k_codes) + ph * P * D;
    float *scale = (which ? v.v_scale : v.k_scale) + ph;
    const bool begun = pos0 < first;  // the page holds earlier tokens
    const float old = here && begun ? *scale : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) red[tid >> 5] = amax;
    __syncthreads();
    if (!here) return;
    for (int w = 0; w < team >> 5; ++w) amax = fmaxf(amax, red[(tid - k0 >> 5) + w]);
    float s = pow2f(scale_exp(amax));
    if (begun) s = fmaxf(s, old);
    const float inv = 1.0f / s;  // exact: s is a power of two
    const bool grow = begun && s > old;
    const float ratio = old * inv;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int k = i * team + k0, pos = pos0 + k / kUnits;
        int d0, d1;
        unit_dims(k % kUnits, rot, p.interleaved, d0, d1);
        uint8_t *row = codes + k / kUnits * D;
        if (pos >= max(first, 0) && pos < q.kv) {
            uint2 a, c;
            a.x = codes4(x[i][0] * inv, x[i][1] * inv, x[i][2] * inv, x[i][3] * inv);
            a.y = codes4(x[i][4] * inv, x[i][5] * inv, x[i][6] * inv, x[i][7] * inv);
            c.x = codes4(y[i][0] * inv, y[i][1] * inv, y[i][2] * inv, y[i][3] * inv);
            c.y = codes4(y[i][4] * inv, y[i][5] * inv, y[i][6] * inv, y[i][7] * inv);
            *reinterpret_cast<uint2 *>(row + d0) = a;
            *reinterpret_cast<uint2 *>(row + d1) = c;
        } else if (grow) {
            uint2 a = *reinterpret_cast<const uint2 *>(row + d0), c = *reinterpret_cast<const uint2 *>(row + d1);
            a.x = rescale4(a.x, ratio), a.y = rescale4(a.y, ratio);
            c.x = rescale4(c.x, ratio), c.y = rescale4(c.y, ratio);
            *reinterpret_cast<uint2 *>(row + d0) = a;
            *reinterpret_cast<uint2 *>(row + d1) = c;
        }
    }
    if (k0 == 0 && s != old) *scale = s;
}

template <int D, bool F16>
cudaError_t launch(const AppendArgs &a, cudaStream_t s) {
    LaunchScope scope(KC_KV_APPEND, s);
    const int q_blocks = a.q ? (a.kv.n_tokens + a.q_tokens - 1) / a.q_tokens : 0;
    const int units = a.kv.P * D / 16;
    const int u = units / kThreads;
    AppendArgs b = a;
    b.page_blocks = u > 1 ? a.page_items : (a.page_items + kThreads / units - 1) / (kThreads / units);
    const int grid = b.page_blocks + q_blocks;
    if (u <= 1) kv_append_kernel<D, 1, F16><<<grid, kThreads, 0, s>>>(b);
    else if (u == 2) kv_append_kernel<D, 2, F16><<<grid, kThreads, 0, s>>>(b);
    else if (u == 4) kv_append_kernel<D, 4, F16><<<grid, kThreads, 0, s>>>(b);
    else kv_append_kernel<D, 8, F16><<<grid, kThreads, 0, s>>>(b);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, int D, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (D == 64) return f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (D == 128) return f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace moe
