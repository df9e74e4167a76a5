// attention.cu -- attention over the paged 8-bit cache, split along the keys: the form for single
// tokens and short query runs.
//
// Per row (token, q head): o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q.k_j), with k_j = 2^ek code
// and v_j = 2^ev code under the page's exponents.  In base 2 and with the value's scale drawn into
// the weight:  z_j = S_j 2^ek c + ev,  w_j = 2^(z_j - m),  o = sum_j w_j code_j / sum_j w_j 2^-ev:
// the products then run on the codes alone, which are exact in fp16, and pages of any scales mix.
//
// Bound: every code byte is read once and takes part in 2 x (rows of its head) products, so a
// decode step is bound by HBM.  Each warp streams its own keys, 16 at a time, through a ring of its
// own in shared memory (cp.async, no barrier between warps; 8 KB a warp in flight at D = 128, 128 KB
// an SM) into the register fragments of mma.sync.m16n8k16.  With keys (or value dims) on the 16-row
// side and 8 query rows on the 8-wide side no product is wasted for a group of 8 heads; the
// contraction index may be permuted freely, so a thread reads its fragments as 16-byte runs of a
// row, placed so that no two lanes meet on a bank.  (tcgen05 would need 128 rows on one side and
// the codes widened in shared memory first: with 8 rows a head the tensor cores are nearly idle
// either way.)
//
// Split: the batch's work is laid out as one line of 128-key steps (sequence by sequence, kv
// head by kv head, row tile by row tile, each with a fixed cost in front) and cut into equal runs, one
// a block, whatever the lengths.  A run that ends inside a segment leaves partial sums, which a second
// kernel joins in order.
//
// Measured, with the join: one token behind 1500 9.9 us, most of it five dependent reads and two
// launches; one behind 131,071, 32 q and 8 kv heads, 54 us (5.0 TB/s, 74% of the measured copy); 48 of very different
// length, up to 32,768, 36 us (4.0 TB/s); 8 runs of up to 4 tokens, D = 256, window 4096, 15 us.  About 10 us
// of each is the same start and end; between them the codes stream at 6 TB/s.
#include "layer.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
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
__device__ __forceinline__ int exponent_of(float s) { return (int)((__float_as_uint(s) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

// The keys that rows of tokens [t0, t1) (of a sequence's n) see at least one of: [lo, hi).
__device__ __forceinline__ void key_range(const AttnArgs &p, const Seq &q, int t0, int t1, int &lo, int &hi) {
    const int pos0 = q.kv - q.n + t0, pos1 = q.kv - q.n + t1 - 1;
    hi = p.causal ? min(q.kv, pos1 + 1) : q.kv;
    lo = p.window > 0 ? max(0, pos0 + 1 - p.window) : 0;
    if (hi < lo) hi = lo;
}

// Cost of a segment beside its steps (finding it, its queries, the first pages, the join), in steps: about
// 2.5 us against 0.5 us a step.
constexpr int kSegCost = 5;
constexpr int kSeqCache = 256;  // sequences kept in shared memory
constexpr float kMostWeight = 15.f;  // log2 of the largest weight under a row's reference: inside fp16

// A sequence's share of the line: tiles * kv heads segments of kSegCost + steps each.
struct SeqWork {
    Seq q;
    int tiles, step0, steps;
};
__device__ __forceinline__ SeqWork seq_work(const AttnArgs &p, const Seq &q, int rows_tile) {
    SeqWork w;
    w.q = q;
    if ((int64_t)w.q.n * p.kv.G >= p.prompt_rows) w.q.n = 0;  // the prompt kernel's
    w.tiles = (int)(((int64_t)w.q.n * p.kv.G + rows_tile - 1) / rows_tile);
    int lo, hi;
    key_range(p, w.q, 0, max(w.q.n, 1), lo, hi);
    w.step0 = lo / kStep;
    w.steps = max((hi + kStep - 1) / kStep - w.step0, 1);  // one at least: it writes the empty rows
    return w;
}
__device__ __forceinline__ int64_t line_length(const AttnArgs &p, const SeqWork &w) {
    return (int64_t)w.tiles * (w.steps + kSegCost) * p.kv.KH;
}

// NB: query row tiles of 8 that share a key tile.
template <int D, int NB>
struct Split {
    static constexpr int kRows = 8 * NB;
    static constexpr int kKLoads = D / 64;   // 16-byte runs of a key row a thread reads
    static constexpr int kVRun = D / 8;      // value dims a thread owns, of 4 keys
    static constexpr int kMT = D / 16;       // 16-dim output tiles
    static constexpr int kPart = kRows * D + 2 * kRows;  // floats of a partial result: sums, m, l
    static constexpr int kTile = 16 * D;     // bytes of 16 keys (or values)
    static constexpr int kRing = 3;          // tiles of K and V in a warp's ring
    static constexpr int kRingBytes = kWarps * kRing * 2 * kTile;
    static constexpr int kMergeBytes = kWarps * kRows * D * 4;  // over the ring, once it is drained
    static constexpr int kSmem = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;
    static constexpr int kBlocks = D * NB <= 128 ? 2 : 1;  // resident a SM
    static constexpr bool kQShared = NB > 1;               // query fragments in shared memory, not registers
    static constexpr int kGrid = kSplitMaxSms * kBlocks;   // blocks at most
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
// Where 16-byte chunk c of row r of a tile lies.  A key fragment is read by 8 lanes at 4 chunks of rows 2x and
// 2x + 1, a value fragment at 2 neighbouring chunks of rows 0, 2, 4, 6 (or 1, 3, 5, 7): both fall on all banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    if (D == 64) return (uint32_t)((r >> 1) * 128 + (((r ^ (r >> 2)) & 1) * 4 + (c ^ (r & 2))) * 16);
    return (uint32_t)(r * D + (c ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) * 16);
}

// Four dims of a row's output, and its lse.
template <int D, bool F16>
__device__ __forceinline__ void finish_row(const AttnArgs &p, int q0, int row, int head, int d, float4 acc, float top, float sum) {
    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
    const int64_t tok = q0 + row / p.kv.G;
    const int qh = head * p.kv.G + row % p.kv.G;
    *reinterpret_cast<uint2 *>(p.out + tok * p.out_ld + (int64_t)qh * D + d) =
        make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
    if (p.lse && d == 0) p.lse[tok * p.kv.QH + qh] = (top + log2f(sum)) * 0.6931471805599453f;
}

// Joins the parts of the segment whose first step block blockIdx.x of the split kernel had.  Its 16 warps
// share the rows evenly; the warps of a row take every n-th part and are added in order: the result is the
// same whatever block was done when.  (One block joining inside the split kernel, the last to arrive,
// took 25 us for the 76 parts of each head of a 131,071-key cache.)
template <int D, int NB, bool F16>
__global__ void __launch_bounds__(512) attn_join_kernel(const __grid_constant__ AttnArgs p) {
    using C = Split<D, NB>;
    constexpr int kPer = D / 32;  // dims a lane
    constexpr int kBatch = D <= 128 ? 16 : 8;  // parts whose loads are in flight together
    __shared__ float sums[16][D], tops[16], totals[16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const SplitDesc d = p.desc[blockIdx.x];
    if (d.parts <= 1) return;
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    int each = 16;  // warps a row, a power of two
    while (each > 1 && each * d.rows > 16) each >>= 1;
    const int w = warp % each;
    // part k: slot 1 of the first block (the segment begins there), slot 0 of the others
    const float *base = p.part + (int64_t)blockIdx.x * 2 * C::kPart;
    auto part = [&](int k) { return base + (int64_t)(2 * k + (k > 0 ? 0 : 1)) * C::kPart; };
    for (int r0 = 0; r0 < d.rows; r0 += 16 / each) {
        const int r = r0 + warp / each;
        const bool live = r < d.rows;
        float acc[kPer], sum = 0.f, top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
        for (int k0 = w; live && k0 < d.parts; k0 += kBatch * each) {
            float y[kBatch][kPer], m[kBatch], l[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int k = k0 + j * each;
                const bool in = k < d.parts;
                const float *x = part(in ? k : w);
                m[j] = in ? __ldcg(x + C::kRows * D + r) : -INFINITY;
                l[j] = __ldcg(x + C::kRows * D + C::kRows + r);
                if (kPer == 2) {
                    *reinterpret_cast<float2 *>(y[j]) = __ldcg(reinterpret_cast<const float2 *>(x + r * D + lane * kPer));
                } else {
#pragma unroll
                    for (int i = 0; i < kPer; i += 4)
                        *reinterpret_cast<float4 *>(y[j] + i) = __ldcg(reinterpret_cast<const float4 *>(x + r * D + lane * kPer + i));
                }
            }
            float to = top;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) to = fmaxf(to, m[j]);
            const float ref = to == -INFINITY ? 0.f : to, f = exp2_fast(top - ref);
            top = to;
            sum *= f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] *= f;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float e = exp2_fast(m[j] - ref);
                sum = fmaf(l[j], e, sum);
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc[i] = fmaf(y[j][i], e, acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) sums[warp][lane + 32 * i] = acc[i];
        if (lane == 0) tops[warp] = top, totals[warp] = sum;
        __syncthreads();
        if (live && w == 0) {
            for (int x = 1; x < each; ++x) top = fmaxf(top, tops[warp + x]);
            const float ref = top == -INFINITY ? 0.f : top;
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
            for (int x = 0; x < each; ++x) {
                const float e = exp2_fast(tops[warp + x] - ref);
                sum = fmaf(totals[warp + x], e, sum);
#pragma unroll
                for (int i = 0; i < kPer; ++i) acc[i] = fmaf(sums[warp + x][lane + 32 * i], e, acc[i]);
            }
            const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
            const int64_t tok = d.q0 + (d.row0 + r) / p.kv.G;
            const int qh = d.head * p.kv.G + (d.row0 + r) % p.kv.G;
            uint32_t *out = reinterpret_cast<uint32_t *>(p.out + tok * p.out_ld + (int64_t)qh * D + lane * kPer);
#pragma unroll
            for (int i = 0; i < kPer; i += 2) out[i / 2] = pack2<F16>(acc[i] * inv, acc[i + 1] * inv);
            if (p.lse && lane == 0) p.lse[tok * p.kv.QH + qh] = (top + log2f(sum)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

template <int D, int NB, bool F16>
__global__ void __launch_bounds__(kThreads, Split<D, NB>::kBlocks) attn_split_kernel(const __grid_constant__ AttnArgs p) {
    using C = Split<D, NB>;
    constexpr int kMT = C::kMT, kRows = C::kRows;
    const KvView &v = p.kv;
    extern __shared__ __align__(128) uint8_t ring[];
    float *merge_o = reinterpret_cast<float *>(ring);  // [kWarps][kRows][D], once the ring is drained
    __shared__ int64_t scan[kWarps];
    __shared__ int64_t found_at;
    __shared__ int found_b;
    __shared__ int seq_q0[kSeqCache], seq_n[kSeqCache], seq_kv[kSeqCache];
    __shared__ float merge_m[kWarps][kRows], merge_l[kWarps][kRows];
    __shared__ uint2 q_frag[C::kQShared ? NB * C::kKLoads * 4 * 32 : 1];  // [nb][run][k-step][lane]
    __shared__ int q_exps[C::kQShared ? kRows : 1];

    const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end by itself
    if (tid == 0) p.desc[blockIdx.x].parts = 0;

    // ------------------------------------------------- this block's run of the line --
    // its length, then the sequence that holds the run's first place
    int64_t total = 0, own0 = 0;
    for (int b = tid; b < v.n_seqs; b += kThreads) {
        const Seq q = load_seq(v, b);
        if (b < kSeqCache) seq_q0[b] = q.q0, seq_n[b] = q.n, seq_kv[b] = q.kv;
        const int64_t own = line_length(p, seq_work(p, q, kRows));
        if (b < kThreads) own0 = own;
        total += own;
    }
    auto seq_at = [&](int b) {
        Seq q;
        if (b < kSeqCache) q.q0 = seq_q0[b], q.n = seq_n[b], q.kv = seq_kv[b];
        else q = load_seq(v, b);
        return seq_work(p, q, kRows);
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) total += scan[w];
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    const int64_t begin = per * blockIdx.x, end = min(total, begin + per);
    if (begin >= end) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    int64_t before = 0;  // the line up to the sequences of this chunk
    for (int b0 = 0;; b0 += kThreads) {
        __syncthreads();
        const int b = b0 + tid;
        const int64_t own = b0 == 0 ? own0 : b < v.n_seqs ? line_length(p, seq_at(b)) : 0;
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
    int64_t seq_begin = found_at;  // where sequence b begins on the line
    SeqWork sw = seq_at(b);

    const uint32_t my_ring = (uint32_t)__cvta_generic_to_shared(ring) + warp * C::kRing * 2 * C::kTile;
    for (int64_t at = begin; at < end;) {
        while (at >= seq_begin + line_length(p, sw)) {
            seq_begin += line_length(p, sw);
            sw = seq_at(++b);
        }
        // ---------------------------------------------------------------- a segment --
        const int seg_len = sw.steps + kSegCost;
        const int64_t seg = (at - seq_begin) / seg_len;  // (head, tile) of the sequence
        const int64_t seg_at = seq_begin + seg * seg_len, seg_end = seg_at + seg_len;
        const int head = (int)(seg / sw.tiles), tile = (int)(seg % sw.tiles);
        const int s0 = max((int)(at - seg_at) - kSegCost, 0), s1 = max((int)(min(end, seg_end) - seg_at) - kSegCost, 0);
        at = min(end, seg_end);
        if (s1 <= s0) continue;  // only the cost in front lies in this run
        const int row0 = tile * kRows, rows = min(kRows, sw.q.n * v.G - row0);
        const int first_pos = sw.q.kv - sw.q.n;

        // tiles of 16 keys: tile n is keys [ks0 + n * kStep, + 16), from the first to the last that a row of this segment sees
        int klo, khi;
        key_range(p, sw.q, row0 / v.G, (row0 + rows - 1) / v.G + 1, klo, khi);
        const int32_t *table = v.table + (int64_t)b * v.max_pages;
        int ks0 = max((sw.step0 + s0) * kStep, klo / kStep * kStep) + warp * 16;
        if (ks0 + 16 <= klo) ks0 += kStep;  // 16 keys that no row sees are not looked up: their page may be gone
        const int ke = min((sw.step0 + s1) * kStep, khi);
        const int tiles = ks0 < ke ? (ke - ks0 + kStep - 1) / kStep : 0;
        // lane x holds page * KH + head and the scales of tile (a multiple of 32) + x, and of the 32 after
        auto page_at = [&](int n) {
            int page = 0;
            if (n < tiles) {
                page = __ldg(table + ((ks0 + n * kStep) >> v.log_p));
                if (page < 0 || page >= v.n_pages) {
                    layer_error(v.status);
                    page = 0;
                }
            }
            return page * v.KH + head;
        };
        int page = page_at(lane), page_next = 0;
        float sk = __ldg(v.k_scale + page), sv = __ldg(v.v_scale + page), sk_next = 1.f, sv_next = 1.f;
        // chunk i of a lane is chunk i * 32 + lane of the tile; rows 4 apart differ in bit 2 of the place
        const int cr = lane / (D / 16), cc = lane % (D / 16);
        uint32_t fill_at = my_ring;  // the ring place that is filled next
        auto fill = [&](int n) {     // tile n
            if (n < tiles) {
                const int pg = __shfl_sync(0xffffffffu, (n & 31) >= C::kRing - 1 || n < 32 ? page : page_next, n & 31);
                const int key = ks0 + n * kStep;
                const int64_t off = (((int64_t)pg << v.log_p) + (key & (v.P - 1))) * D + lane * 16;
                const uint8_t *ks = v.k_codes + off, *vs = v.v_codes + off;
                if (key + 16 <= sw.q.kv) {
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint32_t dst = fill_at + chunk_at<D>(i * (512 / D) + cr, cc);
                        copy16(dst, ks + i * 512);
                        copy16(dst + C::kTile, vs + i * 512);
                    }
                } else {  // slots past the end hold anything: zeros instead
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const int r = i * (512 / D) + cr;
                        copy16_or_zero(fill_at + chunk_at<D>(r, cc), ks + i * 512, key + r < sw.q.kv);
                        copy16_or_zero(fill_at + C::kTile + chunk_at<D>(r, cc), vs + i * 512, key + r < sw.q.kv);
                    }
                }
                fill_at = fill_at == my_ring + (C::kRing - 1) * 2 * C::kTile ? my_ring : fill_at + 2 * C::kTile;
            }
            copies_commit();
        };
#pragma unroll
        for (int n = 0; n < C::kRing - 1; ++n) fill(n);

        // q rows: fragment rows are n = g, dims i*64 + t*16 + 4s of the four k-steps of run i
        uint2 qf[C::kQShared ? 1 : C::kKLoads][4];
        float mul[NB][2];
        int lo[NB][2], hi[NB][2];  // the keys that rows 2t, 2t + 1 see
        int all_lo = 0, all_hi = 0x7fffffff;  // keys in [all_lo, all_hi) are seen by every row
        int q_exp = 0;
        // every warp makes the one tile's fragments, or warp nb those of row tile nb for all
        if (!C::kQShared || warp < NB) {
            const int nb = C::kQShared ? warp : 0;
            float amax = 0.f;
            uint4 qv[C::kKLoads][2];
            const int r = row0 + nb * 8 + g;
            const bool live = nb * 8 + g < rows;
            const uint16_t *row = p.q + (int64_t)(sw.q.q0 + r / v.G) * p.q_ld + (int64_t)(head * v.G + r % v.G) * D + t * 16;
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    qv[i][c] = live ? *reinterpret_cast<const uint4 *>(row + i * 64 + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[8];
                    unpack8<F16>(qv[i][c], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // largest magnitude into [1, 2): fp16 then holds every bf16 digit down to 2^-17 of it
            q_exp = amax > 0.f ? max(min((int)(__float_as_uint(amax) >> 23) - 127, 126), -126) : 0;
            const float inv = pow2f(-q_exp);
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[8];
                    unpack8<F16>(qv[i][c], x);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint2 f = make_uint2(pack2<true>(x[4 * j] * inv, x[4 * j + 1] * inv),
                                                   pack2<true>(x[4 * j + 2] * inv, x[4 * j + 3] * inv));
                        if (C::kQShared) q_frag[((nb * C::kKLoads + i) * 4 + 2 * c + j) * 32 + lane] = f;
                        else qf[i][2 * c + j] = f;
                    }
                }
            if (C::kQShared && t == 0) q_exps[nb * 8 + g] = q_exp;
        }
        if (C::kQShared) __syncthreads();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int rr = nb * 8 + 2 * t + c, pos = first_pos + (row0 + rr) / v.G;
                mul[nb][c] = p.scale_log2 * pow2f(C::kQShared ? q_exps[rr] : __shfl_sync(0xffffffffu, q_exp, (2 * t + c) * 4));
                hi[nb][c] = p.causal ? min(sw.q.kv, pos + 1) : sw.q.kv;
                lo[nb][c] = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
                if (rr < rows) {
                    all_lo = max(all_lo, lo[nb][c]);
                    all_hi = min(all_hi, hi[nb][c]);
                }
            }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
            all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
        }

        float m[NB][2], l[NB][2], o[NB][kMT][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int i = 0; i < kMT; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
        }
        uint32_t read_at = my_ring;
        for (int n = 0; n < tiles; ++n) {
            copies_wait<C::kRing - 2>();
            __syncwarp();  // tile n is there for all lanes, and all are done with the tile before it
            if ((n & 31) == 0 && n + 32 < tiles) page_next = page_at(n + 32 + lane);
            if ((n & 31) == 16 && n + 16 < tiles) sk_next = __ldg(v.k_scale + page_next), sv_next = __ldg(v.v_scale + page_next);
            fill(n + C::kRing - 1);
            const uint32_t kt = read_at, vt = kt + C::kTile;
            read_at = read_at == my_ring + (C::kRing - 1) * 2 * C::kTile ? my_ring : read_at + 2 * C::kTile;
            const float tsk = __shfl_sync(0xffffffffu, sk, n & 31), tsv = __shfl_sync(0xffffffffu, sv, n & 31);
            const int key0 = ks0 + n * kStep;
            // ------------------------------------------------------------ S = K q --
            float s[NB][4], s2[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[nb][i] = s2[nb][i] = 0.f;
#pragma unroll
            for (int i = 0; i < C::kKLoads; ++i) {
                const uint4 x0 = lds16(kt + chunk_at<D>(g, 4 * i + t)), x1 = lds16(kt + chunk_at<D>(8 + g, 4 * i + t));
                const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t a0, a1, a2, a3;
                    widen4(w0[j], a0, a2);
                    widen4(w1[j], a1, a3);
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint2 f = C::kQShared ? q_frag[((nb * C::kKLoads + i) * 4 + j) * 32 + lane] : qf[C::kQShared ? 0 : i][j];
                        mma_f16(j & 1 ? s2[nb] : s[nb], a0, a1, a2, a3, f.x, f.y);
                    }
                }
            }
            // ------------------------------------------------------------- softmax --
            const float ev = (float)exponent_of(tsv), inv_sv = pow2f(-exponent_of(tsv));
            float z[NB][4];  // keys g, g, g + 8, g + 8 of rows 2t, 2t + 1
            bool up = false;
            const bool masked = key0 < all_lo || key0 + 16 > all_hi;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[nb][i] = fmaf(s[nb][i] + s2[nb][i], mul[nb][i & 1] * tsk, ev);
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + g + (i >> 1) * 8;
                        if (key < lo[nb][i & 1] || key >= hi[nb][i & 1]) z[nb][i] = -INFINITY;
                    }
                }
                up |= fmaxf(z[nb][0], z[nb][2]) > m[nb][0] + kMostWeight || fmaxf(z[nb][1], z[nb][3]) > m[nb][1] + kMostWeight;
            }
            // The reference m of a row moves only when a weight would pass 2^15, 2^6 above the largest that it
            // was set by; most steps change nothing.
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(m[nb][c], fmaxf(z[nb][c], z[nb][2 + c]) - kBelowTop);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                        const float f = mx == -INFINITY ? 1.f : exp2_fast(m[nb][c] - mx);
                        m[nb][c] = mx;
                        l[nb][c] *= f;
#pragma unroll
                        for (int i = 0; i < kMT; ++i) {
                            o[nb][i][c] *= f;
                            o[nb][i][2 + c] *= f;
                        }
                    }
            }
            uint32_t b0[NB], b1[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = exp2_fast(z[nb][i] - (m[nb][i & 1] == -INFINITY ? 0.f : m[nb][i & 1]));
                l[nb][0] = fmaf(w[0] + w[2], inv_sv, l[nb][0]);
                l[nb][1] = fmaf(w[1] + w[3], inv_sv, l[nb][1]);
                // w as [key][row] pairs of rows; transposed into [row][key] pairs of keys
                b0[nb] = transpose8(pack2<true>(w[0], w[1]));
                b1[nb] = transpose8(pack2<true>(w[2], w[3]));
            }
            // -------------------------------------------------------- O += V^T w --
            uint32_t vr[4][C::kVRun / 4];  // the thread's dims of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 2 * t + (j & 1) + (j >> 1) * 8;
                if (D == 64) {
                    const uint2 x = lds8(vt + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
                    vr[j][0] = x.x, vr[j][1] = x.y;
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        const uint4 x = lds16(vt + chunk_at<D>(r, i * 8 + g));
                        vr[j][4 * i] = x.x, vr[j][4 * i + 1] = x.y, vr[j][4 * i + 2] = x.z, vr[j][4 * i + 3] = x.w;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < C::kVRun / 4; ++j) {
                // four dims of keys 2t, 2t+1 (and 2t+8, 2t+9): pairs of keys a dim
                const uint32_t x = __byte_perm(vr[0][j], vr[1][j], 0x5140), y = __byte_perm(vr[0][j], vr[1][j], 0x7362);
                const uint32_t x8 = __byte_perm(vr[2][j], vr[3][j], 0x5140), y8 = __byte_perm(vr[2][j], vr[3][j], 0x7362);
                uint32_t a0, a1, a2, a3;
                widen4(x, a0, a1);
                widen4(x8, a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][2 * j], a0, a1, a2, a3, b0[nb], b1[nb]);
                widen4(y, a0, a1);
                widen4(y8, a2, a3);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][2 * j + 1], a0, a1, a2, a3, b0[nb], b1[nb]);
            }
            if ((n & 31) == 31) page = page_next, sk = sk_next, sv = sv_next;
        }

        // ------------------------------------------------ join the block's eight warps --
        copies_wait<0>();
        __syncthreads();  // every ring is drained
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = nb * 8 + 2 * t + c;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nb][c] += __shfl_xor_sync(0xffffffffu, l[nb][c], d);
                if (g == 0) {
                    merge_m[warp][r] = m[nb][c];
                    merge_l[warp][r] = l[nb][c];
                }
#pragma unroll
                for (int j = 0; j < C::kVRun / 4; ++j) {
                    // o[2j][c], o[2j][2+c], o[2j+1][c], o[2j+1][2+c] of thread (g, t): four dims of row 2t + c
                    const int dim = (D == 64) ? g * 8 + 4 * j : (j / 4) * 128 + g * 16 + (j % 4) * 4;
                    *reinterpret_cast<float4 *>(merge_o + (warp * kRows + r) * D + dim) =
                        make_float4(o[nb][2 * j][c], o[nb][2 * j][2 + c], o[nb][2 * j + 1][c], o[nb][2 * j + 1][2 + c]);
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
                const float4 x = *reinterpret_cast<const float4 *>(merge_o + (k * kRows + r) * D + d);
                acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
                acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
                sum = fmaf(merge_l[k][r], f, sum);
            }
            if (whole) {
                finish_row<D, F16>(p, sw.q.q0, row0 + r, head, d, acc, top, sum);
            } else {
                __stcg(reinterpret_cast<float4 *>(slot + r * D + d), acc);
                if (d == 0) {
                    __stcg(slot + kRows * D + r, top);
                    __stcg(slot + kRows * D + kRows + r, sum);
                }
            }
        }
        // the block with the segment's first step tells the join where its parts are
        if (!whole && s0 == 0 && tid == 0)
            p.desc[blockIdx.x] = SplitDesc{(int)((seg_end - 1) / per - blockIdx.x + 1), rows, sw.q.q0, row0, head};
        __syncthreads();  // merge buffers are free again
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the prompt kernel's end: what follows this grid follows both
}

template <int D, int NB, bool F16>
cudaError_t launch(const AttnArgs &a, bool after_prompt, cudaStream_t s) {
    using C = Split<D, NB>;
    cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<D, NB, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const int sms = device_info().sm_count < kSplitMaxSms ? device_info().sm_count : kSplitMaxSms;
    const int grid = sms * C::kBlocks;
    // Each launch may begin before the one before it ends: the split kernel beside the last blocks of the
    // prompt kernel, which it does not read and whose end it awaits at its own; the join while the split
    // kernel drains.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = after_prompt ? 1 : 0;
    {
        LaunchScope scope(KC_ATTN_SPLIT, s);
        e = cudaLaunchKernelEx(&cfg, attn_split_kernel<D, NB, F16>, a);
        if (e != cudaSuccess) return e;
    }
    LaunchScope scope(KC_ATTN_JOIN, s);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, NB, F16>, a);
}

}  // namespace

size_t split_part_floats(int D) {
    auto most = [](size_t a, size_t b) { return a > b ? a : b; };
    if (D == 64) return most(Split<64, 1>::kGrid * 2 * Split<64, 1>::kPart, Split<64, 4>::kGrid * 2 * Split<64, 4>::kPart);
    if (D == 128) return most(Split<128, 1>::kGrid * 2 * Split<128, 1>::kPart, Split<128, 4>::kGrid * 2 * Split<128, 4>::kPart);
    return most(Split<256, 1>::kGrid * 2 * Split<256, 1>::kPart, Split<256, 2>::kGrid * 2 * Split<256, 2>::kPart);
}

template <int D, int NB>
cudaError_t by_dtype(const AttnArgs &a, int dtype, bool after_prompt, cudaStream_t s) {
    return dtype == MOE_DTYPE_F16 ? launch<D, NB, true>(a, after_prompt, s) : launch<D, NB, false>(a, after_prompt, s);
}

// shared: 4 row tiles (2 at D = 256) share each key tile that is read and widened.
// after_prompt: the launch just before, on the same stream, is the same call's prompt kernel.
cudaError_t launch_attn_split(const AttnArgs &a, int D, int dtype, bool shared, bool after_prompt, cudaStream_t s) {
    if (D == 64) return shared ? by_dtype<64, 4>(a, dtype, after_prompt, s) : by_dtype<64, 1>(a, dtype, after_prompt, s);
    if (D == 128) return shared ? by_dtype<128, 4>(a, dtype, after_prompt, s) : by_dtype<128, 1>(a, dtype, after_prompt, s);
    return shared ? by_dtype<256, 2>(a, dtype, after_prompt, s) : by_dtype<256, 1>(a, dtype, after_prompt, s);
}

}  // namespace moe
