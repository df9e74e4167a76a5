// linear_prompt.cu -- moe_linear_attention for runs of many tokens, chunk by chunk on the 5th-generation tensor cores.
//
// A chunk of 64 tokens, G the sums of its log decays from its begin, S0 the state there:
//   o_i = scale (e^{G_i} S0^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S   = e^{G_64} S0 + sum_j e^{G_64 - G_j} k_j v_j^T
// All exponents are at most 0.  Four products a chunk, with the value channels on the rows (lanes) of three of them, so
// that a thread holds a channel's row of the state in fp32 registers from the first chunk to the last:
//   A = Q K^T (tokens x tokens), U^T = (w V)^T K (channels x DK), O1^T = S0^T Q^T, O2^T = V^T P^T (channels x tokens),
// P = A weighted and masked.  The tensor cores take 16-bit operands, so what is rounded for them is split: P and S0
// into two parts, the weighted values into three in bf16 and two in fp16 (a state's error stays below
// that of its fp32 sums).  With fp16, whose range is short, each row of P, each channel of S0 and each chunk's weighted
// values are scaled by a power of two.
//
// A block walks one value head's chunks (128 value channels at most) in order.  The state is what makes it wait: U(c) ->
// registers -> S0(c+1) in TMEM; everything else runs ahead.  Where heads and sequences leave SMs idle, a
// run's chunks are cut into segments: a first kernel computes what each segment adds to the state (K and V only),
// and each segment's block begins with the sum of those before it.
//
// Roles (16 warps): 0-3 the state; 4-7 the output; 8-11 weighted values; 12, 13 P (a row a thread); 14 copies (TMA)
// and decays; 15 the MMAs.
#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kOutWarp = 4, kValueWarp = 8, kWeightWarp = 12, kLoadWarp = 14, kMmaWarp = 15;
// Registers a thread: 128 at launch; of a scheduler's 4 x 128 the state's warp, which holds 128 of them, takes 200.
constexpr int kStateRegs = 200, kOutRegs = 104, kValueRegs = 96, kOtherRegs = 112;
static_assert(kStateRegs + kOutRegs + kValueRegs + kOtherRegs <= 512, "more registers than the block has");
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far above any legitimate wait
constexpr int kBlockBytes = kChunk * 128;    // 64 tokens x 64 channels
constexpr int kSlots = 4;                    // chunks whose decays are in shared memory

// What the warps tell one another of a chunk.
struct alignas(16) Slot {
    float g_hi[kChunk], g_lo[kChunk];  // log2 of the decay from the chunk's begin, in two parts
    float weight[kChunk];              // e^{G_64 - G_j}
    float fade[kChunk];                // e^{G_i}
    float p_unit[kChunk];              // fp16: P's rows hold 1 / p_unit of their values
    float s_unit[128];                 // fp16: and S0's channels
    int bad[128];                      // first token whose value is not finite, of each channel
    float whole;                       // e^{G_64}
    float u_unit;                      // fp16: U holds 1 / u_unit of its values
    int any_bad;
};

template <int DK, int DV, bool F16>
struct Shape {
    static constexpr int kKBlocks = DK / 64, kVBlocks = DV / 64;
    static constexpr int kQ = 0, kK = kKBlocks * kBlockBytes, kV = 2 * kK;  // offsets in a stage
    static constexpr int kStageBytes = kV + kVBlocks * kBlockBytes;
    static constexpr int kStages = 3;
    static constexpr int kParts = F16 ? 2 : 3;  // of a weighted value
    static constexpr int kPartBytes = kVBlocks * kBlockBytes;
    static constexpr int kValues = kStages * kStageBytes, kP = kValues + kParts * kPartBytes;
    static constexpr int kBars = kP + 2 * kBlockBytes, kSlotAt = kBars + 256;
    static constexpr int kSmem = 1024 + kSlotAt + kSlots * (int)sizeof(Slot);
    static constexpr int kLaneWarps = DV / 32;  // warps that hold channels
    // TMEM columns: S0 in two parts, U, A, O1, O2
    static constexpr uint32_t kColS = 0, kColU = DK, kColA = 2 * DK, kColO1 = kColA + 64, kColO2 = kColO1 + 64, kCols = 512;
    static_assert(kColO2 + 64 <= kCols, "TMEM");
    static_assert(kSmem <= 227 * 1024, "shared memory over the per-block limit");
    // (operands of 128 rows whose second half is none of theirs read up to a block further; it is never looked at)
    static_assert(kP + 2 * kBlockBytes <= kSmem - 1024, "operands end in shared memory");
};

struct Maps {
    CUtensorMap q, k, v;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }
// The power of two that brings `largest` (finite or not, >= 0) near 2^14, within fp16's range.
__device__ __forceinline__ int lift(float largest) {
    const int e = (int)(__float_as_uint(largest) >> 23) - 127;
    return largest > 0.f ? min(max(14 - e, -126), 126) : 0;
}
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k]));
}
// (a, b) = hi + lo, both of the 16-bit type.
template <bool F16>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2<F16>(a, b);
    const float2 h = unpack2<F16>(hi);
    lo = pack2<F16>(a - h.x, b - h.y);
}

// Where sequence b's segments lie among the batch's.
__device__ __forceinline__ int segment_base(const LinearArgs &p, int b) { return p.q_start[b] / (p.segment_chunks * kChunk) + b; }

// STATES: what each segment but a run's last adds to the state, and its decay; otherwise the outputs.
template <int DK, int DV, bool F16, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ LinearArgs p, const __grid_constant__ Maps maps) {
    using C = Shape<DK, DV, F16>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBars);  // [kStages] Q, K, V of a chunk
    uint64_t *empty = full + kStages;                                // [kStages]
    uint64_t *g_full = empty + kStages, *g_empty = g_full + kSlots;  // [kSlots] decays
    uint64_t *a_full = g_empty + kSlots, *a_free = a_full + 1;       // A in TMEM; read
    uint64_t *p_full = a_free + 1;                                   // P in shared memory
    uint64_t *v_full = p_full + 1;                                   // weighted values there
    uint64_t *u_full = v_full + 1, *u_free = u_full + 1;             // U in TMEM (and the values read); read
    uint64_t *s_full = u_free + 1, *s_free = s_full + 1;             // S0 in TMEM; read by its product
    uint64_t *o_full = s_free + 1, *o_free = o_full + 1;             // O1 and O2 in TMEM (and P read); read
    uint64_t *m_full = o_free + 1;                                   // fp16: the warps' largest weighted values
    uint64_t *drain = m_full + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    float *most = reinterpret_cast<float *>(tmem_holder + 2);  // [2 x 4] those, of even and odd chunks
    Slot *slots = reinterpret_cast<Slot *>(smem + C::kSlotAt);

    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

    // ------------------------------------------------------------------- the block's chunks --
    const int tiles = p.DV / DV;
    const int tile = (int)blockIdx.x % tiles, head = (int)blockIdx.x / tiles % p.VH, place = (int)blockIdx.x / tiles / p.VH;
    int b;
    {
        int lo = 0, hi = p.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (segment_base(p, mid) <= place) lo = mid; else hi = mid - 1;
        }
        b = lo;
    }
    const Run run = load_run(p, b);
    // (where there is no other kernel, chunk_tokens is 0: a run of padding alone is this one's too)
    if (run.n < p.chunk_tokens) return;
    const int all = (run.n + kChunk - 1) / kChunk, base = segment_base(p, b), seg = place - base;
    const int segs = (all + p.segment_chunks - 1) / p.segment_chunks;
    const int kh = head / p.G, col0 = head * p.DV + tile * DV;  // the block's columns of v and out
    if (!STATES && seg == 0)
        for (int i = tid; i < run.pad * (DV / 2); i += kThreads)
            *reinterpret_cast<uint32_t *>(p.out + (int64_t)(run.q0 - run.pad + i / (DV / 2)) * p.out_ld + col0 + i % (DV / 2) * 2) = 0;
    if (seg < 0 || seg >= segs - (STATES ? 1 : 0)) return;
    const int chunk0 = seg * p.segment_chunks, chunks = min(p.segment_chunks, all - chunk0);
    const int64_t row0 = run.q0 + (int64_t)chunk0 * kChunk;
    const int rows = min(run.n - chunk0 * kChunk, chunks * kChunk);  // tokens

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s], 1), ptx::mbar_init(&empty[s], 1);
        for (int s = 0; s < kSlots; ++s) {
            ptx::mbar_init(&g_full[s], 1);
            ptx::mbar_init(&g_empty[s], 4 + C::kLaneWarps + (STATES ? 0 : 2 + C::kLaneWarps));
        }
        ptx::mbar_init(a_full, 1), ptx::mbar_init(a_free, 2);
        ptx::mbar_init(p_full, 2);
        ptx::mbar_init(v_full, 4);
        // (u_full and o_full: the MMAs' end, and the arrival of the warp that has seen the units of their operands)
        ptx::mbar_init(m_full, 4);
        ptx::mbar_init(u_full, 2), ptx::mbar_init(u_free, C::kLaneWarps);
        ptx::mbar_init(s_full, C::kLaneWarps), ptx::mbar_init(s_free, 1);
        ptx::mbar_init(o_full, 2), ptx::mbar_init(o_free, C::kLaneWarps);
        ptx::mbar_init(drain, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) ptx::tmem_alloc(tmem_holder, C::kCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    auto wait = [&](uint64_t *bar, int phase) {  // of the whole warp
        return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase & 1, kWaitNs, abort_flag)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar);
    };
    bool ok = true;
    int issued = 0;  // chunks whose copies were begun

    if (warp < kOutWarp) {
        ptx::regs_up<kStateRegs>();
        if (warp < C::kLaneWarps) {
            // ------------------------------------------------------------------ the state --
            // Thread t has channel t: S[d] of all key channels d.
            const int64_t state_size = (int64_t)DK * p.DV;
            float *own = p.states + ((int64_t)max(run.slot, 0) * p.VH + head) * state_size + tile * DV + tid;
            auto place_at = [&](int i) {  // of segment i of this run
                return p.seg_states + ((int64_t)(base + i) * p.VH + head) * state_size + tile * DV + tid;
            };
            float S[DK];
#pragma unroll
            for (int d = 0; d < DK; ++d) S[d] = 0.f;
            if (seg == 0) {
                // with several segments, whose last writes the slot, the others find the slot's state at the last one's place
                const float *src = !STATES && segs > 1 ? place_at(segs - 1) : own;
                if (!run.fresh) {
#pragma unroll
                    for (int d = 0; d < DK; ++d) S[d] = src[(int64_t)d * p.DV];
                }
                if (STATES && !run.fresh) {
                    float *dst = place_at(segs - 1);
#pragma unroll
                    for (int d = 0; d < DK; ++d) dst[(int64_t)d * p.DV] = S[d];
                }
            } else if (!STATES) {
                for (int i = 0; i < seg; ++i) {
                    const float *src = place_at(i), f = p.seg_decay[(int64_t)(base + i) * p.VH + head];
#pragma unroll
                    for (int d = 0; d < DK; ++d) S[d] = fmaf(S[d], i == 0 ? 0.f : f, src[(int64_t)d * p.DV]);
                }
            }
            const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
            auto publish = [&](int c) {  // S0 of chunk c, in two parts
                float f = 1.f;
                if (F16) {
                    float m = 0.f;
#pragma unroll
                    for (int d = 0; d < DK; ++d) m = fmaxf(m, fabsf(S[d]));
                    const int e = lift(m);
                    f = pow2f(e);
                    slots[c % kSlots].s_unit[tid] = pow2f(-e);
                }
#pragma unroll
                for (int g = 0; g < DK / 32; ++g) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int d = 0; d < 16; ++d) split2<F16>(S[g * 32 + 2 * d] * f, S[g * 32 + 2 * d + 1] * f, hi[d], lo[d]);
                    ptx::tmem_st_16(lanes + C::kColS + g * 16, hi);
                    ptx::tmem_st_16(lanes + C::kColS + DK / 2 + g * 16, lo);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                arrive(s_full);
            };
            if (!STATES) {
                ok = wait(&g_full[0], 0);
                if (ok) publish(0);
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const Slot &sl = slots[c % kSlots];
                if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(u_full, c))) break;
                ptx::tc_fence_after();
                const float f = sl.whole, unit = F16 ? sl.u_unit : 1.f;
#pragma unroll
                for (int g = 0; g < DK / 32; ++g) {
                    uint32_t u[32];
                    ptx::tmem_ld_32(lanes + C::kColU + g * 32, u);
                    ptx::tmem_ld_wait();
                    tie32(u);
#pragma unroll
                    for (int d = 0; d < 32; ++d) {
                        const float x = F16 ? __uint_as_float(u[d]) * unit : __uint_as_float(u[d]);
                        S[g * 32 + d] = fmaf(S[g * 32 + d], f, x);
                    }
                }
                ptx::tc_fence_before();
                arrive(u_free);
                arrive(&g_empty[c % kSlots]);
                if (!STATES && c + 1 < chunks) {
                    if (!(ok = wait(s_free, c) && wait(&g_full[(c + 1) % kSlots], (c + 1) / kSlots))) break;
                    ptx::tc_fence_after();
                    publish(c + 1);
                }
            }
            if (ok && STATES) {
                float *dst = place_at(seg);
#pragma unroll
                for (int d = 0; d < DK; ++d) dst[(int64_t)d * p.DV] = S[d];
            } else if (ok && seg == segs - 1 && run.slot >= 0) {
#pragma unroll
                for (int d = 0; d < DK; ++d) own[(int64_t)d * p.DV] = S[d];
            }
        }
    } else if (warp < kValueWarp) {
        ptx::regs_down<kOutRegs>();
        if (!STATES && warp - kOutWarp < C::kLaneWarps) {
            // ------------------------------------------------------------------ the output --
            const int ch = (warp - kOutWarp) * 32 + lane;
            const uint32_t lanes = tmem + ((uint32_t)((warp - kOutWarp) * 32) << 16);
            for (int c = 0; c < chunks && ok; ++c) {
                const Slot &sl = slots[c % kSlots];
                if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(o_full, c))) break;
                ptx::tc_fence_after();
                const int valid = min(rows - c * kChunk, kChunk);
                const float f = p.scale * (F16 ? sl.s_unit[ch] : 1.f);
                const int bad = sl.any_bad ? sl.bad[ch] : kChunk;
                uint16_t *dst = p.out + (row0 + (int64_t)c * kChunk) * p.out_ld + col0 + ch;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    uint32_t a[32], x[32];
                    ptx::tmem_ld_32(lanes + C::kColO1 + g * 32, a);
                    ptx::tmem_ld_32(lanes + C::kColO2 + g * 32, x);
                    ptx::tmem_ld_wait();
                    tie32(a);
                    tie32(x);
                    if (g == 1) {
                        ptx::tc_fence_before();
                        arrive(o_free);
                    }
#pragma unroll
                    for (int t = 0; t < 32; ++t) {
                        const int i = g * 32 + t;
                        float o = __uint_as_float(a[t]) * (f * sl.fade[i]);
                        o = fmaf(__uint_as_float(x[t]), F16 ? p.scale * sl.p_unit[i] : p.scale, o);
                        if (i >= bad) o = __int_as_float(0x7fffffff);
                        if (i < valid) dst[(int64_t)i * p.out_ld] = (uint16_t)pack2<F16>(o, 0.f);
                    }
                }
                arrive(&g_empty[c % kSlots]);
            }
        }
    } else if (warp < kWeightWarp) {
        ptx::regs_down<kValueRegs>();
        // ------------------------------------------------------------- weighted values --
        // Thread t has 16-byte pieces t, t + 128, ... of the tile as it lies in shared memory (swizzled): of rows t / 8 + 16 i
        // of each block.  What comes out lies in the same places.
        const int t = tid - kValueWarp * 32, r0 = t >> 3;
        constexpr int kPieces = C::kVBlocks * 4;
        const int ch0 = ((t & 7) ^ (r0 & 7)) * 8;  // its channels in each block (rows differ by multiples of 8)
        for (int c = 0; c < chunks && ok; ++c) {
            Slot &sl = slots[c % kSlots];
            uint8_t *stage = smem + c % kStages * C::kStageBytes;
            if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(&full[c % kStages], c / kStages))) break;
            const int valid = min(rows - c * kChunk, kChunk);
            float x[kPieces][8], sum = 0.f, m = 0.f;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int row = r0 + (i & 3) * 16;
                uint4 *src = reinterpret_cast<uint4 *>(stage + C::kV + t * 16 + i * 2048);
                uint4 w = *src;
                if (row >= valid) {  // behind the run's end, where whatever comes there lies: the products must not see it
                    w = make_uint4(0, 0, 0, 0);
                    *src = w;
                }
                const float f = sl.weight[row];
                unpack8<F16>(w, x[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum = fmaf(x[i][j], 0.f, sum);
                    x[i][j] *= f;
                    if (F16) m = fmaxf(m, fabsf(x[i][j]));
                }
            }
            if (valid < kChunk) {
#pragma unroll
                for (int i = 0; i < C::kKBlocks * 4; ++i)
                    if (r0 + (i & 3) * 16 >= valid)
                        *reinterpret_cast<uint4 *>(stage + C::kK + t * 16 + i * 2048) = make_uint4(0, 0, 0, 0);
            }
            if (__any_sync(0xffffffffu, sum != 0.f)) {  // a value that is not finite: taken out of V, remembered
                m = 0.f;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int row = r0 + (i & 3) * 16;
                    uint16_t *src = reinterpret_cast<uint16_t *>(stage + C::kV + t * 16 + i * 2048);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float raw = load1<F16>(src + j);
                        if (!(fabsf(raw) <= 3.4028234e38f)) {
                            src[j] = 0;
                            atomicMin(&sl.bad[(i >> 2) * 64 + ch0 + j], row);
                            sl.any_bad = 1;
                        } else if (F16) {
                            m = fmaxf(m, fabsf(x[i][j]));
                        }
                    }
                }
            }
            if (F16) {
                m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
                float *all = most + (c & 1) * 4;
                if (lane == 0) all[warp - kValueWarp] = m;
                arrive(m_full);
                if (!(ok = wait(m_full, c))) break;
                const int e = lift(fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3])));
                const float f = pow2f(e);
                if (t == 0) sl.u_unit = pow2f(-e);
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[i][j] *= f;
            }
            if (c > 0 && !(ok = wait(u_full, c - 1))) break;  // the last chunk's values have been read
            uint8_t *dst = smem + C::kValues + t * 16;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
#pragma unroll
                for (int part = 0; part < C::kParts; ++part) {
                    const uint4 w = pack8<F16>(x[i]);
                    *reinterpret_cast<uint4 *>(dst + part * C::kPartBytes + i * 2048) = w;
                    if (part + 1 < C::kParts) {
                        float h[8];
                        unpack8<F16>(w, h);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[i][j] -= h[j];
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            arrive(v_full);
            arrive(&g_empty[c % kSlots]);
        }
    } else {
        ptx::regs_down<kOtherRegs>();
        if (warp < kLoadWarp) {
            if (!STATES) {
                // -------------------------------------------------------------------------- P --
                const int i = tid - kWeightWarp * 32;  // its row
                const uint32_t lanes = tmem + ((uint32_t)((warp - kWeightWarp) * 32) << 16);
                uint8_t *dst = smem + C::kP + i * 128;
                for (int c = 0; c < chunks && ok; ++c) {
                    Slot &sl = slots[c % kSlots];
                    if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(a_full, c))) break;
                    ptx::tc_fence_after();
                    uint32_t a[2][32];
                    ptx::tmem_ld_32(lanes + C::kColA, a[0]);
                    ptx::tmem_ld_32(lanes + C::kColA + 32, a[1]);
                    ptx::tmem_ld_wait();
                    tie32(a[0]);
                    tie32(a[1]);
                    ptx::tc_fence_before();
                    arrive(a_free);
                    const float gh = sl.g_hi[i], gl = sl.g_lo[i];
                    float m = 0.f;
#pragma unroll
                    for (int j0 = 0; j0 < kChunk; j0 += 4) {
                        const float4 h4 = *reinterpret_cast<const float4 *>(&sl.g_hi[j0]), l4 = *reinterpret_cast<const float4 *>(&sl.g_lo[j0]);
                        const float h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = j0 + e;
                            const float w = exp2_fast((gh - h[e]) + (gl - l[e]));
                            const float x = j <= i ? __uint_as_float(a[j >> 5][j & 31]) * w : 0.f;
                            a[j >> 5][j & 31] = __float_as_uint(x);
                            if (F16) m = fmaxf(m, fabsf(x));
                        }
                    }
                    float f = 1.f;
                    if (F16) {
                        const int e = lift(m);
                        f = pow2f(e);
                        sl.p_unit[i] = pow2f(-e);
                    }
                    if (c > 0 && !(ok = wait(o_full, c - 1))) break;  // the last chunk's P has been read
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t *x = &a[j >> 2][(j & 3) * 8 + 2 * e];
                            split2<F16>(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f, hi[e], lo[e]);
                        }
                        uint8_t *at = dst + ((j ^ (i & 7)) << 4);
                        *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(at + kBlockBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    ptx::fence_proxy_async_smem();
                    arrive(p_full);
                    arrive(&g_empty[c % kSlots]);
                }
            }
        } else if (warp == kLoadWarp) {
            // -------------------------------------------------------------- copies, decays --
            double total = 0.0;  // log2 of the segment's decay
            if (lane == 0) {
                ptx::tma_prefetch_desc(&maps.k);
                ptx::tma_prefetch_desc(&maps.v);
                if (!STATES) ptx::tma_prefetch_desc(&maps.q);
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const int st = c % kStages;
                const int64_t row = row0 + (int64_t)c * kChunk;
                const int valid = min(rows - c * kChunk, kChunk);
                // the decays of two tokens a lane, on their way while the stage is waited for
                const float g0 = 2 * lane < valid ? load_decay(p, row + 2 * lane, head) : 0.f;
                const float g1 = 2 * lane + 1 < valid ? load_decay(p, row + 2 * lane + 1, head) : 0.f;
                if (c >= kStages && !(ok = wait(&empty[st], c / kStages - 1))) break;
                if (lane == 0) {
                    uint8_t *stage = smem + st * C::kStageBytes;
                    ptx::mbar_arrive_expect_tx(&full[st], (uint32_t)(C::kStageBytes - (STATES ? C::kK : 0)));
#pragma unroll
                    for (int i = 0; i < C::kKBlocks; ++i) {
                        ptx::tma_load_2d(stage + C::kK + i * kBlockBytes, &maps.k, kh * DK + i * 64, (int)row, &full[st]);
                        if (!STATES) ptx::tma_load_2d(stage + i * kBlockBytes, &maps.q, kh * DK + i * 64, (int)row, &full[st]);
                    }
#pragma unroll
                    for (int i = 0; i < C::kVBlocks; ++i)
                        ptx::tma_load_2d(stage + C::kV + i * kBlockBytes, &maps.v, col0 + i * 64, (int)row, &full[st]);
                }
                issued = c + 1;
                if (c >= kSlots && !(ok = wait(&g_empty[c % kSlots], c / kSlots - 1))) break;
                constexpr double kLog2e = 1.4426950408889634074;
                const double l0 = g0 * kLog2e, l1 = g1 * kLog2e;
                double sum = l0 + l1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double x = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += x;
                }
                const double end = __shfl_sync(0xffffffffu, sum, 31), G[2] = {sum - l1, sum};
                total += end;
                Slot &sl = slots[c % kSlots];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * lane + e;
                    const float hi = (float)G[e];
                    sl.g_hi[j] = hi;
                    sl.g_lo[j] = (float)(G[e] - (double)hi);
                    sl.fade[j] = exp2_fast(hi);
                    sl.weight[j] = exp2_fast((float)(end - G[e]));
                }
                for (int i = lane; i < 128; i += 32) sl.bad[i] = kChunk;
                if (lane == 0) {
                    sl.whole = exp2_fast((float)end);
                    sl.any_bad = 0;
                }
                arrive(&g_full[c % kSlots]);
            }
            if (STATES && ok && lane == 0 && tile == 0) p.seg_decay[(int64_t)place * p.VH + head] = exp2_fast((float)total);
        } else {
            // -------------------------------------------------------------------- the MMAs --
            const uint32_t idesc_a = ptx::idesc_16_f32(F16, 128, kChunk, false, false);
            const uint32_t idesc_u = ptx::idesc_16_f32(F16, 128, DK, true, true);
            const uint32_t idesc_o1 = ptx::idesc_16_f32(F16, 128, kChunk, false, false);
            const uint32_t idesc_o2 = ptx::idesc_16_f32(F16, 128, kChunk, true, false);
            const uint64_t desc_k = ptx::sw128_desc(ptx::smem_u32(smem));                    // K-major operands
            const uint64_t desc_mn = ptx::sw128_desc_mn(ptx::smem_u32(smem), kBlockBytes);  // MN-major ones
            constexpr int kBlock16 = kBlockBytes >> 4;
            auto at = [](int bytes) { return (uint64_t)(bytes >> 4); };
            auto logits = [&](int c) {  // A = Q K^T: 64 rows, and 64 that nobody reads
                if (ptx::elect_one()) {
                    const uint64_t st = desc_k + at(c % kStages * C::kStageBytes);
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const int off = (k >> 2) * kBlock16 + (k & 3) * 2;
                        ptx::mma_f16_ss(tmem + C::kColA, st + off, st + at(C::kK) + off, idesc_a, k > 0);
                    }
                    ptx::mma_commit(a_full);
                }
                __syncwarp();
            };
            if (!STATES) {
                ok = wait(&full[0], 0);
                ptx::tc_fence_after();
                if (ok) logits(0);
            }
            for (int c = 0; c < chunks && ok; ++c) {
                const int stage = c % kStages * C::kStageBytes;
                if (!STATES && c + 1 < chunks) {
                    if (!(ok = wait(&full[(c + 1) % kStages], (c + 1) / kStages) && wait(a_free, c))) break;
                    ptx::tc_fence_after();
                    logits(c + 1);
                }
                // U^T = (w V)^T K
                if (STATES && !(ok = wait(&full[c % kStages], c / kStages))) break;
                if (!(ok = wait(v_full, c) && (c == 0 || wait(u_free, c - 1)))) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part)
#pragma unroll
                        for (int k = 0; k < kChunk / 16; ++k)
                            ptx::mma_f16_ss(tmem + C::kColU, desc_mn + at(C::kValues + part * C::kPartBytes + k * 2048),
                                            desc_mn + at(stage + C::kK + k * 2048), idesc_u, part > 0 || k > 0);
                    ptx::mma_commit(u_full);
                    ptx::mbar_arrive(u_full);
                    if (STATES) ptx::mma_commit(&empty[c % kStages]);
                }
                __syncwarp();
                if (STATES) continue;
                // O1^T = S0^T Q^T
                if (!(ok = wait(s_full, c) && (c == 0 || wait(o_free, c - 1)))) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k)
                            ptx::mma_f16_ts(tmem + C::kColO1, tmem + C::kColS + part * (DK / 2) + k * 8,
                                            desc_k + at(stage) + (k >> 2) * kBlock16 + (k & 3) * 2, idesc_o1, part > 0 || k > 0);
                    ptx::mma_commit(s_free);
                }
                __syncwarp();
                // O2^T = V^T P^T
                if (!(ok = wait(p_full, c))) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < kChunk / 16; ++k)
                            ptx::mma_f16_ss(tmem + C::kColO2, desc_mn + at(stage + C::kV + k * 2048),
                                            desc_k + at(C::kP + part * kBlockBytes) + k * 2, idesc_o2, part > 0 || k > 0);
                    ptx::mma_commit(o_full);
                    ptx::mbar_arrive(o_full);
                    ptx::mma_commit(&empty[c % kStages]);
                }
                __syncwarp();
            }
            if (!ok) {  // nothing of this block may still run when its TMEM is freed
                if (ptx::elect_one()) ptx::mma_commit(drain);
                int zero = 0;
                ptx::mbar_wait(drain, 0, kWaitNs, &zero);
            }
        }
    }
    if (!ok) {
        *abort_flag = 1;
        atomicCAS(p.status, 0, (int)MOE_ERR_TIMEOUT);
        if (warp == kLoadWarp && lane == 0) {  // copies under way land before the shared memory is given up
            int zero = 0;
            for (int c = max(issued - kStages, 0); c < issued; ++c) ptx::mbar_wait(&full[c % kStages], c / kStages & 1, kWaitNs, &zero);
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, C::kCols);
}

template <int DK, int DV, bool F16, bool STATES>
cudaError_t launch_kernel(const LinearArgs &a, const Maps &m, cudaStream_t s) {
    constexpr int smem = Shape<DK, DV, F16>::kSmem;
    auto *kernel = linear_chunk_kernel<DK, DV, F16, STATES>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t segments = linear_segments(a.n_tokens, a.n_seqs, a.segment_chunks), blocks = segments * a.VH * (a.DV / DV);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    LaunchScope scope(STATES ? KC_LINEAR_STATES : KC_LINEAR_CHUNKS, s);
    kernel<<<(unsigned)blocks, kThreads, smem, s>>>(a, m);
    return cudaGetLastError();
}

template <int DK, int DV, bool F16>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
    Maps m;
    if (!encode_tmap_rows(&m.q, a.q, a.n_tokens, (uint64_t)a.KH * DK, a.q_ld, kChunk, 64) ||
        !encode_tmap_rows(&m.k, a.k, a.n_tokens, (uint64_t)a.KH * DK, a.k_ld, kChunk, 64) ||
        !encode_tmap_rows(&m.v, a.v, a.n_tokens, (uint64_t)a.VH * a.DV, a.v_ld, kChunk, 64))
        return cudaErrorInvalidValue;
    if (a.seg_states) {
        const cudaError_t e = launch_kernel<DK, DV, F16, true>(a, m, s);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel<DK, DV, F16, false>(a, m, s);
}

}  // namespace

cudaError_t launch_linear_chunks(const LinearArgs &a, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (a.DK == 64) {
        if (a.DV == 64) return f16 ? launch<64, 64, true>(a, s) : launch<64, 64, false>(a, s);
        return f16 ? launch<64, 128, true>(a, s) : launch<64, 128, false>(a, s);
    }
    if (a.DV == 64) return f16 ? launch<128, 64, true>(a, s) : launch<128, 64, false>(a, s);
    return f16 ? launch<128, 128, true>(a, s) : launch<128, 128, false>(a, s);
}

}  // namespace moe
