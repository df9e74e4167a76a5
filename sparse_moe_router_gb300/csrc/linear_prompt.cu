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
// that of its fp32 sums).  With fp16, whose range is short, each row of P, each channel of S0 and each channel of a chunk's
// weighted values are scaled by a power of two of their own: two parts then hold 22 bits, down to 2^-39 of the largest.  (One power
// for all channels of a chunk took 4% less time, and left a channel 2^-26 as large as another 11 bits.)
//
// A block walks one value head's chunks (128 value channels at most) in order.  The state is what makes it wait: U(c) ->
// registers -> S0(c+1) in TMEM; everything else runs ahead.  Where heads and sequences leave SMs idle, a
// run's chunks are cut into segments: a first kernel computes what each segment adds to the state (K and V only),
// and each segment's block begins with the sum of those before it.
//
// Bound: shared memory.  At DK = DV = 128 a chunk's operands, copies, splits and transposes move some 3800 times 128 bytes (U
// alone, whose values come in three parts, 1280), and 4250 cycles are measured; the tensor cores are busy for 1790 of them.
// Beside that the instruction cache: all loops that need not be unrolled are not (92 KB of straight-line roles took 10,900
// cycles a chunk, most of them waiting for instructions), little may spill (28 bytes of fp16's do; shared memory leaves no L1: 52 bytes
// cost 30%), and what a chunk's decays need is read two chunks ahead.
//
// Measured, 32 value heads and 16 key heads of 128: 8192 tokens 112 us (39 of them the first kernel's) where token by token
// takes 10,270; 512 tokens 21, 64 tokens 7.7; 12 runs of up to 1031 tokens, 20 heads of 64 and 128 in fp16, 52 (its longest run's
// 17 chunks, one after another: fp16's scales of P take a pass of their own).  On the way: decays in 64-bit floats 3000 cycles a
// chunk; outputs stored 2 bytes at a time 10,000; A in one place 97 us for the second kernel where two take 84; weighted values as
// an operand in TMEM, 16 or 32 tokens at a time, 116 to 126 in all.
//
// Roles (16 warps): 0-3 the state; 4-7 the output; 8-11 weighted values; 12, 13 P (a row a thread); 14 copies (TMA)
// and decays; 15 the MMAs.  Without outputs 4-11 weigh values and 12 copies.
#include <atomic>

#include "mixer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kOutWarp = 4, kValueWarp = 8, kWeightWarp = 12, kLoadWarp = 14, kMmaWarp = 15;
// Registers a thread: 128 at launch; of a scheduler's 4 x 128 the state's warp, which holds 128 of them, takes most (less
// and the roles spill, into an L1 that shared memory has left next to nothing of).
template <bool STATES>
struct Regs {
    static constexpr int kState = STATES ? 216 : 232, kOut = 96, kValue = STATES ? 80 : 64, kOther = 120;
    static_assert(kState + kOut + kValue + kOther <= 512, "more registers than the block has");
};
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s, of the waits when a block gives up
constexpr int kBlockBytes = kChunk * 128;    // 64 tokens x 64 channels
constexpr int kFetch = 2;                    // chunks beyond the stages that are brought into L2
constexpr int kTurnRow = 36;                 // words of 32 channels in a transpose buffer, padded for the banks
constexpr int kSlots = 4;                    // chunks whose decays are in shared memory

// What the warps tell one another of a chunk.
struct alignas(16) Slot {
    float g_hi[kChunk], g_lo[kChunk];  // -log2 of the decay from the chunk's begin, in two parts
    float to_end[kChunk];              // e^{G_l - G_j}, l the last of the 16 tokens that j is among
    float weight[kChunk];              // e^{G_64 - G_j}
    float fade[kChunk];                // scale e^{G_i}
    float p_unit[kChunk];              // fp16: P's rows hold scale / p_unit of their values
    float s_unit[128];                 // fp16: and S0's channels
    float u_unit[128];                 // fp16: U's channels hold 1 / u_unit of their values
    int bad[128];                      // first token whose value is not finite, of each channel
    float whole;                       // e^{G_64}
    int any_bad;
};

template <int DK, int DV, bool F16>
struct Shape {
    static constexpr int kKBlocks = DK / 64, kVBlocks = DV / 64;
    static constexpr int kK = kKBlocks * kBlockBytes, kV = 2 * kK;  // offsets in a stage, of Q 0
    static constexpr int kStageBytes = kV + kVBlocks * kBlockBytes;
    static constexpr int kStages = 3;
    static constexpr int kParts = F16 ? 2 : 3;  // of a weighted value
    static constexpr int kPartBytes = kVBlocks * kBlockBytes;
    static constexpr int kValues = kStages * kStageBytes, kP = kValues + kParts * kPartBytes;
    static constexpr int kTurn = kP + 2 * kBlockBytes, kBars = kTurn + kVBlocks * 2 * 8 * kTurnRow * 4, kSlotAt = kBars + 384;
    static constexpr int kSmem = 1024 + kSlotAt + kSlots * (int)sizeof(Slot);
    static constexpr int kLaneWarps = DV / 32;  // warps that hold channels
    // TMEM columns: S0 in two parts, U, A of even and odd chunks, O1, O2
    static constexpr uint32_t kColS = 0, kColU = DK, kColA = 2 * DK, kColO1 = kColA + 2 * 64, kColO2 = kColO1 + 64, kCols = 512;
    static_assert(kColO2 + 64 <= kCols, "TMEM");
    static_assert(kSmem <= 227 * 1024, "shared memory over the per-block limit");
    // (operands of 128 rows whose second half is none of theirs read up to a block further; it is never looked at)
    static_assert(kP + 2 * kBlockBytes <= kSmem - 1024, "operands end in shared memory");
};

template <bool B>
struct Flag {
    static constexpr bool value = B;
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
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// What a rounding to 16 bits left out of x.
template <bool F16>
__device__ __forceinline__ float2 rest(float2 x, uint32_t rounded) {
    return __ffma2_rn(unpack2<F16>(rounded), both(-1.f), x);
}
// x = hi + lo, both of the 16-bit type.
template <bool F16>
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
    hi = pack2<F16>(x.x, x.y);
    const float2 r = rest<F16>(x, hi);
    lo = pack2<F16>(r.x, r.y);
}

// A sum of logs in two floats (48 bits): a chunk's decays differ by what is small beside their sum from its begin, and
// 64-bit floats cost 16 cycles each here.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // a + b exactly (Knuth)
    const float s = a + b, v = s - a;
    return {s, (a - (s - v)) + (b - v)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    const float lo = s.lo + (a.lo + b.lo), hi = s.hi + lo;
    return {hi, lo - (hi - s.hi)};
}
__device__ __forceinline__ Two log2_of(float g) {  // g log2(e)
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f;
    const float hi = g * kHi;
    return {hi, fmaf(g, kLo, fmaf(g, kHi, -hi))};
}

// Where sequence b's segments lie among the batch's.
__device__ __forceinline__ int first_place(const LinearArgs &p, int b) {
    return segment_base(p.q_start[b], b, p.segment_chunks, p.place_tokens);
}

// STATES: what each segment but a run's last adds to the state, and its decay; otherwise the outputs.
template <int DK, int DV, bool F16, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ LinearArgs p, const __grid_constant__ Maps maps) {
    using C = Shape<DK, DV, F16>;
    constexpr int kStages = C::kStages;
    constexpr int kUs = STATES ? 2 : 1;            // places for U
    constexpr int kConvWarps = STATES ? 8 : 4;  // (without outputs their warps weigh values too)
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBars);  // [kStages] Q, K, V of a chunk
    uint64_t *empty = full + kStages;                                // [kStages]
    uint64_t *g_full = empty + kStages, *g_empty = g_full + kSlots;  // [kSlots] decays
    uint64_t *a_full = g_empty + kSlots, *a_free = a_full + 2;       // [2] A of an even or odd chunk in TMEM; read
    uint64_t *p_full = a_free + 2;                                   // P in shared memory
    uint64_t *v_full = p_full + 1, *v_free = v_full + 2;             // [2] weighted values of 32 tokens there; read
    uint64_t *u_full = v_free + 2, *u_free = u_full + 2;             // [2] U in TMEM; read (without outputs: of even and odd chunks)
    uint64_t *s_full = u_free + 2, *s_free = s_full + 1;             // S0 in TMEM; read by its product
    uint64_t *o_full = s_free + 1, *o_free = o_full + 1;             // O1 and O2 in TMEM (and P read); read
    uint64_t *drain = o_free + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    Slot *slots = reinterpret_cast<Slot *>(smem + C::kSlotAt);

    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

    if (!STATES) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the token kernel does not depend on this one)

    // ------------------------------------------------------------------- the block's chunks --
    const int tiles = p.DV / DV;
    const int tile = (int)blockIdx.x % tiles, head = (int)blockIdx.x / tiles % p.VH, place = (int)blockIdx.x / tiles / p.VH;
    int b = 0;  // the last sequence whose places begin at or before this one: 32 probes at a time
    for (int end = p.n_seqs; end - b > 1;) {
        const int step = (end - b + 31) / 32, at = b + lane * step;
        const int n = __popc(__ballot_sync(0xffffffffu, at < end && first_place(p, at) <= place));
        b += max(n - 1, 0) * step;
        end = min(b + step, end);
    }
    const Run run = load_run(p, b);
    // (where there is no other kernel, chunk_tokens is 0: a run of padding alone is this one's too)
    if (run.n < p.chunk_tokens) return;
    const int all = (run.n + kChunk - 1) / kChunk, base = first_place(p, b), seg = place - base;
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
            ptx::mbar_init(&g_empty[s], kConvWarps + C::kLaneWarps + (STATES ? 0 : 2 + C::kLaneWarps));
        }
        ptx::mbar_init(p_full, 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&a_full[i], 1), ptx::mbar_init(&a_free[i], 2);
            ptx::mbar_init(&v_full[i], kConvWarps), ptx::mbar_init(&v_free[i], 1);
        }
        // (u_full and o_full: the MMAs' end, and the arrival of the warp that has seen the units of their operands)
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&u_full[i], 2), ptx::mbar_init(&u_free[i], C::kLaneWarps);
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
        return __all_sync(0xffffffffu, ptx::mbar_sleep_wait(bar, phase & 1, abort_flag)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar);
    };
    bool ok = true;
    int issued = 0;  // chunks whose copies were begun

    // ----------------------------------------------------------------- weighted values --
    // A thread has the 8 channels of one 16-byte column of the tile, of every kRows-th token from r0 on, as they lie in shared
    // memory (swizzled: 8 lanes on 8 rows touch all banks); a warp has all 64 tokens of its channels.  What comes out lies in the
    // same places.  Two halves of 32 tokens, the one's products under way while the other is weighed.
    auto weigh_values = [&]() {
        constexpr int kGroups = DV / 8 / kConvWarps, kRows = 32 / kGroups, kPieces = kChunk / kRows;
        const int conv = warp - (kWeightWarp - kConvWarps), t = conv * 32 + lane, r0 = lane % kRows, group = conv * kGroups + lane / kRows;
        const int place = (group >> 3) * kBlockBytes + r0 * 128 + (((group ^ r0) & 7) << 4);
        for (int c = 0; c < chunks && ok; ++c) {
            Slot &sl = slots[c % kSlots];
            uint8_t *stage = smem + c % kStages * C::kStageBytes;
            if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(&full[c % kStages], c / kStages))) break;
            const int valid = min(rows - c * kChunk, kChunk);
            auto piece = [&](int i) { return reinterpret_cast<uint4 *>(stage + C::kV + place + i * (kRows * 128)); };
            if (valid < kChunk) {  // behind the run's end, where whatever comes there lies: the products must not see it
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int i = 0; i < kPieces; ++i)
                    if (r0 + i * kRows >= valid) *piece(i) = zero;
#pragma unroll 1
                for (int at = t * 16; at < C::kKBlocks * kBlockBytes; at += kConvWarps * 512)
                    if ((at >> 7) % kChunk >= valid) *reinterpret_cast<uint4 *>(stage + C::kK + at) = zero;
            }
            float2 unit[4];  // fp16: a power of two for each channel, by its largest weighted value of the chunk
            if (F16) {
                uint32_t most[4] = {0, 0, 0, 0};  // (rounded to bf16, which has the exponents; a NaN does not count)
                auto larger = [](uint32_t a, uint32_t b) {
                    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
                    return *reinterpret_cast<const uint32_t *>(&m);
                };
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const uint4 w = *piece(i);
                    const uint32_t raw[4] = {w.x, w.y, w.z, w.w};
                    const float2 f = both(sl.weight[r0 + i * kRows]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = __fmul2_rn(unpack2<F16>(raw[j]), f);
                        most[j] = larger(most[j], pack2<false>(x.x, x.y) & 0x7fff7fffu);
                    }
                }
#pragma unroll
                for (int o = kRows / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int j = 0; j < 4; ++j) most[j] = larger(most[j], __shfl_xor_sync(0xffffffffu, most[j], o));
                // from an exponent E of at least 15 to 268 - E, two at a time: the largest comes to lie between 2^14 and 2^15
#pragma unroll
                for (int j = 0; j < 4; ++j) unit[j] = unpack2<false>(0x86008600u - larger(most[j] & 0x7f807f80u, 0x07800780u));
                if (r0 == 0) {  // what undoes them, exponents 254 - (268 - E)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float2 *>(&sl.u_unit[group * 8 + 2 * j]) =
                            make_float2(__int_as_float((254 << 23) - __float_as_int(unit[j].x)), __int_as_float((254 << 23) - __float_as_int(unit[j].y)));
                }
            }
            uint8_t *dst = smem + C::kValues + place;
            float2 sum = both(0.f);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {  // tokens 0..31, 32..63
                if (c > 0 && !(ok = wait(&v_free[half], c - 1))) break;  // the last chunk's have been read
                uint4 raw[kPieces / 2];  // (loads cannot pass the stores by themselves)
                float weight[kPieces / 2];
                const int first = half * (kPieces / 2);
#pragma unroll
                for (int n = 0; n < kPieces / 2; ++n) raw[n] = *piece(first + n), weight[n] = sl.weight[r0 + (first + n) * kRows];
#pragma unroll
                for (int n = 0; n < kPieces / 2; ++n) {
                    float2 x[4] = {unpack2<F16>(raw[n].x), unpack2<F16>(raw[n].y), unpack2<F16>(raw[n].z), unpack2<F16>(raw[n].w)};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum = __ffma2_rn(x[j], both(0.f), sum);
                        x[j] = __fmul2_rn(x[j], both(weight[n]));
                        if (F16) x[j] = __fmul2_rn(x[j], unit[j]);
                    }
#pragma unroll
                    for (int part = 0; part < C::kParts; ++part) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            w[j] = pack2<F16>(x[j].x, x[j].y);
                            if (part + 1 < C::kParts) x[j] = rest<F16>(x[j], w[j]);
                        }
                        *reinterpret_cast<uint4 *>(dst + part * C::kPartBytes + (first + n) * (kRows * 128)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                // A value that is not finite makes its channel of the state that; of the tokens before it the product with P must
                // not see it (0 times it), so it is taken out of V in the end, and remembered for the tokens from it on.
                if (half == 1 && __any_sync(0xffffffffu, sum.x != 0.f || sum.y != 0.f)) {
#pragma unroll 1
                    for (int e = 0; e < kPieces * 8; ++e) {
                        uint16_t *src = reinterpret_cast<uint16_t *>(piece(e >> 3)) + (e & 7);
                        if (fabsf(load1<F16>(src)) <= 3.4028234e38f) continue;
                        *src = 0;
                        atomicMin(&sl.bad[group * 8 + (e & 7)], r0 + (e >> 3) * kRows);
                        sl.any_bad = 1;
                    }
                    __syncwarp();
                }
                ptx::fence_proxy_async_smem();
                arrive(&v_full[half]);
            }
            if (!ok) break;
            arrive(&g_empty[c % kSlots]);
        }
    };

    if (warp < kOutWarp) {
        ptx::regs_up<Regs<STATES>::kState>();
        if (warp < C::kLaneWarps) {
            // ------------------------------------------------------------------ the state --
            // Thread t has channel t: S[d] of all key channels d.
            const int64_t state_size = (int64_t)DK * p.DV;
            float *own = p.states + ((int64_t)max(run.slot, 0) * p.VH + head) * state_size + tile * DV + tid;
            auto place_at = [&](int i) {  // of segment i of this run
                return p.seg_states + ((int64_t)(base + i) * p.VH + head) * state_size + tile * DV + tid;
            };
            float2 S[DK / 2];  // channels 2 d and 2 d + 1
            auto store = [&](float *dst) {
#pragma unroll
                for (int d = 0; d < DK / 2; ++d) {
                    dst[0] = S[d].x;
                    dst[p.DV] = S[d].y;
                    dst += 2 * p.DV;
                }
            };
#pragma unroll
            for (int d = 0; d < DK / 2; ++d) S[d] = both(0.f);
            // The first segment begins with the slot's state (of several segments the last writes the slot: the output's
            // kernel finds the state at the last one's place), the others with what those before them add.
            const int sources = seg > 0 ? (STATES ? 0 : seg) : run.fresh ? 0 : 1;
#pragma unroll 1
            for (int i = 0; i < sources; ++i) {
                const float *src = seg > 0 ? place_at(i) : !STATES && segs > 1 ? place_at(segs - 1) : own;
                const float f = i == 0 ? 0.f : p.seg_decay[(int64_t)(base + i) * p.VH + head];
#pragma unroll
                for (int d = 0; d < DK / 2; ++d) {
                    S[d] = __ffma2_rn(S[d], both(f), make_float2(src[0], src[p.DV]));
                    src += 2 * p.DV;
                    if (d % 32 == 31) asm volatile("" ::: "memory");  // (no more loads at once than there are registers for)
                }
            }
            if (STATES && seg == 0 && !run.fresh) store(place_at(segs - 1));
            const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
            for (int c = 0; c < chunks; ++c) {
                Slot &sl = slots[c % kSlots];
                if (!(ok = wait(&g_full[c % kSlots], c / kSlots))) break;
                if (!STATES) {  // S0 in two parts
                    if (c > 0 && !(ok = wait(s_free, c - 1))) break;
                    ptx::tc_fence_after();
                    float f = 1.f;
                    if (F16) {
                        float m = 0.f;
#pragma unroll
                        for (int d = 0; d < DK / 2; ++d) m = fmaxf(m, fmaxf(fabsf(S[d].x), fabsf(S[d].y)));
                        const int e = lift(m);
                        f = pow2f(e);
                        sl.s_unit[tid] = pow2f(-e);
                    }
#pragma unroll
                    for (int g = 0; g < DK / 32; ++g) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int d = 0; d < 16; ++d) asm volatile("" : "+f"(S[g * 16 + d].x), "+f"(S[g * 16 + d].y));  // (one group after another)
#pragma unroll
                        for (int d = 0; d < 16; ++d) split2<F16>(F16 ? __fmul2_rn(S[g * 16 + d], both(f)) : S[g * 16 + d], hi[d], lo[d]);
                        ptx::tmem_st_16(lanes + C::kColS + g * 16, hi);
                        ptx::tmem_st_16(lanes + C::kColS + DK / 2 + g * 16, lo);
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    arrive(s_full);
                }
                if (!(ok = wait(&u_full[c % kUs], c / kUs))) break;
                ptx::tc_fence_after();
                const float f = sl.whole, unit = F16 ? sl.u_unit[tid] : 1.f;
#pragma unroll
                for (int g = 0; g < DK / 32; ++g) {
                    uint32_t u[32];
                    ptx::tmem_ld_32(lanes + C::kColU + c % kUs * 128 + g * 32, u);
                    ptx::tmem_ld_wait();
                    tie32(u);
#pragma unroll
                    for (int d = 0; d < 16; ++d) {
                        float2 x = make_float2(__uint_as_float(u[2 * d]), __uint_as_float(u[2 * d + 1]));
                        if (F16) x = __fmul2_rn(x, both(unit));
                        S[g * 16 + d] = __ffma2_rn(S[g * 16 + d], both(f), x);
                    }
                }
                ptx::tc_fence_before();
                arrive(&u_free[c % kUs]);
                arrive(&g_empty[c % kSlots]);
            }
            if (ok && (STATES || (seg == segs - 1 && run.slot >= 0))) store(STATES ? place_at(seg) : own);
        }
    } else if (warp < kValueWarp) {
        ptx::regs_down<Regs<STATES>::kOut>();
        if (STATES) {
            weigh_values();
        } else if (warp - kOutWarp < C::kLaneWarps) {
            // ------------------------------------------------------------------ the output --
            // Thread t has channel t of all tokens.  16 tokens at a time go through the warp's own transpose buffer, two tokens
            // of a channel a word, and leave as 16-byte pieces of a token's row.
            const int w = warp - kOutWarp, ch = w * 32 + lane, m = lane >> 2, piece = lane & 3;
            const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16);
            uint32_t *turn = reinterpret_cast<uint32_t *>(smem + C::kTurn) + w * (8 * kTurnRow);
            for (int c = 0; c < chunks && ok; ++c) {
                const Slot &sl = slots[c % kSlots];
                if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(o_full, c))) break;
                ptx::tc_fence_after();
                const int valid = min(rows - c * kChunk, kChunk);
                const float unit = F16 ? sl.s_unit[ch] : 1.f;
                const bool some = sl.any_bad != 0;
                const int bad = some ? sl.bad[ch] : kChunk;
                uint32_t o[32];  // token pairs
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t a[16], x[16];
                    ptx::tmem_ld_16(lanes + C::kColO1 + g * 16, a);
                    ptx::tmem_ld_16(lanes + C::kColO2 + g * 16, x);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int t = 0; t < 16; ++t) asm volatile("" : "+r"(a[t]), "+r"(x[t]));
#pragma unroll
                    for (int t = 0; t < 16; t += 4) {
                        const float4 f4 = *reinterpret_cast<const float4 *>(&sl.fade[g * 16 + t]);
                        float4 p4 = make_float4(p.scale, p.scale, p.scale, p.scale);
                        if (F16) p4 = *reinterpret_cast<const float4 *>(&sl.p_unit[g * 16 + t]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float2 f = e ? make_float2(f4.z, f4.w) : make_float2(f4.x, f4.y);
                            if (F16) f = __fmul2_rn(f, both(unit));
                            float2 v = __fmul2_rn(make_float2(__uint_as_float(a[t + e]), __uint_as_float(a[t + e + 1])), f);
                            v = __ffma2_rn(make_float2(__uint_as_float(x[t + e]), __uint_as_float(x[t + e + 1])),
                                           e ? make_float2(p4.z, p4.w) : make_float2(p4.x, p4.y), v);
                            o[g * 8 + (t + e) / 2] = pack2<F16>(v.x, v.y);
                        }
                    }
                }
                ptx::tc_fence_before();
                arrive(o_free);
                if (some) {
#pragma unroll
                    for (int t = 0; t < 32; ++t) o[t] |= (2 * t >= bad ? 0x7fffu : 0u) | (2 * t + 1 >= bad ? 0x7fff0000u : 0u);
                }
                uint16_t *dst = p.out + (row0 + (int64_t)c * kChunk + 2 * m) * p.out_ld + col0 + w * 32 + piece * 8;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 8; ++k) turn[k * kTurnRow + lane] = o[g * 8 + k];
                    __syncwarp();
                    const uint4 y = *reinterpret_cast<const uint4 *>(&turn[m * kTurnRow + piece * 8]);
                    const uint4 z = *reinterpret_cast<const uint4 *>(&turn[m * kTurnRow + piece * 8 + 4]);
                    if (g * 16 + 2 * m < valid)
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410),
                                                                     __byte_perm(z.x, z.y, 0x5410), __byte_perm(z.z, z.w, 0x5410));
                    if (g * 16 + 2 * m + 1 < valid)
                        *reinterpret_cast<uint4 *>(dst + p.out_ld) =
                            make_uint4(__byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632), __byte_perm(z.x, z.y, 0x7632),
                                       __byte_perm(z.z, z.w, 0x7632));
                    dst += 16 * p.out_ld;
                }
                arrive(&g_empty[c % kSlots]);
            }
        }
    } else if (warp < kWeightWarp) {
        ptx::regs_down<Regs<STATES>::kValue>();
        weigh_values();
    } else {
        ptx::regs_down<Regs<STATES>::kOther>();
        if (warp < kLoadWarp && !(STATES && warp == kWeightWarp)) {
            if (!STATES) {
                // -------------------------------------------------------------------------- P --
                // Rows 0..31 are one warp's, 32..63 the other's: of the four 32 x 32 blocks the first warp has one below the
                // diagonal's and one of zeros, which stays, the second one that no mask touches.
                const int i = tid - kWeightWarp * 32, halves = warp - kWeightWarp + 1;  // its row; its blocks
                const uint32_t lanes = tmem + ((uint32_t)((warp - kWeightWarp) * 32) << 16);
                uint8_t *dst = smem + C::kP + i * 128;
                if (halves == 1) {
#pragma unroll
                    for (int j = 4; j < 8; ++j) {
                        *reinterpret_cast<uint4 *>(dst + ((j ^ (i & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(dst + ((j ^ (i & 7)) << 4) + kBlockBytes) = make_uint4(0, 0, 0, 0);
                    }
                }
                for (int c = 0; c < chunks && ok; ++c) {
                    Slot &sl = slots[c % kSlots];
                    if (!(ok = wait(&g_full[c % kSlots], c / kSlots) && wait(&a_full[c & 1], c >> 1))) break;
                    ptx::tc_fence_after();
                    const float2 gh = both(-sl.g_hi[i]), gl = both(-sl.g_lo[i]);
                    float m = 0.f, f = 1.f;
                    // 16 columns from j0 on: their largest (with fp16, whose rows are scaled), or their two parts into shared memory.
                    // Where all of them lie before the row, their weights are e^{G_i - G_l} e^{G_l - G_j}, l the last of them.
                    auto weigh = [&](int j0, auto diagonal, bool put) {
                        uint32_t a[16];
                        ptx::tmem_ld_16(lanes + C::kColA + (c & 1) * 64 + j0, a);
                        const float since = exp2_fast((gh.x + sl.g_hi[j0 + 15]) + (gl.x + sl.g_lo[j0 + 15])) * f;
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(a[j]));
                        uint32_t hi[8], lo[8];
                        const int last = i - j0;
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float2 x = make_float2(__uint_as_float(a[j]), __uint_as_float(a[j + 1]));
                            if constexpr (decltype(diagonal)::value) {
                                const float4 h4 = *reinterpret_cast<const float4 *>(&sl.g_hi[j0 + (j & ~3)]);
                                const float4 l4 = *reinterpret_cast<const float4 *>(&sl.g_lo[j0 + (j & ~3)]);
                                const float2 h = j & 2 ? make_float2(h4.z, h4.w) : make_float2(h4.x, h4.y);
                                const float2 l = j & 2 ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                                const float2 g = __fadd2_rn(__fadd2_rn(gh, h), __fadd2_rn(gl, l));
                                x = __fmul2_rn(x, make_float2(exp2_fast(g.x), exp2_fast(g.y)));
                                if (j > last) x.x = 0.f;
                                if (j + 1 > last) x.y = 0.f;
                                if (F16) x = __fmul2_rn(x, both(f));
                            } else {
                                const float4 w4 = *reinterpret_cast<const float4 *>(&sl.to_end[j0 + (j & ~3)]);
                                x = __fmul2_rn(x, __fmul2_rn(j & 2 ? make_float2(w4.z, w4.w) : make_float2(w4.x, w4.y), both(since)));
                            }
                            if (F16 && !put) m = fmaxf(m, fmaxf(fabsf(x.x), fabsf(x.y)));
                            else split2<F16>(x, hi[j / 2], lo[j / 2]);
                        }
                        if (F16 && !put) return;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint8_t *at = dst + ((j0 / 8 + k) ^ (i & 7)) * 16;
                            *reinterpret_cast<uint4 *>(at) = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                            *reinterpret_cast<uint4 *>(at + kBlockBytes) = make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                        }
                    };
#pragma unroll 1
                    for (int pass = F16 ? 0 : 1; pass < 2; ++pass) {
                        if (pass == 1 && c > 0 && !(ok = wait(o_full, c - 1))) break;  // the last chunk's P has been read
                        int j0 = 0;
#pragma unroll 1
                        for (; j0 < (halves - 1) * 32; j0 += 16) weigh(j0, Flag<false>{}, pass == 1);
#pragma unroll 1
                        for (; j0 < halves * 32; j0 += 16) weigh(j0, Flag<true>{}, pass == 1);
                        if (F16 && pass == 0) {
                            const int e = lift(m);
                            f = pow2f(e);
                            sl.p_unit[i] = p.scale * pow2f(-e);
                        }
                    }
                    if (!ok) break;
                    ptx::tc_fence_before();
                    arrive(&a_free[c & 1]);
                    ptx::fence_proxy_async_smem();
                    arrive(p_full);
                    arrive(&g_empty[c % kSlots]);
                }
            }
        } else if (warp <= kLoadWarp) {
            // -------------------------------------------------------------- copies, decays --
            // (without outputs each has a warp of its own)
            const bool copy = !STATES || warp == kWeightWarp, weigh = warp == kLoadWarp;
            Two total{0.f, 0.f};  // log2 of the segment's decay
            // Lanes 0, 1 (, 2) copy a chunk's tokens of K, V (and Q); lanes 8, 9 (, 10) bring those of a later chunk into L2.
            constexpr int kBoxes = STATES ? 2 : 3;
            const int box = lane & 7;
            const CUtensorMap *map = box == 0 ? &maps.k : box == 1 ? &maps.v : &maps.q;
            const int box_block = box == 1 ? col0 / 64 : kh * C::kKBlocks, box_at = box == 0 ? C::kK : box == 1 ? C::kV : 0;
            if (copy && lane < kBoxes) ptx::tma_prefetch_desc(map);
            // the decays of two tokens a lane, on their way two chunks ahead
            auto decays = [&](int c) {
                const int i = c * kChunk + 2 * lane;
                return make_float2(weigh && i < rows ? raw_decay(p, row0 + i, head) : 0.f, weigh && i + 1 < rows ? raw_decay(p, row0 + i + 1, head) : 0.f);
            };
            float2 g = decays(0), g1 = decays(1);
            if (copy && lane >= 8 && lane < 8 + kBoxes)
                for (int c = kStages; c < min(kStages + kFetch, chunks); ++c) ptx::tma_prefetch_3d(map, 0, (int)row0 + c * kChunk, box_block);
            for (int c = 0; c < chunks && ok; ++c) {
                const int st = c % kStages, row = (int)row0 + c * kChunk;
                const float2 g2 = decays(c + 2);
                if (copy) {
                    if (c >= kStages && !(ok = wait(&empty[st], c / kStages - 1))) break;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&full[st], (uint32_t)(C::kStageBytes - (STATES ? C::kK : 0)));
                    __syncwarp();
                    if (lane < kBoxes) ptx::tma_load_3d(smem + st * C::kStageBytes + box_at, map, 0, row, box_block, &full[st]);
                    else if (lane >= 8 && lane < 8 + kBoxes && c + kStages + kFetch < chunks)
                        ptx::tma_prefetch_3d(map, 0, row + (kStages + kFetch) * kChunk, box_block);
                    issued = c + 1;
                }
                if (!weigh) continue;
                if (c >= kSlots && !(ok = wait(&g_empty[c % kSlots], c / kSlots - 1))) break;
                const Two l0 = log2_of(checked_decay(p, g.x)), l1 = log2_of(checked_decay(p, g.y));
                g = g1, g1 = g2;
                Two G = l0 + l1;  // up to the lane's second token
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const Two x{__shfl_up_sync(0xffffffffu, G.hi, o), __shfl_up_sync(0xffffffffu, G.lo, o)}, y = x + G;
                    if (lane >= o) G = y;
                }
                const Two end{__shfl_sync(0xffffffffu, G.hi, 31), __shfl_sync(0xffffffffu, G.lo, 31)};
                const Two G0 = G + Two{-l1.hi, -l1.lo};
                total = total + end;
                Slot &sl = slots[c % kSlots];
                const Two last{__shfl_sync(0xffffffffu, G.hi, lane | 7), __shfl_sync(0xffffffffu, G.lo, lane | 7)};  // of 16 tokens
                reinterpret_cast<float2 *>(sl.to_end)[lane] =
                    make_float2(exp2_fast((last.hi - G0.hi) + (last.lo - G0.lo)), exp2_fast((last.hi - G.hi) + (last.lo - G.lo)));
                reinterpret_cast<float2 *>(sl.g_hi)[lane] = make_float2(-G0.hi, -G.hi);
                reinterpret_cast<float2 *>(sl.g_lo)[lane] = make_float2(-G0.lo, -G.lo);
                reinterpret_cast<float2 *>(sl.fade)[lane] = make_float2(p.scale * exp2_fast(G0.hi), p.scale * exp2_fast(G.hi));
                reinterpret_cast<float2 *>(sl.weight)[lane] =
                    make_float2(exp2_fast((end.hi - G0.hi) + (end.lo - G0.lo)), exp2_fast((end.hi - G.hi) + (end.lo - G.lo)));
                for (int i = lane; i < 128; i += 32) sl.bad[i] = kChunk;
                if (lane == 0) {
                    sl.whole = exp2_fast(end.hi);
                    sl.any_bad = 0;
                }
                arrive(&g_full[c % kSlots]);
            }
            if (STATES && weigh && ok && lane == 0 && tile == 0) p.seg_decay[(int64_t)place * p.VH + head] = exp2_fast(total.hi);
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
                        ptx::mma_f16_ss(tmem + C::kColA + (c & 1) * 64, st + off, st + at(C::kK) + off, idesc_a, k > 0);
                    }
                    ptx::mma_commit(&a_full[c & 1]);
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
                    if (!(ok = wait(&full[(c + 1) % kStages], (c + 1) / kStages) && (c == 0 || wait(&a_free[(c + 1) & 1], (c - 1) >> 1)))) break;
                    ptx::tc_fence_after();
                    logits(c + 1);
                }
                // U^T = (w V)^T K
                if (STATES && !(ok = wait(&full[c % kStages], c / kStages))) break;
                if (!(ok = c < kUs || wait(&u_free[c % kUs], c / kUs - 1))) break;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = wait(&v_full[half], c))) break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
#pragma unroll 1
                        for (int part = 0; part < C::kParts; ++part)
#pragma unroll
                            for (int k = 2 * half; k < 2 * half + 2; ++k)
                                ptx::mma_f16_ss(tmem + C::kColU + c % kUs * 128, desc_mn + at(C::kValues + part * C::kPartBytes + k * 2048),
                                                desc_mn + at(stage + C::kK + k * 2048), idesc_u, part > 0 || k > 0);
                        ptx::mma_commit(&v_free[half]);
                        if (half == 1) {
                            ptx::mma_commit(&u_full[c % kUs]);
                            ptx::mbar_arrive(&u_full[c % kUs]);
                            if (STATES) ptx::mma_commit(&empty[c % kStages]);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (STATES) continue;
                // O1^T = S0^T Q^T
                if (!(ok = wait(s_full, c) && (c == 0 || wait(o_free, c - 1)))) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
#pragma unroll 1
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
#pragma unroll 1
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
        if (issued > 0 && lane == 0) {  // copies under way land before the shared memory is given up
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
    static std::atomic<bool> ready[64];  // of each device: the shared-memory opt-in
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const int64_t places = segment_base(a.n_tokens, a.n_seqs, a.segment_chunks, a.place_tokens), blocks = places * a.VH * (a.DV / DV);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    LaunchScope scope(STATES ? KC_LINEAR_STATES : KC_LINEAR_CHUNKS, s);
    kernel<<<(unsigned)blocks, kThreads, smem, s>>>(a, m);
    return cudaGetLastError();
}

template <int DK, int DV, bool F16>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
    Maps m;
    if (!encode_tmap_blocks(&m.q, a.q, a.n_tokens, (uint64_t)a.KH * DK, a.q_ld, kChunk, DK / 64) ||
        !encode_tmap_blocks(&m.k, a.k, a.n_tokens, (uint64_t)a.KH * DK, a.k_ld, kChunk, DK / 64) ||
        !encode_tmap_blocks(&m.v, a.v, a.n_tokens, (uint64_t)a.VH * a.DV, a.v_ld, kChunk, DV / 64))
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
