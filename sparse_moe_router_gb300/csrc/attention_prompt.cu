// attention_prompt.cu -- attention over the paged 8-bit cache for runs of many new tokens, on the
// 5th-generation tensor cores (tcgen05, TMEM).
//
// A block takes 256 query rows (token, q head) of one kv head as two 128-row tiles (one at D = 256,
// where the output of one fills TMEM) and walks the keys they see in tiles of 128.  In halves of 64
// keys a row tile computes S = Q K^T into TMEM, the softmax takes S into registers at once and puts
// the weights back as fp16, and O += P V reads them from there, while the next half's logits are
// computed.  All rows of a group of q heads share each key and value tile, so a tile of K and V
// is widened once for 256 rows.
//
// Bound: 4 D flops a (row, key) on the tensor cores; at D = 128 a tile of keys is 4 x 512 tensor
// cycles for the two row tiles, and their 2 x 16,384 exponentials take 1024 cycles at the SM's 32 a cycle,
// so both have to run at once: logits ahead, two row tiles apart.  The 8-bit codes cannot be an operand
// beside fp16 weights (both operands of an MMA have one type, and queries in 8 bits would lose what
// the 16-bit ones hold), so eight warps read codes from global memory (L2, mostly: all tiles of a head
// read the same pages), widen them exactly to fp16 and store them in the swizzled layout that the MMA
// reads.  At 128 bytes a cycle those 64 KB and the operands (6 KB an MMA of 64 keys' logits, 4 KB of the output)
// take 2560 cycles a tile of keys: at D = 128 shared memory is the nearer limit, and 3500 are measured.  What is
// between is the chain of each half tile (wait, TMEM load, weights, TMEM store, MMAs, each a few hundred
// cycles): leaving out the exponentials gives 2% at D = 128 and 9% at D = 64, the widening 7% and 6%, 7/8 of the
// logits' MMAs 10% and 0.
//
// Scales: the exponents of the pages are drawn into the codes relative to the largest that the block meets, exactly (the
// least code is 2^-9, fp16's least value 2^-24, so 2^15 apart is the most), and one factor a row holds for all keys.  A block
// whose pages lie further apart, one of all zeros or one with an infinity among them, leaves the codes as they are: the
// softmax then goes by 16 keys, which share a page, with the key scale in the factor of the logits and the
// value's exponent in the weights, z = S 2^ek c + ev, w = 2^(z - m), the row's sum taking w 2^-ev.  The converters, which look the
// pages up anyway, hand the scales over in shared memory.  So a row's result does not depend on pages that it does
// not see.  (A page of zeros in each sequence: the five pieces below 82.4 us instead
// of 70.8, 8192 tokens 218.5 instead of 200.7.)
//
// Parts: where the blocks leave SMs idle, several share one's keys, and the rows' parts are joined by a second
// kernel (a warp a row, all parts' loads at once).  8 q heads and 1 kv head of 128 dims, 16,384 keys: 128
// tokens 31 us, 512 44, 1024 72, where one block for all keys takes 200.
//
// Measured, causal: 8192 tokens, 16 q heads and 2 kv heads of 128 dims 201 us (1368 TFLOP/s, 73% of the
// cuBLAS rate measured here, 80% of the sustained one); of 64 dims 161 us (851); 16 and 4 heads of 256
// 519 us (1060), where the split kernel takes 4635; five pieces of up to 1031 tokens behind up to 6007, 24 q heads in groups of 3 of
// 64 dims, 70.6 us (its 152 blocks run at once, and the longest has 1.3 times the mean's keys).  On the way, each against the kernel of its time, at
// D = 128: whole tiles of logits in the place their weights take 214 us; halves from one MMA warp 284 (its waits
// for one row tile hold up the other); two threads a row 232 (a barrier a half tile); four converter warps 277; the
// maximum looked for in every tile 221; scalar instead of paired fp32 in the softmax 219; the next logits
// loaded before the weights are stored 233 (registers).
//
// Roles: warps 0-3 and 4-7 do the softmax of row tiles 0 and 1, one row a thread; warps 8-15 widen K
// and V; warps 16 and 17 issue the MMAs of row tiles 0 and 1 (with kAhead their logits, and 18 and 19
// their outputs).  A row's maximum is not looked for in
// every tile: the weights are taken under the reference so far, and their sum (needed anyway) shows when that
// has become too small; the row's thread then finds the maximum, rescales its row of O and takes the
// weights again.
#include "layer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRowTile = 128;
constexpr int kKeys = 128;  // keys a tile
constexpr int kSoftWarps = 8, kConvWarps = 8, kMmaWarp = 16;
constexpr int kThreads = 20 * 32;
// Registers a thread: 96 at launch (five warps a scheduler); of a scheduler's 5 x 96 the two softmax
// warps, which hold 64 logits and 32 pairs of weights, take 2 x 144, the converters 2 x 80, an MMA warp 32.
constexpr int kLaunchRegs = 96, kSoftRegs = 144, kConvRegs = 80, kMmaRegs = 32;
static_assert(8 * kSoftRegs + 8 * kConvRegs + 4 * kMmaRegs <= 20 * kLaunchRegs, "more registers than the block has");
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far above any legitimate wait
constexpr int kPartTiles = 8;  // key tiles of a part (of 8: 11 us at D = 128), about and at least
constexpr float kMostSum = 65504.f;  // 64 weights of one row may add up to this: fp16's largest value (64 equal ones: 32,768)

// Most that the exponents of a block's pages may differ by to go into the codes: of the keys what is exact, of the values
// less, as a weight is then rounded in units of the row's largest whatever its value's scale.
constexpr int kKeyShift = 15, kValueShift = 8;
// Scales of the 8 times 16 keys of a tile: factors of the keys, exponents of the values and 2^-those, of the last 4
// tiles.  A tile's place is written once the logits of the tile two before (D = 256: one) are done, which begin
// once the weights of the half tile before them are; so whatever still reads is at most 3 tiles behind.
constexpr int kScaleTiles = 4, kScaleFloats = 24, kScaleBytes = kScaleTiles * kScaleFloats * 4;
template <bool B>
struct Flag {
    static constexpr bool value = B;
};

template <int D>
struct Prompt {
    static constexpr int kBlocks = D / 64;                    // 128-byte column blocks of a row
    static constexpr int kBlockBytes = kKeys * 128;           // one column block of a 128-row tile
    static constexpr int kTileBytes = kBlocks * kBlockBytes;  // a tile of Q, K or V
    static constexpr int kTiles = D == 256 ? 1 : 2;           // row tiles a block: TMEM holds one output of 256 dims
    static constexpr int kRows = kTiles * kRowTile;
    static constexpr int kStages = D == 256 ? 2 : 4;          // K and V tiles in flight, in the order K0 V0 K1 V1 ...
    // 1 KB to align; barriers; scales; whether the block writes the output
    static constexpr int kSmem = 1024 + (kTiles + kStages) * kTileBytes + 256 + kScaleBytes + 16;
    static constexpr uint32_t kColO = kTiles * kKeys;         // TMEM: S0 (S1) O0 (O1); S of even and odd halves
    static constexpr uint32_t kCols = 512;
    // Where a half tile's 64 logits and 64 weights (fp16: 32 columns) lie among a row tile's 128 columns, and
    // how far the logits run ahead.  D = 64 and 256, where the softmax sets the pace: two places for logits, the
    // weights in theirs, logits two half tiles ahead from a warp of their own.  D = 128, where the tensor cores and
    // their operands' reads do (64-column logits read 6 KB a 32 cycles): one place for logits and two for weights,
    // one warp for both, so that a row tile's next logits always come before its output.  us with the first
    // form and the second: 8192 tokens at D = 64 (8 q heads a kv head) 162 and 167, at D = 128 207 and 202, at
    // D = 256 510 and 597; five pieces at D = 64 69.5 and 73.6.  (The second with two warps at D = 128: 214.)
    static constexpr bool kAhead = D != 128;
    __device__ static uint32_t s_place(int n) { return kAhead ? (n & 1) * 64 : 0; }
    __device__ static uint32_t p_place(int n) { return kAhead ? (n & 1) * 64 : 64 + (n & 1) * 32; }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ int exponent_of(float s) { return (int)((__float_as_uint(s) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t f) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Values read from TMEM are used only past this point (after the wait that completes the read).
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k]));
}
// A factor of logits that is small beyond fp32 (a tiny query over a tiny page): the logits are 0 either way, but
// masked ones, -infinity before the factor, have to stay it.
__device__ __forceinline__ float positive(float x) { return fmaxf(x, 1.17549435e-38f); }
// a * b + c on two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
    return __ffma2_rn(a, make_float2(b, b), make_float2(c, c));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
template <int R>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Block (slot, head): sequence b owns slots base(b) .. base(b+1)-1 of R rows each of every head, with
// base(b) = q_start[b] G / R + b (its n G rows need at most n G / R + 1 of them).
template <int R>
__device__ __forceinline__ int slot_base(const KvView &v, int b) {
    return (int)((int64_t)v.q_start[b] * v.G / R) + b;
}

// Keys that any of a block's rows sees, in tiles, and how many parts of so many tiles they are worked on in.  The
// host's p.parts goes by what the table can name; a sequence that is shorter has fewer, down to one block that writes
// the output itself (512 tokens of 16 q and 2 kv heads of 128 without a past: 17.0 us in a table of 512, 20.5 in one for 131,072, and
// 35.6 with parts by the table).
struct BlockKeys {
    int lo, hi, tile0, tiles, parts, share;
};
__device__ __forceinline__ BlockKeys block_keys(const AttnArgs &p, const Seq &q, int row0, int rows) {
    BlockKeys k;
    const int first_pos = q.kv - q.n, pos_lo = first_pos + row0 / p.kv.G, pos_hi = first_pos + (row0 + rows - 1) / p.kv.G;
    k.hi = p.causal ? min(q.kv, pos_hi + 1) : q.kv;
    k.lo = p.window > 0 ? max(0, pos_lo + 1 - p.window) : 0;
    k.tile0 = k.lo / kKeys;
    k.tiles = k.hi > k.lo ? (k.hi + kKeys - 1) / kKeys - k.tile0 : 0;
    k.parts = min(p.parts, max((k.tiles + kPartTiles / 2) / kPartTiles, 1));
    k.share = (k.tiles + k.parts - 1) / k.parts;
    if (k.tiles > 0) k.parts = (k.tiles + k.share - 1) / k.share;
    return k;
}

template <int D, bool F16, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ AttnArgs p, int slots) {
    using C = Prompt<D>;
    constexpr int kStages = C::kStages, kTiles = C::kTiles, kRows = C::kRows;
    const KvView &v = p.kv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *q_smem = smem, *kv_smem = smem + kTiles * C::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(kv_smem + kStages * C::kTileBytes);
    uint64_t *full = bars, *empty = bars + kStages;  // of a stage
    uint64_t *s_full = empty + kStages;              // [2 x 2] 64 logits of a row tile, even and odd half tiles, are in TMEM
                                                     // (and their keys' scales in shared memory)
    uint64_t *p_full = s_full + 4;                   // [2 x 2] and their weights are, in their place
    uint64_t *o_half = p_full + 4;                   // [2 x 2] and have gone into the output
    uint64_t *o_full = o_half + 4;                   // [2] all have
    uint64_t *s_free = o_full + 2;                   // [2] the logits are in registers
    uint64_t *q_full = s_free + 2;
    uint64_t *drain = q_full + 1;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *max_exp = reinterpret_cast<int *>(tmem_holder + 2);              // [4] largest of K and V, smallest negated
    float *scales = reinterpret_cast<float *>(kv_smem + kStages * C::kTileBytes + 256);
    volatile int *in_parts = reinterpret_cast<int *>(scales + kScaleTiles * kScaleFloats);

    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the split kernel does not depend on this one)

    // ------------------------------------------------------------------- the block's rows --
    // Blocks begin in the order of their number, so the ones with most keys come first: of up to 32 sequences the
    // longest, and of each its last rows (a causal row sees the more the later it is).
    const int head = (int)blockIdx.x % v.KH;
    int b, row0;
    if (v.n_seqs <= 32) {
        Seq own{0, 0, 0};
        if (lane < v.n_seqs) own = load_seq(v, lane);
        const int64_t own_rows = (int64_t)own.n * v.G;
        const int count = own_rows >= p.prompt_rows ? (int)((own_rows + kRows - 1) / kRows) : 0;
        int base = 0;  // blocks of the sequences before this lane's
        for (int c = 0; c < v.n_seqs; ++c) {
            const int kv = __shfl_sync(0xffffffffu, own.kv, c), n = __shfl_sync(0xffffffffu, count, c);
            if (kv > own.kv || (kv == own.kv && c < lane)) base += n;
        }
        const int slot = (int)blockIdx.x / v.KH;
        const uint32_t mine = __ballot_sync(0xffffffffu, slot >= base && slot < base + count);
        if (mine == 0) return;
        b = __ffs(mine) - 1;
        row0 = (__shfl_sync(0xffffffffu, base + count, b) - 1 - slot) * kRows;
    } else {
        const int slot = slots - 1 - (int)blockIdx.x / v.KH;
        int lo_b = 0, hi_b = v.n_seqs - 1;
        while (lo_b < hi_b) {
            const int mid = (lo_b + hi_b + 1) >> 1;
            if (slot_base<kRows>(v, mid) <= slot) lo_b = mid; else hi_b = mid - 1;
        }
        b = lo_b;
        row0 = (slot - slot_base<kRows>(v, b)) * kRows;
    }
    const Seq q = load_seq(v, b);
    const int rows = min(kRows, q.n * v.G - row0);
    if (row0 < 0 || rows <= 0 || q.n * v.G < p.prompt_rows) return;  // (short runs are the split kernel's)
    const int first_pos = q.kv - q.n;
    const BlockKeys all = block_keys(p, q, row0, rows);
    int key_lo = all.lo, key_hi = all.hi, tile0 = all.tile0, tiles = all.tiles;
    if (PARTS) {  // this block's part of them
        if ((int)blockIdx.y >= all.parts) {  // the join takes -infinity for no such part
            const int tok = q.q0 + (row0 + tid) / v.G, qh = head * v.G + (row0 + tid) % v.G;
            if (tid < rows) p.part_lse[((int64_t)blockIdx.y * v.n_tokens + tok) * v.QH + qh] = -INFINITY;
            return;
        }
        tile0 += (int)blockIdx.y * all.share;
        tiles = min(all.share, tiles - (int)blockIdx.y * all.share);
        key_lo = max(key_lo, tile0 * kKeys);
        key_hi = min(key_hi, (tile0 + tiles) * kKeys);
    }
    const int halves = tiles > 0 ? (key_hi - tile0 * kKeys + 63) / 64 : 0;  // half tiles of 64 keys
    const int32_t *table = v.table + (int64_t)b * v.max_pages;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], kConvWarps);
            ptx::mbar_init(&empty[s], kTiles);  // every row tile is done with it
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s_full[2 * i], 2);  // the MMAs' end, and the arrival of the warp that has seen the scales
            ptx::mbar_init(&s_full[2 * i + 1], 2);
            ptx::mbar_init(&p_full[2 * i], 4);
            ptx::mbar_init(&p_full[2 * i + 1], 4);
            ptx::mbar_init(&o_half[2 * i], 1);
            ptx::mbar_init(&o_half[2 * i + 1], 1);
            ptx::mbar_init(&o_full[i], 1);
            ptx::mbar_init(&s_free[i], 4);
        }
        ptx::mbar_init(q_full, 4 * kTiles);
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&drain[i], 1);
        *abort_flag = 0;
        *in_parts = PARTS && all.parts > 1;
        for (int i = 0; i < 4; ++i) max_exp[i] = -200;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) ptx::tmem_alloc(tmem_holder, C::kCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // the largest and smallest exponents among the pages that a row of the block sees
    {
        int e[4] = {-200, -200, -200, -200};
        const int pages0 = key_lo >> v.log_p, pages1 = (key_hi + v.P - 1) >> v.log_p;
        for (int i = pages0 + tid; tiles > 0 && i < pages1; i += kThreads) {
            int page = __ldg(table + i);
            if (page < 0 || page >= v.n_pages) {
                layer_error(v.status);
                page = 0;
            }
            const int ek = exponent_of(__ldg(v.k_scale + (int64_t)page * v.KH + head));
            const int ev = exponent_of(__ldg(v.v_scale + (int64_t)page * v.KH + head));
            e[0] = max(e[0], ek), e[1] = max(e[1], ev), e[2] = max(e[2], -ek), e[3] = max(e[3], -ev);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __reduce_max_sync(0xffffffffu, e[i]);
        if (lane < 4) atomicMax(&max_exp[lane], lane == 0 ? e[0] : lane == 1 ? e[1] : lane == 2 ? e[2] : e[3]);
    }
    __syncthreads();
    // Read where they are needed: in registers over the softmax they cost 4% at D = 64.
    struct Exps {
        int k, v;
        bool by16;
    };
    auto exps = [&]() {
        const volatile int *e = max_exp;
        const int k = e[0], v = e[1];
        return Exps{k, v, k + e[2] > kKeyShift || v + e[3] > kValueShift};
    };
    bool ok = true;

    if (warp < kSoftWarps) {
        regs_up<kSoftRegs>();
        if (warp < 4 * kTiles) {
        // ---------------------------------------------------------------------- softmax --
        // Thread t has row t of the block: lane t % 128 of row tile t / 128.
        const int i = warp >> 2, r = tid, rr = r & (kRowTile - 1);
        const bool live = r < rows;
        const int tok = (row0 + r) / v.G, qh = head * v.G + (row0 + r) % v.G;
        const int pos = first_pos + tok;
        const int hi = min(p.causal ? min(q.kv, pos + 1) : q.kv, key_hi);
        const int lo = max(p.window > 0 ? max(0, pos + 1 - p.window) : 0, key_lo);
        const bool sees = live && hi > lo;
        // Q: the row scaled by a power of two into [1, 2) at its largest, as fp16, K-major swizzled
        int q_exp;
        {
            const uint16_t *src = p.q + (int64_t)(q.q0 + tok) * p.q_ld + (int64_t)qh * D;
            uint8_t *dst = q_smem + i * C::kTileBytes + rr * 128;
            constexpr int kHeld = D < 256 ? D / 8 : 16;  // pieces kept in registers; a wide row is read twice
            uint4 qv[kHeld];
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                if (c % kHeld == 0) {
#pragma unroll
                    for (int x = 0; x < kHeld; ++x)
                        qv[x] = live ? __ldg(reinterpret_cast<const uint4 *>(src + (c + x) * 8)) : make_uint4(0, 0, 0, 0);
                }
                float f[8];
                unpack8<F16>(qv[c % kHeld], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
            }
            q_exp = amax > 0.f ? max(min((int)(__float_as_uint(amax) >> 23) - 127, 126), -126) : 0;
            const float q_inv = pow2f(-q_exp);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                if (D / 8 > kHeld && c % kHeld == 0) {
#pragma unroll
                    for (int x = 0; x < kHeld; ++x)
                        qv[x] = live ? __ldg(reinterpret_cast<const uint4 *>(src + (c + x) * 8)) : make_uint4(0, 0, 0, 0);
                }
                float f[8];
                unpack8<F16>(qv[c % kHeld], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= q_inv;
                *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kBlockBytes + (((c & 7) ^ (rr & 7)) << 4)) = pack8<true>(f);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full);
        }
        const Exps pages = exps();
        const float q_mul = p.scale_log2 * pow2f(q_exp), mul = pages.by16 ? q_mul : positive(q_mul * pow2f(pages.k));
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_addr = tmem + lanes + C::kColO + i * D;
        float m = 0.f, l = 0.f;  // reference of the weights, and their sum (0: none so far)
        auto walk = [&](auto flag) {
        constexpr bool kBy16 = decltype(flag)::value;
        for (int n = 0; n < halves; ++n) {
            ok = __all_sync(0xffffffffu, ptx::mbar_wait(&s_full[2 * i + (n & 1)], n >> 1 & 1, kWaitNs, abort_flag)) != 0;
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t s_addr = tmem + lanes + i * kKeys + C::s_place(n);
            uint32_t s[2][32], w[32];
            ptx::tmem_ld_32(s_addr, s[0]);
            ptx::tmem_ld_32(s_addr + 32, s[1]);
            ptx::tmem_ld_wait();
            tie32(s[0]);
            tie32(s[1]);
            if (!C::kAhead) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&s_free[i]);
            }
            const int key0 = tile0 * kKeys + n * 64, c_lo = lo - key0, c_hi = hi - key0;
            if (__any_sync(0xffffffffu, live && (c_lo > 0 || c_hi < 64))) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c * 32 + k < c_lo || c * 32 + k >= c_hi) s[c][k] = 0xff800000u;  // -inf
            }
            // The sum of the weights itself tells when the reference is too small: as long as it stays within
            // kMostSum every weight fits fp16.  Only then (and where a row begins) is the maximum looked for.
            const float *c16 = scales + (n >> 1) % kScaleTiles * kScaleFloats + (n & 1) * 4;  // with kBy16
            float add = 0.f;                                                                  // what the weights add to l
            auto weights = [&]() {
                float2 sum = make_float2(0.f, 0.f);
                if constexpr (!kBy16) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 z =
                                fma2(make_float2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), mul, -m);
                            const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                            sum = __fadd2_rn(sum, e);
                            w[c * 16 + k] = pack2<true>(e.x, e.y);
                        }
                    return add = sum.x + sum.y;
                } else {
                    float all = 0.f;
                    add = 0.f;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float factor = positive(mul * c16[g]), offset = c16[8 + g] - m;
                        sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t *x = s[g >> 1] + (g & 1) * 16 + 2 * k;
                            const float2 z = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), factor, offset);
                            const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                            sum = __fadd2_rn(sum, e);
                            w[g * 8 + k] = pack2<true>(e.x, e.y);
                        }
                        all += sum.x + sum.y;
                        add = fmaf(sum.x + sum.y, c16[16 + g], add);
                    }
                    return all;
                }
            };
            bool renew = __any_sync(0xffffffffu, l == 0.f && sees);
            if (!renew) renew = __any_sync(0xffffffffu, !(weights() <= kMostSum));
            if (renew) {
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint32_t *x = s[g >> 1] + (g & 1) * 16;
                    float t = kBy16 ? -INFINITY : top;
#pragma unroll
                    for (int k = 0; k < 16; k += 2) t = max3(t, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                    top = kBy16 ? fmaxf(top, fmaf(t, positive(mul * c16[g]), c16[8 + g])) : t;
                }
                top = (kBy16 ? top : top * mul) - kBelowTop;  // mul > 0
                float f = 1.f;
                if (l == 0.f) {
                    m = top == -INFINITY ? 0.f : top;
                } else if (top > m) {
                    f = exp2_fast(m - top);
                    m = top;
                }
                l *= f;
                if (n > 0) {  // O under the old reference, once the product of the half tile before is in it
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(&o_half[2 * i + ((n - 1) & 1)], (n - 1) >> 1 & 1, kWaitNs, abort_flag)) != 0;
                    ptx::tc_fence_after();
                    uint32_t o[16];
                    constexpr int kUnroll = D == 256 ? 1 : D / 16;  // (16 addresses would be kept over the whole loop)
#pragma unroll kUnroll
                    for (int c = 0; c < D / 16; ++c) {
                        ptx::tmem_ld_16(o_addr + c * 16, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            asm volatile("" : "+r"(o[k]));
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        }
                        ptx::tmem_st_16(o_addr + c * 16, o);
                    }
                }
                weights();
            }
            l += add;
            ptx::tmem_st_32(tmem + lanes + i * kKeys + C::p_place(n), w);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            // (a barrier for even and one for odd: a warp may be a half tile ahead of another)
            if (lane == 0) ptx::mbar_arrive(&p_full[2 * i + (n & 1)]);
            if (!ok) break;
        }
        };
        if (pages.by16) walk(Flag<true>{});
        else walk(Flag<false>{});
        // ---------------------------------------------------------------- output, normalised --
        if (ok && tiles > 0) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&o_full[i], 0, kWaitNs, abort_flag)) != 0;
        if (ok) {
            ptx::tc_fence_after();
            const Exps pages = exps();
            const float unit = pages.by16 ? 1.f : pow2f(pages.v);
            const float inv = (l > 0.f || l != l) && tiles > 0 ? unit / l : 0.f;
            uint16_t *out = p.out + (int64_t)(q.q0 + tok) * p.out_ld + (int64_t)qh * D;
            const int64_t row = ((int64_t)blockIdx.y * v.n_tokens + q.q0 + tok) * v.QH + qh;  // among the parts'
            const bool part = PARTS && *in_parts != 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (tiles > 0) {
                    ptx::tmem_ld_32(o_addr + c * 32, o);
                    ptx::tmem_ld_wait();
                    tie32(o);
                }
#pragma unroll
                for (int k = 0; k < 4 && live; ++k) {
                    float f[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] = inv == 0.f ? 0.f : __uint_as_float(o[8 * k + x]) * inv;
                    if (part) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_out + row * D + c * 32 + k * 8);
                        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                        dst[1] = make_float4(f[4], f[5], f[6], f[7]);
                    } else {
                        *reinterpret_cast<uint4 *>(out + c * 32 + k * 8) = pack8<F16>(f);
                    }
                }
            }
            if (live && PARTS) p.part_lse[row] = part ? m + log2f(l) : INFINITY;  // infinity: the output is written
            if (live && !part && p.lse) p.lse[(int64_t)(q.q0 + tok) * v.QH + qh] = (m + log2f(l)) * 0.6931471805599453f;
        }
        }
    } else if (warp < kMmaWarp) {
        regs_down<kConvRegs>();
        // ------------------------------------------------------------- K and V, widened --
        // Warp w owns keys 16 w .. 16 w + 15 of every tile: they lie in one page.  A load takes whole rows
        // (2 of 256 codes, 4 of 128, 8 of 64), so that it reads full lines, 16 codes a lane; lanes are laid
        // out so that each 8 of them hold 4 pieces of two neighbouring rows, whose 16-byte stores fall on
        // all the banks.  The registers of a tile's codes take the next tile's as soon as they are
        // widened, so a load has a whole tile's time to arrive (at D = 256, where K and V take turns in
        // the same registers, half of it).
        constexpr int kRowsLoad = 512 / D, kLoads = 16 / kRowsLoad;
        const int cw = warp - kSoftWarps;
        const int piece = D == 256 ? (lane >> 3 << 2) | (lane & 3) : D == 128 ? (lane >> 1 & 4) | (lane & 3) : lane & 3;
        const int sub = D == 256 ? lane >> 2 & 1 : D == 128 ? (lane >> 3 & 2) | (lane >> 2 & 1) : lane >> 2;
        auto page_at = [&](int tile) {  // page * KH + head
            const int key = (tile0 + tile) * kKeys + cw * 16;
            int page = 0;
            if (key < key_hi) page = __ldg(table + (key >> v.log_p));
            return (page < 0 || page >= v.n_pages ? 0 : page) * v.KH + head;  // (reported above)
        };
        const Exps pages = exps();
        const bool by16 = pages.by16;
        auto factor = [&](float scale, int largest) {  // 2^(exponent - the block's largest)
            const int e = by16 ? 0 : min(exponent_of(scale) - largest, 0);  // (keys not looked up: any page)
            const __half2 f = __float2half2_rn(e < -kKeyShift ? 0.f : pow2f(e));
            return *reinterpret_cast<const uint32_t *>(&f);
        };
        const int log_pd = v.log_p + (D == 256 ? 8 : D == 128 ? 7 : 6);
        auto load = [&](uint4 (&raw)[kLoads], int tile, int page, const uint8_t *codes, int end) {
            const int key0 = (tile0 + tile) * kKeys + cw * 16;
            const uint8_t *src = codes + ((uint64_t)(uint32_t)page << log_pd) + ((key0 & (v.P - 1)) + sub) * D + piece * 16;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                raw[n] = make_uint4(0, 0, 0, 0);
                if (key0 + n * kRowsLoad + sub < end)  // slots past the end hold anything
                    raw[n] = load_codes16(src + n * kRowsLoad * D);
            }
        };
        // offsets of a piece's two stores in the rows of the first load; later loads' rows differ in their upper bits
        const uint32_t base = (uint32_t)(piece >> 2) * C::kBlockBytes + (uint32_t)(cw * 16 + sub) * 128;
        const uint32_t c0 = ((2 * (piece & 3)) ^ sub) << 4, c1 = c0 ^ 16u;
        auto widen = [&](const uint4 (&raw)[kLoads], int it, uint32_t f) {
            uint8_t *st = kv_smem + it % kStages * C::kTileBytes + base;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const uint32_t w[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
                uint32_t h[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    widen4(w[k], h[2 * k], h[2 * k + 1]);
                    h[2 * k] = mul2(h[2 * k], f);
                    h[2 * k + 1] = mul2(h[2 * k + 1], f);
                }
                const uint32_t flip = (n * kRowsLoad & 7) << 4;  // of the swizzle
                uint8_t *dst = st + n * kRowsLoad * 128;
                *reinterpret_cast<uint4 *>(dst + (c0 ^ flip)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(dst + (c1 ^ flip)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
        };
        auto free_stage = [&](int it) {
            bool f = it < kStages || ptx::mbar_wait(&empty[it % kStages], (it / kStages - 1) & 1, kWaitNs, abort_flag);
            return __all_sync(0xffffffffu, f) != 0;
        };
        auto publish = [&](int it) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&full[it % kStages]);
        };
        constexpr bool kBoth = D < 256;
        uint4 rk[kLoads], rv[kBoth ? kLoads : 1];
        // In the first tile 16 keys may lie before all that the rows see: their page may be gone and is not looked up.
        const bool gone = tile0 * kKeys + cw * 16 + 16 <= key_lo;
        const int first_end = gone ? 0 : key_hi;
        int end = first_end;  // of the keys of the tile in hand (at D = 256 by its number: 518 us instead of 528)
        int page1 = gone ? head : page_at(0), page2 = page_at(1);
        float sk = __ldg(v.k_scale + page1), sv = __ldg(v.v_scale + page1);
        if (tiles > 0) {
            load(rk, 0, page1, v.k_codes, end);
            if constexpr (kBoth) load(rv, 0, page1, v.v_codes, end);
        }
        for (int j = 0; j < tiles; ++j) {
            const uint32_t fk = factor(sk, pages.k), fv = factor(sv, pages.v);
            const int ek = exponent_of(sk), ev = exponent_of(sv);
            const int page0 = page1;
            page1 = page2;  // of tile j + 1
            sk = __ldg(v.k_scale + page1), sv = __ldg(v.v_scale + page1);
            page2 = page_at(j + 2);
            if (!(ok = free_stage(2 * j))) break;
            if (by16 && lane == 0) {  // (not looked up: 1)
                const bool in = (tile0 + j) * kKeys + cw * 16 < (kBoth ? end : j == 0 ? first_end : key_hi);
                float *sc = scales + j % kScaleTiles * kScaleFloats + cw;
                sc[0] = in ? pow2f(ek) : 1.f, sc[8] = in ? (float)ev : 0.f, sc[16] = in ? pow2f(-ev) : 1.f;
            }
            widen(rk, 2 * j, fk);
            if constexpr (kBoth) {
                if (j + 1 < tiles) load(rk, j + 1, page1, v.k_codes, key_hi);
                publish(2 * j);
                if (!(ok = free_stage(2 * j + 1))) break;
                widen(rv, 2 * j + 1, fv);
                if (j + 1 < tiles) load(rv, j + 1, page1, v.v_codes, key_hi);
            } else {
                load(rk, j, page0, v.v_codes, j == 0 ? first_end : key_hi);
                publish(2 * j);
                if (!(ok = free_stage(2 * j + 1))) break;
                widen(rk, 2 * j + 1, fv);
                if (j + 1 < tiles) load(rk, j + 1, page1, v.k_codes, key_hi);
            }
            publish(2 * j + 1);
            if constexpr (kBoth) end = key_hi;
        }
    } else {
        regs_down<kMmaRegs>();
        const int i = warp & 1;
        if (i < kTiles && (C::kAhead || warp < kMmaWarp + 2) && tiles > 0) {
            // ------------------------------------------------------------------ the MMAs --
            // A warp for each row tile: the next 64 logits as soon as the last are in registers, then the output of
            // the last's weights.
            const uint32_t idesc_s = ptx::idesc_f16_f32(kRowTile, 64, false);
            const uint32_t idesc_o = ptx::idesc_f16_f32(kRowTile, D, true);
            const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(q_smem));
            const uint64_t k_desc = ptx::sw128_desc(ptx::smem_u32(kv_smem));
            const uint64_t v_desc = ptx::sw128_desc_mn(ptx::smem_u32(kv_smem), C::kBlockBytes);
            auto wait = [&](uint64_t *bar, int parity) {
                return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity & 1, kWaitNs, abort_flag)) != 0;
            };
            auto logits = [&](int n) {  // S = Q K^T for the 64 keys of half tile n
                const int s = n / 2 * 2 % kStages;
                if (ptx::elect_one()) {
                    const uint64_t qd = q_desc + (uint64_t)(i * (C::kTileBytes >> 4));
                    const uint64_t kd = k_desc + (uint64_t)(s * (C::kTileBytes >> 4) + (n & 1) * (64 * 128 >> 4));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        constexpr int kBlock16 = C::kBlockBytes >> 4;
                        const int off = (k >> 2) * kBlock16 + (k & 3) * 2;
                        ptx::mma_f16_ss(tmem + i * kKeys + C::s_place(n), qd + off, kd + off, idesc_s, k > 0);
                    }
                    ptx::mma_commit(&s_full[2 * i + (n & 1)]);
                    ptx::mbar_arrive(&s_full[2 * i + (n & 1)]);
                    if ((n & 1) || n + 1 == halves) ptx::mma_commit(&empty[s]);
                }
                __syncwarp();
            };
            auto output = [&](int n) {  // O += P V
                const int s = (n / 2 * 2 + 1) % kStages;
                if (ptx::elect_one()) {
                    const uint64_t vd = v_desc + (uint64_t)(s * (C::kTileBytes >> 4) + (n & 1) * (64 * 128 >> 4));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        ptx::mma_f16_ts(tmem + C::kColO + i * D, tmem + i * kKeys + C::p_place(n) + k * 8,
                                        vd + k * (2048 >> 4), idesc_o, n > 0 || k > 0);
                    ptx::mma_commit(&o_half[2 * i + (n & 1)]);
                    if ((n & 1) || n + 1 == halves) ptx::mma_commit(&empty[s]);
                    if (n + 1 == halves) ptx::mma_commit(&o_full[i]);
                }
                __syncwarp();
            };
            auto filled = [&](int it) { return wait(&full[it % kStages], it / kStages); };
            if (!C::kAhead) {
                ok = wait(q_full, 0) && filled(0);
                ptx::tc_fence_after();
                if (ok) logits(0);
                for (int n = 0; n < halves && ok; ++n) {
                    if (n + 1 < halves) {
                        ok = (!(n & 1) || filled(n + 1)) && wait(&s_free[i], n);  // K of the next tile
                        ptx::tc_fence_after();
                        if (ok) logits(n + 1);
                    }
                    ok = ok && ((n & 1) || filled(n + 1)) && wait(&p_full[2 * i + (n & 1)], n >> 1);  // V of this one
                    ptx::tc_fence_after();
                    if (ok) output(n);
                }
            } else if (warp < kMmaWarp + 2) {
                ok = wait(q_full, 0) && filled(0);
                ptx::tc_fence_after();
                for (int n = 0; n < halves && ok; ++n) {
                    if (n > 1) {  // K; the weights whose place the logits take have been read
                        ok = ((n & 1) || filled(n)) && wait(&o_half[2 * i + (n & 1)], (n - 2) >> 1);
                        ptx::tc_fence_after();
                    }
                    if (ok) logits(n);
                }
            } else {
                for (int n = 0; n < halves && ok; ++n) {
                    ok = ((n & 1) || filled(n + 1)) && wait(&p_full[2 * i + (n & 1)], n >> 1);  // V, weights
                    ptx::tc_fence_after();
                    if (ok) output(n);
                }
            }
            if (!ok) {  // nothing of this block may still run when its TMEM is freed
                if (ptx::elect_one()) ptx::mma_commit(&drain[warp - kMmaWarp]);
                int zero = 0;
                ptx::mbar_wait(&drain[warp - kMmaWarp], 0, kWaitNs, &zero);
            }
        }
    }
    if (!ok) {
        *abort_flag = 1;
        atomicCAS(v.status, 0, (int)MOE_ERR_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, C::kCols);
}

// Joins the parts of each row that has several, a warp a row (up to 32 sequences).  Parts in which a row sees nothing, or
// that there are not, have -infinity and are not read.
template <int D, bool F16>
__global__ void __launch_bounds__(256) attn_prompt_join_kernel(const __grid_constant__ AttnArgs p) {
    const KvView &v = p.kv;
    const int lane = (int)threadIdx.x & 31;
    const int64_t rows = (int64_t)v.n_tokens * v.QH, row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int tok = (int)(row / v.QH), qh = (int)(row % v.QH);
    const float lse = lane < p.parts ? p.part_lse[lane * rows + row] : -INFINITY;
    const uint32_t there = __ballot_sync(0xffffffffu, lse != -INFINITY);
    if (__shfl_sync(0xffffffffu, lse, 0) == INFINITY) return;  // one part: its block has written the row
    const int b = __popc(__ballot_sync(0xffffffffu, lane < v.n_seqs && v.q_start[min(lane + 1, v.n_seqs)] <= tok));
    if (b >= v.n_seqs) return;
    const Seq q = load_seq(v, b);
    if (tok < q.q0 || tok >= q.q0 + q.n || q.n * v.G < p.prompt_rows) return;  // no row, or the split kernel's
    float top = lse;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float w = top == -INFINITY && lse == lse ? 0.f : exp2_fast(lse - top);
    float sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t *out = p.out + (int64_t)tok * p.out_ld + (int64_t)qh * D;
    for (int d0 = 0; d0 < D; d0 += 128) {
        const int d = d0 + lane * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float4 o[kPromptParts];
#pragma unroll
        for (int i = 0; i < kPromptParts; ++i)
            o[i] = (there >> i & 1) && d < D ? *reinterpret_cast<const float4 *>(p.part_out + (i * rows + row) * D + d) : acc;
#pragma unroll
        for (int i = 0; i < kPromptParts; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            acc.x = fmaf(wi, o[i].x, acc.x), acc.y = fmaf(wi, o[i].y, acc.y);
            acc.z = fmaf(wi, o[i].z, acc.z), acc.w = fmaf(wi, o[i].w, acc.w);
        }
        if (d < D)
            *reinterpret_cast<uint2 *>(out + d) = make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
    }
    if (lane == 0 && p.lse) p.lse[row] = (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, bool F16, bool PARTS>
cudaError_t launch_kernel(const AttnArgs &a, cudaStream_t s) {
    constexpr int smem = Prompt<D>::kSmem;
    static_assert(smem <= 227 * 1024, "shared memory over the per-block limit");
    cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<D, F16, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    static_assert(Prompt<D>::kRows == (D == 256 ? 128 : 256), "prompt_block_rows");
    const int slots = (int)((int64_t)a.kv.n_tokens * a.kv.G / Prompt<D>::kRows) + a.kv.n_seqs;
    LaunchScope scope(KC_ATTN_PROMPT, s);
    attn_prompt_kernel<D, F16, PARTS><<<dim3(slots * a.kv.KH, a.parts), kThreads, smem, s>>>(a, slots);
    return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
    if (a.parts == 1) return launch_kernel<D, F16, false>(a, s);
    const cudaError_t e = launch_kernel<D, F16, true>(a, s);
    if (e != cudaSuccess) return e;
    LaunchScope scope(KC_ATTN_JOIN, s);
    const int64_t rows = (int64_t)a.kv.n_tokens * a.kv.QH;
    attn_prompt_join_kernel<D, F16><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs &a, int D, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (D == 64) return f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    if (D == 128) return f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    return f16 ? launch<256, true>(a, s) : launch<256, false>(a, s);
}

}  // namespace moe
