// attention_prompt.cu -- attention over the paged 8-bit cache for runs of many new tokens, on the
// 5th-generation tensor cores (tcgen05, TMEM).
//
// A block takes 256 query rows (token, q head) of one kv head as two 128-row tiles and walks the
// keys they see in tiles of 128: S = Q K^T into TMEM, softmax weights back into TMEM as fp16 over S,
// O += P V from there.  All rows of a group of q heads share each key and value tile, so a tile
// of K and V is widened once for 256 rows.
//
// Bound: 4 D flops a (row, key) on the tensor cores; one tile pair is 4 x 512 tensor cycles at
// D = 128, and the weights of its 2 x 16,384 logits take about as long on two warpgroups, so the two
// row tiles alternate: while the tensor cores work on one, the other's softmax runs.  The 8-bit
// codes cannot be an operand beside fp16 weights (both operands of an MMA have one type, and queries in 8
// bits would lose what the 16-bit ones hold), so eight warps read codes from global memory (L2,
// mostly: all tiles of a head read the same pages), widen them exactly to fp16 and store them in the
// swizzled layout that the MMA reads: 96 KB of shared-memory traffic a tile against the MMA's own
// 192 KB.  The exponents of the pages are drawn into the codes relative to the largest one the block
// will meet (exact in fp16 unless a page is 2^-15 below it, and then off by at most 2^-25 of the
// largest), so one factor a row holds for all keys.
//
// Roles: warps 0-3 and 4-7 are row tiles 0 and 1, one row a thread; a thread of each also issues its
// tile's MMAs, so the hand-over from weights to products is one barrier.  Warps 8-15 widen K and V.  Row maxima move lazily: a row's reference changes only when a
// logit passes it by 2^8 (weights stay below 256), so O is rarely rescaled, by the thread that
// owns the row.
#include "layer.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRowTile = 128, kRowsBlock = 2 * kRowTile;
constexpr int kKeys = 128;  // keys a tile
constexpr int kStages = 4;  // K and V tiles in flight, in the order K0 V0 K1 V1 ...
constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kThreads = (kSoftWarps + kConvWarps) * 32;
// Registers a thread: 128 at launch (four warps a scheduler); the softmax warps hold a row's 128
// logits and take 2 x 168 of a scheduler's 4 x 128, the others keep 88.
constexpr int kSoftRegs = 168, kOtherRegs = 88;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s: far above any legitimate wait
constexpr float kLazy = 8.f;

template <int D>
struct Prompt {
    static constexpr int kBlocks = D / 64;                    // 128-byte column blocks of a row
    static constexpr int kBlockBytes = kKeys * 128;           // one column block of a 128-row tile
    static constexpr int kTileBytes = kBlocks * kBlockBytes;  // a tile of Q, K or V
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 256;
    static constexpr uint32_t kColO = 2 * kKeys;              // TMEM: S0 S1 O0 O1
    static constexpr uint32_t kCols = 512;
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ int exponent_of(float s) { return (int)((__float_as_uint(s) >> 23) & 0xffu) - 127; }
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((min(max(e, -126), 127) + 127) << 23); }
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t f) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&f));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Values read from TMEM are used only past this point (after the wait that completes the read).
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
    for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(r[k]));
}
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

// Block (slot, head): sequence b owns the 256-row slots base(b) .. base(b+1)-1 of every head, with
// base(b) = q_start[b] G / 256 + b (its n G rows need at most n G / 256 + 1 of them).
__device__ __forceinline__ int slot_base(const KvView &v, int b) {
    return (int)((int64_t)v.q_start[b] * v.G / kRowsBlock) + b;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ AttnArgs p, int slots) {
    using C = Prompt<D>;
    const KvView &v = p.kv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *q_smem = smem, *kv_smem = smem + 2 * C::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(kv_smem + kStages * C::kTileBytes);
    uint64_t *full = bars, *empty = bars + kStages;  // of a stage
    uint64_t *s_full = empty + kStages;              // [2] logits of a row tile are in TMEM
    uint64_t *p_full = s_full + 2;                   // [2] its weights are
    uint64_t *o_full = p_full + 2;                   // [2] its output is complete
    uint64_t *q_full = o_full + 2;                   // [2] its queries are in shared memory
    uint64_t *drain = q_full + 2;                    // [2]
    uint64_t *turn = drain + 2;                      // [2] the row tile may issue its next MMAs
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(turn + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    int *max_exp = reinterpret_cast<int *>(tmem_holder + 2);  // [2] of K and V

    const int tid = (int)threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

    // ------------------------------------------------------------------- the block's rows --
    const int head = (int)blockIdx.x % v.KH;
    const int slot = slots - 1 - (int)blockIdx.x / v.KH;  // a sequence's last rows see most keys: first
    int lo_b = 0, hi_b = v.n_seqs - 1;
    while (lo_b < hi_b) {
        const int mid = (lo_b + hi_b + 1) >> 1;
        if (slot_base(v, mid) <= slot) lo_b = mid; else hi_b = mid - 1;
    }
    const int b = lo_b;
    const Seq q = load_seq(v, b);
    const int row0 = (slot - slot_base(v, b)) * kRowsBlock;
    const int rows = min(kRowsBlock, q.n * v.G - row0);
    if (row0 < 0 || rows <= 0 || q.n * v.G < p.prompt_rows) return;  // (short runs are the split kernel's)
    const int first_pos = q.kv - q.n;
    // keys that any of the rows sees
    const int pos_lo = first_pos + row0 / v.G, pos_hi = first_pos + (row0 + rows - 1) / v.G;
    const int key_hi = p.causal ? min(q.kv, pos_hi + 1) : q.kv;
    const int key_lo = p.window > 0 ? max(0, pos_lo + 1 - p.window) : 0;
    const int tile0 = key_lo / kKeys;
    const int tiles = key_hi > key_lo ? (key_hi + kKeys - 1) / kKeys - tile0 : 0;
    const int32_t *table = v.table + (int64_t)b * v.max_pages;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&full[s], kConvWarps);
            ptx::mbar_init(&empty[s], 2);  // both row tiles are done with it
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 4);
            ptx::mbar_init(&o_full[i], 1);
            ptx::mbar_init(&q_full[i], 4);
            ptx::mbar_init(&drain[i], 1);
            ptx::mbar_init(&turn[i], 1);
        }
        *abort_flag = 0;
        max_exp[0] = max_exp[1] = -127;
        ptx::fence_mbar_init();
    }
    if (warp == 0) ptx::tmem_alloc(tmem_holder, C::kCols);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // the largest exponents among the pages the block reads
    {
        int ek = -127, ev = -127;
        const int pages0 = (tile0 * kKeys) >> v.log_p, pages1 = (key_hi + v.P - 1) >> v.log_p;
        for (int i = pages0 + tid; tiles > 0 && i < pages1; i += kThreads) {
            int page = __ldg(table + i);
            if (page < 0 || page >= v.n_pages) {
                layer_error(v.status);
                page = 0;
            }
            ek = max(ek, exponent_of(__ldg(v.k_scale + (int64_t)page * v.KH + head)));
            ev = max(ev, exponent_of(__ldg(v.v_scale + (int64_t)page * v.KH + head)));
        }
        ek = __reduce_max_sync(0xffffffffu, ek);
        ev = __reduce_max_sync(0xffffffffu, ev);
        if (lane == 0) {
            atomicMax(&max_exp[0], ek);
            atomicMax(&max_exp[1], ev);
        }
    }
    __syncthreads();
    const int k_exp = max_exp[0], v_exp = max_exp[1];
    bool ok = true;

    if (warp < kSoftWarps) {
        regs_up<kSoftRegs>();
        // ----------------------------------------------------------------- softmax, rows --
        const int i = warp >> 2;                        // row tile
        const int r = i * kRowTile + (warp & 3) * 32 + lane;  // row of the block = TMEM lane of tile i
        const bool live = r < rows;
        const int tok = (row0 + r) / v.G, qh = head * v.G + (row0 + r) % v.G;
        const int pos = first_pos + tok;
        const int hi = p.causal ? min(q.kv, pos + 1) : q.kv;
        const int lo = p.window > 0 ? max(0, pos + 1 - p.window) : 0;
        // Q: the row scaled by a power of two into [1, 2) at its largest, as fp16, K-major swizzled
        const int rr = r & (kRowTile - 1);
        uint8_t *dst = q_smem + i * C::kTileBytes + rr * 128;
        float amax = 0.f;
        uint4 qv[D / 8];
        const uint16_t *src = p.q + (int64_t)(q.q0 + tok) * p.q_ld + (int64_t)qh * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            qv[c] = live ? *reinterpret_cast<const uint4 *>(src + c * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            float f[8];
            unpack8<F16>(qv[c], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
        }
        const int q_exp = amax > 0.f ? max(min((int)(__float_as_uint(amax) >> 23) - 127, 126), -126) : 0;
        const float q_inv = pow2f(-q_exp);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
            float f[8];
            unpack8<F16>(qv[c], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= q_inv;
            *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kBlockBytes + (((c & 7) ^ (rr & 7)) << 4)) = pack8<true>(f);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&q_full[i]);

        // --------------------------------------- the MMAs, by one warp of each row tile --
        const bool issuer = (warp & 3) == 0;
        const uint32_t idesc_s = ptx::idesc_f16_f32(kRowTile, kKeys, false);
        const uint32_t idesc_o = ptx::idesc_f16_f32(kRowTile, D, true);
        const uint32_t s_tmem = tmem + i * kKeys, o_tmem = tmem + C::kColO + i * D;
        const uint64_t q_desc = ptx::sw128_desc(ptx::smem_u32(q_smem) + i * C::kTileBytes);
        const uint64_t k_desc = ptx::sw128_desc(ptx::smem_u32(kv_smem));
        const uint64_t v_desc = ptx::sw128_desc_mn(ptx::smem_u32(kv_smem), C::kBlockBytes);
        auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
        auto filled = [&](int it) { return ptx::mbar_wait(&full[it % kStages], (it / kStages) & 1, kWaitNs, abort_flag); };
        auto logits = [&](int j) {  // S = Q K_j^T
            const int s = 2 * j % kStages;
            if (!all(filled(2 * j))) return false;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                const uint64_t kd = k_desc + (uint64_t)(s * (C::kTileBytes >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    constexpr int kBlock16 = C::kBlockBytes >> 4;
                    const int off = (k >> 2) * kBlock16 + (k & 3) * 2;
                    ptx::mma_f16_ss(s_tmem, q_desc + off, kd + off, idesc_s, k > 0);
                }
                ptx::mma_commit(&s_full[i]);
                ptx::mma_commit(&empty[s]);
            }
            __syncwarp();
            return true;
        };
        auto output = [&](int j) {  // O += P V_j
            const int s = (2 * j + 1) % kStages;
            if (!all(filled(2 * j + 1))) return false;
            ptx::tc_fence_after();
            if (ptx::elect_one()) {
                const uint64_t vd = v_desc + (uint64_t)(s * (C::kTileBytes >> 4));
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    ptx::mma_f16_ts(o_tmem, s_tmem + k * 8, vd + k * (2048 >> 4), idesc_o, j > 0 || k > 0);
                ptx::mma_commit(&empty[s]);
                if (j + 1 == tiles) ptx::mma_commit(&o_full[i]);
            }
            __syncwarp();
            return true;
        };
        // The tiles take turns: O_0, S_0, O_1, S_1, ...  Issued at will, the two tiles' MMAs interleave, both
        // softmaxes get their logits at the same time, and the tensor cores idle while both run.
        auto my_turn = [&](int n) { return ptx::mbar_wait(&turn[i], n & 1, kWaitNs, abort_flag); };
        if (issuer && tiles > 0) {
            ok = all(ptx::mbar_wait(&q_full[i], 0, kWaitNs, abort_flag) && (i == 0 || my_turn(0)));
            if (ok) ok = logits(0);
            if (lane == 0) ptx::mbar_arrive(&turn[i ^ 1]);
        }

        const float mul = p.scale_log2 * pow2f(q_exp) * pow2f(k_exp);
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lanes + i * kKeys, o_addr = tmem + lanes + C::kColO + i * D;
        float m = -INFINITY;
        float2 l0 = make_float2(0.f, 0.f), l1 = l0;  // sums of every fourth column's weights
        for (int j = 0; j < tiles && ok; ++j) {
            ok = ptx::mbar_wait(&s_full[i], j & 1, kWaitNs, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const int key0 = (tile0 + j) * kKeys;
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) ptx::tmem_ld_32(s_addr + c * 32, s[c]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) tie32(s[c]);
            if (__any_sync(0xffffffffu, live && (key0 < lo || key0 + kKeys > hi))) {
                const int c_lo = lo - key0, c_hi = hi - key0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c * 32 + k < c_lo || c * 32 + k >= c_hi) s[c][k] = 0xff800000u;  // -inf
            }
            float tops[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                tops[c] = max3(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]), __uint_as_float(s[c][2]));
#pragma unroll
                for (int k = 3; k < 31; k += 2) tops[c] = max3(tops[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
                tops[c] = fmaxf(tops[c], __uint_as_float(s[c][31]));
            }
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * mul;  // mul > 0
            if (__any_sync(0xffffffffu, top > m + kLazy)) {
                const float to = fmaxf(m, top);
                const float f = to == -INFINITY ? 1.f : exp2_fast(m - to);
                m = to;
                l0.x *= f, l0.y *= f, l1.x *= f, l1.y *= f;
                if (j > 0) {  // the logits came after the last product of this tile was complete
                    uint32_t o[16];
                    __syncwarp();
#pragma unroll
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
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 z = fma2(make_float2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), mul, -ref);
                    const float2 e = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                    if (k & 1) l1 = __fadd2_rn(l1, e); else l0 = __fadd2_rn(l0, e);
                    w[k] = pack2<true>(e.x, e.y);
                }
                ptx::tmem_st_16(s_addr + c * 16, w);  // over S, all of which is in registers
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&p_full[i]);
            if (issuer) {
                ok = all(ptx::mbar_wait(&p_full[i], j & 1, kWaitNs, abort_flag) && my_turn(j + i));
                if (ok) ok = output(j);
                if (ok && j + 1 < tiles) ok = logits(j + 1);
                if (lane == 0) ptx::mbar_arrive(&turn[i ^ 1]);
            }
        }
        if (!ok && issuer) {  // nothing of this block may still run when its TMEM is freed
            if (ptx::elect_one()) ptx::mma_commit(&drain[i]);
            int zero = 0;
            ptx::mbar_wait(&drain[i], 0, kWaitNs, &zero);
        }
        const float l = l0.x + l0.y + (l1.x + l1.y);
        if (ok && tiles > 0) ok = ptx::mbar_wait(&o_full[i], 0, kWaitNs, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            ptx::tc_fence_after();
            const float inv = (l > 0.f || l != l) && tiles > 0 ? pow2f(v_exp) / l : 0.f;
            uint16_t *out = p.out + (int64_t)(q.q0 + tok) * p.out_ld + (int64_t)qh * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (tiles > 0) {
                    ptx::tmem_ld_32(o_addr + c * 32, o);
                    ptx::tmem_ld_wait();
                }
#pragma unroll
                for (int k = 0; k < 4 && live; ++k) {
                    float f[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] = inv == 0.f ? 0.f : __uint_as_float(o[8 * k + x]) * inv;
                    *reinterpret_cast<uint4 *>(out + c * 32 + k * 8) = pack8<F16>(f);
                }
            }
            if (live && p.lse) p.lse[(int64_t)(q.q0 + tok) * v.QH + qh] = (m + log2f(l)) * 0.6931471805599453f;
        }
    } else {
        regs_down<kOtherRegs>();
        // ------------------------------------------------------------- K and V, widened --
        // Warp w owns keys 16 w .. 16 w + 15 of every tile: they lie in one page.  A load takes 8 rows x 64
        // codes: lane = 4 * row + 16-code piece, so that the two 16-byte stores of 8 lanes fall on
        // all the banks.  The registers of a tile's codes take the next tile's as soon as they are
        // widened, so a load has a whole tile's time to arrive.
        constexpr int kLoads = 2 * C::kBlocks;
        const int cw = warp - kSoftWarps, piece = lane & 3, sub = lane >> 2;
        auto page_at = [&](int tile) {  // page * KH + head
            const int key = (tile0 + tile) * kKeys + cw * 16;
            int page = 0;
            if (key < key_hi) page = __ldg(table + (key >> v.log_p));
            return (page < 0 || page >= v.n_pages ? 0 : page) * v.KH + head;  // (reported above)
        };
        auto factor = [&](float scale, int largest) {  // 2^(exponent - the block's largest)
            const int e = min(exponent_of(scale) - largest, 0);  // (past the end: any page)
            const __half2 f = __float2half2_rn(e < -24 ? 0.f : pow2f(e));
            return *reinterpret_cast<const uint32_t *>(&f);
        };
        const int log_pd = v.log_p + (D == 128 ? 7 : 6);
        auto load = [&](uint4 (&raw)[kLoads], int tile, int page, const uint8_t *codes) {
            const int key0 = (tile0 + tile) * kKeys + cw * 16;
            const uint8_t *src = codes + ((uint64_t)(uint32_t)page << log_pd) + ((key0 & (v.P - 1)) + sub) * D + piece * 16;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                raw[n] = make_uint4(0, 0, 0, 0);
                if (key0 + n / C::kBlocks * 8 + sub < key_hi)  // slots past the end hold anything
                    raw[n] = __ldg(reinterpret_cast<const uint4 *>(src + n / C::kBlocks * 8 * D + n % C::kBlocks * 64));
            }
        };
        const uint32_t row_off = (uint32_t)(cw * 16 + sub) * 128;
        const uint32_t off0 = row_off + (((2 * piece) ^ sub) << 4), off1 = row_off + (((2 * piece + 1) ^ sub) << 4);
        auto widen = [&](const uint4 (&raw)[kLoads], int it, uint32_t f) {
            uint8_t *st = kv_smem + it % kStages * C::kTileBytes;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) {
                const uint32_t w[4] = {raw[n].x, raw[n].y, raw[n].z, raw[n].w};
                uint32_t h[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[2 * k] = mul2(widen2(w[k] & 0xffffu), f);
                    h[2 * k + 1] = mul2(widen2(w[k] >> 16), f);
                }
                uint8_t *dst = st + n % C::kBlocks * C::kBlockBytes + n / C::kBlocks * 8 * 128;
                *reinterpret_cast<uint4 *>(dst + off0) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(dst + off1) = make_uint4(h[4], h[5], h[6], h[7]);
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
        uint4 rk[kLoads], rv[kLoads];
        int page1 = page_at(0), page2 = page_at(1);
        float sk = __ldg(v.k_scale + page1), sv = __ldg(v.v_scale + page1);
        if (tiles > 0) {
            load(rk, 0, page1, v.k_codes);
            load(rv, 0, page1, v.v_codes);
        }
        for (int j = 0; j < tiles; ++j) {
            const uint32_t fk = factor(sk, k_exp), fv = factor(sv, v_exp);
            page1 = page2;  // of tile j + 1
            sk = __ldg(v.k_scale + page1), sv = __ldg(v.v_scale + page1);
            page2 = page_at(j + 2);
            if (!(ok = free_stage(2 * j))) break;
            widen(rk, 2 * j, fk);
            if (j + 1 < tiles) load(rk, j + 1, page1, v.k_codes);
            publish(2 * j);
            if (!(ok = free_stage(2 * j + 1))) break;
            widen(rv, 2 * j + 1, fv);
            if (j + 1 < tiles) load(rv, j + 1, page1, v.v_codes);
            publish(2 * j + 1);
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
    if (warp == 0) ptx::tmem_dealloc(tmem, C::kCols);
}

template <int D, bool F16>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
    constexpr int smem = Prompt<D>::kSmem;
    static_assert(smem <= 227 * 1024, "shared memory over the per-block limit");
    cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    LaunchScope scope(KC_ATTN_PROMPT, s);
    const int slots = (int)((int64_t)a.kv.n_tokens * a.kv.G / kRowsBlock) + a.kv.n_seqs;
    attn_prompt_kernel<D, F16><<<slots * a.kv.KH, kThreads, smem, s>>>(a, slots);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs &a, int D, int dtype, cudaStream_t s) {
    const bool f16 = dtype == MOE_DTYPE_F16;
    if (D == 64) return f16 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return f16 ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace moe
