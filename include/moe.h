/*
 * moe.h -- C ABI of the GB300-native top-k routed Mixture-of-Experts FFN layer (libmoe.so).
 *
 * The layer.  The pages describe the layer only in prose: a network of many expert
 * sub-networks of which each token activates a small part ("AI MAX+ 395部署Qwen3大模型：
 * GFX1151引擎实测优化解析", explanatory MoE paragraph under "MOE 内核优化"), executed on the
 * timed path of a batch-1 BF16 engine by a "selected-MoE" kernel ("AIMA AMD395 Qwen3.6 35B
 * Windows Engine", section "性能优化做了什么").  This library computes the standard reading of
 * that layer, for T tokens of hidden size H, E routed experts, top-k, expert intermediate I
 * and a shared expert of intermediate Is:
 *   logits   l[t,e] = sum_h x[t,h] Wr[e,h] (+ b[e])                     fp32
 *   route    ids[t,0..k) = the k largest logits (lower index first on equal logits),
 *            descending; w[t,j] = exp(l[t,ids_j]) / sum_i exp(l[t,ids_i])   (softmax over
 *            all E followed by renormalisation over the k chosen; the full denominator cancels)
 *   permute  stable counting sort of the T*k pairs p = t*k + j by expert id
 *   experts  h = bf16( silu(Wg[e] x) * (Wu[e] x) ),  y = Wd[e] h        fp32 accumulate
 *   shared   the same SwiGLU with the shared weights, weight 1, for every token
 *   combine  out[t] = bf16( sum_j w[t,j] y[t,j] + y_shared[t] )
 * and composes long prompts from q8192 / q4096 / q2048 / q1024 pieces plus an exact tail
 * ("AIMA AMD395 Qwen3.6 35B Windows Engine", "性能优化做了什么": prompts split into a q8192
 * tile, q1024 and a tail; "AIMA AMD395 Qwen3.6 35B Linux Engine", "Read this boundary first":
 * resident q1024/q2048/q4096/q8192 buckets).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers (caller-allocated, caller-owned), row-major and
 *     contiguous, 16-byte aligned, in the [out, in] linear convention.  bf16 tensors are passed
 *     as moe_bf16 (the 16-bit pattern).  The library never allocates device memory and keeps no
 *     state between calls other than per-device launch attributes and the optional timing table.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call is
 *     asynchronous on that stream; inputs must stay valid until the stream reaches the work.
 *   - Arguments are validated on the host before any launch; an invalid call launches
 *     nothing and returns an error status.  T == 0 returns MOE_OK and does nothing.
 *   - Device-side failures (a bounded wait that ran out, an expert id out of range) are
 *     recorded in a status word in the workspace and read with moe_check_status().
 *   - Supported shapes: H % 128 == 0, I % 128 == 0, Is % 128 == 0 (or Is == 0: no shared
 *     expert), 1 <= k <= min(E, 32), E <= 1024, H <= 16384, I, Is <= 8192.  Router logits
 *     must be finite.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t moe_bf16; /* bit pattern of a bfloat16 value */

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,        /* null pointer, negative size, k > E, misalignment, ... */
    MOE_ERR_WORKSPACE_TOO_SMALL = 2,
    MOE_ERR_UNSUPPORTED_SHAPE = 3,  /* outside the supported shapes listed above */
    MOE_ERR_CUDA = 4,               /* a CUDA runtime/driver call failed */
    MOE_ERR_TIMEOUT = 5,            /* a device-side bounded wait ran out (see moe_check_status) */
    MOE_ERR_NOT_IMPLEMENTED = 6
} moe_status;

/* Layer shape.  shared_inter == 0 means no shared expert. */
typedef struct {
    int hidden;       /* H */
    int n_experts;    /* E */
    int top_k;        /* k */
    int inter;        /* I */
    int shared_inter; /* Is */
} moe_config;

/* Device pointers to one layer's weights (bf16 unless noted). */
typedef struct {
    const moe_bf16 *w_router; /* [E, H] */
    const float *b_router;    /* [E] fp32 router bias, or NULL (no bias) */
    const moe_bf16 *w_gate;   /* [E, I, H] */
    const moe_bf16 *w_up;     /* [E, I, H] */
    const moe_bf16 *w_down;   /* [E, H, I] */
    const moe_bf16 *ws_gate;  /* [Is, H]  (NULL when Is == 0) */
    const moe_bf16 *ws_up;    /* [Is, H]  (NULL when Is == 0) */
    const moe_bf16 *ws_down;  /* [H, Is]  (NULL when Is == 0) */
} moe_weights;

/* One layer with quantised expert weights: every expert matrix as E4M3 codes (1 sign, 4
 * exponent bits with bias 7, 3 fraction bits; no infinities) with one fp32 scale per output row,
 * weight[r, c] = scale[r] * code[r, c].  The router stays bf16.  ("AI MAX+ 395部署Qwen3大模型：
 * GFX1151引擎实测优化解析", "两种权重格式：HGN 与 GGUF 的统一支持": 8-bit float weights for the large
 * modules; the row scales are this library's reading, the page gives no layout.)  Code arrays
 * 16-byte aligned; moe_quantize_e4m3 produces them from bf16 matrices. */
typedef struct {
    const moe_bf16 *w_router; /* [E, H] bf16 */
    const float *b_router;    /* [E] fp32, or NULL */
    const uint8_t *q_gate;    /* [E, I, H] codes */
    const uint8_t *q_up;      /* [E, I, H] */
    const uint8_t *q_down;    /* [E, H, I] */
    const float *s_gate;      /* [E, I] row scales */
    const float *s_up;        /* [E, I] */
    const float *s_down;      /* [E, H] */
    const uint8_t *qs_gate;   /* [Is, H] (NULL when Is == 0) */
    const uint8_t *qs_up;     /* [Is, H] */
    const uint8_t *qs_down;   /* [H, Is] */
    const float *ss_gate;     /* [Is] */
    const float *ss_up;       /* [Is] */
    const float *ss_down;     /* [H] */
} moe_weights_q8;

/* One layer with 4-bit integer expert weights ("Q4": 4-bit integer codes, as the GFX1151 page's
 * explanatory paragraph on weight formats calls them; the block layout is this library's
 * reading, the page gives none).  Each row of every expert matrix is cut into blocks of 32
 * consecutive columns; a block has one fp32 scale and 32 codes in [-7, 7], two's-complement
 * nibbles, column 2j in the low and 2j+1 in the high nibble of byte j of the row (cols / 2 bytes a
 * row); weight = scale * code.  The router stays bf16.  H and I (and Is) multiples of 128; code
 * arrays 16-byte aligned; moe_quantize_q4 produces them from bf16 matrices. */
typedef struct {
    const moe_bf16 *w_router; /* [E, H] bf16 */
    const float *b_router;    /* [E] fp32, or NULL */
    const uint8_t *q_gate;    /* [E, I, H/2] codes */
    const uint8_t *q_up;      /* [E, I, H/2] */
    const uint8_t *q_down;    /* [E, H, I/2] */
    const float *s_gate;      /* [E, I, H/32] block scales */
    const float *s_up;        /* [E, I, H/32] */
    const float *s_down;      /* [E, H, I/32] */
    const uint8_t *qs_gate;   /* [Is, H/2] (NULL when Is == 0) */
    const uint8_t *qs_up;     /* [Is, H/2] */
    const uint8_t *qs_down;   /* [H, Is/2] */
    const float *ss_gate;     /* [Is, H/32] */
    const float *ss_up;       /* [Is, H/32] */
    const float *ss_down;     /* [H, Is/32] */
} moe_weights_q4;

/* Text for a status code (static storage). */
const char *moe_status_string(moe_status s);

/* Bytes of device workspace needed by any call below for up to max_T tokens (moe_forward
 * needs only min(max_T, 8192) tokens' worth, since it works piece by piece).  Returns 0 for
 * an invalid or unsupported config.  The workspace must be 256-byte aligned.  Its first 256
 * bytes hold the device status word: zero them once after allocating the workspace (kernels
 * only ever change the word from 0 to an error code; moe_check_status clears it).  The rest
 * is scratch that every call overwrites. */
size_t moe_workspace_size(const moe_config *cfg, int max_T);

/* Router: logits, softmax, top-k and renormalisation.  Passage: each token activates only a few
 * of many experts ("AI MAX+ 395部署Qwen3大模型：GFX1151引擎实测优化解析", explanatory MoE
 * paragraph under "MOE 内核优化"); the selection rule (largest logits, lower index on ties,
 * weights renormalised over the k) is this library's reading, the pages give no formula.
 * x [T,H] bf16 -> topk_ids [T,k] int32 and topk_w [T,k] fp32, slots in descending logit
 * order.  logits_out [T,E] fp32 may be NULL; when given it receives the exact fp32 logits the
 * selection used.  ws: workspace of moe_workspace_size(cfg, T) bytes (holds the logits when
 * logits_out is NULL).  Computed on tensor cores (bf16 x bf16 -> fp32 accumulate); for the
 * 1 to 4 tokens moe_forward runs on the decode path, by that path's GEMV, so the logits are
 * the ones moe_forward selects on. */
moe_status moe_route(const moe_config *cfg, const moe_weights *w, const moe_bf16 *x, int T,
                     float *logits_out, int32_t *topk_ids, float *topk_w, void *ws,
                     size_t ws_bytes, void *stream);

/* Softmax + top-k + renormalisation only, from given fp32 logits [T,E] (the routing step of
 * the same passage as moe_route).  Bit-exact ids for
 * identical logits (the selection compares fp32 values exactly, lower index first on ties). */
moe_status moe_route_from_logits(const moe_config *cfg, const float *logits, int T,
                                 int32_t *topk_ids, float *topk_w, void *stream);

/* Permutation of the T*k (token, slot) pairs by expert: a stable counting sort.  Passage: the
 * "selected-MoE" kernel runs only the experts each token selected ("AIMA AMD395 Qwen3.6 35B
 * Windows Engine", "性能优化做了什么"), which needs each expert's tokens gathered together; the
 * page does not describe how, so the grouping is this library's (a textbook stable sort).
 * topk_ids [T,k] -> expert_offsets [E+1] (exclusive prefix sum of the per-expert counts,
 * offsets[E] == T*k), perm [T*k] (row of the expert-sorted order -> pair index t*k+j),
 * inv [T*k] (pair index -> row).  Pairs of one expert keep increasing pair order.  Bit-exact.
 * ws: workspace of moe_workspace_size(cfg, T) bytes.  Ids outside [0,E) are a caller error:
 * they are detected on the device, flagged in the status word, and the pair is dropped
 * (inv = -1). */
moe_status moe_permute(const moe_config *cfg, const int32_t *topk_ids, int T,
                       int32_t *expert_offsets, int32_t *perm, int32_t *inv, void *ws,
                       size_t ws_bytes, void *stream);

/* moe_permute without a workspace, for callers that cannot allocate device memory where
 * they route tokens (a serving process that reserves all device memory at start-up, host
 * code with no allocator at hand).  The pages have no counterpart: this is a convenience of
 * this library.  Same outputs as moe_permute (bit-identical), but the per-chunk count table
 * lives in a fixed array inside the library (160 KiB on every device that loads it, kept
 * until the process exits), so the call allocates nothing and takes no workspace.
 * Limits: T*k <= 65536 pairs, E <= 1024, k <= 32; larger problems return
 * MOE_ERR_UNSUPPORTED_SHAPE (use moe_permute).  Ids outside [0,E) get inv = -1 and are not
 * otherwise reported (no status word).  The first call on each device looks up the array's
 * device address (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  All calls share the one array: calls that overlap on the GPU
 * (different streams or threads) race and must be serialised by the caller. */
moe_status moe_permute_noalloc(const moe_config *cfg, const int32_t *topk_ids, int T,
                               int32_t *expert_offsets, int32_t *perm, int32_t *inv,
                               void *stream);

/* Expert FFNs, unfused (for step-by-step checking).  Passage: the selected experts' own
 * sub-networks ("AI MAX+ 395部署Qwen3大模型：GFX1151引擎实测优化解析", "MOE 内核优化": the MoE
 * kernel that bounds prefill), read as SwiGLU experts plus an always-on shared expert.
 * Routed rows in the permuted order:
 * h_rows [T*k, I] bf16 = bf16(silu(Wg[e] x_t) * (Wu[e] x_t)) and y_rows [T*k, H] fp32 =
 * Wd[e] h, for row r of expert e holding pair perm[r] of token perm[r]/k.  When shared_y is not
 * NULL and Is > 0, also shared_y [T,H] fp32 = the shared expert applied to every token.
 * expert_offsets/perm as produced by moe_permute.  ws: moe_workspace_size(cfg, T) bytes. */
moe_status moe_expert_ffn(const moe_config *cfg, const moe_weights *w, const moe_bf16 *x, int T,
                          const int32_t *expert_offsets, const int32_t *perm, moe_bf16 *h_rows,
                          float *y_rows, float *shared_y, void *ws, size_t ws_bytes,
                          void *stream);

/* Weighted combine (the last step of the selected-MoE layer, "AIMA AMD395 Qwen3.6 35B Windows
 * Engine", "性能优化做了什么"; the weighting by the renormalised routing weights is this
 * library's reading): out[t] = bf16( sum_j topk_w[t,j] * y_rows[inv[t*k+j]] + shared_y[t] ).
 * shared_y may be NULL (no shared term).  Deterministic (fixed slot order, fp32). */
moe_status moe_combine(const moe_config *cfg, const float *y_rows, const int32_t *inv,
                       const float *topk_w, const float *shared_y, int T, moe_bf16 *out,
                       void *stream);

/* The whole layer, fused: x [T,H] -> out [T,H] bf16.  T is split greedily into pieces of
 * 8192, 4096, 2048 and 1024 tokens and an exact tail (no padding); every piece runs the same
 * kernels, so the result equals the concatenation of per-piece calls.  A call (or tail) of 1
 * to 4 tokens with T*H <= 32768 takes the decode path: a router GEMV, then every selected
 * expert's weights streamed once for all the tokens that chose it, its partial products
 * added in fp32 with atomics (so not bit-reproducible) and rounded to bf16 once.  x_next may
 * be NULL; when given it receives bf16(resid + out), the residual-stream update of a layer
 * stack, fused into the last kernel; resid [T,H] may be NULL, meaning x.  x_next may alias
 * resid (not x, when they differ).  ws: moe_workspace_size(cfg, T) bytes.  Rounding on the
 * prefill path: h is rounded to bf16 once, each weighted expert row w*y (and the shared
 * expert's row) is stored as bf16, the k+1 rows of a token are summed in fp32 in slot order,
 * and the sum is rounded to bf16 once.  No atomics there: the result is bit-reproducible.
 * Any T >= 0 (int) is accepted: the pieces are walked one after another, so there is no limit
 * on their number. */
moe_status moe_forward(const moe_config *cfg, const moe_weights *w, const moe_bf16 *x, int T,
                       moe_bf16 *out, const moe_bf16 *resid, moe_bf16 *x_next, void *ws,
                       size_t ws_bytes, void *stream);

/* moe_forward for a layer with quantised expert weights (moe_weights_q8): the same piece
 * composition, router (bf16 weights), selection, permutation, rounding points and combine, with
 * every expert matrix streamed as its E4M3 codes, one byte a weight ("AI MAX+ 395部署Qwen3大模型：
 * GFX1151引擎实测优化解析", "两种权重格式：HGN 与 GGUF 的统一支持": 8-bit float weights for the large
 * modules).  The grouped GEMMs widen each code exactly to bf16 in shared memory (every E4M3 value
 * is a bf16 value), multiply with bf16 tokens into fp32, and scale each weight row's accumulator
 * by its fp32 row scale; h = bf16(silu(g) * u) as in moe_forward.  Every piece, however short,
 * takes this grouped path (there is no E4M3 variant of the 1-4-token kernels in moe_forward;
 * moe_decode_chain_q8 is the quantised decode step).  Same arguments, workspace, alignment and
 * errors as moe_forward. */
moe_status moe_forward_q8(const moe_config *cfg, const moe_weights_q8 *w, const moe_bf16 *x, int T,
                          moe_bf16 *out, const moe_bf16 *resid, moe_bf16 *x_next, void *ws,
                          size_t ws_bytes, void *stream);

/* A layer stack captured once as a CUDA graph and replayed (the resident prefill buckets of
 * "AIMA AMD395 Qwen3.6 35B Linux Engine", release boundary v1.5.0: one graph per bucket size,
 * kept resident with its workspace).  The graph holds n_layers (1..64) moe_forward calls on T
 * tokens with these exact pointers: layer 0 reads x0; layer l writes out and
 * x_{l+1} = bf16(r + out_l), r = resid when given, else x_l; layer l+1 reads x_{l+1}.  The
 * intermediate x_l alternate between x_last and scratch so that x_last receives x_{n_layers};
 * both [T,H] bf16, required when n_layers > 1 (x_last may be NULL for one layer; scratch is
 * then unused), distinct from x0, resid and out.  Every buffer, the weights and ws must stay
 * allocated and unchanged in place while the graph lives; their contents may change between
 * launches (a new x0 is simply copied into x0's buffer).
 * moe_graph_create validates as moe_forward does, runs the stack once on `stream` (this
 * warms the library's per-device launch caches and writes the outputs), then captures it on a
 * private stream and instantiates it.  moe_graph_launch replays it on `stream`, asynchronously;
 * moe_launch_count() advances by the graph's kernel count.  Calls sharing ws must not overlap.
 * moe_graph_destroy frees the graph (NULL is a no-op). */
typedef struct moe_graph_s *moe_graph;
moe_status moe_graph_create(const moe_config *cfg, const moe_weights *layers, int n_layers, int T,
                            const moe_bf16 *x0, const moe_bf16 *resid, moe_bf16 *out, moe_bf16 *x_last,
                            moe_bf16 *scratch, void *ws, size_t ws_bytes, void *stream, moe_graph *graph);
moe_status moe_graph_launch(moe_graph graph, void *stream);
/* Kernel nodes in the graph (-1 for NULL). */
int moe_graph_kernel_count(moe_graph graph);
moe_status moe_graph_destroy(moe_graph graph);

/* One token through a stack of n_layers MoE layers (1 <= n_layers <= 64), each with its own
 * weights layers[l] (a host array of device pointers), in ONE cooperative kernel launch: the
 * batch-1 greedy decode step the pages run ("AIMA AMD395 Qwen3.6 35B Windows Engine",
 * "产品定位"), with the MoE layers back to back.  x_0 = x0 [H] bf16; for each layer
 * out_l = the layer applied to x_l (as moe_forward with T = 1: same router rows, selection and
 * rounding points) and x_{l+1} = bf16(r + out_l), r = resid [H] when given, else x_l (the
 * residual stream).  out [H] receives the last layer's out; x_last [H] (may be NULL) receives
 * x_{n_layers}.  The layers are separated by grid barriers instead of kernel boundaries; the
 * fp32 atomics of the split-K down projection make the last bit run-dependent, as at T = 1.
 * Requires T = 1 to fit the decode path (H <= 16384).  x0, resid, out, x_last 16-byte aligned;
 * out and x_last must not alias x0 or resid.  ws: moe_workspace_size(cfg, 1) bytes; the call
 * writes its barrier words there, so calls sharing a workspace must not overlap.  A barrier
 * wait that runs out (2 s) records MOE_ERR_TIMEOUT in the workspace status word and every
 * block returns.  MOE_ERR_UNSUPPORTED_SHAPE for more than 64 layers or a too-large H. */
moe_status moe_decode_chain(const moe_config *cfg, const moe_weights *layers, int n_layers,
                            const moe_bf16 *x0, const moe_bf16 *resid, moe_bf16 *out,
                            moe_bf16 *x_last, void *ws, size_t ws_bytes, void *stream);

/* moe_decode_chain for layers with quantised expert weights (moe_weights_q8): every expert
 * row streamed as its E4M3 codes (half the bytes of bf16) and its scale, widened exactly and
 * accumulated in fp32; otherwise the same steps, rounding points, barriers and errors. */
moe_status moe_decode_chain_q8(const moe_config *cfg, const moe_weights_q8 *layers, int n_layers,
                               const moe_bf16 *x0, const moe_bf16 *resid, moe_bf16 *out,
                               moe_bf16 *x_last, void *ws, size_t ws_bytes, void *stream);

/* moe_decode_chain for layers with 4-bit expert weights (moe_weights_q4): every expert row
 * streamed as its codes (a quarter of the bytes of bf16) and block scales, each block's codes
 * dotted in fp32 and scaled; otherwise the same steps, rounding points, barriers and errors. */
moe_status moe_decode_chain_q4(const moe_config *cfg, const moe_weights_q4 *layers, int n_layers,
                               const moe_bf16 *x0, const moe_bf16 *resid, moe_bf16 *out,
                               moe_bf16 *x_last, void *ws, size_t ws_bytes, void *stream);

/* Block-wise 4-bit quantisation of a bf16 matrix w [rows, cols] (device pointers; cols a multiple
 * of 32): per block of 32 columns, scale = max |w| / 7 (1 for an all-zero block) and code =
 * round-half-even(w / scale) clamped to [-7, 7], in fp32 with IEEE division (a function of the
 * block alone).  q [rows, cols/2] packed nibbles (column 2j low, 2j+1 high), scale [rows, cols/32]
 * fp32.  Blocks holding an infinity or a NaN give unspecified codes.  Asynchronous on `stream`;
 * rows or cols of 0 do nothing; a negative size, cols not a multiple of 32 or a NULL pointer is
 * MOE_ERR_INVALID_ARG. */
moe_status moe_quantize_q4(const moe_bf16 *w, int rows, int cols, uint8_t *q, float *scale, void *stream);

/* Row-wise E4M3 quantisation of a bf16 matrix w [rows, cols] (device pointers): scale[r] =
 * max_c |w[r,c]| / 448 (1 for an all-zero row) and q[r,c] = the E4M3 code nearest to
 * w[r,c] / scale[r] (ties to even; magnitudes past 448 saturate), in fp32 with IEEE division,
 * so the result is a function of the row alone.  q [rows, cols] bytes, scale [rows] fp32.
 * Rows holding an infinity or a NaN give unspecified codes.  Asynchronous on `stream`; rows or
 * cols of 0 do nothing; a negative size or a NULL pointer is MOE_ERR_INVALID_ARG. */
moe_status moe_quantize_e4m3(const moe_bf16 *w, int rows, int cols, uint8_t *q, float *scale,
                             void *stream);

/* ---- the rest of a decoder layer: block norms, the paged 8-bit cache, attention ----
 *
 * The MoE layer above is one half of a decoder layer; these three calls are the other half
 * ("AIMA AMD395 Qwen3.6 35B Windows Engine", "性能优化做了什么": the engine whose timed path the
 * MoE kernel is part of; the pages give no formulas for the rest, so every reading is this
 * library's).  The conventions above hold, with these differences: activations are bf16 or
 * fp16 (moe_dtype), rows may lie apart (a row stride in elements, a multiple of 8, so that q,
 * k and v can be columns of one product), and the workspace is moe_attn_workspace_size's. */

typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F16 = 1 } moe_dtype;

typedef enum {
    MOE_GATE_NONE = 0,    /* g = 1 */
    MOE_GATE_CHANNEL = 1, /* gate [H]: one value a channel (a learned layer scale) */
    MOE_GATE_TOKEN = 2,   /* gate [T], row stride gate_ld: one value a token */
    MOE_GATE_ELEMENT = 3  /* gate [T,H], row stride gate_ld */
} moe_gate;

/* Norms before and after a block, fused with its gate and residual scale. */
typedef struct {
    int hidden;           /* H, a multiple of 8, at most 16384 */
    int dtype;            /* moe_dtype of every tensor of the call, weights included */
    int gate;             /* moe_gate */
    int gate_sigmoid;     /* 1: g = 1 / (1 + e^-gate) */
    int unit_offset;      /* 1: the norm weights are stored as w - 1 */
    float eps;            /* added to the mean square, >= 0 */
    float residual_scale; /* alpha */
} moe_norm_config;

typedef struct {
    const void *x;      /* [T,H] the block's output, or NULL: no block, only the norm before one */
    const void *resid;  /* [T,H] the residual stream, or NULL: 0 */
    const void *gate;   /* see moe_gate; NULL with MOE_GATE_NONE */
    const void *w_post; /* [H] weight of the norm after the block, or NULL: no such norm */
    const void *w_pre;  /* [H] weight of the norm before the next block; needed with y */
    void *resid_out;    /* [T,H] the new residual stream, or NULL; may be resid */
    void *y;            /* [T,H] the next block's input, or NULL; may be x */
    int64_t x_ld, resid_ld, gate_ld, resid_out_ld, y_ld; /* row strides in elements */
} moe_norm_io;

/* Per row, in fp32, each output rounded once:
 *   n  = x * w_post / sqrt(mean(x^2) + eps)    (n = x when w_post is NULL)
 *   r' = resid + alpha * g * n                 -> resid_out
 *   y  = r' * w_pre / sqrt(mean(r'^2) + eps)   (from r' before its rounding) -> y
 * At least one of x and resid, and one of resid_out and y, must be given.  No workspace;
 * deterministic.  Tensors 16-byte aligned (a per-token gate: 2), strides multiples of 8 and at
 * least H (gate_ld of a per-token gate: at least 1). */
moe_status moe_block_norm(const moe_norm_config *cfg, const moe_norm_io *io, int T, void *stream);

/* Heads and cache layout.  kv head h serves q heads h*G .. h*G+G-1, G = q_heads / kv_heads. */
typedef struct {
    int q_heads;     /* a multiple of kv_heads, G <= 128 */
    int kv_heads;
    int head_dim;    /* D: 64, 128 or 256 */
    int page_size;   /* P tokens a page: 16, 32, 64 or 128 */
    int rotary_dim;  /* leading dims that are rotated: 0, or a multiple of 16 up to D */
    int interleaved; /* 0: pairs (i, i + rotary_dim/2); 1: pairs (2i, 2i+1) */
    int dtype;       /* moe_dtype of q, k, v and the outputs */
} moe_attn_config;

/* The paged cache: keys (after the rotation) and values as E4M3 codes, each page's tokens of one
 * kv head under one fp32 scale: value = scale * code.  Scales are powers of two, 2^-60 .. 2^120:
 * the code is a float itself, so a finer scale would not add precision, and with a power of
 * two a page can move to a larger scale by an exact shift of its codes (those that become
 * subnormal round once more). */
typedef struct {
    uint8_t *k_codes; /* [n_pages, kv_heads, P, D] */
    uint8_t *v_codes; /* [n_pages, kv_heads, P, D] */
    float *k_scale;   /* [n_pages, kv_heads] */
    float *v_scale;   /* [n_pages, kv_heads] */
    int n_pages;
} moe_kv_cache;

/* A batch of sequences.  Sequence b's new tokens are rows q_start[b] .. q_start[b+1]-1 of q, k
 * and v; with n of them they have positions kv_len[b] - n .. kv_len[b] - 1.  Position p lies in
 * page page_table[b, p / P], slot p % P. */
typedef struct {
    int n_seqs;                /* B >= 0, at most 65536 */
    int n_tokens;              /* T = q_start[B] */
    int max_pages;             /* columns of page_table */
    const int32_t *q_start;    /* [B+1], q_start[0] = 0, not descending */
    const int32_t *kv_len;     /* [B] cached tokens, this batch's included */
    const int32_t *page_table; /* [B, max_pages] */
} moe_kv_batch;

/* Bytes of workspace for the two calls below on batches of up to max_seqs sequences and max_tokens
 * new tokens (the lengths in the cache do not matter).  0 for an invalid or unsupported config.
 * 256-byte aligned; zero its first 256 bytes once after allocating: they hold the status word that
 * moe_check_status reads.  The rest is scratch.  Calls that overlap must not share one. */
size_t moe_attn_workspace_size(const moe_attn_config *cfg, int max_seqs, int max_tokens);

/* Rotates q and k at their positions, writes q to q_out and k and v into the cache.
 *   rotation  (a, b) -> (a cos - b sin, b cos + a sin), cos/sin from row p of rope, fp32
 *             [rope_rows, rotary_dim]: rotary_dim/2 cosines, then rotary_dim/2 sines
 *   q_out     the rotated q rounded once to dtype (correctly: from the exact value; a pair with an
 *             infinity may give NaN)
 *   scale     per (page, kv head) the smallest power of two s with |value| <= 448 s over the
 *             page's new tokens; a page that held tokens before keeps its scale if that is
 *             larger, else its codes are re-rounded (to nearest even) under the new one
 *   codes     the E4M3 value nearest to value / s, ties to even, of the exact rotated value
 * A page written by one sequence of a call must not be written by another.  Tokens at negative
 * positions (padding in front) are not cached and give q_out rows of 0; so do rows from q_start[B] on
 * (a batch held for more tokens than it has).
 * Reported as MOE_ERR_INVALID_ARG in the status word: NaN, stored as 0; infinities (rotated
 * values past fp32 among them), stored as +-448 s under the largest scale, as 0 where the rotation's
 * formula makes them NaN; a position past rope, stored as zeros, its q_out row 0; a page id outside [0, n_pages), whose tokens are not cached; a
 * kv_len past the table (the sequence's pages and q_out rows are then unspecified).
 * q [T, q_heads, D] row stride q_ld, k and v [T, kv_heads, D] strides k_ld, v_ld, q_out stride
 * q_out_ld (q_out may be q).  q and q_out may both be NULL. */
moe_status moe_kv_append(const moe_attn_config *cfg, const moe_kv_cache *cache, const moe_kv_batch *batch,
                         const void *q, int64_t q_ld, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
                         const float *rope, int rope_rows, void *q_out, int64_t q_out_ld, void *ws,
                         size_t ws_bytes, void *stream);

/* Attention of the batch's rows over their sequences' cached tokens:
 *   out[t, h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(softmax_scale * q[t,h] . k_j)
 * over the positions j < kv_len that the masks leave for the row's position p: causal != 0:
 * j <= p; window > 0 (of any size): j > p - window.  A row that sees nothing (a negative position, an empty
 * cache) gives 0, and lse -infinity.  lse [T, q_heads] fp32 (natural log of the sum) or NULL.
 * Slots past kv_len are never used, whatever they hold; table entries of pages that no row sees (past
 * kv_len, behind every row's window) are not looked up and may hold anything.  q rows are scaled by a power of two
 * into fp16 and multiplied with the exact codes, sums and softmax statistics in fp32; for the
 * product with the values' codes, p (or p times its value's scale) is rounded to fp16, to 11 bits
 * down to 2^-23 of the row's largest, and by at most 2^-34 of it below; out is rounded once.  A row
 * does not depend on keys that it does not see, nor on their pages' scales.
 * softmax_scale > 0.  Deterministic.  A bad page id or a kv_len past the table is reported in
 * the status word (those rows are then unspecified).  Rows from q_start[B] on stay untouched. */
moe_status moe_attention(const moe_attn_config *cfg, const moe_kv_cache *cache, const moe_kv_batch *batch,
                         const void *q, int64_t q_ld, float softmax_scale, int causal, int window, void *out,
                         int64_t out_ld, float *lse, void *ws, size_t ws_bytes, void *stream);

/* ---- a recurrent token mixer: linear attention over a state, the heads' norm, products ----
 *
 * What a decoder layer without a key/value cache runs in place of the attention above ("AIMA AMD395 Qwen3.6
 * 35B Linux Engine", the HTTP prompt-length paragraph: the engine's model carries a recurrent state from piece to
 * piece of a prompt; the page gives no formula, so the readings are this library's).  The conventions of the
 * calls above hold: activations in bf16 or fp16, rows that may lie apart, a status word at the begin of the workspace. */

/* Heads.  Key head j serves the value heads j*G .. j*G+G-1, G = value_heads / key_heads. */
typedef struct {
    int key_heads;   /* KH */
    int value_heads; /* VH, a multiple of KH, at most 1024 */
    int key_dim;     /* DK: 64 or 128 */
    int value_dim;   /* DV: 64, 128 or 256 */
    int dtype;       /* moe_dtype of q, k, v and out */
} moe_linear_config;

/* The sequences' states, each [VH, DK, DV] in fp32: 16-byte aligned. */
typedef struct {
    float *states; /* [n_slots, VH, DK, DV] */
    int n_slots;
} moe_state_pool;

/* A batch of sequences.  Sequence b's new tokens are rows q_start[b] .. q_start[b+1]-1 of q, k and v; with n of
 * them they have positions kv_len[b] - n .. kv_len[b] - 1, as in moe_kv_batch. */
typedef struct {
    int n_seqs;             /* B >= 0, at most 65536 */
    int n_tokens;           /* T = q_start[B], at most 2^22 */
    const int32_t *q_start; /* [B+1], q_start[0] = 0, not descending */
    const int32_t *kv_len;  /* [B] tokens of the sequence so far, this batch's included */
    const int32_t *slots;   /* [B] where its state lies in the pool */
    int longest;            /* the most new tokens that a sequence has, or 0 where the host does not know.  Kernels are
                             * chosen by it: a value that is not so costs time, no result hangs on it */
} moe_state_batch;

/* Bytes of workspace for moe_linear_attention on batches of up to max_seqs sequences and max_tokens new
 * tokens.  0 for an invalid or unsupported config.  256-byte aligned; zero its first 256 bytes once after
 * allocating (the status word).  The rest is scratch.  Calls that overlap must not share one. */
size_t moe_linear_workspace_size(const moe_linear_config *cfg, int max_seqs, int max_tokens);

/* Linear attention with a decay for each value head.  Token by token, for every value head h and its key head j:
 *   S   = e^g S + k v^T          S [DK, DV] the sequence's state, g the token's log decay
 *   out = scale * S^T q
 * A sequence whose first new token has position 0 (kv_len = n) begins with S = 0, whatever its slot holds; any other
 * begins with its slot's state.  The state after its last new token is written to the slot: who may want to take tokens
 * back copies the slot first.  A sequence without new tokens leaves its slot alone.  Tokens at negative positions (padding in front) do not count, and get out rows of 0.
 * Rows from q_start[B] on stay untouched.
 * q, k [T, KH, DK], v, out [T, VH, DV], row strides q_ld, k_ld, v_ld, out_ld.  decay fp32, g <= 0: [T, VH] with row
 * stride decay_ld >= VH, or with decay_ld = 0 one value a head, [VH]; NULL: g = 0.  g = -infinity forgets the
 * state; below -10,000 a decay counts as that (its factor is 0 either way).
 * States and sums are fp32.  Long runs are computed chunk by chunk, 64 tokens each, on tensor cores, whose operands are sums
 * of 16-bit values.  What enters a state, a token's value times its decay up to the chunk's end, has 24 bits with bf16 and 22
 * with fp16; what an output sees, the state at the chunk's begin and the decayed products of queries and keys, 16 with bf16
 * and 22 with fp16.  With fp16 that holds down to 2^-17, and what is smaller is kept to 2^-39, of the largest one of the same
 * channel and chunk, channel of the state, or query.  out is rounded once.  Factors below 2^-126 count as 0.  Deterministic, but a run's length decides which kernel takes it, so the last bits of a
 * state depend on how a prompt is cut.  A value of v that is not finite makes its channel not finite from its token on.
 * Reported as MOE_ERR_INVALID_ARG in the status word: a slot outside [0, n_slots) (the sequence begins with S = 0
 * and its state is not kept); a range of rows outside the batch (no tokens); a decay above 0 or NaN (taken as 0).
 * Two sequences of a call must not have the same slot.  out must not overlap q, k, v or decay. */
moe_status moe_linear_attention(const moe_linear_config *cfg, const moe_state_pool *pool, const moe_state_batch *batch,
                                const void *q, int64_t q_ld, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
                                const float *decay, int64_t decay_ld, float scale, void *out, int64_t out_ld, void *ws,
                                size_t ws_bytes, void *stream);

typedef enum {
    MOE_HEAD_GATE_NONE = 0,
    MOE_HEAD_GATE_SIGMOID = 1, /* 1 / (1 + e^-gate) */
    MOE_HEAD_GATE_SILU = 2     /* gate / (1 + e^-gate) */
} moe_head_gate;

typedef struct {
    int heads;       /* >= 1; heads * dim at most 65536 */
    int dim;         /* D, a multiple of 8, at most 1024 */
    int dtype;       /* moe_dtype of every tensor of the call */
    int center;      /* 1: the head's mean is taken off first */
    int gate;        /* moe_head_gate */
    int weight_each; /* 0: one weight [D] for all heads; 1: [heads, D] */
    int unit_offset; /* 1: the weights are stored as w - 1 */
    float eps;       /* added to the mean square, >= 0 */
} moe_head_norm_config;

/* The norm of each head of each row, with its weight and gate, in fp32, rounded once:
 *   y = (x - m) * w / sqrt(mean((x - m)^2) + eps) * act(gate),  m = mean(x) with center, else 0
 * x, gate, y [T, heads, D], row strides x_ld, gate_ld, y_ld in elements (multiples of 8, at least heads * D); y may be
 * x or gate.  act is good to 2^-16, and 0 below gate = -87.  weight may be NULL (1); gate is NULL with MOE_HEAD_GATE_NONE
 * only.  16-byte aligned.  No workspace; deterministic. */
moe_status moe_head_norm(const moe_head_norm_config *cfg, const void *x, int64_t x_ld, const void *weight,
                         const void *gate, int64_t gate_ld, void *y, int64_t y_ld, int T, void *stream);

typedef enum {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,
    MOE_ACT_GELU = 2, /* z (1 + erf(z / sqrt(2))) / 2 */
    MOE_ACT_SILU = 3,
    MOE_ACT_SIGMOID = 4,
    MOE_ACT_LOG_SIGMOID = 5 /* -log(1 + e^-z): a log decay */
} moe_act;

typedef struct {
    int inputs;  /* K, a multiple of 8, at most 65536 */
    int outputs; /* N, a multiple of 8, at most 2^20 */
    int dtype;   /* moe_dtype of x, w and bias */
    int out_f32; /* 1: y and resid are fp32, 0: of dtype */
    int act;     /* moe_act */
    float scale; /* alpha */
} moe_project_config;

typedef struct {
    const void *x;     /* [T,K] */
    const void *w;     /* [N,K] */
    const void *bias;  /* [N] or NULL */
    const void *resid; /* [T,N] or NULL; may be y */
    void *y;           /* [T,N] */
    int64_t x_ld, w_ld, resid_ld, y_ld; /* row strides in elements, multiples of 8 */
} moe_project_io;

/* Bytes of workspace for moe_project on up to max_T rows, as above (status word, then scratch). */
size_t moe_project_workspace_size(const moe_project_config *cfg, int max_T);

/* y = resid + alpha * act(x w^T + bias): 16-bit products, sums and epilogue in fp32, rounded once.
 * With 16-bit y the sigmoid's e^-z is good to 2^-16, and below z = -87 sigmoid and SiLU are 0; with fp32 y both keep a few
 * ulp of the result down to fp32's least value.
 * Deterministic.  T of 0 does nothing, more than 2^30 rows are not supported.  y must not overlap x or w. */
moe_status moe_project(const moe_project_config *cfg, const moe_project_io *io, int T, void *ws, size_t ws_bytes,
                       void *stream);

/* Reads and clears the device status word in `ws` (synchronises `stream`).  *device_status
 * receives MOE_OK or the first error recorded by a kernel (MOE_ERR_TIMEOUT for a wait that
 * ran out, MOE_ERR_INVALID_ARG for an out-of-range expert id).  Returns MOE_ERR_CUDA if the
 * copy fails. */
moe_status moe_check_status(void *ws, size_t ws_bytes, int *device_status, void *stream);

/* Diagnostics, not a step of the layer: one device thread waits on a barrier with the same
 * bounded wait every pipeline of this library uses.  With arrive != 0 the barrier completes
 * first and the wait returns at once; with arrive == 0 nothing arrives, the wait gives up after
 * limit_ns nanoseconds (at most 1e9) and records MOE_ERR_TIMEOUT in the workspace status word,
 * which moe_check_status then reports.  No fault, trap or hang: the kernel returns, and the
 * stream and context stay usable.  ws: at least the 256-byte status area of a workspace
 * (256-byte aligned).  Returns MOE_ERR_INVALID_ARG for a bad workspace or limit. */
moe_status moe_selftest_wait(void *ws, size_t ws_bytes, unsigned long long limit_ns, int arrive,
                             void *stream);

/* Sizes of the pieces moe_forward splits T into: writes up to max_pieces sizes to `pieces`
 * and returns the number of pieces (host only, no device work); -1 if T < 0. */
int moe_plan_pieces(int T, int *pieces, int max_pieces);

/* Number of kernels this library has launched in this process (host counter). */
uint64_t moe_launch_count(void);

/* Optional per-kernel timing.  While enabled, every kernel launch is bracketed by CUDA events
 * on its stream; moe_timing_read() synchronises them and returns, for kernel class `name`
 * (see moe_timing_name()), the number of launches and their total device time in ms, then
 * forgets them.  Returns MOE_ERR_INVALID_ARG for an unknown name.  Not for use inside CUDA
 * graph capture. */
moe_status moe_timing_enable(int enable);
moe_status moe_timing_read(const char *name, int *launches, double *total_ms);
/* 1 when this library was built with MOE_DEBUG: every kernel then checks each index it reads from
 * device data (permutation rows, caller-given expert offsets, combine rows, GEMM output rows)
 * before using it, records MOE_ERR_INVALID_ARG in the workspace status word (moe_combine has
 * none) and skips the access.  0 for the ordinary build, which does not check them. */
int moe_debug_build(void);

/* Name of kernel class i (0 <= i < moe_timing_classes()), or NULL. */
const char *moe_timing_name(int i);
int moe_timing_classes(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
