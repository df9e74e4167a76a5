// layer_abi.cu -- the extern "C" entry points of the decoder layer's other half (include/moe.h):
// argument checks, workspace carving, launches.
#include <climits>
#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "layer.h"

namespace moe {
namespace {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool good_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

#define MOE_TRY(expr)                  \
    do {                               \
        moe_status _st = (expr);       \
        if (_st != MOE_OK) return _st; \
    } while (0)
#define MOE_CUDA(expr) MOE_TRY((expr) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA)

// A row of `width` 16-bit values read or written in 16-byte pieces.
bool good_rows(const void *p, int64_t ld, int64_t width) { return p && aligned16(p) && ld >= width && ld % 8 == 0; }

moe_status check_attn_config(const moe_attn_config *c) {
    if (!c || c->q_heads <= 0 || c->kv_heads <= 0 || !good_dtype(c->dtype)) return MOE_ERR_INVALID_ARG;
    if (c->rotary_dim < 0 || (c->interleaved != 0 && c->interleaved != 1)) return MOE_ERR_INVALID_ARG;
    if (c->q_heads % c->kv_heads) return MOE_ERR_INVALID_ARG;
    if (c->q_heads / c->kv_heads > 128 || c->q_heads > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c->rotary_dim > c->head_dim) return MOE_ERR_INVALID_ARG;
    if (c->rotary_dim % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// Limits on a batch's size: they keep every count of rows, pages and steps inside 32 bits.
constexpr int kMaxSeqs = 65536;
constexpr int kMaxTokens = 1 << 22;

moe_status check_batch(const moe_attn_config &c, const moe_kv_cache *k, const moe_kv_batch *b) {
    if (!k || !b) return MOE_ERR_INVALID_ARG;
    if (b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages < 0 || k->n_pages < 0) return MOE_ERR_INVALID_ARG;
    if (b->n_seqs == 0 && b->n_tokens > 0) return MOE_ERR_INVALID_ARG;
    if (b->n_seqs > kMaxSeqs || b->n_tokens > kMaxTokens) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)b->max_pages * c.page_size > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((int64_t)k->n_pages * c.kv_heads > INT_MAX) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (b->n_tokens == 0) return MOE_OK;
    if (!b->q_start || !b->kv_len) return MOE_ERR_INVALID_ARG;
    if (b->max_pages > 0 && !b->page_table) return MOE_ERR_INVALID_ARG;
    if (k->n_pages < 1 || !k->k_codes || !k->v_codes || !k->k_scale || !k->v_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(k->k_codes) || !aligned16(k->v_codes)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Query rows a kv head from which a sequence goes to the prompt kernel.
constexpr int kPromptRows = 128;
// Mean rows a sequence and kv head below which a batch is a decode step, all of it the split kernel's.
constexpr int kPromptMean = 33;
// Rows in all (tokens x q heads) from which the prompt kernel is worth it: a block of it takes 256 rows (D = 256: 128)
// at the price of a long start and a join of parts, the split kernel 8.  us of the prompt kernel and the split one,
// 8 q heads, 1 kv head: 2048 rows, D = 64, 1024 keys 17.7 and 17.7, 4096 26.8 and 25.4, 16,384 26.8 and 57.6; D = 128, 22.9
// and 23.4, 33.0 and 36.3, 31.8 and 89.0; D = 256, 28.1 and 29.2, 41 and 54, 52 and 155; 1024 rows, D = 128, 23.0 and 17.8,
// 28.5 and 27.9, 29.7 and 52.4.  A prompt without a past, D = 128: 1024 rows 12.9 and 8.9, 2048 14.3 and 13.7, 4096 17.8
// and 22.4.  So half as many from 8192 keys on.  Several sequences, some of which may be short and the split
// kernel's after the other two, need twice as many: 6 of up to 247 tokens, 8 and 4 heads of 128, 4000 rows, 2356
// keys, 45.7 and 32.4.
constexpr int64_t kPromptWork = 2048, kPromptKeys = 8192;
// From this many steps a block times row tiles a sequence (4 at most), the split kernel's row tiles share key
// tiles.  Below, the SMs are short of work and more, smaller segments end sooner.  us shared and not, at 304 blocks,
// D = 128, groups of 8, 2 kv heads: 4 tiles, 8 sequences of 4000 keys (26) 20.5 and 20.0, of 10,000 (66) 27.9
// and 29.8, of 32,000 (211) 53.6 and 76.6; 3 tiles, 16 of 4000 (30) 25.2 and 24.0, 32 of 4000 (61) 37.3 and 40.2;
// 2 tiles, 32 of 4000 (27) 35.0 and 30.3, 32 of 16,000 (105) 87.1 and 94.1; D = 256, 4 kv heads, 4 tiles: 8 of
// 4000 (54) 27.4 and 27.3, of 16,000 (211) 59.6 and 89.4.
constexpr int kManySteps = 56;

// Rows of partial results that the prompt kernel's parts may have: a block an SM twice over.
int64_t part_rows(const moe_attn_config &c, int64_t n_tokens) {
    const int64_t rows = n_tokens * c.q_heads, most = (int64_t)kSplitMaxBlocks * prompt_block_rows(c.head_dim);
    return rows * kPromptParts < most ? rows * kPromptParts : most;
}
struct Layout {
    size_t desc, part, prompt_out, prompt_lse, total;
};
Layout layout(const moe_attn_config &c, int n_tokens) {
    Layout l;
    l.desc = 256;  // behind the status word
    l.part = l.desc + (kSplitMaxBlocks * sizeof(SplitDesc) + 255) / 256 * 256;
    l.prompt_out = l.part + (split_part_floats(c.head_dim) * sizeof(float) + 255) / 256 * 256;
    l.prompt_lse = l.prompt_out + part_rows(c, n_tokens) * c.head_dim * sizeof(float);
    l.total = l.prompt_lse + part_rows(c, n_tokens) * sizeof(float);
    return l;
}

// Parts of a prompt's keys: where its blocks leave SMs idle, each block's keys are shared out over several: as
// many as end soonest, in tiles of 128 keys (1.4 us at D = 128), a block's start counted as 5 and the join as 4.
int prompt_parts(const moe_attn_config &c, const moe_kv_batch &b, int64_t rows, int64_t keys) {
    const int sms = device_info().sm_count, block = prompt_block_rows(c.head_dim);
    const int64_t blocks = (rows + block - 1) / block * c.kv_heads, all = (int64_t)b.n_tokens * c.q_heads;
    if (blocks >= sms || b.n_seqs > 32) return 1;
    int best = 1;
    const double tiles = (double)keys / 128;
    double least = tiles + 5;
    for (int k = 2; k <= kPromptParts && k * all <= part_rows(c, b.n_tokens) && k * 1024 <= keys; ++k) {
        const double cost = (double)((blocks * k + sms - 1) / sms) * (tiles / k + 5) + 4 + 0.2 * k;
        if (cost < least) least = cost, best = k;
    }
    return best;
}

moe_status check_ws(const moe_attn_config &c, int n_tokens, const void *ws, size_t bytes) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOE_ERR_INVALID_ARG;
    if (bytes < layout(c, n_tokens).total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    return MOE_OK;
}

KvView view(const moe_attn_config &c, const moe_kv_cache &k, const moe_kv_batch &b, void *ws) {
    KvView v{};
    v.q_start = b.q_start;
    v.kv_len = b.kv_len;
    v.table = b.page_table;
    v.k_codes = k.k_codes;
    v.v_codes = k.v_codes;
    v.k_scale = k.k_scale;
    v.v_scale = k.v_scale;
    v.n_seqs = b.n_seqs;
    v.n_tokens = b.n_tokens;
    v.max_pages = b.max_pages;
    v.n_pages = k.n_pages;
    v.QH = c.q_heads;
    v.KH = c.kv_heads;
    v.G = c.q_heads / c.kv_heads;
    v.P = c.page_size;
    while ((1 << v.log_p) < v.P) ++v.log_p;
    v.status = static_cast<int *>(ws);
    return v;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_block_norm(const moe_norm_config *cfg, const moe_norm_io *io, int T, void *stream) {
    NvtxRange nvtx_range("moe_block_norm");
    if (!cfg || T < 0 || !good_dtype(cfg->dtype) || cfg->hidden <= 0) return MOE_ERR_INVALID_ARG;
    if (cfg->gate < MOE_GATE_NONE || cfg->gate > MOE_GATE_ELEMENT) return MOE_ERR_INVALID_ARG;
    if (!(cfg->eps >= 0.f) || !std::isfinite(cfg->eps) || !std::isfinite(cfg->residual_scale)) return MOE_ERR_INVALID_ARG;
    if (cfg->hidden % 8 || cfg->hidden > 16384) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!io) return MOE_ERR_INVALID_ARG;
    const int64_t H = cfg->hidden;
    if (!io->x && !io->resid) return MOE_ERR_INVALID_ARG;
    if (!io->resid_out && !io->y) return MOE_ERR_INVALID_ARG;
    if (io->x && !good_rows(io->x, io->x_ld, H)) return MOE_ERR_INVALID_ARG;
    if (io->resid && !good_rows(io->resid, io->resid_ld, H)) return MOE_ERR_INVALID_ARG;
    if (io->resid_out && !good_rows(io->resid_out, io->resid_out_ld, H)) return MOE_ERR_INVALID_ARG;
    if (io->y && (!good_rows(io->y, io->y_ld, H) || !io->w_pre)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(io->w_post) || !aligned16(io->w_pre)) return MOE_ERR_INVALID_ARG;
    // without a block there is nothing for a gate or a post norm to act on
    if (!io->x && (io->w_post || cfg->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((cfg->gate == MOE_GATE_NONE) != (io->gate == nullptr)) return MOE_ERR_INVALID_ARG;
    if (cfg->gate == MOE_GATE_CHANNEL && !aligned16(io->gate)) return MOE_ERR_INVALID_ARG;
    if (cfg->gate == MOE_GATE_ELEMENT && !good_rows(io->gate, io->gate_ld, H)) return MOE_ERR_INVALID_ARG;
    if (cfg->gate == MOE_GATE_TOKEN && (io->gate_ld < 1 || (reinterpret_cast<uintptr_t>(io->gate) & 1u)))
        return MOE_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = static_cast<const uint16_t *>(io->x);
    a.resid = static_cast<const uint16_t *>(io->resid);
    a.gate = static_cast<const uint16_t *>(io->gate);
    a.w_post = static_cast<const uint16_t *>(io->w_post);
    a.w_pre = static_cast<const uint16_t *>(io->w_pre);
    a.resid_out = static_cast<uint16_t *>(io->resid_out);
    a.y = static_cast<uint16_t *>(io->y);
    a.x_ld = io->x_ld;
    a.resid_ld = io->resid_ld;
    a.gate_ld = io->gate_ld;
    a.resid_out_ld = io->resid_out_ld;
    a.y_ld = io->y_ld;
    a.T = T;
    a.H = cfg->hidden;
    a.gate_kind = cfg->gate;
    a.sigmoid = cfg->gate_sigmoid;
    a.unit_offset = cfg->unit_offset;
    a.eps = cfg->eps;
    a.alpha = cfg->residual_scale;
    MOE_CUDA(launch_block_norm(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

size_t moe_attn_workspace_size(const moe_attn_config *cfg, int max_seqs, int max_tokens) {
    if (check_attn_config(cfg) != MOE_OK || max_seqs < 0 || max_tokens < 0) return 0;
    if (max_seqs > kMaxSeqs || max_tokens > kMaxTokens) return 0;
    return layout(*cfg, max_tokens).total;
}

moe_status moe_kv_append(const moe_attn_config *cfg, const moe_kv_cache *cache, const moe_kv_batch *batch,
                         const void *q, int64_t q_ld, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
                         const float *rope, int rope_rows, void *q_out, int64_t q_out_ld, void *ws,
                         size_t ws_bytes, void *stream) {
    NvtxRange nvtx_range("moe_kv_append");
    MOE_TRY(check_attn_config(cfg));
    const moe_attn_config &c = *cfg;
    MOE_TRY(check_batch(c, cache, batch));
    if (batch->n_tokens == 0) return MOE_OK;
    const int64_t D = c.head_dim;
    if (!good_rows(k, k_ld, c.kv_heads * D) || !good_rows(v, v_ld, c.kv_heads * D)) return MOE_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr)) return MOE_ERR_INVALID_ARG;
    if (q && (!good_rows(q, q_ld, c.q_heads * D) || !good_rows(q_out, q_out_ld, c.q_heads * D))) return MOE_ERR_INVALID_ARG;
    if (c.rotary_dim > 0 && (!rope || !aligned16(rope) || rope_rows < 1)) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_ws(c, batch->n_tokens, ws, ws_bytes));
    AppendArgs a{};
    a.kv = view(c, *cache, *batch, ws);
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.q_out_ld = q_out_ld;
    a.rope = rope;
    a.rope_rows = rope_rows;
    a.rot = c.rotary_dim;
    a.interleaved = c.interleaved;
    const int64_t items = ((int64_t)(batch->n_tokens >> a.kv.log_p) + 2 * (int64_t)batch->n_seqs) * 2 * c.kv_heads;
    if (items > (1 << 30)) return MOE_ERR_UNSUPPORTED_SHAPE;
    a.page_items = (int)items;
    // a block of the q part takes as many tokens as fill its threads once, fewer while that leaves SMs idle
    const int groups = (c.q_heads + 1) / 2, once = 256 / (c.head_dim / 16) / groups;
    const int spread = batch->n_tokens / (2 * device_info().sm_count);
    a.q_tokens = spread < 1 || once < 1 ? 1 : spread > once ? once : spread;
    MOE_CUDA(launch_kv_append(a, c.head_dim, c.dtype, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

moe_status moe_attention(const moe_attn_config *cfg, const moe_kv_cache *cache, const moe_kv_batch *batch,
                         const void *q, int64_t q_ld, float softmax_scale, int causal, int window, void *out,
                         int64_t out_ld, float *lse, void *ws, size_t ws_bytes, void *stream) {
    NvtxRange nvtx_range("moe_attention");
    MOE_TRY(check_attn_config(cfg));
    const moe_attn_config &c = *cfg;
    MOE_TRY(check_batch(c, cache, batch));
    if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale) || window < 0) return MOE_ERR_INVALID_ARG;
    if (batch->n_tokens == 0) return MOE_OK;
    const int64_t width = (int64_t)c.q_heads * c.head_dim;
    if (!good_rows(q, q_ld, width) || !good_rows(out, out_ld, width)) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(lse) & 3u) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_ws(c, batch->n_tokens, ws, ws_bytes));
    const Layout l = layout(c, batch->n_tokens);
    AttnArgs a{};
    a.kv = view(c, *cache, *batch, ws);
    a.q = static_cast<const uint16_t *>(q);
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.q_ld = q_ld;
    a.out_ld = out_ld;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.causal = causal != 0;
    // A window as long as the table masks nothing (a position is less than its length); the kernels' 32-bit
    // pos + 1 - window, pos >= -n_tokens, could not hold a much longer one.
    const int64_t table = (int64_t)batch->max_pages * c.page_size;
    a.window = window < table ? window : 0;
    a.desc = reinterpret_cast<SplitDesc *>(static_cast<char *>(ws) + l.desc);
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + l.part);
    a.part_out = reinterpret_cast<float *>(static_cast<char *>(ws) + l.prompt_out);
    a.part_lse = reinterpret_cast<float *>(static_cast<char *>(ws) + l.prompt_lse);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Which sequences the prompt kernel takes goes by their own rows, which only the device knows.  The host
    // leaves a kernel out that has none for sure, and the prompt kernel in a step of few tokens a
    // sequence: its launch would cost more (5 us) than the rare long run among them.
    const int64_t rows = (int64_t)batch->n_tokens * a.kv.G, mean = rows / batch->n_seqs;
    // keys a sequence has to look at, at most
    const int64_t seen = a.window > 0 ? (int64_t)a.window + batch->n_tokens : INT64_MAX, keys = seen < table ? seen : table;
    const int64_t work = kPromptWork * (batch->n_seqs == 1 ? 2 : 4) / (keys >= kPromptKeys ? 4 : 2);
    const bool prompts = rows >= kPromptRows && mean >= kPromptMean && rows * c.kv_heads >= work;
    a.prompt_rows = !prompts ? INT_MAX : batch->n_seqs == 1 ? 1 : kPromptRows;
    a.parts = prompts ? prompt_parts(c, *batch, rows, keys) : 1;
    if (prompts) MOE_CUDA(launch_attn_prompt(a, c.head_dim, c.dtype, s));
    if (batch->n_seqs > 1 || !prompts) {
        // steps of the split kernel with one row tile a segment, at most
        const int64_t steps = (rows + 7) / 8 * c.kv_heads * ((keys + 127) / 128), tiles = mean > 24 ? 4 : (mean + 7) / 8;
        const bool shared = tiles > 1 && steps * tiles >= (int64_t)kManySteps * 2 * device_info().sm_count;
        MOE_CUDA(launch_attn_split(a, c.head_dim, c.dtype, shared, prompts && a.parts == 1, s));
    }
    return MOE_OK;
}

}  // extern "C"
