// mixer_abi.cu -- the extern "C" entry points of the recurrent token mixer (include/moe.h): argument checks,
// workspace carving, launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include <nvtx3/nvToolsExt.h>

#include "mixer.h"

namespace moe {
namespace {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool good_dtype(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

#define MOE_TRY(expr)                  \
    do {                               \
        moe_status _st = (expr);       \
        if (_st != MOE_OK) return _st; \
    } while (0)
#define MOE_CUDA(expr) MOE_TRY(cuda_status(expr))

// A row of `width` values read or written in 16-byte pieces.
bool good_rows(const void *p, int64_t ld, int64_t width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0; }

// Limits on a batch's size: they keep counts of rows inside 32 bits.
constexpr int kMaxSeqs = 65536;
constexpr int kMaxTokens = 1 << 22;

moe_status check_linear_config(const moe_linear_config *c) {
    if (!c || c->key_heads <= 0 || c->value_heads <= 0 || !good_dtype(c->dtype)) return MOE_ERR_INVALID_ARG;
    if (c->value_heads % c->key_heads) return MOE_ERR_INVALID_ARG;
    if (c->value_heads > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c->key_dim != 64 && c->key_dim != 128) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (c->value_dim != 64 && c->value_dim != 128 && c->value_dim != 256) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// New tokens from which a run is the chunk kernel's, and the same with several heads an SM, where the SMs are busy either way.
// us token by token and in chunks, 32 heads of 128 and 128: one run of 8 tokens 12 and 8; 16 sequences of 8 30 and 38, of 16 47 and
// 39; 64 of 16 159 and 137, of 32 275 and 139; 200 of 8 289 and 410.
constexpr int kChunkTokens = 8, kManyTokens = 16;
// Segments times heads times column tiles that a batch may have when its runs are cut: the states they add are in the workspace.
constexpr int64_t kMostSegments = 640;

int value_tiles(const moe_linear_config &c) { return c.value_dim > 128 ? 2 : 1; }
int64_t most_segments(const moe_linear_config &c, int64_t n_seqs, int64_t n_tokens) {
    const int64_t n = (n_tokens / kChunk + n_seqs) * c.value_heads * value_tiles(c);
    return n < kMostSegments ? n : kMostSegments;
}
struct LinearLayout {
    size_t decay, states, total;
};
LinearLayout linear_layout(const moe_linear_config &c, int n_seqs, int n_tokens) {
    const size_t n = (size_t)most_segments(c, n_seqs, n_tokens);
    LinearLayout l;
    l.decay = 256;  // behind the status word
    l.states = l.decay + (n * sizeof(float) + 255) / 256 * 256;
    l.total = l.states + n * c.key_dim * (c.value_dim / value_tiles(c)) * sizeof(float);
    return l;
}

// Chunks a segment: as many as end soonest.  Measured, us: a block of the output kernel 8, 2.2 a chunk and 0.6 a segment
// before its own, a block of the first kernel 5 and 1.2 a chunk.
int segment_chunks(const moe_linear_config &c, int64_t n_seqs, int64_t n_tokens) {
    const int sms = device_info().sm_count;
    const double chunks = (double)((n_tokens + kChunk - 1) / kChunk), per = (double)c.value_heads * value_tiles(c) / sms;
    // a batch's longest run: all of it, or of several four times the mean
    const double longest = n_seqs == 1 ? chunks : fmin(chunks, 4 * chunks / n_seqs + 1);
    // time of `n` blocks a head of up to l chunks: equal ones go by rounds, ragged ones fill gaps
    auto walk = [&](double n, double l, double start, double each) {
        if (n_seqs == 1) return ceil(n * per) * (start + each * l);
        return fmax(start + each * l, n * per * start + chunks * per * each + each * l / 2);
    };
    int64_t best = (int64_t)chunks;
    double least = walk((double)n_seqs, longest, 8, 2.2);
    for (int64_t l = 2; l < longest; l += l < 32 ? 1 : l / 16) {
        if ((n_tokens / (l * kChunk) + n_seqs) * c.value_heads * value_tiles(c) > kMostSegments) continue;
        const double n = n_seqs == 1 ? ceil(chunks / l) : chunks / l + 0.6 * n_seqs;
        const double cost = walk(n, (double)l, 8 + 0.6 * (n_seqs == 1 ? n : longest / l), 2.2) + walk(n_seqs == 1 ? n - 1 : chunks / l, (double)l, 5, 1.2);
        if (cost < least) least = cost, best = l;
    }
    return (int)best;
}

moe_status check_project_config(const moe_project_config *c) {
    if (!c || c->inputs <= 0 || c->outputs <= 0 || !good_dtype(c->dtype)) return MOE_ERR_INVALID_ARG;
    if (c->out_f32 != 0 && c->out_f32 != 1) return MOE_ERR_INVALID_ARG;
    if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_LOG_SIGMOID || !std::isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
    if (c->inputs % 8 || c->outputs % 8 || c->inputs > 65536 || c->outputs > 1 << 20) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

size_t project_workspace(const moe_project_config &, int) { return 256; }

moe_status check_ws(const void *ws, size_t bytes, size_t need) {
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    return bytes < need ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_config *cfg, int max_seqs, int max_tokens) {
    if (check_linear_config(cfg) != MOE_OK || max_seqs < 0 || max_tokens < 0) return 0;
    if (max_seqs > kMaxSeqs || max_tokens > kMaxTokens) return 0;
    return linear_layout(*cfg, max_seqs, max_tokens).total;
}

moe_status moe_linear_attention(const moe_linear_config *cfg, const moe_state_pool *pool, const moe_state_batch *batch,
                                const void *q, int64_t q_ld, const void *k, int64_t k_ld, const void *v, int64_t v_ld,
                                const float *decay, int64_t decay_ld, float scale, void *out, int64_t out_ld, void *ws,
                                size_t ws_bytes, void *stream) {
    NvtxRange nvtx_range("moe_linear_attention");
    MOE_TRY(check_linear_config(cfg));
    const moe_linear_config &c = *cfg;
    if (!pool || !batch || batch->n_seqs < 0 || batch->n_tokens < 0 || pool->n_slots < 0) return MOE_ERR_INVALID_ARG;
    if (batch->longest < 0 || (batch->n_seqs == 0 && batch->n_tokens > 0)) return MOE_ERR_INVALID_ARG;
    if (batch->n_seqs > kMaxSeqs || batch->n_tokens > kMaxTokens) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    if (batch->n_tokens == 0) return MOE_OK;
    if (!batch->q_start || !batch->kv_len || !batch->slots) return MOE_ERR_INVALID_ARG;
    if (pool->n_slots < 1 || !pool->states || !aligned(pool->states, 16)) return MOE_ERR_INVALID_ARG;
    const int64_t kw = (int64_t)c.key_heads * c.key_dim, vw = (int64_t)c.value_heads * c.value_dim;
    if (!good_rows(q, q_ld, kw) || !good_rows(k, k_ld, kw) || !good_rows(v, v_ld, vw) || !good_rows(out, out_ld, vw))
        return MOE_ERR_INVALID_ARG;
    if (decay && (!aligned(decay, 4) || (decay_ld != 0 && decay_ld < c.value_heads))) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_ws(ws, ws_bytes, linear_layout(c, batch->n_seqs, batch->n_tokens).total));
    LinearArgs a{};
    a.q_start = batch->q_start;
    a.kv_len = batch->kv_len;
    a.slots = batch->slots;
    a.states = pool->states;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.decay = decay;
    a.out = static_cast<uint16_t *>(out);
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.out_ld = out_ld;
    a.decay_ld = decay_ld;
    a.n_seqs = batch->n_seqs;
    a.n_tokens = batch->n_tokens;
    a.n_slots = pool->n_slots;
    a.KH = c.key_heads;
    a.VH = c.value_heads;
    a.G = c.value_heads / c.key_heads;
    a.DK = c.key_dim;
    a.DV = c.value_dim;
    a.scale = scale;
    a.status = static_cast<int *>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Which runs the chunk kernel takes goes by their own lengths, which only the device knows.  The host leaves a
    // kernel out that has none for sure, and the chunk kernel in steps of a few tokens a sequence (drafts), where its launch
    // would cost more than a longer run among them (of up to 64 tokens, 1.2 us each).  Where the caller does not say how long runs
    // are, it is taken that every sequence has a token in batches of up to 127 tokens, and nothing in larger ones, where one may have
    // all of them: their launch may be in vain (us without and with it, single tokens, 32 heads of 128 and 128: 128 sequences 88
    // and 92, 200 136 and 142, 1000 683 and 709), but 1050 tokens among 999 empty sequences took 815 without it and take 129.
    const int n = batch->n_tokens, more = n - batch->n_seqs;
    const int longest = batch->longest > 0 ? std::min(batch->longest, n) : n >= 128 ? n : more + 1;
    const bool chunks = batch->n_seqs == 1 ? n >= kChunkTokens : longest > 64 || n >= kChunkTokens * batch->n_seqs;
    const bool many = (int64_t)batch->n_seqs * c.value_heads * value_tiles(c) > 2 * device_info().sm_count;
    a.chunk_tokens = !chunks ? INT_MAX : batch->n_seqs == 1 ? 0 : many ? kManyTokens : kChunkTokens;
    if (chunks) {
        a.place_tokens = many && batch->n_tokens / kManyTokens < batch->n_seqs ? kManyTokens : 0;
        a.segment_chunks = segment_chunks(c, batch->n_seqs, batch->n_tokens);
        const LinearLayout l = linear_layout(c, batch->n_seqs, batch->n_tokens);
        if ((int64_t)a.segment_chunks * kChunk < batch->n_tokens) {
            a.seg_decay = reinterpret_cast<float *>(static_cast<char *>(ws) + l.decay);
            a.seg_states = reinterpret_cast<float *>(static_cast<char *>(ws) + l.states);
        }
        MOE_CUDA(launch_linear_chunks(a, c.dtype, s));
    }
    // Beside the chunk kernel, but for a launch that may well be in vain: single tokens take a tenth longer beside one
    // (200 sequences 153 us for 142).
    const bool beside = chunks && (batch->longest > 0 || more >= 64);
    if (!chunks || batch->n_seqs > 1) MOE_CUDA(launch_linear_tokens(a, c.dtype, beside, s));
    return MOE_OK;
}

moe_status moe_head_norm(const moe_head_norm_config *cfg, const void *x, int64_t x_ld, const void *weight,
                         const void *gate, int64_t gate_ld, void *y, int64_t y_ld, int T, void *stream) {
    NvtxRange nvtx_range("moe_head_norm");
    if (!cfg || T < 0 || cfg->heads <= 0 || cfg->dim <= 0 || !good_dtype(cfg->dtype)) return MOE_ERR_INVALID_ARG;
    if (cfg->gate < MOE_HEAD_GATE_NONE || cfg->gate > MOE_HEAD_GATE_SILU) return MOE_ERR_INVALID_ARG;
    if (!(cfg->eps >= 0.f) || !std::isfinite(cfg->eps)) return MOE_ERR_INVALID_ARG;
    if (cfg->dim % 8 || cfg->dim > 1024 || (int64_t)cfg->heads * cfg->dim > 65536) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    const int64_t width = (int64_t)cfg->heads * cfg->dim;
    if (!good_rows(x, x_ld, width) || !good_rows(y, y_ld, width) || !aligned(weight, 16)) return MOE_ERR_INVALID_ARG;
    if ((cfg->gate == MOE_HEAD_GATE_NONE) != (gate == nullptr)) return MOE_ERR_INVALID_ARG;
    if (gate && !good_rows(gate, gate_ld, width)) return MOE_ERR_INVALID_ARG;
    HeadNormArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.weight = static_cast<const uint16_t *>(weight);
    a.gate = static_cast<const uint16_t *>(gate);
    a.y = static_cast<uint16_t *>(y);
    a.x_ld = x_ld;
    a.gate_ld = gate_ld;
    a.y_ld = y_ld;
    a.T = T;
    a.heads = cfg->heads;
    a.dim = cfg->dim;
    a.center = cfg->center;
    a.gate_kind = cfg->gate;
    a.weight_each = cfg->weight_each;
    a.unit_offset = cfg->unit_offset;
    a.eps = cfg->eps;
    MOE_CUDA(launch_head_norm(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
    return MOE_OK;
}

size_t moe_project_workspace_size(const moe_project_config *cfg, int max_T) {
    if (check_project_config(cfg) != MOE_OK || max_T < 0) return 0;
    return project_workspace(*cfg, max_T);
}

moe_status moe_project(const moe_project_config *cfg, const moe_project_io *io, int T, void *ws, size_t ws_bytes,
                       void *stream) {
    NvtxRange nvtx_range("moe_project");
    MOE_TRY(check_project_config(cfg));
    const moe_project_config &c = *cfg;
    if (T < 0) return MOE_ERR_INVALID_ARG;
    if (T > 1 << 30) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!io || !good_rows(io->x, io->x_ld, c.inputs) || !good_rows(io->w, io->w_ld, c.inputs)) return MOE_ERR_INVALID_ARG;
    if (!good_rows(io->y, io->y_ld, c.outputs) || !aligned(io->bias, 16)) return MOE_ERR_INVALID_ARG;
    if (io->resid && !good_rows(io->resid, io->resid_ld, c.outputs)) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_ws(ws, ws_bytes, project_workspace(c, T)));
    ProjectArgs a{};
    a.x = static_cast<const uint16_t *>(io->x);
    a.w = static_cast<const uint16_t *>(io->w);
    a.bias = static_cast<const uint16_t *>(io->bias);
    a.resid = io->resid;
    a.y = io->y;
    a.x_ld = io->x_ld;
    a.w_ld = io->w_ld;
    a.resid_ld = io->resid_ld;
    a.y_ld = io->y_ld;
    a.T = T;
    a.K = c.inputs;
    a.N = c.outputs;
    a.act = !c.out_f32 ? c.act : c.act == MOE_ACT_SILU ? kSilu32 : c.act == MOE_ACT_SIGMOID ? kSigmoid32 : c.act;
    a.out_f32 = c.out_f32;
    a.scale = c.scale;
    a.status = static_cast<int *>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One row, or a few and few weights, go row by row: the tensor cores' start and end would take longer.  us by rows and in a
    // batch: 1 row of 2048, 12,288 outputs 10.0 and 11.6, of 4096, 2048 outputs 4.0 and 6.0; 2 of 2048 and 12,288 16.8 and 11.8;
    // 4 of 1024 and 4096 (2^22 products for each four rows) 4.6 and 4.6; 16 of 2048 and 256 2.9 and 4.6, and 1024 5.8 and 4.9.
    if (T == 1 || (T <= 32 && (int64_t)((T + 3) / 4) * c.inputs * c.outputs <= 1 << 22)) {
        MOE_CUDA(launch_project_rows(a, c.dtype, s));
        return MOE_OK;
    }
    // A short side is a batch's while its parts of K share the SMs in one round; with more tiles than that the other kernel,
    // whose blocks stay, is ahead.  By estimates; measured, us, in a batch and in tiles: 256 rows of 8192, 4096 outputs 25 and 32,
    // 8192 outputs 43 and 34; 64 rows of 2048, 12,288 outputs 14 and 15, 256 rows 29 and 17; 2048 rows of 2048, 96 outputs 8.0
    // and 11.3, 256 outputs 13.4 and 11.5.
    if (T <= 256 || c.outputs <= 256) {
        double us = 0;
        MOE_CUDA(project_batch_time(a, c.dtype, &us));
        if (us <= project_tiles_time(a)) {
            MOE_CUDA(launch_project_batch(a, c.dtype, s));
            return MOE_OK;
        }
    }
    MOE_CUDA(launch_project_tiles(a, c.dtype, s));
    return MOE_OK;
}

}  // extern "C"
