// C ABI of the token mixers: argument checks and dispatch.  Declarations and
// conventions: include/lmoe.h.

#include <cmath>
#include <cstring>

#include "lmoe_mixers.cuh"

using namespace lmoe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA; }

int check_attn(const lmoe_attn_cfg* c) {
    if (c == nullptr || c->n_heads <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0)
        return LMOE_ERR_ARG;
    if (c->n_heads % c->n_kv_heads || c->n_heads > 1024) return LMOE_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return LMOE_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return LMOE_ERR_UNSUPPORTED;
    if (c->kv_fmt != LMOE_KV_INT8 && c->kv_fmt != LMOE_KV_E4M3) return LMOE_ERR_UNSUPPORTED;
    return LMOE_OK;
}

size_t attn_ws(const lmoe_attn_cfg& c) { return kAttnCtrlBytes + attend_ws_bytes(c.head_dim); }

// Checks what every call on a cache shares and fills the parameters; *empty:
// a valid call without anything to do.
int kv_params(const lmoe_attn_cfg* cfg, const lmoe_kv_cache* cache, const lmoe_kv_batch* b, void* ws, size_t ws_bytes,
              KvParams* p, bool* empty) {
    int s = check_attn(cfg);
    if (s != LMOE_OK) return s;
    if (!cache || !b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_new < 0 || b->pages_per_seq < 0 || cache->n_pages < 0)
        return LMOE_ERR_ARG;
    *empty = b->n_seqs == 0 || b->n_tokens == 0 || b->max_new == 0;
    if (*empty) return LMOE_OK;
    if (!cache->k || !cache->v || !cache->k_scale || !cache->v_scale || !aligned(cache->k, 16) ||
        !aligned(cache->v, 16) || !aligned(cache->k_scale, 16) || !aligned(cache->v_scale, 16) || cache->n_pages < 1)
        return LMOE_ERR_ARG;
    if (!b->q_start || !b->kv_len || !b->page_table || !aligned(b->q_start, 4) || !aligned(b->kv_len, 4) ||
        !aligned(b->page_table, 4) || b->pages_per_seq < 1)
        return LMOE_ERR_ARG;
    if (!ws || !aligned(ws, 256)) return LMOE_ERR_ARG;
    if (ws_bytes < attn_ws(*cfg)) return LMOE_ERR_WORKSPACE;
    p->Hq = cfg->n_heads;
    p->Hk = cfg->n_kv_heads;
    p->G = cfg->n_heads / cfg->n_kv_heads;
    p->D = cfg->head_dim;
    p->fmt = cfg->kv_fmt;
    p->page_log2 = 0;
    while ((1 << p->page_log2) < cfg->page_size) ++p->page_log2;
    p->k = static_cast<uint8_t*>(cache->k);
    p->v = static_cast<uint8_t*>(cache->v);
    p->ks = cache->k_scale;
    p->vs = cache->v_scale;
    p->n_pages = cache->n_pages;
    p->q_start = b->q_start;
    p->kv_len = b->kv_len;
    p->table = b->page_table;
    p->n_seqs = b->n_seqs;
    p->table_stride = b->pages_per_seq;
    p->n_tokens = b->n_tokens;
    p->max_new = b->max_new < b->n_tokens ? b->max_new : b->n_tokens;
    // query rows of a sequence and key head are counted in an int
    if ((long long)p->max_new * p->G > 0x7fffffff - 1024) return LMOE_ERR_UNSUPPORTED;
    p->ctrl = static_cast<Ctrl*>(ws);
    return LMOE_OK;
}

// bf16 rows: pointer, alignment, stride.
bool rows_ok(const void* x, size_t stride, size_t width) {
    return x && aligned(x, 16) && stride % 8 == 0 && stride >= width;
}

int check_delta(const lmoe_delta_cfg* c) {
    if (c == nullptr || c->n_heads <= 0 || c->n_qk_heads <= 0 || c->head_k <= 0 || c->head_v <= 0) return LMOE_ERR_ARG;
    if (c->n_heads % c->n_qk_heads || c->n_heads > 1024) return LMOE_ERR_UNSUPPORTED;
    if ((c->head_k != 64 && c->head_k != 128) || (c->head_v != 64 && c->head_v != 128)) return LMOE_ERR_UNSUPPORTED;
    return LMOE_OK;
}

size_t delta_ws(const lmoe_delta_cfg& c, int n_tokens, int n_seqs, int max_new) {
    return kAttnCtrlBytes + delta_chunk_ws_bytes(c.n_heads, n_tokens, n_seqs, max_new);
}

}  // namespace

extern "C" {

int lmoe_attn_cfg_check(const lmoe_attn_cfg* cfg) { return check_attn(cfg); }

size_t lmoe_attn_workspace_bytes(const lmoe_attn_cfg* cfg) { return check_attn(cfg) == LMOE_OK ? attn_ws(*cfg) : 0; }

int lmoe_kv_append(const lmoe_attn_cfg* cfg, const lmoe_kv_cache* cache, const lmoe_kv_batch* batch, const void* k,
                   const void* v, size_t k_stride, size_t v_stride, void* ws, size_t ws_bytes, void* stream) {
    KvParams p;
    bool empty = false;
    const int s = kv_params(cfg, cache, batch, ws, ws_bytes, &p, &empty);
    if (s != LMOE_OK || empty) return s;
    const size_t width = (size_t)p.Hk * p.D;
    if (!rows_ok(k, k_stride, width) || !rows_ok(v, v_stride, width)) return LMOE_ERR_ARG;
    return cuda_status(run_kv_append(p, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), k_stride,
                                     v_stride, static_cast<cudaStream_t>(stream)));
}

int lmoe_kv_read(const lmoe_attn_cfg* cfg, const lmoe_kv_cache* cache, const lmoe_kv_batch* batch, void* k, void* v,
                 size_t k_stride, size_t v_stride, void* ws, size_t ws_bytes, void* stream) {
    KvParams p;
    bool empty = false;
    const int s = kv_params(cfg, cache, batch, ws, ws_bytes, &p, &empty);
    if (s != LMOE_OK || empty) return s;
    const size_t width = (size_t)p.Hk * p.D;
    if (!rows_ok(k, k_stride, width) || !rows_ok(v, v_stride, width)) return LMOE_ERR_ARG;
    return cuda_status(run_kv_read(p, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), k_stride, v_stride,
                                   static_cast<cudaStream_t>(stream)));
}

int lmoe_attend(const lmoe_attn_cfg* cfg, const lmoe_kv_cache* cache, const lmoe_kv_batch* batch, const void* q,
                size_t q_stride, float softmax_scale, int causal, int window, void* out, float* lse, void* ws,
                size_t ws_bytes, void* stream) {
    AttendParams p;
    bool empty = false;
    const int s = kv_params(cfg, cache, batch, ws, ws_bytes, &p, &empty);
    if (s != LMOE_OK) return s;
    const float scale_log2 = softmax_scale * 1.4426950408889634f;
    if (window < 0 || (window > 0 && !causal) || !std::isfinite(scale_log2)) return LMOE_ERR_ARG;
    if (empty) return LMOE_OK;
    if (!rows_ok(q, q_stride, (size_t)p.Hq * p.D) || !out || !aligned(out, 16) || (lse && !aligned(lse, 4)))
        return LMOE_ERR_ARG;
    p.q = static_cast<const uint16_t*>(q);
    p.q_stride = q_stride;
    p.scale_log2 = scale_log2;
    p.causal = causal != 0;
    // a window as wide as the cache hides nothing (and position - window stays in an int)
    p.window = window < ((long long)p.table_stride << p.page_log2) ? window : 0;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    return cuda_status(run_attend(p, static_cast<char*>(ws) + kAttnCtrlBytes, static_cast<cudaStream_t>(stream)));
}

int lmoe_delta_cfg_check(const lmoe_delta_cfg* cfg) { return check_delta(cfg); }

size_t lmoe_delta_workspace_bytes(const lmoe_delta_cfg* cfg, int n_tokens, int n_seqs, int max_new) {
    if (check_delta(cfg) != LMOE_OK || n_tokens < 0 || n_seqs < 0 || max_new < 0) return 0;
    return delta_ws(*cfg, n_tokens, n_seqs, max_new);
}

int lmoe_delta_rule(const lmoe_delta_cfg* cfg, const lmoe_delta_batch* b, const void* q, const void* k, const void* v,
                    size_t q_stride, size_t k_stride, size_t v_stride, const float* log_decay, const float* beta,
                    float scale, float* states, void* out, void* ws, size_t ws_bytes, void* stream) {
    const int s = check_delta(cfg);
    if (s != LMOE_OK) return s;
    if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_new < 0 || b->n_states < 0 || !std::isfinite(scale))
        return LMOE_ERR_ARG;
    if (b->n_seqs == 0) return LMOE_OK;
    if (!b->q_start || !b->src || !b->dst || !aligned(b->q_start, 4) || !aligned(b->src, 4) || !aligned(b->dst, 4))
        return LMOE_ERR_ARG;
    if (b->n_states > 0 && (!states || !aligned(states, 16))) return LMOE_ERR_ARG;
    if (b->n_tokens > 0) {
        const size_t wk = (size_t)cfg->n_qk_heads * cfg->head_k, wv = (size_t)cfg->n_heads * cfg->head_v;
        if (!rows_ok(q, q_stride, wk) || !rows_ok(k, k_stride, wk) || !rows_ok(v, v_stride, wv)) return LMOE_ERR_ARG;
        if (!log_decay || !beta || !out || !aligned(log_decay, 4) || !aligned(beta, 4) || !aligned(out, 16))
            return LMOE_ERR_ARG;
    }
    if ((long long)b->n_seqs * cfg->n_heads * (cfg->head_v / 32) > 0x7fffffff) return LMOE_ERR_UNSUPPORTED;   // blocks of a launch
    if (!ws || !aligned(ws, 256)) return LMOE_ERR_ARG;
    if (ws_bytes < delta_ws(*cfg, b->n_tokens, b->n_seqs, b->max_new)) return LMOE_ERR_WORKSPACE;
    DeltaParams p;
    std::memset(&p, 0, sizeof(p));
    p.H = cfg->n_heads;
    p.Hq = cfg->n_qk_heads;
    p.group = cfg->n_heads / cfg->n_qk_heads;
    p.DK = cfg->head_k;
    p.DV = cfg->head_v;
    p.l2norm = cfg->l2norm != 0;
    p.q_start = b->q_start;
    p.src = b->src;
    p.dst = b->dst;
    p.n_seqs = b->n_seqs;
    p.n_states = b->n_states;
    p.n_tokens = b->n_tokens;
    p.max_new = b->max_new < b->n_tokens ? b->max_new : b->n_tokens;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.qs = q_stride;
    p.ks = k_stride;
    p.vs = v_stride;
    p.log_decay = log_decay;
    p.beta = beta;
    p.scale = scale;
    p.states = states;
    p.out = static_cast<uint16_t*>(out);
    p.ctrl = static_cast<Ctrl*>(ws);
    p.chunk_ws = static_cast<char*>(ws) + kAttnCtrlBytes;
    return cuda_status(run_delta(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
