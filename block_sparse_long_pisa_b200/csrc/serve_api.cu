// Host side of the calls around the attention: norm and rotation of queries and keys, the K/V cache,
// and the attention of drafted tokens over it. Argument checks (which never touch the GPU), layouts
// and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "pisa.h"
#include "pisa_internal.h"

namespace pisa {

static bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// a required pointer of the given alignment
static bool good(const void* p, uintptr_t n) { return p != nullptr && aligned(p, n); }
static bool good_or_null(const void* p, uintptr_t n) { return p == nullptr || aligned(p, n); }

static bool strides_ok(const int64_t* s) {
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0 || s[i] % 8 != 0) return false;
    return true;
}

// Whether rows of D elements at these strides are disjoint: of the dims larger than one, ordered by
// stride, each stride clears everything inside it.
static bool rows_disjoint(const int64_t* stride, int64_t n0, int64_t n1, int64_t n2, int64_t D) {
    const int64_t n[3] = {n0, n1, n2};
    bool done[3] = {n0 <= 1, n1 <= 1, n2 <= 1};
    int64_t span = D;  // elements from the first to past the last, of the dims taken so far
    for (int k = 0; k < 3; ++k) {
        int at = -1;
        for (int i = 0; i < 3; ++i)
            if (!done[i] && (at < 0 || stride[i] < stride[at])) at = i;
        if (at < 0) break;
        if (stride[at] < span) return false;
        if (stride[at] > (int64_t(1) << 62) / n[at]) return false;
        span += stride[at] * (n[at] - 1);
        done[at] = true;
    }
    return true;
}

// The shape, without its output strides.
static pisa_status check_norm_rope(const pisa_norm_rope_shape* s) {
    if (s == nullptr) return PISA_ERR_INVALID_ARG;
    if (s->batch < 1 || s->tokens < 1 || s->heads_q < 1 || s->heads_kv < 1 || s->head_dim < 1 || s->rotary_dim < 0 ||
        s->rotary_dim > s->head_dim || (s->interleaved != 0 && s->interleaved != 1) || !(s->eps >= 0.f) ||
        isinf(s->eps) || !strides_ok(s->xq_stride) || !strides_ok(s->xk_stride))
        return PISA_ERR_INVALID_ARG;
    if (s->head_dim != 64 && s->head_dim != 128) return PISA_ERR_UNSUPPORTED;
    if (s->rotary_dim % 16 != 0) return PISA_ERR_UNSUPPORTED;
    if (s->heads_q > 32768 || s->heads_kv > 32768) return PISA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s->batch) * s->tokens >= (int64_t(1) << 31)) return PISA_ERR_UNSUPPORTED;
    return PISA_OK;
}

static NormRopeParams norm_rope_params(const pisa_norm_rope_shape* s, const void* Xq, const void* Xk, const float* wq,
                                       const float* wk, const float* inv_freq, const int32_t* pos) {
    NormRopeParams p{};
    p.Xq = static_cast<const __nv_bfloat16*>(Xq);
    p.Xk = static_cast<const __nv_bfloat16*>(Xk);
    p.wq = wq;
    p.wk = wk;
    p.inv_freq = inv_freq;
    p.pos = pos;
    for (int i = 0; i < 3; ++i) {
        p.xq[i] = s->xq_stride[i];
        p.xk[i] = s->xk_stride[i];
        p.dxq[i] = s->dxq_stride[i];
        p.dxk[i] = s->dxk_stride[i];
    }
    p.ntokens = static_cast<int64_t>(s->batch) * s->tokens;
    p.T = s->tokens;
    p.Hq = s->heads_q;
    p.Hkv = s->heads_kv;
    p.R = s->rotary_dim;
    p.eps = s->eps;
    return p;
}

static size_t norm_rope_ws(const pisa_norm_rope_shape* s) {
    return static_cast<size_t>(kNormRopeBlocks) * s->head_dim * sizeof(float);
}

static pisa_status check_cache(const pisa_cache_shape* s) {
    if (s == nullptr || s->batch < 1 || s->heads_kv < 1 || s->capacity < 1 || s->head_dim < 1 ||
        (s->format != PISA_CACHE_BF16 && s->format != PISA_CACHE_E4M3))
        return PISA_ERR_INVALID_ARG;
    if (s->head_dim != 64 && s->head_dim != 128) return PISA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s->batch) * s->heads_kv >= (int64_t(1) << 31) / s->capacity) return PISA_ERR_UNSUPPORTED;
    return PISA_OK;
}

// The cache's buffers for its format.
static bool cache_buffers_ok(int32_t format, const void* Kc, const void* Vc, const uint8_t* ke, const uint8_t* ve) {
    if (!good(Kc, 16) || !good(Vc, 16)) return false;
    return format == PISA_CACHE_E4M3 ? good(ke, 16) && good(ve, 16) : ke == nullptr && ve == nullptr;
}

struct TreePlan {
    int32_t g, gh, hsel, rows, rm, mt, runs;
    size_t total;
};

static pisa_status tree_plan(const pisa_tree_shape* s, TreePlan* t) {
    if (s == nullptr) return PISA_ERR_INVALID_ARG;
    if (s->batch < 1 || s->heads_q < 1 || s->heads_kv < 1 || s->drafts < 1 || s->capacity < 1 || s->head_dim < 1 ||
        (s->format != PISA_CACHE_BF16 && s->format != PISA_CACHE_E4M3) || s->block < 1 || s->topk < 0 ||
        s->seq_kv < 0 || (s->select_per_qhead != 0 && s->select_per_qhead != 1) || !(s->scale == s->scale) ||
        isinf(s->scale) || s->heads_q % s->heads_kv != 0 || s->capacity % s->block != 0)
        return PISA_ERR_INVALID_ARG;
    if (s->topk == 0 && (s->seq_kv != 0 || s->select_per_qhead != 0)) return PISA_ERR_INVALID_ARG;
    if (s->topk > 0 && (s->seq_kv < s->block || s->seq_kv % s->block != 0 || s->seq_kv > s->capacity))
        return PISA_ERR_INVALID_ARG;
    if (s->head_dim != 64 && s->head_dim != 128) return PISA_ERR_UNSUPPORTED;
    if (s->block != 64 && s->block != 128) return PISA_ERR_UNSUPPORTED;
    if (s->drafts > 64 || s->topk > PISA_MAX_CANDIDATES) return PISA_ERR_UNSUPPORTED;
    // row coordinates of the copies, and every row index of the outputs, stay below 2^31
    const int64_t planes = static_cast<int64_t>(s->batch) * s->heads_kv;
    if (planes >= (int64_t(1) << 31) / s->capacity || planes >= (int64_t(1) << 31) / s->drafts)
        return PISA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s->batch) * s->heads_q >= (int64_t(1) << 31) / s->drafts) return PISA_ERR_UNSUPPORTED;
    t->g = s->heads_q / s->heads_kv;
    t->gh = s->select_per_qhead ? 1 : t->g;
    t->hsel = s->select_per_qhead ? s->heads_q : s->heads_kv;
    if (static_cast<int64_t>(t->gh) * s->drafts > (1 << 20)) return PISA_ERR_UNSUPPORTED;
    t->rows = t->gh * s->drafts;
    t->rm = tree_row_tile(t->rows, s->drafts, s->format == PISA_CACHE_E4M3);
    t->mt = (t->rows + t->rm - 1) / t->rm;
    if (static_cast<int64_t>(s->batch) * t->hsel * t->mt >= (int64_t(1) << 31)) return PISA_ERR_UNSUPPORTED;
    t->runs = kTreeRuns * tree_ctas_per_sm(t->rm, s->format == PISA_CACHE_E4M3);
    t->total = kStatusBytes + size_t(2) * t->runs * t->rm * (s->head_dim + 2) * sizeof(float);
    return PISA_OK;
}

}  // namespace pisa

using namespace pisa;

extern "C" {

pisa_status pisa_qk_norm_rope(const pisa_norm_rope_shape* shape, const void* Xq, const void* Xk, const float* wq,
                              const float* wk, const float* inv_freq, const int32_t* pos, void* Q, void* K,
                              pisa_stream_t stream) {
    g_launches = 0;
    const pisa_status s = check_norm_rope(shape);
    if (s != PISA_OK) return s;
    if (!good(Xq, 16) || !good(Xk, 16) || !good(Q, 16) || !good(K, 16) || !good_or_null(wq, 4) ||
        !good_or_null(wk, 4) || !good_or_null(inv_freq, 4) || !good_or_null(pos, 4))
        return PISA_ERR_INVALID_ARG;
    if (shape->rotary_dim > 0 && (inv_freq == nullptr || pos == nullptr)) return PISA_ERR_INVALID_ARG;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    NormRopeParams p = norm_rope_params(shape, Xq, Xk, wq, wk, inv_freq, pos);
    p.Q = static_cast<__nv_bfloat16*>(Q);
    p.K = static_cast<__nv_bfloat16*>(K);
    if (!launch_norm_rope(p, shape->head_dim, shape->interleaved != 0, reinterpret_cast<cudaStream_t>(stream)))
        return PISA_ERR_CUDA;
    ++g_launches;
    return PISA_OK;
}

pisa_status pisa_norm_rope_workspace_size(const pisa_norm_rope_shape* shape, size_t* bytes) {
    if (bytes == nullptr) return PISA_ERR_INVALID_ARG;
    const pisa_status s = check_norm_rope(shape);
    if (s == PISA_OK) *bytes = norm_rope_ws(shape);
    return s;
}

pisa_status pisa_qk_norm_rope_backward(const pisa_norm_rope_shape* shape, const void* Xq, const void* Xk,
                                       const float* wq, const float* wk, const float* inv_freq, const int32_t* pos,
                                       const void* dQ, const void* dK, void* dXq, void* dXk, float* dwq, float* dwk,
                                       void* ws, size_t ws_bytes, pisa_stream_t stream) {
    g_launches = 0;
    const pisa_status s = check_norm_rope(shape);
    if (s != PISA_OK) return s;
    if (!strides_ok(shape->dxq_stride) || !strides_ok(shape->dxk_stride) ||
        !rows_disjoint(shape->dxq_stride, shape->batch, shape->tokens, shape->heads_q, shape->head_dim) ||
        !rows_disjoint(shape->dxk_stride, shape->batch, shape->tokens, shape->heads_kv, shape->head_dim))
        return PISA_ERR_INVALID_ARG;
    if (!good(Xq, 16) || !good(Xk, 16) || !good(dQ, 16) || !good(dK, 16) || !good(dXq, 16) || !good(dXk, 16) ||
        !good_or_null(wq, 4) || !good_or_null(wk, 4) || !good_or_null(inv_freq, 4) || !good_or_null(pos, 4) ||
        !good_or_null(dwq, 4) || !good_or_null(dwk, 4) || !good(ws, 16))
        return PISA_ERR_INVALID_ARG;
    if (shape->rotary_dim > 0 && (inv_freq == nullptr || pos == nullptr)) return PISA_ERR_INVALID_ARG;
    if (ws_bytes < norm_rope_ws(shape)) return PISA_ERR_WORKSPACE;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    NormRopeParams p = norm_rope_params(shape, Xq, Xk, wq, wk, inv_freq, pos);
    p.dQ = static_cast<const __nv_bfloat16*>(dQ);
    p.dK = static_cast<const __nv_bfloat16*>(dK);
    p.dXq = static_cast<__nv_bfloat16*>(dXq);
    p.dXk = static_cast<__nv_bfloat16*>(dXk);
    p.part = static_cast<float*>(ws);
    return launch_norm_rope_backward(p, shape->head_dim, shape->interleaved != 0, dwq, dwk,
                                     reinterpret_cast<cudaStream_t>(stream), &g_launches)
               ? PISA_OK
               : PISA_ERR_CUDA;
}

pisa_status pisa_cache_write(const pisa_cache_shape* shape, int32_t tokens, const void* K, const void* V,
                             const int64_t* k_stride, const int64_t* v_stride, const int32_t* start,
                             const int32_t* count, void* Kc, void* Vc, uint8_t* k_exp, uint8_t* v_exp, void* ws,
                             pisa_stream_t stream) {
    g_launches = 0;
    const pisa_status s = check_cache(shape);
    if (s != PISA_OK) return s;
    if (tokens < 1 || tokens > shape->capacity || k_stride == nullptr || v_stride == nullptr ||
        !strides_ok(k_stride) || !strides_ok(v_stride) || !good(K, 16) || !good(V, 16) || !good_or_null(start, 4) ||
        !good_or_null(count, 4) || !cache_buffers_ok(shape->format, Kc, Vc, k_exp, v_exp) || !good(ws, 16))
        return PISA_ERR_INVALID_ARG;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    CacheParams p{};
    p.K = static_cast<const __nv_bfloat16*>(K);
    p.V = static_cast<const __nv_bfloat16*>(V);
    p.Kc = Kc;
    p.Vc = Vc;
    p.ke = k_exp;
    p.ve = v_exp;
    p.start = start;
    p.count = count;
    p.status = static_cast<uint32_t*>(ws);
    for (int i = 0; i < 3; ++i) {
        p.ks[i] = k_stride[i];
        p.vs[i] = v_stride[i];
    }
    p.B = shape->batch;
    p.H = shape->heads_kv;
    p.cap = shape->capacity;
    p.tokens = tokens;
    if (!launch_cache_write(p, shape->head_dim, shape->format == PISA_CACHE_E4M3,
                            reinterpret_cast<cudaStream_t>(stream)))
        return PISA_ERR_CUDA;
    ++g_launches;
    return PISA_OK;
}

pisa_status pisa_cache_read(const pisa_cache_shape* shape, int32_t tokens, const void* Kc, const void* Vc,
                            const uint8_t* k_exp, const uint8_t* v_exp, const int32_t* start, const int32_t* count,
                            void* K, void* V, void* ws, pisa_stream_t stream) {
    g_launches = 0;
    const pisa_status s = check_cache(shape);
    if (s != PISA_OK) return s;
    if (tokens < 1 || tokens > shape->capacity || !good(K, 16) || !good(V, 16) || !good_or_null(start, 4) ||
        !good_or_null(count, 4) || !cache_buffers_ok(shape->format, Kc, Vc, k_exp, v_exp) || !good(ws, 16))
        return PISA_ERR_INVALID_ARG;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    CacheParams p{};
    p.Ko = static_cast<__nv_bfloat16*>(K);
    p.Vo = static_cast<__nv_bfloat16*>(V);
    p.Kc = const_cast<void*>(Kc);
    p.Vc = const_cast<void*>(Vc);
    p.ke = const_cast<uint8_t*>(k_exp);
    p.ve = const_cast<uint8_t*>(v_exp);
    p.start = start;
    p.count = count;
    p.status = static_cast<uint32_t*>(ws);
    p.B = shape->batch;
    p.H = shape->heads_kv;
    p.cap = shape->capacity;
    p.tokens = tokens;
    if (!launch_cache_read(p, shape->head_dim, shape->format == PISA_CACHE_E4M3,
                           reinterpret_cast<cudaStream_t>(stream)))
        return PISA_ERR_CUDA;
    ++g_launches;
    return PISA_OK;
}

pisa_status pisa_cache_append_pyramid(const pisa_shape* shape, const void* Kc, const uint8_t* k_exp, float* pyramid,
                                      int32_t seq_kv_old, pisa_stream_t stream) {
    g_launches = 0;
    Plan pl;
    const pisa_status s = make_plan(shape, &pl);
    if (s != PISA_OK) return s;
    if (!good(Kc, 16) || !good(k_exp, 16) || !good(pyramid, 16)) return PISA_ERR_INVALID_ARG;
    if (seq_kv_old < 0 || seq_kv_old > shape->seq_kv || seq_kv_old % pl.blk != 0) return PISA_ERR_INVALID_ARG;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    if (seq_kv_old == shape->seq_kv) return PISA_OK;
    CachePyramidParams p{};
    p.K = static_cast<const uint8_t*>(Kc);
    p.e = k_exp;
    p.pyr = pyramid;
    p.planes = pl.B * pl.Hkv;
    p.N = pl.N;
    p.D = pl.D;
    p.blk = pl.blk;
    p.factor = pl.f;
    p.L = pl.L;
    p.plane_rows = pl.total_nodes;
    p.n0 = pl.n0;
    p.b_lo = seq_kv_old / pl.blk;
    p.b_hi = pl.n0;
    for (int l = 0; l < pl.L; ++l) {
        p.lsize[l] = pl.lsize[l];
        p.loff[l] = pl.loff[l];
    }
    return launch_cache_pyramid(p, reinterpret_cast<cudaStream_t>(stream), &g_launches) ? PISA_OK : PISA_ERR_CUDA;
}

pisa_status pisa_tree_workspace_size(const pisa_tree_shape* shape, size_t* bytes) {
    if (bytes == nullptr) return PISA_ERR_INVALID_ARG;
    TreePlan t;
    const pisa_status s = tree_plan(shape, &t);
    if (s == PISA_OK) *bytes = t.total;
    return s;
}

pisa_status pisa_tree_attention(const pisa_tree_shape* shape, const void* Q, const void* K, const void* V,
                                const uint64_t* mask, const void* Kc, const void* Vc, const uint8_t* k_exp,
                                const uint8_t* v_exp, const int32_t* cache_len, const int32_t* idx, void* O,
                                float* lse, void* ws, size_t ws_bytes, pisa_stream_t stream) {
    g_launches = 0;
    TreePlan t;
    const pisa_status s = tree_plan(shape, &t);
    if (s != PISA_OK) return s;
    if (!good(Q, 16) || !good(K, 16) || !good(V, 16) || !good(mask, 8) ||
        !cache_buffers_ok(shape->format, Kc, Vc, k_exp, v_exp) || !good(cache_len, 4) || !good_or_null(idx, 4) ||
        (shape->topk > 0) != (idx != nullptr) || !good(O, 16) || !good_or_null(lse, 4) || !good(ws, 16))
        return PISA_ERR_INVALID_ARG;
    if (ws_bytes < t.total) return PISA_ERR_WORKSPACE;
    if (injected_launch_failure()) return PISA_ERR_CUDA;
    TreeParams p{};
    p.Q = static_cast<const __nv_bfloat16*>(Q);
    p.DV = static_cast<const __nv_bfloat16*>(V);
    p.mask = mask;
    p.k_exp = k_exp;
    p.v_exp = v_exp;
    p.len = cache_len;
    p.idx = idx;
    p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kStatusBytes);
    p.O = static_cast<__nv_bfloat16*>(O);
    p.lse = lse;
    p.status = static_cast<uint32_t*>(ws);
    p.B = shape->batch;
    p.Hq = shape->heads_q;
    p.Hkv = shape->heads_kv;
    p.Hsel = t.hsel;
    p.g = t.g;
    p.gh = t.gh;
    p.T = shape->drafts;
    p.cap = shape->capacity;
    p.seq = shape->seq_kv;
    p.topk = shape->topk;
    p.n0 = shape->seq_kv / shape->block;
    p.per_qhead = shape->select_per_qhead;
    p.upb = shape->block / 64;
    p.mt = t.mt;
    p.rows_per_seq = t.hsel * t.mt;
    p.rpt = (t.rows + t.mt - 1) / t.mt;
    p.runs = t.runs;
    p.min_units = kTreeMinUnits;
    p.tp = (shape->drafts + 15) / 16 * 16;
    const float scale = shape->scale > 0.f ? shape->scale : 1.0f / sqrtf(static_cast<float>(shape->head_dim));
    p.scale_log2 = scale * 1.4426950408889634f;
    return launch_attn_tree(p, shape->head_dim, shape->format == PISA_CACHE_E4M3, t.rm, K, Kc, Vc,
                            reinterpret_cast<cudaStream_t>(stream), &g_launches)
               ? PISA_OK
               : PISA_ERR_CUDA;
}

}  // extern "C"
