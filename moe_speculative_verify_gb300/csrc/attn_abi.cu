// attn_abi.cu -- host side of the attention part of the C ABI declared in
// include/moe_verify.h: argument checks, the cache's tensor maps and kernel
// launches.  As in abi.cu: no allocation, no host synchronisation.
#include <cmath>
#include <cstring>

#include "attn.h"
#include "host.h"

namespace {

using moe::aligned;
using moe::cuda_status;
using moe::device_info;

bool stride_ok(int64_t elems, int64_t es) {
    return elems > 0 && elems <= (int64_t(1) << 40) / es - 1 && (elems * es) % 16 == 0;
}

moe_status_t check_cache(const moe_kv_cache_t* c, bool rows) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_KV_BF16 && c->dtype != MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
    if (c->n_kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->n_pages < 0)
        return MOE_ERR_INVALID_ARG;
    if (c->n_kv_heads > MOE_MAX_HEADS || (c->head_dim != 64 && c->head_dim != 128) ||
        (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128))
        return MOE_ERR_UNSUPPORTED;
    if (!rows) return MOE_OK;
    const int64_t es = c->dtype == MOE_KV_E4M3 ? 1 : 2;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16) || c->n_pages == 0)
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(c->page_stride, es) || !stride_ok(c->head_stride, es) ||
        !stride_ok(c->token_stride, es))
        return MOE_ERR_INVALID_ARG;
    if (c->dtype == MOE_KV_E4M3 &&
        (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t check_seqs(const moe_seqs_t* s, bool queries) {
    if (!s || s->n_seqs < 0 || s->max_pages < 0) return MOE_ERR_INVALID_ARG;
    if (s->n_seqs > MOE_MAX_SEQS || s->max_pages > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if (s->n_seqs == 0) return MOE_OK;
    if (!s->kv_len || !aligned(s->kv_len, 4)) return MOE_ERR_INVALID_ARG;
    if (s->max_pages > 0 && (!s->block_table || !aligned(s->block_table, 4)))
        return MOE_ERR_INVALID_ARG;
    if (queries && (!s->cu_q || !aligned(s->cu_q, 4) || s->max_q < 1)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t check_attn(const moe_attn_t* a, const moe_kv_cache_t* c) {
    if (!a || a->n_q_heads <= 0 || a->n_q_heads % c->n_kv_heads || !std::isfinite(a->scale) ||
        a->window < 0)
        return MOE_ERR_INVALID_ARG;
    if (a->n_q_heads > MOE_MAX_HEADS) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t check_tokens(int32_t n) {
    if (n < 0) return MOE_ERR_INVALID_ARG;
    return n > MOE_MAX_TOKENS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// A [tokens, heads, head_dim] bf16 tensor's pointer and token stride.
bool rows_ok(const void* p, int64_t stride, int64_t row) {
    return p && aligned(p, 16) && stride >= row && stride % 8 == 0 && stride < (int64_t(1) << 32);
}

moe::KvArgs kv_args(const moe_kv_cache_t* c) {
    moe::KvArgs k{};
    k.k = static_cast<uint8_t*>(c->k);
    k.v = static_cast<uint8_t*>(c->v);
    k.k_scale = c->k_scale;
    k.v_scale = c->v_scale;
    k.page_stride = c->page_stride;
    k.head_stride = c->head_stride;
    k.token_stride = c->token_stride;
    k.e4m3 = c->dtype == MOE_KV_E4M3;
    k.n_pages = c->n_pages;
    k.page = c->page_size;
    while ((1 << k.page_log2) < k.page) ++k.page_log2;
    k.heads = c->n_kv_heads;
    k.dim = c->head_dim;
    return k;
}

moe::SeqArgs seq_args(const moe_seqs_t* s, int32_t tokens) {
    return moe::SeqArgs{s->cu_q, s->kv_len, s->block_table, s->n_seqs, s->max_pages, tokens};
}

struct KvMapKey {
    const void* k;
    const void* v;
    int64_t ps, hs, ts;
    int32_t dtype, n_pages, page, heads, dim, box;
};

// K and V as 4-D tensors (d, token, head, page), boxes of `box` tokens and 128
// bytes (64 for e4m3 heads of 64 elements), swizzled at that width.
bool make_kv_maps(const moe_kv_cache_t* c, int box, moe::KvMaps* m) {
    KvMapKey key;
    std::memset(&key, 0, sizeof(key));
    key.k = c->k;
    key.v = c->v;
    key.ps = c->page_stride;
    key.hs = c->head_stride;
    key.ts = c->token_stride;
    key.dtype = c->dtype;
    key.n_pages = c->n_pages;
    key.page = c->page_size;
    key.heads = c->n_kv_heads;
    key.dim = c->head_dim;
    key.box = box;
    thread_local moe::MapCache<KvMapKey, moe::KvMaps> cache;
    if (const moe::KvMaps* hit = cache.find(key)) {
        *m = *hit;
        return true;
    }
    auto fn = moe::encode_fn();
    if (!fn) return false;
    const bool e4m3 = c->dtype == MOE_KV_E4M3;
    const cuuint64_t es = e4m3 ? 1 : 2;
    const cuuint32_t width = e4m3 ? cuuint32_t(c->head_dim) : 64;
    const cuuint64_t dims[4] = {cuuint64_t(c->head_dim), cuuint64_t(c->page_size),
                                cuuint64_t(c->n_kv_heads), cuuint64_t(c->n_pages)};
    const cuuint64_t strides[3] = {c->token_stride * es, c->head_stride * es, c->page_stride * es};
    const cuuint32_t bx[4] = {width, cuuint32_t(box < c->page_size ? box : c->page_size), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle sw = width * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    void* base[2] = {c->k, c->v};
    CUtensorMap* map[2] = {&m->k, &m->v};
    for (int i = 0; i < 2; ++i)
        if (fn(map[i], e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
               base[i], dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    cache.put(key, *m);
    return true;
}

struct QMapKey {
    const void* q;
    int64_t stride;
    int32_t dim, heads, tokens, box_heads, box_tokens;
};

// q as a 3-D tensor (d, head, token): boxes of 64 elements x box_heads x
// box_tokens, 128-byte swizzled; tokens and heads past the end read as zeros.
bool make_q_map(const void* q, int64_t stride, int dim, int heads, int tokens, int box_heads,
                int box_tokens, CUtensorMap* m) {
    QMapKey key;
    std::memset(&key, 0, sizeof(key));
    key.q = q;
    key.stride = stride;
    key.dim = dim;
    key.heads = heads;
    key.tokens = tokens;
    key.box_heads = box_heads;
    key.box_tokens = box_tokens;
    thread_local moe::MapCache<QMapKey, CUtensorMap> cache;
    if (const CUtensorMap* hit = cache.find(key)) {
        *m = *hit;
        return true;
    }
    auto fn = moe::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    cache.put(key, *m);
    return true;
}

moe::AttnArgs attn_args(const moe_attn_t* at, const moe_kv_cache_t* c, const moe_seqs_t* s,
                        const void* q, int64_t q_stride, const uint64_t* draft, int32_t tokens,
                        void* ws) {
    moe::AttnArgs a{};
    a.kv = kv_args(c);
    a.sq = seq_args(s, tokens);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.draft = draft;
    a.q_heads = at->n_q_heads;
    a.group = at->n_q_heads / c->n_kv_heads;
    a.group_magic = a.group > 1 ? static_cast<uint32_t>(((uint64_t(1) << 32) + a.group - 1) / a.group) : 0u;
    a.scale = at->scale;
    a.causal = at->causal != 0;
    a.window = at->window < moe::kMaxWindow ? at->window : moe::kMaxWindow;
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.err = reinterpret_cast<int32_t*>(base);
    a.notes = reinterpret_cast<moe::SplitNote*>(base + moe::kAttnNotes);
    a.partials = reinterpret_cast<float*>(base + moe::kAttnPartials);
    a.timeout_ns = uint64_t(at->wait_timeout_us ? at->wait_timeout_us : 2000000u) * 1000ull;
    return a;
}

moe_status_t check_ws(const void* ws, size_t bytes, size_t need) {
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    return bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_rope_freqs(int32_t rot_dim, double base, int32_t kind, double factor,
                            int32_t original_len, double beta_fast, double beta_slow,
                            float* freqs_host, float* magnitude_host) {
    if (rot_dim < 0 || rot_dim % 16 || !freqs_host || !magnitude_host || !(base > 1.0) ||
        !std::isfinite(base))
        return MOE_ERR_INVALID_ARG;
    if (rot_dim > 128) return MOE_ERR_UNSUPPORTED;
    if (kind != MOE_ROPE_PLAIN && kind != MOE_ROPE_LINEAR && kind != MOE_ROPE_RAMP)
        return MOE_ERR_INVALID_ARG;
    if (kind != MOE_ROPE_PLAIN && !(factor > 0.0 && std::isfinite(factor))) return MOE_ERR_INVALID_ARG;
    if (kind == MOE_ROPE_RAMP &&
        !(original_len > 0 && beta_slow > 0.0 && beta_fast >= beta_slow && std::isfinite(beta_fast)))
        return MOE_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    double lo = 0.0, hi = 0.0;
    *magnitude_host = 1.0f;
    if (kind == MOE_ROPE_RAMP) {
        // pair index at which a pair turns `turns` times within original_len
        auto index = [&](double turns) {
            return rot_dim * std::log(original_len / (turns * two_pi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(index(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(index(beta_slow)), rot_dim - 1.0);
        if (factor > 1.0) *magnitude_host = static_cast<float>(0.1 * std::log(factor) + 1.0);
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (kind == MOE_ROPE_LINEAR) f /= factor;
        if (kind == MOE_ROPE_RAMP) {
            const double r = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
            f = f * (1.0 - r) + f / factor * r;
        }
        f /= two_pi;
        const float h = static_cast<float>(f);
        freqs_host[2 * i] = h;
        freqs_host[2 * i + 1] = static_cast<float>(f - static_cast<double>(h));
    }
    return MOE_OK;
}

moe_status_t moe_rope_append(const moe_rope_t* rope, const moe_kv_cache_t* cache,
                             const moe_seqs_t* seqs, const void* q, int64_t q_stride,
                             const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, int32_t n_tokens, int32_t n_q_heads,
                             void* q_out, int64_t q_out_stride, moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_seqs(seqs, true)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (!rope || rope->rot_dim < 0 || rope->rot_dim % 16 || rope->rot_dim > cache->head_dim ||
        !std::isfinite(rope->magnitude) || n_q_heads <= 0)
        return MOE_ERR_INVALID_ARG;
    if (n_q_heads > MOE_MAX_HEADS) return MOE_ERR_UNSUPPORTED;
    if (n_tokens == 0) return MOE_OK;
    const int64_t d = cache->head_dim;
    if (!rows_ok(q, q_stride, n_q_heads * d) || !rows_ok(q_out, q_out_stride, n_q_heads * d) ||
        !rows_ok(k, k_stride, cache->n_kv_heads * d) || !rows_ok(v, v_stride, cache->n_kv_heads * d))
        return MOE_ERR_INVALID_ARG;
    if (!positions || !aligned(positions, 4) ||
        (rope->rot_dim > 0 && (!rope->freqs || !aligned(rope->freqs, 4))) || !aligned(rope->err, 4))
        return MOE_ERR_INVALID_ARG;
    moe::RopeArgs a{};
    a.kv = kv_args(cache);
    a.sq = seq_args(seqs, n_tokens);
    a.freqs = rope->freqs;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved != 0;
    a.magnitude = rope->magnitude;
    a.q = static_cast<const uint16_t*>(q);
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = q_out_stride;
    a.pos = positions;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.q_heads = n_q_heads;
    a.err = rope->err;
    return cuda_status(moe::launch_rope(a, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_attn_workspace_bytes(const moe_attn_t* attn, const moe_kv_cache_t* cache) {
    if (check_cache(cache, false) != MOE_OK || check_attn(attn, cache) != MOE_OK) return 0;
    return static_cast<size_t>(moe::attn_workspace_bytes(cache->head_dim));
}

moe_status_t moe_paged_attention(const moe_attn_t* attn, const moe_kv_cache_t* cache,
                                 const moe_seqs_t* seqs, const void* q, int64_t q_stride,
                                 const uint64_t* draft_mask, int32_t n_tokens, void* out,
                                 float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_attn(attn, cache)) != MOE_OK) return st;
    if ((st = check_seqs(seqs, true)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (n_tokens == 0) return MOE_OK;
    if (seqs->n_seqs == 0) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(q, q_stride, int64_t(attn->n_q_heads) * cache->head_dim) || !out || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(draft_mask, 8))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe_attn_workspace_bytes(attn, cache))) != MOE_OK) return st;
    moe::KvMaps maps;
    const int64_t rows = int64_t(seqs->max_q) * (attn->n_q_heads / cache->n_kv_heads);
    const bool few = rows <= moe::kAttnFewRows;
    if (!make_kv_maps(cache, few ? moe::kAttnTile : moe::kAttnBigTile, &maps)) return MOE_ERR_CUDA;
    moe::AttnArgs a = attn_args(attn, cache, seqs, q, q_stride, draft_mask, n_tokens, ws);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return cuda_status(few ? moe::launch_attn_rows(a, maps, device_info().sms, s)
                           : moe::launch_attn_tile(a, maps, device_info().sms, s));
}

moe_status_t moe_key_weights(const moe_attn_t* attn, const moe_kv_cache_t* cache,
                             const moe_seqs_t* seqs, const void* q, int64_t q_stride,
                             const uint64_t* draft_mask, int32_t n_tokens, const float* lse,
                             float decay, const float* scores, float* scores_out,
                             int64_t score_stride, void* ws, size_t ws_bytes,
                             moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_attn(attn, cache)) != MOE_OK) return st;
    if ((st = check_seqs(seqs, true)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (seqs->n_seqs == 0) return n_tokens == 0 ? MOE_OK : MOE_ERR_INVALID_ARG;
    if (n_tokens == 0) {          // no rows: the scores decay; the row arguments are not read
        q = cache->k;
        q_stride = int64_t(attn->n_q_heads) * cache->head_dim;
        lse = static_cast<const float*>(ws);
        draft_mask = nullptr;
    }
    if (!rows_ok(q, q_stride, int64_t(attn->n_q_heads) * cache->head_dim) || !lse || !aligned(lse, 4) ||
        !aligned(draft_mask, 8) || !scores || !scores_out || !aligned(scores, 4) ||
        !aligned(scores_out, 4) || score_stride < 1 || !std::isfinite(decay))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe_attn_workspace_bytes(attn, cache))) != MOE_OK) return st;
    moe::KeywArgs a{};
    a.a = attn_args(attn, cache, seqs, q, q_stride, draft_mask, n_tokens, ws);
    a.a.lse = const_cast<float*>(lse);
    a.decay = decay;
    a.scores = scores;
    a.scores_out = scores_out;
    a.score_stride = score_stride;
    a.tile_heads = a.a.group < 128 ? a.a.group : 128;
    a.tile_tokens = 128 / a.tile_heads < seqs->max_q ? 128 / a.tile_heads : seqs->max_q;
    a.tile_magic = a.tile_tokens > 1 ? static_cast<uint32_t>(((uint64_t(1) << 32) + a.tile_tokens - 1) / a.tile_tokens) : 0u;
    moe::KeywMaps maps;
    moe::KvMaps kv;
    if (!make_kv_maps(cache, moe::kAttnBigTile, &kv) ||
        !make_q_map(q, q_stride, cache->head_dim, attn->n_q_heads, n_tokens > 0 ? n_tokens : 1, a.tile_heads,
                    a.tile_tokens, &maps.q))
        return MOE_ERR_CUDA;
    maps.k = kv.k;
    return cuda_status(moe::launch_keyw(a, maps, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_cache_evict(const moe_kv_cache_t* cache, const moe_seqs_t* seqs,
                             const float* scores, int64_t score_stride, int32_t budget,
                             int32_t n_recent, const int32_t* to_table, int32_t to_pages,
                             int32_t* kept, float* scores_out, int32_t* new_len, void* ws,
                             size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_seqs(seqs, false)) != MOE_OK) return st;
    if (budget < 1 || n_recent < 0 || n_recent > budget || score_stride < 1 || to_pages < 1 ||
        int64_t(to_pages) * cache->page_size < budget)
        return MOE_ERR_INVALID_ARG;
    if (seqs->n_seqs == 0) return MOE_OK;
    if (!scores || !scores_out || scores == scores_out || !to_table || !kept || !new_len ||
        !aligned(scores, 4) || !aligned(scores_out, 4) || !aligned(to_table, 4) ||
        !aligned(kept, 4) || !aligned(new_len, 4) || new_len == seqs->kv_len)
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe::kAttnNotes)) != MOE_OK) return st;
    moe::EvictArgs a{};
    a.kv = kv_args(cache);
    a.sq = seq_args(seqs, 0);
    a.scores = scores;
    a.score_stride = score_stride;
    a.budget = budget;
    a.recent = n_recent;
    a.to_table = to_table;
    a.to_pages = to_pages;
    a.kept = kept;
    a.scores_out = scores_out;
    a.new_len = new_len;
    a.err = static_cast<int32_t*>(ws);
    const int64_t places = int64_t(seqs->max_pages) * cache->page_size;
    const int64_t longest = places < score_stride ? places : score_stride;
    return cuda_status(moe::launch_evict(a, static_cast<int>(longest < (1 << 30) ? longest : 1 << 30),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
