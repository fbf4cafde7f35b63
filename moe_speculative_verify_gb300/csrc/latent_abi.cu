// latent_abi.cu -- host side of the latent-cache part of the C ABI declared in
// include/moe_verify.h: argument checks and kernel launches.  As in abi.cu: no
// allocation, no host synchronisation.
#include <cmath>

#include "host.h"
#include "latent.h"

namespace {

using moe::aligned;
using moe::cuda_status;
using moe::device_info;

// (a tensor map's strides are below 2^40 bytes, that of eight tokens among them)
bool stride_ok(int64_t elems, int64_t es, int64_t least) {
    return elems >= least && elems <= (int64_t(1) << 37) / es - 1 && (elems * es) % 16 == 0;
}

// Strides of rows of bf16 elements that are read in 16-byte pieces.
bool row_stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0 && s < (int64_t(1) << 32); }

bool rows_ok(const void* p, int64_t stride, int64_t least) { return p && aligned(p, 16) && row_stride_ok(stride, least); }

moe_status_t check_cache(const moe_latent_cache_t* c, bool rows) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_KV_BF16 && c->dtype != MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
    if (c->latent_dim <= 0 || c->page_size <= 0 || c->n_pages < 0) return MOE_ERR_INVALID_ARG;
    if ((c->latent_dim != 256 && c->latent_dim != 512) ||
        (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128))
        return MOE_ERR_UNSUPPORTED;
    const bool e4m3 = c->dtype == MOE_KV_E4M3;
    if (e4m3 && (c->scale_log2 < MOE_LATENT_MIN_SCALE || c->scale_log2 > MOE_LATENT_MAX_SCALE)) return MOE_ERR_UNSUPPORTED;
    if (!rows) return MOE_OK;
    const int64_t es = e4m3 ? 1 : 2;
    if (!c->latent || !c->rope || !aligned(c->latent, 16) || !aligned(c->rope, 16) || c->n_pages == 0)
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(c->latent_page_stride, es, c->latent_dim) || !stride_ok(c->latent_token_stride, es, c->latent_dim) ||
        !stride_ok(c->rope_page_stride, 2, moe::kLatentRot) || !stride_ok(c->rope_token_stride, 2, moe::kLatentRot))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t check_seqs(const moe_seqs_t* s, bool queries, bool table) {
    if (!s || s->n_seqs < 0 || s->max_pages < 0) return MOE_ERR_INVALID_ARG;
    if (s->n_seqs > MOE_MAX_SEQS || s->max_pages > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    if (s->n_seqs == 0) return MOE_OK;
    if (!s->kv_len || !aligned(s->kv_len, 4)) return MOE_ERR_INVALID_ARG;
    if (table && s->max_pages > 0 && (!s->block_table || !aligned(s->block_table, 4))) return MOE_ERR_INVALID_ARG;
    if (queries && (!s->cu_q || !aligned(s->cu_q, 4) || s->max_q < 1)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t check_attn(const moe_attn_t* a) {
    if (!a || a->n_q_heads <= 0 || !std::isfinite(a->scale) || a->window < 0) return MOE_ERR_INVALID_ARG;
    return a->n_q_heads > MOE_MAX_HEADS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t check_tokens(int32_t n) {
    if (n < 0) return MOE_ERR_INVALID_ARG;
    return n > MOE_MAX_TOKENS ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t check_ws(const void* ws, size_t bytes, size_t need) {
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    return bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe::LatentArgs latent_args(const moe_latent_cache_t* c) {
    moe::LatentArgs k{};
    k.latent = static_cast<uint8_t*>(c->latent);
    k.rope = static_cast<uint16_t*>(c->rope);
    k.lat_page = c->latent_page_stride;
    k.lat_token = c->latent_token_stride;
    k.rope_page = c->rope_page_stride;
    k.rope_token = c->rope_token_stride;
    k.e4m3 = c->dtype == MOE_KV_E4M3;
    k.scale_log2 = k.e4m3 ? c->scale_log2 : 0;
    k.n_pages = c->n_pages;
    k.page = c->page_size;
    while ((1 << k.page_log2) < k.page) ++k.page_log2;
    k.dim = c->latent_dim;
    return k;
}

moe::SeqArgs seq_args(const moe_seqs_t* s, int32_t tokens) {
    return moe::SeqArgs{s->cu_q, s->kv_len, s->block_table, s->n_seqs, s->max_pages, tokens};
}

// What both attention calls share; `heads` kv heads, rows of `dim` output elements.
moe::AttnArgs attn_args(const moe_attn_t* at, const moe_seqs_t* s, const void* q, int64_t q_stride, const uint64_t* draft,
                        int32_t tokens, void* out, float* lse, void* ws, int heads, int dim) {
    moe::AttnArgs a{};
    a.kv.heads = heads;
    a.kv.dim = dim;
    a.sq = seq_args(s, tokens);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.draft = draft;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_heads = at->n_q_heads;
    a.group = at->n_q_heads / heads;
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

// The cache's tensor maps, encoded anew by every call: nothing is kept by an address.
bool make_maps(const moe_latent_cache_t* c, moe::LatentMaps* m) {
    auto fn = moe::encode_fn();
    if (!fn) return false;
    const bool e4m3 = c->dtype == MOE_KV_E4M3;
    const cuuint64_t es = e4m3 ? 1 : 2, part = 128 / es;         // 128 bytes
    const cuuint64_t dims[5] = {part, 8, c->latent_dim / part, cuuint64_t(c->page_size) / 8, cuuint64_t(c->n_pages)};
    const cuuint64_t token = c->latent_token_stride * es;
    const cuuint64_t strides[4] = {token, 128, 8 * token, c->latent_page_stride * es};
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    auto latent = [&](CUtensorMap* map, int tokens, int dim) {
        const cuuint32_t box[5] = {cuuint32_t(part), 8, cuuint32_t(dim / part),
                                   cuuint32_t(c->page_size < tokens ? c->page_size : tokens) / 8, 1};
        return fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, c->latent, dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const int keys = moe::kLatentKeys / 2;
    const cuuint64_t rdims[3] = {moe::kLatentRot, cuuint64_t(c->page_size), cuuint64_t(c->n_pages)};
    const cuuint64_t rstrides[2] = {cuuint64_t(c->rope_token_stride) * 2, cuuint64_t(c->rope_page_stride) * 2};
    const cuuint32_t rbox[3] = {moe::kLatentRot, cuuint32_t(c->page_size < keys ? c->page_size : keys), 1};
    return latent(&m->keys, keys, c->latent_dim) && latent(&m->values, moe::kLatentKeys, c->latent_dim / 2) &&
           fn(&m->rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c->rope, rdims, rstrides, rbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_q_map(const moe::LatentAttnArgs& a, bool few, moe::LatentMaps* m) {
    const cuuint64_t row = a.c.dim + moe::kLatentRot;
    const cuuint64_t dims[3] = {64, cuuint64_t(a.a.sq.tokens) * a.a.q_heads, row / 64}, strides[2] = {row * 2, 128};
    const cuuint32_t box[3] = {64, cuuint32_t(moe::kLatentRows / (few ? 4 : 2)), cuuint32_t(row / 64)}, one[3] = {1, 1, 1};
    return moe::encode_fn()(&m->q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.a.q), dims, strides, box, one,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_maps(const moe::ExpandedArgs& a, moe::ExpandedMaps* m) {
    auto fn = moe::encode_fn();
    if (!fn) return false;
    const cuuint64_t n = a.n_keys, h = a.a.q_heads;
    const cuuint32_t one[4] = {1, 1, 1, 1}, rows = moe::kExpandedKeys / 2;
    auto map = [&](CUtensorMap* to, const uint16_t* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
        return fn(to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<uint16_t*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t qd[4] = {64, cuuint64_t(a.a.sq.tokens), cuuint64_t(a.dim) / 64 + 1, h};
    const cuuint64_t qs[3] = {cuuint64_t(a.a.q_stride) * 2, 128, (cuuint64_t(a.dim) + moe::kLatentRot) * 2};
    const cuuint32_t qb[4] = {64, 128, cuuint32_t(a.dim) / 64 + 1, 1};
    const cuuint64_t kd[4] = {64, n, cuuint64_t(a.dim) / 64, h}, ks[3] = {cuuint64_t(a.k_token) * 2, 128, cuuint64_t(a.k_head) * 2};
    const cuuint32_t kb[4] = {64, rows, cuuint32_t(a.dim) / 64, 1};
    const cuuint64_t rd[2] = {moe::kLatentRot, n}, rs[1] = {cuuint64_t(a.rope_token) * 2};
    const cuuint32_t rb[2] = {moe::kLatentRot, rows};
    const cuuint64_t vd[3] = {cuuint64_t(a.dim), n, h}, vs[2] = {cuuint64_t(a.v_token) * 2, cuuint64_t(a.v_head) * 2};
    const cuuint32_t vb[3] = {64, moe::kExpandedKeys, 1};
    return map(&m->q, a.a.q, 4, qd, qs, qb) && map(&m->k, a.k, 4, kd, ks, kb) && map(&m->rope, a.rope, 2, rd, rs, rb) && map(&m->v, a.v, 3, vd, vs, vb);
}

}  // namespace

extern "C" {

moe_status_t moe_latent_append(const moe_rope_t* rope, const moe_latent_cache_t* cache,
                               const moe_seqs_t* seqs, const void* kv, int64_t kv_stride,
                               const float* gamma, float eps, const void* q_rope,
                               int64_t q_token_stride, int64_t q_head_stride,
                               const int32_t* positions, int32_t n_tokens, int32_t n_q_heads,
                               void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                               moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_seqs(seqs, true, true)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (!rope || rope->rot_dim != moe::kLatentRot || !std::isfinite(rope->magnitude) || n_q_heads <= 0 ||
        !std::isfinite(eps) || eps < 0.0f)
        return MOE_ERR_INVALID_ARG;
    if (n_q_heads > MOE_MAX_HEADS) return MOE_ERR_UNSUPPORTED;
    if (n_tokens == 0) return MOE_OK;
    if (!rows_ok(kv, kv_stride, cache->latent_dim + moe::kLatentRot) || !aligned(gamma, 16) ||
        !rows_ok(q_rope, q_token_stride, moe::kLatentRot) || !row_stride_ok(q_head_stride, moe::kLatentRot) ||
        !rows_ok(q_out, q_out_token_stride, moe::kLatentRot) || !row_stride_ok(q_out_head_stride, moe::kLatentRot))
        return MOE_ERR_INVALID_ARG;
    if (!positions || !aligned(positions, 4) || !rope->freqs || !aligned(rope->freqs, 4) || !aligned(rope->err, 4))
        return MOE_ERR_INVALID_ARG;
    moe::LatentAppendArgs a{};
    a.c = latent_args(cache);
    a.sq = seq_args(seqs, n_tokens);
    a.freqs = rope->freqs;
    a.interleaved = rope->interleaved != 0;
    a.magnitude = rope->magnitude;
    a.gamma = gamma;
    a.eps = eps;
    a.kv = static_cast<const uint16_t*>(kv);
    a.kv_stride = kv_stride;
    a.q = static_cast<const uint16_t*>(q_rope);
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.q_out = static_cast<uint16_t*>(q_out);
    a.out_token = q_out_token_stride;
    a.out_head = q_out_head_stride;
    a.pos = positions;
    a.q_heads = n_q_heads;
    a.err = rope->err;
    return cuda_status(moe::launch_latent_append(a, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_latent_workspace_bytes(const moe_attn_t* attn, const moe_latent_cache_t* cache) {
    if (check_cache(cache, false) != MOE_OK || check_attn(attn) != MOE_OK) return 0;
    return static_cast<size_t>(moe::latent_workspace_bytes(cache->latent_dim));
}

moe_status_t moe_latent_attention(const moe_attn_t* attn, const moe_latent_cache_t* cache,
                                  const moe_seqs_t* seqs, const void* q, int64_t q_stride,
                                  const uint64_t* draft_mask, int32_t n_tokens, void* out,
                                  float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_attn(attn)) != MOE_OK) return st;
    if ((st = check_seqs(seqs, true, true)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (n_tokens == 0) return MOE_OK;
    if (seqs->n_seqs == 0) return MOE_ERR_INVALID_ARG;
    if (!rows_ok(q, q_stride, int64_t(attn->n_q_heads) * (cache->latent_dim + moe::kLatentRot)) || !out || !aligned(out, 16) ||
        !aligned(lse, 4) || !aligned(draft_mask, 8))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe_latent_workspace_bytes(attn, cache))) != MOE_OK) return st;
    moe::LatentAttnArgs a{};
    a.a = attn_args(attn, seqs, q, q_stride, draft_mask, n_tokens, out, lse, ws, 1, cache->latent_dim);
    a.c = latent_args(cache);
    a.a.kv.page = a.c.page;
    a.a.kv.page_log2 = a.c.page_log2;
    a.a.kv.n_pages = a.c.n_pages;
    const bool few = int64_t(seqs->max_q) * attn->n_q_heads <= moe::kLatentRows / 2;
    a.q_flat = q_stride == int64_t(attn->n_q_heads) * (cache->latent_dim + moe::kLatentRot);
    moe::LatentMaps maps{};
    if (!make_maps(cache, &maps)) return MOE_ERR_CUDA;
    if (a.q_flat && !make_q_map(a, few, &maps)) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_latent_attn(a, maps, few, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_latent_gather(const moe_latent_cache_t* cache, const moe_seqs_t* seqs,
                               const int32_t* cu_k, int32_t n_rows, void* out, int64_t out_stride,
                               void* ws, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_cache(cache, true);
    if (st != MOE_OK) return st;
    if ((st = check_seqs(seqs, false, true)) != MOE_OK) return st;
    if (n_rows < 0) return MOE_ERR_INVALID_ARG;
    if (n_rows > MOE_MAX_KV_LEN) return MOE_ERR_UNSUPPORTED;
    if (n_rows == 0) return MOE_OK;
    if (seqs->n_seqs == 0) return MOE_ERR_INVALID_ARG;
    if (!cu_k || !aligned(cu_k, 4) || !rows_ok(out, out_stride, cache->latent_dim + moe::kLatentRot)) return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe::kCtlBytes)) != MOE_OK) return st;
    moe::LatentGatherArgs a{};
    a.c = latent_args(cache);
    a.sq = seq_args(seqs, 0);
    a.cu_k = cu_k;
    a.rows = n_rows;
    a.out = static_cast<uint16_t*>(out);
    a.out_stride = out_stride;
    a.err = static_cast<int32_t*>(ws);
    return cuda_status(moe::launch_latent_gather(a, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t moe_expanded_workspace_bytes(const moe_attn_t* attn, int32_t v_dim) {
    if (check_attn(attn) != MOE_OK || (v_dim != 64 && v_dim != 128)) return 0;
    return static_cast<size_t>(moe::expanded_workspace_bytes(v_dim));
}

moe_status_t moe_expanded_attention(const moe_attn_t* attn, const moe_seqs_t* seqs,
                                    const int32_t* cu_k, int32_t n_keys, int32_t v_dim,
                                    const void* q, int64_t q_stride, const void* k,
                                    int64_t k_token_stride, int64_t k_head_stride,
                                    const void* k_rope, int64_t rope_stride, const void* v,
                                    int64_t v_token_stride, int64_t v_head_stride,
                                    int32_t n_tokens, void* out, float* lse, void* ws,
                                    size_t ws_bytes, moe_stream_t stream) {
    moe_status_t st = check_attn(attn);
    if (st != MOE_OK) return st;
    if ((st = check_seqs(seqs, true, false)) != MOE_OK) return st;
    if ((st = check_tokens(n_tokens)) != MOE_OK) return st;
    if (n_keys < 0 || v_dim <= 0) return MOE_ERR_INVALID_ARG;
    if (v_dim != 64 && v_dim != 128) return MOE_ERR_UNSUPPORTED;
    if (n_tokens == 0) return MOE_OK;
    if (seqs->n_seqs == 0 || n_keys == 0) return MOE_ERR_INVALID_ARG;
    if (n_keys > MOE_MAX_KV_LEN) return MOE_ERR_UNSUPPORTED;
    if (!cu_k || !aligned(cu_k, 4) || !rows_ok(q, q_stride, int64_t(attn->n_q_heads) * (v_dim + moe::kLatentRot)) ||
        !rows_ok(k, k_token_stride, v_dim) || !row_stride_ok(k_head_stride, v_dim) ||
        !rows_ok(k_rope, rope_stride, moe::kLatentRot) || !rows_ok(v, v_token_stride, v_dim) ||
        !row_stride_ok(v_head_stride, v_dim) || !out || !aligned(out, 16) || !aligned(lse, 4))
        return MOE_ERR_INVALID_ARG;
    if ((st = check_ws(ws, ws_bytes, moe_expanded_workspace_bytes(attn, v_dim))) != MOE_OK) return st;
    moe::ExpandedArgs a{};
    a.a = attn_args(attn, seqs, q, q_stride, nullptr, n_tokens, out, lse, ws, attn->n_q_heads, v_dim);
    a.a.kv.page = 1;
    a.a.sq.max_pages = n_keys;
    a.cu_k = cu_k;
    a.n_keys = n_keys;
    a.dim = v_dim;
    a.k = static_cast<const uint16_t*>(k);
    a.rope = static_cast<const uint16_t*>(k_rope);
    a.v = static_cast<const uint16_t*>(v);
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.rope_token = rope_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    moe::ExpandedMaps maps;
    if (!make_maps(a, &maps)) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_expanded(a, maps, device_info().sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
