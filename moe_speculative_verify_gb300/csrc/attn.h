// attn.h -- arguments, workspace layout and launch entry points of the
// attention-side kernels (rope.cu, attn.cu, keyw.cu, evict.cu), used by their
// host ABI (attn_abi.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// The paged cache as the kernels see it (strides in elements).
struct KvArgs {
    uint8_t* k;
    uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    int64_t page_stride, head_stride, token_stride;
    int32_t e4m3;
    int32_t n_pages, page, page_log2, heads, dim;
};

struct SeqArgs {
    const int32_t* cu_q;
    const int32_t* kv_len;
    const int32_t* table;
    int32_t n, max_pages, tokens;
};

// A split item that begins in CTA i: written there by every call's CTA i.
struct SplitNote {
    int32_t pieces;          // 0: none
    int32_t rows, row0;      // rows of the item, the first one's index in its sequence
    int32_t q0, head;        // its sequence's first token, its kv head
    int32_t pad[3];
};

// Workspace of the attention calls: the control block (error word), one note
// per CTA, then the pieces of split items: one slot per CTA for an item that
// begins there, after these one per CTA for an item that began before.  A slot
// has kAttnSlotRows rows, fp32: sums [dim/4][row][4], then (reference in log2
// units, sum of powers) [row][2].
constexpr int kAttnMaxCtas = 160;       // >= SMs of the card; larger grids are cut to it
constexpr int kAttnSlotRows = 256;
constexpr int64_t kAttnNotes = 256;     // byte offset
constexpr int64_t kAttnPartials = kAttnNotes + ((kAttnMaxCtas * sizeof(SplitNote) + 255) / 256) * 256;

inline int64_t attn_workspace_bytes(int dim) {
    return kAttnPartials + int64_t(2) * kAttnMaxCtas * kAttnSlotRows * (dim + 2) * 4;
}

struct RopeArgs {
    KvArgs kv;
    SeqArgs sq;
    const float* freqs;
    int32_t rot, interleaved;
    float magnitude;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride, out_stride;
    const int32_t* pos;
    uint16_t* q_out;
    int32_t q_heads;
    int32_t* err;            // may be NULL
};

struct AttnArgs {
    KvArgs kv;
    SeqArgs sq;
    const uint16_t* q;
    int64_t q_stride;
    const uint64_t* draft;   // NULL: causal or full
    uint16_t* out;
    float* lse;              // may be NULL
    int32_t q_heads, group;  // group = q_heads / kv heads
    float scale;
    int32_t causal, window;
    uint32_t group_magic;    // ceil(2^32 / group), 0 for a group of 1
    int32_t* err;
    SplitNote* notes;
    float* partials;
    uint64_t timeout_ns;

#ifdef __CUDACC__
    // row / group: exact for row * group < 2^32 (rows < 2^24, groups <= 256)
    __device__ __forceinline__ int query_of(int row) const {
        return group_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), group_magic)) : row;
    }
#endif
};

struct KeywArgs {
    AttnArgs a;              // out, notes and partials unused; lse is read
    float decay;
    const float* scores;
    float* scores_out;
    int64_t score_stride;
    int32_t tile_heads;      // rows of a tile: the query heads of a kv head (at most 128 at a time)
    int32_t tile_tokens;     // by so many tokens
    uint32_t tile_magic;     // ceil(2^32 / tile_tokens), 0 for one token

#ifdef __CUDACC__
    __device__ __forceinline__ int tile_of(int query) const {
        return tile_magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(query), tile_magic)) : query;
    }
#endif
};

struct EvictArgs {
    KvArgs kv;
    SeqArgs sq;              // cu_q unused
    const float* scores;
    int64_t score_stride;
    int32_t budget, recent;
    const int32_t* to_table;
    int32_t to_pages;
    int32_t* kept;
    float* scores_out;
    int32_t* new_len;
    int32_t* err;
};

// Tensor maps of K and V: 4-D (d, token, head, page), 128 bytes wide boxes
// (64 for e4m3 heads of 64) of min(page, tile) tokens, swizzled at that width.
struct KvMaps {
    CUtensorMap k, v;
};

// K as above, and q as a 3-D tensor (d, head, token) in boxes of 64 elements,
// tile_heads heads and tile_tokens tokens.
struct KeywMaps {
    CUtensorMap k, q;
};

// The widest window the kernels take, so that the place of a query (at least
// -MOE_MAX_TOKENS, where new tokens outnumber keys) less the window stays in 32
// bits; no sequence is long enough for a wider one to matter.
constexpr int kMaxWindow = 0x7FFFFFFF - 0x10000 - 1;

// Rows a kv head (new tokens of a sequence times query heads a kv head) up to
// which the few-rows kernel is taken: one 16-row matrix tile.
constexpr int kAttnFewRows = 16;
constexpr int kAttnTile = 64;       // keys of a tile of the few-rows kernel
constexpr int kAttnBigTile = 128;   // and of the tensor-memory kernel

cudaError_t launch_rope(const RopeArgs& a, int n_sms, cudaStream_t s);
cudaError_t launch_attn_rows(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s);
cudaError_t launch_attn_join(const AttnArgs& a, int n_notes, cudaStream_t s);
cudaError_t launch_attn_tile(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s);
cudaError_t launch_keyw(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s);
cudaError_t launch_evict(const EvictArgs& a, int max_len, cudaStream_t s);

}  // namespace moe
