// latent.h -- arguments, workspace layout and launch entry points of the
// operators over a latent cache (latent_rows.cu, latent_attn.cu) and of the
// expanded form's attention (expanded.cu), used by their host ABI
// (latent_abi.cu).
#pragma once

#include "attn.h"

namespace moe {

constexpr int kLatentRot = MOE_LATENT_ROPE_DIM;   // 64: the rotary part of a row

// The latent cache as the kernels see it (strides in elements).
struct LatentArgs {
    uint8_t* latent;
    uint16_t* rope;
    int64_t lat_page, lat_token, rope_page, rope_token;
    int32_t e4m3, scale_log2;
    int32_t n_pages, page, page_log2, dim;
};

// 2^e, exactly, for the exponents that a cache may have and their opposites.
#ifdef __CUDACC__
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
#endif

struct LatentAppendArgs {
    LatentArgs c;
    SeqArgs sq;
    const float* freqs;
    int32_t interleaved;
    float magnitude;
    const float* gamma;      // NULL: no normalisation
    float eps;
    const uint16_t* kv;
    int64_t kv_stride;
    const uint16_t* q;
    int64_t q_token, q_head;
    uint16_t* q_out;
    int64_t out_token, out_head;
    const int32_t* pos;
    int32_t q_heads;
    int32_t* err;            // may be NULL
};

struct LatentGatherArgs {
    LatentArgs c;
    SeqArgs sq;              // cu_q unused
    const int32_t* cu_k;
    int32_t rows;
    uint16_t* out;
    int64_t out_stride;
    int32_t* err;
};

// Workspaces: the control block, one note per pair of CTAs (attn.h), then the pieces
// of split items, two slots a pair as there.  A slot has an item's rows, fp32: sums [dim/4][row][4], then (reference in log2 units, sum
// of powers) [row][2].
constexpr int kLatentRows = 128;        // rows of an item
constexpr int kLatentKeys = 64;         // keys of a tile
constexpr int kMaxPairs = kAttnMaxCtas / 2;

constexpr int kExpandedRows = 512;      // rows of an item of the expanded form
constexpr int kExpandedKeys = 128;

inline int64_t latent_workspace_bytes(int dim) {
    return kAttnPartials + int64_t(2) * kMaxPairs * kLatentRows * (dim + 2) * 4;
}

inline int64_t expanded_workspace_bytes(int dim) {
    return kAttnPartials + int64_t(2) * kMaxPairs * kExpandedRows * (dim + 2) * 4;
}

// Tensor maps of the cache: the latent as a 5-D tensor (64 elements or 128 codes of a
// row, eight tokens, such part of the row, such eight tokens, page), keys in boxes of
// whole rows of min(page, 32) tokens, values of half rows of min(page, 64); the rotary
// key as a 3-D one (element, token, page) in boxes as the keys'; q, if its rows lie one
// behind another, as a 3-D one (64 elements, row, such part of the row) in boxes of a
// CTA's rows.  128-byte swizzled.
struct LatentMaps {
    CUtensorMap keys, values, rope, q;
};

// Absorbed attention: `a` with one kv head of the latent's width and its rows the
// query heads of a token; q has the latent part and the rotary one side by side.
struct LatentAttnArgs {
    AttnArgs a;
    LatentArgs c;
    bool q_flat;             // q has no gaps between tokens
};

// Tensor maps of the expanded form: q and k as 4-D tensors (64 elements, token, such
// part of the head, head) in boxes of 128 and 64 tokens and the whole head; the rotary key (element,
// token) in boxes of 64 tokens; v (element, token, head) in boxes of 64 elements and 128
// tokens.  128-byte swizzled; what lies outside reads as zeros.
struct ExpandedMaps {
    CUtensorMap q, k, rope, v;
};

// Expanded attention: `a` with a kv head of its own for every query head, and
// pages of one token, so that lengths are cut to the n_keys rows there are.
struct ExpandedArgs {
    AttnArgs a;
    const int32_t* cu_k;
    int32_t n_keys, dim;     // dim: a head's own part of q and k, and v
    const uint16_t* k;
    const uint16_t* rope;
    const uint16_t* v;
    int64_t k_token, k_head, rope_token, v_token, v_head;
};

cudaError_t launch_latent_append(const LatentAppendArgs& a, int n_sms, cudaStream_t s);
cudaError_t launch_latent_gather(const LatentGatherArgs& a, int n_sms, cudaStream_t s);
// few: up to half of kLatentRows query rows a sequence (it only picks the kernel)
cudaError_t launch_latent_attn(const LatentAttnArgs& a, const LatentMaps& m, bool few, int n_sms, cudaStream_t s);
cudaError_t launch_expanded(const ExpandedArgs& a, const ExpandedMaps& m, int n_sms, cudaStream_t s);

}  // namespace moe
