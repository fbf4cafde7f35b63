// evict.cu -- cuts the cache to a budget of keys per kv head by accumulated
// attention weight (sm_103a).
//
// One cluster of CTAs per (sequence, kv head).  The budget-th largest key is
// found by radix selection, 8 bits a pass, on the scores' ordered bits: each
// CTA counts its contiguous slice of the places in shared memory, the counts
// are added through distributed shared memory, and every CTA finds the same
// digit.  A key above the threshold is kept, of those equal to it the lowest
// places; a scan over the slices then gives each kept place its rank, which
// is the row it moves to.  Integer counts only, so the result does not depend
// on any order.  The rows then move in 16-byte pieces, the bulk of the bytes.
#include <cooperative_groups.h>

#include "attn.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kCluster = 8;

// Order of the scores as an unsigned integer: NaN lowest, -0 = +0, the recent
// keys above every score.
__device__ __forceinline__ uint32_t score_key(float v, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (v != v) return 0u;
    if (v == 0.0f) v = 0.0f;
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
    __shared__ int s_hist[2][256];
    __shared__ int s_sum[256];
    __shared__ int s_digit, s_rest;
    __shared__ int2 s_count;                    // this CTA's (above, equal)
    __shared__ int2 s_warp[kThreads / 32];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int cr = static_cast<int>(cl.block_rank());
    const int bh = blockIdx.x / kCluster, b = bh / a.kv.heads, h = bh - b * a.kv.heads;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t cap = min(int64_t(a.sq.max_pages) * a.kv.page, a.score_stride);
    const int len = a.sq.kv_len[b];
    const int n = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
    if (n != len && tid == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
    const int keep = min(n, a.budget), first_recent = n - a.recent;
    const float* sc = a.scores + int64_t(bh) * a.score_stride;
    int32_t* kept = a.kept + int64_t(bh) * a.budget;
    float* so = a.scores_out + int64_t(bh) * a.score_stride;
    // this CTA's slice of the places, in order
    const int s0 = static_cast<int>(int64_t(n) * cr / kCluster);
    const int s1 = static_cast<int>(int64_t(n) * (cr + 1) / kCluster);

    uint32_t prefix = 0;                         // digits of the threshold so far
    int need = keep;                             // of the keys with that prefix
    if (n > keep) {
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            int* hist = s_hist[pass & 1];
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = s0 + tid; j < s1; j += kThreads) {
                const uint32_t k = score_key(sc[j], j >= first_recent);
                if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            cl.sync();
            if (tid < 256) {
                int v = 0;
#pragma unroll
                for (int c = 0; c < kCluster; ++c) v += cl.map_shared_rank(hist, c)[tid];
                s_sum[tid] = v;
            }
            __syncthreads();
            if (tid < 32) {                      // the digit whose keys hold the need-th largest
                int v[8], mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine += v[i] = s_sum[255 - 8 * tid - i];
                int incl = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (lane >= d) incl += o;
                }
                int before = incl - mine;
                if (before < need && need <= incl) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (before < need && need <= before + v[i]) {
                            s_digit = 255 - 8 * tid - i;
                            s_rest = need - before;
                        }
                        before += v[i];
                    }
                }
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(s_digit) << shift;
            need = s_rest;
        }
    }
    // --- ranks: keys above the threshold, and the first `need` equal to it
    const bool all = n <= keep;
    int2 mine = make_int2(0, 0);
    // a thread's places are contiguous, so ranks follow the places' order
    const int len_c = s1 - s0, per = (len_c + kThreads - 1) / kThreads;
    const int j0 = min(s1, s0 + tid * per), j1 = min(s1, j0 + per);
    for (int j = j0; j < j1; ++j) {
        const uint32_t k = score_key(sc[j], j >= first_recent);
        mine.x += all || k > prefix;
        mine.y += !all && k == prefix;
    }
    int2 incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl.x, d), y = __shfl_up_sync(0xFFFFFFFFu, incl.y, d);
        if (lane >= d) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 31) s_warp[wid] = incl;
    __syncthreads();
    int2 at = make_int2(incl.x - mine.x, incl.y - mine.y);
    int2 sum = make_int2(0, 0);
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < wid) {
            at.x += s_warp[w].x;
            at.y += s_warp[w].y;
        }
        sum.x += s_warp[w].x;
        sum.y += s_warp[w].y;
    }
    if (tid == 0) s_count = sum;
    cl.sync();
    for (int c = 0; c < cr; ++c) {
        const int2 o = *cl.map_shared_rank(&s_count, c);
        at.x += o.x;
        at.y += o.y;
    }
    for (int j = j0; j < j1; ++j) {
        const float v = sc[j];
        const uint32_t k = score_key(v, j >= first_recent);
        const bool eq = !all && k == prefix;
        if (all || k > prefix || (eq && at.y < need)) {
            const int r = at.x + min(at.y, need);
            kept[r] = j;
            so[r] = v;
        }
        at.x += all || k > prefix;
        at.y += eq;
    }
    for (int r = keep + cr * kThreads + tid; r < a.budget; r += kCluster * kThreads) kept[r] = -1;
    if (h == 0 && cr == 0 && tid == 0) a.new_len[b] = keep;
    cl.sync();                                   // the kept list is whole; no CTA's counts are read any more
    // --- move the rows: a row is rb/16 threads' work, K and V together
    const int rb = a.kv.dim * (a.kv.e4m3 ? 1 : 2), lanes = rb / 16, es = a.kv.e4m3 ? 1 : 2;
    const int sub = tid % lanes;
    const int32_t* from = a.sq.table + int64_t(b) * a.sq.max_pages;
    const int32_t* to = a.to_table + int64_t(b) * a.to_pages;
    const int rows_c = kThreads / lanes;
    for (int r = cr * rows_c + tid / lanes; r < keep; r += kCluster * rows_c) {
        const int j = __ldcg(kept + r);
        const int ps = from[j >> a.kv.page_log2], pd = to[r >> a.kv.page_log2];
        if (ps < 0 || ps >= a.kv.n_pages || pd < 0 || pd >= a.kv.n_pages) {
            if (sub == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
            continue;
        }
        const int64_t src = es * (ps * a.kv.page_stride + h * a.kv.head_stride +
                                  (j & (a.kv.page - 1)) * a.kv.token_stride) + 16 * sub;
        const int64_t dst = es * (pd * a.kv.page_stride + h * a.kv.head_stride +
                                  (r & (a.kv.page - 1)) * a.kv.token_stride) + 16 * sub;
        const uint4 x = *reinterpret_cast<const uint4*>(a.kv.k + src);
        const uint4 y = *reinterpret_cast<const uint4*>(a.kv.v + src);
        *reinterpret_cast<uint4*>(a.kv.k + dst) = x;
        *reinterpret_cast<uint4*>(a.kv.v + dst) = y;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
    const cudaError_t e = launch_pdl_cluster(evict_kernel, dim3(a.sq.n * a.kv.heads * kCluster), dim3(kThreads),
                                             kCluster, 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
