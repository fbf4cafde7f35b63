// evict.cu -- cuts the cache to a budget of keys per kv head by accumulated
// attention weight (sm_103a).
//
// Selection: one CTA per (sequence, kv head) finds the budget-th largest key
// by radix selection on the scores' ordered bits, which it keeps in shared
// memory: 11, 11 and 10 bits a pass (the first digit has sign, exponent and two
// fraction bits, so that scores of one magnitude still fall into several
// bins).  A key above the threshold is kept, of those equal to it the lowest
// places; a scan over the places gives each kept one its rank, which is the
// row it moves to.  Integer counts only, so the result does not depend on any
// order.  (A cluster of 8 or 16 CTAs a pair, with the counts
// added through distributed shared memory: its five cluster barriers and
// remote reads took longer, 12 to 16 us for 8192 places.)
//
// The move, all but a few percent of the bytes, is a kernel of its own, so
// that its blocks spread evenly over the card whatever the pairs: a thread
// has four rows' 16-byte pieces of K and V in flight.
//
// Measured (8 kv heads of 128): one sequence of 8,191 keys cut to 4,096 (bf16) 15
// us, most of it the selection's dependent passes; 16 of 5,003 to 32,003 keys
// cut to 8,000 (e4m3) 108 us, 4.8 TB/s.
#include "attn.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 49152;               // places whose keys shared memory holds

// Order of the scores as an unsigned integer: NaN lowest, -0 = +0, the recent
// keys above every score.
__device__ __forceinline__ uint32_t score_key(float v, bool recent) {
    if (recent) return 0xFFFFFFFFu;
    if (v != v) return 0u;
    if (v == 0.0f) v = 0.0f;
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads, 1) select_kernel(const EvictArgs a, int held_cap) {
    extern __shared__ __align__(16) uint32_t s_key[];   // the keys, where they fit
    __shared__ int s_hist[2048];
    __shared__ int s_digit, s_rest;
    __shared__ int2 s_warp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int bh = blockIdx.x, b = bh / a.kv.heads, h = bh - b * a.kv.heads;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t cap = min(min(int64_t(a.sq.max_pages) * a.kv.page, a.score_stride), int64_t(MOE_MAX_KV_LEN));
    const int len = a.sq.kv_len[b];
    const int n = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
    if (n != len && tid == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
    const int keep = min(n, a.budget), first_recent = n - a.recent;
    const float* sc = a.scores + int64_t(bh) * a.score_stride;
    int32_t* kept = a.kept + int64_t(bh) * a.budget;
    float* so = a.scores_out + int64_t(bh) * a.score_stride;
    // each warp's part of the places, in order, a lane four places at a time
    const int64_t per = (int64_t(n) + 4 * kThreads - 1) / (4 * kThreads) * 128;
    const int w0 = static_cast<int>(min(int64_t(n), wid * per)), w1 = static_cast<int>(min(int64_t(n), (wid + 1) * per));
    const bool held = n <= held_cap;
    // keys of places j .. j + 3, j a multiple of 4 (past the end: whatever)
    auto keys_at = [&](int j, uint32_t (&k)[4]) {
        if (held) {
            const uint4 x = *reinterpret_cast<const uint4*>(s_key + j);
            k[0] = x.x;
            k[1] = x.y;
            k[2] = x.z;
            k[3] = x.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) k[i] = j + i < n ? score_key(sc[j + i], j + i >= first_recent) : 0u;
        }
    };

    const bool all = n <= keep;
    uint32_t prefix = 0;                         // digits of the threshold so far
    int need = keep;                             // of the keys with that prefix
    if (!all) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), above = pass == 1 ? 21 : 10;
            const uint32_t mask = pass == 2 ? 1023u : 2047u;
            for (int i = tid; i < 2048; i += kThreads) s_hist[i] = 0;
            __syncthreads();
            // (adds of one to one address are added up by the hardware across a warp)
            if (pass == 0) {
                for (int j0 = w0; j0 < w1; j0 += 32 * 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + 32 * i + lane;
                        v[i] = j < w1 ? __ldg(sc + j) : 0.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + 32 * i + lane;
                        const uint32_t k = score_key(v[i], j >= first_recent);
                        if (j < w1) {
                            if (held) s_key[j] = k;
                            atomicAdd(&s_hist[k >> 21], 1);
                        }
                    }
                }
            } else {
#pragma unroll 2
                for (int j = w0 + 4 * lane; j < w1; j += 128) {
                    uint32_t k[4];
                    keys_at(j, k);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (j + i < w1 && (k[i] >> above) == (prefix >> above)) atomicAdd(&s_hist[(k[i] >> shift) & mask], 1);
                }
            }
            __syncthreads();
            // the digit whose keys hold the need-th largest: thread t has digits 2047 - 2t and one below
            const int c0 = s_hist[2047 - 2 * tid], c1 = s_hist[2046 - 2 * tid];
            int incl = c0 + c1;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                if (lane >= d) incl += o;
            }
            if (lane == 31) s_warp[wid].x = incl;
            __syncthreads();
            int o = lane < wid ? s_warp[lane].x : 0;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) o += __shfl_xor_sync(0xFFFFFFFFu, o, d);
            const int before = o + incl - c0 - c1;
            if (before < need && need <= before + c0 + c1) {
                const bool second = need > before + c0;
                s_digit = 2047 - 2 * tid - (second ? 1 : 0);
                s_rest = need - before - (second ? c0 : 0);
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(s_digit) << shift;
            need = s_rest;
        }
    }
    // --- ranks: keys above the threshold, and the first `need` equal to it
    // four places' kinds: bit i above, bit 4 + i equal
    auto kinds_at = [&](int j) {
        uint32_t k[4], m = 0;
        if (!all) keys_at(j, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i < w1) m |= all || k[i] > prefix ? 1u << i : (k[i] == prefix ? 16u << i : 0u);
        return m;
    };
    int2 sum = make_int2(0, 0);
    for (int j = w0 + 4 * lane; j < w1; j += 128) {
        const uint32_t m = kinds_at(j);
        sum.x += __popc(m & 15u);
        sum.y += __popc(m >> 4);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, d);
        sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, d);
    }
    if (lane == 0) s_warp[wid] = sum;
    __syncthreads();
    int2 at = make_int2(0, 0);
    {
        int2 o = s_warp[lane];                   // (32 warps)
        if (lane >= wid) o = make_int2(0, 0);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, d);
            o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, d);
        }
        at = o;
    }
    for (int j0 = w0; j0 < w1; j0 += 128) {
        const int j = j0 + 4 * lane;
        const uint32_t m = j < w1 ? kinds_at(j) : 0u;
        const uint32_t mine = __popc(m & 15u) | (__popc(m >> 4) << 16);
        uint32_t incl = mine;                    // counts of the lanes up to this one, packed
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        int gt = at.x + static_cast<int>((incl - mine) & 0xFFFFu), eq = at.y + static_cast<int>((incl - mine) >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool is_gt = (m >> i) & 1u, is_eq = (m >> (4 + i)) & 1u;
            if (is_gt || (is_eq && eq < need)) {
                const int r = gt + min(eq, need);
                kept[r] = j + i;
                so[r] = sc[j + i];
            }
            gt += is_gt;
            eq += is_eq;
        }
        const uint32_t last = __shfl_sync(0xFFFFFFFFu, incl, 31);
        at.x += last & 0xFFFFu;
        at.y += last >> 16;
    }
    for (int r = keep + tid; r < a.budget; r += kThreads) kept[r] = -1;
    if (h == 0 && tid == 0) a.new_len[b] = keep;
}

constexpr int kMoveThreads = 256, kFlight = 4;

// LANES threads move a row (16 bytes of K and of V each); a block
// kFlight * kMoveThreads / LANES rows of one pair, from row block `block0` on.
// Pairs are the grid's x, which alone may pass 65,535.
template <int LANES, int ES>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a, int block0) {
    constexpr int kRows = kMoveThreads / LANES;
    pdl_wait();
    pdl_launch_dependents();
    const int bh = blockIdx.x, b = bh / a.kv.heads, h = bh - b * a.kv.heads;
    const int keep = a.new_len[b], r0 = (block0 + static_cast<int>(blockIdx.y)) * kFlight * kRows + threadIdx.x / LANES;
    const int32_t* kept = a.kept + int64_t(bh) * a.budget;
    const int32_t* from = a.sq.table + int64_t(b) * a.sq.max_pages;
    const int32_t* to = a.to_table + int64_t(b) * a.to_pages;
    const int64_t head = h * a.kv.head_stride;
    const int sub = 16 * (threadIdx.x % LANES);
    int j[kFlight], pd[kFlight], ps[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
        const int r = r0 + i * kRows;
        j[i] = r < keep ? kept[r] : -1;
        pd[i] = r < keep ? to[r >> a.kv.page_log2] : -1;
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) ps[i] = j[i] >= 0 ? from[j[i] >> a.kv.page_log2] : -1;
    uint4 x[kFlight], y[kFlight];
    int64_t dst[kFlight];
    unsigned bad = 0;                            // bit i: row i has no source page; 16: a row has no destination page
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
        const int r = r0 + i * kRows;
        dst[i] = -1;
        if (j[i] < 0) continue;
        if (pd[i] < 0 || pd[i] >= a.kv.n_pages) {
            bad |= 16u;
            continue;
        }
        if (ps[i] < 0 || ps[i] >= a.kv.n_pages) {        // its own destination is loaded, zeros are stored
            bad |= 1u << i;
            ps[i] = pd[i];
            j[i] = r;
        }
        const int64_t src = ES * (ps[i] * a.kv.page_stride + head + (j[i] & (a.kv.page - 1)) * a.kv.token_stride) + sub;
        dst[i] = ES * (pd[i] * a.kv.page_stride + head + (r & (a.kv.page - 1)) * a.kv.token_stride) + sub;
        x[i] = *reinterpret_cast<const uint4*>(a.kv.k + src);
        y[i] = *reinterpret_cast<const uint4*>(a.kv.v + src);
    }
    if (bad) {
        if (sub == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if ((bad >> i) & 1u) x[i] = y[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
        if (dst[i] >= 0) {
            *reinterpret_cast<uint4*>(a.kv.k + dst[i]) = x[i];
            *reinterpret_cast<uint4*>(a.kv.v + dst[i]) = y[i];
        }
}

template <int LANES, int ES>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
    constexpr int kMost = 65535;                 // row blocks of a launch
    const int rows = kFlight * kMoveThreads / LANES, most = a.budget < MOE_MAX_KV_LEN ? a.budget : MOE_MAX_KV_LEN;
    const int blocks = (most + rows - 1) / rows;
    cudaError_t e = cudaSuccess;
    for (int k = 0; k < blocks && e == cudaSuccess; k += kMost)
        e = launch_pdl(move_kernel<LANES, ES>, dim3(a.sq.n * a.kv.heads, blocks - k < kMost ? blocks - k : kMost),
                       dim3(kMoveThreads), 0, s, a, k);
    return e;
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int max_len, cudaStream_t s) {
    const int cap = max_len < kHeld ? max_len : kHeld;
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(select_kernel), kHeld * 4);
    if (e != cudaSuccess) return e;
    e = launch_pdl(select_kernel, dim3(a.sq.n * a.kv.heads), dim3(kThreads), (size_t(cap) + 3) / 4 * 16, s, a, cap);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.kv.dim == 128)
        e = a.kv.e4m3 ? launch_move<8, 1>(a, s) : launch_move<16, 2>(a, s);
    else
        e = a.kv.e4m3 ? launch_move<4, 1>(a, s) : launch_move<8, 2>(a, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
