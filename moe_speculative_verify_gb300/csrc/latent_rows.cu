// latent_rows.cu -- rows of a latent cache written and read back (sm_103a):
// the step's latents normalised, rotary positions on the shared keys and on the
// queries' rotary parts, rows stored; and cached rows gathered as bf16.
//
// A latent x of C elements becomes x * rsqrt(sum x^2 / C + eps) * gamma, the sum
// in fp32 in a fixed order (of x times a power of two where squares would leave
// fp32's range); e4m3 rows hold the code of that times 2^-e, which is exact, so
// the code is the only rounding.  Pairs turn as in rope.cu, with angles
// right to fp32 at any |position| < 2^24.
//
// Both are copies bound by HBM at chunk sizes and by latency at verify sizes:
// each element is read and written once, in 16-byte pieces.
#include "attn.cuh"
#include "latent.h"

namespace moe {

namespace {

constexpr int kAppendThreads = 128;

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// 16 elements of a rotary part, as two pieces of 8 that hold whole pairs: piece w
// of four.  Interleaved: elements 16 w .. 16 w + 15; else 8 w .. and 32 + 8 w ...
struct Part {
    uint4 x, y;
};

__device__ __forceinline__ int part_e0(bool inter, int w) { return inter ? 16 * w : 8 * w; }
__device__ __forceinline__ int part_e1(bool inter, int w) { return inter ? 16 * w + 8 : 32 + 8 * w; }

__device__ __forceinline__ Part load_part(const uint16_t* p, bool inter, int w) {
    Part r;
    r.x = *reinterpret_cast<const uint4*>(p + part_e0(inter, w));
    r.y = *reinterpret_cast<const uint4*>(p + part_e1(inter, w));
    return r;
}

__device__ __forceinline__ void turn_store(uint16_t* o, const Part& r, bool inter, int w, const float2* cs, bool zero) {
    float x[8], y[8];
    unpack8(r.x, x);
    unpack8(r.y, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 c = cs[8 * w + i];
        float* p1 = inter ? (i < 4 ? &x[2 * i] : &y[2 * i - 8]) : &x[i];
        float* p2 = inter ? p1 + 1 : &y[i];
        const float x1 = *p1, x2 = *p2;
        *p1 = __fsub_rn(__fmul_rn(x1, c.x), __fmul_rn(x2, c.y));
        *p2 = __fadd_rn(__fmul_rn(x2, c.x), __fmul_rn(x1, c.y));
    }
    const uint4 z = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(o + part_e0(inter, w)) = zero ? z : pack8(x);
    *reinterpret_cast<uint4*>(o + part_e1(inter, w)) = zero ? z : pack8(y);
}

// A block takes one token, or a share of its heads when there are few tokens
// (blockIdx.y); the first share also has the token's row.
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const LatentAppendArgs a) {
    __shared__ float2 s_cs[kLatentRot / 2];
    __shared__ float s_sum[kAppendThreads / 32];
    __shared__ int s_seq, s_bad;                 // lowest sequence with this token; first one that does not fit
    const int t = blockIdx.x, tid = threadIdx.x;
    const bool inter = a.interleaved != 0, row = blockIdx.y == 0;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_seq = s_bad = a.sq.n;
    __syncthreads();
    for (int b = tid; b < a.sq.n; b += kAppendThreads) {
        const int c0 = a.sq.cu_q[b], c1 = a.sq.cu_q[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.sq.tokens)
            atomicMin(&s_bad, b);
        else if (t >= c0 && t < c1)
            atomicMin(&s_seq, b);
    }
    // the thread's first pieces are on their way while the angles are worked out
    const uint16_t* kv = a.kv + t * a.kv_stride;
    const int pieces = a.c.dim / 8, units = 4 * a.q_heads;
    const bool mine = row && tid < pieces;
    uint4 lat = make_uint4(0, 0, 0, 0);
    if (mine) lat = *reinterpret_cast<const uint4*>(kv + 8 * tid);
    Part key{lat, lat};
    const int kw = tid - (kAppendThreads - 4);                   // the last four threads: the shared key
    if (row && kw >= 0) key = load_part(kv + a.c.dim, inter, kw);
    const int step = gridDim.y * kAppendThreads;
    int u = blockIdx.y * kAppendThreads + tid;
    Part q{lat, lat};
    auto fetch = [&](int v) { return load_part(a.q + t * a.q_token + (v >> 2) * a.q_head, inter, v & 3); };
    if (u < units) q = fetch(u);
    if (tid < kLatentRot / 2) {
        const float pos = static_cast<float>(a.pos[t]);
        const float hi = a.freqs[2 * tid], lo = a.freqs[2 * tid + 1];
        const float p = __fmul_rn(pos, hi);
        const float e = __fmaf_rn(pos, lo, __fmaf_rn(pos, hi, -p));
        float sn, cs;
        sincospif(2.0f * __fadd_rn(p - rintf(p), e), &sn, &cs);
        s_cs[tid] = make_float2(cs * a.magnitude, sn * a.magnitude);
    }
    float x[8];
    unpack8(lat, x);
    const bool norm = row && a.gamma;
    auto add_squares = [&](float f) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i] * f, x[i] * f, sum);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
    };
    auto mean = [&](float eps) { return __fadd_rn((s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) / a.c.dim, eps); };
    if (norm) add_squares(1.0f);
    __syncthreads();
    float p2 = 1.0f, r = 1.0f;                   // x r p2 is the normalised row
    if (norm) {
        float m = mean(a.eps);
        if (m == INFINITY || m < 0x1p-100f) {    // (all of the block: squares past fp32's end, or below where it keeps their bits)
            p2 = m == INFINITY ? 0x1p-70f : 0x1p70f;
            __syncthreads();
            add_squares(p2);
            __syncthreads();
            m = mean(a.eps * p2 * p2);
        }
        r = 1.0f / sqrtf(m);
    }
    // (from the first sequence on whose offsets do not fit, none has new tokens)
    const int b = s_seq < s_bad ? s_seq : -1;
    if (row) {
        // this token's place in the cache; pg < 0: not stored
        int pg = -1;
        int64_t at = 0;
        bool lost = s_bad < a.sq.n;
        if (b >= 0) {
            at = int64_t(a.sq.kv_len[b]) - a.sq.cu_q[b + 1] + t;
            if (at >= 0 && (at >> a.c.page_log2) < a.sq.max_pages) {
                pg = a.sq.table[int64_t(b) * a.sq.max_pages + (at >> a.c.page_log2)];
                if (pg >= a.c.n_pages) pg = -1;
            }
            lost = lost || (at >= 0 && pg < 0);
        }
        if (lost && tid == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
        at &= a.c.page - 1;
        if (pg >= 0 && mine) {
            if (a.gamma) {
                const float4 g0 = reinterpret_cast<const float4*>(a.gamma)[2 * tid];
                const float4 g1 = reinterpret_cast<const float4*>(a.gamma)[2 * tid + 1];
                const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(__fmul_rn(x[i], r), p2), g[i]);
            }
            const int64_t o = pg * a.c.lat_page + at * a.c.lat_token + 8 * tid;
            if (a.c.e4m3) {
                const float f = pow2(-a.c.scale_log2);
                *reinterpret_cast<uint2*>(a.c.latent + o) =
                    make_uint2(to_e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f), to_e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
            } else {
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.c.latent) + o) = pack8(x);
            }
        }
        if (pg >= 0 && kw >= 0) turn_store(a.c.rope + pg * a.c.rope_page + at * a.c.rope_token, key, inter, kw, s_cs, false);
    }
    while (u < units) {
        turn_store(a.q_out + t * a.out_token + (u >> 2) * a.out_head, q, inter, u & 3, s_cs, b < 0);
        u += step;
        if (u < units) q = fetch(u);
    }
}

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 8;              // rows of a warp at a time
constexpr int kGatherFlight = 4;            // of them in flight

// Rows of the output, kGatherRows a warp in turn.  Lanes 0 .. 7 each look a row's
// place up, then the warp copies the rows in 16-byte pieces.
__global__ void __launch_bounds__(kGatherThreads) latent_gather_kernel(const LatentGatherArgs a) {
    __shared__ int s_bad;                        // first sequence whose offsets do not fit
    const int tid = threadIdx.x, lane = tid & 31, n = a.sq.n;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_bad = n;
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < n; b += kGatherThreads) {
        const int c0 = a.cu_k[b], c1 = a.cu_k[b + 1], len = a.sq.kv_len[b];
        if (c0 < 0 || c1 < c0 || c1 > a.rows) {
            atomicMin(&s_bad, b);
            bad = true;
        }
        bad = bad || len < 0 || len > min(int64_t(a.sq.max_pages) * a.c.page, int64_t(MOE_MAX_KV_LEN));
    }
    if (bad) record_error(a.err, MOE_ERR_INVALID_ARG);
    __syncthreads();
    const int seqs = s_bad, C = a.c.dim;
    const int warps = gridDim.x * (kGatherThreads / 32);
    const int lat_pieces = C / 8, all = (C + kLatentRot) / 8;
    for (int r0 = (blockIdx.x * (kGatherThreads / 32) + (tid >> 5)) * kGatherRows; r0 < a.rows; r0 += warps * kGatherRows) {
        // this lane's row: its page and its place there, page < 0 where there is none
        int page = -1, slot = 0;
        const int r = r0 + lane;
        if (lane < kGatherRows && r < a.rows && seqs > 0 && r >= a.cu_k[0]) {
            int lo = 0, hi = seqs;               // the last sequence of the first `seqs` that begins at or before r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.cu_k[mid] <= r)
                    lo = mid;
                else
                    hi = mid;
            }
            const int64_t at = r - a.cu_k[lo];
            if (r < a.cu_k[lo + 1] && at < a.sq.kv_len[lo] && (at >> a.c.page_log2) < a.sq.max_pages) {
                page = a.sq.table[int64_t(lo) * a.sq.max_pages + (at >> a.c.page_log2)];
                slot = static_cast<int>(at) & (a.c.page - 1);
                if (page < 0 || page >= a.c.n_pages) {
                    page = -1;
                    record_error(a.err, MOE_ERR_INVALID_ARG);
                }
            }
        }
        __syncwarp();
        const int count = min(kGatherRows, a.rows - r0);
        for (int k0 = 0; k0 < count; k0 += kGatherFlight) {
            int64_t lat[kGatherFlight], rot[kGatherFlight];
            bool on[kGatherFlight];
#pragma unroll
            for (int k = 0; k < kGatherFlight; ++k) {
                const int pg = __shfl_sync(0xFFFFFFFFu, page, k0 + k), sl = __shfl_sync(0xFFFFFFFFu, slot, k0 + k);
                on[k] = pg >= 0;
                lat[k] = on[k] ? pg * a.c.lat_page + sl * a.c.lat_token : 0;
                rot[k] = on[k] ? pg * a.c.rope_page + sl * a.c.rope_token : 0;
            }
            const uint4 zero = make_uint4(0, 0, 0, 0);
            if (!a.c.e4m3) {
                const uint16_t* src = reinterpret_cast<const uint16_t*>(a.c.latent);
                for (int p = lane; p < all; p += 32) {
                    uint4 v[kGatherFlight];
#pragma unroll
                    for (int k = 0; k < kGatherFlight; ++k) {
                        v[k] = zero;
                        if (on[k] && k0 + k < count)
                            v[k] = p < lat_pieces ? *reinterpret_cast<const uint4*>(src + lat[k] + 8 * p)
                                                  : *reinterpret_cast<const uint4*>(a.c.rope + rot[k] + 8 * (p - lat_pieces));
                    }
#pragma unroll
                    for (int k = 0; k < kGatherFlight; ++k)
                        if (k0 + k < count)
                            *reinterpret_cast<uint4*>(a.out + int64_t(r0 + k0 + k) * a.out_stride + 8 * p) = v[k];
                }
            } else {
                const float f = pow2(a.c.scale_log2);                            // code * f is a bf16
                for (int p = lane; p < all; p += 32) {
                    uint4 v[kGatherFlight];
#pragma unroll
                    for (int k = 0; k < kGatherFlight; ++k) {
                        v[k] = zero;
                        if (on[k] && k0 + k < count) {
                            if (p < lat_pieces) {
                                const uint2 w = *reinterpret_cast<const uint2*>(a.c.latent + lat[k] + 8 * p);
                                v[k].x = w.x;
                                v[k].y = w.y;
                            } else {
                                v[k] = *reinterpret_cast<const uint4*>(a.c.rope + rot[k] + 8 * (p - lat_pieces));
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kGatherFlight; ++k) {
                        if (k0 + k >= count) continue;
                        uint4 o = v[k];
                        if (p < lat_pieces) {
                            const uint32_t h[4] = {e4m3x2_to_f16x2(v[k].x), e4m3x2_to_f16x2(v[k].x >> 16),
                                                   e4m3x2_to_f16x2(v[k].y), e4m3x2_to_f16x2(v[k].y >> 16)};
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
                                w[e] = pack_bf16(y.x * f, y.y * f);
                            }
                            o = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        *reinterpret_cast<uint4*>(a.out + int64_t(r0 + k0 + k) * a.out_stride + 8 * p) = o;
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, int n_sms, cudaStream_t s) {
    int parts = n_sms / a.sq.tokens;                       // few tokens: a token's heads over several blocks
    const int most = (4 * a.q_heads + kAppendThreads - 1) / kAppendThreads;
    parts = parts < 1 ? 1 : (parts > most ? most : parts);
    cudaError_t e = launch_pdl(latent_append_kernel, dim3(a.sq.tokens, parts), dim3(kAppendThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherArgs& a, int n_sms, cudaStream_t s) {
    const int per = kGatherRows * (kGatherThreads / 32);
    const int want = (a.rows + per - 1) / per, most = 8 * n_sms;
    cudaError_t e = launch_pdl(latent_gather_kernel, dim3(want < most ? want : most), dim3(kGatherThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
