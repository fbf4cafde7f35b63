// rope.cu -- rotary positions on the step's new q and k, and k and v stored
// into the paged cache (sm_103a).
//
// Pair i of a head turns by the angle 2 pi pos f_i: y1 = m (x1 cos - x2 sin),
// y2 = m (x2 cos + x1 sin).  f_i comes as fp32 hi + lo; pos*hi is split
// exactly into p + e with one fma, whole turns leave p exactly, so the
// fraction of a turn is right to fp32 rounding at any |pos| < 2^24, where the
// product alone would lose all its fraction bits.
//
// Bound by HBM at chunk sizes and by latency at verify sizes: each element is
// read and written once, in 16-byte pieces.  A CTA takes one token (or a part
// of its heads when there are few tokens), so a token's cos and sin are
// computed once, into shared memory.
#include "attn.cuh"

namespace moe {

namespace {

// Small blocks: a block is a token's chain of latencies (its sequence, its
// page, its angles), and more of them share an SM.  Measured for 4096 tokens,
// 64 + 16 heads of 128: 128 threads 30.8 us (5.4 TB/s of the 6.7 of a copy), 256
// 34.7, 512 52.6; two units of a thread in flight 32.1, three of 256 threads 37.1.
constexpr int kRopeThreads = 128;
constexpr int kFlight = 1;                  // units of a thread in flight

struct Vec8 {
    float v[8];
};

__device__ __forceinline__ Vec8 unpack8(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return r;
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const Vec8& r) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]),
                                              pack_bf16(r.v[4], r.v[5]), pack_bf16(r.v[6], r.v[7]));
}

__device__ __forceinline__ void store8_e4m3(uint8_t* p, const Vec8& r, float scale) {
    uint2 w;
    w.x = to_e4m3x4(r.v[0] / scale, r.v[1] / scale, r.v[2] / scale, r.v[3] / scale);
    w.y = to_e4m3x4(r.v[4] / scale, r.v[5] / scale, r.v[6] / scale, r.v[7] / scale);
    *reinterpret_cast<uint2*>(p) = w;
}

// A unit is 16 elements of a head: two pieces of 8 that hold whole pairs.
struct Unit {
    const uint16_t* src;     // the head
    int kind;                // 0: q, 1: k, 2: v, -1: past the last unit
    int head, e0, e1;        // its two pieces
    int pair;                // first pair of it
    bool turn;
};

struct Raw {
    uint4 x, y;
};

__device__ __forceinline__ Unit unit_of(const RopeArgs& a, int t, int u, int units, int per, int half) {
    Unit r;
    int head = u / per;
    const int w = u - head * per;
    r.kind = u >= units ? -1 : (head < a.q_heads ? 0 : (head < a.q_heads + a.kv.heads ? 1 : 2));
    head -= r.kind <= 0 ? 0 : (r.kind == 1 ? a.q_heads : a.q_heads + a.kv.heads);
    r.head = head;
    r.turn = r.kind != 2 && w < a.rot / 16;
    const bool halves = r.turn && !a.interleaved;
    r.e0 = halves ? 8 * w : 16 * w;
    r.e1 = halves ? half + 8 * w : 16 * w + 8;
    r.pair = 8 * w;
    r.src = (r.kind <= 0 ? a.q + t * a.q_stride : (r.kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride)) +
            head * a.kv.dim;
    return r;
}

__device__ __forceinline__ Raw load_unit(const Unit& u) {
    Raw r{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (u.kind >= 0) {
        r.x = *reinterpret_cast<const uint4*>(u.src + u.e0);
        r.y = *reinterpret_cast<const uint4*>(u.src + u.e1);
    }
    return r;
}

__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    __shared__ float2 s_cs[64];
    __shared__ int s_seq, s_bad;                 // lowest sequence with this token; first one that does not fit
    const int t = blockIdx.x, tid = threadIdx.x;
    const int half = a.rot >> 1;
    pdl_wait();
    pdl_launch_dependents();
    if (tid == 0) s_seq = s_bad = a.sq.n;
    __syncthreads();
    for (int b = tid; b < a.sq.n; b += kRopeThreads) {
        const int c0 = a.sq.cu_q[b], c1 = a.sq.cu_q[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.sq.tokens)
            atomicMin(&s_bad, b);
        else if (t >= c0 && t < c1)
            atomicMin(&s_seq, b);
    }
    // the thread's first units are on their way while the angles are worked out
    const int D = a.kv.dim, per = D / 16, units = (a.q_heads + 2 * a.kv.heads) * per;
    const int step = gridDim.y * kRopeThreads;
    Unit un[kFlight];
    Raw raw[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
        un[k] = unit_of(a, t, blockIdx.y * kRopeThreads + tid + k * step, units, per, half);
        raw[k] = load_unit(un[k]);
    }
    if (tid < half) {
        const float pos = static_cast<float>(a.pos[t]);
        const float hi = a.freqs[2 * tid], lo = a.freqs[2 * tid + 1];
        const float p = __fmul_rn(pos, hi);
        const float e = __fmaf_rn(pos, lo, __fmaf_rn(pos, hi, -p));
        float sn, cs;
        sincospif(2.0f * __fadd_rn(p - rintf(p), e), &sn, &cs);
        s_cs[tid] = make_float2(cs * a.magnitude, sn * a.magnitude);
    }
    __syncthreads();
    // (from the first sequence on whose offsets do not fit, none has new tokens)
    const int b = s_seq < s_bad ? s_seq : -1;
    // this token's place in the cache; dst < 0: not stored
    int64_t dst = -1;
    bool lost = s_bad < a.sq.n;
    if (b >= 0) {
        const int64_t at = int64_t(a.sq.kv_len[b]) - a.sq.cu_q[b + 1] + t;
        if (at >= 0 && (at >> a.kv.page_log2) < a.sq.max_pages) {
            const int pg = a.sq.table[int64_t(b) * a.sq.max_pages + (at >> a.kv.page_log2)];
            if (pg >= 0 && pg < a.kv.n_pages)
                dst = pg * a.kv.page_stride + (at & (a.kv.page - 1)) * a.kv.token_stride;
        }
        lost = lost || (at >= 0 && dst < 0);
    }
    if (lost && tid == 0) record_error(a.err, MOE_ERR_INVALID_ARG);
    for (int u0 = blockIdx.y * kRopeThreads + tid;;) {
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const Unit& n = un[k];
            if (n.kind < 0) continue;
            Vec8 x = unpack8(raw[k].x), y = unpack8(raw[k].y);
            if (n.turn) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 c = s_cs[n.pair + i];
                    float* p1 = a.interleaved ? (i < 4 ? &x.v[2 * i] : &y.v[2 * i - 8]) : &x.v[i];
                    float* p2 = a.interleaved ? p1 + 1 : &y.v[i];
                    const float x1 = *p1, x2 = *p2;
                    *p1 = __fsub_rn(__fmul_rn(x1, c.x), __fmul_rn(x2, c.y));
                    *p2 = __fadd_rn(__fmul_rn(x2, c.x), __fmul_rn(x1, c.y));
                }
            }
            if (n.kind == 0) {
                uint16_t* o = a.q_out + t * a.out_stride + n.head * D;
                if (b < 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x.v[i] = y.v[i] = 0.0f;
                }
                store8_bf16(o + n.e0, x);
                store8_bf16(o + n.e1, y);
            } else if (dst >= 0) {
                const int64_t o = dst + n.head * a.kv.head_stride;
                uint8_t* base = n.kind == 1 ? a.kv.k : a.kv.v;
                if (a.kv.e4m3) {
                    const float sc = (n.kind == 1 ? a.kv.k_scale : a.kv.v_scale)[n.head];
                    store8_e4m3(base + o + n.e0, x, sc);
                    store8_e4m3(base + o + n.e1, y, sc);
                } else {
                    uint16_t* p = reinterpret_cast<uint16_t*>(base) + o;
                    store8_bf16(p + n.e0, x);
                    store8_bf16(p + n.e1, y);
                }
            }
        }
        u0 += kFlight * step;
        if (u0 >= units) break;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            un[k] = unit_of(a, t, u0 + k * step, units, per, half);
            raw[k] = load_unit(un[k]);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int n_sms, cudaStream_t s) {
    const int units = (a.q_heads + 2 * a.kv.heads) * (a.kv.dim / 16);
    int parts = n_sms / a.sq.tokens;                       // few tokens: a token's heads over several CTAs
    const int most = (units + kRopeThreads - 1) / kRopeThreads;
    parts = parts < 1 ? 1 : (parts > most ? most : parts);
    cudaError_t e = launch_pdl(rope_kernel, dim3(a.sq.tokens, parts), dim3(kRopeThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
