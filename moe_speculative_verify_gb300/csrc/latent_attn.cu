// latent_attn.cu -- attention over a latent cache, absorbed form (sm_103a).
//
// With q in latent space, s_j = scale * (q_c . c_j + q_r . r_j) and the output
// is sum_j p_j c_j / sum_j p_j: a cached row serves as key and as value of every
// head.  A warp takes a token's head: lanes share the row's elements, one pass
// over the keys with a running maximum and sum.
#include "attn.cuh"
#include "latent.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

// The sequence of token t and its index there; b < 0: a pad row.
__device__ __forceinline__ int find_seq(const AttnArgs& a, int t, Seq& s) {
    for (int b = 0; b < a.sq.n; ++b) {
        bool fits;
        s = load_seq(a.sq, a.kv.page, b, a.err, &fits);
        if (!fits) return -1;
        if (t >= s.q0 && t < s.q0 + s.nq) return b;
    }
    return -1;
}

template <int C>
__global__ void __launch_bounds__(kThreads) latent_attn_kernel(const LatentAttnArgs la) {
    constexpr int kOwn = C / 32;
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31;
    const int64_t u = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (u >= int64_t(a.sq.tokens) * a.q_heads) return;
    const int t = static_cast<int>(u / a.q_heads), h = static_cast<int>(u % a.q_heads);
    Seq s;
    const int b = find_seq(a, t, s);
    uint16_t* out = a.out + u * C;
    float o[kOwn] = {};
    float top = kNegInf, sum = 0.0f;
    if (b >= 0) {
        const uint16_t* q = a.q + t * a.q_stride + h * (C + kLatentRot);
        float qc[kOwn], qr[2];
        for (int i = 0; i < kOwn; ++i) qc[i] = bf16_bits_to_f32(q[lane + 32 * i]);
        for (int i = 0; i < 2; ++i) qr[i] = bf16_bits_to_f32(q[C + lane + 32 * i]);
        const RowView v = row_view(a, s, t - s.q0);
        const bool draft = a.draft != nullptr;
        const float f = la.c.e4m3 ? pow2(la.c.scale_log2) : 1.0f;
        for (int j = max(v.lo, 0); j < v.hi; ++j) {
            if (!row_sees(v, draft, s.first, j)) continue;
            const int pg = a.sq.table[int64_t(b) * a.sq.max_pages + (j >> la.c.page_log2)];
            const int sl = j & (la.c.page - 1);
            float x[kOwn] = {}, r[2] = {};
            if (pg < 0 || pg >= la.c.n_pages) {
                record_error(a.err, MOE_ERR_INVALID_ARG);
            } else {
                const int64_t at = pg * la.c.lat_page + sl * la.c.lat_token;
                for (int i = 0; i < kOwn; ++i) {
                    if (la.c.e4m3) {
                        const uint32_t hw = e4m3x2_to_f16x2(la.c.latent[at + lane + 32 * i]);
                        x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(hw & 0xFFFFu))) * f;
                    } else {
                        x[i] = bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(la.c.latent)[at + lane + 32 * i]);
                    }
                }
                for (int i = 0; i < 2; ++i) r[i] = bf16_bits_to_f32(la.c.rope[pg * la.c.rope_page + sl * la.c.rope_token + lane + 32 * i]);
            }
            float d = qr[0] * r[0] + qr[1] * r[1];
            for (int i = 0; i < kOwn; ++i) d = fmaf(qc[i], x[i], d);
            for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, k);
            const float z = d * a.scale * kLog2e;
            const float now = fmaxf(top, z);
            const float keep = top == kNegInf ? 0.0f : exp2f(top - now), p = now == kNegInf && z == z ? 0.0f : exp2f(z - now);
            sum = sum * keep + p;
            for (int i = 0; i < kOwn; ++i) o[i] = o[i] * keep + p * x[i];
            top = now;
        }
    }
    const bool none = top == kNegInf && !(sum != sum);
    for (int i = 0; i < kOwn; ++i)
        out[lane + 32 * i] = static_cast<uint16_t>(pack_bf16(none ? 0.0f : o[i] / sum, 0.0f));
    if (lane == 0 && a.lse) a.lse[u] = none ? kNegInf : (top + log2f(sum)) * kLn2;
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnArgs& a, int n_sms, cudaStream_t s) {
    const int64_t warps = int64_t(a.a.sq.tokens) * a.a.q_heads;
    const dim3 grid(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cudaError_t e = a.c.dim == 512 ? launch_pdl(latent_attn_kernel<512>, grid, dim3(kThreads), 0, s, a)
                                   : launch_pdl(latent_attn_kernel<256>, grid, dim3(kThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
