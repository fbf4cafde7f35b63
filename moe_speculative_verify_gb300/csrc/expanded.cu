// expanded.cu -- attention of the expanded form of a latent cache's layer
// (sm_103a): a head's key is a part of its own beside the rotary part that the
// heads share, its values have the own part's width.
//
// A warp takes a token's head, one pass over the keys with a running maximum
// and sum.
#include "attn.cuh"
#include "latent.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <int D>
__global__ void __launch_bounds__(kThreads) expanded_kernel(const ExpandedArgs x) {
    constexpr int kOwn = D / 32;
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 31;
    const int64_t u = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (u >= int64_t(a.sq.tokens) * a.q_heads) return;
    const int t = static_cast<int>(u / a.q_heads), h = static_cast<int>(u % a.q_heads);
    Seq s;
    int b = -1;
    for (int i = 0; i < a.sq.n; ++i) {
        bool fits;
        s = load_seq(a.sq, 1, i, a.err, &fits);
        if (!fits) break;
        if (t >= s.q0 && t < s.q0 + s.nq) {
            b = i;
            break;
        }
    }
    uint16_t* out = a.out + u * D;
    float o[kOwn] = {};
    float top = kNegInf, sum = 0.0f;
    if (b >= 0) {
        const uint16_t* q = a.q + t * a.q_stride + h * (D + kLatentRot);
        float qc[kOwn], qr[2];
        for (int i = 0; i < kOwn; ++i) qc[i] = bf16_bits_to_f32(q[lane + 32 * i]);
        for (int i = 0; i < 2; ++i) qr[i] = bf16_bits_to_f32(q[D + lane + 32 * i]);
        const RowView v = row_view(a, s, t - s.q0);
        const int k0 = x.cu_k[b];
        for (int j = max(v.lo, 0); j < v.hi; ++j) {
            float kx[kOwn] = {}, r[2] = {}, vx[kOwn] = {};
            const int64_t row = int64_t(k0) + j;
            if (row < 0 || row >= x.n_keys) {
                record_error(a.err, MOE_ERR_INVALID_ARG);
            } else {
                for (int i = 0; i < kOwn; ++i) {
                    kx[i] = bf16_bits_to_f32(x.k[row * x.k_token + h * x.k_head + lane + 32 * i]);
                    vx[i] = bf16_bits_to_f32(x.v[row * x.v_token + h * x.v_head + lane + 32 * i]);
                }
                for (int i = 0; i < 2; ++i) r[i] = bf16_bits_to_f32(x.rope[row * x.rope_token + lane + 32 * i]);
            }
            float d = qr[0] * r[0] + qr[1] * r[1];
            for (int i = 0; i < kOwn; ++i) d = fmaf(qc[i], kx[i], d);
            for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, k);
            const float z = d * a.scale * kLog2e;
            const float now = fmaxf(top, z);
            const float keep = top == kNegInf ? 0.0f : exp2f(top - now), p = now == kNegInf && z == z ? 0.0f : exp2f(z - now);
            sum = sum * keep + p;
            for (int i = 0; i < kOwn; ++i) o[i] = o[i] * keep + p * vx[i];
            top = now;
        }
    }
    const bool none = top == kNegInf && !(sum != sum);
    for (int i = 0; i < kOwn; ++i)
        out[lane + 32 * i] = static_cast<uint16_t>(pack_bf16(none ? 0.0f : o[i] / sum, 0.0f));
    if (lane == 0 && a.lse) a.lse[u] = none ? kNegInf : (top + log2f(sum)) * kLn2;
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, int n_sms, cudaStream_t s) {
    const int64_t warps = int64_t(a.a.sq.tokens) * a.a.q_heads;
    const dim3 grid(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
    cudaError_t e = a.dim == 128 ? launch_pdl(expanded_kernel<128>, grid, dim3(kThreads), 0, s, a)
                                 : launch_pdl(expanded_kernel<64>, grid, dim3(kThreads), 0, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
