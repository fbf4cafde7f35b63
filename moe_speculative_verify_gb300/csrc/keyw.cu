// keyw.cu -- the attention weight that each cached key received in a step,
// added to the running scores that eviction goes by (sm_103a).
//
// w_j = sum over the rows that see key j of 2^(c q.k_j - lse log2 e).  A unit
// is 64 keys of one sequence and kv head; its CTA holds their K rows in
// registers as matrix fragments and passes over every row that sees them, so
// K is read once, each key's sum is one CTA's, and no atomics are needed.
#include "attn.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kKeys = 64;                  // keys of a unit: 16 a warp
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// 16-bit fragments of one 16-column step, two per 16 bytes of bf16 (32
// columns, lane t of a quad the columns 8t..8t+7) and four per 16 e4m3 codes
// (64 columns, 16t..16t+15): the k index is permuted alike on both sides.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) keyw_kernel(const KeywArgs ka) {
    extern __shared__ int64_t s_pre[];     // units before sequence b
    __shared__ int64_t s_warp[kWarps];
    const AttnArgs& a = ka.a;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_launch_dependents();
    const int per = (a.sq.n + kThreads - 1) / kThreads;
    const int b0 = min(a.sq.n, tid * per), b1 = min(a.sq.n, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
        s_pre[b + 1] = mine;
        mine += int64_t(a.kv.heads) * ((load_seq(a.sq, a.kv.page, b, a.err).len + kKeys - 1) / kKeys);
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) s_warp[wid] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < wid) before += s_warp[w];
        total += s_warp[w];
    }
    for (int b = b0; b < b1; ++b) s_pre[b + 1] += before;   // units before sequence b, at b + 1
    __syncthreads();

    const bool draft = a.draft != nullptr;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        // the last sequence whose first unit is at or before u (it has units)
        int lo = 0, hi = a.sq.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_pre[mid + 1] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int b = lo;
        const Seq s = load_seq(a.sq, a.kv.page, b, nullptr);
        const int tiles = (s.len + kKeys - 1) / kKeys;
        const int in = static_cast<int>(u - s_pre[b + 1]);
        const int h = in / tiles, j0 = (in - h * tiles) * kKeys;
        // --- this warp's 16 K rows
        const int32_t* table = a.sq.table + int64_t(b) * a.sq.max_pages;
        uint4 kf[2][E4M3 ? D / 64 : D / 32];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = j0 + 16 * wid + 8 * n + g;
            int pg = -1;
            if (j < s.len) {
                pg = table[j >> a.kv.page_log2];
                if (pg < 0 || pg >= a.kv.n_pages) {
                    pg = -1;
                    record_error(a.err, MOE_ERR_INVALID_ARG);
                }
            }
            const int64_t at = pg * a.kv.page_stride + h * a.kv.head_stride +
                               (j & (a.kv.page - 1)) * a.kv.token_stride;
#pragma unroll
            for (int c = 0; c < (E4M3 ? D / 64 : D / 32); ++c) {
                const uint8_t* src = E4M3 ? a.kv.k + at + 64 * c + 16 * t
                                          : a.kv.k + 2 * (at + 32 * c + 8 * t);
                kf[n][c] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
            }
        }
        const float ck = a.scale * kLog2e * (E4M3 ? a.kv.k_scale[h] : 1.0f);
        float w[2][2] = {};
        const int rows = s.nq * a.group;
        const int j1 = min(j0 + kKeys, s.len);
        int rt0 = 0;                       // causal: rows before the unit's first key see none of it
        if (!draft && a.causal && j0 > s.first) rt0 = (j0 - s.first) * a.group / 16;
        for (int rt = rt0; rt * 16 < rows; ++rt) {
            const int rl = min(rows, rt * 16 + 16) - 1, i0 = rt * 16 / a.group, i1 = rl / a.group;
            const int2 range = rows_range(a, s, i0, i1);
            if (range.x >= j1) break;      // window: later rows are further right still
            if (range.y <= j0) continue;
            const bool whole = rows_see_all(a, s, i0, i1, j0, j0 + kKeys);
            RowView view[2];
            float c[2], off[2];
            uint4 qf[2][D / 32];
            bool live[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rt * 16 + g + 8 * r;
                live[r] = row < rows;
                const int i = live[r] ? row / a.group : 0;
                const int hd = h * a.group + (live[r] ? row - i * a.group : 0);
                const uint16_t* src = a.q + (s.q0 + i) * a.q_stride + hd * D;
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    qf[r][k] = live[r] ? __ldg(reinterpret_cast<const uint4*>(
                                             src + (E4M3 ? 64 * (k >> 1) + 16 * t + 8 * (k & 1) : 32 * k + 8 * t)))
                                       : make_uint4(0, 0, 0, 0);
                const float z = live[r] ? a.lse[int64_t(s.q0 + i) * a.q_heads + hd] : kNegInf;
                if (fabsf(z) == INFINITY) live[r] = false;
                off[r] = z * kLog2e;
                view[r] = RowView{0, 0, 0ull};
                if (live[r] && !whole) view[r] = row_view(a, s, i);
                c[r] = ck;
            }
            if constexpr (E4M3) {          // f16 beside the codes: see pow2_norm
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t* x = reinterpret_cast<uint32_t*>(qf[r]);
                    float amax = 0.0f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16_bits_to_f32(x[k] & 0xFFFFu)),
                                                 fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                    const float f = pow2_norm(amax);
                    c[r] = ck / f;
#pragma unroll
                    for (int k = 0; k < D / 8; ++k)
                        x[k] = pack_f16(bf16_bits_to_f32(x[k] & 0xFFFFu) * f,
                                        __uint_as_float(x[k] & 0xFFFF0000u) * f);
                }
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float d[4] = {};
                if constexpr (!E4M3) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        mma16<false>(d, qf[0][k].x, qf[1][k].x, qf[0][k].y, qf[1][k].y, kf[n][k].x, kf[n][k].y);
                        mma16<false>(d, qf[0][k].z, qf[1][k].z, qf[0][k].w, qf[1][k].w, kf[n][k].z, kf[n][k].w);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const uint32_t ww[4] = {kf[n][k].x, kf[n][k].y, kf[n][k].z, kf[n][k].w};
                        const uint32_t q0[8] = {qf[0][2 * k].x, qf[0][2 * k].y, qf[0][2 * k].z, qf[0][2 * k].w,
                                                qf[0][2 * k + 1].x, qf[0][2 * k + 1].y, qf[0][2 * k + 1].z, qf[0][2 * k + 1].w};
                        const uint32_t q1[8] = {qf[1][2 * k].x, qf[1][2 * k].y, qf[1][2 * k].z, qf[1][2 * k].w,
                                                qf[1][2 * k + 1].x, qf[1][2 * k + 1].y, qf[1][2 * k + 1].z, qf[1][2 * k + 1].w};
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4)
                            mma16<true>(d, q0[2 * k4], q1[2 * k4], q0[2 * k4 + 1], q1[2 * k4 + 1],
                                        e4m3x2_to_f16x2(ww[k4] & 0xFFFFu), e4m3x2_to_f16x2(ww[k4] >> 16));
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = k >> 1, j = j0 + 16 * wid + 8 * n + 2 * t + (k & 1);
                    const bool see = live[r] && (whole || row_sees(view[r], draft, s.first, j));
                    w[n][k & 1] += see ? fast_exp2(fmaf(d[k], c[r], -off[r])) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = w[n][e];
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
                const int j = j0 + 16 * wid + 8 * n + 2 * t + e;
                if (g == 0 && j < s.len && j < ka.score_stride) {
                    const int64_t at = (int64_t(b) * a.kv.heads + h) * ka.score_stride + j;
                    ka.scores_out[at] = x + (j < s.first ? ka.decay * ka.scores[at] : 0.0f);
                }
            }
    }
}

template <int D, bool E4M3>
cudaError_t launch(const KeywArgs& a, int n_sms, cudaStream_t s) {
    const size_t smem = sizeof(int64_t) * (a.a.sq.n + 1);
    const cudaError_t e = launch_pdl(keyw_kernel<D, E4M3>, dim3(4 * n_sms), dim3(kThreads), smem, s, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_keyw(const KeywArgs& a, int n_sms, cudaStream_t s) {
    if (a.a.kv.dim == 128) return a.a.kv.e4m3 ? launch<128, true>(a, n_sms, s) : launch<128, false>(a, n_sms, s);
    return a.a.kv.e4m3 ? launch<64, true>(a, n_sms, s) : launch<64, false>(a, n_sms, s);
}

}  // namespace moe
