// pair.cuh -- what the kernels that work in pairs of SMs share (latent_attn.cu,
// expanded.cu): cluster barriers, tcgen05 forms of a pair of CTAs, and the join of
// items that several pairs worked on.
#pragma once

#include "attn_mma.cuh"
#include "latent.h"

namespace moe {

// --------------------------------------------------------------- cluster ----
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrives on the barrier at this address of the pair's first CTA.  What was written
// before lies in this CTA's shared memory and is read by its own tensor core, so the
// CTA's order does; a release to the cluster would wait for memory (1000 to 2500
// clocks, a third of a tile's time).
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// All 512 columns of tensor memory, by a warp of each CTA.
__device__ __forceinline__ void pair_alloc(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(512) : "memory");
}

// One step (K = 16) of D[tmem] (+)= A B^T of the pair, A and B in both CTAs' shared
// memory at the same offsets.
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// The same with A in tensor memory, at the same columns of both CTAs.
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// Arrives on the barrier at this address of both CTAs once the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Joins the pieces of the split items, out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k
// in pair order.  Slots have ROWS rows of C columns.  A thread has four columns of a row, kBatch pieces of them in flight; a
// warp has eight rows, which are a line of the pieces' layout, by four such columns, a
// sector of the output.  (Rows as units of whole blocks, the pieces shared out among
// their threads: 76 us behind a chunk whose 76 pairs share 40 MB, 17 now.)
constexpr int kJoinRows = 8, kJoinThreads = 512;

template <int C, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, 2) pair_join_kernel(const AttnArgs a, int n_notes) {
    constexpr int64_t kSlot = ROWS * (C + 2);
    constexpr int kBatch = 4, kUnit = kJoinRows * C / 4;         // threads' work of eight rows
    __shared__ SplitNote s_note[kMaxPairs];
    __shared__ int s_end[128];                                   // units up to note i, inclusive
    static_assert(kMaxPairs <= 128, "four notes a lane");
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < n_notes; i += kJoinThreads) s_note[i] = a.notes[i];
    __syncthreads();
    if (threadIdx.x < 32) {
        int u[4], sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = threadIdx.x * 4 + k;
            u[k] = i < n_notes && s_note[i].pieces > 0 ? (s_note[i].rows + kJoinRows - 1) / kJoinRows : 0;
            sum += u[k];
        }
        int before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (threadIdx.x >= d) before += o;
        }
        before -= sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) s_end[threadIdx.x * 4 + k] = before += u[k];
    }
    __syncthreads();
    const int total = s_end[127] * kUnit;
    for (int w = blockIdx.x * kJoinThreads + threadIdx.x; w < total; w += gridDim.x * kJoinThreads) {
        const int u = w / kUnit, cell = w - u * kUnit;
        int i = 0;
#pragma unroll
        for (int step = 64; step > 0; step >>= 1)
            if (s_end[i + step - 1] <= u) i += step;
        const SplitNote& n = s_note[i];
        const int row = (u - (i > 0 ? s_end[i - 1] : 0)) * kJoinRows + cell % kJoinRows, d4 = cell / kJoinRows;
        if (row >= n.rows) continue;
        // the piece of the pair where the item begins, and (k >= 1) of the k-th pair after it
        const float* head = a.partials + int64_t(i) * kSlot;
        const float* rest = a.partials + (int64_t(kMaxPairs) + i) * kSlot;
        const int ml = ROWS * C + 2 * row, od = (d4 * ROWS + row) * 4, pieces = n.pieces;
        float top = kNegInf, sum = 0.0f;
        float4 s = make_float4(0, 0, 0, 0);
        for (int k0 = 0; k0 < pieces; k0 += kBatch) {
            float2 x[kBatch];
            float4 y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int k = k0 + j;
                const float* p = k == 0 ? head : rest + k * kSlot;
                x[j] = make_float2(kNegInf, 0.0f);
                y[j] = make_float4(0, 0, 0, 0);
                if (k < pieces) {
                    x[j] = *reinterpret_cast<const float2*>(p + ml);
                    y[j] = *reinterpret_cast<const float4*>(p + od);
                }
            }
            float now = top;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) now = fmaxf(now, x[j].x);
            const float ref = now == kNegInf ? 0.0f : now, keep = fast_exp2(top - ref);
            sum *= keep;
            s = make_float4(s.x * keep, s.y * keep, s.z * keep, s.w * keep);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float f = fast_exp2(x[j].x - ref);
                sum = fmaf(x[j].y, f, sum);
                s.x = fmaf(y[j].x, f, s.x);
                s.y = fmaf(y[j].y, f, s.y);
                s.z = fmaf(y[j].z, f, s.z);
                s.w = fmaf(y[j].w, f, s.w);
            }
            top = now;
        }
        const int r = n.row0 + row, q = a.query_of(r), hd = n.head * a.group + r - q * a.group;
        const int64_t at = int64_t(n.q0 + q) * a.q_heads + hd;
        if (top == kNegInf) s = make_float4(0, 0, 0, 0);             // no key has weight, whatever its values
        const float inv = top == kNegInf ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint2*>(a.out + at * C + 4 * d4) = make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
        if (d4 == 0 && a.lse) a.lse[at] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
    }
}

template <int C, int ROWS>
cudaError_t launch_pair_join(const AttnArgs& a, int pairs, int n_sms, cudaStream_t s) {
    cudaError_t e = launch_pdl(pair_join_kernel<C, ROWS>, dim3(2 * n_sms), dim3(kJoinThreads), 0, s, a, pairs);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
