// attn.cuh -- device helpers shared by the attention-side kernels: the
// sequences' numbers made safe, which keys a row sees, and the 16-bit matrix
// instruction on registers.
#pragma once

#include <cuda_fp16.h>

#include "attn.h"
#include "common.cuh"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -INFINITY;

// One sequence: its first row of the step's tensors, new tokens, cached keys
// and the cache place of its first new token.  Numbers that do not fit are
// cut to what does, and recorded.  Rows go by the offsets up to the first pair
// that does not fit: from that sequence on none has new tokens (a later offset
// could claim rows of an earlier sequence); `fits` is that sequence's.
struct Seq {
    int q0, nq, len, first;
};

__device__ __forceinline__ Seq load_seq(const SeqArgs& s, int page, int b, int32_t* err, bool* fits = nullptr) {
    const int c0 = s.cu_q[b], c1 = s.cu_q[b + 1], len = s.kv_len[b];
    Seq r;
    r.q0 = c0;
    r.nq = c1 - c0;
    const bool bad_q = c0 < 0 || c1 < c0 || c1 > s.tokens;
    if (bad_q) {
        r.q0 = 0;
        r.nq = 0;
    }
    const int64_t cap = min(int64_t(s.max_pages) * page, int64_t(MOE_MAX_KV_LEN));
    r.len = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
    r.first = r.len - r.nq;
    if (bad_q || r.len != len) record_error(err, MOE_ERR_INVALID_ARG);
    if (fits) *fits = !bad_q;
    return r;
}

// The keys that row i of a sequence can see: [lo, hi), and among the new keys
// (from `first` on) those of its draft mask.
struct RowView {
    int lo, hi;
    uint64_t draft;
};

__device__ __forceinline__ RowView row_view(const AttnArgs& a, const Seq& s, int i) {
    RowView r;
    r.hi = s.len;
    r.draft = ~0ull;
    if (a.draft)
        r.draft = a.draft[s.q0 + i];
    else if (a.causal)
        r.hi = min(s.len, s.first + i + 1);
    r.lo = a.window > 0 ? max(0, s.first + i - a.window + 1) : 0;
    return r;
}

__device__ __forceinline__ bool row_sees(const RowView& r, bool draft, int first, int j) {
    bool ok = j >= r.lo && j < r.hi;
    if (draft) {
        const int c = j - first;
        ok = ok && (c < 0 || (c < 64 && ((r.draft >> (c & 63)) & 1ull)));
    }
    return ok;
}

// row_sees() of the 32 keys from k0 on, key k0 + e at bit e.
__device__ __forceinline__ uint32_t row_bits(const RowView& r, bool draft, int first, int k0) {
    const int lo = min(max(r.lo - k0, 0), 32), hi = min(max(r.hi - k0, 0), 32);
    uint32_t bits = lo >= hi ? 0u : (0xFFFFFFFFu << lo) & (0xFFFFFFFFu >> (32 - hi));
    if (draft) {
        const int d = first - k0;                 // bit of the first new key
        if (d <= 0)
            bits &= -d >= 64 ? 0u : static_cast<uint32_t>(r.draft >> -d);
        else if (d < 32)
            bits &= static_cast<uint32_t>(r.draft << d) | ((1u << d) - 1u);
    }
    return bits;
}

// Keys that some row of the rows i0 .. i1 of a sequence can see, as a range.
__device__ __forceinline__ int2 rows_range(const AttnArgs& a, const Seq& s, int i0, int i1) {
    int hi = s.len;
    if (a.draft)
        hi = min(s.len, max(s.first, 0) + 64);
    else if (a.causal)
        hi = min(s.len, s.first + i1 + 1);
    const int lo = a.window > 0 ? max(0, s.first + i0 - a.window + 1) : 0;
    return make_int2(lo, max(hi, 0));
}

// Keys that every one of those rows sees, as a range.
__device__ __forceinline__ int2 rows_whole(const AttnArgs& a, const Seq& s, int i0, int i1) {
    int hi = s.len;
    if (a.draft)
        hi = min(hi, s.first);
    else if (a.causal)
        hi = min(hi, s.first + i0 + 1);
    return make_int2(a.window > 0 ? s.first + i1 - a.window + 1 : 0, hi);
}

// Whether every key of [j0, j1) is seen by every one of those rows.
__device__ __forceinline__ bool rows_see_all(const AttnArgs& a, const Seq& s, int i0, int i1,
                                             int j0, int j1) {
    const int2 w = rows_whole(a, s, i0, i1);
    return j0 >= w.x && j1 <= w.y;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (d0, d1) = (a0, a1) * b + c, and (d0, d1) += (a0, a1), as one packed
// instruction each, rounded as the scalar ones.
__device__ __forceinline__ void fma2_to(float& d0, float& d1, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
        "mov.b64 pa, {%2, %3};\n\t"
        "mov.b64 pb, {%4, %4};\n\t"
        "mov.b64 pc, {%5, %5};\n\t"
        "fma.rn.f32x2 pc, pa, pb, pc;\n\t"
        "mov.b64 {%0, %1}, pc;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

__device__ __forceinline__ void fma2_off(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
        "mov.b64 pa, {%2, %3};\n\t"
        "mov.b64 pb, {%4, %4};\n\t"
        "mov.b64 pc, {%5, %6};\n\t"
        "fma.rn.f32x2 pc, pa, pb, pc;\n\t"
        "mov.b64 {%0, %1}, pc;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n\t.reg .b64 pa, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\t"
        "mov.b64 pd, {%0, %1};\n\t"
        "add.rn.f32x2 pd, pd, pa;\n\t"
        "mov.b64 {%0, %1}, pd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// Two fp32 as bf16x2 / f16x2, `lo` in the low half, nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low 16 bits) as f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(r)
        : "r"(codes));
    return r;
}

// Four e4m3 codes as bf16 pairs, exactly, without the conversion unit (which
// the powers need): a code's exponent and fraction bits moved to where bf16
// has them give the value times 2^-120, subnormals included.  NaN codes come
// out as +-480, which no other code does: `most` keeps the largest bits of two
// columns of codes for e4m3_had_nan, and e4m3_nan_again puts them right.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t codes, uint32_t& lo, uint32_t& hi, uint32_t& most) {
    const uint32_t a = __byte_perm(codes, 0, 0x1404), b = __byte_perm(codes, 0, 0x3424);
    const uint32_t ma = (a >> 4) & 0x07F007F0u, mb = (b >> 4) & 0x07F007F0u;
    constexpr uint32_t k2p120 = 0x7B807B80u;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(ma | (a & 0x80008000u)), "r"(k2p120));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(mb | (b & 0x80008000u)), "r"(k2p120));
    asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(ma));
    asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(mb));
}

__device__ __forceinline__ bool e4m3_had_nan(uint32_t most) { return ((most + 0x00100010u) & 0x08000800u) != 0u; }

// A pair of those results with +-480 as NaN.
__device__ __forceinline__ uint32_t e4m3_nan_again(uint32_t pair) {
    if ((pair & 0x7FFFu) == 0x43F0u) pair |= 0x7FC0u;
    if ((pair & 0x7FFF0000u) == 0x43F00000u) pair |= 0x7FC00000u;
    return pair;
}

// D[16x8] += A[16x16] B[16x8]: bf16 or f16 operands, fp32 sums.  Lane l = 4g+t
// holds A rows g, g+8 at columns 2t,2t+1 (a0, a1) and 2t+8,2t+9 (a2, a3), B
// column g at rows 2t,2t+1 (b0) and 2t+8,2t+9 (b1), D rows g (d0, d1) and g+8
// (d2, d3) at columns 2t, 2t+1.
template <bool F16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that takes a bf16 query row's largest element to [2^14,
// 2^15), near the end of f16 (or as near as fp32 has it), where the row
// multiplies e4m3 codes: elements keep their 8 bits down to 2^-31 of the
// largest, and below it err by at most 2^-39 of it.  Non-finite rows stay as
// they are.
__device__ __forceinline__ float pow2_norm(float amax) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23);
    return e == 255 ? 1.0f : __uint_as_float(static_cast<uint32_t>(min(268 - e, 253)) << 23);
}

// 4-D tiled bulk tensor load global -> shared; c0 (innermost, elements) starts
// on a 16-byte boundary.  A coordinate out of range reads as zeros.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
        "r"(c3)
        : "memory");
}

// Same, 3-D.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// A CTA ends after its copies and products, also where a wait ran out (they
// would write into shared or tensor memory that is no longer its own).  The waits
// for that have a limit of their own, far above what a copy or a burst of products
// takes, whatever the caller's limit is; they end at once unless the GPU has
// stopped answering.  A stage is given back only by a thread that saw it full: a
// second copy into one whose first is still in flight would count into the
// first one's phase.
constexpr uint64_t kDrainNs = 2000000000ull;

// A wait of a whole warp whose lanes go on or stop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* err, uint64_t timeout_ns) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, err, timeout_ns));
}

// ------------------------------------------------------------ work split ----
// The attention kernels cut a call into items -- (sequence, kv head, tile of
// MT query rows), rows r = i * group + g -- of one unit per KT-key tile that
// some row of the item sees (one unit when none does), and give every CTA an
// equal run of units in item order.  A CTA so meets at most two items that
// it shares with its neighbours: it leaves its pieces of those in its two
// slots (one for an item that begins with it, one for an item that began
// before), the CTA where an item begins notes the split, and the join kernel (attn.cu) adds an item's
// pieces up in CTA order.
struct Item {
    int b, h, rt;          // sequence, kv head, row tile
    int lo, hi;            // keys some row sees
    int tile0, n;          // first key tile, units
    int t0, t1;            // this CTA's units of it
    int64_t u;             // global index of its first unit
    Seq s;
};

template <int MT, int KT>
struct Work {
    __device__ __forceinline__ static int row_tiles(const AttnArgs& a, const Seq& s) {
        return (s.nq * a.group + MT - 1) / MT;
    }
    // keys and units of row tile rt
    __device__ __forceinline__ static void extent(const AttnArgs& a, const Seq& s, int rt, int& lo,
                                                  int& hi, int& tile0, int& n) {
        const int r1 = min(s.nq * a.group, (rt + 1) * MT) - 1;
        const int2 k = rows_range(a, s, a.query_of(rt * MT), a.query_of(r1));
        lo = k.x;
        hi = k.y;
        tile0 = lo / KT;
        n = max(1, (hi + KT - 1) / KT - tile0);
        if (hi <= lo) n = 1;
    }
    __device__ __forceinline__ static int64_t head_units(const AttnArgs& a, const Seq& s) {
        const int rts = row_tiles(a, s);
        int64_t u = 0;
        for (int rt = 0; rt < rts; ++rt) {
            int lo, hi, t0, n;
            extent(a, s, rt, lo, hi, t0, n);
            u += n;
        }
        return u;
    }
};

// a / b for 0 <= a, 0 < b, by the 32-bit division where that does.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// What a CTA knows of the call's split once plan_work() has run: CTA c of
// `ctas` takes `share` units, the first `extra` CTAs one more.
struct Plan {
    int64_t u0, u1;        // this CTA's units
    int64_t share, extra;
    int64_t off;           // unit u0 lies `off` units into row tile rt of head h of sequence b
    int b, h, rt;
    int ctas;              // CTAs that take part
    int seqs;              // sequences with rows: those before the first whose offsets do not fit

    __device__ __forceinline__ int owner(int64_t u) const {
        const int64_t head = extra * (share + 1);
        return static_cast<int>(u < head ? div64(u, share + 1) : extra + div64(u - head, share));
    }
};

// All threads of the block.  s_warp: one int64 per warp, s_plan: shared.
template <int MT, int KT>
__device__ __forceinline__ void plan_work(const AttnArgs& a, int min_units, int64_t* s_warp,
                                          Plan* s_plan) {
    using W = Work<MT, KT>;
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wid = tid >> 5;
    const int per = (a.sq.n + nt - 1) / nt;
    int seqs = a.sq.n, b0;
    int64_t mine, head = 0, incl;              // units of the thread's sequences, of a head of the last one
    for (;;) {
        b0 = min(seqs, tid * per);
        const int b1 = min(seqs, b0 + per);
        bool fits = true;
        int bad = b1;
        mine = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            head = W::head_units(a, load_seq(a.sq, a.kv.page, b, a.err, &fits));
            mine += a.kv.heads * head;
            if (!fits) {
                bad = b;
                break;
            }
        }
        incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) s_warp[wid] = incl;
        if (!__syncthreads_or(!fits)) break;
        // once more, with the sequences before the first one that does not fit
        if (tid == 0) s_plan->seqs = seqs;
        __syncthreads();
        if (!fits) atomicMin(&s_plan->seqs, bad);
        __syncthreads();
        seqs = s_plan->seqs;
    }
    int64_t before = 0, total = 0;
    for (int w = 0; w < (nt >> 5); ++w) {
        const int64_t v = s_warp[w];
        before += w < wid ? v : 0;
        total += v;
    }
    const int64_t want = div64(total + min_units - 1, min_units);
    const int C = static_cast<int>(want < int64_t(gridDim.x) ? (want > 0 ? want : 1) : gridDim.x);
    const int c = blockIdx.x;
    const int64_t share = div64(total, C), extra = total - share * C;
    const int64_t u0 = c < C ? c * share + min(int64_t(c), extra) : total;
    const int64_t u1 = c < C ? u0 + share + (c < extra ? 1 : 0) : total;
    if (tid == 0) {
        s_plan->u0 = u0;
        s_plan->u1 = u1;
        s_plan->share = share;
        s_plan->extra = extra;
        s_plan->ctas = C;
        s_plan->seqs = seqs;
        a.notes[c].pieces = 0;
    }
    const int64_t pre = before + incl - mine;
    if (u0 < u1 && pre <= u0 && u0 < pre + mine) {
        int64_t off = u0 - pre;
        int b = b0;
        Seq s = load_seq(a.sq, a.kv.page, b, nullptr);
        if (per > 1) {
#pragma unroll 1
            for (;;) {
                head = W::head_units(a, s);
                if (off < a.kv.heads * head) break;
                off -= a.kv.heads * head;
                s = load_seq(a.sq, a.kv.page, ++b, nullptr);
            }
        }
        const int h = static_cast<int>(div64(off, head));
        off -= h * head;
        int rt = 0;
#pragma unroll 1
        for (;; ++rt) {
            int lo, hi, t0, n;
            W::extent(a, s, rt, lo, hi, t0, n);
            if (off < n) break;
            off -= n;
        }
        s_plan->b = b;
        s_plan->h = h;
        s_plan->rt = rt;
        s_plan->off = off;
    }
    __syncthreads();
}

// Walks a CTA's units item by item; every warp keeps its own copy.
template <int MT, int KT>
struct Walk {
    using W = Work<MT, KT>;
    Seq s;
    int b, h, rt, rts;
    int64_t off, u, left;      // units to skip in the first item, next unit, units left

    __device__ __forceinline__ void start(const AttnArgs& a, const Plan& p) {
        left = p.u1 - p.u0;
        u = p.u0;
        b = h = rt = rts = 0;
        off = 0;
        if (left <= 0) return;
        b = p.b;
        h = p.h;
        rt = p.rt;
        off = p.off;
        s = load_seq(a.sq, a.kv.page, b, nullptr);
        rts = W::row_tiles(a, s);
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, Item& it) {
        if (left <= 0) return false;
        while (rt >= rts) {
            rt = 0;
            if (++h >= a.kv.heads || rts == 0) {
                h = 0;
                if (++b >= a.sq.n) return false;
                s = load_seq(a.sq, a.kv.page, b, nullptr);
                rts = W::row_tiles(a, s);
            }
        }
        W::extent(a, s, rt, it.lo, it.hi, it.tile0, it.n);
        it.s = s;
        it.b = b;
        it.h = h;
        it.rt = rt;
        it.t0 = static_cast<int>(off);
        it.t1 = static_cast<int>(left < it.n - off ? off + left : it.n);
        it.u = u - off;
        u += it.t1 - it.t0;
        left -= it.t1 - it.t0;
        off = 0;
        ++rt;
        return true;
    }
};

// One thread, for each item of the CTA: notes the split item that begins here.
__device__ __forceinline__ void note_split(const AttnArgs& a, const Item& it, int rows, int mt, const Plan& p) {
    if (it.t0 != 0 || it.t1 >= it.n) return;
    // the last item of the CTA's run, so its note is not written over
    SplitNote n;
    n.pieces = p.owner(it.u + it.n - 1) - static_cast<int>(blockIdx.x) + 1;
    n.rows = rows;
    n.row0 = it.rt * mt;
    n.q0 = it.s.q0;
    n.head = it.h;
    a.notes[blockIdx.x] = n;
}

// Zeroes the output rows that belong to no sequence: those before and after
// the rows of the sequences that fit, which follow one another.
__device__ __forceinline__ void zero_pad_rows(const AttnArgs& a, int seqs) {
    const int first = seqs > 0 ? a.sq.cu_q[0] : a.sq.tokens, last = seqs > 0 ? a.sq.cu_q[seqs] : a.sq.tokens;
    const int n = first + (a.sq.tokens - last);
    for (int p = blockIdx.x; p < n; p += gridDim.x) {
        const int64_t t = p < first ? p : last + (p - first);
        uint4* o = reinterpret_cast<uint4*>(a.out + t * a.q_heads * a.kv.dim);
        for (int i = threadIdx.x; i < a.q_heads * a.kv.dim / 8; i += blockDim.x)
            o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = threadIdx.x; i < a.q_heads; i += blockDim.x)
                a.lse[t * a.q_heads + i] = kNegInf;
    }
}

}  // namespace moe
