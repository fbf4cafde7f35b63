// attn.cu -- attention of the step's new tokens over the paged cache (sm_103a):
// the kernel for few query rows a kv head (single tokens; attn_tile.cu is the
// one for more).
//
// out_i = sum_j p_ij v_j / sum_j p_ij with p_ij = 2^(c (s_ij) - m_i), m_i the
// running row maximum: one pass over K and V, with the sums rescaled when the
// maximum grows.
//
// Few rows per kv head read each K and V row once for 2 * rows flops a byte:
// bound by HBM.  So the kernel is a stream: one producer warp keeps a ring of
// 64-key K and V tiles in flight with TMA (a page or half a page per box),
// eight warps take 16 keys each of two alternating tiles and keep their own
// maximum, sum and 16 x D sums in registers, with no exchange between warps
// until an item ends.  The key axis is cut into equal runs over all SMs
// (attn.cuh), so lengths of 1 : 1000 in a batch load them alike.
//
// Measured (8 kv heads of 8 query heads of 128, bf16): 48 single tokens over
// 251 to 32,011 keys 241 us, 5.9 TB/s of a copy's 6.7 (over e4m3 281, 2.5 TB/s:
// the conversions to f16); one over 60,000 keys 53 us (4.6 TB/s), over 6,011 20.8
// and over 8 keys 9.6: a fixed cost of the plan, an item's start and end and
// the join's launch.
#include "attn.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRows = 16;                   // query rows of an item
constexpr int kTile = kAttnTile;            // keys of a tile
constexpr int kConsumers = 8;               // warps; four to a tile
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kBarMerge = 1;                // named barrier of the consumer warps

// e4m3: f16 probabilities at 2^15 times their share of a warp's largest, near the
// end of f16: 8 bits down to 2^-32 of it, some down to 2^-39.  (bf16 ones, which
// have no such end, need bf16 codes, four times the instructions of f16 ones in a
// kernel that they bound.)
template <bool E4M3>
constexpr float kBias = E4M3 ? 15.0f : 0.0f;

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kRowBytes = E4M3 ? D : 2 * D;
    static constexpr int kTileBytes = kTile * kRowBytes;
    // Even, so that a stage always serves the same group of warps: a warp
    // waits for every use of its stages in turn, and one that skipped a use
    // would take the phase before it for its own (parities repeat every two).
    static constexpr int kStages = kTileBytes >= 16384 ? 6 : 10;
    static_assert(kStages % 2 == 0, "two groups take tiles in turn");
    static constexpr int kRing = 2 * kTileBytes * kStages;
    static constexpr int kMergeFloats = 4 * kRows * D;
    static constexpr size_t kSmem = 1024 + kRing + kMergeFloats * 4;
};

constexpr int kItems = 4;                    // items handed on ahead

struct Shared {
    alignas(16) Item item[kItems];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t full[10];
    uint64_t empty[10];
    int64_t warp_sum[kConsumers + 1];
    Plan plan;
    float2 ml[kConsumers][kRows];            // maximum (log2) and sum of a warp's keys
};

// The TMA warp.  It walks the CTA's items and hands them to the other warps,
// which so need not look up sequences themselves, and prefetches their rows.
// A step is a key tile, K and V, a box or two a page, each page issued by a
// lane of its own, one after the other; the next tile's page indices are read
// a step ahead.
template <int D, bool E4M3>
__device__ __forceinline__ void produce(const AttnArgs& a, const KvMaps& maps, Shared& sh, uint8_t* ring) {
    using C = Cfg<D, E4M3>;
    constexpr int kBox = E4M3 ? D : 64, kBoxBytes = E4M3 ? D : 128, kParts = D / kBox;
    const int lane = threadIdx.x & 31;
    const int page = a.kv.page, pl = a.kv.page_log2, n_pages = a.kv.n_pages;
    const int rows = page < kTile ? page : kTile;       // tokens of a box
    const int np = kTile / rows;                        // pages of a tile
    uint8_t* box = ring + lane * rows * kBoxBytes;
    Walk<kRows, kTile> wk;
    wk.start(a, sh.plan);
    Item it;
    int st = 0, slot = 0;
    uint32_t ph = 1, ip = 1;
    bool dead = false, more = true;
    while (more && !dead) {
        more = wk.next(a, it);
        if (!more) it.b = -1;
        // (after a wait that ran out nothing is handed on: the slot may still be read)
        if (!warp_wait(&sh.item_empty[slot], ip, a.err, a.timeout_ns)) break;
        if (lane == 0) {
            sh.item[slot] = it;
            mbar_arrive(&sh.item_full[slot]);
        }
        __syncwarp();
        if (++slot == kItems) {
            slot = 0;
            ip ^= 1;
        }
        if (!more) break;
        {
            const int r = it.rt * kRows + (lane & 15);
            if (r < it.s.nq * a.group) {
                const int i = a.query_of(r), hd = it.h * a.group + r - i * a.group;
                const uint16_t* p = a.q + (it.s.q0 + i) * a.q_stride + hd * D + (lane >> 4) * 64;
                if (lane < 16 || D > 64) asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
            }
        }
        const int32_t* table = a.sq.table + int64_t(it.b) * a.sq.max_pages;
        // pages with a seen key (none where no key is seen)
        const int p_lo = it.lo >> pl, p_hi = it.hi > it.lo ? (it.hi + page - 1) >> pl : p_lo;
        int j0 = (it.tile0 + it.t0) * kTile;
        auto mine = [&]() {
            const int p = (j0 >> pl) + lane;
            return lane < np && p >= p_lo && p < p_hi;
        };
        int pg = mine() ? table[(j0 >> pl) + lane] : 0;
        for (int t = it.t0; t < it.t1; ++t) {
            const int first = j0 >> pl;
            const bool issue = mine();
            const int bytes = max(0, min(first + np, p_hi) - max(first, p_lo)) * rows * C::kRowBytes * 2;
            if (issue && (pg < 0 || pg >= n_pages)) {
                record_error(a.err, MOE_ERR_INVALID_ARG);
                pg = n_pages;                           // out of range: reads as zeros
            }
            if (!warp_wait(&sh.empty[st], ph, a.err, a.timeout_ns)) {
                dead = true;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], bytes);
            __syncwarp();
            for (int b = 0; b < np; ++b) {
                if (lane == b && issue) {
#pragma unroll
                    for (int x = 0; x < kParts; ++x) {
                        uint8_t* dst = box + st * 2 * C::kTileBytes + x * kTile * 128;
                        tma_load_4d(dst, &maps.k, &sh.full[st], x * kBox, j0 & (page - 1), it.h, pg);
                        tma_load_4d(dst + C::kTileBytes, &maps.v, &sh.full[st], x * kBox, j0 & (page - 1), it.h, pg);
                    }
                }
                __syncwarp();
            }
            if (++st == C::kStages) {
                st = 0;
                ph ^= 1;
            }
            j0 += kTile;
            if (t + 1 < it.t1 && mine()) pg = table[(j0 >> pl) + lane];
        }
    }
    // each stage's last copy
    for (int k = 0; k < C::kStages; ++k) {
        mbar_wait(&sh.full[st], ph, a.err, kDrainNs);
        if (++st == C::kStages) {
            st = 0;
            ph ^= 1;
        }
    }
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(addr)
                 : "memory");
    return r;
}

__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
    return r;
}

// One consumer warp's query rows as A fragments.  bf16 caches: columns in
// order.  e4m3: lane t of a quad holds 16 consecutive columns per 64, so that
// a K row's codes come as one 16-byte load; the k index of the product is
// permuted alike on both sides.
template <int D, bool E4M3>
struct QFrag {
    uint32_t a[D / 16][4];
    float mul[2];             // factor taken out of rows g and g+8 (e4m3)

    __device__ __forceinline__ void load(const AttnArgs& at, const Item& it) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = it.s.nq * at.group;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = it.rt * kRows + g + 8 * r;
            const bool ok = row < rows;
            const int i = ok ? at.query_of(row) : 0;
            const int hd = it.h * at.group + (ok ? row - i * at.group : 0);
            const uint16_t* src = at.q + (it.s.q0 + i) * at.q_stride + hd * D;
            mul[r] = 1.0f;
            if constexpr (!E4M3) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    a[s][r] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * t) : 0u;
                    a[s][2 + r] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * t) : 0u;
                }
            } else {
                uint32_t w[D / 64][8];
                float amax = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint4 x = ok ? *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t + 8 * v)
                                           : make_uint4(0, 0, 0, 0);
                        w[c][4 * v] = x.x;
                        w[c][4 * v + 1] = x.y;
                        w[c][4 * v + 2] = x.z;
                        w[c][4 * v + 3] = x.w;
                    }
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        amax = fmaxf(amax, fabsf(bf16_bits_to_f32(w[c][v] & 0xFFFFu)));
                        amax = fmaxf(amax, fabsf(__uint_as_float(w[c][v] & 0xFFFF0000u)));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                const float f = pow2_norm(amax);
                mul[r] = 1.0f / f;
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const uint32_t x = w[s / 4][2 * (s & 3) + v];
                        a[s][2 * v + r] = pack_f16(bf16_bits_to_f32(x & 0xFFFFu) * f,
                                                   __uint_as_float(x & 0xFFFF0000u) * f);
                    }
            }
        }
    }
};

template <int D, bool E4M3>
__device__ __forceinline__ void consume(const AttnArgs& a, Shared& sh, uint8_t* ring,
                                        float* merge) {
    using C = Cfg<D, E4M3>;
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int grp = wid >> 2, key0 = (wid & 3) * 16;     // this warp's keys of its group's tiles
    const int ctid = threadIdx.x;                        // consumers are threads 0 .. 255
    const bool draft = a.draft != nullptr;
    const int slot_floats = kAttnSlotRows * (D + 2);
    int run = 0, slot = 0;
    uint32_t ip = 0;
    bool dead = false;
    for (;;) {
        if (!dead && !mbar_wait(&sh.item_full[slot], ip, a.err, a.timeout_ns)) dead = true;
        // all warps go on or none (the merge's barriers); its room has been read
        if (!bar_and(kBarMerge, !dead, 32 * kConsumers)) break;
        const Item it = sh.item[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[slot]);
        if (++slot == kItems) {
            slot = 0;
            ip ^= 1;
        }
        if (it.b < 0) break;
        QFrag<D, E4M3> q;
        q.load(a, it);
        const int rows = min(kRows, it.s.nq * a.group - it.rt * kRows);
        const int i0 = a.query_of(it.rt * kRows), i1 = a.query_of(it.rt * kRows + rows - 1);
        RowView view[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = g + 8 * r;
            view[r] = RowView{0, 0, 0ull};
            if (row < rows) view[r] = row_view(a, it.s, a.query_of(it.rt * kRows + row));
        }
        float c[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
            c[r] = a.scale * kLog2e * (E4M3 ? a.kv.k_scale[it.h] * q.mul[r] : 1.0f);
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[n][k] = 0.0f;

        for (int tt = it.t0; tt < it.t1; ++tt, ++run) {
            if ((run & 1) != grp) continue;
            const int st = run % C::kStages, ph = (run / C::kStages) & 1;
            const uint32_t kb = smem_u32(ring + st * 2 * C::kTileBytes), vb = kb + C::kTileBytes;
            if (!dead && !mbar_wait(&sh.full[st], ph, a.err, a.timeout_ns)) dead = true;   // (all warps leave after this item)
            const int j0 = (it.tile0 + tt) * kTile + key0;
            // --- scores of 16 rows x 16 keys
            float s[2][4] = {};
            if constexpr (!E4M3) {
                // lanes 0-7: keys 0-7 of chunk 2s, 8-15: the same keys of chunk 2s+1, 16-31: keys 8-15
                const int key = key0 + (lane & 7) + ((lane & 16) >> 1);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const int chunk = 2 * ks + ((lane >> 3) & 1);
                    uint32_t r[4];
                    ldsm4(kb + (chunk >> 3) * (kTile * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), r);
                    mma16<false>(s[0], q.a[ks][0], q.a[ks][1], q.a[ks][2], q.a[ks][3], r[0], r[1]);
                    mma16<false>(s[1], q.a[ks][0], q.a[ks][1], q.a[ks][2], q.a[ks][3], r[2], r[3]);
                }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int key = key0 + 8 * n + g;
#pragma unroll
                    for (int cc = 0; cc < D / 64; ++cc) {
                        const int chunk = 4 * cc + t;
                        const uint4 w = D == 128
                                            ? lds16(kb + key * 128 + ((chunk ^ (key & 7)) << 4))
                                            : lds16(kb + key * 64 + ((chunk ^ ((key >> 1) & 3)) << 4));
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const int ks = 4 * cc + k4;
                            mma16<true>(s[n], q.a[ks][0], q.a[ks][1], q.a[ks][2], q.a[ks][3],
                                        e4m3x2_to_f16x2(ww[k4] & 0xFFFFu), e4m3x2_to_f16x2(ww[k4] >> 16));
                        }
                    }
                }
            }
            // --- in log2 units, unseen keys at -inf
            const bool whole = rows_see_all(a, it.s, i0, i1, j0, j0 + 16);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[n][k] *= c[k >> 1];
            if (!whole) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!row_sees(view[k >> 1], draft, it.s.first, j0 + 8 * n + 2 * t + (k & 1)))
                            s[n][k] = kNegInf;
            }
            // --- running maximum
            float top[2];
            bool grew = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
                grew = grew || top[r] > m[r];
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float nm = fmaxf(m[r], top[r]);
                    const float f = m[r] == kNegInf ? 0.0f : fast_exp2(m[r] - nm);
                    m[r] = nm;
                    l[r] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][2 * r] *= f;
                        o[n][2 * r + 1] *= f;
                    }
                }
            }
            // --- probabilities: summed in fp32, rounded for the product to the 16-bit type that the
            // matrix instruction takes beside V (bf16: 2^-8 of each at most; f16 beside codes: 2^-11)
            const float ref[2] = {m[0] == kNegInf ? 0.0f : m[0] - kBias<E4M3>, m[1] == kNegInf ? 0.0f : m[1] - kBias<E4M3>};
            float p[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[n][k] = fast_exp2(s[n][k] - ref[k >> 1]);
                    l[k >> 1] += p[n][k];
                }
            uint32_t pa[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    pa[2 * n + r] = E4M3 ? pack_f16(p[n][2 * r], p[n][2 * r + 1])
                                         : pack_bf16(p[n][2 * r], p[n][2 * r + 1]);
            // V rows that no row of the item sees may hold anything: zero them
            // (0 * NaN is NaN).  Lane's keys: 2t, 2t+1 (b0), 2t+8, 2t+9 (b1).
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
            const bool clean = j0 >= it.lo && j0 + 16 <= it.hi;
            if (!clean) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = j0 + 8 * n + 2 * t;
                    keep[n] = (j >= it.lo && j < it.hi ? 0xFFFFu : 0u) |
                              (j + 1 >= it.lo && j + 1 < it.hi ? 0xFFFF0000u : 0u);
                }
            }
            if constexpr (!E4M3) {
                const int key = key0 + (lane & 15);
#pragma unroll
                for (int n2 = 0; n2 < D / 16; ++n2) {
                    const int chunk = 2 * n2 + (lane >> 4);
                    uint32_t r[4];
                    ldsm4t(vb + (chunk >> 3) * (kTile * 128) + key * 128 + (((chunk & 7) ^ (key & 7)) << 4), r);
                    if (!clean) {
                        r[0] &= keep[0];
                        r[1] &= keep[1];
                        r[2] &= keep[0];
                        r[3] &= keep[1];
                    }
                    mma16<false>(o[2 * n2], pa[0], pa[1], pa[2], pa[3], r[0], r[1]);
                    mma16<false>(o[2 * n2 + 1], pa[0], pa[1], pa[2], pa[3], r[2], r[3]);
                }
            } else {
                // column g of block j is element (D/8) g + j: a lane's 16 (or 8)
                // bytes of one key serve every block
                uint32_t w[4][D / 32];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = key0 + 2 * t + (k & 1) + 8 * (k >> 1);
                    if constexpr (D == 128) {
                        const uint4 x = lds16(vb + key * 128 + ((g ^ (key & 7)) << 4));
                        w[k][0] = x.x;
                        w[k][1] = x.y;
                        w[k][2] = x.z;
                        w[k][3] = x.w;
                    } else {
                        const uint2 x = lds8(vb + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (g & 1));
                        w[k][0] = x.x;
                        w[k][1] = x.y;
                    }
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    const uint32_t sel = (n & 3) | (((n & 3) + 4) << 4);
                    uint32_t b0 = e4m3x2_to_f16x2(__byte_perm(w[0][n >> 2], w[1][n >> 2], sel));
                    uint32_t b1 = e4m3x2_to_f16x2(__byte_perm(w[2][n >> 2], w[3][n >> 2], sel));
                    if (!clean) {
                        b0 &= keep[0];
                        b1 &= keep[1];
                    }
                    mma16<true>(o[n], pa[0], pa[1], pa[2], pa[3], b0, b1);
                }
            }
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(&sh.empty[st]);
        }

        // --- join the eight warps
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (l[r] != l[r]) m[r] = fmaxf(m[r], 0.0f);   // a NaN is a result, not an empty row
            m[r] -= kBias<E4M3>;
            if (t == 0) sh.ml[wid][g + 8 * r] = make_float2(m[r], l[r]);
        }
        named_bar(kBarMerge, 32 * kConsumers);
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = kNegInf;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, sh.ml[w][g + 8 * r].x);
            f[r] = m[r] == kNegInf ? 0.0f : fast_exp2(m[r] - top);
        }
        float* buf = merge + (wid & 3) * kRows * D;
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if ((wid >> 2) == half) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = E4M3 ? (D / 8) * (2 * t + (k & 1)) + n : 8 * n + 2 * t + (k & 1);
                        float* at = buf + (g + 8 * (k >> 1)) * D + d;
                        const float v = m[k >> 1] == kNegInf ? 0.0f : o[n][k] * f[k >> 1];
                        *at = half ? v : *at + v;
                    }
            }
            named_bar(kBarMerge, 32 * kConsumers);
        }
        // --- write: the item's output, or this CTA's piece of it
        const bool piece = it.t0 > 0 || it.t1 < it.n;
        float* slot = a.partials + (int64_t(it.t0 == 0 ? 0 : kAttnMaxCtas) + blockIdx.x) * slot_floats;
        const float vs = E4M3 ? a.kv.v_scale[it.h] : 1.0f;
        for (int e = ctid; e < rows * (D / 4); e += 32 * kConsumers) {
            const int row = e / (D / 4), d4 = e % (D / 4);
            float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(merge + (w * kRows + row) * D + 4 * d4);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            float top = kNegInf, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, sh.ml[w][row].x);
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
                const float2 x = sh.ml[w][row];
                sum += x.x == kNegInf ? 0.0f : x.y * fast_exp2(x.x - top);
            }
            if (piece) {
                *reinterpret_cast<float4*>(slot + (d4 * kAttnSlotRows + row) * 4) =
                    make_float4(v.x * vs, v.y * vs, v.z * vs, v.w * vs);
                if (d4 == 0) *reinterpret_cast<float2*>(slot + kAttnSlotRows * D + 2 * row) = make_float2(top, sum);
            } else {
                const int r = it.rt * kRows + row, i = a.query_of(r), hd = it.h * a.group + r - i * a.group;
                const int64_t at = int64_t(it.s.q0 + i) * a.q_heads + hd;
                const float inv = top == kNegInf ? 0.0f : vs / sum;
                *reinterpret_cast<uint2*>(a.out + at * D + 4 * d4) =
                    make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
                if (d4 == 0 && a.lse) a.lse[at] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
            }
        }
        if (ctid == 0) note_split(a, it, rows, kRows, sh.plan);
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) attn_rows_kernel(const AttnArgs a,
                                                               const __grid_constant__ KvMaps maps) {
    using C = Cfg<D, E4M3>;
    extern __shared__ uint8_t dyn[];
    __shared__ Shared sh;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    float* merge = reinterpret_cast<float*>(ring + C::kRing);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kConsumers / 2);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kConsumers);
        }
        fence_barrier_init();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    pdl_wait();
    pdl_launch_dependents();
    plan_work<kRows, kTile>(a, 1, sh.warp_sum, &sh.plan);
    zero_pad_rows(a, sh.plan.seqs);
    if (threadIdx.x >= 32 * kConsumers)
        produce<D, E4M3>(a, maps, sh, ring);
    else
        consume<D, E4M3>(a, sh, ring, merge);
}

template <int D, bool E4M3>
cudaError_t launch_rows(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<D, E4M3>::kSmem;
    static_assert(smem + sizeof(Shared) <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(attn_rows_kernel<D, E4M3>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int grid = n_sms < kAttnMaxCtas ? n_sms : kAttnMaxCtas;
    e = launch_pdl(attn_rows_kernel<D, E4M3>, dim3(grid), dim3(kThreads), smem, s, a, m);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_join(a, grid, s);
}

// Joins the pieces of the split items:
// out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k over the pieces in CTA
// order.  A kernel of its own, not the work of the piece that comes last: that
// CTA alone would read a verify block's 19 pieces of 64 rows (630 KB) at one
// SM's rate, here every SM reads some.
// A unit is kJoinRows rows of a split item; the blocks share the units of all
// items out among them (each adds up the notes for itself).  Four threads have
// four columns of a row, each a quarter of the pieces, kBatch of them in
// flight at a time (more take registers from the second block of an SM: with
// eight, 2048 tokens over 16,384 keys 793 -> 850 us, whose many items are split
// in two; one verify block, split in 20, 21.5 -> 20.8).  The first piece is added before the loop over the others,
// which lie at one distance from each other: with the first one's place chosen
// inside an unrolled loop, joins of 128 columns whose first quarter counted a
// multiple of eight pieces ended in a misaligned access.
constexpr int kJoinRows = 4, kJoinParts = 4;

template <int D>
__global__ void __launch_bounds__(kJoinRows* kJoinParts* D / 4, 1) attn_join_kernel(const AttnArgs a, int n_notes) {
    constexpr int64_t kSlot = kAttnSlotRows * (D + 2);
    constexpr int kCells = kJoinRows * D / 4;                                  // threads of a part
    constexpr int kPer = kAttnMaxCtas / 32, kBatch = 3;
    __shared__ float4 s_v[kJoinParts][kCells];
    __shared__ float s_sum[kJoinParts][kJoinRows];
    __shared__ int s_end[kAttnMaxCtas];                                        // units up to note i, inclusive
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) {
        int u[kPer], sum = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = threadIdx.x * kPer + k;
            u[k] = i < n_notes && a.notes[i].pieces > 0 ? (a.notes[i].rows + kJoinRows - 1) / kJoinRows : 0;
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
        for (int k = 0; k < kPer; ++k) s_end[threadIdx.x * kPer + k] = before += u[k];
    }
    __syncthreads();
    const int total = s_end[kAttnMaxCtas - 1];
    const int cell = threadIdx.x % kCells, part = threadIdx.x / kCells;
    const int rl = cell % kJoinRows, d4 = cell / kJoinRows;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int i = 0;
#pragma unroll
        for (int step = 128; step > 0; step >>= 1)
            if (i + step <= kAttnMaxCtas - 1 && s_end[i + step - 1] <= u) i += step;
        const SplitNote n = a.notes[i];
        const int row0 = (u - (i > 0 ? s_end[i - 1] : 0)) * kJoinRows;
        // the piece of the CTA where the item begins, and (k >= 1) of the k-th CTA after it
        const float* head = a.partials + int64_t(i) * kSlot;
        const float* rest = a.partials + (int64_t(kAttnMaxCtas) + i) * kSlot;
        const int row = min(row0 + rl, n.rows - 1);
        const int ml = kAttnSlotRows * D + 2 * row, od = (d4 * kAttnSlotRows + row) * 4;
        float top = head[ml];
        for (int k0 = 1; k0 < n.pieces; k0 += kBatch) {
            float t[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) t[j] = k0 + j < n.pieces ? rest[(k0 + j) * kSlot + ml] : kNegInf;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) top = fmaxf(top, t[j]);
        }
        const float ref = top == kNegInf ? 0.0f : top;
        float sum = 0.0f;
        float4 v = make_float4(0, 0, 0, 0);
        auto add = [&](const float2& x, const float4& y) {
            const float w = fast_exp2(x.x - ref);
            sum += x.y * w;
            v.x += y.x * w;
            v.y += y.y * w;
            v.z += y.z * w;
            v.w += y.w * w;
        };
        float2 hx = make_float2(kNegInf, 0.0f);
        float4 hy = make_float4(0, 0, 0, 0);
        if (part == 0) {
            hx = *reinterpret_cast<const float2*>(head + ml);
            hy = *reinterpret_cast<const float4*>(head + od);
        }
        for (int k0 = part > 0 ? part : kJoinParts; k0 < n.pieces || k0 == kJoinParts; k0 += kBatch * kJoinParts) {
            float2 x[kBatch];
            float4 y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int k = k0 + j * kJoinParts;
                x[j] = make_float2(kNegInf, 0.0f);
                y[j] = make_float4(0, 0, 0, 0);
                if (k < n.pieces) {
                    x[j] = *reinterpret_cast<const float2*>(rest + k * kSlot + ml);
                    y[j] = *reinterpret_cast<const float4*>(rest + k * kSlot + od);
                }
            }
            if (k0 == kJoinParts) add(hx, hy);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (k0 + j * kJoinParts < n.pieces) add(x[j], y[j]);
        }
        s_v[part][cell] = v;
        if (d4 == 0) s_sum[part][rl] = sum;
        __syncthreads();
        if (part == 0 && row0 + rl < n.rows) {
            sum = 0.0f;
            v = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int p = 0; p < kJoinParts; ++p) {
                const float4 y = s_v[p][cell];
                sum += s_sum[p][rl];
                v.x += y.x;
                v.y += y.y;
                v.z += y.z;
                v.w += y.w;
            }
            const int r = n.row0 + row, q = a.query_of(r), hd = n.head * a.group + r - q * a.group;
            const int64_t at = int64_t(n.q0 + q) * a.q_heads + hd;
            const float inv = top == kNegInf ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(a.out + at * D + 4 * d4) =
                make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (d4 == 0 && a.lse) a.lse[at] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs& a, int n_notes, cudaStream_t s) {
    // two blocks an SM: the pieces' loads of one beside the sums of the other
    const cudaError_t e =
        a.kv.dim == 128
            ? launch_pdl(attn_join_kernel<128>, dim3(2 * n_notes), dim3(kJoinRows * kJoinParts * 32), 0, s, a, n_notes)
            : launch_pdl(attn_join_kernel<64>, dim3(2 * n_notes), dim3(kJoinRows * kJoinParts * 16), 0, s, a, n_notes);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_attn_rows(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s) {
    if (a.kv.dim == 128)
        return a.kv.e4m3 ? launch_rows<128, true>(a, m, n_sms, s) : launch_rows<128, false>(a, m, n_sms, s);
    return a.kv.e4m3 ? launch_rows<64, true>(a, m, n_sms, s) : launch_rows<64, false>(a, m, n_sms, s);
}

}  // namespace moe
