// latent_attn.cu -- attention over a latent cache, absorbed form, on tensor
// memory of pairs of SMs (sm_103a).
//
// With q in latent space, s_j = scale * (q_c . c_j + q_r . r_j) and the output is
// sum_j p_j c_j / sum_j p_j: a cached row is key and value of every head, so a
// row of C + 64 elements takes 2 (2 C + 64) operations a query row.  An item is up to
// 128 query rows (tokens times heads) of one sequence, worked on by a cluster
// of two CTAs, 64 rows each, over tiles of 128 keys:
//   S = Q K^T     one tcgen05.mma of the pair, M = N = 128: each CTA holds its rows
//                 of Q and 64 of the keys, all C + 64 elements;
//   softmax       a warpgroup a CTA; tensor memory has a row's keys 0 .. 63 in lane
//                 r and 64 .. 127 in lane 64 + r;
//   O += P V      M = 128, N = 256: each CTA holds its rows of P, all 128 keys'
//                 elements of its half of C, and its rows of all of O.
// Why pairs: O of 128 rows would fill an SM's tensor memory and Q its shared
// memory; a single SM with 64 rows runs its matrix instructions at less than
// half rate (measured, 64 rows by 64 keys by 16: 61 clocks), while the pair's
// 128 x 128 x 16 takes the ideal 32 and 128 x 256 x 16 64.  The price is that keys
// are held twice, once by key and once by element: 17 panels of 64 x 64 an SM for a
// tile's 9.  They are copied by group and given back by group, so that a group's
// copy has a tile's time to land.
//
// A row's sums use a reference that follows the running maximum only when that has
// grown by more than 2^kLag (see attn_tile.cu).  e4m3 rows are turned to bf16 in
// shared memory, exactly (their scale is a power of two), by two warpgroups.
#include "attn_mma.cuh"
#include "kernels.h"
#include "latent.h"

namespace moe {

namespace {

constexpr int kMT = kLatentRows, kKT = kLatentKeys;
constexpr int kHalf = 64;                // rows and keys of a CTA
constexpr int kPanel = kHalf * 128;      // 64 rows of 64 bf16 elements
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 128;          // S of tile g at column 64 (g & 1), O behind
constexpr float kLag = 8.0f;             // log2 of what powers may grow to
// 4 softmax warps; copies of K, of V, MMA, a warp that passes K on; 4 warps that
// pass V on; e4m3: 4 warps that convert K, 4 that convert V
template <bool E4M3>
constexpr int kThreads = E4M3 ? 512 : 384;
constexpr int kBarSoft = 1, kBarV = 2, kBarK = 3;                // named barriers, 128 threads each

template <int C>
struct Cfg {
    static constexpr int kGroups = C / 128;                      // of two panels of K, beside the rotary one
    static constexpr int kVPanels = C / 128;                     // of a CTA's half of C, for 64 keys
    static constexpr int kNV = C / 256;                          // MMAs of P V a step
    static constexpr int kQBytes = (C / 64 + 1) * kPanel;
    static constexpr int kPBytes = 2 * kPanel;
    static constexpr int kKBytes = kQBytes;
    static constexpr int kVBytes = 2 * kVPanels * kPanel;
    static constexpr size_t kSmem = kQBytes + kPBytes + kKBytes + kVBytes;   // then Shared
};

// A role's place in the pair's work, in shared memory; THREADS threads share it, at
// named barrier `bar`.
struct Ctx {
    Walk<kMT, kKT> wk;
    Item it;
    int more;
    int rows, half;          // rows of the item, and of its first CTA
    int tiles;               // of this pair (0: nothing seen)
    int wlo, whi;            // keys that every row of the item sees

    template <int THREADS>
    __device__ __forceinline__ void sync(int bar) {
        if constexpr (THREADS == 32)
            __syncwarp();
        else
            named_bar(bar, THREADS);
    }
    template <int THREADS>
    __device__ __forceinline__ void start(const AttnArgs& a, const Plan& p) {
        if (threadIdx.x % THREADS == 0) wk.start(a, p);
    }
    template <int THREADS>
    __device__ __forceinline__ bool next(const AttnArgs& a, int bar = 0) {
        sync<THREADS>(bar);
        if (threadIdx.x % THREADS == 0) {
            more = wk.next(a, it);
            if (more) {
                rows = min(kMT, it.s.nq * a.group - it.rt * kMT);
                half = (rows + 1) / 2;
                tiles = it.hi > it.lo ? it.t1 - it.t0 : 0;
                const int2 w = rows_whole(a, it.s, a.query_of(it.rt * kMT), a.query_of(it.rt * kMT + rows - 1));
                wlo = w.x;
                whi = w.y;
            }
        }
        sync<THREADS>(bar);
        return more != 0;
    }
    __device__ __forceinline__ int key0(int tile) const { return (it.tile0 + it.t0 + tile) * kKT; }
};

struct Shared {
    float top[2][2][kHalf];                 // a row's maximum by half of a tile's keys, two tiles in turn
    float sum[2][kHalf];
    int64_t scan[16];                       // plan_work's
    // of this CTA: copies that landed, room that the pair's products gave back
    uint64_t k_full[5], k_empty[5], v_full[2], v_empty[2];
    // of the pair, in its first CTA: operands in place in both
    uint64_t k_ready[5], v_ready[2], p_ready, q_ready;
    // of this CTA: the pair's products are done
    uint64_t s_full[2], pv_done, done;
    Plan plan;
    Ctx ctx[6];                             // softmax, copies of K and V, MMA, K and V passed on
    uint32_t tmem;
};

// --------------------------------------------------------------- cluster ----
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrives on the barrier at this address of the pair's first CTA.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [r];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// mbar_wait for arrivals of either CTA.
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, int32_t* err, uint64_t timeout_ns) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0; it < (1u << 30); ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((it & 63u) == 63u && globaltimer_ns() - t0 > timeout_ns) break;
    }
    record_error(err, MOE_ERR_TIMEOUT);
    return false;
}

__device__ __forceinline__ void pair_alloc(uint32_t* dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kTmemCols) : "memory");
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

// Arrives on the barrier at this address of both CTAs once the products issued so far are done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ----------------------------------------------------------------- copies ----
// The boxes of 64 keys from k0 on: lane p has the p-th, of `tokens` keys.
struct Boxes {
    int tokens, n, bytes;    // bytes: of those of the 64 keys' boxes that are read, for one panel
    bool mine;
    int page, slot;

    __device__ __forceinline__ void set(const LatentArgs& c, const AttnArgs& a, const Item& it, int k0) {
        tokens = min(c.page, kHalf);
        n = kHalf / tokens;
        const int lane = threadIdx.x & 31, k = k0 + lane * tokens;
        mine = lane < n && k < it.hi && k + tokens > it.lo;
        slot = k & (c.page - 1);
        page = 0;
        if (mine) page = a.sq.table[int64_t(it.b) * a.sq.max_pages + (k >> c.page_log2)];
        if (page < 0 || page >= c.n_pages) {
            record_error(a.err, MOE_ERR_INVALID_ARG);
            page = c.n_pages;                                    // out of range: reads as zeros
        }
        bytes = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * tokens * 128;
    }
};

// Copies `panels` (bf16) or panels / 2 parts of codes (e4m3: into the second of each two
// panels, see convert_row) of the boxes' rows, from panel p0 on.
template <bool E4M3>
__device__ __forceinline__ void copy_panels(const Boxes& b, const LatentMaps& maps, uint8_t* dst, int p0, int panels, uint64_t* full) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) mbar_arrive_expect_tx(full, b.bytes * (E4M3 ? panels / 2 : panels));
    __syncwarp();
    if (b.mine) {
        uint8_t* at = dst + lane * b.tokens * 128;
        if constexpr (E4M3) {
            for (int x = 0; x < panels; x += 2) tma_load_4d(at + (x + 1) * kPanel, &maps.latent, full, 0, b.slot, (p0 + x) / 2, b.page);
        } else {
            const int step = b.tokens == kHalf ? 2 : 1;
            for (int x = 0; x < panels; x += step) tma_load_4d(at + x * kPanel, &maps.latent, full, 0, b.slot, p0 + x, b.page);
        }
    }
    __syncwarp();
}

// This CTA's 64 keys of each tile, all elements: the rotary part, then the groups.
template <int C, bool E4M3>
__device__ __forceinline__ void produce_k(const LatentAttnArgs& la, const LatentMaps& maps, Shared& sh, uint8_t* ks, uint32_t rank) {
    using F = Cfg<C>;
    const AttnArgs& a = la.a;
    Ctx& ctx = sh.ctx[1];
    ctx.start<32>(a, sh.plan);
    int uses = 0;
    uint32_t ph = 1u;
    bool dead = false;
    while (!dead && ctx.next<32>(a)) {
        const int T = ctx.tiles;
        for (int j = 0; j < T && !dead; ++j, ph ^= 1u) {
            Boxes b;
            b.set(la.c, a, ctx.it, ctx.key0(j) + static_cast<int>(rank) * kHalf);
            for (int g = 0; g <= F::kGroups; ++g) {              // g = 0: the rotary part
                dead = !warp_wait(&sh.k_empty[g], ph, a.err, a.timeout_ns);
                if (dead) break;
                if (g == 0) {
                    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&sh.k_full[0], b.bytes);
                    __syncwarp();
                    if (b.mine)
                        tma_load_3d(ks + (C / 64) * kPanel + (threadIdx.x & 31) * b.tokens * 128, &maps.rope, &sh.k_full[0], 0, b.slot, b.page);
                    __syncwarp();
                } else {
                    copy_panels<E4M3>(b, maps, ks + (g - 1) * 2 * kPanel, (g - 1) * 2, 2, &sh.k_full[g]);
                }
                ++uses;
            }
        }
    }
    // each group's last copy
    for (int g = 0; g <= F::kGroups; ++g) {
        const int n = (uses + F::kGroups - g) / (F::kGroups + 1);
        if (n > 0) mbar_wait(&sh.k_full[g], (n - 1) & 1, a.err, kDrainNs);
    }
}

// All 128 keys of each tile, this CTA's half of the elements: by half of the keys.
template <int C, bool E4M3>
__device__ __forceinline__ void produce_v(const LatentAttnArgs& la, const LatentMaps& maps, Shared& sh, uint8_t* vs, uint32_t rank) {
    using F = Cfg<C>;
    const AttnArgs& a = la.a;
    Ctx& ctx = sh.ctx[2];
    ctx.start<32>(a, sh.plan);
    int uses = 0;
    uint32_t ph = 1u;
    bool dead = false;
    while (!dead && ctx.next<32>(a)) {
        const int T = ctx.tiles;
        for (int j = 0; j < T && !dead; ++j, ph ^= 1u) {
            for (int h = 0; h < 2; ++h) {
                Boxes b;
                b.set(la.c, a, ctx.it, ctx.key0(j) + h * kHalf);
                dead = !warp_wait(&sh.v_empty[h], ph, a.err, a.timeout_ns);
                if (dead) break;
                copy_panels<E4M3>(b, maps, vs + h * F::kVPanels * kPanel, static_cast<int>(rank) * F::kVPanels, F::kVPanels, &sh.v_full[h]);
                ++uses;
            }
        }
    }
    for (int h = 0; h < 2; ++h) {
        const int n = (uses + 1 - h) / 2;
        if (n > 0) mbar_wait(&sh.v_full[h], (n - 1) & 1, a.err, kDrainNs);
    }
}

// ------------------------------------------------------------ passing on ----
// What landed in this CTA is told to the first one, whose MMA warp waits for both.
// Values of keys that no row of the item sees may be anything: they are zeroed here,
// as are, in tiles where some row does not see some key, those of a key with an
// element that is not finite (its score is not finite for the rows that do see it, so
// that they become NaN all the same; a probability of 0 would make the others NaN).
template <int C>
__device__ __forceinline__ void pass_k(const LatentAttnArgs& la, Shared& sh) {
    const AttnArgs& a = la.a;
    Ctx& ctx = sh.ctx[4];
    ctx.start<32>(a, sh.plan);
    uint32_t ph = 0;
    bool dead = false;
    while (!dead && ctx.next<32>(a)) {
        for (int j = 0; j < ctx.tiles && !dead; ++j, ph ^= 1u) {
            for (int g = 0; g <= Cfg<C>::kGroups; ++g) {
                dead = !warp_wait(&sh.k_full[g], ph, a.err, a.timeout_ns);
                if (dead) break;
                if ((threadIdx.x & 31) == 0) arrive_first(&sh.k_ready[g]);
            }
        }
    }
}

__device__ __forceinline__ bool any_nonfinite(const uint4& w) {
    bool bad = false;
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (x[i] & 0x7F800000u) == 0x7F800000u || (x[i] & 0x7F80u) == 0x7F80u;
    return bad;
}

template <int C>
__device__ __forceinline__ void pass_v(const LatentAttnArgs& la, Shared& sh, uint8_t* vs) {
    using F = Cfg<C>;
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    Ctx& ctx = sh.ctx[5];
    ctx.start<128>(a, sh.plan);
    uint32_t ph = 0;
    bool dead = false;
    while (ctx.next<128>(a, kBarV)) {
        for (int j = 0; j < ctx.tiles && !dead; ++j, ph ^= 1u) {
            for (int h = 0; h < 2; ++h) {
                dead = !warp_wait(&sh.v_full[h], ph, a.err, a.timeout_ns);
                if (dead) break;
                const int j0 = ctx.key0(j) + h * kHalf, lo = max(ctx.it.lo, ctx.wlo), hi = min(ctx.it.hi, ctx.whi);
                if (j0 < lo || j0 + kHalf > hi) {
                    // a key's elements, 16 bytes a lane
                    uint8_t* v = vs + h * F::kVPanels * kPanel + (lane >> 3) * kPanel + (lane & 7) * 16;
                    for (int r = warp; r < kHalf; r += 4) {
                        uint4* p = reinterpret_cast<uint4*>(v + r * 128);
                        bool bad = j0 + r < ctx.it.lo || j0 + r >= ctx.it.hi;
                        if (lane < 8 * F::kVPanels) bad = bad || any_nonfinite(*p);
                        if (__any_sync(0xFFFFFFFFu, bad) && lane < 8 * F::kVPanels) *p = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                if (lane == 0) arrive_first(&sh.v_ready[h]);
            }
        }
    }
}

// e4m3: 128 codes of a key, which landed in row r of the second of two panels, to
// bf16 in row r of both, by one thread: all are read before any is written.
__device__ __forceinline__ void convert_row(uint8_t* two, int r, uint32_t factor, bool nan_again, uint32_t nan_bits, bool zero,
                                            bool zero_nan) {
    uint8_t* first = two + r * 128;
    uint8_t* second = first + kPanel;
    uint4 raw[8];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) raw[ch] = *reinterpret_cast<const uint4*>(second + ((ch ^ (r & 7)) << 4));
    uint32_t most = 0;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
        const uint32_t x[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // as e4m3x4_to_bf16, with the row's power of two in the factor
            const uint32_t p = __byte_perm(x[e], 0, 0x1404), q = __byte_perm(x[e], 0, 0x3424);
            const uint32_t mp = (p >> 4) & 0x07F007F0u, mq = (q >> 4) & 0x07F007F0u;
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y[2 * e]) : "r"(mp | (p & 0x80008000u)), "r"(factor));
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y[2 * e + 1]) : "r"(mq | (q & 0x80008000u)), "r"(factor));
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(mp));
            asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(mq));
        }
        uint8_t* to = ch < 4 ? first : second;
        const int c2 = (2 * ch) & 7;
        *reinterpret_cast<uint4*>(to + ((c2 ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(to + (((c2 + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
    }
    const bool had_nan = e4m3_had_nan(most);
    if (zero || (had_nan && zero_nan)) {
#pragma unroll 1
        for (int ch = 0; ch < 16; ++ch)
            *reinterpret_cast<uint4*>((ch < 8 ? first : second) + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
    } else if (had_nan && nan_again) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>((i < 32 ? first : second)) + (i & 31);
            uint32_t v = *w;
            if ((v & 0x7FFFu) == nan_bits) v |= 0x7FC0u;
            if ((v & 0x7FFF0000u) == nan_bits << 16) v |= 0x7FC00000u;
            *w = v;
        }
    }
}

// The factor of convert_row and what a NaN code comes out as: 480 times the scale.
__device__ __forceinline__ uint32_t code_factor(int scale_log2) {
    const uint32_t f = static_cast<uint32_t>(127 + 120 + scale_log2) << 7;
    return f | (f << 16);
}
__device__ __forceinline__ uint32_t code_nan(int scale_log2) { return 0x43F0u + static_cast<uint32_t>(scale_log2 * 128); }

// K: two warps a group, two groups at a time.
template <int C>
__device__ __forceinline__ void convert_k(const LatentAttnArgs& la, Shared& sh, uint8_t* ks) {
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31, t = threadIdx.x & 127, side = t >> 6;
    const uint32_t factor = code_factor(la.c.scale_log2), nan_bits = code_nan(la.c.scale_log2);
    Ctx& ctx = sh.ctx[4];
    ctx.start<128>(a, sh.plan);
    uint32_t ph = 0;
    bool dead = false;
    while (ctx.next<128>(a, kBarK)) {
        for (int j = 0; j < ctx.tiles && !dead; ++j, ph ^= 1u) {
            if (t < 32) {
                dead = !warp_wait(&sh.k_full[0], ph, a.err, a.timeout_ns);
                if (dead) break;
                if (lane == 0) arrive_first(&sh.k_ready[0]);
            }
            for (int g = side; g < Cfg<C>::kGroups; g += 2) {
                dead = !warp_wait(&sh.k_full[g + 1], ph, a.err, a.timeout_ns);
                if (dead) break;
                convert_row(ks + g * 2 * kPanel, t & 63, factor, true, nan_bits, false, false);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive_first(&sh.k_ready[g + 1]);
            }
        }
    }
}

// V: a thread a key and 128 elements.
template <int C>
__device__ __forceinline__ void convert_v(const LatentAttnArgs& la, Shared& sh, uint8_t* vs) {
    using F = Cfg<C>;
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31, t = threadIdx.x & 127, r = t & 63, side = t >> 6;
    const uint32_t factor = code_factor(la.c.scale_log2), nan_bits = code_nan(la.c.scale_log2);
    Ctx& ctx = sh.ctx[5];
    ctx.start<128>(a, sh.plan);
    uint32_t ph = 0;
    bool dead = false;
    while (ctx.next<128>(a, kBarV)) {
        for (int j = 0; j < ctx.tiles && !dead; ++j, ph ^= 1u) {
            for (int h = 0; h < 2; ++h) {
                dead = !warp_wait(&sh.v_full[h], ph, a.err, a.timeout_ns);
                if (dead) break;
                const int j0 = ctx.key0(j) + h * kHalf, key = j0 + r;
                const bool part = j0 < ctx.wlo || j0 + kHalf > ctx.whi;
                if (2 * side < F::kVPanels)
                    convert_row(vs + (h * F::kVPanels + 2 * side) * kPanel, r, factor, true, nan_bits,
                                key < ctx.it.lo || key >= ctx.it.hi, part);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive_first(&sh.v_ready[h]);
            }
        }
    }
}

// --------------------------------------------------------------- products ----
// The MMA warp of the first CTA: Q K^T of a tile, then P V of the one before, so
// that one tile's softmax runs beside another's products.
template <int C>
__device__ __forceinline__ void multiply(const LatentAttnArgs& la, Shared& sh, uint8_t* qs, uint8_t* ps, uint8_t* ks, uint8_t* vs) {
    using F = Cfg<C>;
    constexpr uint32_t kIdQK = idesc(false, kKT), kIdPV = idesc(true, 256);
    const AttnArgs& a = la.a;
    const uint32_t colS = sh.tmem, colO = sh.tmem + kColO;
    const uint64_t qd = sdesc(smem_u32(qs), 16, 1024), pd = sdesc(smem_u32(ps), 16, 1024);
    const uint64_t kd = sdesc(smem_u32(ks), 16, 1024), vd = sdesc(smem_u32(vs), kPanel, 1024);
    Ctx& ctx = sh.ctx[3];
    ctx.start<32>(a, sh.plan);
    uint32_t qp = 0, pp = 0, kp = 0, vp = 0, g = 0;              // phases; tiles so far
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !__all_sync(0xFFFFFFFFu, pair_wait(bar, parity, a.err, a.timeout_ns));
    };
    while (!dead && ctx.next<32>(a)) {
        const int T = ctx.tiles;
        if (T == 0) continue;
        wait(&sh.q_ready, qp);
        qp ^= 1u;
        for (int i = 0; i <= T && !dead; ++i) {
            if (i < T) {
#pragma unroll 1
                for (int x = 0; x <= F::kGroups; ++x) {
                    wait(&sh.k_ready[x], kp);
                    if (dead) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const int p0 = x == 0 ? C / 64 : 2 * (x - 1), n = x == 0 ? 4 : 8;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            if (k >= n) break;
                            const uint32_t off = ((p0 + (k >> 2)) * kPanel + (k & 3) * 32) >> 4;
                            pair_mma(colS + 64 * (g & 1u), qd + off, kd + off, kIdQK, x > 0 || k > 0);
                        }
                        pair_commit(&sh.k_empty[x]);
                        if (x == F::kGroups) pair_commit(&sh.s_full[g & 1u]);
                    }
                    __syncwarp();
                }
                kp ^= 1u;
                ++g;
            }
            if (i > 0 && !dead) {
                wait(&sh.p_ready, pp);
                pp ^= 1u;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    wait(&sh.v_ready[h], vp);
                    if (dead) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
#pragma unroll
                            for (int n = 0; n < F::kNV; ++n)
                                pair_mma(colO + 128 * n, pd + ((h * kPanel + k * 32) >> 4),
                                         vd + (((h * F::kVPanels + 2 * n) * kPanel + k * 2048) >> 4), kIdPV,
                                         i > 1 || h > 0 || k > 0);
                        }
                        pair_commit(&sh.v_empty[h]);
                        if (h == 1) pair_commit(&sh.pv_done);
                    }
                    __syncwarp();
                }
                vp ^= 1u;
            }
        }
    }
    // the products end before the accumulators are given back
    if (elect_one()) pair_commit(&sh.done);
    __syncwarp();
    mbar_wait(&sh.done, 0, a.err, kDrainNs);
}

// ---------------------------------------------------------------- softmax ----
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The CTA's rows of Q into shared memory, K-major with the 128-byte swizzle, by 128
// threads in whole rows; rows past the last are zeros.
template <int C>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Item& it, int row0, int count, bool negate, uint8_t* qs) {
    constexpr int kChunks = (C + kLatentRot) / 8, kBatch = 9;
    const uint32_t flip = negate ? 0x80008000u : 0u;
#pragma unroll 1
    for (int e0 = 0; e0 < kHalf * kChunks; e0 += 128 * kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int e = e0 + 128 * k + static_cast<int>(threadIdx.x), r = e / kChunks, ch = e - r * kChunks;
            w[k] = make_uint4(0, 0, 0, 0);
            if (r < count) {
                const int row = row0 + r, qi = a.query_of(row), hd = row - qi * a.group;
                w[k] = __ldg(reinterpret_cast<const uint4*>(a.q + int64_t(it.s.q0 + qi) * a.q_stride + hd * (C + kLatentRot) + 8 * ch));
                w[k] = make_uint4(w[k].x ^ flip, w[k].y ^ flip, w[k].z ^ flip, w[k].w ^ flip);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int e = e0 + 128 * k + static_cast<int>(threadIdx.x), r = e / kChunks, ch = e - r * kChunks;
            if (r < kHalf) *reinterpret_cast<uint4*>(qs + (ch >> 3) * kPanel + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = w[k];
        }
    }
    fence_async_smem();
}

template <int C>
__device__ __forceinline__ void soften(const LatentAttnArgs& la, Shared& sh, uint8_t* qs, uint8_t* ps, int pair, uint32_t rank) {
    using F = Cfg<C>;
    const AttnArgs& a = la.a;
    const int tid = threadIdx.x, lr = tid & 63, half = tid >> 6, lane = tid & 31;
    const uint32_t tm = sh.tmem + (static_cast<uint32_t>(tid & 96) << 16);
    const uint32_t colO = tm + kColO;
    uint8_t* p_row = ps + half * kPanel + lr * 128;
    const bool draft = a.draft != nullptr;
    Ctx& ctx = sh.ctx[0];
    ctx.start<128>(a, sh.plan);
    const Item& it = ctx.it;
    uint32_t g = 0, pv = 0;                                      // tiles so far; phase of pv_done
    bool pending = false, dead = false;                          // a P V that has not been waited for
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
        tc_fence_after();
    };
    auto wait_pv = [&]() {
        if (!pending) return;
        wait(&sh.pv_done, pv);
        pv ^= 1u;
        pending = false;
    };
    // log2 units a product: at least 1.2e-38 (an unseen key's -inf times it stays -inf), or NaN; the sign goes to the queries
    const float cs = a.scale * kLog2e;
    const float c = fmaxf(fabsf(cs), 1.2e-38f);
    while (ctx.next<128>(a, kBarSoft)) {
        const int row0 = static_cast<int>(rank) * ctx.half, count = rank ? ctx.rows - ctx.half : ctx.half;
        const int T = ctx.tiles;
        const bool valid = lr < count;
        const int r = it.rt * kMT + row0 + (valid ? lr : 0), qi = a.query_of(r), hd = r - qi * a.group;
        RowView view{0, 0, 0ull};
        if (valid) view = row_view(a, it.s, qi);
        if (T > 0) {
            load_queries<C>(a, it, it.rt * kMT + row0, count, cs < 0.0f, qs);
            __syncwarp();
            if (lane == 0) arrive_first(&sh.q_ready);
        }
        float ref = kNegInf, sum0 = 0.0f, sum1 = 0.0f;
        for (int j = 0; j < T; ++j, ++g) {
            const int j0 = ctx.key0(j);
            wait(&sh.s_full[g & 1u], (g >> 1) & 1u);
            float x[2][32];
            tmem_ld32(tm + 64 * (g & 1u), x[0]);
            tmem_ld32(tm + 64 * (g & 1u) + 32, x[1]);
            tmem_wait_ld();
            if (j0 < ctx.wlo || j0 + kKT > ctx.whi) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t bits = row_bits(view, draft, it.s.first, j0 + half * kHalf + 32 * q);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((bits >> e) & 1u)) x[q][e] = kNegInf;
                }
            }
            float m4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int e = 0; e < 32; e += 4)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x[q][e + k]);
            float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            sh.top[g & 1u][half][lr] = top;
            named_bar(kBarSoft, 128);
            top = fmaxf(top, sh.top[g & 1u][half ^ 1][lr]) * c;
            if (!(top > kNegInf)) top = kNegInf;                 // (NaN: the sums carry it)
            const bool grow = top > ref + kLag || (ref == kNegInf && top > kNegInf);
            if (j > 0 && __any_sync(0xFFFFFFFFu, grow)) {
                wait_pv();
                const float f = !grow ? 1.0f : (ref == kNegInf ? 0.0f : fast_exp2(ref - top));
                sum0 *= f;
                sum1 *= f;
#pragma unroll 1
                for (int q = 0; q < F::kNV * 8; ++q) {
                    float o[16];
                    tmem_ld16(colO + 16 * q, o);
                    tmem_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(f == 0.0f ? 0.0f : o[e] * f);
                    tmem_st16(colO + 16 * q, u);
                }
                tmem_wait_st();
            }
            if (grow) ref = top;
            const float off = ref == kNegInf ? 0.0f : -ref;
            uint32_t u[32];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float p0, p1;
                    fma2_to(p0, p1, x[q][e], x[q][e + 1], c, off);
                    p0 = fast_exp2(p0);
                    p1 = fast_exp2(p1);
                    add2(sum0, sum1, p0, p1);
                    u[16 * q + e / 2] = pack_bf16(p0, p1);
                }
            wait_pv();                                           // P's room has been read
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
                *reinterpret_cast<uint4*>(p_row + ((ch ^ (lr & 7)) << 4)) =
                    make_uint4(u[4 * ch], u[4 * ch + 1], u[4 * ch + 2], u[4 * ch + 3]);
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first(&sh.p_ready);
            pending = true;
        }
        // --- the item's rows: normalised, or this pair's piece of them
        sh.sum[half][lr] = sum0 + sum1;
        named_bar(kBarSoft, 128);
        const float sum = sh.sum[0][lr] + sh.sum[1][lr];
        if (sum != sum) ref = fmaxf(ref, 0.0f);                  // a NaN is a result, not an empty row
        const bool piece = it.t0 > 0 || it.t1 < it.n;
        float* slot = a.partials + (int64_t(it.t0 == 0 ? 0 : kLatentMaxPairs) + pair) * (kLatentRows * (C + 2));
        const int64_t at = int64_t(it.s.q0 + qi) * a.q_heads + hd;
        const float weight = ref == kNegInf || T == 0 ? 0.0f : (piece ? 1.0f : 1.0f / sum);
        if (valid && half == 0) {
            if (piece)
                *reinterpret_cast<float2*>(slot + kLatentRows * C + 2 * (row0 + lr)) = make_float2(ref, sum);
            else if (a.lse)
                a.lse[at] = ref == kNegInf ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
        wait_pv();
        if (__any_sync(0xFFFFFFFFu, valid)) {
#pragma unroll 1
            for (int q = 0; q < F::kNV * 8; ++q) {
                float o[16];
                tmem_ld16(colO + 16 * q, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = weight != 0.0f ? o[e] * weight : 0.0f;
                const int d0 = half * (C / 2) + 16 * q;
                if (valid) {
                    if (piece) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(slot + ((d0 / 4 + e) * kLatentRows + row0 + lr) * 4) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4*>(a.out + at * C + d0 + 8 * e) =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        if (tid == 0 && rank == 0) note_split(a, it, ctx.rows, kMT, sh.plan, pair);
    }
}

template <int C, bool E4M3>
__global__ void __launch_bounds__(kThreads<E4M3>, 1) latent_attn_kernel(const LatentAttnArgs la, const __grid_constant__ LatentMaps maps) {
    using F = Cfg<C>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    uint8_t* qs = dyn;
    uint8_t* ps = qs + F::kQBytes;
    uint8_t* ks = ps + F::kPBytes;
    uint8_t* vs = ks + F::kKBytes;
    Shared& sh = *reinterpret_cast<Shared*>(dyn + F::kSmem);
    const AttnArgs& a = la.a;
    const int warp = threadIdx.x >> 5, pair = blockIdx.x >> 1;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 5; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.k_ready[i], E4M3 && i > 0 ? 4 : 2);    // both CTAs: the passing warp, or the group's two that convert
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.v_ready[i], 8);
            mbar_init(&sh.s_full[i], 1);
        }
        mbar_init(&sh.p_ready, 8);
        mbar_init(&sh.q_ready, 8);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.done, 1);
        fence_barrier_init();
        prefetch_tensormap(&maps.latent);
        prefetch_tensormap(&maps.rope);
    }
    if (warp == 6) pair_alloc(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // both CTAs' barriers are there
    pdl_wait();
    pdl_launch_dependents();
    plan_work<kMT, kKT>(a, 1, sh.scan, &sh.plan, pair, gridDim.x >> 1, rank == 0);   // (its barriers publish sh.tmem)
    tc_fence_after();
    zero_pad_rows(a, sh.plan.seqs);
    if (warp < 4)
        soften<C>(la, sh, qs, ps, pair, rank);
    else if (warp == 4)
        produce_k<C, E4M3>(la, maps, sh, ks, rank);
    else if (warp == 5)
        produce_v<C, E4M3>(la, maps, sh, vs, rank);
    else if (warp == 6) {
        if (rank == 0) multiply<C>(la, sh, qs, ps, ks, vs);
    } else if (warp >= 8) {
        if constexpr (E4M3) {
            if (warp < 12)
                convert_k<C>(la, sh, ks);
            else
                convert_v<C>(la, sh, vs);
        } else {
            pass_v<C>(la, sh, vs);
        }
    } else if (!E4M3) {
        pass_k<C>(la, sh);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // nothing of the pair is in flight
    tc_fence_after();
    if (warp == 6) pair_dealloc(sh.tmem);
}

// Joins the pieces of the split items, out = sum_k 2^(m_k - m) O_k / sum_k 2^(m_k - m) l_k
// in pair order.  A unit is two rows of a split item; the blocks share the units
// of all items out.  Four threads have four columns of a row, each a quarter of the pieces.
constexpr int kJoinRows = 2, kJoinParts = 4;

template <int C>
__global__ void __launch_bounds__(kJoinRows* kJoinParts* C / 4, 1) latent_join_kernel(const AttnArgs a, int n_notes) {
    constexpr int64_t kSlot = kLatentRows * (C + 2);
    constexpr int kCells = kJoinRows * C / 4, kBatch = 3;
    __shared__ float4 s_v[kJoinParts][kCells];
    __shared__ float s_sum[kJoinParts][kJoinRows];
    __shared__ int s_end[96];                                    // units up to note i, inclusive
    static_assert(kLatentMaxPairs <= 96, "three notes a lane");
    pdl_wait();
    pdl_launch_dependents();
    if (threadIdx.x < 32) {
        int u[3], sum = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int i = threadIdx.x * 3 + k;
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
        for (int k = 0; k < 3; ++k) s_end[threadIdx.x * 3 + k] = before += u[k];
    }
    __syncthreads();
    const int total = s_end[95];
    const int cell = threadIdx.x % kCells, part = threadIdx.x / kCells;
    const int rl = cell % kJoinRows, d4 = cell / kJoinRows;
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
        int i = 0;
        while (s_end[i] <= u) ++i;
        const SplitNote n = a.notes[i];
        const int row0 = (u - (i > 0 ? s_end[i - 1] : 0)) * kJoinRows;
        // the piece of the pair where the item begins, and (k >= 1) of the k-th pair after it
        const float* head = a.partials + int64_t(i) * kSlot;
        const float* rest = a.partials + (int64_t(kLatentMaxPairs) + i) * kSlot;
        const int row = min(row0 + rl, n.rows - 1);
        const int ml = kLatentRows * C + 2 * row, od = (d4 * kLatentRows + row) * 4;
        float top = head[ml];
        for (int k = 1; k < n.pieces; ++k) top = fmaxf(top, rest[k * kSlot + ml]);
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
        if (part == 0) add(*reinterpret_cast<const float2*>(head + ml), *reinterpret_cast<const float4*>(head + od));
        for (int k0 = part > 0 ? part : kJoinParts; k0 < n.pieces; k0 += kBatch * kJoinParts) {
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
            const int r = n.row0 + row, q = a.query_of(r), hd = r - q * a.group;
            const int64_t at = int64_t(n.q0 + q) * a.q_heads + hd;
            const float inv = top == kNegInf ? 0.0f : 1.0f / sum;
            *reinterpret_cast<uint2*>(a.out + at * C + 4 * d4) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
            if (d4 == 0 && a.lse) a.lse[at] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
        }
        __syncthreads();
    }
}

template <int C, bool E4M3>
cudaError_t launch(const LatentAttnArgs& a, const LatentMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<C>::kSmem + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(latent_attn_kernel<C, E4M3>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int pairs = n_sms / 2 < kLatentMaxPairs ? n_sms / 2 : kLatentMaxPairs;
    e = launch_pdl_cluster(latent_attn_kernel<C, E4M3>, dim3(2 * pairs), dim3(kThreads<E4M3>), 2, smem, s, a, m);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_pdl(latent_join_kernel<C>, dim3(n_sms), dim3(kJoinRows * kJoinParts * C / 4), 0, s, a.a, pairs);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnArgs& a, const LatentMaps& m, int n_sms, cudaStream_t s) {
    if (a.c.dim == 512) return a.c.e4m3 ? launch<512, true>(a, m, n_sms, s) : launch<512, false>(a, m, n_sms, s);
    return a.c.e4m3 ? launch<256, true>(a, m, n_sms, s) : launch<256, false>(a, m, n_sms, s);
}

}  // namespace moe
