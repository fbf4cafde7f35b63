// latent_attn.cu -- attention over a latent cache, absorbed form, on tensor
// memory of pairs of SMs (sm_103a).
//
// With q in latent space, s_j = scale * (q_c . c_j + q_r . r_j) and the output is
// sum_j p_j c_j / sum_j p_j: a cached row is key and value of every head, so a
// row of C + 64 elements takes 2 (2 C + 64) operations a query row.  An item is up to
// 128 query rows (tokens times heads) of one sequence, worked on by a cluster
// of two CTAs, 64 rows each, over tiles of 64 keys:
//   S = Q K^T     one tcgen05.mma of the pair, M = 128, N = 64: each CTA holds its
//                 rows of Q and 32 of the keys, all C + 64 elements;
//   softmax       a warpgroup a CTA; tensor memory has a row's keys 0 .. 31 in lane
//                 r and 32 .. 63 in lane 64 + r;
//   O += P V      M = 128, N = 256: each CTA holds its rows of P, all 64 keys'
//                 elements of its half of C, and its rows of all of O.
// Why pairs: O of 128 rows would fill an SM's tensor memory and Q its shared
// memory; a single SM with 64 rows runs its matrix instructions at less than
// half rate (measured, 64 rows by 64 keys by 16: 61 clocks, by 256: 147), while the pair's
// 128 x 64 x 16 takes 25 and 128 x 256 x 16 the ideal 64.  The price is that a key is
// held twice, whole in one CTA and by halves in both, and copied for each from L2.
// (The halves copied from shared memory to shared memory instead: such copies run at
// some 14 bytes a clock, 60 clocks a key.)
//
// A row's sums use a reference that follows the running maximum only when that has
// grown by more than 2^kLag (see attn_tile.cu).  e4m3 rows are turned to bf16 in
// shared memory, exactly (their scale is a power of two), by two warpgroups.
#include "kernels.h"
#include "pair.cuh"

namespace moe {

namespace {

constexpr int kKT = kLatentKeys;
constexpr int kRows = 64;                // rows of a CTA, as the products take them
constexpr int kKeys = kKT / 2;           // whole keys of a CTA
constexpr int kRowPanel = kRows * 128;   // 64 elements of its rows
// K and V lie in atoms of 8 keys by 64 elements (1 KB, swizzled), eight keys' atoms
// beside each other, so that a copy reads eight whole rows at a time (element by
// element of all rows, memory gave 4.7 TB/s).  The rotary part of K has its own place.
constexpr int kAtom = 1024;
constexpr uint32_t kColO = 64;           // S of tile g at column 32 (g & 1), O behind
constexpr float kLag = 8.0f;             // log2 of what powers may grow to
// 4 softmax warps; copies of keys, MMA, copies of values, one that passes keys on; 4
// that pass values on; e4m3: 4 that convert keys and pass them on
template <bool E4M3>
constexpr int kThreads = E4M3 ? 512 : 384;
constexpr int kBarSoft = 1, kBarV = 2, kBarK = 3;                // named barriers, 128 threads each
constexpr int kBarTop = 4;                                       // and two of the 64 that share 32 rows

constexpr int kAhead = 3;                // items that the copying warp may be ahead by

// FEW: items of up to 64 rows, 32 a CTA (single tokens of up to 64 heads). Their
// queries take half the room, which a third stage of keys gets: such calls are bound by
// memory, and two stages of keys are too few bytes on their way (48 single tokens over
// 251 to 32,011 rows: 103 -> 97 us). The products still take 64 rows a CTA: those
// past the 32 are whatever lies behind a panel, and reach no other row.
template <int C, bool FEW>
struct Cfg {
    static constexpr int kItem = FEW ? kLatentRows / 2 : kLatentRows;   // rows of an item
    static constexpr int kHeld = kItem / 2;                      // of them a CTA's
    static constexpr int kQPanel = kHeld * 128;
    static constexpr int kKStages = FEW ? 3 : 2;
    static constexpr int kParts = C / 128;                       // of two panels each: of a key, beside the rotary one
    static constexpr int kVPanels = C / 128;                     // of a CTA's half of C
    static constexpr int kNV = C / 256;                          // MMAs of P V a step
    static constexpr int kQBytes = (C / 64 + 1) * kQPanel;
    static constexpr int kPBytes = kRowPanel;
    static constexpr int kKGroup = C / 64 * kAtom;               // of eight keys
    static constexpr int kVGroup = kVPanels * kAtom;
    static constexpr int kRope = kKeys / 8 * kKGroup;            // offset of the rotary part in a stage
    static constexpr int kKBytes = kRope + kKeys / 8 * kAtom;
    static constexpr int kVBytes = kKT / 8 * kVGroup;
    static constexpr size_t kSmem = kQBytes + kKStages * kKBytes + 2 * (kPBytes + kVBytes);   // then Shared
};

// An item as the CTA's warps work on it.  The warp that copies keys walks the pair's
// items and queues them here; each other role takes its own way through the queue.
struct Job {
    Item it;
    int more;                // 0: none; no other field holds
    int rows, half;          // rows of the item, and of its first CTA
    int tiles;               // of this pair (0: nothing seen)
    int wlo, whi;            // keys that every row of the item sees

    template <int MT>
    __device__ __forceinline__ void set(const AttnArgs& a, const Item& i) {
        const int n = min(MT, i.s.nq * a.group - i.rt * MT);
        const int2 w = rows_whole(a, i.s, a.query_of(i.rt * MT), a.query_of(i.rt * MT + n - 1));
        it = i;
        rows = n;
        half = (n + 1) / 2;
        tiles = i.hi > i.lo ? i.t1 - i.t0 : 0;
        wlo = w.x;
        whi = w.y;
    }
    __device__ __forceinline__ int key0(int tile) const { return (it.tile0 + it.t0 + tile) * kKT; }
};

// Barriers of the stages of K and of the two of V, S and P, a tile each in turn.
struct Shared {
    float top[2][2][kRows];                 // a row's maximum by half of a tile's keys, two tiles in turn
    float sum[2][kRows];
    uint8_t odd[2][kRows];                  // a key that the row sees scored -inf in a tile that some row sees in part
    int64_t scan[16];                       // plan_work's
    // of this CTA: what landed, and the room that the products gave back
    uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2], q_full, q_empty;
    // of the pair, in its first CTA: operands in place in both
    uint64_t k_ready[3], v_ready[2], p_ready[2], q_ready;
    // of this CTA: the pair's products are done
    uint64_t s_full[2], pv_done[2], done;
    Plan plan;
    Job job[kAhead];
    uint64_t job_full[kAhead], job_empty[kAhead];
    uint32_t tmem;
};

// A warp's way through the queue.
struct Jobs {
    int n = 0;
    __device__ __forceinline__ const Job* next(Shared& sh, const AttnArgs& a) {
        if (!warp_wait(&sh.job_full[n % kAhead], (n / kAhead) & 1, a.err, a.timeout_ns)) return nullptr;
        const Job* j = &sh.job[n % kAhead];
        return j->more ? j : nullptr;
    }
    // by all of the warp, once it has read what it needs of the item
    __device__ __forceinline__ void done(Shared& sh) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.job_empty[n % kAhead]);
        ++n;
    }
};

// A warpgroup's next item: all of it goes on or stops, at the named barrier `id`.
__device__ __forceinline__ const Job* next_of_group(Jobs& jobs, Shared& sh, const AttnArgs& a, int id, bool dead) {
    const Job* j = dead ? nullptr : jobs.next(sh, a);
    return bar_and(id, j != nullptr, 128) ? j : nullptr;
}

// A place in a ring of N stages.
template <int N>
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++st == N) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// ----------------------------------------------------------------- copies ----
// 5-D tiled bulk tensor load global -> shared; c0 (innermost, elements) starts on a
// 16-byte boundary.  A coordinate out of range reads as zeros.
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1, int32_t c2,
                                            int32_t c3, int32_t c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// The two warps that copy from memory: keys (this CTA's 32 of each tile, all elements
// and the rotary part) and values (all 64 keys, this CTA's half of the elements).  A
// box a page, each page by a lane of its own.  e4m3: the codes land in the second half
// of their stage, see convert.
template <int C, bool FEW, bool E4M3, bool V>
__device__ __forceinline__ void produce(const LatentAttnArgs& la, const LatentMaps& maps, Shared& sh, uint8_t* qs, uint8_t* ring, uint32_t rank) {
    using F = Cfg<C, FEW>;
    constexpr int kN = V ? kKT : kKeys, kGroup = (V ? F::kVGroup : F::kKGroup) / (E4M3 ? 2 : 1);   // eight keys' bytes
    constexpr int kStages = V ? 2 : F::kKStages;
    const AttnArgs& a = la.a;
    uint64_t* fulls = V ? sh.v_full : sh.k_full;
    uint64_t* empties = V ? sh.v_empty : sh.k_empty;
    const CUtensorMap* map = V ? &maps.values : &maps.keys;
    const int lane = threadIdx.x & 31, p0 = V ? static_cast<int>(rank) * F::kVPanels / (E4M3 ? 2 : 1) : 0;
    const int tokens = min(la.c.page, kN), boxes = kN / tokens;
    Walk<F::kItem, kKT> walk;                                    // keys: every lane's own, in registers
    if (!V) walk.start(a, sh.plan);
    Jobs jobs;
    Ring<kStages> at;
    int uses = 0, queries = 0;                                   // copies of tiles, of queries
    bool dead = false;
    while (!dead) {
        const Job* job;
        if constexpr (V) {
            job = jobs.next(sh, a);
            if (!job) break;
        } else {
            Job& next = sh.job[jobs.n % kAhead];
            if (!warp_wait(&sh.job_empty[jobs.n % kAhead], ((jobs.n / kAhead) & 1) ^ 1, a.err, a.timeout_ns)) break;
            Item it;                                             // (the others' waits for it run out too)
            const bool more = walk.next(a, it);
            if (lane == 0) {
                next.more = more;
                if (more) next.set<F::kItem>(a, it);
                mbar_arrive(&sh.job_full[jobs.n % kAhead]);
            }
            __syncwarp();
            if (!more) break;
            job = &next;
            ++jobs.n;
        }
        const Item& it = job->it;
        const int32_t* table = a.sq.table + int64_t(it.b) * a.sq.max_pages;
        for (int j = 0; j < job->tiles; ++j, ++uses, at.step()) {
            const int k = job->key0(j) + (V ? 0 : static_cast<int>(rank) * kKeys) + lane * tokens;
            const bool mine = lane < boxes && k < it.hi && k + tokens > it.lo;
            int page = mine ? table[k >> la.c.page_log2] : 0;
            if (page < 0 || page >= la.c.n_pages) {
                record_error(a.err, MOE_ERR_INVALID_ARG);
                page = la.c.n_pages;                             // out of range: reads as zeros
            }
            const int rows = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * tokens;
            dead = !warp_wait(&empties[at.st], at.ph ^ 1u, a.err, a.timeout_ns);
            if (dead) break;
            uint64_t* full = &fulls[at.st];
            if (lane == 0) mbar_arrive_expect_tx(full, rows / 8 * (kGroup + (V ? 0 : kAtom)));
            __syncwarp();
            if (mine) {
                const int slot = k & (la.c.page - 1);
                uint8_t* stage = ring + at.st * (V ? F::kVBytes : F::kKBytes);
                uint8_t* to = stage + (E4M3 ? kN / 8 * kGroup : 0) + lane * (tokens / 8) * kGroup;
                if (!V) tma_load_3d(stage + F::kRope + lane * (tokens / 8) * kAtom, &maps.rope, full, 0, slot, page);
                tma_load_5d(to, map, full, 0, 0, p0, slot / 8, page);
            }
            __syncwarp();
            if (!V && j == 0 && la.q_flat) {
                dead = !warp_wait(&sh.q_empty, (queries & 1) ^ 1, a.err, a.timeout_ns);
                if (dead) {
                    ++uses;                                      // (this tile's copy is under way)
                    break;
                }
                if (lane == 0) {
                    const int row = it.s.q0 * a.group + it.rt * F::kItem + static_cast<int>(rank) * job->half;
                    mbar_arrive_expect_tx(&sh.q_full, F::kQBytes);
                    tma_load_3d(qs, &maps.q, &sh.q_full, 0, row, 0);
                }
                __syncwarp();
                ++queries;
            }
        }
        if constexpr (V) jobs.done(sh);
    }
    if (queries > 0) mbar_wait(&sh.q_full, (queries - 1) & 1, a.err, kDrainNs);
    // each stage's last copy
    for (int st = 0; st < kStages; ++st) {
        const int n = (uses + kStages - 1 - st) / kStages;
        if (n > 0) mbar_wait(&fulls[st], (n - 1) & 1, a.err, kDrainNs);
    }
}

// ------------------------------------------------------------ passing on ----
// What landed in this CTA is told to the first one, whose MMA warp waits for both.
// By a warp of each CTA, of an item's queries.
__device__ __forceinline__ bool pass_q(const AttnArgs& a, Shared& sh, uint32_t& parity) {
    const bool ok = warp_wait(&sh.q_full, parity, a.err, a.timeout_ns);
    if (ok && (threadIdx.x & 31) == 0) arrive_first(&sh.q_ready);
    parity ^= 1u;
    return ok;
}

template <int C, bool FEW>
__device__ __forceinline__ void pass_k(const LatentAttnArgs& la, Shared& sh) {
    const AttnArgs& a = la.a;
    uint32_t qp = 0;
    Jobs jobs;
    Ring<Cfg<C, FEW>::kKStages> at;
    bool dead = false;
    while (const Job* job = dead ? nullptr : jobs.next(sh, a)) {
        for (int j = 0; j < job->tiles; ++j, at.step()) {
            dead = !warp_wait(&sh.k_full[at.st], at.ph, a.err, a.timeout_ns);
            if (dead) break;
            if ((threadIdx.x & 31) == 0) arrive_first(&sh.k_ready[at.st]);
            if (j == 0) dead = !pass_q(a, sh, qp);
            if (dead) break;
        }
        jobs.done(sh);
    }
}

__device__ __forceinline__ bool any_nonfinite(const uint4& w) {
    bool bad = false;
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (x[i] & 0x7F800000u) == 0x7F800000u || (x[i] & 0x7F80u) == 0x7F80u;
    return bad;
}

// Four warps.  Values of keys that no row of the item sees may be anything: they are
// zeroed, as are, in tiles where some row does not see some key, those of a key with an
// element that is not finite (a probability of 0 would make the rows that do not see it
// NaN).  The rows that do see it have a score of it that is not finite either: NaN or
// +inf make all of the row NaN; after -inf, which is a weight of 0, soften puts the NaN of 0
// times an infinite value back.
template <int C, bool FEW>
__device__ __forceinline__ void pass_v(const LatentAttnArgs& la, Shared& sh, uint8_t* vs) {
    using F = Cfg<C, FEW>;
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    Jobs jobs;
    Ring<2> at;
    bool dead = false;
    while (const Job* job = dead ? nullptr : jobs.next(sh, a)) {
        for (int j = 0; j < job->tiles; ++j, at.step()) {
            dead = !warp_wait(&sh.v_full[at.st], at.ph, a.err, a.timeout_ns);
            if (dead) break;
            const int j0 = job->key0(j), lo = max(job->it.lo, job->wlo), hi = min(job->it.hi, job->whi);
            if (j0 < lo || j0 + kKT > hi) {
                // a key's elements, 16 bytes a lane
                uint8_t* v = vs + at.st * F::kVBytes + (lane >> 3) * kAtom + (lane & 7) * 16;
                for (int r = warp; r < kKT; r += 4) {
                    uint4* p = reinterpret_cast<uint4*>(v + (r >> 3) * F::kVGroup + (r & 7) * 128);
                    bool bad = j0 + r < job->it.lo || j0 + r >= job->it.hi;
                    if (lane < 8 * F::kVPanels) bad = bad || any_nonfinite(*p);
                    if (__any_sync(0xFFFFFFFFu, bad) && lane < 8 * F::kVPanels) *p = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) arrive_first(&sh.v_ready[at.st]);
        }
        jobs.done(sh);
    }
}

// e4m3: 128 codes of a key, as read, to bf16 in the key's row of two atoms.  A NaN
// code comes out as `nan_bits`, which no other does; `zero` and, where it has NaN
// codes, `zero_nan` make the row zeros (see pass_v).
__device__ __forceinline__ void convert_row(const uint4 (&raw)[8], uint8_t* first, int r, uint32_t factor, uint32_t nan_bits, bool zero,
                                            bool zero_nan) {
    uint8_t* second = first + kAtom;
    uint32_t most = 0;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
        const uint32_t x[4] = {raw[ch].x, raw[ch].y, raw[ch].z, raw[ch].w};
        uint32_t y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // as e4m3x4_to_bf16, with the cache's power of two in the factor
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
    } else if (had_nan) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(i < 32 ? first : second) + (i & 31);
            uint32_t v = *w;
            if ((v & 0x7FFFu) == nan_bits) v |= 0x7FC0u;
            if ((v & 0x7FFF0000u) == nan_bits << 16) v |= 0x7FC00000u;
            *w = v;
        }
    }
}

// e4m3: four warps each for keys and values, a thread a key and 128 codes.  All codes
// are read before any atom is written over them.  Both run the same instructions, what
// differs are numbers: with a copy of their own each, 184 us for 145 (16 verify blocks
// over 4,099 to 16,411 rows), the softmax's, these and the products' no longer fitting the
// instruction caches.
template <int C, bool FEW>
__device__ __forceinline__ void convert(const LatentAttnArgs& la, Shared& sh, uint8_t* ring, const bool values) {
    using F = Cfg<C, FEW>;
    const int n = values ? kKT : kKeys, group = values ? F::kVGroup : F::kKGroup, units = values ? F::kVPanels / 2 : F::kParts;
    const int bytes = values ? F::kVBytes : F::kKBytes, stages = values ? 2 : F::kKStages, id = values ? kBarV : kBarK;
    static_assert(kKT * (F::kVPanels / 2) <= 128 && kKeys * F::kParts <= 128, "a row's part a thread");
    uint64_t* full = values ? sh.v_full : sh.k_full;
    uint64_t* ready = values ? sh.v_ready : sh.k_ready;
    const AttnArgs& a = la.a;
    const int lane = threadIdx.x & 31, t = threadIdx.x & 127, r = t & (n - 1), part = t / n;
    const uint32_t from = n / 8 * (group / 2) + (r >> 3) * (group / 2) + part * kAtom + (r & 7) * 128;
    const uint32_t to = (r >> 3) * group + 2 * part * kAtom + (r & 7) * 128;
    // 2^120 times the cache's power of two (see e4m3x4_to_bf16), and 480 times it
    const uint32_t f = static_cast<uint32_t>(127 + 120 + la.c.scale_log2) << 7, factor = f | (f << 16);
    const uint32_t nan_bits = 0x43F0u + static_cast<uint32_t>(la.c.scale_log2 * 128);
    Jobs jobs;
    int st = 0;
    uint32_t ph = 0, qp = 0;
    bool dead = false, q_ok = true;                              // (q: the first warp's)
    while (const Job* job = next_of_group(jobs, sh, a, id, dead || !q_ok)) {
#pragma unroll 1
        for (int j = 0; j < job->tiles; ++j) {
            uint8_t* stage = ring + st * bytes;
            const bool ok = mbar_wait(&full[st], ph, a.err, a.timeout_ns);
            uint4 raw[8];
            if (part < units) {
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) raw[ch] = *reinterpret_cast<const uint4*>(stage + from + ((ch ^ (r & 7)) << 4));
            }
            dead = !bar_and(id, ok && q_ok, 128);
            if (dead) break;
            if (part < units) {
                const int j0 = job->key0(j), key = j0 + r;
                convert_row(raw, stage + to, r, factor, nan_bits, values && (key < job->it.lo || key >= job->it.hi),
                            values && (j0 < job->wlo || j0 + kKT > job->whi));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive_first(&ready[st]);
            if (!values && j == 0 && t < 32) q_ok = pass_q(a, sh, qp);
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        jobs.done(sh);
    }
}

// --------------------------------------------------------------- products ----
// The MMA warp of the first CTA: Q K^T of a tile, then P V of the one before, so that
// one tile's softmax runs beside another's products.
template <int C, bool FEW>
__device__ __forceinline__ void multiply(const LatentAttnArgs& la, Shared& sh, uint8_t* qs, uint8_t* ps, uint8_t* ks, uint8_t* vs) {
    using F = Cfg<C, FEW>;
    constexpr uint32_t kIdQK = idesc(false, kKT), kIdPV = idesc(true, 256);
    const AttnArgs& a = la.a;
    const uint32_t colS = sh.tmem, colO = sh.tmem + kColO;
    const uint64_t qd = sdesc(smem_u32(qs), 16, 1024), pd = sdesc(smem_u32(ps), 16, 1024);
    const uint64_t kd = sdesc(smem_u32(ks), 16, F::kKGroup), rd = sdesc(smem_u32(ks) + F::kRope, 16, kAtom);
    const uint64_t vd = sdesc(smem_u32(vs), kAtom, F::kVGroup);
    Jobs jobs;
    Ring<F::kKStages> ka;                                        // K
    Ring<2> sa, pa;                                              // S; P and V
    uint32_t qp = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !warp_wait(bar, parity, a.err, a.timeout_ns);
    };
    while (const Job* job = dead ? nullptr : jobs.next(sh, a)) {
        const int T = job->tiles;
        if (T > 0) {
            wait(&sh.q_ready, qp);
            qp ^= 1u;
        }
        for (int i = 0; i <= T && T > 0 && !dead; ++i) {
            if (i < T) {
                wait(&sh.k_ready[ka.st], ka.ph);
                if (dead) break;
                tc_fence_after();
                if (elect_one()) {
                    // (bases and constants: each operand worked out on its own would cost as much as its product)
                    const uint64_t kk = kd + ka.st * (F::kKBytes >> 4), rr = rd + ka.st * (F::kKBytes >> 4);
#pragma unroll
                    for (int x = 0; x <= C / 64; ++x)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            pair_mma(colS + 32 * sa.st, qd + ((x * F::kQPanel + k * 32) >> 4),
                                     x < C / 64 ? kk + ((x * kAtom + k * 32) >> 4) : rr + (k * 32 >> 4), kIdQK, x > 0 || k > 0);
                    pair_commit(&sh.s_full[sa.st]);
                    pair_commit(&sh.k_empty[ka.st]);
                    if (i == T - 1) pair_commit(&sh.q_empty);
                }
                __syncwarp();
                ka.step();
                sa.step();
            }
            if (i > 0) {
                wait(&sh.v_ready[pa.st], pa.ph);
                wait(&sh.p_ready[pa.st], pa.ph);
                if (dead) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t pp = pd + pa.st * (F::kPBytes >> 4), vv = vd + pa.st * (F::kVBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int n = 0; n < F::kNV; ++n)
                            pair_mma(colO + 128 * n, pp + (k * 32 >> 4), vv + ((2 * n * kAtom + 2 * k * F::kVGroup) >> 4), kIdPV,
                                     i > 1 || k > 0);
                    pair_commit(&sh.v_empty[pa.st]);
                    pair_commit(&sh.pv_done[pa.st]);
                }
                __syncwarp();
                pa.step();
            }
        }
        jobs.done(sh);
    }
    // the products end before the accumulators are given back
    if (elect_one()) pair_commit(&sh.done);
    __syncwarp();
    mbar_wait(&sh.done, 0, a.err, kDrainNs);
}

// ---------------------------------------------------------------- softmax ----
// The CTA's rows of Q into shared memory where tokens have gaps between them (else one
// tensor copy does it, see produce), K-major with the 128-byte swizzle: a warp copies
// whole rows, all of its 16 on their way at once; rows past the last are zeros.
// (By registers, nine pieces a thread at a time, an item's start took 18,000 clocks.)
template <int C, bool FEW>
__device__ __forceinline__ void load_queries(const AttnArgs& a, const Item& it, int row0, int count, uint8_t* qs) {
    constexpr int kChunks = (C + kLatentRot) / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto place = [&](int r, int ch) { return qs + (ch >> 3) * Cfg<C, FEW>::kQPanel + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
#pragma unroll 4
    for (int r = warp; r < Cfg<C, FEW>::kHeld; r += 4) {
        const int row = row0 + min(r, count - 1), qi = a.query_of(row), hd = row - qi * a.group;
        const uint16_t* src = a.q + int64_t(it.s.q0 + qi) * a.q_stride + hd * (C + kLatentRot);
        const uint32_t bytes = r < count ? 16u : 0u;
#pragma unroll
        for (int ch = lane; ch < kChunks; ch += 32)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(r, ch))), "l"(src + 8 * ch), "r"(bytes)
                         : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_async_smem();
}

// Which of 32 elements are infinite or NaN, a bit each.
__device__ __forceinline__ uint32_t nonfinite32(const uint16_t* p) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(p + 8 * i);
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((x[k] & 0x7F80u) == 0x7F80u) bits |= 1u << (8 * i + 2 * k);
            if ((x[k] & 0x7F800000u) == 0x7F800000u) bits |= 2u << (8 * i + 2 * k);
        }
    }
    return bits;
}

// Of the elements d0 .. d0 + 31, those that are not finite in some key that a row sees in
// the tiles where pass_v zeroed such keys.
__device__ __noinline__ uint32_t lost_elements(const LatentAttnArgs& la, const Job& job, int lo, int hi, uint64_t draft, int d0) {
    const AttnArgs& a = la.a;
    const RowView view{lo, hi, draft};
    const int32_t* table = a.sq.table + int64_t(job.it.b) * a.sq.max_pages;
    uint32_t bits = 0;
    for (int t = 0; t < job.tiles; ++t) {
        const int j0 = job.key0(t);
        if (j0 >= job.wlo && j0 + kKT <= job.whi) continue;
        for (int j = max(j0, view.lo); j < min(j0 + kKT, view.hi); ++j) {
            if (!row_sees(view, a.draft != nullptr, job.it.s.first, j)) continue;
            const int page = table[j >> la.c.page_log2];
            if (page < 0 || page >= la.c.n_pages) continue;
            bits |= nonfinite32(reinterpret_cast<const uint16_t*>(la.c.latent) + page * la.c.lat_page +
                                (j & (la.c.page - 1)) * la.c.lat_token + d0);
        }
    }
    return bits;
}

template <int C, bool FEW, bool E4M3>
__device__ __forceinline__ void soften(const LatentAttnArgs& la, Shared& sh, uint8_t* qs, uint8_t* ps, int pair, uint32_t rank) {
    using F = Cfg<C, FEW>;
    const AttnArgs& a = la.a;
    const int tid = threadIdx.x, lr = tid & 63, half = tid >> 6, lane = tid & 31;
    const uint32_t tm = sh.tmem + (static_cast<uint32_t>(tid & 96) << 16);
    const uint32_t colO = tm + kColO;
    uint8_t* p_row = ps + lr * 128;
    const bool draft = a.draft != nullptr;
    Jobs jobs;
    uint32_t g = 0;                                              // tiles so far
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
        tc_fence_after();
    };
    auto wait_pv = [&](uint32_t tile) { wait(&sh.pv_done[tile & 1u], (tile >> 1) & 1u); };
    // log2 units a product: at least 1.2e-38 (an unseen key's -inf times it stays -inf), or NaN; the sign goes to the scores
    const float cs = a.scale * kLog2e;
    const float c = fmaxf(fabsf(cs), 1.2e-38f);
    while (const Job* job = next_of_group(jobs, sh, a, kBarSoft, __any_sync(0xFFFFFFFFu, dead))) {
        const Item& it = job->it;
        const int row0 = static_cast<int>(rank) * job->half, count = rank ? job->rows - job->half : job->half;
        const int T = job->tiles;
        const bool valid = lr < count, warp_on = __any_sync(0xFFFFFFFFu, valid);   // (both warps of 32 rows alike)
        const int r = it.rt * F::kItem + row0 + (valid ? lr : 0), qi = a.query_of(r), hd = r - qi * a.group;
        RowView view{0, 0, 0ull};
        if (valid) view = row_view(a, it.s, qi);
        if (T > 0 && !la.q_flat) {
            load_queries<C, FEW>(a, it, it.rt * F::kItem + row0, count, qs);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.q_full);
        }
        float ref = kNegInf, sum0 = 0.0f, sum1 = 0.0f;
        bool odd = false;                                        // (codes have no infinity)
        for (int j = 0; j < T; ++j, ++g) {
            const int j0 = job->key0(j);
            wait(&sh.s_full[g & 1u], (g >> 1) & 1u);
            if (warp_on) {
                float x[32];
                tmem_ld32(tm + 32 * (g & 1u), x);
                tmem_wait_ld();
                if (cs < 0.0f) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = -x[e];
                }
                if (j0 < job->wlo || j0 + kKT > job->whi) {
                    const uint32_t bits = row_bits(view, draft, it.s.first, j0 + half * kKeys);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        if (!E4M3) odd = odd || (((bits >> e) & 1u) && x[e] == kNegInf);
                        if (!((bits >> e) & 1u)) x[e] = kNegInf;
                    }
                }
                float m4[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int e = 0; e < 32; e += 4)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], x[e + k]);
                float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                sh.top[g & 1u][half][lr] = top;
                // powers by the reference so far, while the row's other half says its maximum: summed in
                // fp32, rounded to bf16 for the product with bf16 values (its range holds any power)
                uint32_t u[16];
                float s0, s1;
                auto powers = [&]() {
                    const float off = ref == kNegInf ? 0.0f : -ref;
                    s0 = sum0;
                    s1 = sum1;
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float p0, p1;
                        fma2_to(p0, p1, x[e], x[e + 1], c, off);
                        p0 = fast_exp2(p0);
                        p1 = fast_exp2(p1);
                        add2(s0, s1, p0, p1);
                        u[e / 2] = pack_bf16(p0, p1);
                    }
                };
                if (j > 0) powers();
                named_bar(kBarTop + ((tid >> 5) & 1), 64);
                top = fmaxf(top, sh.top[g & 1u][half ^ 1][lr]) * c;
                if (!(top > kNegInf)) top = kNegInf;                 // (NaN: the sums carry it)
                const bool grow = top > ref + kLag || (ref == kNegInf && top > kNegInf);
                if (__any_sync(0xFFFFFFFFu, grow) || j == 0) {
                    const float f = !grow ? 1.0f : (ref == kNegInf ? 0.0f : fast_exp2(ref - top));
                    sum0 *= f;
                    sum1 *= f;
                    if (grow) ref = top;
                    if (j > 0) {
                        wait_pv(g - 1);
#pragma unroll 1
                        for (int q = 0; q < F::kNV * 8; ++q) {
                            float o[16];
                            tmem_ld16(colO + 16 * q, o);
                            tmem_wait_ld();
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);   // (what is not finite stays so)
                            tmem_st16(colO + 16 * q, w);
                        }
                        tmem_wait_st();
                    }
                    powers();
                }
                sum0 = s0;
                sum1 = s1;
                // (P's room has been read: S of this tile came after P V of two before)
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    *reinterpret_cast<uint4*>(p_row + (g & 1u) * F::kPBytes + (((4 * half + ch) ^ (lr & 7)) << 4)) =
                        make_uint4(u[4 * ch], u[4 * ch + 1], u[4 * ch + 2], u[4 * ch + 3]);
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_first(&sh.p_ready[g & 1u]);
        }
        // --- the item's rows: normalised, or this pair's piece of them
        sh.sum[half][lr] = sum0 + sum1;
        if (!E4M3) sh.odd[half][lr] = odd;
        named_bar(kBarSoft, 128);
        const float sum = sh.sum[0][lr] + sh.sum[1][lr];
        if (!E4M3) odd = valid && (sh.odd[0][lr] | sh.odd[1][lr]) != 0;
        if (sum != sum) ref = fmaxf(ref, 0.0f);                  // a NaN is a result, not an empty row
        const bool piece = it.t0 > 0 || it.t1 < it.n;
        float* slot = a.partials + (int64_t(it.t0 == 0 ? 0 : kMaxPairs) + pair) * (kLatentRows * (C + 2));
        const int64_t at = int64_t(it.s.q0 + qi) * a.q_heads + hd;
        // a piece whose keys all have weight 0 still says where 0 times infinity is
        const float weight = T == 0 ? 0.0f : (piece ? 1.0f : (ref == kNegInf ? 0.0f : 1.0f / sum));
        if (valid && half == 0) {
            if (piece)
                *reinterpret_cast<float2*>(slot + kLatentRows * C + 2 * (row0 + lr)) = make_float2(ref, sum);
            else if (a.lse)
                a.lse[at] = ref == kNegInf ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
        if (T > 0) wait_pv(g - 1);
        if (warp_on) {
#pragma unroll 1
            for (int q = 0; q < F::kNV * 4; ++q) {
                float o[32];
                tmem_ld32(colO + 32 * q, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = weight != 0.0f ? o[e] * weight : 0.0f;
                const int d0 = half * (C / 2) + 32 * q;
                if (!E4M3 && odd && weight != 0.0f) {
                    const uint32_t lost = lost_elements(la, *job, view.lo, view.hi, view.draft, d0);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if ((lost >> e) & 1u) o[e] = __uint_as_float(0x7FFFFFFFu);
                }
                if (valid) {
                    if (piece) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4*>(slot + ((d0 / 4 + e) * kLatentRows + row0 + lr) * 4) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(a.out + at * C + d0 + 8 * e) =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();
        if (tid == 0 && rank == 0) note_split(a, it, job->rows, F::kItem, sh.plan, pair);
        jobs.done(sh);
    }
}

template <int C, bool FEW, bool E4M3>
__global__ void __launch_bounds__(kThreads<E4M3>, 1) latent_attn_kernel(const LatentAttnArgs la, const __grid_constant__ LatentMaps maps) {
    using F = Cfg<C, FEW>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    uint8_t* qs = dyn;
    uint8_t* ps = qs + F::kQBytes;
    uint8_t* ks = ps + 2 * F::kPBytes;
    uint8_t* vs = ks + F::kKStages * F::kKBytes;
    Shared& sh = *reinterpret_cast<Shared*>(dyn + F::kSmem);
    const AttnArgs& a = la.a;
    const int warp = threadIdx.x >> 5, pair = blockIdx.x >> 1;
    const uint32_t rank = cta_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::kKStages; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.k_ready[i], E4M3 ? 8 : 2);             // both CTAs' passing warps
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], 4 + 1 + (E4M3 ? 4 : 1) + 4 + (rank == 0 ? 1 : 0));   // softmax, values, passing on, MMA
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.v_ready[i], 8);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_ready[i], 8);
            mbar_init(&sh.pv_done[i], 1);
        }
        mbar_init(&sh.q_full, la.q_flat ? 1 : 4);                // the copy, or the softmax warps
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.q_ready, 2);
        mbar_init(&sh.done, 1);
        fence_barrier_init();
        prefetch_tensormap(&maps.keys);
        prefetch_tensormap(&maps.values);
        prefetch_tensormap(&maps.rope);
    }
    if (warp == 6) pair_alloc(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // both CTAs' barriers are there
    pdl_wait();
    pdl_launch_dependents();
    plan_work<F::kItem, kKT>(a, 1, sh.scan, &sh.plan, pair, gridDim.x >> 1, rank == 0);   // (its barriers publish sh.tmem)
    tc_fence_after();
    if (warp < 4)
        soften<C, FEW, E4M3>(la, sh, qs, ps, pair, rank);
    else if (warp == 4)
        produce<C, FEW, E4M3, false>(la, maps, sh, qs, ks, rank);
    else if (warp == 5) {
        if (rank == 0)
            multiply<C, FEW>(la, sh, qs, ps, ks, vs);
        else                                                     // (it has nothing else to do)
            zero_pad_rows(a, sh.plan.seqs, pair, gridDim.x >> 1, threadIdx.x & 31, 32);
    } else if (warp == 6)
        produce<C, FEW, E4M3, true>(la, maps, sh, qs, vs, rank);
    else if (warp >= 8) {
        if constexpr (E4M3) {
            convert<C, FEW>(la, sh, warp < 12 ? vs : ks, warp < 12);
        } else {
            pass_v<C, FEW>(la, sh, vs);
        }
    } else if (!E4M3) {
        pass_k<C, FEW>(la, sh);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // nothing of the pair is in flight
    tc_fence_after();
    if (warp == 6) {
        // the last commit's arrival, which the first CTA's MMA warp has seen in its own shared memory, in this CTA's too
        mbar_wait(&sh.done, 0, a.err, kDrainNs);
        __syncwarp();
        pair_dealloc(sh.tmem);
    }
}

template <int C, bool FEW, bool E4M3>
cudaError_t launch(const LatentAttnArgs& a, const LatentMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<C, FEW>::kSmem + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(latent_attn_kernel<C, FEW, E4M3>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int pairs = n_sms / 2 < kMaxPairs ? n_sms / 2 : kMaxPairs;
    e = launch_pdl_cluster(latent_attn_kernel<C, FEW, E4M3>, dim3(2 * pairs), dim3(kThreads<E4M3>), 2, smem, s, a, m);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pair_join<C, kLatentRows>(a.a, pairs, n_sms, s);
}

}  // namespace

cudaError_t launch_latent_attn(const LatentAttnArgs& a, const LatentMaps& m, bool few, int n_sms, cudaStream_t s) {
    if (a.c.dim == 512) {
        if (few) return a.c.e4m3 ? launch<512, true, true>(a, m, n_sms, s) : launch<512, true, false>(a, m, n_sms, s);
        return a.c.e4m3 ? launch<512, false, true>(a, m, n_sms, s) : launch<512, false, false>(a, m, n_sms, s);
    }
    if (few) return a.c.e4m3 ? launch<256, true, true>(a, m, n_sms, s) : launch<256, true, false>(a, m, n_sms, s);
    return a.c.e4m3 ? launch<256, false, true>(a, m, n_sms, s) : launch<256, false, false>(a, m, n_sms, s);
}

}  // namespace moe
