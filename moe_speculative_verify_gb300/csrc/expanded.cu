// expanded.cu -- attention of the expanded form of a latent cache's layer, on tensor
// memory of pairs of SMs (sm_103a): a head's key is a part of D elements of its own
// beside the 64 of the rotary part that the heads share, its values have D elements.
//
// An item is up to 512 query rows of one sequence and head, worked on by a cluster
// of two CTAs as two streams of 256 rows, 128 a CTA, over tiles of 128 keys:
//   S = Q K^T     one tcgen05.mma of the pair, M = 256, N = 128: each CTA holds its
//                 rows of Q and 64 of the keys;
//   softmax       of each stream by a warpgroup a CTA, a thread a row;
//   O += P V      M = 256, N = D, P from tensor memory: each CTA holds its rows of P,
//                 all keys' values of its half of D, and its rows of all of O.
// So a tile's keys and values are read by one CTA each (half by half), and one stream's
// products run while the other's softmax does.  Pairs, because their products run at
// the tensor core's full rate (256 x 128 x 16 in 64 clocks) where a single SM's from
// shared memory, 128 x 128 x 16, takes 102 for its 64.
//
// The reference of a row's sums lags as in attn_tile.cu.
#include "kernels.h"
#include "pair.cuh"

namespace moe {

namespace {

constexpr int kMT = kExpandedRows, kKT = kExpandedKeys;
constexpr int kStream = kMT / 2;         // rows of a stream
constexpr int kKeys = kKT / 2;           // keys of a CTA
constexpr int kPanel = 128 * 128;        // 128 rows of 64 elements
constexpr int kThreads = 384;            // 8 softmax warps; copies, an MMA warp a stream, one that passes on what landed
constexpr int kStages = 3;
// Registers a thread, moved between the warpgroups after the launch at 168:
// 8 * 208 + 4 * 80 = 1984 a lane column of the 12 * 168 = 2016 launched.
constexpr int kRegsSoft = 208, kRegsRest = 80;
constexpr int kAhead = 4;                // items that the copying warp may be ahead by
constexpr uint32_t kColO = 256;          // S/P of stream s at column 128 s, O at 256 + 128 s
constexpr float kLag = 8.0f;             // log2 of what powers may grow to

template <int D>
struct Cfg {
    static constexpr int kQBytes = (D / 64 + 1) * kPanel;        // of a stream: 128 rows
    static constexpr int kKPanel = kKeys * 128;
    static constexpr int kKBytes = (D / 64 + 1) * kKPanel;
    static constexpr int kVBytes = kPanel;                       // 128 keys, D / 2 elements used of 64
    static constexpr size_t kSmem = 2 * kQBytes + kStages * (kKBytes + kVBytes);   // then Shared
};

// An item as the CTA's warps work on it.  The copying warp walks the pair's items and
// queues them here; each other role takes its own way through the queue.
struct Job {
    Item it;
    int more;                // 0: none; no other field holds
    int rows;                // rows of the item
    int tiles;               // key tiles of this pair (0: nothing seen)
    int a[2], b[2];          // stream s takes local tiles a .. b-1
    int wlo[2], whi[2];      // keys that every row of the stream sees
    int lo_all, hi_all;      // and of the item

    __device__ __forceinline__ void set(const AttnArgs& at, const Item& it) {
        const int r0 = it.rt * kMT;
        const int n = min(kMT, it.s.nq - r0), m = it.hi > it.lo ? it.t1 - it.t0 : 0;
        const int2 all = rows_whole(at, it.s, r0, r0 + n - 1);
        rows = n;
        tiles = m;
        lo_all = all.x;
        hi_all = all.y;
        const int base = it.tile0 + it.t0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int i0 = r0 + s * kStream, i1 = min(i0 + kStream, r0 + n) - 1;
            a[s] = b[s] = 0;
            wlo[s] = whi[s] = 0;
            if (i1 < i0) continue;
            const int2 k = rows_range(at, it.s, i0, i1), w = rows_whole(at, it.s, i0, i1);
            wlo[s] = w.x;
            whi[s] = w.y;
            const int first = min(max(k.x / kKT - base, 0), m);
            a[s] = first;
            b[s] = k.y > k.x ? max(min((k.y + kKT - 1) / kKT - base, m), first) : first;
        }
    }
    __device__ __forceinline__ int first(int s) const { return s ? a[1] : a[0]; }
    __device__ __forceinline__ int last(int s) const { return s ? b[1] : b[0]; }
    __device__ __forceinline__ int key0(int tile) const { return (it.tile0 + it.t0 + tile) * kKT; }
};

struct Shared {
    int64_t scan[16];                       // plan_work's
    // of this CTA: what landed, and the room that both streams' products gave back
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t q_full[2], q_empty[2];
    // of the pair, in its first CTA: operands in place in both
    uint64_t k_ready[kStages], v_ready[kStages], q_ready[2], p_ready[2];
    // of this CTA: the pair's products are done
    uint64_t s_full[2], o_full[2], done[2];
    Plan plan;
    Job job[kAhead];
    uint64_t job_full[kAhead], job_empty[kAhead];
    uint32_t tmem;
    // by place in the queue: 1 + the last item that had values put right which are not finite.  Its
    // number only grows, so that nothing has to clear it: an item that finds that of a later
    // one in its place looks its own values over for nothing.
    int bad[kAhead];
};

struct Slot {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++st == kStages) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// A warp's way through the queue.
struct Jobs {
    int n = 0;
    __device__ __forceinline__ const Job* next(Shared& sh, const AttnArgs& a) {
        if (!warp_wait(&sh.job_full[n % kAhead], (n / kAhead) & 1, a.err, a.timeout_ns)) return nullptr;
        const Job* j = &sh.job[n % kAhead];
        return j->more ? j : nullptr;
    }
    // by one thread of the warp, once all have read what they need of the item
    __device__ __forceinline__ void done(Shared& sh) { mbar_arrive(&sh.job_empty[n % kAhead]); }
};

// The warp that copies: this CTA's 64 keys of each tile, then its half of the tile's
// values; an item's queries after its first tile, as soon as the last one's have been
// used, beside that item's end.  Rows past the sequence's are read as they lie there,
// or as zeros past the last.
template <int D>
__device__ __forceinline__ void produce(const ExpandedArgs& x, const ExpandedMaps& maps, Shared& sh, uint8_t* qs, uint8_t* ks, uint8_t* vs,
                                        int rank) {
    using F = Cfg<D>;
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 31;
    Walk<kMT, kKT> walk;                                         // every lane's own, in registers
    walk.start(a, sh.plan);
    Slot at;
    int uses = 0, used[2] = {0, 0};                              // tiles begun; items of a stream
    bool dead = false;
    for (int n = 0;; ++n) {
        Job& job = sh.job[n % kAhead];
        dead = dead || !warp_wait(&sh.job_empty[n % kAhead], ((n / kAhead) & 1) ^ 1, a.err, a.timeout_ns);
        if (dead) break;                                         // (the others' waits for it run out too)
        Item next;
        const bool more = walk.next(a, next);
        if (lane == 0) {
            job.more = more;
            if (more) {
                job.it = next;
                job.set(a, next);
            }
            mbar_arrive(&sh.job_full[n % kAhead]);
        }
        __syncwarp();
        if (!more) break;
        const Item& it = job.it;
        const int64_t k0 = x.cu_k[it.b];
        if (lane == 0 && (k0 < 0 || k0 + it.s.len > x.n_keys)) record_error(a.err, MOE_ERR_INVALID_ARG);
        for (int j = 0; j < job.tiles && !dead; ++j) {
            // (a place far outside stays outside, whatever 32 bits make of the sum)
            const int row = static_cast<int>(min(max(k0 + job.key0(j), int64_t(-(1 << 30))), int64_t(x.n_keys)));
            dead = !warp_wait(&sh.k_empty[at.st], at.ph ^ 1u, a.err, a.timeout_ns);
            if (dead) break;
            if (lane == 0) {
                uint8_t* k = ks + at.st * F::kKBytes;
                mbar_arrive_expect_tx(&sh.k_full[at.st], F::kKBytes);
                tma_load_4d(k, &maps.k, &sh.k_full[at.st], 0, row + rank * kKeys, 0, it.h);
                tma_load_2d(k + (D / 64) * F::kKPanel, &maps.rope, &sh.k_full[at.st], 0, row + rank * kKeys);
            }
            __syncwarp();
            dead = !warp_wait(&sh.v_empty[at.st], at.ph ^ 1u, a.err, a.timeout_ns);
            if (dead) {                                          // this stage's K alone
                mbar_wait(&sh.k_full[at.st], at.ph, a.err, kDrainNs);
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&sh.v_full[at.st], F::kVBytes);
                tma_load_3d(vs + at.st * F::kVBytes, &maps.v, &sh.v_full[at.st], rank * (D / 2), row, it.h);
            }
            __syncwarp();
            at.step();
            ++uses;
            for (int s = 0; s < 2 && j == 0; ++s) {
                if (job.last(s) <= job.first(s)) continue;
                dead = dead || !warp_wait(&sh.q_empty[s], (used[s] & 1) ^ 1, a.err, a.timeout_ns);
                if (dead) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_full[s], F::kQBytes);
                    tma_load_4d(qs + s * F::kQBytes, &maps.q, &sh.q_full[s], 0, it.s.q0 + it.rt * kMT + s * kStream + rank * 128, 0, it.h);
                }
                __syncwarp();
                ++used[s];
            }
        }
    }
    // the last copies
    for (int st = 0; st < kStages; ++st) {
        const int n = (uses + kStages - 1 - st) / kStages;
        if (n > 0) {
            mbar_wait(&sh.k_full[st], (n - 1) & 1, a.err, kDrainNs);
            mbar_wait(&sh.v_full[st], (n - 1) & 1, a.err, kDrainNs);
        }
    }
    for (int s = 0; s < 2; ++s)
        if (used[s] > 0) mbar_wait(&sh.q_full[s], (used[s] - 1) & 1, a.err, kDrainNs);
}

// Of a pair of bf16: bits 15 and 31 are set where one is not finite (its exponent
// carries into them), and the pair with such as zeros.
__device__ __forceinline__ uint32_t carry2(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    const uint32_t n = carry2(w);
    return w & ((n & 0x8000u ? 0u : 0xFFFFu) | (n & 0x80000000u ? 0u : 0xFFFF0000u));
}

// Puts a tile's values right, keys from j0 on of which the item's rows see see0 .. see1 - 1 and
// all of them wlo .. whi - 1: where some row does not see some key, elements that are not
// finite become zeros (a probability of 0 would make them NaN for that row).  The rows
// that do see such a key get them when the item ends.
__device__ __forceinline__ void mend_values(Shared& sh, int item, uint8_t* tile, int j0, int see0, int see1, int wlo, int whi) {
    if (j0 >= max(see0, wlo) && j0 + kKT <= min(see1, whi)) return;
    // 16 bytes of eight keys at a time: in all but few tiles all is finite and nothing to be put right
    const int lane = threadIdx.x & 31;
    uint8_t* v = tile + lane * 16;
    uint32_t odd = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < kKT / 4; e0 += 8) {
        uint4 w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = *reinterpret_cast<const uint4*>(v + (e0 + e) * 512);
#pragma unroll
        for (int e = 0; e < 8; ++e) odd |= carry2(w[e].x) | carry2(w[e].y) | carry2(w[e].z) | carry2(w[e].w);
    }
    if (!__any_sync(0xFFFFFFFFu, (odd & 0x80008000u) != 0)) return;
    bool any = false;
#pragma unroll 1
    for (int e = 0; e < kKT / 4; ++e) {
        const int key = j0 + (lane >> 3) + 4 * e;
        uint4* p = reinterpret_cast<uint4*>(v + e * 512);
        const uint4 w = *p;
        if (((carry2(w.x) | carry2(w.y) | carry2(w.z) | carry2(w.w)) & 0x80008000u) == 0) continue;
        *p = make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
        any = any || (key >= see0 && key < see1);
    }
    if (any) {                                                   // in both CTAs: each has all columns of its rows
        for (uint32_t r = 0; r < 2; ++r)
            asm volatile("{\n\t.reg .b32 p;\n\tmapa.shared::cluster.u32 p, %0, %1;\n\tst.shared::cluster.u32 [p], %2;\n\t}" ::"r"(
                             smem_u32(&sh.bad[item % kAhead])),
                         "r"(r), "r"(item + 1)
                         : "memory");
        asm volatile("fence.acq_rel.cluster;" ::: "memory");
    }
    fence_async_smem();
    __syncwarp();
}

// The warp that tells the first CTA, whose MMA warps wait for both, what landed here.
template <int D>
__device__ __forceinline__ void pass_on(const ExpandedArgs& x, Shared& sh, uint8_t* vs) {
    using F = Cfg<D>;
    const AttnArgs& a = x.a;
    const int lane = threadIdx.x & 31;
    Slot at;
    Jobs jobs;
    uint32_t qp[2] = {0, 0};
    bool dead = false;
    while (const Job* job = dead ? nullptr : jobs.next(sh, a)) {
        for (int j = 0; j < job->tiles; ++j, at.step()) {
            dead = !warp_wait(&sh.k_full[at.st], at.ph, a.err, a.timeout_ns);
            if (dead) break;
            if (lane == 0) arrive_first(&sh.k_ready[at.st]);
            dead = !warp_wait(&sh.v_full[at.st], at.ph, a.err, a.timeout_ns);
            if (dead) break;
            mend_values(sh, jobs.n, vs + at.st * F::kVBytes, job->key0(j), job->it.lo, job->it.hi, job->lo_all, job->hi_all);
            if (lane == 0) arrive_first(&sh.v_ready[at.st]);
            for (int s = 0; s < 2 && j == 0; ++s) {
                if (job->last(s) <= job->first(s)) continue;
                dead = dead || !warp_wait(&sh.q_full[s], s ? qp[1] : qp[0], a.err, a.timeout_ns);
                if (lane == 0 && !dead) arrive_first(&sh.q_ready[s]);
                qp[s] ^= 1u;
            }
            if (dead) break;
        }
        __syncwarp();
        if (lane == 0) jobs.done(sh);
        ++jobs.n;
    }
}

// The MMA warp of stream s, in the first CTA.  The streams go their own ways, through
// items too; a burst is PV of a tile, then QK of the next (which writes S over that
// P).  A warp's waits run beside the other's burst.  (Bursts in strict turns left the one
// stream waiting for the other's last tiles under a causal mask, and both for each
// other's items: 573 us for 4 ragged chunks of 64 heads where this takes 522; a lock
// about a burst 552.)
template <int D>
__device__ __forceinline__ void multiply(const ExpandedArgs& x, Shared& sh, uint8_t* qs, uint8_t* ks, uint8_t* vs, int s) {
    using F = Cfg<D>;
    constexpr uint32_t kM256 = static_cast<uint32_t>(128 >> 4) << 24;   // beyond idesc's M = 128
    constexpr uint32_t kIdQK = idesc(false, kKT) + kM256, kIdPV = idesc(true, D) + kM256;
    const AttnArgs& a = x.a;
    const uint32_t colS = sh.tmem + 128 * s, colO = sh.tmem + kColO + 128 * s;
    const uint64_t qd = sdesc(smem_u32(qs + s * F::kQBytes), 16, 1024);
    const uint64_t kd = sdesc(smem_u32(ks), 16, 1024), vd = sdesc(smem_u32(vs), kPanel, 1024);
    Slot ka, va;
    Jobs jobs;
    uint32_t qp = 0, pp = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !warp_wait(bar, parity, a.err, a.timeout_ns);
    };
    while (const Job* job = dead ? nullptr : jobs.next(sh, a)) {
        const int T = job->tiles, a0 = job->first(s), b0 = job->last(s);
        if (b0 > a0) {
            wait(&sh.q_ready[s], qp);
            qp ^= 1u;
        }
        for (int i = 0; i <= T && T > 0; ++i) {
            const bool do_v = i > a0 && i <= b0, do_k = i >= a0 && i < b0, has_v = i > 0, has_k = i < T;
            const int vst = va.st, kst = ka.st;
            if (has_v) {
                wait(&sh.v_ready[vst], va.ph);
                va.step();
            }
            if (has_k) {
                wait(&sh.k_ready[kst], ka.ph);
                ka.step();
            }
            if (do_v) {
                wait(&sh.p_ready[s], pp);
                pp ^= 1u;
            }
            tc_fence_after();
            // (a base and constants: each operand worked out on its own would cost as much as its product)
            const uint64_t kk = kd + kst * (F::kKBytes >> 4), vv = vd + vst * (F::kVBytes >> 4);
            const uint32_t more = i - 1 > a0;
            if (elect_one() && !dead) {
                if (do_v) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) pair_mma_ts(colO, colS + 8 * k, vv + (k * 2048 >> 4), kIdPV, k > 0 ? 1u : more);
                    if (i == b0) pair_commit(&sh.o_full[s]);
                }
                if (has_v) pair_commit(&sh.v_empty[vst]);
                if (do_k) {
#pragma unroll
                    for (int k = 0; k < D / 16 + 4; ++k)
                        pair_mma(colS, qd + (((k >> 2) * kPanel + (k & 3) * 32) >> 4),
                                 kk + (((k >> 2) * F::kKPanel + (k & 3) * 32) >> 4), kIdQK, k > 0);
                    pair_commit(&sh.s_full[s]);
                    if (i == b0 - 1) pair_commit(&sh.q_empty[s]);
                }
                if (has_k) pair_commit(&sh.k_empty[kst]);
            }
            __syncwarp();
        }
        if ((threadIdx.x & 31) == 0) jobs.done(sh);
        ++jobs.n;
    }
    // the products end before the accumulators are given back
    if (elect_one()) pair_commit(&sh.done[s]);
    __syncwarp();
    mbar_wait(&sh.done[s], 0, a.err, kDrainNs);
}

// What a softmax thread carries through an item: its row's reference (log2 units)
// and sum of powers, in two parts.
struct RowState {
    float ref, sum0, sum1;
};

__device__ __forceinline__ float max32(const float (&x)[32]) {
    float t[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
    for (int e = 0; e < 32; e += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = fmaxf(t[k], fmaxf(x[e + 2 * k], x[e + 2 * k + 1]));
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// Takes a tile's maximum into the reference, and O with it where the reference moves
// (its products are complete: S came after them in the MMA thread's order).
template <int D>
__device__ __forceinline__ void follow(uint32_t colO, float top, bool started, RowState& st) {
    if (!(top > kNegInf)) top = kNegInf;                         // (NaN: the sums carry it)
    const bool grow = top > st.ref + kLag || (st.ref == kNegInf && top > kNegInf);
    if (started && __any_sync(0xFFFFFFFFu, grow)) {
        const float f = !grow ? 1.0f : (st.ref == kNegInf ? 0.0f : fast_exp2(st.ref - top));
        st.sum0 *= f;
        st.sum1 *= f;
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
            float o[16];
            tmem_ld16(colO + 16 * q, o);
            tmem_wait_ld();
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);   // (what is not finite stays so)
            tmem_st16(colO + 16 * q, u);
        }
    }
    if (grow) st.ref = top;
}

// 32 scores to powers: summed in fp32, rounded to bf16 (the products' type, whose
// range holds any power), stored as P of their keys: 16 columns of pairs.
__device__ __forceinline__ void powers(uint32_t colP, const float (&x)[32], float c, float off, RowState& st) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float p0, p1;
        fma2_to(p0, p1, x[e], x[e + 1], c, off);
        p0 = fast_exp2(p0);
        p1 = fast_exp2(p1);
        add2(st.sum0, st.sum1, p0, p1);
        u[e / 2] = pack_bf16(p0, p1);
    }
    tmem_st16(colP, u);
}

// Tells the MMA warp of the P stored so far.
__device__ __forceinline__ void hand_over(uint64_t* bar) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_first(bar);
}

// Adds to a thread's row, as it was written, the values that are not finite, of the keys
// lo .. hi - 1 in the tiles where mend_values takes such out: a piece's sums, or the output.  By
// all of a warp, 32 keys at a time: a lane reads a key, and says of each element which
// infinity it is (a NaN is both); a row takes what the keys say that it sees.  (One such
// value in a call of 0.18 ms makes it 0.25, all of them 1.1.  Each thread its own keys, element by
// element, took 1.2 ms an item of 512 rows.  On the sums in registers, before
// they are written, the code beside the main loop cost 4 ragged chunks of 64 heads 25 of
// 531 us.)
template <int D>
__device__ __noinline__ void add_nonfinite(const ExpandedArgs& x, const Job& job, int lo, int hi, float* sums, uint16_t* out) {
    const int lane = threadIdx.x & 31;
    const int64_t k0 = x.cu_k[job.it.b];
    uint32_t up[D / 32] = {}, down[D / 32] = {};                 // the row's infinities, a bit an element
#pragma unroll 1
    for (int j0 = job.key0(0); j0 < job.key0(job.tiles); j0 += 32) {
        const int tile = j0 - j0 % kKT, j = j0 + lane;
        if (tile >= max(job.it.lo, job.lo_all) && tile + kKT <= min(job.it.hi, job.hi_all)) continue;
        const bool there = j >= job.it.lo && j < job.it.hi && k0 + j >= 0 && k0 + j < x.n_keys;
        const uint4* v = reinterpret_cast<const uint4*>(x.v + (there ? (k0 + j) * x.v_token : 0) + job.it.h * x.v_head);
        const int l = min(max(lo - j0, 0), 32), h = min(max(hi - j0, 0), 32);
        const uint32_t seen = l >= h ? 0u : (0xFFFFFFFFu << l) & (0xFFFFFFFFu >> (32 - h));
        uint4 w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) w[i] = there ? v[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint32_t odd = carry2(w[i].x) | carry2(w[i].y) | carry2(w[i].z) | carry2(w[i].w);
            if (!__any_sync(0xFFFFFFFFu, (odd & 0x80008000u) != 0)) continue;
            const uint32_t p[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t n = (p[e / 2] >> (16 * (e & 1))) & 0xFFFFu, bit = 1u << ((8 * i + e) & 31);
                const bool bad = (n & 0x7F80u) == 0x7F80u, nan = (n & 0x7Fu) != 0;
                if (__ballot_sync(0xFFFFFFFFu, bad && (nan || n < 0x8000u)) & seen) up[i / 4] |= bit;
                if (__ballot_sync(0xFFFFFFFFu, bad && (nan || n >= 0x8000u)) & seen) down[i / 4] |= bit;
            }
        }
    }
#pragma unroll
    for (int d = 0; d < D; d += 4) {
        const uint32_t u = up[d / 32] >> (d & 31), n = down[d / 32] >> (d & 31);
        if (((u | n) & 15u) == 0) continue;
        float add[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) add[e] = ((u >> e) & 1u ? INFINITY : 0.0f) + ((n >> e) & 1u ? -INFINITY : 0.0f);
        if (sums) {
            float4* at = reinterpret_cast<float4*>(sums + d * kMT);
            const float4 o = *at;
            *at = make_float4(o.x + add[0], o.y + add[1], o.z + add[2], o.w + add[3]);
        } else {
            uint2* at = reinterpret_cast<uint2*>(out + d);
            const uint2 o = *at;
            *at = make_uint2(pack_bf16(bf16_bits_to_f32(o.x & 0xFFFFu) + add[0], __uint_as_float(o.x & 0xFFFF0000u) + add[1]),
                             pack_bf16(bf16_bits_to_f32(o.y & 0xFFFFu) + add[2], __uint_as_float(o.y & 0xFFFF0000u) + add[3]));
        }
    }
    __syncwarp();
}

template <int D>
__device__ __forceinline__ void soften(const ExpandedArgs& xa, Shared& sh, int pair, int rank) {
    const AttnArgs& a = xa.a;
    const int tid = threadIdx.x, s = tid >> 7, lr = tid & 127;
    const uint32_t tm = sh.tmem + (static_cast<uint32_t>(tid & 96) << 16);
    const uint32_t colS = tm + 128 * s, colO = tm + kColO + 128 * s;
    Jobs jobs;
    uint32_t sp = 0, op = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
        tc_fence_after();
    };
    // log2 units a product: at least 1.2e-38 (an unseen key's -inf times it stays -inf); the sign goes to the scores
    const float cs = a.scale * kLog2e;
    const float c = fmaxf(fabsf(cs), 1.2e-38f);
    while (const Job* job = jobs.next(sh, a)) {
        const Item& it = job->it;
        const int row0 = s * kStream + rank * 128, count = min(max(job->rows - row0, 0), 128);
        const int t0 = job->first(s), n = job->last(s) - t0;
        const int wlo = s ? job->wlo[1] : job->wlo[0], whi = s ? job->whi[1] : job->whi[0];
        const bool valid = lr < count, warp_on = __any_sync(0xFFFFFFFFu, valid);
        const int qi = it.rt * kMT + row0 + (valid ? lr : 0);
        RowView view{0, 0, 0ull};
        if (valid) view = row_view(a, it.s, qi);
        RowState st{kNegInf, 0.0f, 0.0f};
        for (int i = 0; i < n; ++i) {
            const int j0 = job->key0(t0 + i);
            wait(&sh.s_full[s], sp);
            sp ^= 1u;
            if (warp_on) {
                const bool whole = j0 >= wlo && j0 + kKT <= whi;
                float x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32(colS + 32 * q, x[q]);
                tmem_wait_ld();
                if (cs < 0.0f) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[q][e] = -x[q][e];
                }
                if (!whole) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t bits = row_bits(view, false, it.s.first, j0 + 32 * q);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) x[q][e] = kNegInf;
                    }
                }
                const float top = fmaxf(fmaxf(max32(x[0]), max32(x[1])), fmaxf(max32(x[2]), max32(x[3])));
                follow<D>(colO, top * c, i > 0, st);
                const float off = st.ref == kNegInf ? 0.0f : -st.ref;
                powers(colS, x[0], c, off, st);
                powers(colS + 16, x[1], c, off, st);
                powers(colS + 32, x[2], c, off, st);
                powers(colS + 48, x[3], c, off, st);
            }
            hand_over(&sh.p_ready[s]);
        }
        // --- the item's rows: normalised, or this pair's piece of them
        const float sum = st.sum0 + st.sum1;
        float ref = st.ref;
        if (sum != sum) ref = fmaxf(ref, 0.0f);                  // a NaN is a result, not an empty row
        const bool piece = it.t0 > 0 || it.t1 < it.n;
        float* slot = a.partials + (int64_t(it.t0 == 0 ? 0 : kMaxPairs) + pair) * (kMT * (D + 2));
        const int64_t at = int64_t(it.s.q0 + qi) * a.q_heads + it.h;
        // a piece whose keys all have weight 0 still says where 0 times infinity is
        const float weight = n == 0 ? 0.0f : (piece ? 1.0f : (ref == kNegInf ? 0.0f : 1.0f / sum));
        if (valid) {
            if (piece)
                *reinterpret_cast<float2*>(slot + kMT * D + 2 * (row0 + lr)) = make_float2(ref, sum);
            else if (a.lse)
                a.lse[at] = ref == kNegInf ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
        if (n > 0) {
            wait(&sh.o_full[s], op);
            op ^= 1u;
        }
        const bool bad = __any_sync(0xFFFFFFFFu, *const_cast<volatile int*>(&sh.bad[jobs.n % kAhead]) > jobs.n);
        if (warp_on) {
            float o[D / 32][32];
#pragma unroll
            for (int q = 0; q < D / 32; ++q) tmem_ld32(colO + 32 * q, o[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[q][e] = weight != 0.0f ? o[q][e] * weight : 0.0f;
                if (valid) {
                    if (piece) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4*>(slot + ((8 * q + e) * kMT + row0 + lr) * 4) =
                                make_float4(o[q][4 * e], o[q][4 * e + 1], o[q][4 * e + 2], o[q][4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(a.out + at * D + 32 * q + 8 * e) =
                                make_uint4(pack_bf16(o[q][8 * e], o[q][8 * e + 1]), pack_bf16(o[q][8 * e + 2], o[q][8 * e + 3]),
                                           pack_bf16(o[q][8 * e + 4], o[q][8 * e + 5]), pack_bf16(o[q][8 * e + 6], o[q][8 * e + 7]));
                    }
                }
            }
            if (bad)
                add_nonfinite<D>(xa, *job, view.lo, valid && weight != 0.0f ? view.hi : 0, piece ? slot + (row0 + lr) * 4 : nullptr,
                                 a.out + at * D);
        }
        tc_fence_before();
        if (tid == 0 && rank == 0) note_split(a, it, job->rows, kMT, sh.plan, pair);
        __syncwarp();
        if ((tid & 31) == 0) jobs.done(sh);
        ++jobs.n;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const ExpandedArgs x, const __grid_constant__ ExpandedMaps maps) {
    using F = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t dyn[];
    uint8_t* qs = dyn;
    uint8_t* ks = qs + 2 * F::kQBytes;
    uint8_t* vs = ks + kStages * F::kKBytes;
    Shared& sh = *reinterpret_cast<Shared*>(dyn + F::kSmem);
    const AttnArgs& a = x.a;
    const int warp = threadIdx.x >> 5, pair = blockIdx.x >> 1, rank = static_cast<int>(cta_rank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.k_empty[i], 2);                        // both streams' products
            mbar_init(&sh.v_empty[i], 2);
            mbar_init(&sh.k_ready[i], 2);                        // both CTAs' passing warps
            mbar_init(&sh.v_ready[i], 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.q_full[s], 1);
            mbar_init(&sh.q_empty[s], 1);
            mbar_init(&sh.q_ready[s], 2);
            mbar_init(&sh.p_ready[s], 8);
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.done[s], 1);
        }
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&sh.job_full[i], 1);
            mbar_init(&sh.job_empty[i], 8 + 1 + (rank == 0 ? 2 : 0));   // softmax warps, passing on, MMA
        }
        for (int i = 0; i < kAhead; ++i) sh.bad[i] = 0;
        fence_barrier_init();
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.rope);
        prefetch_tensormap(&maps.v);
    }
    if (warp == 8) pair_alloc(&sh.tmem);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // both CTAs' barriers are there
    pdl_wait();
    pdl_launch_dependents();
    plan_work<kMT, kKT>(a, 1, sh.scan, &sh.plan, pair, gridDim.x >> 1, rank == 0);   // (its barriers publish sh.tmem)
    tc_fence_after();
    zero_pad_rows(a, sh.plan.seqs);
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        soften<D>(x, sh, pair, rank);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == 8)
            produce<D>(x, maps, sh, qs, ks, vs, rank);
        else if (warp == 11)
            pass_on<D>(x, sh, vs);
        else if (rank == 0)
            multiply<D>(x, sh, qs, ks, vs, warp - 9);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                              // nothing of the pair is in flight
    tc_fence_after();
    if (warp == 8) {
        // the last commits' arrivals, which the first CTA's MMA warps have seen in its own shared memory, in this CTA's too
        for (int s = 0; s < 2; ++s) mbar_wait(&sh.done[s], 0, a.err, kDrainNs);
        __syncwarp();
        pair_dealloc(sh.tmem);
    }
}

template <int D>
cudaError_t launch(const ExpandedArgs& a, const ExpandedMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<D>::kSmem + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(expanded_kernel<D>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int pairs = n_sms / 2 < kMaxPairs ? n_sms / 2 : kMaxPairs;
    e = launch_pdl_cluster(expanded_kernel<D>, dim3(2 * pairs), dim3(kThreads), 2, smem, s, a, m);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_pair_join<D, kMT>(a.a, pairs, n_sms, s);
}

}  // namespace

cudaError_t launch_expanded(const ExpandedArgs& a, const ExpandedMaps& m, int n_sms, cudaStream_t s) {
    return a.dim == 128 ? launch<128>(a, m, n_sms, s) : launch<64>(a, m, n_sms, s);
}

}  // namespace moe
