// attn_tile.cu -- paged attention on tensor memory (sm_103a): verify blocks of
// many heads per kv head, and prefill chunks.
//
// An item is up to 256 query rows of one sequence and kv head, worked on as
// two streams of 128-row tiles.  Above 128 rows the streams are the two row
// tiles, which share every K and V tile; up to 128 rows both hold the same
// rows and take alternate key tiles, and are joined when the item ends; with
// 64 (or 32) rows or fewer the rows are repeated in the tile's other lanes,
// and each copy takes its half (quarter) of a tile's keys through the softmax,
// so all eight warps work on few rows too.  Each
// stream's step is S = Q K^T (tcgen05.mma, shared x shared), the softmax of a
// warpgroup with a thread per row, and O += P V (P from tensor memory), so one
// stream's products run while the other's softmax does.
//
// A row's sums use a reference that follows the running maximum only when
// that has grown by more than 2^kLag: the rescaling of O in tensor memory is
// rare then, and every power stays within the 16-bit types.
//
// e4m3 tiles are turned to bf16 in shared memory (exactly) by a warpgroup of
// their own, once for all of an item's rows, and multiplied as a bf16 cache's:
// queries keep their bits, and a probability its 8 bits at any size.  (8-bit
// products with a probability as two codes, which need no conversion, lose
// probabilities far below a row's largest: behind a first key that takes most
// of the weight the output was 10 % off.)
//
// Measured (64 query heads, 8 kv heads of 128): 2048 tokens over 16,384 keys
// more 0.80 ms in bf16, 1.46 PFLOP/s where the library's matrix product runs at
// 1.91 (a step's two products leave the tensor pipe idle between bursts, see
// multiply), 1.00 ms over e4m3 (the conversion's instructions); 16 verify blocks of
// up to 8 tokens over 4,099 to 16,411 keys 128 us in bf16 (4.9 TB/s), 139 over e4m3
// (2.3 TB/s: a stage is filled, converted and used in turn); one block over 6,011
// keys 21.6 us, over e4m3 24.0.
#include "attn_mma.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMT = 256;                 // rows of an item
constexpr int kKT = 128;                 // keys of a tile
// 2 softmax warpgroups; TMA warp, 2 MMA warps and an idle one; e4m3: a warpgroup that converts
template <bool E4M3>
constexpr int kThreads = E4M3 ? 512 : 384;
// Registers a thread, moved between the warpgroups after the launch at 168:
// 8 * 208 + 4 * 80 = 1984 a lane column of the 12 * 168 = 2016 launched; with
// the converting warps, launched at 128: 8 * 192 + 8 * 64 = 2048 of 16 * 128.
template <bool E4M3>
constexpr int kRegsSoft = E4M3 ? 192 : 208;
template <bool E4M3>
constexpr int kRegsRest = E4M3 ? 64 : 80;
constexpr int kSoft = 256;
constexpr int kBarAll = 1, kBarGroup = 2, kBarMma = 4;   // named barriers: both warpgroups, each, the MMA warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;          // S/P of stream s at column 128 s, O at 256 + 128 s

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kTileBytes = kKT * 2 * D;                 // bf16
    // e4m3: the tile as it is cached lands kRaw bytes into its stage: at D = 128
    // the upper half, whose rows are also those of the bf16 tile's elements 64 on
    static constexpr int kRaw = E4M3 ? 16384 : 0;
    static constexpr int kStageBytes = E4M3 && D == 64 ? kTileBytes + kKT * D : kTileBytes;
    static constexpr int kQBytes = 128 * 2 * D;
    static constexpr int kStages = D == 128 || E4M3 ? 5 : 10;
    static constexpr int kMerge = 128 * D * 4;                     // == 2 * kQBytes: stream 1's O
    static constexpr size_t kSmem = 2 * kQBytes + kStages * kStageBytes;   // then Shared
};

constexpr float kLag = 8.0f;             // log2 of what powers may grow to

// An item as its CTA works on it: mode, tiles, and each stream's share.
struct Share {
    int pair;                // two row tiles; else alternate key tiles of one
    int rows;                // rows of the item
    int tiles;               // key tiles of this CTA (0: nothing seen)
    int a[2], b[2];          // pair: stream s takes local tiles a .. b-1
    int wlo[2], whi[2];      // keys that every row of the stream sees

    __device__ __forceinline__ void set(const AttnArgs& at, const Item& it) {
        rows = min(kMT, it.s.nq * at.group - it.rt * kMT);
        pair = rows > 128;
        tiles = it.hi > it.lo ? it.t1 - it.t0 : 0;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r0 = it.rt * kMT + (pair ? 128 * s : 0);
            const int r1 = pair ? min(r0 + 128, it.rt * kMT + rows) : r0 + rows;
            const int i0 = at.query_of(r0), i1 = at.query_of(r1 - 1);
            const int2 k = rows_range(at, it.s, i0, i1), w = rows_whole(at, it.s, i0, i1);
            wlo[s] = w.x;
            whi[s] = w.y;
            a[s] = 0;
            b[s] = tiles;
            if (pair) {
                const int base = it.tile0 + it.t0;
                a[s] = min(max(k.x / kKT - base, 0), tiles);
                b[s] = k.y > k.x ? max(min((k.y + kKT - 1) / kKT - base, tiles), a[s]) : a[s];
            }
        }
    }
    // tiles of stream s, and its n-th
    __device__ __forceinline__ int count(int s) const {
        return pair ? (s ? b[1] - a[1] : b[0] - a[0]) : (tiles + 1 - s) / 2;
    }
    __device__ __forceinline__ int tile(int s, int n) const { return pair ? (s ? a[1] : a[0]) + n : 2 * n + s; }
};

// A role's place in the CTA's work (a softmax warpgroup's, the TMA warp's, the
// MMA warps'), kept in shared memory so that it takes no registers from the
// loops over the tiles.  THREADS threads share it, at named barrier `bar`.
struct Ctx {
    Walk<kMT, kKT> wk;
    Item it;
    Share sr;
    int more;

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
            if (more) sr.set(a, it);
        }
        sync<THREADS>(bar);
        return more != 0;
    }
};

struct Shared {
    alignas(16) float2 ml[2][128];          // a lane's reference and sum, among a row's sharers
    uint64_t kv_full[10];                   // e4m3: from kStages on, those of the tiles as they are cached
    uint64_t kv_empty[10];
    uint64_t s_full[2], p_ready[2], o_full[2], q_ready[2], turn[2], done[2];
    Plan plan;
    Ctx ctx[4];                             // the softmax warpgroups', the TMA warp's, the MMA warps'
    uint32_t tmem;
    int raw_end;                            // e4m3: uses of the ring, once all are on their way
};

// The K/V ring's order: K V of a tile (two row tiles), or K K V V of two tiles
// (alternate tiles).  The TMA warp fills stages in that order and both MMA
// warps wait for every stage in that order, their own or not: a warp that
// skipped a use of a stage would take the phase before it for its own
// (parities repeat every two).
template <int NS>
struct Slot {
    int st;
    uint32_t ph;
    __device__ __forceinline__ void step() {
        if (++st == NS) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// The TMA warp.  A tile is a box or two a page, each page issued by a lane of
// its own, one after the other; page indices are read a group of tiles ahead.
template <int D, bool E4M3>
__device__ __forceinline__ void produce(const AttnArgs& a, const KvMaps& maps, Shared& sh, uint8_t* ring) {
    using C = Cfg<D, E4M3>;
    constexpr int kBox = E4M3 ? D : 64, kBoxBytes = E4M3 ? D : 128, kParts = D / kBox;
    uint64_t* full = sh.kv_full + (E4M3 ? C::kStages : 0);
    int uses = 0;
    const int lane = threadIdx.x & 31;
    const int page = a.kv.page, pl = a.kv.page_log2, np = kKT >> pl, n_pages = a.kv.n_pages;
    // lanes 0 .. np-1: the pages of a group's first tile, np .. 2 np - 1: of its second
    const int i = lane >= np ? 1 : 0;
    uint8_t* box = ring + C::kRaw + (lane - i * np) * page * kBoxBytes;
    Ctx& ctx = sh.ctx[2];
    ctx.start<32>(a, sh.plan);
    Slot<C::kStages> at{0, 1u};
    bool dead = false;
    while (!dead && ctx.next<32>(a)) {
        const Item& it = ctx.it;
        const int32_t* table = a.sq.table + int64_t(it.b) * a.sq.max_pages;
        const int p_lo = it.lo >> pl, p_hi = (it.hi + page - 1) >> pl, head = it.h;
        const int T = ctx.sr.tiles, group = ctx.sr.pair ? 1 : 2;
        int p = (((it.tile0 + it.t0) * kKT) >> pl) + lane;       // this lane's page
        auto mine = [&]() { return lane < group * np && p >= p_lo && p < p_hi; };
        int pg = T > 0 && mine() ? table[p] : 0;
        for (int j = 0; j < T && !dead; j += group) {
            const bool issue = mine() && j + i < T;
            if (issue && (pg < 0 || pg >= n_pages)) {
                record_error(a.err, MOE_ERR_INVALID_ARG);
                pg = n_pages;                                    // out of range: reads as zeros
            }
            const int p0 = p - lane, m = min(group, T - j);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                for (int t = 0; t < m && !dead; ++t) {
                    const int bytes = max(0, min(p0 + (t + 1) * np, p_hi) - max(p0 + t * np, p_lo)) * page * kParts * kBoxBytes;
                    dead = !warp_wait(&sh.kv_empty[at.st], at.ph, a.err, a.timeout_ns);
                    if (dead) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[at.st], bytes);
                    __syncwarp();
                    for (int b = t * np; b < (t + 1) * np; ++b) {
                        if (lane == b && issue) {
#pragma unroll
                            for (int x = 0; x < kParts; ++x)
                                tma_load_4d(box + at.st * C::kStageBytes + x * kKT * 128, v ? &maps.v : &maps.k,
                                            &full[at.st], x * kBox, 0, head, pg);
                        }
                        __syncwarp();
                    }
                    at.step();
                    ++uses;
                }
            }
            p += group * np;
            if (j + group < T && mine()) pg = table[p];
        }
    }
    if constexpr (E4M3) {                                        // one more, empty: the converting warps end there
        if (!dead && warp_wait(&sh.kv_empty[at.st], at.ph, a.err, a.timeout_ns)) {
            if (lane == 0) {
                sh.raw_end = uses;
                mbar_arrive(&full[at.st]);
            }
            __syncwarp();
            at.step();
        }
    }
    // each stage's last copy
    for (int k = 0; k < C::kStages; ++k, at.step()) mbar_wait(&full[at.st], at.ph, a.err, kDrainNs);
}

// e4m3: a stage's tile to bf16 where it is, by a warpgroup with a thread a key and
// without the conversion unit, which the powers need (see e4m3x4_to_bf16).  A
// thread's 16-byte pieces go in order: the two it writes for piece ch lie in the
// first half, or over pieces 2 ch - 8 and 2 ch - 7 of its own row, which it has
// read.  Code size decides: 2048 tokens over 16,384 keys take 1.00 ms with two
// pieces a turn and 1.04 with one; with all eight, and NaN codes looked for a
// piece at a time, the code did not fit the instruction caches beside the other
// roles' (1.9 ms).  A ring of its own for the tiles as they are cached (4 + 2
// stages for 5) 1.05, a second warpgroup 1.00 (16 verify blocks 139 -> 150 us).
template <int D>
__device__ __forceinline__ void convert(const AttnArgs& a, Shared& sh, uint8_t* ring) {
    using C = Cfg<D, true>;
    const int lr = threadIdx.x & 127, lane = threadIdx.x & 31;
    Slot<C::kStages> at{0, 0u};
    for (int use = 0;; ++use, at.step()) {
        if (!warp_wait(&sh.kv_full[C::kStages + at.st], at.ph, a.err, a.timeout_ns)) break;
        if (use == *const_cast<volatile int*>(&sh.raw_end)) break;
        uint8_t* dst = ring + at.st * C::kStageBytes + lr * 128;
        const uint8_t* raw = ring + at.st * C::kStageBytes + C::kRaw + lr * D;
        auto from = [&](int ch) { return raw + ((D == 128 ? ch ^ (lr & 7) : ch ^ ((lr >> 1) & 3)) << 4); };
        auto to = [&](int c2) { return dst + (c2 >> 3) * 16384 + (((c2 & 7) ^ (lr & 7)) << 4); };
        uint4 next = *reinterpret_cast<const uint4*>(from(0));
        uint32_t most = 0;
#pragma unroll 2
        for (int ch = 0; ch < D / 16; ++ch) {
            const uint32_t x[4] = {next.x, next.y, next.z, next.w};
            next = *reinterpret_cast<const uint4*>(from((ch + 1) & (D / 16 - 1)));
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_bf16(x[e], y[2 * e], y[2 * e + 1], most);
            *reinterpret_cast<uint4*>(to(2 * ch)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(to(2 * ch + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        if (e4m3_had_nan(most)) {
#pragma unroll 1
            for (int c2 = 0; c2 < D / 8; ++c2) {
                uint4 w = *reinterpret_cast<const uint4*>(to(c2));
                w.x = e4m3_nan_again(w.x);
                w.y = e4m3_nan_again(w.y);
                w.z = e4m3_nan_again(w.z);
                w.w = e4m3_nan_again(w.w);
                *reinterpret_cast<uint4*>(to(c2)) = w;
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kv_full[at.st]);
    }
}

// The MMA warp of stream s: one thread issues, the whole warp waits.  The
// streams' warps take turns, a burst each: PV of a tile, then QK of the next
// (which writes S over that P).  Two warps, because the tensor pipe holds only
// a few instructions: a warp's waits for its data run beside the other's
// burst (one warp for both: 862 us for a chunk of 2048 over 16384 keys, its
// four to six waits a burst leaving the pipe idle for 105 to 230 of 1025 cycles).
// In turns, because bursts that mix finish together, and both softmaxes then
// wait together (1049 us).  Descriptors are a constant plus the stage's offset
// (the 14-bit address field cannot carry: shared memory lies below 256 KB).
template <int D, bool E4M3>
__device__ __forceinline__ void multiply(const AttnArgs& a, Shared& sh, uint8_t* qs, uint8_t* ring, int s) {
    using C = Cfg<D, E4M3>;
    constexpr uint32_t kIdQK = idesc(false, kKT), kIdPV = idesc(true, D);
    const int lane = threadIdx.x & 31;
    const uint32_t colS = sh.tmem + 128 * s, colO = sh.tmem + kColO + 128 * s;
    const uint64_t q_desc = sdesc(smem_u32(qs + s * C::kQBytes), 16, 1024);
    const uint64_t k_desc = sdesc(smem_u32(ring), 16, 1024), v_desc = sdesc(smem_u32(ring), 16384, 1024);
    Ctx& ctx = sh.ctx[3];
    ctx.start<64>(a, sh.plan);
    const Item& it = ctx.it;
    const Share& sr = ctx.sr;
    Slot<C::kStages> at{0, 0u};
    uint32_t qp = 0, pp = 0, tp = 0;                             // phases of q_ready, p_ready, turn
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
    };
    if (s == 1 && lane == 0) mbar_arrive(&sh.turn[0]);           // stream 0 begins
    while (ctx.next<64>(a, kBarMma)) {
        const int T = sr.tiles, pair = sr.pair;
        if (T == 0) continue;
        // slots: this stream's tiles, or (two row tiles) all tiles, of which it uses a0 .. b0 - 1
        const int slots = pair ? T : (T + 1) / 2;
        const int a0 = pair ? (s ? sr.a[1] : sr.a[0]) : 0, b0 = pair ? (s ? sr.b[1] : sr.b[0]) : sr.count(s);
        const int have = pair ? T : b0;                          // slots whose tile is this warp's to look at
        const int lo = it.lo - (it.tile0 + it.t0) * kKT, hi = it.hi - (it.tile0 + it.t0) * kKT;
        int op = 0;                                              // ring uses of this item waited for
        // the stage of use `to`, once it and those before it are full; the others' are passed on
        auto take = [&](int to) {
            for (;; ++op, at.step()) {
                wait(&sh.kv_full[at.st], at.ph);
                if (op == to) break;
                if (lane == 0 && !dead) mbar_arrive(&sh.kv_empty[at.st]);
                __syncwarp();
            }
            const int st = at.st;
            ++op;
            at.step();
            return st;
        };
        if (b0 > a0) {
            wait(&sh.q_ready[s], qp);
            qp ^= 1;
        }
        for (int i = 0; i <= slots; ++i) {
            const bool do_v = i > a0 && i <= b0, do_k = i >= a0 && i < b0;
            int vs = 0, ks = 0;
            const bool has_v = i > 0 && i <= have, has_k = i < have;
            if (has_v) vs = take(pair ? 2 * i - 1 : 4 * (i - 1) + s + min(2, T - 2 * (i - 1)));
            if (has_k) ks = take(pair ? 2 * i : 4 * i + s);
            if (do_v) {
                // V rows of keys that no row of the item sees may hold anything: zero them (in a pair both warps do)
                const int j0 = (pair ? i - 1 : 2 * (i - 1) + s) * kKT;
                if (j0 < lo || j0 + kKT > hi) {
                    uint8_t* v = ring + vs * C::kStageBytes;
                    const int head = min(max(lo - j0, 0), kKT) * 128, tail = min(max(hi - j0, 0), kKT) * 128;
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {
                        uint8_t* part = v + x * kKT * 128;
                        for (int e = 16 * lane; e < head; e += 512)
                            *reinterpret_cast<uint4*>(part + e) = make_uint4(0, 0, 0, 0);
                        for (int e = tail + 16 * lane; e < kKT * 128; e += 512)
                            *reinterpret_cast<uint4*>(part + e) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                wait(&sh.p_ready[s], pp);
                pp ^= 1;
            }
            wait(&sh.turn[s], tp);
            tp ^= 1;
            tc_fence_after();
            const uint64_t kd = k_desc + ks * (C::kStageBytes >> 4), vd = v_desc + vs * (C::kStageBytes >> 4);
            const uint32_t acc = i - 1 > a0 ? 1u : 0u;
            if (elect_one() && !dead) {
                if (do_v) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        mma_ts(colO, colS + 8 * k, vd + (k * 2048 >> 4), kIdPV, k > 0 ? 1u : acc);
                    }
                    if (i == b0) mma_commit(&sh.o_full[s]);
                    mma_commit(&sh.kv_empty[vs]);
                } else if (has_v) {
                    mbar_arrive(&sh.kv_empty[vs]);
                }
                if (do_k) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                        mma_ss(colS, q_desc + off, kd + off, kIdQK, k > 0);
                    }
                    mma_commit(&sh.s_full[s]);
                    mma_commit(&sh.kv_empty[ks]);
                } else if (has_k) {
                    mbar_arrive(&sh.kv_empty[ks]);
                }
                mbar_arrive(&sh.turn[s ^ 1]);
            }
            __syncwarp();
        }
        // the other stream's last uses
        for (; op < 2 * T; ++op, at.step()) {
            wait(&sh.kv_full[at.st], at.ph);
            if (lane == 0 && !dead) mbar_arrive(&sh.kv_empty[at.st]);
            __syncwarp();
        }
    }
    // the products end before the accumulators are given back
    if (elect_one()) mma_commit(&sh.done[s]);
    mbar_wait(&sh.done[s], 0, a.err, kDrainNs);
}

// 16 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// What a softmax thread carries through an item: its row's reference (log2
// units) and sum of powers, in two parts.
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

// Takes a tile's maximum into the reference: the reference follows when it
// lags by more than kLag, and O in tensor memory with it (its products are
// complete: S came after them in the MMA thread's order).
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
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(f == 0.0f ? 0.0f : o[e] * f);
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
    for (int e = 0; e < 32; e += 4) {
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            fma2_to(p[k], p[k + 1], x[e + k], x[e + k + 1], c, off);
            p[k] = fast_exp2(p[k]);
            p[k + 1] = fast_exp2(p[k + 1]);
            add2(st.sum0, st.sum1, p[k], p[k + 1]);
        }
        u[e / 2] = pack_bf16(p[0], p[1]);
        u[e / 2 + 1] = pack_bf16(p[2], p[3]);
    }
    tmem_st16(colP, u);
}

__device__ __forceinline__ float power_offset(const RowState& st) {
    return st.ref == kNegInf ? 0.0f : -st.ref;
}

// Hands P to the MMA warp.
__device__ __forceinline__ void p_done(uint64_t* bar) {
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A key tile that every row sees, N pieces of 32 keys from piece `from` on
// this copy's (4: all of it) and the others' P zero: the long calls' loops, S
// held in registers.
template <int D, int N>
__device__ __forceinline__ void soft_tile_whole(uint32_t colS, uint32_t colO, int from, float c, bool started,
                                                uint64_t* ready, RowState& st) {
    float x[N][32];
#pragma unroll
    for (int q = 0; q < N; ++q) tmem_ld32(colS + 32 * (from + q), x[q]);
    tmem_wait_ld();
    float top = max32(x[0]);
#pragma unroll
    for (int q = 1; q < N; ++q) top = fmaxf(top, max32(x[q]));
    follow<D>(colO, top * c, started, st);
    const float off = power_offset(st);
    if constexpr (N < 4) {
        const uint32_t z[16] = {};
#pragma unroll
        for (int q = N; q < 4; ++q) tmem_st16(colS + 16 * ((from + q) & 3), z);
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
        powers(colS + 16 * (from + q), x[q], c, off, st);
    }
    p_done(ready);
}

// Any other: `count` pieces of 32 keys from piece `from` on are this copy's,
// the others' P is zero.  A loop of small code over the pieces, S read twice:
// a short call runs its code once, from cold instruction caches.
template <int D>
__device__ __forceinline__ void soft_tile_part(uint32_t colS, uint32_t colO, int from, int count, float c, bool started,
                                               bool whole, const RowView& view, bool draft, int first, int j0,
                                               uint64_t* ready, RowState& st) {
    float x[32];
    auto piece = [&](int q) {
        tmem_ld32(colS + 32 * q, x);
        tmem_wait_ld();
        if (!whole) {
            const uint32_t bits = row_bits(view, draft, first, j0 + 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) x[e] = kNegInf;
        }
    };
    float top = kNegInf;
#pragma unroll 1
    for (int q = from; q < from + count; ++q) {
        piece(q);
        top = fmaxf(top, max32(x));
    }
    follow<D>(colO, top * c, started, st);
    const float off = power_offset(st);
    // P of piece q lies at columns 16 q, in S pieces that have been read
#pragma unroll 1
    for (int q = from; q < from + count; ++q) {
        if (count > 1) piece(q);
        powers(colS + 16 * q, x, c, off, st);
    }
    const uint32_t z[16] = {};
#pragma unroll 1
    for (int q = 0; q < 4; ++q)
        if (q < from || q >= from + count) tmem_st16(colS + 16 * q, z);
    p_done(ready);
}

// A warp's 32 query rows into shared memory, K-major with the 128-byte swizzle.
// `src` is the lane's own row; the warp reads whole rows, D / 8 lanes to one, so
// that a load touches 4 lines and not 32, a few loads at a time before their use
// (few, because a short call runs this code from cold instruction caches).
template <int D>
__device__ __forceinline__ void load_queries(const uint16_t* src, bool valid, bool negate, uint8_t* qt) {
    constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes, kBatch = 8;
    const int lane = threadIdx.x & 31, ch = lane % kLanes, sub = lane / kLanes;
    const int row0 = threadIdx.x & 96;                           // the warp's first row of the tile
    const uint32_t flip = negate ? 0x80008000u : 0u, on = __ballot_sync(0xFFFFFFFFu, valid);
    const unsigned long long mine = reinterpret_cast<unsigned long long>(src);
#pragma unroll 1
    for (int i0 = 0; i0 < kLanes; i0 += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int rl = (i0 + k) * kRowsAt + sub;
            const uint16_t* p = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, mine, rl));
            w[k] = __ldg(reinterpret_cast<const uint4*>(p + 8 * ch));
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int rl = (i0 + k) * kRowsAt + sub, r = row0 + rl;
            const uint32_t keep = (on >> rl) & 1u ? 0xFFFFFFFFu : 0u;
            *reinterpret_cast<uint4*>(qt + r * 128 + (ch >> 3) * 16384 + (((ch & 7) ^ (r & 7)) << 4)) =
                make_uint4((w[k].x ^ flip) & keep, (w[k].y ^ flip) & keep, (w[k].z ^ flip) & keep, (w[k].w ^ flip) & keep);
        }
    }
    fence_async_smem();
}

template <int D, bool E4M3>
__device__ __forceinline__ void soften(const AttnArgs& a, Shared& sh, uint8_t* qs) {
    using C = Cfg<D, E4M3>;
    const int tid = threadIdx.x, s = tid >> 7, lr = tid & 127, lane = tid & 31, wq = (tid >> 5) & 3;
    const uint32_t tm_lane = sh.tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t colS = tm_lane + 128 * s, colO = tm_lane + kColO + 128 * s;
    const bool draft = a.draft != nullptr;
    Ctx& ctx = sh.ctx[s];
    ctx.start<128>(a, sh.plan);
    const Item& it = ctx.it;
    const Share& sr = ctx.sr;
    uint32_t sp = 0, op0 = 0, op1 = 0;
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
        tc_fence_after();
    };
    while (ctx.next<128>(a, kBarGroup + s)) {
        // this thread's row, and its copy where the rows repeat
        const int copies = sr.pair || sr.rows > 64 ? 1 : (sr.rows > 32 ? 2 : 4);
        const int span = 128 / copies, copy = lr / span;
        const int row = sr.pair ? 128 * s + lr : lr - copy * span;
        const bool valid = row < sr.rows;
        const bool warp_on = __any_sync(0xFFFFFFFFu, valid);
        const int n = sr.count(s);
        RowView view{0, 0, 0ull};
        // log2 units a product: at least 1.2e-38 (an unseen key's -inf times it stays -inf), or NaN; the sign goes to the queries
        const float cs = a.scale * kLog2e * (E4M3 ? a.kv.k_scale[it.h] : 1.0f);
        const float c = cs != cs ? cs : fmaxf(fabsf(cs), 1.2e-38f);
        {
            const int r = it.rt * kMT + (valid ? row : 0), qi = a.query_of(r), hd = it.h * a.group + r - qi * a.group;
            if (valid) view = row_view(a, it.s, qi);
            load_queries<D>(a.q + (it.s.q0 + qi) * a.q_stride + hd * D, valid, cs < 0.0f, qs + s * C::kQBytes);
            __syncwarp();
            if (lane == 0 && n > 0) mbar_arrive(&sh.q_ready[s]);
        }
        RowState st{kNegInf, 0.0f, 0.0f};
        {
            const int base = (it.tile0 + it.t0 + sr.tile(s, 0)) * kKT, step = sr.pair ? kKT : 2 * kKT;
            const int wlo = s ? sr.wlo[1] : sr.wlo[0], whi = s ? sr.whi[1] : sr.whi[0], first = it.s.first;
            for (int i = 0; i < n; ++i) {
                const int j0 = base + i * step;
                wait(&sh.s_full[s], sp);
                sp ^= 1;
                const bool whole = j0 >= wlo && j0 + kKT <= whi;
                if (!warp_on) {
                    p_done(&sh.p_ready[s]);
                } else if (whole && copies == 1) {
                    soft_tile_whole<D, 4>(colS, colO, 0, c, i > 0, &sh.p_ready[s], st);
                } else if (whole && copies == 2) {
                    soft_tile_whole<D, 2>(colS, colO, 2 * copy, c, i > 0, &sh.p_ready[s], st);
                } else {
                    soft_tile_part<D>(colS, colO, copy * (span >> 5), span >> 5, c, i > 0, whole, view, draft,
                                            first, j0, &sh.p_ready[s], st);
                }
            }
        }
        // --- the item's rows: normalised, or this CTA's piece of them
        float ref = st.ref, sum = st.sum0 + st.sum1;             // (lanes of no row: whatever)
        if (sum != sum) ref = fmaxf(ref, 0.0f);                  // a NaN is a result, not an empty row
        const bool piece = it.t0 > 0 || it.t1 < it.n;
        const int n0 = sr.count(0), n1 = sr.count(1);
        float* slot = a.partials + (int64_t(it.t0 == 0 ? 0 : kAttnMaxCtas) + blockIdx.x) * (kAttnSlotRows * (D + 2));
        // What a row's sums are multiplied with here: its weight among the lanes that share the row (the
        // streams of one row tile, the copies), v_scale and, unless the row goes on elsewhere, 1 / its sum.
        float weight = ref == kNegInf ? 0.0f : 1.0f, top = ref;
        const int sharers = sr.pair ? 0 : 2 * copies;
        if (sharers) {
            sh.ml[s][lr] = make_float2(ref, sum);
            named_bar(kBarAll, kSoft);
            for (int k = 0; k < sharers; ++k) top = fmaxf(top, sh.ml[k & 1][(lr & (span - 1)) + (k >> 1) * span].x);
            sum = 0.0f;
            for (int k = 0; k < sharers; ++k) {
                const float2 x = sh.ml[k & 1][(lr & (span - 1)) + (k >> 1) * span];
                sum += x.x == kNegInf ? 0.0f : x.y * fast_exp2(x.x - top);
            }
            weight = ref == kNegInf ? 0.0f : fast_exp2(ref - top);
        }
        weight *= (E4M3 ? a.kv.v_scale[it.h] : 1.0f) * (piece || top == kNegInf ? 1.0f : 1.0f / sum);
        const int r = it.rt * kMT + (valid ? row : 0), qi = a.query_of(r), hd = it.h * a.group + r - qi * a.group;
        const int64_t at = int64_t(it.s.q0 + qi) * a.q_heads + hd;
        if (valid && (sr.pair || (s == 0 && copy == 0))) {
            if (piece)
                *reinterpret_cast<float2*>(slot + kAttnSlotRows * D + 2 * row) = make_float2(top, sum);
            else if (a.lse)
                a.lse[at] = top == kNegInf ? kNegInf : (top + log2f(sum)) * kLn2;
        }
        // four columns of a row, finished
        auto put = [&](int64_t at_, int row_, int d4, const float4& y) {
            if (piece)
                *reinterpret_cast<float4*>(slot + (d4 * kAttnSlotRows + row_) * 4) = y;
            else
                *reinterpret_cast<uint2*>(a.out + at_ * D + 4 * d4) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        };
        if (n > 0) wait(&sh.o_full[s], s ? op1 : op0);
        if (sr.pair) {
            if (warp_on) {
#pragma unroll 1
                for (int q = 0; q < D / 16; ++q) {
                    float o[16];
                    tmem_ld16(colO + 16 * q, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = weight != 0.0f && n > 0 ? o[e] * weight : 0.0f;
                    if (valid) {
                        if (piece) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                put(at, row, 4 * q + e, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                *reinterpret_cast<uint4*>(a.out + at * D + 16 * q + 8 * e) =
                                    make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                               pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                        }
                    }
                    __syncwarp();
                }
            }
        } else {
            // The streams' sums meet in the query tiles' room, once both streams' products are done: each
            // warpgroup leaves one half of its columns there, then adds the other's half to its own.
            float* merge = reinterpret_cast<float*>(qs);
            auto cell = [&](int l, int d4) { return reinterpret_cast<float4*>(merge + l * D + ((d4 ^ (l & 7)) << 2)); };
            if (s == 0 ? n1 > 0 : n0 > 0) wait(&sh.o_full[s ^ 1], s ? op0 : op1);
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                const int c0 = (s ^ step ^ 1) * (D / 2);
                if (warp_on) {
#pragma unroll 2
                    for (int q = 0; q < D / 32; ++q) {
                        float o[16];
                        tmem_ld16(colO + c0 + 16 * q, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d4 = c0 / 4 + 4 * q + e;
                            float4 y = make_float4(0, 0, 0, 0);
                            if (step) y = *cell(lr, d4);
                            if (weight != 0.0f && n > 0) {
                                y.x = fmaf(o[4 * e], weight, y.x);
                                y.y = fmaf(o[4 * e + 1], weight, y.y);
                                y.z = fmaf(o[4 * e + 2], weight, y.z);
                                y.w = fmaf(o[4 * e + 3], weight, y.w);
                            }
                            if (step == 0 || copies > 1)
                                *cell(lr, d4) = y;
                            else if (valid)
                                put(at, row, d4, y);
                        }
                        __syncwarp();
                    }
                }
                named_bar(kBarAll, kSoft);
            }
            if (copies > 1) {
                // thread: a row and every eighth (fourth) piece of four columns
                const int tr = tid & (span - 1), rr = it.rt * kMT + tr, qj = a.query_of(rr);
                const int64_t to = int64_t(it.s.q0 + qj) * a.q_heads + it.h * a.group + rr - qj * a.group;
                if (tr < sr.rows) {
#pragma unroll 4
                    for (int d4 = tid / span; d4 < D / 4; d4 += kSoft / span) {
                        float4 y = *cell(tr, d4);
#pragma unroll
                        for (int k = 1; k < 4; ++k) {
                            if (k >= copies) break;
                            const float4 u = *cell(tr + k * span, d4);
                            y.x += u.x;
                            y.y += u.y;
                            y.z += u.z;
                            y.w += u.w;
                        }
                        put(to, tr, d4, y);
                    }
                }
            }
        }
        tc_fence_before();
        if (n0 > 0) op0 ^= 1;
        if (n1 > 0) op1 ^= 1;
        if (!sr.pair) named_bar(kBarAll, kSoft);                 // the query tiles' room has been read
        if (tid == 0) note_split(a, it, sr.rows, kMT, sh.plan);
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads<E4M3>, 1) attn_tile_kernel(const AttnArgs a,
                                                                const __grid_constant__ KvMaps maps) {
    using C = Cfg<D, E4M3>;
    static_assert(C::kMerge == 2 * C::kQBytes, "stream 1's sums fit the two query tiles");
    extern __shared__ __align__(1024) uint8_t dyn[];
    uint8_t* qs = dyn;
    uint8_t* ring = qs + 2 * C::kQBytes;
    Shared& sh = *reinterpret_cast<Shared*>(dyn + C::kSmem);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sh.kv_full[i], E4M3 ? 4 : 1);         // the converting warps, or the TMA warp
            mbar_init(&sh.kv_empty[i], 2);
            if (E4M3) mbar_init(&sh.kv_full[C::kStages + i], 1);
        }
        sh.raw_end = -1;
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_ready[s], 4);
            mbar_init(&sh.turn[s], 1);
            mbar_init(&sh.done[s], 1);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.q_ready[s], 4);
        }
        fence_barrier_init();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();
    pdl_launch_dependents();
    plan_work<kMT, kKT>(a, 1, reinterpret_cast<int64_t*>(sh.ml), &sh.plan);   // (its barriers publish sh.tmem)
    tc_fence_after();
    zero_pad_rows(a, sh.plan.seqs);
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft<E4M3>));
        soften<D, E4M3>(a, sh, qs);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest<E4M3>));
        if (warp == 8)
            produce<D, E4M3>(a, maps, sh, ring);
        else if (warp < 11)
            multiply<D, E4M3>(a, sh, qs, ring, warp - 9);
        else if (E4M3 && warp >= 12)
            convert<D>(a, sh, ring);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(sh.tmem, kTmemCols);
}

template <int D, bool E4M3>
cudaError_t launch(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<D, E4M3>::kSmem + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(attn_tile_kernel<D, E4M3>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int grid = n_sms < kAttnMaxCtas ? n_sms : kAttnMaxCtas;
    e = launch_pdl(attn_tile_kernel<D, E4M3>, dim3(grid), dim3(kThreads<E4M3>), smem, s, a, m);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_join(a, grid, s);
}

}  // namespace

cudaError_t launch_attn_tile(const AttnArgs& a, const KvMaps& m, int n_sms, cudaStream_t s) {
    if (a.kv.dim == 128) return a.kv.e4m3 ? launch<128, true>(a, m, n_sms, s) : launch<128, false>(a, m, n_sms, s);
    return a.kv.e4m3 ? launch<64, true>(a, m, n_sms, s) : launch<64, false>(a, m, n_sms, s);
}

}  // namespace moe
