// keyw.cu -- the attention weight that each cached key received in a step,
// added to the running scores that eviction goes by (sm_103a).
//
// w_j = sum over the rows that see key j of 2^(c q.k_j - lse log2 e), from the
// transposed product S^T = K Q^T (tcgen05.mma, keys on the tensor-memory
// lanes, rows on the columns): a thread has a key, and its sum runs over the
// columns of its own lane, with no exchange between threads and no atomics.
//
// An item is 256 keys of a sequence and kv head: two 128-key tiles, held in
// shared memory while the query rows that see them pass through in tiles of
// up to 128 (TMA boxes of whole tokens: the heads of a kv head by as many
// tokens as fit).  K is so read once, and a Q tile feeds two products; each
// tile's products go to two S buffers in turn, and a warpgroup a tile takes
// the powers of one while the next is made.  Few rows: bound by the K stream
// (the next item's tiles load meanwhile).  Many rows: the products take 512
// cycles a 128 x 128 tile on an SM, the powers as many; measured, the two overlap
// for a small part only (both units active 43 %).
//
// e4m3 keys are turned to bf16 in shared memory first (exact), which a tile
// pays once however many rows see it, by two warpgroups of their own (as part
// of the powers' warpgroups' round it held up the stream: 16 verify blocks 92 us).
// Queries as two e4m3 codes an element, beside K as it is cached, were no
// faster (87 us: waiting for instructions was the warps' largest stall) and
// slower for chunks, where a query tile is coded again for every item.
//
// Measured (64 query heads, 8 kv heads of 128): 8 single tokens over 1,021 to
// 8,209 keys 16 us (4.4 TB/s); 16 verify blocks of up to 8 over 4,099 to 16,411
// keys 61 us in bf16 (5.3 TB/s of a copy's 6.7), 84 over e4m3 (2.0: the powers'
// and the conversion's instructions, not bytes); 1024 tokens over
// 8,192 157 us in bf16 (0.93 PFLOP/s), 160 over e4m3.
#include "attn_mma.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kKeys = 128;                  // keys of a tile; two an item
// 2 warpgroups for the powers, K warp, Q warp, 2 MMA warps; e4m3: 2 warpgroups that convert
template <bool E4M3>
constexpr int kThreads = E4M3 ? 640 : 384;

// e4m3 and more than 64 rows a tile: registers a thread, moved to the powers'
// warpgroups after the launch at 96: 8 * 128 + 12 * 72 = 1888 a lane column of
// the 20 * 96 = 1920 launched.  1024 tokens over 8,192 keys 190 -> 162 us with
// the powers of a full tile unrolled; with fewer rows, whose tiles are never full,
// both cost more code and the conversion registers (16 verify blocks 86 -> 90).
constexpr int kRegsPowers = 128, kRegsRest = 72;

constexpr int kMaxBufs = 8;                 // K buffers a tile
constexpr int kItems = 4;                   // items ahead

// Shared memory: the query tiles (their rows rounded up to 8, in parts of 64
// elements), the e4m3 keys' bf16 tiles (two of each where rows are few: with
// one, a tile's conversion waits for the products of the one before it), and
// as many K buffers a tile as fit: the fewer rows, the more of K in flight.
template <int D, bool E4M3>
struct Cfg {
    static constexpr int kQStages = E4M3 ? 2 : 3;
    static constexpr int kRaw = kKeys * (E4M3 ? D : 2 * D);    // a K tile as it is cached
    static constexpr int kTile = kKeys * 2 * D;                // bf16
    static constexpr int kTotal = 232448 - 3072;               // then Shared

    __host__ __device__ __forceinline__ static int part(const KeywArgs& a) {
        return (a.tile_tokens * a.tile_heads + 7) / 8 * 1024;
    }
    __host__ __device__ __forceinline__ static int q_tile(const KeywArgs& a) { return part(a) * (D / 64); }
    __host__ __device__ __forceinline__ static int conv(const KeywArgs& a) {      // bf16 tiles a key tile
        return !E4M3 ? 0 : (a.tile_tokens * a.tile_heads <= 64 ? 2 : 1);
    }
    __host__ __device__ __forceinline__ static int k16(const KeywArgs& a) { return kQStages * q_tile(a); }
    __host__ __device__ __forceinline__ static int raw(const KeywArgs& a) { return k16(a) + 2 * conv(a) * kTile; }
    __host__ __device__ __forceinline__ static int bufs(const KeywArgs& a) {
        const int n = (kTotal - raw(a)) / (2 * kRaw);
        return n < kMaxBufs ? n : kMaxBufs;
    }
};

struct Shared {
    alignas(16) float off[2][2][128];       // [tile][buffer] -lse log2 e of the columns' rows
    uint32_t live[2][2][4];                 // which columns count
    alignas(16) int item[kItems][12];       // see Item
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t k_full[2][kMaxBufs], k_empty[2][kMaxBufs];   // [tile][buffer]
    uint64_t k_bf16[2][2], k_free[2][2];    // e4m3, [tile][bf16 tile]: it is there, is no longer read
    uint64_t q_full[3], q_empty[3];
    uint64_t s_full[2][2], s_empty[2][2];   // [tile][buffer]
    uint64_t done[2];
    uint32_t tmem;
};

// An item as the roles read it; b < 0: no more.
struct Item {
    int b, h, j0, q0;
    int nq, first, len, t0;                 // row tiles t0 .. t1 - 1 see some of its keys
    int t1;
};

// A place in a ring of buffers, and the phase of its barriers.
struct Turn {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step(int n) {
        if (++st == n) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// A warp's waits: after one that ran out the others return at once.
struct Waiter {
    const AttnArgs& a;
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
        if (!dead) dead = !warp_wait(bar, parity, a.err, a.timeout_ns);
    }
};

// Items in the order (sequence, key group, head), CTA c taking every
// gridDim.x-th.  The K warp walks them once for the CTA and hands them to the
// other roles through a small ring (every warp on its own walk: 12 to 20 times
// the bookkeeping, which then paced the stream of verify blocks).
struct Scheduler {
    Seq s;
    int b, g, h, groups, dg, dh;
    int64_t skip;                           // items still to pass before this CTA's next, past (g, h)
    bool rows;                              // no sequence so far whose offsets do not fit

    __device__ __forceinline__ void start(const KeywArgs& ka) {
        b = -1;
        g = h = groups = 0;
        dg = gridDim.x / ka.a.kv.heads;
        dh = gridDim.x - dg * ka.a.kv.heads;
        skip = blockIdx.x;
        rows = true;
    }
    __device__ __forceinline__ bool next(const KeywArgs& ka, Item& it) {
        const AttnArgs& a = ka.a;
        if (b >= 0) {                       // gridDim.x items on
            g += dg;
            h += dh;
            if (h >= a.kv.heads) {
                h -= a.kv.heads;
                ++g;
            }
            skip = int64_t(g - groups) * a.kv.heads + h;     // past this sequence's end, if it is not below 0
        }
        while (b < 0 || g >= groups) {
            if (++b >= a.sq.n) return false;
            bool fits;
            s = load_seq(a.sq, a.kv.page, b, a.err, &fits);
            rows = rows && fits;
            if (!rows) {
                s.q0 = s.nq = 0;
                s.first = s.len;
            }
            groups = (s.len + 2 * kKeys - 1) / (2 * kKeys);
            const int64_t count = int64_t(groups) * a.kv.heads;
            if (skip >= count) {
                skip -= count;
                g = groups;
                continue;
            }
            g = static_cast<int>(skip / a.kv.heads);
            h = static_cast<int>(skip - int64_t(g) * a.kv.heads);
        }
        const int j0 = g * 2 * kKeys, j1 = min(j0 + 2 * kKeys, s.len);
        int i0 = 0, i1 = s.nq;              // queries that see some of these keys
        if (!a.draft && a.causal) i0 = min(max(0, j0 - s.first), s.nq);
        if (a.window > 0) i1 = static_cast<int>(min(int64_t(s.nq), max(int64_t(0), int64_t(j1) - 1 - s.first + a.window)));
        const int t0 = ka.tile_of(i0), t1 = i1 > i0 ? ka.tile_of(i1 - 1) + 1 : t0;
        it = Item{b, h, j0, s.q0, s.nq, s.first, s.len, t0, t1};
        return true;
    }
};

// A role's place in the ring of items; next() copies one out, false after the
// last or once a wait ran out.  One warp each.
struct Feed {
    Shared& sh;
    Waiter& wait;
    Turn at;

    __device__ __forceinline__ bool next(Item& it) {
        wait(&sh.item_full[at.st], at.ph);
        const int4 x = *reinterpret_cast<const int4*>(&sh.item[at.st][0]);
        const int4 y = *reinterpret_cast<const int4*>(&sh.item[at.st][4]);
        it = Item{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, sh.item[at.st][8]};
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.item_empty[at.st]);
        at.step(kItems);
        return !wait.dead && it.b >= 0;
    }
};

template <int D, bool E4M3>
__device__ __forceinline__ void load_keys(const KeywArgs& ka, const CUtensorMap& map, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    constexpr int kBox = E4M3 ? D : 64, kBoxBytes = E4M3 ? D : 128, kParts = D / kBox;
    const AttnArgs& a = ka.a;
    const int lane = threadIdx.x & 31, page = a.kv.page, pl = a.kv.page_log2, np = kKeys >> pl;
    const int bufs = C::bufs(ka), raw = C::raw(ka);
    Scheduler sc;
    sc.start(ka);
    Waiter wait{a};
    Turn use[2], slot;
    int p0 = 0, p_hi = 0, pg = 0, head = 0;
    bool mine = false;
    // the next item, handed on, and its page indices, read a step ahead
    // (after a wait that ran out nothing is handed on: the slot may still be read)
    auto fetch = [&]() {
        Item it{-1, 0, 0, 0, 0, 0, 0, 0, 0};
        const bool more = sc.next(ka, it);
        wait(&sh.item_empty[slot.st], slot.ph ^ 1u);
        if (wait.dead) return false;
        if (lane == 0) {
            *reinterpret_cast<int4*>(&sh.item[slot.st][0]) = make_int4(it.b, it.h, it.j0, it.q0);
            *reinterpret_cast<int4*>(&sh.item[slot.st][4]) = make_int4(it.nq, it.first, it.len, it.t0);
            sh.item[slot.st][8] = it.t1;
            mbar_arrive(&sh.item_full[slot.st]);
        }
        __syncwarp();
        slot.step(kItems);
        if (!more) return false;
        p0 = it.j0 >> pl;
        p_hi = (it.len + page - 1) >> pl;
        head = it.h;
        mine = lane < 2 * np && p0 + lane < p_hi;
        pg = mine ? a.sq.table[int64_t(it.b) * a.sq.max_pages + p0 + lane] : 0;
        return true;
    };
    bool more = fetch();
    while (more && !wait.dead) {
        if (mine && (pg < 0 || pg >= a.kv.n_pages)) {
            record_error(a.err, MOE_ERR_INVALID_ARG);
            pg = a.kv.n_pages;                                  // out of range: reads as zeros
        }
        const int c0 = p0, c_hi = p_hi, c_pg = pg, c_head = head;
        const bool c_mine = mine;
        more = fetch();
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int first = c0 + w * np, boxes = min(first + np, c_hi) - first;
            if (boxes <= 0) continue;
            const int buf = use[w].st;
            wait(&sh.k_empty[w][buf], use[w].ph ^ 1u);
            if (wait.dead) break;
            use[w].step(bufs);
            uint8_t* dst = smem + raw + (w * bufs + buf) * C::kRaw;
            if (lane == 0) mbar_arrive_expect_tx(&sh.k_full[w][buf], boxes * page * (E4M3 ? D : 2 * D));
            __syncwarp();
            for (int k = 0; k < np; ++k) {
                if (lane == w * np + k && c_mine) {
#pragma unroll
                    for (int x = 0; x < kParts; ++x)
                        tma_load_4d(dst + k * page * kBoxBytes + x * kKeys * 128, &map, &sh.k_full[w][buf], x * kBox, 0,
                                    c_head, c_pg);
                }
                __syncwarp();
            }
        }
    }
    // each buffer's last copy
    for (int w = 0; w < 2; ++w)
        for (int k = 0; k < bufs; ++k) {
            mbar_wait(&sh.k_full[w][use[w].st], use[w].ph ^ 1u, a.err, kDrainNs);
            use[w].step(bufs);
        }
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_rows(const KeywArgs& ka, const CUtensorMap& map, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const int lane = threadIdx.x & 31;
    const uint32_t bytes = ka.tile_tokens * ka.tile_heads * D * 2;
    const int q_tile = C::q_tile(ka), part = C::part(ka);
    Item it;
    Waiter wait{a};
    Feed feed{sh, wait};
    Turn q;
    while (feed.next(it)) {
        for (int t = it.t0; t < it.t1; ++t)
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                wait(&sh.q_empty[q.st], q.ph ^ 1u);
                if (wait.dead) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_full[q.st], bytes);
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_3d(smem + q.st * q_tile + x * part, &map, &sh.q_full[q.st], 64 * x,
                                    it.h * a.group + hc, it.q0 + t * ka.tile_tokens);
                }
                __syncwarp();
                q.step(C::kQStages);
            }
    }
    for (int k = 0; k < C::kQStages; ++k) {                      // each stage's last copy
        mbar_wait(&sh.q_full[q.st], q.ph ^ 1u, a.err, kDrainNs);
        q.step(C::kQStages);
    }
}

template <int D, bool E4M3>
__device__ __forceinline__ void multiply(const KeywArgs& ka, Shared& sh, uint8_t* smem, int w) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const uint64_t q_desc = sdesc(smem_u32(smem), 16, 1024);
    const int q_tile = C::q_tile(ka), part = C::part(ka), bufs = C::bufs(ka), raw = C::raw(ka);
    Item it;
    Waiter wait{a};
    Feed feed{sh, wait};
    Turn q, key, buf;
    const int conv = C::conv(ka), k16 = C::k16(ka);
    while (feed.next(it)) {
        const bool on = it.j0 + w * kKeys < it.len;
        int kb = 0;
        uint64_t k_desc = 0;
        if (on) {
            if constexpr (E4M3) {
                kb = key.st;
                wait(&sh.k_bf16[w][kb], key.ph);
                key.step(conv);
                k_desc = sdesc(smem_u32(smem + k16 + (w * conv + kb) * C::kTile), 16, 1024);
            } else {
                kb = key.st;
                wait(&sh.k_full[w][kb], key.ph);
                key.step(bufs);
                k_desc = sdesc(smem_u32(smem + raw + (w * bufs + kb) * C::kRaw), 16, 1024);
            }
        }
        for (int t = it.t0; t < it.t1; ++t) {
            const int tokens = min(ka.tile_tokens, it.nq - t * ka.tile_tokens);
            const uint32_t id = idesc(false, (tokens * ka.tile_heads + 15) & ~15);
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                wait(&sh.q_full[q.st], q.ph);
                const int sb = buf.st;
                if (on) {
                    wait(&sh.s_empty[w][sb], buf.ph ^ 1u);
                    buf.step(2);
                }
                if (wait.dead) break;
                tc_fence_after();
                const uint64_t qd = q_desc + (q.st * q_tile >> 4);
                const uint32_t d = sh.tmem + (2 * w + sb) * 128;
                if (elect_one()) {
                    if (on) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            mma_ss(d, k_desc + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                                          qd + (((k >> 2) * part + (k & 3) * 32) >> 4), id, k > 0);
                        }
                        mma_commit(&sh.s_full[w][sb]);
                        mma_commit(&sh.q_empty[q.st]);
                    } else {
                        mbar_arrive(&sh.q_empty[q.st]);
                    }
                }
                __syncwarp();
                q.step(C::kQStages);
            }
        }
        if (on && !wait.dead) {
            if (elect_one()) mma_commit(E4M3 ? &sh.k_free[w][kb] : &sh.k_empty[w][kb]);
            __syncwarp();
        }
    }
    // the products end before the accumulators are given back
    if (elect_one()) mma_commit(&sh.done[w]);
    mbar_wait(&sh.done[w], 0, a.err, kDrainNs);
}

// e4m3: one tile of the items' pairs to bf16.
template <int D>
__device__ __forceinline__ void convert(const KeywArgs& ka, Shared& sh, uint8_t* smem, int w) {
    using C = Cfg<D, true>;
    const int lr = threadIdx.x & 127, lane = threadIdx.x & 31;
    Item it;
    Waiter wait{ka.a};
    Feed feed{sh, wait};
    const int bufs = C::bufs(ka), conv = C::conv(ka);
    Turn key, out;
    while (feed.next(it)) {
        if (it.j0 + w * kKeys >= it.len) continue;
        const int kb = key.st;
        wait(&sh.k_full[w][kb], key.ph);
        key.step(bufs);
        const uint8_t* raw = smem + C::raw(ka) + (w * bufs + kb) * C::kRaw;
        uint8_t* dst = smem + C::k16(ka) + (w * conv + out.st) * C::kTile;
        uint4 in[D / 16];
#pragma unroll
        for (int ch = 0; ch < D / 16; ++ch)
            in[ch] = *reinterpret_cast<const uint4*>(
                raw + lr * D + ((D == 128 ? ch ^ (lr & 7) : ch ^ ((lr >> 1) & 3)) << 4));
        wait(&sh.k_free[w][out.st], out.ph ^ 1u);
        if (wait.dead) break;
        uint32_t most = 0;
#pragma unroll
        for (int ch = 0; ch < D / 16; ++ch) {
            const uint4 x = in[ch];
            uint32_t y[8];
            e4m3x4_to_bf16(x.x, y[0], y[1], most);
            e4m3x4_to_bf16(x.y, y[2], y[3], most);
            e4m3x4_to_bf16(x.z, y[4], y[5], most);
            e4m3x4_to_bf16(x.w, y[6], y[7], most);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c2 = 2 * ch + e;
                *reinterpret_cast<uint4*>(dst + (c2 >> 3) * 16384 + lr * 128 + (((c2 & 7) ^ (lr & 7)) << 4)) =
                    make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
            }
        }
        if (e4m3_had_nan(most)) {             // a NaN code makes its key's scores NaN: one NaN in the row does
            *reinterpret_cast<uint16_t*>(dst + lr * 128 + ((lr & 7) << 4)) = 0x7FC0u;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&sh.k_empty[w][kb]);
            mbar_arrive(&sh.k_bf16[w][out.st]);
        }
        out.step(conv);
    }
}

// 16 (or 32) columns: powers of the masked scores, added to two partial sums.
template <int N, bool MASK>
__device__ __forceinline__ void add_powers(uint32_t col, const float* off, float c, uint32_t bits, float& t0, float& t1) {
    float x[N];
    tmem_ld<N>(col, x);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 o = *reinterpret_cast<const float4*>(off + e);
        float p[4];
        fma2_off(p[0], p[1], x[e], x[e + 1], c, o.x, o.y);
        fma2_off(p[2], p[3], x[e + 2], x[e + 3], c, o.z, o.w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            p[k] = fast_exp2(p[k]);
            if (MASK && !((bits >> (e + k)) & 1u)) p[k] = 0.0f;
        }
        add2(t0, t1, p[0], p[1]);
        add2(t0, t1, p[2], p[3]);
    }
}

template <int D, bool E4M3, bool MANY>
__device__ __forceinline__ void weigh(const KeywArgs& ka, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const int tid = threadIdx.x, w = tid >> 7, lr = tid & 127, lane = tid & 31, wq = (tid >> 5) & 3;
    const uint32_t tm = sh.tmem + (static_cast<uint32_t>(wq * 32) << 16) + 2 * w * 128;
    const bool draft = a.draft != nullptr;
    // the row of column lr: token and head within a tile
    const int r_tok = lr / ka.tile_heads, r_head = lr - r_tok * ka.tile_heads;
    const int heads = a.group;
    // an item of this tile, its key's place in the scores, the score, and the log-sum-exp of its first
    // row tile's columns: read an item ahead
    Waiter wait{a};
    Feed feed{sh, wait};
    struct Ahead {
        Item it;
        bool more;
        int64_t at;
        bool store;
        float before, z;
    };
    auto row_lse = [&](const Item& it, int t, int hc) {
        const int i = t * ka.tile_tokens + r_tok, hd = hc + r_head;
        const bool ok = t < it.t1 && r_tok < ka.tile_tokens && i < it.nq && hd < heads;
        return ok ? __ldg(a.lse + int64_t(it.q0 + i) * a.q_heads + it.h * heads + hd) : kNegInf;
    };
    auto fetch = [&](Ahead& x) {
        do {
            x.more = bar_and(1 + w, feed.next(x.it), 128);       // all four warps go on or none: they meet below
        } while (x.more && x.it.j0 + w * kKeys >= x.it.len);
        if (!x.more) return;
        const int j = x.it.j0 + w * kKeys + lr;
        x.at = (int64_t(x.it.b) * a.kv.heads + x.it.h) * ka.score_stride + j;
        x.store = j < x.it.len && j < ka.score_stride;
        x.before = x.store && j < x.it.first ? ka.scores[x.at] : 0.0f;
        x.z = row_lse(x.it, x.it.t0, 0);
    };
    Ahead nx;
    fetch(nx);
    Turn buf;
    while (nx.more) {
        const Item it = nx.it;
        const int jt = it.j0 + w * kKeys, j = jt + lr;
        const int64_t at = nx.at;
        const bool store = nx.store;
        const float before = ka.decay * nx.before;
        float z = nx.z, sum = 0.0f;
        fetch(nx);
        const float c = a.scale * kLog2e * (E4M3 ? a.kv.k_scale[it.h] : 1.0f);
        for (int t = it.t0; t < it.t1; ++t) {
            const int i0 = t * ka.tile_tokens, tokens = min(ka.tile_tokens, it.nq - i0);
            const bool seen = (draft ? jt + kKeys <= it.first : !a.causal || jt + kKeys <= it.first + i0 + 1) &&
                              !(a.window > 0 && jt <= it.first + i0 + tokens - 1 - a.window);
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                const int sb = buf.st, rows = tokens * min(ka.tile_heads, a.group - hc);
                const bool live = fabsf(z) != INFINITY;
                sh.off[w][sb][lr] = live ? -z * kLog2e : 0.0f;
                const uint32_t word = __ballot_sync(0xFFFFFFFFu, live);
                if (lane == 0) sh.live[w][sb][wq] = word;
                named_bar(1 + w, 128);
                z = hc + ka.tile_heads < heads ? row_lse(it, t, hc + ka.tile_heads) : row_lse(it, t + 1, 0);
                wait(&sh.s_full[w][sb], buf.ph);
                buf.step(2);
                tc_fence_after();
                const uint32_t col = tm + sb * 128;
                const float* off = sh.off[w][sb];
                const uint32_t* words = sh.live[w][sb];
                float p0 = 0.0f, p1 = 0.0f;
                // columns of rows that see key j: a range by token, or by the rows' draft masks
                const int th = ka.tile_heads;
                int lo = 0, hi = rows;
                if (!seen) {
                    const int64_t rel = int64_t(j) - it.first - i0;             // j's place less the tile's first token's
                    if (!draft && a.causal) lo = static_cast<int>(max(int64_t(0), min(rel, int64_t(128)))) * th;
                    if (a.window > 0) hi = min(hi, static_cast<int>(max(int64_t(0), min(rel + a.window, int64_t(128)))) * th);
                }
                const bool whole = MANY && seen && rows == 128 &&
                                   (words[0] & words[1] & words[2] & words[3]) == 0xFFFFFFFFu;
                if (whole) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) add_powers<32, false>(col + 32 * q, off + 32 * q, c, 0, p0, p1);
                }
#pragma unroll 1
                for (int q = 0; q < 4 && !whole; ++q) {
                    if (32 * q >= rows) break;
                    const uint32_t word = words[q];
                    if (seen && word == 0xFFFFFFFFu) {
                        add_powers<32, false>(col + 32 * q, off + 32 * q, c, 0, p0, p1);
                        continue;
                    }
#pragma unroll 1
                    for (int n = 32 * q; n < min(32 * q + 32, rows); n += 16) {
                        uint32_t bits = (word >> (n & 16)) & 0xFFFFu;
                        if (!seen) {
                            const int l = min(max(lo - n, 0), 16), u = min(max(hi - n, 0), 16);
                            bits &= ((1u << u) - 1u) & ~((1u << l) - 1u);
                            const int place = j - it.first;
                            if (draft && place >= 0) {
                                for (int e = 0; e < 16 && n + e < rows; ++e) {
                                    const uint64_t m = a.draft[it.q0 + i0 + (n + e) / th];
                                    if (place >= 64 || !((m >> place) & 1ull)) bits &= ~(1u << e);
                                }
                            }
                            __syncwarp();
                        }
                        add_powers<16, true>(col + n, off + n, c, bits, p0, p1);
                    }
                }
                sum += p0 + p1;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty[w][sb]);
            }
        }
        if (store) ka.scores_out[at] = before + sum;
    }
}

// MANY: tiles of more than 64 rows.
template <int D, bool E4M3, bool MANY>
__global__ void __launch_bounds__(kThreads<E4M3>, 1) keyw_kernel(const KeywArgs ka, const __grid_constant__ KeywMaps maps) {
    using C = Cfg<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kTotal);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sh.done[w], 1);
            for (int i = 0; i < kMaxBufs; ++i) {
                mbar_init(&sh.k_full[w][i], 1);
                mbar_init(&sh.k_empty[w][i], E4M3 ? 4 : 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.k_bf16[w][i], 4);
                mbar_init(&sh.k_free[w][i], 1);
                mbar_init(&sh.s_full[w][i], 1);
                mbar_init(&sh.s_empty[w][i], 4);
            }
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kThreads<E4M3> / 32 - 1);   // every warp but the K warp
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 2);
        }
        fence_barrier_init();
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.q);
    }
    if (warp == 10) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_launch_dependents();
    if (warp < 8) {
        if constexpr (E4M3 && MANY) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsPowers));
        weigh<D, E4M3, MANY>(ka, sh, smem);
    } else {
        if constexpr (E4M3 && MANY) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == 8)
            load_keys<D, E4M3>(ka, maps.k, sh, smem);
        else if (warp == 9)
            load_rows<D, E4M3>(ka, maps.q, sh, smem);
        else if (warp < 12)
            multiply<D, E4M3>(ka, sh, smem, warp - 10);
        else if constexpr (E4M3)
            convert<D>(ka, sh, smem, (warp - 12) >> 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10) tmem_dealloc(sh.tmem, 512);
}

template <int D, bool E4M3, bool MANY>
cudaError_t launch(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<D, E4M3>::kTotal + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(keyw_kernel<D, E4M3, MANY>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(keyw_kernel<D, E4M3, MANY>, dim3(n_sms), dim3(kThreads<E4M3>), smem, s, a, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool E4M3>
cudaError_t launch(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s) {
    const bool many = a.tile_tokens * a.tile_heads > 64;
    if (a.a.kv.dim == 128) return many ? launch<128, E4M3, true>(a, m, n_sms, s) : launch<128, E4M3, false>(a, m, n_sms, s);
    return many ? launch<64, E4M3, true>(a, m, n_sms, s) : launch<64, E4M3, false>(a, m, n_sms, s);
}

}  // namespace

cudaError_t launch_keyw(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s) {
    return a.a.kv.e4m3 ? launch<true>(a, m, n_sms, s) : launch<false>(a, m, n_sms, s);
}

}  // namespace moe
