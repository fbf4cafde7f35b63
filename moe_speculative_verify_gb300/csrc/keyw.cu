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
// cycles a 128 x 128 tile on an SM, the powers as many.
//
// e4m3 keys are turned to bf16 in shared memory first (exact), which a tile
// pays once however many rows see it.
#include "attn_mma.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kKeys = 128;                  // keys of a tile; two an item
constexpr int kThreads = 384;               // 2 warpgroups, K warp, Q warp, 2 MMA warps
constexpr int kQStages = 3;

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kRaw = kKeys * (E4M3 ? D : 2 * D);    // a K tile as it is cached
    static constexpr int kTile = kKeys * 2 * D;                // bf16
    static constexpr int kQTile = 128 * 2 * D;
    static constexpr int oRaw = 0;                             // [tile][buffer]
    static constexpr int oK = 4 * kRaw;                        // e4m3: [tile] in bf16
    static constexpr int oQ = oK + (E4M3 ? 2 * kTile : 0);
    static constexpr int kBytes = oQ + kQStages * kQTile;      // then Shared
};

struct Shared {
    alignas(16) float off[2][2][128];       // [tile][buffer] -lse log2 e of the columns' rows
    uint32_t live[2][2][4];                 // which columns count
    uint64_t k_full[2][2], k_empty[2][2];   // [tile][buffer]
    uint64_t k_bf16[2];
    uint64_t q_full[kQStages], q_empty[kQStages];
    uint64_t s_full[2][2], s_empty[2][2];   // [tile][buffer]
    uint32_t tmem;
};

// Items in the order (sequence, key group, head), CTA c taking every
// gridDim.x-th; every role walks them for itself.
struct Items {
    Seq s;
    int b, h, j0;
    int t0, t1;                             // row tiles that see some of its keys
    int64_t idx, base;                      // this item, items before sequence b
    int64_t count;                          // items of it

    __device__ __forceinline__ void start(const KeywArgs& ka) {
        b = -1;
        base = count = 0;
        idx = int64_t(blockIdx.x) - gridDim.x;
    }
    __device__ __forceinline__ bool next(const KeywArgs& ka) {
        const AttnArgs& a = ka.a;
        idx += gridDim.x;
        while (idx >= base + count) {
            base += count;
            if (++b >= a.sq.n) return false;
            s = load_seq(a.sq, a.kv.page, b, a.err);
            count = int64_t(a.kv.heads) * ((s.len + 2 * kKeys - 1) / (2 * kKeys));
        }
        const int in = static_cast<int>(idx - base), g = in / a.kv.heads;
        h = in - g * a.kv.heads;
        j0 = g * 2 * kKeys;
        const int j1 = min(j0 + 2 * kKeys, s.len);
        int i0 = 0, i1 = s.nq;              // queries that see some of these keys
        if (!a.draft && a.causal) i0 = max(0, j0 - s.first);
        if (a.window > 0) i1 = static_cast<int>(min(int64_t(s.nq), max(int64_t(0), int64_t(j1) - 1 - s.first + a.window)));
        t0 = i0 / ka.tile_tokens;
        t1 = i1 > i0 ? (i1 + ka.tile_tokens - 1) / ka.tile_tokens : t0;
        return true;
    }
};

// A counted use of a two-buffer resource.
struct Turn {
    uint32_t n = 0;
    __device__ __forceinline__ int buf() const { return n & 1; }
    __device__ __forceinline__ uint32_t phase() const { return (n >> 1) & 1u; }
};

struct QSlot {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step() {
        if (++st == kQStages) {
            st = 0;
            ph ^= 1u;
        }
    }
};

struct Waiter {
    const AttnArgs& a;
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
        if (!dead && !mbar_wait(bar, parity, a.err, a.timeout_ns)) dead = true;
    }
};

template <int D, bool E4M3>
__device__ __forceinline__ void load_keys(const KeywArgs& ka, const CUtensorMap& map, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    constexpr int kBox = E4M3 ? D : 64, kBoxBytes = E4M3 ? D : 128, kParts = D / kBox;
    const AttnArgs& a = ka.a;
    const int lane = threadIdx.x & 31, page = a.kv.page, pl = a.kv.page_log2, np = kKeys >> pl;
    Items it;
    it.start(ka);
    Waiter wait{a};
    Turn use[2];
    while (it.next(ka)) {
        const int32_t* table = a.sq.table + int64_t(it.b) * a.sq.max_pages;
        const int p_hi = (it.s.len + page - 1) >> pl, p0 = it.j0 >> pl, p = p0 + lane;
        const bool mine = lane < 2 * np && p < p_hi;
        int pg = mine ? table[p] : 0;
        if (mine && (pg < 0 || pg >= a.kv.n_pages)) {
            record_error(a.err, MOE_ERR_INVALID_ARG);
            pg = a.kv.n_pages;                                  // out of range: reads as zeros
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int first = p0 + w * np, boxes = min(first + np, p_hi) - first;
            if (boxes <= 0) continue;
            const int buf = use[w].buf();
            wait(&sh.k_empty[w][buf], use[w].phase() ^ 1u);
            ++use[w].n;
            uint8_t* dst = smem + C::oRaw + (2 * w + buf) * C::kRaw;
            if (lane == 0)
                mbar_arrive_expect_tx(&sh.k_full[w][buf], wait.dead ? 0 : boxes * page * (E4M3 ? D : 2 * D));
            __syncwarp();
            for (int k = 0; k < np; ++k) {
                if (lane == w * np + k && mine && !wait.dead) {
#pragma unroll
                    for (int x = 0; x < kParts; ++x)
                        tma_load_4d(dst + k * page * kBoxBytes + x * kKeys * 128, &map, &sh.k_full[w][buf], x * kBox, 0,
                                    it.h, pg);
                }
                __syncwarp();
            }
        }
    }
}

template <int D, bool E4M3>
__device__ __forceinline__ void load_rows(const KeywArgs& ka, const CUtensorMap& map, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const int lane = threadIdx.x & 31;
    const uint32_t bytes = ka.tile_tokens * ka.tile_heads * D * 2;
    Items it;
    it.start(ka);
    Waiter wait{a};
    QSlot q;
    while (it.next(ka)) {
        for (int t = it.t0; t < it.t1; ++t)
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                wait(&sh.q_empty[q.st], q.ph ^ 1u);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_full[q.st], wait.dead ? 0 : bytes);
                    if (!wait.dead) {
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_3d(smem + C::oQ + q.st * C::kQTile + x * 16384, &map, &sh.q_full[q.st], 64 * x,
                                        it.h * a.group + hc, it.s.q0 + t * ka.tile_tokens);
                    }
                }
                __syncwarp();
                q.step();
            }
    }
}

template <int D, bool E4M3>
__device__ __forceinline__ void multiply(const KeywArgs& ka, Shared& sh, uint8_t* smem, int w) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const uint64_t q_desc = sdesc(smem_u32(smem + C::oQ), 16, 1024, kSw128);
    Items it;
    it.start(ka);
    Waiter wait{a};
    QSlot q;
    Turn key, buf;
    uint32_t kp = 0;
    while (it.next(ka)) {
        const bool on = it.j0 + w * kKeys < it.s.len;
        int kb = 0;
        uint64_t k_desc = 0;
        if (on) {
            if constexpr (E4M3) {
                wait(&sh.k_bf16[w], kp);
                kp ^= 1u;
                k_desc = sdesc(smem_u32(smem + C::oK + w * C::kTile), 16, 1024, kSw128);
            } else {
                kb = key.buf();
                wait(&sh.k_full[w][kb], key.phase());
                ++key.n;
                k_desc = sdesc(smem_u32(smem + C::oRaw + (2 * w + kb) * C::kRaw), 16, 1024, kSw128);
            }
        }
        for (int t = it.t0; t < it.t1; ++t) {
            const int tokens = min(ka.tile_tokens, it.s.nq - t * ka.tile_tokens);
            const uint32_t id = idesc(1, 1, false, (tokens * ka.tile_heads + 15) & ~15);
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                wait(&sh.q_full[q.st], q.ph);
                const int sb = buf.buf();
                if (on) {
                    wait(&sh.s_empty[w][sb], buf.phase() ^ 1u);
                    ++buf.n;
                }
                tc_fence_after();
                const uint64_t qd = q_desc + q.st * (C::kQTile >> 4);
                const uint32_t d = sh.tmem + (2 * w + sb) * 128;
                if (elect_one()) {
                    if (on) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                            mma_ss<false>(d, k_desc + off, qd + off, id, k > 0);
                        }
                        mma_commit(&sh.s_full[w][sb]);
                        mma_commit(&sh.q_empty[q.st]);
                    } else {
                        mbar_arrive(&sh.q_empty[q.st]);
                    }
                }
                __syncwarp();
                q.step();
            }
        }
        if (!E4M3 && on) {
            if (elect_one()) mma_commit(&sh.k_empty[w][kb]);
            __syncwarp();
        }
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

template <int D, bool E4M3>
__device__ __forceinline__ void weigh(const KeywArgs& ka, Shared& sh, uint8_t* smem) {
    using C = Cfg<D, E4M3>;
    const AttnArgs& a = ka.a;
    const int tid = threadIdx.x, w = tid >> 7, lr = tid & 127, lane = tid & 31, wq = (tid >> 5) & 3;
    const uint32_t tm = sh.tmem + (static_cast<uint32_t>(wq * 32) << 16) + 2 * w * 128;
    const bool draft = a.draft != nullptr;
    // the row of column lr: token and head within a tile
    const int r_tok = lr / ka.tile_heads, r_head = lr - r_tok * ka.tile_heads;
    Items it;
    it.start(ka);
    Waiter wait{a};
    Turn key, buf;
    while (it.next(ka)) {
        const int jt = it.j0 + w * kKeys;
        if (jt >= it.s.len) continue;
        if constexpr (E4M3) {
            const int kb = key.buf();
            wait(&sh.k_full[w][kb], key.phase());
            ++key.n;
            const uint8_t* raw = smem + C::oRaw + (2 * w + kb) * C::kRaw;
            uint8_t* dst = smem + C::oK + w * C::kTile;         // (its last products are done: their S was waited for)
#pragma unroll
            for (int ch = 0; ch < D / 16; ++ch) {
                const uint4 x = *reinterpret_cast<const uint4*>(
                    raw + lr * D + ((D == 128 ? ch ^ (lr & 7) : ch ^ ((lr >> 1) & 3)) << 4));
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = unpack_e4m3((xs[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
                    y[e] = pack_bf16(f.x, f.y);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c2 = 2 * ch + e;
                    *reinterpret_cast<uint4*>(dst + (c2 >> 3) * 16384 + lr * 128 + (((c2 & 7) ^ (lr & 7)) << 4)) =
                        make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.k_empty[w][kb]);
                mbar_arrive(&sh.k_bf16[w]);
            }
        }
        const int j = jt + lr;
        const int64_t at = (int64_t(it.b) * a.kv.heads + it.h) * ka.score_stride + j;
        const bool store = j < it.s.len && j < ka.score_stride;
        const float before = store && j < it.s.first ? ka.decay * ka.scores[at] : 0.0f;
        const float c = a.scale * kLog2e * (E4M3 ? a.kv.k_scale[it.h] : 1.0f);
        const int heads_left = a.group;
        // the next tile's log-sum-exp of this thread's column, a tile ahead
        auto row_lse = [&](int t, int hc) {
            const int i = t * ka.tile_tokens + r_tok, hd = hc + r_head;
            const bool ok = t < it.t1 && r_tok < ka.tile_tokens && i < it.s.nq && hd < heads_left;
            return ok ? __ldg(a.lse + int64_t(it.s.q0 + i) * a.q_heads + it.h * a.group + hd) : kNegInf;
        };
        float z = row_lse(it.t0, 0), sum = 0.0f;
        for (int t = it.t0; t < it.t1; ++t) {
            const int i0 = t * ka.tile_tokens, tokens = min(ka.tile_tokens, it.s.nq - i0);
            const bool seen = (draft ? jt + kKeys <= it.s.first : !a.causal || jt + kKeys <= it.s.first + i0 + 1) &&
                              !(a.window > 0 && jt <= it.s.first + i0 + tokens - 1 - a.window);
            for (int hc = 0; hc < a.group; hc += ka.tile_heads) {
                const int sb = buf.buf(), rows = tokens * min(ka.tile_heads, a.group - hc);
                const bool live = fabsf(z) != INFINITY;
                sh.off[w][sb][lr] = live ? -z * kLog2e : 0.0f;
                const uint32_t word = __ballot_sync(0xFFFFFFFFu, live);
                if (lane == 0) sh.live[w][sb][wq] = word;
                named_bar(1 + w, 128);
                z = hc + ka.tile_heads < a.group ? row_lse(t, hc + ka.tile_heads) : row_lse(t + 1, 0);
                wait(&sh.s_full[w][sb], buf.phase());
                ++buf.n;
                tc_fence_after();
                const uint32_t col = tm + sb * 128;
                const float* off = sh.off[w][sb];
                const uint32_t* words = sh.live[w][sb];
                float p0 = 0.0f, p1 = 0.0f;
                if (seen && rows == 128 && (words[0] & words[1] & words[2] & words[3]) == 0xFFFFFFFFu) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) add_powers<32, false>(col + 32 * q, off + 32 * q, c, 0, p0, p1);
                } else {
                    // columns of rows that see key j: a range by token, or by the rows' draft masks
                    int lo = 0, hi = rows;
                    const int64_t rel = int64_t(j) - it.s.first - i0;         // j's place less the tile's first token's
                    const int th = ka.tile_heads;
                    if (!draft && a.causal) lo = static_cast<int>(max(int64_t(0), min(rel, int64_t(128)))) * th;
                    if (a.window > 0) hi = min(hi, static_cast<int>(max(int64_t(0), min(rel + a.window, int64_t(128)))) * th);
#pragma unroll 1
                    for (int n = 0; n < rows; n += 16) {
                        uint32_t bits = (words[n >> 5] >> (n & 16)) & 0xFFFFu;
                        if (!seen) {
                            const int l = min(max(lo - n, 0), 16), u = min(max(hi - n, 0), 16);
                            bits &= ((1u << u) - 1u) & ~((1u << l) - 1u);
                            const int place = j - it.s.first;
                            if (draft && place >= 0) {
                                for (int e = 0; e < 16 && n + e < rows; ++e) {
                                    const uint64_t m = a.draft[it.s.q0 + i0 + (n + e) / th];
                                    if (place >= 64 || !((m >> place) & 1ull)) bits &= ~(1u << e);
                                }
                            }
                        }
                        add_powers<16, true>(col + n, off + n, c, bits, p0, p1);
                        __syncwarp();
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

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1) keyw_kernel(const KeywArgs ka, const __grid_constant__ KeywMaps maps) {
    using C = Cfg<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int w = 0; w < 2; ++w) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.k_full[w][i], 1);
                mbar_init(&sh.k_empty[w][i], E4M3 ? 4 : 1);
                mbar_init(&sh.s_full[w][i], 1);
                mbar_init(&sh.s_empty[w][i], 4);
            }
            mbar_init(&sh.k_bf16[w], 4);
        }
        for (int i = 0; i < kQStages; ++i) {
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
    if (warp < 8)
        weigh<D, E4M3>(ka, sh, smem);
    else if (warp == 8)
        load_keys<D, E4M3>(ka, maps.k, sh, smem);
    else if (warp == 9)
        load_rows<D, E4M3>(ka, maps.q, sh, smem);
    else
        multiply<D, E4M3>(ka, sh, smem, warp - 10);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10) tmem_dealloc(sh.tmem, 512);
}

template <int D, bool E4M3>
cudaError_t launch(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s) {
    constexpr size_t smem = Cfg<D, E4M3>::kBytes + sizeof(Shared);
    static_assert(smem <= 232448, "227 KB a CTA");
    cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(keyw_kernel<D, E4M3>), static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(keyw_kernel<D, E4M3>, dim3(n_sms), dim3(kThreads), smem, s, a, m);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_keyw(const KeywArgs& a, const KeywMaps& m, int n_sms, cudaStream_t s) {
    if (a.a.kv.dim == 128) return a.a.kv.e4m3 ? launch<128, true>(a, m, n_sms, s) : launch<128, false>(a, m, n_sms, s);
    return a.a.kv.e4m3 ? launch<64, true>(a, m, n_sms, s) : launch<64, false>(a, m, n_sms, s);
}

}  // namespace moe
