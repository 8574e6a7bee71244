// kv_attend.cu -- attention of new tokens over the dense paged cache
// (csla_kv_attend): requests of more than 16 rows per KV head (shorter ones
// are kv_few.cu's), and the join of rows whose keys were cut.
//
//   s_j = scale <R(p) norm(q), K_j>,  o = sum_j e^{s_j} V_j / (e^{sink} + sum_j e^{s_j})
//
// Rows.  The T new tokens of a request and the G query heads of one KV head
// make T*G rows of one matrix (row = token * G + head): they share every key.
// A page (128 tokens of one KV head) is one tile of keys and values.
//
// Work.  A CTA works on items.  A request of 17 to 128 rows per KV head is
// one row tile, its keys cut into chunks of tiles; one item is a chunk, and
// the CTA's two streams take its tiles in turn.  A request of more rows is
// cut into row tiles of 256; one item is such a tile (and a chunk of its keys
// when there are few row tiles), each stream takes 128 of the rows and both
// share every key tile.  How a request is cut depends on its own T and len
// and the layer's shape alone (kv_plan), so its results do not depend on the
// batch.  Rows whose keys were cut are left as partial (m, l, O) in the
// workspace and joined, in order, by kv_join_kernel.
//
// Roles (one persistent CTA per SM, 16 warps):
//   warps 0-3, 4-7  softmax of stream 0, 1: a thread per row; a running maximum
//                   and sum in fp32, P in bf16 back to tensor memory.  O is
//                   rescaled only when the maximum has grown by more than 2^8:
//                   a row's weights are all formed with one reference, so any
//                   reference cancels in O / sum, and 2^8 keeps both in range;
//   warps 8-11      Q: norm and rotation in fp32, rounded to bf16 into the
//                   swizzled operand;
//   warp 12         tcgen05.mma S = Q K^T;
//   warp 13         TMA: K and V tiles into a ring each;
//   warp 14         the items: walks the batch 32 requests at a time;
//   warp 15         tcgen05.mma O += P V (P from tensor memory).
// Tensor memory (512 columns): O of both streams 256, P of both 128, and one S
// of 128 that the streams use in turn.  A softmax thread takes its whole row of
// S into registers at once, so the S columns are free for the other stream's
// scores while it forms its weights, and a stream's next scores wait for it.
//
// Roundings.  P is rounded to bf16 (half a step of each weight; their sum is
// of the unrounded ones).  The rotated query is rounded to bf16, and what the
// rounding left is kept as a second bf16 operand: its S costs twice, which a
// row tile bound by its keys' bytes has to spare, and so has one of 64 dims, which is
// bound by the exponentials (a mixed batch of 28 heads x 64: 67 us without, 68
// with, error 0.0025 and 0.0020 of the output).  A row tile of 256 rows of 128
// dims has neither the shared memory for it nor tensor time to spare (half again
// as many products): its scores carry half a bf16 step of the query (error
// 0.0025 to 0.0029, where 0.0023 is the rounding of P and of the output).
//
// Bound and measured (32 query and 8 KV heads of 128 dims, unless said).
// Row tiles of 256 are bound by the tensor cores and, beside them, by the
// exponentials (16 per clock and SM: 128 x 128 take 1024 clocks, the tile's
// products 1024 too): 4096 tokens after 16384 (4 KV heads) take 1.09 ms, 1.13 PFLOP/s, 0.69
// of what one large library product measures in a burst; at that length the
// clock falls to about 1.4 GHz under the power limit.  2048 tokens alone: 57 us
// (0.37; 256 items of 1 to 16 tiles on 148 SMs).  One chunk of 17 to 128
// rows waits for its chain of S, softmax and P V: 32 requests of 20 rows 132 us for
// 526 MB (4.0 TB/s), 4 requests of 64 rows on one KV head over 262144
// tokens 149 us for 537 MB (3.6 TB/s); with the pages in L2 they take as long:
// 2350 clocks per tile and some 12 000 per item, between its last product and
// the next item's first.
#include "kv.cuh"

namespace csla {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = CSLA_PAGE_TOKENS;   // keys per tile
constexpr int kItems = 3;                 // items in flight between the roles
constexpr int kFlags = 16;                // tiles of page flags

template <int D>
struct Cfg {
    static constexpr int kKB = D / 64;                  // 64-dim blocks (128-byte rows)
    static constexpr int kBlk = 128 * 128;              // bytes of a block: 128 rows x 128 B
    static constexpr int kTileBytes = kKB * kBlk;
    static constexpr int kKStages = D == 128 ? 3 : 5, kVStages = D == 128 ? 2 : 5;
    static constexpr int kOffQ = 0;
    // the rounding's rest of Q, behind both streams' operands with 64 dims; with 128
    // only a single row tile has one, in the other stream's place
    static constexpr bool kPairedRest = D == 64;
    static constexpr int kOffRest = (kPairedRest ? 2 : 1) * kTileBytes;
    static constexpr int kOffK = (kPairedRest ? 4 : 2) * kTileBytes;
    static constexpr int kOffV = kOffK + kKStages * kTileBytes;
    static constexpr int kOffMisc = kOffV + kVStages * kTileBytes;
    // TMEM columns: one S, which the streams use in turn, P of each stream, O of each stream
    static constexpr int kColS = 0, kColP = 128, kColO = 256;
};

struct Item {
    int end;             // no more items
    int paired;          // two row tiles on the same keys; else one row tile, tiles in turn
    int n0, T, pos0;     // request: first row of q and out, new tokens, position of the first
    int slot, hk;
    int row0, rows;      // first row of the item, rows of the request
    int tok0, head0;     // token and head (of the KV head's) of row0
    int rows_s;          // rows whose keys are cut
    int lo, hi;          // key tiles [lo, hi)
    int hi0, lo1;        // paired: stream 0 takes [lo, hi0), stream 1 [lo1, hi)
    int k_lo, k_hi;      // positions that some row of the row tile sees: [k_lo, k_hi)
    int part;            // index of the item's (first) partial, -1: rows are written out
    long long base;      // first partial row of the request
};

struct Misc {
    Item item[kItems];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t k_full[5], k_empty[5], v_full[5], v_empty[5];
    uint64_t q_full[2], q_empty[2], s_full[2], s_free[2], p_full[2], pv_done[2], drain[2];
    int bad[kFlags];     // tile's page is not mapped
    unsigned long long turn[64];   // rotation frequencies
    uint32_t tmem;
    int abort;
};

template <int D>
constexpr int smem_bytes() {
    return Cfg<D>::kOffMisc + (int)sizeof(Misc) + 1024;
}

// ---------------------------------------------------------------- items
// Item `local` of a request, in the order: row tiles from the last (the longest
// under the causal mask) to the first; heads inside, unless the request's
// keys would not stay in L2 while all heads are in use.
__device__ __forceinline__ bool make_item(const KvAttendArgs &a, const KvReq &r, const KvPlan &p, int local,
                                          long long base, Item *it) {
    int i, hk, j = 0, n = a.HK * (p.R - p.Rs), top = p.R - 1, tiles = p.R - p.Rs;   // whole row tiles first
    if (local >= n) {
        local -= n;
        const int x = kv_div(local, p.nch);
        j = local - x * p.nch;
        local = x;
        top = p.Rs - 1;
        tiles = p.Rs;
    }
    const bool cut = top < p.Rs;
    if (p.heads_inside) {
        const int x = kv_div(local, a.HK);
        hk = local - x * a.HK;
        i = top - x;
    } else {
        hk = kv_div(local, tiles);
        i = top - (local - hk * tiles);
    }
    const KvRange g = kv_range(p, r.L - r.T, i, a.window);
    const int lo = g.lo + j * p.c, hi = cut ? min(g.hi, lo + p.c) : g.hi;
    if (lo >= hi) return false;
    it->end = 0;
    it->paired = p.kind == kKvPaired;
    it->n0 = r.n0;
    it->T = r.T;
    it->pos0 = r.L - r.T;
    it->slot = r.slot;
    it->hk = hk;
    it->row0 = i * 256;
    it->tok0 = kv_div(i * 256, p.G);
    it->head0 = i * 256 - it->tok0 * p.G;
    it->rows = p.rows;
    it->rows_s = p.rows_s;
    it->lo = lo;
    it->hi = hi;
    it->hi0 = min(hi, g.hi0);
    it->lo1 = max(lo, g.lo1);
    it->k_lo = g.k_lo;
    it->k_hi = g.k_hi;
    const int parts = kv_parts(p, g, i);
    it->part = parts > 1 ? (p.kind == kKvPaired ? j : 2 * j) : -1;
    it->base = base;
    return true;
}

__device__ void sched_role(const KvAttendArgs &a, Misc *ms) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    kv_walk(a, 1u << kKvSingle | 1u << kKvPaired, [&](const KvWalk &w, bool more, int src, int local) {
        Item it;
        it.end = 1;
        bool have = true;
        if (more && lane == src) have = make_item(a, w.r, w.p, local, w.part_before + w.part_excl, &it);
        if (!__shfl_sync(0xffffffffu, (int)have, src)) return true;   // (a chunk behind a short row tile's keys)
        const int slot = n % kItems;
        if (n >= kItems && !warp_all(kv_wait(&ms->item_empty[slot], (n / kItems - 1) & 1, &ms->abort, kItemLimitNs))) return false;
        if (lane == src) ms->item[slot] = it;
        if (n == 0 && lane == 0) CSLA_TL_MARK_ANY(0);
        mbar_arrive_warp(&ms->item_full[slot]);
        ++n;
        return true;
    });
}

// The next item for a role's warp; false when there is none (or on an abort).
__device__ __forceinline__ bool next_item(Misc *ms, int n, Item *it) {
    const int slot = n % kItems;
    if (!warp_all(kv_wait(&ms->item_full[slot], (n / kItems) & 1, &ms->abort))) return false;
    *it = ms->item[slot];
    mbar_arrive_warp(&ms->item_empty[slot]);
    return !it->end;
}

// ---------------------------------------------------------------- TMA role
// A ring's next stage and the parity of its phase.
template <int N>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == N) {
            stage = 0;
            phase ^= 1;
        }
    }
};

template <int D>
struct Loader {
    using C = Cfg<D>;
    const KvAttendArgs &a;
    uint8_t *smem;
    Misc *ms;
    int lane;
    Ring<C::kKStages> kr;     // (phase of the stage's next filling)
    Ring<C::kVStages> vr;
    int ks = 0, vs = 0;       // tiles issued
    // page ids of 64 tiles from `at` on, two per lane
    int at = 0, pg0 = -1, pg1 = -1;

    __device__ __forceinline__ int fetch(const Item &it, int t) const {
        return t < it.hi ? a.bt.block_table[(long long)it.slot * a.bt.bt_stride + t] : -1;
    }
    __device__ __forceinline__ void begin(const Item &it) {
        at = it.lo;
        pg0 = fetch(it, at + lane);
        pg1 = fetch(it, at + 32 + lane);
    }
    __device__ __forceinline__ int page(const Item &it, int t) {
        // tiles are asked for in ascending order, V two behind K at most
        if (t >= at + 64) {
            at += 32;
            pg0 = pg1;
            pg1 = fetch(it, at + 32 + lane);
        }
        const int d = t - at;
        return d < 32 ? __shfl_sync(0xffffffffu, pg0, d & 31) : __shfl_sync(0xffffffffu, pg1, d & 31);
    }
    template <int N>
    __device__ __forceinline__ bool load(const CUtensorMap &map, Ring<N> &r, int issued, uint64_t *full, uint64_t *empty,
                                         uint8_t *ring, int row) {
        if (issued >= N && !warp_all(kv_wait(&empty[r.stage], r.phase ^ 1, &ms->abort))) return false;
        if (lane == 0) {
            uint64_t *bar = &full[r.stage];
            mbar_arrive_expect_tx(bar, C::kTileBytes);
            uint8_t *dst = ring + r.stage * C::kTileBytes;
#pragma unroll
            for (int kb = 0; kb < C::kKB; ++kb) tma_load_2d(dst + kb * C::kBlk, &map, 64 * kb, row, bar);
        }
        __syncwarp();
        r.next();
        return true;
    }
    __device__ __forceinline__ bool load_k(const Item &it, int t, const CUtensorMap &map) {
        const int pg = page(it, t);
        const bool bad = pg < 0 || pg >= a.bt.n_pages;
        if (lane == 0) {
            ms->bad[ks % kFlags] = bad;
            if (bad) set_dev_err(CSLA_DEVERR_PAGE);
        }
        // (an unmapped page's tile is page 0's, masked)
        return load(map, kr, ks++, ms->k_full, ms->k_empty, smem + C::kOffK, ((bad ? 0 : pg) * a.HK + it.hk) * kTile);
    }
    __device__ __forceinline__ bool load_v(const Item &it, int t, const CUtensorMap &map) {
        const int pg = page(it, t);
        const bool bad = pg < 0 || pg >= a.bt.n_pages;
        return load(map, vr, vs++, ms->v_full, ms->v_empty, smem + C::kOffV, ((bad ? 0 : pg) * a.HK + it.hk) * kTile);
    }
};

template <int D>
__device__ void load_role(const KvAttendArgs &a, const CUtensorMap &km, const CUtensorMap &vm, uint8_t *smem, Misc *ms) {
    using C = Cfg<D>;
    Loader<D> L{a, smem, ms, (int)(threadIdx.x & 31)};
    bool ok = true;
    Item it;
    for (int n = 0; ok && next_item(ms, n, &it); ++n) {
        L.begin(it);
        const int d = it.paired ? 1 : 2;   // V follows its K by d tiles: the order in which they are used
        for (int t = it.lo; ok && t < it.hi + d; ++t) {
            if (t < it.hi) ok = L.load_k(it, t, km);
            if (ok && t - d >= it.lo) ok = L.load_v(it, t - d, vm);
        }
    }
    // copies in flight land before the CTA exits (all have, unless a wait gave up)
    for (int i = max(0, L.ks - C::kKStages); i < L.ks; ++i)
        kv_wait(&ms->k_full[i % C::kKStages], (i / C::kKStages) & 1, nullptr);
    for (int i = max(0, L.vs - C::kVStages); i < L.vs; ++i)
        kv_wait(&ms->v_full[i % C::kVStages], (i / C::kVStages) & 1, nullptr);
}

// ---------------------------------------------------------------- Q role
// Q rows of one stream's operand by four warps (warp = 0..3 of them): norm and
// rotation in fp32, rounded to bf16 into the swizzled operand, the rounding's
// rest into another where there is one.
template <int D, bool QBF16>
struct QRows {
    using C = Cfg<D>;
    static constexpr int kLanes = D / 8, kPer = 32 / kLanes;   // lanes per row, rows per step
    // Rows of a lane at a time: enough for two chains of latencies to overlap, and
    // little code, which the instruction cache has lost since the item before.
    static constexpr int kGroup = 2;
    const KvAttendArgs &a;
    uint8_t *smem;
    Misc *ms;
    int warp, lane, sub, G, b0, b1;
    RowLane rl;
    float g[8];
    unsigned long long turn[4];

    __device__ __forceinline__ QRows(const KvAttendArgs &a_, uint8_t *smem_, Misc *ms_) : a(a_), smem(smem_), ms(ms_) {
        warp = (threadIdx.x >> 5) & 3;
        lane = threadIdx.x & 31;
        const int c = lane % kLanes;
        sub = lane / kLanes;
        G = a.HQ / a.HK;
        rl = row_lane<D>(c, a.d_rope, a.pairs);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = a.gamma_q ? a.gamma_q[i < 4 ? rl.d0 + i : rl.d1 + i - 4] : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) turn[j] = rl.pair >= 0 ? ms->turn[rl.pair + j] : 0;
        // byte offsets of the lane's runs in a row of the operand (row 0's swizzle)
        b0 = (rl.d0 >> 6) * C::kBlk + (rl.d0 & 63) * 2;
        b1 = (rl.d1 >> 6) * C::kBlk + (rl.d1 & 63) * 2;
    }
    // Operand s of the CTA's n-th item.
    __device__ __forceinline__ bool stage(const Item &it, int s, int n) {
        // a lane takes kGroup neighbouring rows (mostly heads of one token: one
        // rotation for all), the four warps kPass rows
        constexpr int kPass = 4 * kGroup * kPer;
        const int r0 = it.row0 + 128 * s, first = kGroup * (warp * kPer + sub);
        const int groups = min(128 / kPass, (it.rows - r0 - kGroup * warp * kPer + kPass - 1) / kPass);
        Raw8<QBF16> next[kGroup];
        int npos[kGroup];
        auto fetch = [&](int gr) {
            // (row - row0 + head0 < 384, G <= 128: exact)
            const int y = r0 - it.row0 + first + kPass * gr + it.head0, of = y * a.inv_g >> 16;
            int tok = it.tok0 + of, head = y - of * G;
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int t = min(tok, it.T - 1);   // (rows that are not there: any)
                npos[k] = it.pos0 + t;
                next[k] = load8<QBF16>(a.q, (long long)(it.n0 + t) * a.q_stride + (it.hk * G + head) * D, rl);
                if (++head == G) {
                    head = 0;
                    ++tok;
                }
            }
        };
        bool waited = n == 0;
        if (groups > 0) fetch(0);
#pragma unroll 1
        for (int gr = 0; gr < groups; ++gr) {
            Raw8<QBF16> raw[kGroup];
            int pos[kGroup];
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                raw[k] = next[k];
                pos[k] = npos[k];
            }
            if (gr + 1 < groups) fetch(gr + 1);   // a group ahead
            // (the first rows' loads are in flight while the operand is still in use)
            if (!waited) {
                if (!warp_all(kv_wait(&ms->q_empty[s], (n - 1) & 1, &ms->abort, kItemLimitNs))) return false;
                if (!it.paired && !warp_all(kv_wait(&ms->q_empty[1], (n - 1) & 1, &ms->abort, kItemLimitNs))) return false;
                waited = true;
            }
            float x[kGroup][8];
#pragma unroll
            for (int k = 0; k < kGroup; ++k) widen8<QBF16>(raw[k], x[k]);
            if (a.gamma_q) rows_norm<D>(x, g, a.eps);
            if (a.d_rope) {
                float2 cs[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) cs[j] = kv_cos_sin(pos[0], turn[j]);   // (turn 0: unchanged)
                const bool one = __all_sync(0xffffffffu, pos[0] == pos[kGroup - 1]);
                row_rope(x[0], a.pairs, cs);
                if (one) {
#pragma unroll
                    for (int k = 1; k < kGroup; ++k) row_rope(x[k], a.pairs, cs);
                } else {
#pragma unroll
                    for (int k = 1; k < kGroup; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) cs[j] = kv_cos_sin(pos[k], turn[j]);
                        row_rope(x[k], a.pairs, cs);
                    }
                }
            }
            const int i0 = first + kPass * gr;   // first row of the operand, a multiple of kGroup
            uint8_t *dst = smem + C::kOffQ + s * C::kTileBytes + i0 * 128;
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int sw = ((i0 & 7) + k) << 4;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint2 o = make_uint2(pack_bf16(x[k][4 * h], x[k][4 * h + 1]),
                                               pack_bf16(x[k][4 * h + 2], x[k][4 * h + 3]));
                    *reinterpret_cast<uint2 *>(dst + k * 128 + ((h ? b1 : b0) ^ sw)) = o;
                    x[k][4 * h] -= __uint_as_float(o.x << 16);
                    x[k][4 * h + 1] -= __uint_as_float(o.x & 0xFFFF0000u);
                    x[k][4 * h + 2] -= __uint_as_float(o.y << 16);
                    x[k][4 * h + 3] -= __uint_as_float(o.y & 0xFFFF0000u);
                }
            }
            if (C::kPairedRest || !it.paired) {   // the rest of the rounding
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const int sw = ((i0 & 7) + k) << 4;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<uint2 *>(dst + C::kOffRest + k * 128 + ((h ? b1 : b0) ^ sw)) =
                            make_uint2(pack_bf16(x[k][4 * h], x[k][4 * h + 1]),
                                       pack_bf16(x[k][4 * h + 2], x[k][4 * h + 3]));
                }
            }
        }
        if (!waited) {   // (no row of this warp: the operand's phases are kept in step all the same)
            if (!warp_all(kv_wait(&ms->q_empty[s], (n - 1) & 1, &ms->abort, kItemLimitNs))) return false;
            if (!it.paired && !warp_all(kv_wait(&ms->q_empty[1], (n - 1) & 1, &ms->abort, kItemLimitNs))) return false;
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&ms->q_full[s]);
        if (!it.paired) mbar_arrive_warp(&ms->q_full[1]);
        return true;
    }
};

template <int D, bool QBF16>
__device__ void q_role(const KvAttendArgs &a, uint8_t *smem, Misc *ms) {
    QRows<D, QBF16> q(a, smem, ms);
    Item it;
    for (int n = 0; next_item(ms, n, &it); ++n) {
        if (n == 0) continue;   // the softmax warps', which have nothing else to do yet
#pragma unroll 1
        for (int s = 0; s <= it.paired; ++s)
            if (!q.stage(it, s, n)) return;
    }
}

// ---------------------------------------------------------------- MMA roles
// The products of a step are 8 to 16 instructions of 64 tensor cycles each,
// and the tensor cores queue little: what the issuing thread does between two
// steps is time they stand still.  So S and PV have a warp each, their only
// order is what the barriers say, and a step's descriptors are a warp-uniform base
// plus constants in the low word (address and leading offset, in 16-byte
// units); the high word is the same for all operands (stride of 8-row groups
// 1024 bytes, version 1, 128-byte swizzle).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (kLayoutSW128 << 29);
__device__ constexpr uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) { return (saddr >> 4) | (lbo_bytes >> 4) << 16; }

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
        : "memory");
}

template <int D>
__device__ void s_role(uint8_t *smem, Misc *ms) {
    using C = Cfg<D>;
    constexpr uint32_t kId = idesc_bf16(128, kTile, false, false);
    const uint32_t d = uniform(ms->tmem) + C::kColS;
    const uint32_t q0 = uniform(desc_lo(smem_u32(smem + C::kOffQ), 16)), k0 = uniform(desc_lo(smem_u32(smem + C::kOffK), 16));
    Ring<C::kKStages> kr;
    uint32_t free0 = 0, free1 = 0;   // phases of s_free
    int pending = -1;                // stream of the last S, not yet waited for
    Item it;
    // S of stream s = Q K^T (both terms of Q where it has two) from K's stage, once the scores before it have been read
    auto step = [&](int s, bool paired, bool last) {
        if (pending >= 0) {
            if (!warp_all(kv_wait(&ms->s_free[pending], pending ? free1 : free0, &ms->abort))) return false;
            if (pending) free1 ^= 1;
            else free0 ^= 1;
        }
        pending = s;
        tc_fence_after();
        const uint32_t k = uniform(k0 + (uint32_t)kr.stage * (C::kTileBytes >> 4));
        const uint32_t q = uniform(q0 + (paired && s ? C::kTileBytes >> 4 : 0));
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4 * C::kKB; ++i) {
                const uint32_t off = ((i >> 2) * C::kBlk + (i & 3) * 32) >> 4;
                umma_ss(d, q + off, k + off, kId, i > 0);
            }
            if (C::kPairedRest || !paired) {
#pragma unroll
                for (int i = 0; i < 4 * C::kKB; ++i) {
                    const uint32_t off = ((i >> 2) * C::kBlk + (i & 3) * 32) >> 4;
                    umma_ss(d, q + (C::kOffRest >> 4) + off, k + off, kId, 1);
                }
            }
            umma_commit(&ms->s_full[s]);
            if (last) {   // Q is free
                umma_commit(&ms->q_empty[s]);
                if (!paired) umma_commit(&ms->q_empty[s ^ 1]);
            }
        }
        __syncwarp();
        return true;
    };
    bool ok = true;
    for (int n = 0; ok && next_item(ms, n, &it); ++n) {
        ok = warp_all(kv_wait(&ms->q_full[0], n & 1, &ms->abort) && kv_wait(&ms->q_full[1], n & 1, &ms->abort));
        if (n == 0 && (threadIdx.x & 31) == 0) CSLA_TL_MARK_ANY(1);
        const bool paired = it.paired;
#pragma unroll 1
        for (int t = it.lo; ok && t < it.hi; ++t) {
            ok = warp_all(kv_wait(&ms->k_full[kr.stage], kr.phase, &ms->abort));
            if (!ok) break;
            if (paired) {
                if (t < it.hi0) ok = step(0, true, t + 1 == it.hi0);
                if (ok && t >= it.lo1) ok = step(1, true, t + 1 == it.hi);
            } else {
                ok = step((t - it.lo) & 1, false, t + 1 == it.hi);
            }
            if (elect_one()) umma_commit(&ms->k_empty[kr.stage]);
            __syncwarp();
            kr.next();
        }
        // a stream without a key tile has not used its Q
        if (ok && paired && elect_one()) {
            if (it.hi0 <= it.lo) umma_commit(&ms->q_empty[0]);
            if (it.lo1 >= it.hi) umma_commit(&ms->q_empty[1]);
        }
        __syncwarp();
    }
    // products in flight end before tensor memory is freed (all have, unless a wait gave up)
    if (elect_one()) umma_commit(&ms->drain[0]);
    __syncwarp();
    kv_wait(&ms->drain[0], 0, nullptr);
}

template <int D>
__device__ void pv_role(uint8_t *smem, Misc *ms) {
    using C = Cfg<D>;
    constexpr uint32_t kId = idesc_bf16(128, D, false, true);
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = uniform(ms->tmem), v0 = uniform(desc_lo(smem_u32(smem + C::kOffV), C::kBlk));
    Ring<C::kVStages> vr;
    uint32_t p0 = 0, p1 = 0;   // phases of p_full
    int tiles = 0;
    Item it;
    // O of stream s (+)= P V once P is there
    auto step = [&](int s, bool first) {
        if (!warp_all(kv_wait(&ms->p_full[s], s ? p1 : p0, &ms->abort))) return false;
        if (s) p1 ^= 1;
        else p0 ^= 1;
        tc_fence_after();
        const uint32_t v = uniform(v0 + (uint32_t)vr.stage * (C::kTileBytes >> 4)), acc = uniform(first ? 0u : 1u);
        const uint32_t o = uniform(tmem + C::kColO + D * s), p = uniform(tmem + C::kColP + 64 * s);
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kTile / 16; ++i) umma_ts(o, p + 8 * i, v + (i * 2048 >> 4), kId, i > 0 ? 1u : acc);
            umma_commit(&ms->pv_done[s]);
        }
        __syncwarp();
        return true;
    };
    bool ok = true;
    for (int n = 0; ok && next_item(ms, n, &it); ++n) {
        const bool paired = it.paired;
#pragma unroll 1
        for (int t = it.lo; ok && t < it.hi; ++t) {
            ok = warp_all(kv_wait(&ms->v_full[vr.stage], vr.phase, &ms->abort));
            if (!ok) break;
            // V rows that no row of the item sees are set to zero: their
            // weights are zero, but 0 * NaN is not
            const bool bad = ms->bad[(tiles + t - it.lo) % kFlags];
            const int lo = it.k_lo - t * kTile, hi = bad ? 0 : it.k_hi - t * kTile;
            if (lo > 0 || hi < kTile) {
                uint8_t *v = smem + C::kOffV + vr.stage * C::kTileBytes;
                for (int i = lane; i < kTile * 8; i += 32) {
                    const int row = i >> 3;
                    if (row >= lo && row < hi) continue;
#pragma unroll
                    for (int kb = 0; kb < C::kKB; ++kb)
                        *reinterpret_cast<uint4 *>(v + kb * C::kBlk + i * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (paired) {
                if (t < it.hi0) ok = step(0, t == it.lo);
                if (ok && t >= it.lo1) ok = step(1, t == it.lo1);
            } else {
                ok = step((t - it.lo) & 1, t < it.lo + 2);
            }
            if (elect_one()) umma_commit(&ms->v_empty[vr.stage]);
            __syncwarp();
            vr.next();
        }
        tiles += it.hi - it.lo;
    }
    if (elect_one()) umma_commit(&ms->drain[1]);
    __syncwarp();
    kv_wait(&ms->drain[1], 0, nullptr);
}

// ---------------------------------------------------------------- softmax role
// 32 bytes of a row: one whole sector per thread.
__device__ __forceinline__ void store32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d),
                 "r"(e), "r"(f), "r"(g), "r"(h)
                 : "memory");
}
// Two fp32 lanes of one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float *a, float *b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

template <int D, bool QBF16, bool OBF16>
__device__ void softmax_role(const KvAttendArgs &a, uint8_t *smem, Misc *ms, int s) {
    using C = Cfg<D>;
    const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const uint32_t tw = ms->tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t ts = tw + C::kColS, tp = tw + C::kColP + 64 * s, to = tw + C::kColO + D * s;
    const int G = a.HQ / a.HK;
    const float sc = a.scale * kLog2e;
    int s_count = 0, tiles = 0;   // S tiles taken; the PV of tile s_count - 1 frees P and leaves O
    for (int n = 0;; ++n) {
        // the item stays in its slot to the end: what the key loop does not
        // need is read there again, its registers hold scores
        const int slot = n % kItems;
        if (!warp_all(kv_wait(&ms->item_full[slot], (n / kItems) & 1, &ms->abort))) return;
        const Item &it = ms->item[slot];
        if (it.end) {
            mbar_arrive_warp(&ms->item_empty[slot]);
            return;
        }
        const bool paired = it.paired;
        // the first item's Q is on nobody's time but the SM's: each stream's
        // four warps stage their own (256 rows: 11 us by the Q warps, half by these)
        if (n == 0 && (paired || s == 0)) {
            QRows<D, QBF16> q(a, smem, ms);
            if (!q.stage(it, s, 0)) return;
        }
        const int row = it.row0 + (it.paired ? 128 * s : 0) + 32 * warp + lane;
        const bool mine = row < it.rows;
        const bool idle = it.row0 + (it.paired ? 128 * s : 0) + 32 * warp >= it.rows;   // no row of the warp is real
        const int r = min(row, it.rows - 1);
        // (row - row0 + head0 < 384, G <= 128: exact)
        const int y = r - it.row0 + it.head0, pos = it.pos0 + it.tok0 + (y * a.inv_g >> 16);
        const int low = a.window > 0 ? pos - a.window + 1 : 0;
        float m = -INFINITY, l = 0.f;   // m: the maximum the weights are formed with (score * sc)
        bool any = false;
        const int lo = it.lo, t0 = paired ? (s == 0 ? lo : it.lo1) : lo + s, t1 = paired && s == 0 ? it.hi0 : it.hi;
        for (int t = t0; t < t1; t += paired ? 1 : 2) {
            if (!warp_all(kv_wait(&ms->s_full[s], s_count & 1, &ms->abort))) return;
            if (s == 0 && s_count == 0 && threadIdx.x == 0) CSLA_TL_MARK_ANY(2);
            ++s_count;
            tc_fence_after();
            if (!idle) {
                const bool bad = ms->bad[(tiles + t - lo) % kFlags];
                const int last = bad ? -1 : pos - t * kTile, from = low - t * kTile;   // visible columns
                const bool cut = __any_sync(0xffffffffu, last < kTile - 1 || from > 0);
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32x32(ts + 32 * c, v[c]);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive_warp(&ms->s_free[s]);
                if (cut) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        // bit i: column 32 c + i is visible
                        const uint32_t below = last < 32 * c ? 0u : (last >= 32 * c + 31 ? ~0u : (2u << (last - 32 * c)) - 1u);
                        const uint32_t above = from <= 32 * c ? ~0u : (from > 32 * c + 31 ? 0u : ~0u << (from - 32 * c));
                        const uint32_t see = below & above;
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[c][i] = see >> i & 1 ? v[c][i] : 0xFF800000u;
                    }
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
                    for (int i = 2; i < 32; i += 2)
                        mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(v[c][i])), __uint_as_float(v[c][i + 1]));
                }
                const float least = last >= 0 && from < kTile ? fmaxf(m, kLeast) : m;   // (from <= last)
                const float mn = fmaxf(least, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc);
                const bool grow = mn > m + kGrow;   // (also from -inf)
                if (any) {   // P and O of the tile before
                    if (!warp_all(kv_wait(&ms->pv_done[s], s_count & 1, &ms->abort))) return;
                    tc_fence_after();
                }
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? (m == -INFINITY ? 0.f : ex2(m - mn)) : 1.f;
                    if (grow) m = mn;
                    l *= f;
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld32x16(to + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32x16(to + 16 * c, o);
                        }
                    }
                }
                const float sub = m == -INFINITY ? 0.f : m;
                const uint64_t sc2 = pack2(sc, sc), sub2 = pack2(-sub, -sub);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x0, x1;
                        unpack2(fma2(pack2(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1])), sc2, sub2), &x0, &x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        sum[i & 1] = add2(sum[i & 1], pack2(p0, p1));
                        o[i] = pack_bf16(p0, p1);
                    }
                    tmem_st32x16(tp + 16 * c, o);
                }
                float l0, l1;
                unpack2(add2(sum[0], sum[1]), &l0, &l1);
                l += l0 + l1;
                tmem_wait_st();
                any = true;
            } else {
                mbar_arrive_warp(&ms->s_free[s]);
                // (this warp's arrival for P must not come a tile early)
                if (any && !warp_all(kv_wait(&ms->pv_done[s], s_count & 1, &ms->abort))) return;
                any = true;
            }
            tc_fence_before();
            if (s == 0 && s_count == 1 && threadIdx.x == 0) CSLA_TL_MARK_ANY(3);
            mbar_arrive_warp(&ms->p_full[s]);
        }
        tiles += it.hi - it.lo;
        if (t0 < t1) {
            if (!warp_all(kv_wait(&ms->pv_done[s], (s_count - 1) & 1, &ms->abort))) return;
            tc_fence_after();
        }
        if (idle) {
            tc_fence_before();
            mbar_arrive_warp(&ms->item_empty[slot]);
            continue;
        }
        const bool none = m == -INFINITY && l == 0.f;   // no token at all (scores that are all NaN leave l NaN)
        if (it.part >= 0) {
            // partial: O and (m, l), of part `part` (+ s for a shared row tile)
            const long long pr = it.base + ((long long)(it.part + (it.paired ? 0 : s)) * a.HK + it.hk) * it.rows_s + r;
            if (mine) a.part_ml[pr] = make_float2(m, l);
            if (t0 < t1) {
                float *po = a.part_o + pr * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tmem_ld32x32(to + 32 * c, v);
                    tmem_wait_ld();
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            store32(po + 32 * c + i, v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]);
                    }
                }
            }
        } else if (t0 < t1) {
            const int t = pos - it.pos0, hq = it.hk * G + y - (t - it.tok0) * G;
            const float sink = a.sink ? a.sink[hq] * kLog2e : -INFINITY;
            const float top = fmaxf(m, sink);
            const float f = none ? 0.f : ex2(m - top);
            const float den = fmaf(l, f, a.sink && !none ? ex2(sink - top) : 0.f);
            const float w = none ? 0.f : f / den;
            const long long at = ((long long)(it.n0 + t) * a.HQ + hq) * D;
            const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // (16 bytes are promised)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_ld32x32(to + 32 * c, v);
                tmem_wait_ld();
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = none ? 0.f : __uint_as_float(v[i]) * w;
                if (mine) {
                    if constexpr (OBF16) {
                        uint16_t *p = reinterpret_cast<uint16_t *>(a.out) + at + 32 * c;
                        uint32_t y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                        if (wide) {
                            store32(p, y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
                            store32(p + 16, y[8], y[9], y[10], y[11], y[12], y[13], y[14], y[15]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                *reinterpret_cast<uint4 *>(p + 8 * i) = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                        }
                    } else {
                        float *p = reinterpret_cast<float *>(a.out) + at + 32 * c;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                }
            }
        }
        tc_fence_before();
        mbar_arrive_warp(&ms->item_empty[slot]);
        if (s == 0 && n == 0 && threadIdx.x == 0) CSLA_TL_MARK_ANY(5);
    }
}

// ---------------------------------------------------------------- kernel
template <int D, bool QBF16, bool OBF16>
__global__ void __launch_bounds__(kThreads, 1) kv_attend_kernel(const __grid_constant__ KvAttendArgs a,
                                                                const __grid_constant__ CUtensorMap km,
                                                                const __grid_constant__ CUtensorMap vm) {
    CSLA_TL_SCOPE(kTlKvAttend);
    using C = Cfg<D>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + C::kOffMisc);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x >= 64 && threadIdx.x < 128) ms->turn[threadIdx.x - 64] = a.freq.turn[threadIdx.x - 64];
    if (warp == 12) {
        tmem_alloc(&ms->tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ms->item_full[i], 1);
            mbar_init(&ms->item_empty[i], 15);   // softmax 8, Q 4, S, PV, TMA
        }
        for (int i = 0; i < 5; ++i) {
            mbar_init(&ms->k_full[i], 1);
            mbar_init(&ms->k_empty[i], 1);
            mbar_init(&ms->v_full[i], 1);
            mbar_init(&ms->v_empty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ms->q_full[s], 4);
            mbar_init(&ms->q_empty[s], 1);
            mbar_init(&ms->s_full[s], 1);
            mbar_init(&ms->p_full[s], 4);
            mbar_init(&ms->s_free[s], 4);
            mbar_init(&ms->pv_done[s], 1);
        }
        mbar_init(&ms->drain[0], 1);
        mbar_init(&ms->drain[1], 1);
        ms->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    CSLA_TL_WAITED();
    // registers: 2 x 128 x 176 + 128 x 96 + 128 x 64 = 65536, the launch's 512 x 128
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        softmax_role<D, QBF16, OBF16>(a, smem, ms, warp >> 2);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        q_role<D, QBF16>(a, smem, ms);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 12)
            s_role<D>(smem, ms);
        else if (warp == 13)
            load_role<D>(a, km, vm, smem, ms);
        else if (warp == 14)
            sched_role(a, ms);
        else
            pv_role<D>(smem, ms);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(ms->tmem, 512);
    }
}

// ---------------------------------------------------------------- join
// Rows whose keys were cut: o = sum_p w_p O_p / (sum_p w_p l_p + w_sink),
// w_p = 2^(m_p - M), parts in a fixed order.  A row of few parts is a warp's;
// one of many is a block's, a range of parts per warp, the warps' sums added
// in order (a long context of one KV head leaves hundreds of parts on a few
// rows: 4 rows x 64 heads x 256 parts took 75 us with a warp per row).
// Bound by the partials' bytes, which the attention has just left in L2: 8
// requests of 16384 tokens and 32 heads, 10.0 us beside 94 us of attention.
constexpr int kJoinWarps = 8, kJoinFew = 32;

// o += sum of w_i O_i over n <= 32 parts `step` rows apart from row pr on, with
// w_i = 2^(m_i - top) in lane i's w.  The parts' loads are issued eight at a
// time, ahead of their weights.
template <int D>
__device__ __forceinline__ void join_parts(const float *part_o, long long pr, long long step, int n, float w, float (&o)[D / 32]) {
    constexpr int kDims = D / 32;
    const int lane = threadIdx.x & 31;
    const float *src = part_o + pr * D + kDims * lane;
    for (int j = 0; j < n; j += 8) {
        float v[8][kDims];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float *p = src + min(j + i, n - 1) * step * D;
            if constexpr (kDims == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(p);
                v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(p);
                v[i][0] = x.x; v[i][1] = x.y;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, (j + i) & 31);
            // (a part of weight zero may never have been written; past n there is none)
#pragma unroll
            for (int d = 0; d < kDims; ++d) o[d] = j + i < n && wi != 0.f ? fmaf(wi, v[i][d], o[d]) : o[d];
        }
    }
}

template <int D, bool OBF16>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const __grid_constant__ KvAttendArgs a) {
    CSLA_TL_SCOPE(kTlKvJoin);
    constexpr int kDims = D / 32;
    __shared__ float sum[kJoinWarps][D];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.HQ / a.HK;
    pdl_wait();
    CSLA_TL_WAITED();
    const KvJoin rq = a.part_req[blockIdx.y];
    if (rq.rows_s == 0) return;
    KvPlan p;
    if (rq.parts == 0) p = kv_plan(rq.T, rq.L, G, a.HK, a.window, D);   // parts by row tile
    const long long step = (long long)a.HK * rq.rows_s;
    const bool block = rq.parts > kJoinFew;
    const int per = block ? 1 : kJoinWarps, units = rq.rows_s * a.HK;
    for (int u0 = blockIdx.x * per; u0 < units; u0 += gridDim.x * per) {
        const int u = block ? u0 : u0 + warp;   // row of the partials, head by head
        if (u >= units) break;
        const int hk = kv_div(u, rq.rows_s), r = u - hk * rq.rows_s, t = kv_div(r, G), hq = hk * G + r - t * G;
        const int parts = rq.parts ? rq.parts : kv_parts(p, kv_range(p, rq.L - rq.T, r / 256, a.window), r / 256);
        if (parts <= 1) continue;
        const long long pr = rq.base + u;
        const float sink = a.sink ? a.sink[hq] * kLog2e : -INFINITY;
        float o[kDims] = {};
        float inv;
        if (parts <= 32 && !block) {
            const float2 ml = lane < parts ? a.part_ml[pr + lane * step] : make_float2(-INFINITY, 0.f);
            const float mx = warp_max(ml.x), top = mx == -INFINITY ? 0.f : fmaxf(mx, sink);
            const float w = ex2(ml.x - top);   // (-inf: 0)
            const float all = warp_sum(w * ml.y);
            inv = mx == -INFINITY && all == 0.f ? 0.f : 1.f / (all + (a.sink ? ex2(sink - top) : 0.f));
            join_parts<D>(a.part_o, pr, step, parts, w, o);
        } else {
            // the largest maximum and the sum over all parts (every warp the
            // same), then O over all parts, or over this warp's share
            float mx = -INFINITY;
            for (int i = lane; i < parts; i += 32) mx = fmaxf(mx, a.part_ml[pr + i * step].x);
            mx = warp_max(mx);
            const float top = mx == -INFINITY ? 0.f : fmaxf(mx, sink);
            float den = 0.f;
            for (int i = lane; i < parts; i += 32) {
                const float2 ml = a.part_ml[pr + i * step];
                den += ex2(ml.x - top) * ml.y;
            }
            den = warp_sum(den);
            inv = mx == -INFINITY && den == 0.f ? 0.f : 1.f / (den + (a.sink ? ex2(sink - top) : 0.f));
            const int share = block ? (parts + kJoinWarps - 1) / kJoinWarps : parts;
            const int i0 = block ? min(parts, warp * share) : 0, i1 = min(parts, i0 + share);
            for (int i = i0; i < i1; i += 32) {
                const float w = i + lane < i1 ? ex2(a.part_ml[pr + (i + lane) * step].x - top) : 0.f;
                join_parts<D>(a.part_o, pr + i * step, step, min(32, i1 - i), w, o);
            }
        }
        if (block) {
#pragma unroll
            for (int d = 0; d < kDims; ++d) sum[warp][kDims * lane + d] = o[d];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                    for (int d = 0; d < kDims; ++d) o[d] += sum[w][kDims * lane + d];
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        const long long at = ((long long)(rq.n0 + t) * a.HQ + hq) * D + kDims * lane;
        if constexpr (OBF16) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(a.out) + at);
#pragma unroll
            for (int d = 0; d < kDims; d += 2) dst[d / 2] = pack_bf16(o[d] * inv, o[d + 1] * inv);
        } else {
            float *dst = reinterpret_cast<float *>(a.out) + at;
#pragma unroll
            for (int d = 0; d < kDims; ++d) dst[d] = o[d] * inv;
        }
    }
}

template <int D, bool QB, bool OB>
cudaError_t launch(const KvAttendArgs &a, const CUtensorMap &km, const CUtensorMap &vm, unsigned grid, cudaStream_t s) {
    auto kern = kv_attend_kernel<D, QB, OB>;
    static KvSmemOnce once;
    const cudaError_t e = once.allow(kern, smem_bytes<D>());
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(kThreads), smem_bytes<D>(), s, a, km, vm);
}
template <int D>
cudaError_t launch_types(const KvAttendArgs &a, bool qb, bool ob, const CUtensorMap &km, const CUtensorMap &vm,
                         unsigned grid, cudaStream_t s) {
    if (qb) return ob ? launch<D, true, true>(a, km, vm, grid, s) : launch<D, true, false>(a, km, vm, grid, s);
    return ob ? launch<D, false, true>(a, km, vm, grid, s) : launch<D, false, false>(a, km, vm, grid, s);
}

}  // namespace

cudaError_t kv_attend_dev_err(unsigned int *bits) {
    *bits = 0;
#ifdef CSLA_UNIT_ALONE
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_dev_err, sizeof(*bits));
    const unsigned int zero = 0;
    if (e == cudaSuccess && *bits) e = cudaMemcpyToSymbol(g_dev_err, &zero, sizeof(zero));
    return e;
#else
    return cudaSuccess;
#endif
}

cudaError_t launch_kv_attend(const KvAttendArgs &a, bool q_bf16, bool out_bf16, const CUtensorMap &km,
                             const CUtensorMap &vm, int num_sms, long long items, cudaStream_t stream) {
    const unsigned grid = (unsigned)(items < num_sms ? items : num_sms);
    return a.D == 64 ? launch_types<64>(a, q_bf16, out_bf16, km, vm, grid, stream)
                     : launch_types<128>(a, q_bf16, out_bf16, km, vm, grid, stream);
}

cudaError_t launch_kv_join(const KvAttendArgs &a, bool out_bf16, int num_sms, cudaStream_t stream) {
    const long long rows = (long long)(a.max_new < a.bt.N ? a.max_new : a.bt.N) * a.HQ;
    const long long most = 8ll * num_sms / a.bt.B + 1;
    const long long x = rows < most ? rows : most;
    const dim3 grid((unsigned)x, (unsigned)a.bt.B), block(32 * kJoinWarps);
    if (a.D == 64)
        return out_bf16 ? launch_pdl(kv_join_kernel<64, true>, grid, block, 0, stream, a)
                        : launch_pdl(kv_join_kernel<64, false>, grid, block, 0, stream, a);
    return out_bf16 ? launch_pdl(kv_join_kernel<128, true>, grid, block, 0, stream, a)
                    : launch_pdl(kv_join_kernel<128, false>, grid, block, 0, stream, a);
}

}  // namespace csla
