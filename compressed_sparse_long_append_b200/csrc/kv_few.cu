// kv_few.cu -- attention of requests of few rows (up to 16 per KV head:
// decode) over the dense paged cache: a part of csla_kv_attend.
//
//   s_j = scale <R(p) norm(q), K_j>,  o = sum_j e^{s_j} V_j / (e^{sink} + sum_j e^{s_j})
//
// Each K and V byte is used by at most 16 rows, so the kernel is bound by HBM
// and by how much of it is asked for at a time; the products are small.  So
// they stay in registers: mma.sync on 16-row fragments needs no tensor
// memory, no handing over between roles and no padding to 128 rows, and its
// rate is several times what the bytes leave time for.
//
// An item is a chunk of pages of one (request, KV head).  Two persistent CTAs
// per SM; a CTA's producer warp walks the batch and streams K and V stages
// (16 KB each) by TMA into a ring, across items; four consumer warps each
// take a quarter of the stage's tokens with a running maximum m, sum l and O
// of their own:
//   S = Q K^T (Q as two bf16 terms: the rounding of the rotated query is kept),
//   P = 2^(S - m) straight from the accumulators into the A operand of O += P V
//       (rounded to bf16, half a step of each weight).
// At the end of an item the four (m, l, O) are joined through shared memory in
// a fixed order and written out, or left as a partial for kv_join_kernel
// when the request's keys were cut.
//
// Measured (8 KV heads of 128 dims, 4 or 8 query heads each, join included): 8
// requests of 131072 tokens 636 to 656 us for 4.29 GB (boxes differ), 6.75 to
// 6.55 TB/s or 1.03 to 1.00 of a plain copy's rate (which writes half of its
// bytes); 64 ragged requests of 1 to
// 32768 tokens 134 us for 757 MB (5.6 TB/s: the last items' latency and the
// join); a window of 1000 in 32 requests (64 dims, 16 KV heads) 31.6 us for
// 131 MB.  One request of 901 tokens: 11.7 us, 10.6 in a graph, a chain of two
// launches and one item's latency.  The same items in the tensor-memory kernel took 1.17 ms, 156
// us and 47 us; with rows as rows only (no narrow_item) 657 us, 141 us and 36 us.
#include "kv.cuh"

namespace csla {
namespace {

constexpr int kConsumers = 4;   // warps, a quarter of a stage's tokens each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kRows = 16;       // of an item
constexpr int kNarrow = 8;      // rows up to which the products are taken with the rows as columns
constexpr int kItems = 4;
constexpr int kMaxStages = 6;

template <int D>
struct Cfg {
    static constexpr int kTok = D == 128 ? 64 : 128;      // tokens per stage
    static constexpr int kKB = D / 64;                    // 128-byte blocks of a row
    static constexpr int kBlk = kTok * 128;
    static constexpr int kStage = kKB * kBlk;             // 16 KB
    static constexpr int kPer = CSLA_PAGE_TOKENS / kTok;  // stages per page
    static constexpr int kStages = 6;
    static constexpr int kWT = kTok / kConsumers;         // tokens of a stage per warp
    static constexpr int kOut = kRows * D * 2;           // half the dims of one warp's O
    // work area: the Q terms [2][16][D] bf16; at an item's end half of two O, or
    // three whole O of up to 8 rows, and their (m, l)
    static constexpr int kOffWork = kStages * kStage;
    static constexpr int kMl = 32 * 16;                  // (m, l) of both row groups, per lane
    static constexpr int kOffMl = kOffWork + 3 * kOut;
    static constexpr int kOffMisc = kOffMl + 3 * kMl;
};

struct Item {
    int end, n0, T, pos0, slot, hk, rows;
    int lo, hi;          // pages
    int k_lo, k_hi;      // positions that some row sees
    int part;            // partial's index, -1: written out
    long long base;
};

struct Misc {
    Item item[kItems];
    uint64_t item_full[kItems], item_empty[kItems], full[kMaxStages], empty[kMaxStages];
    int bad[kMaxStages];
    unsigned long long turn[64];
    int abort;
};

template <int D>
constexpr int smem_bytes() {
    return Cfg<D>::kOffMisc + (int)sizeof(Misc) + 1024;
}

// The loads and products are plain (not volatile) statements, so that the
// compiler can run loads ahead of products; held() ties them to the waits and
// arrivals around them: an address that passed through it after a wait is not
// loaded from before the wait, a sum that passed through it before an
// arrival has its operands loaded by then.
__device__ __forceinline__ uint32_t held(uint32_t x) {
    asm volatile("" : "+r"(x)::"memory");
    return x;
}
__device__ __forceinline__ void held(float (&c)[4]) {
    asm volatile("" : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])::"memory");
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ void sync_consumers() {
    asm volatile("bar.sync 1, %0;" ::"n"(32 * N) : "memory");
}
// The barrier, and whether `ok` holds in every consumer thread.
template <int N>
__device__ __forceinline__ bool all_consumers(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "n"(32 * N)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- producer
template <int D>
__device__ void producer(const KvAttendArgs &a, const CUtensorMap &km, const CUtensorMap &vm, uint8_t *smem, Misc *ms) {
    using C = Cfg<D>;
    const int lane = threadIdx.x & 31;
    int st = 0, issued = 0, n = 0;
    kv_walk(a, 1u << kKvFew, [&](const KvWalk &w, bool more, int src, int local) {
        Item it;
        it.end = !more;
        if (more && lane == src) {
            const int head = kv_div(local, w.p.nch), j = local - head * w.p.nch;
            const KvRange g = kv_range(w.p, w.r.L - w.r.T, 0, a.window);
            it.n0 = w.r.n0;
            it.T = w.r.T;
            it.pos0 = w.r.L - w.r.T;
            it.slot = w.r.slot;
            it.hk = head;
            it.rows = w.p.rows;
            it.lo = g.lo + j * w.p.c;
            it.hi = min(g.hi, it.lo + w.p.c);   // (with a window the last chunk may be empty)
            it.k_lo = g.k_lo;
            it.k_hi = g.k_hi;
            it.part = kv_parts(w.p, g, 0) > 1 ? j : -1;
            it.base = w.part_before + w.part_excl;
        }
        const int lo = __shfl_sync(0xffffffffu, it.lo, src), hi = __shfl_sync(0xffffffffu, it.hi, src);
        if (more && lo >= hi) return true;
        const int slot = n % kItems;
        if (n >= kItems && !warp_all(kv_wait(&ms->item_empty[slot], (n / kItems - 1) & 1, &ms->abort))) return false;
        if (lane == src) ms->item[slot] = it;
        mbar_arrive_warp(&ms->item_full[slot]);
        ++n;
        if (!more) return true;
        const int req_slot = __shfl_sync(0xffffffffu, it.slot, src), hk = __shfl_sync(0xffffffffu, it.hk, src);
        const int32_t *table = a.bt.block_table + (long long)req_slot * a.bt.bt_stride;
        int pages = -1, ahead = lo + lane < hi ? table[lo + lane] : -1;
        for (int p = lo; p < hi; ++p) {
            if (((p - lo) & 31) == 0) {
                pages = ahead;
                ahead = p + 32 + lane < hi ? table[p + 32 + lane] : -1;
            }
            const int pg = __shfl_sync(0xffffffffu, pages, (p - lo) & 31);
            const bool bad = pg < 0 || pg >= a.bt.n_pages;
            if (bad && lane == 0) set_dev_err(CSLA_DEVERR_PAGE);
            // (an unmapped page's tokens are page 0's, masked)
            const int row = ((bad ? 0 : pg) * a.HK + hk) * CSLA_PAGE_TOKENS;
            for (int h = 0; h < 2 * C::kPer; ++h) {   // K then V of each part of the page
                if (issued >= C::kStages && !warp_all(kv_wait(&ms->empty[st], (issued / C::kStages - 1) & 1, &ms->abort)))
                    return false;
                if (lane == 0) {
                    ms->bad[st] = bad;
                    mbar_arrive_expect_tx(&ms->full[st], C::kStage);
#pragma unroll
                    for (int kb = 0; kb < C::kKB; ++kb)
                        tma_load_2d(smem + st * C::kStage + kb * C::kBlk, (h & 1) ? &vm : &km, 64 * kb,
                                    row + (h >> 1) * C::kTok, &ms->full[st]);
                }
                __syncwarp();
                ++issued;
                st = st + 1 == C::kStages ? 0 : st + 1;
            }
        }
        return true;
    });
    // copies in flight land before the CTA exits (all have, unless a wait gave up)
    for (int i = max(0, issued - C::kStages); i < issued; ++i)
        kv_wait(&ms->full[i % C::kStages], (i / C::kStages) & 1, nullptr);
}

// ---------------------------------------------------------------- consumers
// Q rows of the item as two bf16 terms, rows of 2D bytes, 16-byte chunk ^ (row & 7):
// the terms 16 rows apart, or in rows r and r + 8 of one operand (up to 8 rows).
template <int D, bool QBF16>
__device__ void stage_q(const KvAttendArgs &a, const Item &it, uint8_t *qs, const Misc *ms) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
    const int G = a.HQ / a.HK;
    const RowLane rl = row_lane<D>(c, a.d_rope, a.pairs);
    const int rest = (it.rows <= kNarrow ? kNarrow : kRows) * 2 * D;
#pragma unroll 1
    for (int r0 = warp * kPer; r0 < it.rows; r0 += kConsumers * kPer) {
        const int r = min(r0 + sub, it.rows - 1), t = r * a.inv_g >> 16;
        const Raw8<QBF16> raw = load8<QBF16>(a.q, (long long)(it.n0 + t) * a.q_stride + (it.hk * G + r - t * G) * D, rl);
        float2 cs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) cs[j] = kv_cos_sin(it.pos0 + t, rl.pair >= 0 ? ms->turn[rl.pair + j] : 0);
        float xr[1][8], (&x)[8] = xr[0];
        widen8<QBF16>(raw, x);
        if (a.gamma_q) {
            float g[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = a.gamma_q[i < 4 ? rl.d0 + i : rl.d1 + i - 4];
            rows_norm<D>(xr, g, a.eps);
        }
        if (a.d_rope) row_rope(x, a.pairs, cs);
        if (r0 + sub < it.rows) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int byte = 2 * (h ? rl.d1 : rl.d0);
                uint8_t *p = qs + (r0 + sub) * 2 * D + ((byte & ~15) ^ ((r0 + sub) & 7) << 4) + (byte & 15);
                const uint2 o = make_uint2(pack_bf16(x[4 * h], x[4 * h + 1]), pack_bf16(x[4 * h + 2], x[4 * h + 3]));
                *reinterpret_cast<uint2 *>(p) = o;
                *reinterpret_cast<uint2 *>(p + rest) =
                    make_uint2(pack_bf16(x[4 * h] - __uint_as_float(o.x << 16), x[4 * h + 1] - __uint_as_float(o.x & 0xFFFF0000u)),
                               pack_bf16(x[4 * h + 2] - __uint_as_float(o.y << 16),
                                         x[4 * h + 3] - __uint_as_float(o.y & 0xFFFF0000u)));
            }
        }
    }
}

// An item of up to 8 rows.  The terms of Q are the two halves of one operand
// (rows r and r + 8), kept in registers, so one product gives both terms'
// scores; and P, as it lies in the accumulators of S, is the B operand of
// O^T += V^T P^T: half the products, and half the sums, of 16 rows.
//   S, P: row lane / 4, tokens 2 (lane % 4) + {0, 1} of each 8;
//   o[i]: dims 16 i + lane / 4 (+ 8), rows 2 (lane % 4) + {0, 1}.
// Returns false when a wait gave up; the barriers are passed all the same.
template <int D, bool OBF16>
__device__ __forceinline__ bool narrow_item(const KvAttendArgs &a, const Item &it, uint8_t *smem, Misc *ms, int &taken) {
    using C = Cfg<D>;
    constexpr int kNT = C::kWT / 8;   // 8-token tiles per warp and stage
    constexpr int kDT = D / 16;       // 16-dim tiles of O
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, mi = lane >> 3, mr = lane & 7;
    const int tok0 = warp * C::kWT, G = a.HQ / a.HK;
    const float sc = a.scale * kLog2e;
    const uint32_t ring = smem_u32(smem), work = held(smem_u32(smem + C::kOffWork));
    uint32_t q[D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const int row = 8 * (mi & 1) + mr, ch = 2 * k + (mi >> 1);
        ldsm(q[k], work + row * 2 * D + ((ch ^ (row & 7)) << 4));
    }
    const int row = lane >> 2;
    const int pos = it.pos0 + (min(row, it.rows - 1) * a.inv_g >> 16), low = a.window > 0 ? pos - a.window + 1 : 0;
    float m = -INFINITY, l = 0.f, o[kDT][4];
#pragma unroll
    for (int i = 0; i < kDT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // a row's value for the lanes that hold its column of O
    auto column = [&](float x, int e) { return __shfl_sync(0xffffffffu, x, 8 * (lane & 3) + 4 * e); };
    const int parts = (it.hi - it.lo) * C::kPer;
    bool ok = true;
#pragma unroll 1
    for (int s = 0; s < parts; ++s) {
        // ---- S
        const int ks = taken % C::kStages;
        ok = warp_all(kv_wait(&ms->full[ks], (taken / C::kStages) & 1, &ms->abort));
        if (!ok) break;
        ++taken;
        const bool bad = ms->bad[ks];
        const int t0 = it.lo * CSLA_PAGE_TOKENS + s * C::kTok + tok0;   // position of the warp's first token
        float acc[kNT][2][4];   // (two chains of products)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][0][e] = acc[j][1][e] = 0.f;
        const uint32_t kb = held(ring + ks * C::kStage);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < kNT / 2; ++j) {
                uint32_t b[4];
                const int tok = tok0 + 16 * j + 8 * (mi >> 1) + mr, ch = 2 * k + (mi & 1);
                ldsm(b, kb + (ch >> 3) * C::kBlk + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
                mma16816(acc[2 * j][k & 1], q[k], b[0], b[1]);
                mma16816(acc[2 * j + 1][k & 1], q[k], b[2], b[3]);
            }
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
            held(acc[j][0]);
            held(acc[j][1]);
        }
        mbar_arrive_warp(&ms->empty[ks]);
        // ---- both terms together, mask, maximum, P
        float x[kNT][2];
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                x[j][e] = (acc[j][0][e] + acc[j][1][e]) + (acc[j][0][e + 2] + acc[j][1][e + 2]);
        const int vs = taken % C::kStages;
        const bool edge = bad || t0 + C::kWT > it.pos0 + 1 || t0 < it.k_lo + it.T;   // some row may not see some token
        if (edge) {
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = t0 + 8 * j + 2 * (lane & 3) + e;
                    if (bad || t > pos || t < low) x[j][e] = -INFINITY;
                }
        }
        float mn = fmaxf(x[0][0], x[0][1]);
#pragma unroll
        for (int j = 1; j < kNT; ++j) mn = fmaxf(mn, fmaxf(x[j][0], x[j][1]));
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
        const bool some = !bad && t0 <= pos && t0 + C::kWT > low;   // the row sees a token of the warp's
        mn = fmaxf(some ? fmaxf(m, kLeast) : m, mn * sc);
        const bool grow = mn > m + kGrow;
        if (__any_sync(0xffffffffu, grow)) {
            const float f = !grow ? 1.f : (m == -INFINITY ? 0.f : ex2(m - mn));
            if (grow) m = mn;
            l *= f;
            const float f0 = column(f, 0), f1 = column(f, 1);
#pragma unroll
            for (int i = 0; i < kDT; ++i) {
                o[i][0] *= f0;
                o[i][1] *= f1;
                o[i][2] *= f0;
                o[i][3] *= f1;
            }
        }
        const float sub = m == -INFINITY ? 0.f : m;
        uint32_t p[kNT];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
            const float p0 = ex2(fmaf(x[j][0], sc, -sub)), p1 = ex2(fmaf(x[j][1], sc, -sub));
            sum += p0 + p1;
            p[j] = pack_bf16(p0, p1);
        }
        l += sum;
        // ---- O^T += V^T P^T
        ok = warp_all(kv_wait(&ms->full[vs], (taken / C::kStages) & 1, &ms->abort));
        if (!ok) break;
        ++taken;
        const uint32_t vb = held(ring + vs * C::kStage);
#pragma unroll
        for (int k = 0; k < kNT / 2; ++k) {
            // tokens that no row sees count nothing, whatever they hold (0 * NaN is not 0)
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
            if (edge) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = t0 + 16 * k + 8 * h + 2 * (lane & 3);
                    keep[h] = bad ? 0u
                                  : (t >= it.k_lo && t < it.k_hi ? 0xFFFFu : 0u) |
                                        (t + 1 >= it.k_lo && t + 1 < it.k_hi ? 0xFFFF0000u : 0u);
                }
            }
#pragma unroll
            for (int i = 0; i < kDT; ++i) {
                uint32_t v[4];
                const int tok = tok0 + 16 * k + 8 * (mi >> 1) + mr, ch = 2 * i + (mi & 1);
                ldsm_t(v, vb + (ch >> 3) * C::kBlk + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
                if (edge) {
                    v[0] &= keep[0];
                    v[1] &= keep[0];
                    v[2] &= keep[1];
                    v[3] &= keep[1];
                }
                mma16816(o[i], v, p[2 * k], p[2 * k + 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < kDT; ++i) held(o[i]);
        mbar_arrive_warp(&ms->empty[vs]);
    }

    // ---- join the four token groups, in order, by the first warp
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    sync_consumers<kConsumers>();   // Q is in everyone's registers
    if (warp > 0) {
        float4 *buf = reinterpret_cast<float4 *>(smem + C::kOffWork + (warp - 1) * C::kOut);
#pragma unroll
        for (int i = 0; i < kDT; ++i) buf[i * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        reinterpret_cast<float2 *>(smem + C::kOffMl + (warp - 1) * C::kMl)[lane] = make_float2(m, l);
    }
    sync_consumers<kConsumers>();
    if (warp > 0 || *(volatile int *)&ms->abort) return ok;
    float mo[kConsumers], lo[kConsumers];
    mo[0] = m;
    lo[0] = l;
#pragma unroll
    for (int w = 1; w < kConsumers; ++w) {
        const float2 y = reinterpret_cast<const float2 *>(smem + C::kOffMl + (w - 1) * C::kMl)[lane];
        mo[w] = y.x;
        lo[w] = y.y;
        m = fmaxf(m, y.x);
    }
    const float base = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
        const float f = ex2(mo[w] - base), f0 = column(f, 0), f1 = column(f, 1);
        l += lo[w] * f;
        const float4 *buf = reinterpret_cast<const float4 *>(smem + C::kOffWork + (w - 1) * C::kOut);
#pragma unroll
        for (int i = 0; i < kDT; ++i) {
            if (w == 0) {
                o[i][0] *= f0;
                o[i][1] *= f1;
                o[i][2] *= f0;
                o[i][3] *= f1;
            } else {
                const float4 y = buf[i * 32 + lane];
                o[i][0] = fmaf(y.x, f0, o[i][0]);
                o[i][1] = fmaf(y.y, f1, o[i][1]);
                o[i][2] = fmaf(y.z, f0, o[i][2]);
                o[i][3] = fmaf(y.w, f1, o[i][3]);
            }
        }
    }
    // two neighbouring dims of one row per lane: an even lane / 4 takes its first
    // row's dims d, d + 1, an odd one its second row's d - 1, d
    const bool odd = row & 1;
    const int r = 2 * (lane & 3) + odd, d = row & 6;
    auto pair = [&](float c0, float c1) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 4);
        return odd ? make_float2(got, c1) : make_float2(c0, got);
    };
    if (it.part >= 0) {
        const long long first = it.base + ((long long)it.part * a.HK + it.hk) * it.rows;
        if ((lane & 3) == 0 && row < it.rows) a.part_ml[first + row] = make_float2(m, l);
        float *po = a.part_o + (first + r) * D + d;
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 y = pair(o[i][2 * h], o[i][2 * h + 1]);
                if (r < it.rows) *reinterpret_cast<float2 *>(po + 16 * i + 8 * h) = y;
            }
    } else {
        const int own = min(row, it.rows - 1), hq0 = it.hk * G + own - (own * a.inv_g >> 16) * G;
        const bool no = m == -INFINITY && l == 0.f;   // no token at all (scores that are all NaN leave l NaN)
        const float sink = a.sink ? a.sink[hq0] * kLog2e : -INFINITY;
        const float top = fmaxf(m, sink);
        const float f = no ? 0.f : ex2(m - top);
        const float w = no ? 0.f : f / fmaf(l, f, a.sink ? ex2(sink - top) : 0.f);
        const float mine = __shfl_sync(0xffffffffu, w, 4 * r);
        const bool none = __shfl_sync(0xffffffffu, (int)no, 4 * r);
        const int real = min(r, it.rows - 1), t = real * a.inv_g >> 16, hq = it.hk * G + real - t * G;
        const long long at = ((long long)(it.n0 + t) * a.HQ + hq) * D + d;
#pragma unroll
        for (int i = 0; i < kDT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 y = pair(o[i][2 * h], o[i][2 * h + 1]);
                y = none ? make_float2(0.f, 0.f) : make_float2(y.x * mine, y.y * mine);
                if (r < it.rows) {
                    if constexpr (OBF16)
                        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(a.out) + at + 16 * i + 8 * h) = pack_bf16(y.x, y.y);
                    else
                        *reinterpret_cast<float2 *>(reinterpret_cast<float *>(a.out) + at + 16 * i + 8 * h) = y;
                }
            }
    }
    return ok;
}

template <int D, bool QBF16, bool OBF16>
__device__ void consumer(const KvAttendArgs &a, uint8_t *smem, Misc *ms) {
    using C = Cfg<D>;
    constexpr int kNT = C::kWT / 8;   // 8-token tiles per warp and stage
    constexpr int kDT = D / 8;        // 8-dim tiles of O
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.HQ / a.HK;
    const float sc = a.scale * kLog2e;
    const uint32_t ring = smem_u32(smem), work0 = smem_u32(smem + C::kOffWork);
    // ldmatrix addresses: K (rows = tokens): matrix i = lane / 8 is (tokens 8 (i>>1), dims 8 (i&1));
    // V (transposed): (tokens 8 (i&1), dims 8 (i>>1)); Q: (rows 8 (i&1), dims 8 (i>>1))
    const int mi = lane >> 3, mr = lane & 7;
    const int tok0 = warp * C::kWT;
    int taken = 0;
    bool ok = true;
    for (int n = 0;; ++n) {
        const int islot = n % kItems;
        // the warps go on together or not at all: whatever gave up, every
        // warp passes the same barriers (which also say that the last
        // item's join is done with the work area)
        ok = ok && warp_all(kv_wait(&ms->item_full[islot], (n / kItems) & 1, &ms->abort));
        if (!all_consumers<kConsumers>(ok)) return;
        const Item it = ms->item[islot];
        mbar_arrive_warp(&ms->item_empty[islot]);
        if (it.end) return;
        stage_q<D, QBF16>(a, it, smem + C::kOffWork, ms);
        sync_consumers<kConsumers>();
        if (it.rows <= kNarrow) {
            ok = narrow_item<D, OBF16>(a, it, smem, ms, taken);
            continue;
        }

        float m[2], l[2], o[kDT][4];
        int pos[2], low[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
            pos[h] = it.pos0 + (min(8 * h + (lane >> 2), it.rows - 1) * a.inv_g >> 16);
            low[h] = a.window > 0 ? pos[h] - a.window + 1 : 0;
#pragma unroll
            for (int j = 0; j < kDT; ++j) o[j][2 * h] = o[j][2 * h + 1] = 0.f;
        }
        const int parts = (it.hi - it.lo) * C::kPer;
#pragma unroll 1
        for (int s = 0; s < parts; ++s) {
            // ---- S
            const int ks = taken % C::kStages;
            ok = warp_all(kv_wait(&ms->full[ks], (taken / C::kStages) & 1, &ms->abort));
            if (!ok) break;
            ++taken;
            const bool bad = ms->bad[ks];
            const int t0 = it.lo * CSLA_PAGE_TOKENS + s * C::kTok + tok0;   // position of the warp's first token
            // one sum per term of Q: two chains of products, half as long
            float acc[kNT][4], rest[kNT][4];
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = rest[j][e] = 0.f;
            const uint32_t kb = held(ring + ks * C::kStage), work = held(work0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[kNT / 2][4];
#pragma unroll
                for (int j = 0; j < kNT / 2; ++j) {
                    const int tok = tok0 + 16 * j + 8 * (mi >> 1) + mr, ch = 2 * k + (mi & 1);
                    ldsm(b[j], kb + (ch >> 3) * C::kBlk + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
                }
#pragma unroll
                for (int term = 0; term < 2; ++term) {
                    uint32_t q[4];
                    const int row = 8 * (mi & 1) + mr, ch = 2 * k + (mi >> 1);
                    ldsm(q, work + term * (kRows * 2 * D) + row * 2 * D + ((ch ^ (row & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < kNT / 2; ++j) {
                        mma16816(term ? rest[2 * j] : acc[2 * j], q, b[j][0], b[j][1]);
                        mma16816(term ? rest[2 * j + 1] : acc[2 * j + 1], q, b[j][2], b[j][3]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                held(acc[j]);
                held(rest[j]);
            }
            mbar_arrive_warp(&ms->empty[ks]);
#pragma unroll
            for (int j = 0; j < kNT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] += rest[j][e];
            // ---- mask, maximum, P
            const int vs = taken % C::kStages;
            const bool edge = bad || t0 + C::kWT > it.pos0 + 1 || t0 < it.k_lo + it.T;   // some row may not see some token
            if (edge) {
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = t0 + 8 * j + 2 * (lane & 3) + (e & 1);
                        if (bad || t > pos[e >> 1] || t < low[e >> 1]) acc[j][e] = -INFINITY;
                    }
            }
            float mn[2];
            bool grow = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x = fmaxf(acc[0][2 * h], acc[0][2 * h + 1]);
#pragma unroll
                for (int j = 1; j < kNT; ++j) x = fmaxf(x, fmaxf(acc[j][2 * h], acc[j][2 * h + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                const bool some = !bad && t0 <= pos[h] && t0 + C::kWT > low[h];   // the row sees a token of the warp's
                mn[h] = fmaxf(some ? fmaxf(m[h], kLeast) : m[h], x * sc);
                grow |= mn[h] > m[h] + kGrow;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (mn[h] > m[h] + kGrow) {
                        const float f = m[h] == -INFINITY ? 0.f : ex2(m[h] - mn[h]);
                        m[h] = mn[h];
                        l[h] *= f;
#pragma unroll
                        for (int j = 0; j < kDT; ++j) {
                            o[j][2 * h] *= f;
                            o[j][2 * h + 1] *= f;
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float sub = m[h] == -INFINITY ? 0.f : m[h];
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    acc[j][2 * h] = ex2(fmaf(acc[j][2 * h], sc, -sub));
                    acc[j][2 * h + 1] = ex2(fmaf(acc[j][2 * h + 1], sc, -sub));
                    sum += acc[j][2 * h] + acc[j][2 * h + 1];
                }
                l[h] += sum;
            }
            // ---- O += P V
            ok = warp_all(kv_wait(&ms->full[vs], (taken / C::kStages) & 1, &ms->abort));
            if (!ok) break;
            ++taken;
            const uint32_t vb = held(ring + vs * C::kStage);
#pragma unroll
            for (int k = 0; k < kNT / 2; ++k) {
                const uint32_t p[4] = {pack_bf16(acc[2 * k][0], acc[2 * k][1]), pack_bf16(acc[2 * k][2], acc[2 * k][3]),
                                       pack_bf16(acc[2 * k + 1][0], acc[2 * k + 1][1]),
                                       pack_bf16(acc[2 * k + 1][2], acc[2 * k + 1][3])};
                // tokens that no row sees count nothing, whatever they hold (0 * NaN is not 0)
                uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (edge) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = t0 + 16 * k + 8 * h + 2 * (lane & 3);
                        keep[h] = bad ? 0u
                                      : (t >= it.k_lo && t < it.k_hi ? 0xFFFFu : 0u) |
                                            (t + 1 >= it.k_lo && t + 1 < it.k_hi ? 0xFFFF0000u : 0u);
                    }
                }
#pragma unroll
                for (int j = 0; j < kDT / 2; ++j) {
                    uint32_t b[4];
                    const int tok = tok0 + 16 * k + 8 * (mi & 1) + mr, ch = 2 * j + (mi >> 1);
                    ldsm_t(b, vb + (ch >> 3) * C::kBlk + tok * 128 + (((ch & 7) ^ (tok & 7)) << 4));
                    if (edge) {
                        b[0] &= keep[0];
                        b[1] &= keep[1];
                        b[2] &= keep[0];
                        b[3] &= keep[1];
                    }
                    mma16816(o[2 * j], p, b[0], b[1]);
                    mma16816(o[2 * j + 1], p, b[2], b[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < kDT; ++j) held(o[j]);
            mbar_arrive_warp(&ms->empty[vs]);
        }

        // ---- join the four token groups: 2 into 0 and 3 into 1, then 1 into 0
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        sync_consumers<kConsumers>();   // Q is no longer read
#pragma unroll 1
        for (int step = 2; step >= 1; --step) {
            // (step 2: groups 2, 3 write buffers 0, 1; step 1: group 1 writes buffer 1)
            const bool gives = warp >= step && warp < 2 * step, takes = warp < step;
            const int side = gives || step == 2 ? warp & 1 : 1;
            float4 *buf = reinterpret_cast<float4 *>(smem + C::kOffWork + side * C::kOut);
            float4 *ml = reinterpret_cast<float4 *>(smem + C::kOffMl + side * C::kMl);
            float f[2] = {1.f, 1.f}, g[2] = {0.f, 0.f};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (gives) {
#pragma unroll
                    for (int j = 0; j < kDT / 2; ++j) {
                        const int i = half * (kDT / 2) + j;
                        buf[j * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                    }
                    if (half == 0) ml[lane] = make_float4(m[0], l[0], m[1], l[1]);
                }
                sync_consumers<kConsumers>();
                if (takes) {
                    if (half == 0) {
                        const float4 x = ml[lane];
                        const float mo[2] = {x.x, x.z}, lo[2] = {x.y, x.w};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float top = fmaxf(m[h], mo[h]), base = top == -INFINITY ? 0.f : top;
                            f[h] = ex2(m[h] - base);
                            g[h] = ex2(mo[h] - base);
                            m[h] = top;
                            l[h] = l[h] * f[h] + lo[h] * g[h];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kDT / 2; ++j) {
                        const int i = half * (kDT / 2) + j;
                        const float4 y = buf[j * 32 + lane];
                        o[i][0] = o[i][0] * f[0] + y.x * g[0];
                        o[i][1] = o[i][1] * f[0] + y.y * g[0];
                        o[i][2] = o[i][2] * f[1] + y.z * g[1];
                        o[i][3] = o[i][3] * f[1] + y.w * g[1];
                    }
                }
                sync_consumers<kConsumers>();
            }
        }
        if (warp == 0 && !*(volatile int *)&ms->abort) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 8 * h + (lane >> 2);
                if (r >= it.rows) continue;
                const int d = 2 * (lane & 3);
                if (it.part >= 0) {
                    const long long pr = it.base + ((long long)it.part * a.HK + it.hk) * it.rows + r;
                    if (d == 0) a.part_ml[pr] = make_float2(m[h], l[h]);
#pragma unroll
                    for (int j = 0; j < kDT; ++j)
                        *reinterpret_cast<float2 *>(a.part_o + pr * D + 8 * j + d) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
                } else {
                    const int t = r * a.inv_g >> 16, hq = it.hk * G + r - t * G;
                    const bool none = m[h] == -INFINITY && l[h] == 0.f;   // no token at all (scores that are all NaN leave l NaN)
                    const float sink = a.sink ? a.sink[hq] * kLog2e : -INFINITY;
                    const float top = fmaxf(m[h], sink);
                    const float f = none ? 0.f : ex2(m[h] - top);
                    const float w = none ? 0.f : f / fmaf(l[h], f, a.sink ? ex2(sink - top) : 0.f);
                    const long long at = ((long long)(it.n0 + t) * a.HQ + hq) * D + d;
#pragma unroll
                    for (int j = 0; j < kDT; ++j) {
                        const float x = none ? 0.f : o[j][2 * h] * w, y = none ? 0.f : o[j][2 * h + 1] * w;
                        if constexpr (OBF16)
                            *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(a.out) + at + 8 * j) = pack_bf16(x, y);
                        else
                            *reinterpret_cast<float2 *>(reinterpret_cast<float *>(a.out) + at + 8 * j) = make_float2(x, y);
                    }
                }
            }
        }
    }
}

template <int D, bool QBF16, bool OBF16>
__global__ void __launch_bounds__(kThreads, 2) kv_few_kernel(const __grid_constant__ KvAttendArgs a,
                                                             const __grid_constant__ CUtensorMap km,
                                                             const __grid_constant__ CUtensorMap vm) {
    CSLA_TL_SCOPE(kTlKvFew);
    using C = Cfg<D>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    Misc *ms = reinterpret_cast<Misc *>(smem + C::kOffMisc);
    if (threadIdx.x < 64) ms->turn[threadIdx.x] = a.freq.turn[threadIdx.x];
    if (threadIdx.x == 64) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&ms->item_full[i], 1);
            mbar_init(&ms->item_empty[i], kConsumers);
        }
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&ms->full[i], 1);
            mbar_init(&ms->empty[i], kConsumers);
        }
        ms->abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&km);
        tma_prefetch_desc(&vm);
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();   // (before the wait: one user's 901 tokens 11.0 us instead of 10.7 in a graph)
    CSLA_TL_WAITED();
    if (threadIdx.x >= 32 * kConsumers)
        producer<D>(a, km, vm, smem, ms);
    else
        consumer<D, QBF16, OBF16>(a, smem, ms);
}

template <int D, bool QB, bool OB>
cudaError_t launch(const KvAttendArgs &a, const CUtensorMap &km, const CUtensorMap &vm, unsigned grid, cudaStream_t s) {
    auto kern = kv_few_kernel<D, QB, OB>;
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

cudaError_t launch_kv_few(const KvAttendArgs &a, bool q_bf16, bool out_bf16, const CUtensorMap &km,
                          const CUtensorMap &vm, int num_sms, long long items, cudaStream_t stream) {
    const unsigned grid = (unsigned)(items < 2 * num_sms ? items : 2 * num_sms);
    return a.D == 64 ? launch_types<64>(a, q_bf16, out_bf16, km, vm, grid, stream)
                     : launch_types<128>(a, q_bf16, out_bf16, km, vm, grid, stream);
}

}  // namespace csla
