// kv.cuh -- what the dense paged layers' kernels share: a request of the
// ragged batch, and the norm and rotation of a row held 8 dims per lane.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace csla {

// Request b of a dense call: rows n0 .. n0+T-1, context L (new tokens
// included), state-cache slot.  ok == false: the request is skipped (`err`
// says why, 0 for one without new tokens).
struct KvReq {
    int n0, T, L, slot;
    unsigned err;
    bool ok;
};
__device__ __forceinline__ KvReq kv_request(const KvBatch &a, int b, int max_new, int max_len) {
    KvReq r{0, 0, 0, 0, 0u, false};
    if (a.q_start) {
        r.n0 = a.q_start[b];
        const int n1 = a.q_start[b + 1];
        if (r.n0 < 0 || n1 < r.n0 || n1 > a.N) {
            r.err = CSLA_DEVERR_INDEX;
            return r;
        }
        r.T = n1 - r.n0;
    } else {
        r.T = a.T;
        r.n0 = b * a.T;
    }
    if (r.T == 0) return r;   // nothing to do, whatever its slot
    r.slot = a.slots[b];
    if (r.slot < 0 || r.slot >= a.n_slots) {
        r.err = CSLA_DEVERR_INDEX;
        return r;
    }
    r.L = a.len[r.slot];
    if (r.T > max_new || r.L < r.T || r.L > max_len || r.L > (long long)a.bt_stride * CSLA_PAGE_TOKENS)
        r.err = CSLA_DEVERR_LEN;
    r.ok = !r.err;
    return r;
}

// ------------------------------------------------------------ items of a persistent CTA
// A warp's walk over the batch: the items of the requests whose kind is in
// `kinds`, numbered through the batch; this CTA takes item c, 2*grid-1-c,
// 2*grid+c, ... (there and back, so that sizes that fall along the
// numbering even out).  32 requests are held at a time, one per lane, those
// of the largest chunks first.
struct KvWalk {
    int first = -32, total = 0, before = 0, round = 0, incl = 0;
    long long part_before = 0, part_total = 0, part_excl = 0;
    KvReq r{};
    KvPlan p{};

    // The next item: true with *src = the lane that holds its request (its r, p
    // and the request's first partial row part_before + part_excl) and *local
    // = its number in the request; false when there is none.  All lanes call it.
    __device__ __forceinline__ bool next(const KvAttendArgs &a, unsigned kinds, int *src, int *local) {
        const int lane = threadIdx.x & 31, grid = gridDim.x;
        const int u = (round & 1) ? (round + 1) * grid - 1 - (int)blockIdx.x : round * grid + (int)blockIdx.x;
        ++round;
        while (u >= before + total) {
            before += total;
            part_before += part_total;
            first += 32;
            if (first >= a.bt.B) return false;
            int b = first + lane;
            int items = 0;
            long long parts = 0;
            if (b < a.bt.B) {
                r = kv_request(a.bt, b, a.max_new, a.max_len);
                if (r.err && blockIdx.x == 0) set_dev_err(r.err);
                if (r.ok) {
                    p = kv_plan(r.T, r.L, a.HQ / a.HK, a.HK, a.window, a.D);
                    items = (kinds >> p.kind) & 1 ? kv_items(p, a.HK) : 0;
                    parts = kv_part_rows(p, a.HK);
                }
            }
            // largest chunks first: the CTAs' loads even out on the small ones
            if (a.bt.B > 1) {
                unsigned key = (unsigned)(r.ok && b < a.bt.B ? p.c : 0) << 5 | (31 - lane);
#pragma unroll 1
                for (int k = 2; k <= 32; k <<= 1)
#pragma unroll 1
                    for (int j = k >> 1; j > 0; j >>= 1) {
                        const unsigned o = __shfl_xor_sync(0xffffffffu, key, j);
                        const bool larger = ((lane & k) == 0) == ((lane & j) == 0);
                        key = larger ? max(key, o) : min(key, o);
                    }
                const int from = 31 - (int)(key & 31);
                auto take = [&](int &x) { x = __shfl_sync(0xffffffffu, x, from); };
                take(b); take(items);
                parts = __shfl_sync(0xffffffffu, parts, from);
                take(r.n0); take(r.T); take(r.L); take(r.slot);
                take(p.rows); take(p.R); take(p.Rs); take(p.rows_s); take(p.kind); take(p.c); take(p.nch);
                take(p.T); take(p.G); take(p.heads_inside);
            }
            incl = items;
            long long pincl = parts;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                const long long w = __shfl_up_sync(0xffffffffu, pincl, o);
                if (lane >= o) {
                    incl += v;
                    pincl += w;
                }
            }
            part_excl = pincl - parts;
            total = __shfl_sync(0xffffffffu, incl, 31);
            part_total = __shfl_sync(0xffffffffu, pincl, 31);
            // (every attention kernel of the call writes the same)
            if (a.part_req && blockIdx.x == 0 && b < a.bt.B) {
                const int same = p.kind != kKvPaired && parts ? kv_parts(p, kv_range(p, r.L - r.T, 0, a.window), 0) : 0;
                a.part_req[b] = KvJoin{r.n0, parts && same != 1 ? p.rows_s : 0, same, r.T, r.L, 0, part_before + part_excl};
            }
        }
        *src = __ffs(__ballot_sync(0xffffffffu, incl > u - before)) - 1;
        const int prev = __shfl_sync(0xffffffffu, incl, max(*src - 1, 0));
        *local = u - before - (*src ? prev : 0);
        return true;
    }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;   // log2 growth of a row's maximum that its sums tolerate before they are rescaled
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Bounded wait of the attention kernels' roles: they hand tiles over every few
// hundred nanoseconds, so they poll (each poll parks the warp for the
// hardware's own short time) instead of asking to be put to sleep.
__device__ __forceinline__ bool kv_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (int i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            if (abort && *abort) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                set_dev_err(CSLA_DEVERR_TIMEOUT);
                if (abort) *abort = 1;
                return false;
            }
        }
    }
}

// ------------------------------------------------------------ rows, 8 dims per lane
// A row of D dims is held by D/8 consecutive lanes of a warp, 8 dims per lane
// in two runs of four, d0.. and d1..: lanes of unrotated dims hold eight
// neighbours, and so do lanes of adjacent pairs (0,1) (2,3) (4,5) (6,7);
// with pairs of halves a lane holds four dims of the first half and their
// partners, pairs (0,4) (1,5) (2,6) (3,7).  So every rotation stays in its lane.
struct RowLane {
    int d0, d1;   // first dims of the two runs
    int pair;     // first of the lane's four pairs, -1: not rotated
};
template <int D>
__device__ __forceinline__ RowLane row_lane(int c, int d_rope, int pairs) {
    RowLane l;
    const int d = 8 * c - (D - d_rope);   // within the rotated dims (d_rope is a multiple of 16)
    l.d0 = 8 * c;
    l.d1 = 8 * c + 4;
    l.pair = d < 0 ? -1 : d / 2;
    if (d >= 0 && pairs == CSLA_ROPE_HALVES) {
        l.d0 = D - d_rope + d / 2;
        l.d1 = l.d0 + d_rope / 2;
    }
    return l;
}

template <bool BF16>
struct Raw8 {   // 8 elements as loaded
    typename std::conditional<BF16, uint2, uint4>::type v[2];
};
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void *base, long long elem, const RowLane &l) {
    Raw8<BF16> r;
    const char *p = reinterpret_cast<const char *>(base) + elem * (BF16 ? 2 : 4);
    constexpr int kB = BF16 ? 2 : 4;
    using V = typename std::conditional<BF16, uint2, uint4>::type;
    r.v[0] = __ldg(reinterpret_cast<const V *>(p + l.d0 * kB));
    r.v[1] = __ldg(reinterpret_cast<const V *>(p + l.d1 * kB));
    return r;
}
template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &r, float (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (BF16) {
            x[4 * h] = __uint_as_float(r.v[h].x << 16);
            x[4 * h + 1] = __uint_as_float(r.v[h].x & 0xFFFF0000u);
            x[4 * h + 2] = __uint_as_float(r.v[h].y << 16);
            x[4 * h + 3] = __uint_as_float(r.v[h].y & 0xFFFF0000u);
        } else {
            x[4 * h] = __uint_as_float(r.v[h].x);
            x[4 * h + 1] = __uint_as_float(r.v[h].y);
            x[4 * h + 2] = __uint_as_float(r.v[h].z);
            x[4 * h + 3] = __uint_as_float(r.v[h].w);
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// RMSNorm over each of N rows (all lanes of a row take part; fixed-order sum).
// The rows' chains of shuffles run beside one another, so callers take several
// rows through a step, not one row through all steps.
template <int D, int N>
__device__ __forceinline__ void rows_norm(float (&x)[N][8], const float (&g)[8], float eps) {
    float s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = (x[k][0] * x[k][0] + x[k][1] * x[k][1]) + (x[k][2] * x[k][2] + x[k][3] * x[k][3]);
        s[k] += (x[k][4] * x[k][4] + x[k][5] * x[k][5]) + (x[k][6] * x[k][6] + x[k][7] * x[k][7]);
    }
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const float f = rsqrtf(s[k] * (1.0f / D) + eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = x[k][i] * f * g[i];
    }
}

// cos and sin of position times frequency (turns, see KvFreq): the integer
// product wraps at whole turns, its upper half is the angle to 2^-32 turn.
// The angle is then within [-pi, pi], where the fast sine and cosine are good
// to 2^-20, far below the bf16 step (2^-8) that the rotated row is rounded to.
__device__ __forceinline__ float2 kv_cos_sin(int pos, unsigned long long turn) {
    const int t = (int)((unsigned long long)(unsigned)pos * turn >> 32);
    const float x = (float)t * (6.283185307179586f * 0x1p-32f);
    return make_float2(__cosf(x), __sinf(x));
}

// Rotate the lane's four pairs by cs[j] = (cos, sin).
__device__ __forceinline__ void row_rope(float (&x)[8], int pairs, const float2 (&cs)[4]) {
    if (pairs == CSLA_ROPE_ADJACENT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], w = x[2 * j + 1];
            x[2 * j] = u * cs[j].x - w * cs[j].y;
            x[2 * j + 1] = u * cs[j].y + w * cs[j].x;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[j], w = x[4 + j];
            x[j] = u * cs[j].x - w * cs[j].y;
            x[4 + j] = u * cs[j].y + w * cs[j].x;
        }
    }
}

}  // namespace csla
