// kv_walk.cuh -- a request of a dense layer's ragged batch, the walk that finds
// a persistent CTA's items in it, and the bounded wait of the CTA's roles.
// Written against the warp intrinsics and mbar_try_wait, globaltimer_ns,
// kWaitLimitNs and set_dev_err (common.cuh) alone, so that it also runs as
// host code, one fiber per lane.
#pragma once

#include <limits.h>

#include "kernels.h"

namespace csla {

// Request b of a dense call: rows n0 .. n0+T-1, context L (new tokens
// included), state-cache slot.  ok == false: the request is skipped (`err`
// says why, 0 for one without new tokens).  Its two offsets are checked
// against each other and N here, against the requests before it by the caller.
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
    int top = 0;         // largest start so far, once one has fallen below another
    bool fell = false;
    long long part_before = 0, part_total = 0, part_excl = 0;
    KvReq r{};
    KvPlan p{};

    // The next item: true with *src = the lane that holds its request (its r, p
    // and the request's first partial row part_before + part_excl) and *local
    // = its number in the request; false when there is none, or when the caller
    // wants no more (`rest`: the batch is walked to its end).  All lanes call it.
    __device__ __forceinline__ bool next(const KvAttendArgs &a, unsigned kinds, bool rest, int *src, int *local) {
        const int lane = threadIdx.x & 31, grid = gridDim.x;
        const int u = rest ? INT_MAX
                           : ((round & 1) ? (round + 1) * grid - 1 - (int)blockIdx.x : round * grid + (int)blockIdx.x);
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
            }
            // Requests whose offsets are in order on their own may still overlap
            // where a start falls below an earlier one, and the workspace is
            // sized for N rows in all: those are refused.  (Nothing has fallen as
            // long as no request's end lies below its start.)
            if (a.bt.q_start && (fell || __any_sync(0xffffffffu, b < a.bt.B && r.err))) {
                const int start0 = __shfl_sync(0xffffffffu, r.n0, 0);   // (of the group's first: none before is larger yet)
                if (!fell) top = start0;
                fell = true;
                int hi = b < a.bt.B ? r.n0 : top;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, hi, o);
                    if (lane >= o) hi = max(hi, v);
                }
                hi = max(hi, top);
                if (b < a.bt.B && r.n0 < hi) {
                    r.err = CSLA_DEVERR_INDEX;
                    r.ok = false;
                }
                top = __shfl_sync(0xffffffffu, hi, 31);
            }
            if (b < a.bt.B) {
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
            // the join's entries, whatever the requests' kinds
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
// The items of a CTA: take(w, true, src, local) for each, then take(w, false, 0,
// 0).  When take gives up (returns false) it is not called again, but the walk
// goes on to the end of the batch all the same: the join reads an entry of every
// request, and CTA 0's walk writes them.
template <typename Take>
__device__ __forceinline__ void kv_walk(const KvAttendArgs &a, unsigned kinds, Take take) {
    KvWalk w;
    for (bool rest = false, more = true; more;) {
        int src = 0, local = 0;
        more = w.next(a, kinds, rest, &src, &local);
        rest = rest || !take(w, more, src, local);
    }
}

// Bounded wait of the attention kernels' roles: they hand tiles over every few
// hundred nanoseconds, so they poll (each poll parks the warp for the
// hardware's own short time) instead of asking to be put to sleep.  A wait for
// a tile gives up after kWaitLimitNs, one for the end of an item after
// kItemLimitNs: an item is 2^20 key tiles at most, of 2.2 us each where every SM
// is busy.  (A CTA that stands still ends by its waits for tiles all the same,
// whose *abort the longer waits look at.)
constexpr uint64_t kItemLimitNs = 8 * kWaitLimitNs;
__device__ __forceinline__ bool kv_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                        uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (int i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15) == 0) {
            if (abort && *abort) return false;
            if (globaltimer_ns() - t0 > limit_ns) {
                set_dev_err(CSLA_DEVERR_TIMEOUT);
                if (abort) *abort = 1;
                return false;
            }
        }
    }
}

}  // namespace csla
