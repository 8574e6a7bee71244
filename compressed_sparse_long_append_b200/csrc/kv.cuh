// kv.cuh -- what the dense paged layers' kernels share: a request of the
// ragged batch, and the norm and rotation of a row held 8 dims per lane.
#pragma once

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

// ------------------------------------------------------------ rows, 8 dims per lane
// A row of D dims is held by D/8 consecutive lanes of a warp, lane c of the
// row holding dims 8c .. 8c+7 in fp32.

template <bool BF16>
struct Raw8 {   // 8 elements as loaded
    uint4 v[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void *base, long long elem) {
    Raw8<BF16> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) + elem * (BF16 ? 2 : 4));
    r.v[0] = __ldg(p);
    if constexpr (!BF16) r.v[1] = __ldg(p + 1);
    return r;
}
template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &r, float (&x)[8]) {
    if constexpr (BF16) {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        x[0] = __uint_as_float(r.v[0].x); x[1] = __uint_as_float(r.v[0].y);
        x[2] = __uint_as_float(r.v[0].z); x[3] = __uint_as_float(r.v[0].w);
        x[4] = __uint_as_float(r.v[1].x); x[5] = __uint_as_float(r.v[1].y);
        x[6] = __uint_as_float(r.v[1].z); x[7] = __uint_as_float(r.v[1].w);
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// RMSNorm over the row (all lanes of the row take part; fixed-order sum).
template <int D>
__device__ __forceinline__ void row_norm(float (&x)[8], const float (&g)[8], float eps) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float f = 1.0f / sqrtf(s * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g[i];
}

// Which pairs the 8 dims of a lane belong to: pair of dim i = first + i
// (halves) or first + i/2 (adjacent); role 0: not rotated, 1: first half of
// the pairs (or adjacent), 2: second half.
struct RopeLane {
    int first, role;
};
template <int D>
__device__ __forceinline__ RopeLane rope_lane(int c, int d_rope, int pairs) {
    const int d = 8 * c - (D - d_rope);   // 8c within the rotated dims (d_rope is a multiple of 16)
    RopeLane l{0, 0};
    if (d < 0) return l;
    if (pairs == CSLA_ROPE_ADJACENT) {
        l.first = d / 2;
        l.role = 1;
    } else {
        l.role = d < d_rope / 2 ? 1 : 2;
        l.first = l.role == 1 ? d : d - d_rope / 2;
    }
    return l;
}
// Rotate the row: cs[j] = (cos, sin) of the lane's j-th pair (4 adjacent
// pairs, or 8 pairs whose other dims another lane holds).  All 32 lanes call it.
__device__ __forceinline__ void row_rope(float (&x)[8], const RopeLane &l, int c, int d_rope, int pairs,
                                         const float2 *cs) {
    if (pairs == CSLA_ROPE_ADJACENT) {
        if (l.role == 0) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], w = x[2 * j + 1];
            x[2 * j] = u * cs[j].x - w * cs[j].y;
            x[2 * j + 1] = u * cs[j].y + w * cs[j].x;
        }
    } else {
        const int lane = threadIdx.x & 31, hop = d_rope / 16;
        const int src = l.role == 1 ? lane + hop : (l.role == 2 ? lane - hop : lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float o = __shfl_sync(0xffffffffu, x[j], src);
            if (l.role == 1) x[j] = x[j] * cs[j].x - o * cs[j].y;
            if (l.role == 2) x[j] = o * cs[j].y + x[j] * cs[j].x;
        }
    }
}

}  // namespace csla
