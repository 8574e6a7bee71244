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

// RMSNorm over the row (all lanes of the row take part; fixed-order sum).
template <int D>
__device__ __forceinline__ void row_norm(float (&x)[8], const float (&g)[8], float eps) {
    float s = (x[0] * x[0] + x[1] * x[1]) + (x[2] * x[2] + x[3] * x[3]);
    s += (x[4] * x[4] + x[5] * x[5]) + (x[6] * x[6] + x[7] * x[7]);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float f = rsqrtf(s * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g[i];
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
