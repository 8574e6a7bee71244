// kv.cuh -- what the dense paged layers' kernels share: the norm and rotation
// of a row held 8 dims per lane (requests and items: kv_walk.cuh).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kv_walk.cuh"

namespace csla {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.0f;   // log2 growth of a row's maximum that its sums tolerate before they are rescaled
// A row's running maximum from its first visible token on, at least: with -inf
// left to rows that have seen no token, one whose visible scores are all -inf
// ends as 0 / (0 + the sink), not as a row of no tokens.
constexpr float kLeast = -3.0e38f;
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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
