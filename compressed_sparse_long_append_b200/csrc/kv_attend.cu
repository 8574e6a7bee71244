// kv_attend.cu -- attention of new tokens over the dense paged cache
// (csla_kv_attend).
//
//   s_j = scale <R(p) norm(q), K_j>,  o = sum_j e^{s_j} V_j / (e^{sink} + sum_j e^{s_j})
//
// One warp per (token, query head): it walks the visible tokens, four at a
// time, with a running maximum and sum in fp32.
#include "kv.cuh"

namespace csla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;

template <int D, bool QBF16, bool OBF16>
__global__ void __launch_bounds__(32 * kWarps) kv_attend_kernel(const __grid_constant__ KvAttendArgs a) {
    CSLA_TL_SCOPE(kTlKvAttend);
    constexpr int kLanes = D / 8, kPer = 32 / kLanes;   // lanes per row, rows per warp step
    pdl_trigger();
    pdl_wait();
    CSLA_TL_WAITED();
    const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
    const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= (long long)a.bt.N * a.HQ) return;
    const int n = (int)(unit / a.HQ), hq = (int)(unit % a.HQ), hk = hq / (a.HQ / a.HK);
    // the request of row n: the last one that starts at or below it
    int b = n / max(a.bt.T, 1);
    if (a.bt.q_start) {
        int cnt = 0;
        for (int j = lane + 1; j <= a.bt.B; j += 32) cnt += a.bt.q_start[j] <= n;
        b = __reduce_add_sync(0xffffffffu, cnt);
    }
    if (b >= a.bt.B) return;
    const KvReq r = kv_request(a.bt, b, a.max_new, a.max_len);
    if (!r.ok || n < r.n0 || n >= r.n0 + r.T) {
        if (r.err) set_dev_err(r.err);
        return;
    }
    const int pos = r.L - r.T + (n - r.n0);
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;

    float q[8], g[8];
    widen8<QBF16>(load8<QBF16>(a.q, (long long)n * a.q_stride + (long long)hq * D + 8 * c), q);
    if (a.gamma_q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = a.gamma_q[8 * c + i];
        row_norm<D>(q, g, a.eps);
    }
    if (a.d_rope) {
        const RopeLane rl = rope_lane<D>(c, a.d_rope, a.pairs);
        float2 cs[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            rope_cos_sin(pos, a.freq.inv[min(rl.first + j, a.d_rope / 2 - 1)], &cs[j].x, &cs[j].y);
        row_rope(q, rl, c, a.d_rope, a.pairs, cs);
    }
    const float sc = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f, o[8] = {};
    bool bad = false;
    for (int j0 = lo; j0 <= pos; j0 += kPer) {
        const int j = j0 + sub;
        float s = -INFINITY, v[8] = {};
        if (j <= pos) {
            const int page = a.bt.block_table[(long long)r.slot * a.bt.bt_stride + j / CSLA_PAGE_TOKENS];
            if (page >= 0 && page < a.bt.n_pages) {
                const long long at = (((long long)page * a.HK + hk) * CSLA_PAGE_TOKENS + j % CSLA_PAGE_TOKENS) * D + 8 * c;
                float k[8];
                widen8<true>(load8<true>(a.k, at), k);
                widen8<true>(load8<true>(a.v, at), v);
                s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
            } else {
                bad = true;
            }
        }
#pragma unroll
        for (int x = kLanes / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= sc;
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - base), p = exp2f(s - base);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = o[i] * f + p * v[i];
        m = mn;
    }
    if (bad) set_dev_err(CSLA_DEVERR_PAGE);
    // join the warp's row groups, in a fixed order, and the sink
    float mt = m;
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
    const float sink = a.sink ? a.sink[hq] * kLog2e : -INFINITY;
    const bool none = mt == -INFINITY;
    const float top = fmaxf(mt, sink), base = top == -INFINITY ? 0.f : top;
    const float f = exp2f(m - base);
    l *= f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= f;
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], x);
    }
    l += a.sink ? exp2f(sink - base) : 0.f;
    const float inv = none ? 0.f : 1.f / l;
    if (sub == 0) {
        const long long at = ((long long)n * a.HQ + hq) * D + 8 * c;
        if constexpr (OBF16) {
            uint4 w;
            w.x = pack_bf16(o[0] * inv, o[1] * inv);
            w.y = pack_bf16(o[2] * inv, o[3] * inv);
            w.z = pack_bf16(o[4] * inv, o[5] * inv);
            w.w = pack_bf16(o[6] * inv, o[7] * inv);
            *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.out) + at) = w;
        } else {
            float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at);
            p[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
            p[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
        }
    }
}

template <int D>
cudaError_t launch(const KvAttendArgs &a, bool qb, bool ob, cudaStream_t s) {
    const dim3 grid((unsigned)(((long long)a.bt.N * a.HQ + kWarps - 1) / kWarps)), block(32 * kWarps);
    if (qb) return ob ? launch_pdl(kv_attend_kernel<D, true, true>, grid, block, 0, s, a)
                      : launch_pdl(kv_attend_kernel<D, true, false>, grid, block, 0, s, a);
    return ob ? launch_pdl(kv_attend_kernel<D, false, true>, grid, block, 0, s, a)
              : launch_pdl(kv_attend_kernel<D, false, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_kv_attend(const KvAttendArgs &a, bool q_bf16, bool out_bf16, cudaStream_t stream) {
    return a.D == 64 ? launch<64>(a, q_bf16, out_bf16, stream) : launch<128>(a, q_bf16, out_bf16, stream);
}

}  // namespace csla
