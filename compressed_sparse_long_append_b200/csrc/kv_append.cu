// kv_append.cu -- keys and values of new tokens into the dense layers' pages
// (csla_kv_append).
//
//   K row = bf16(R(p) (k / sqrt(mean(k^2) + eps) * gamma_k)),  V row = bf16(v)
//
// A block takes a few consecutive tokens of the ragged batch.  It finds their
// requests (a token's ends at the first start above it), resolves each
// token's page once, and evaluates the rotation's cosines and sines once
// per token and pair in shared memory; then D/8 lanes move one (token, head)
// row, 16 or 32 bytes per lane: the K rows of its tokens, then the V rows (a
// copy), two rows of a thread at a time and the next two in flight.
// The bytes bound a long call (each row read once and written once) and leave
// about 170 instructions per warp for two rows, so a thread's (token, head) is
// carried from row to row, not divided out: 8192 tokens of 8 heads x 128 take
// 15.9 us for 67 MB, 4.2 TB/s or 0.64 of a plain copy's rate, with instruction issue
// 62 % busy (norm and rotation) and one round of blocks, whose start and end
// are not overlapped by another.  Short calls are bound by the
// chain offsets -> slot -> length -> page, which runs while the first rows'
// loads are in flight (8 tokens: 2.9 us in a graph), and by the call itself on
// the host (7.5 us).
#include <limits.h>

#include "kv.cuh"

namespace csla {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;   // tokens per block
constexpr int kFly = 2;       // rows of a thread at a time (and as many in flight)
constexpr int kBlocks = 4;    // blocks per SM
constexpr int kPass = 8;      // K rows of a thread in a long call, at most

// Where a thread is among the rows of a block: rows go head by head through
// the tokens, kRows apart for a thread.
struct RowPos {
    int t, h;
};
__device__ __forceinline__ void advance(RowPos &p, int dt, int dh, int HK) {
    p.t += dt;
    p.h += dh;
    if (p.h >= HK) {
        p.h -= HK;
        ++p.t;
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kBlocks) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int tok) {
    CSLA_TL_SCOPE(kTlKvAppend);
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;   // rows per pass
    __shared__ int s_end[kMaxTok];         // first j with q_start[j] just above token i (the last token: any above it)
    __shared__ int s_pos[kMaxTok];
    __shared__ long long s_dst[kMaxTok];   // element of the token's row in head 0, -1: skipped
    __shared__ float2 s_cs[kMaxTok][D / 2];
    __shared__ unsigned long long s_turn[D / 2];
    pdl_trigger();
    const int tid = threadIdx.x, c = tid % kLanes;
    const int n0 = blockIdx.x * tok, nt = min(tok, a.bt.N - n0);
    const int half = a.d_rope / 2;
    const RowLane rl = row_lane<D>(c, a.d_rope, a.pairs);
    if (tid < kMaxTok) s_end[tid] = INT_MAX;
    if (tid < half) s_turn[tid] = a.freq.turn[tid];
    // (row / HK of the at most 32 rows of a pass, HK <= 1024: exact)
    const int dt = kRows * a.inv_hk >> 16, dh = kRows - dt * a.HK, row = tid / kLanes, t0 = row * a.inv_hk >> 16;
    const RowPos start{t0, row - t0 * a.HK};
    pdl_wait();
    CSLA_TL_WAITED();

    Raw8<BF16> raw[kFly], ahead[kFly];
    // the next kFly rows of a thread from p on
    auto fetch = [&](const void *src, long long stride, RowPos &p, Raw8<BF16> (&x)[kFly]) {
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            if (p.t < nt) x[j] = load8<BF16>(src, (long long)(n0 + p.t) * stride + p.h * D, rl);
            advance(p, dt, dh, a.HK);
        }
    };
    RowPos load = start;
    fetch(a.k_new, a.k_stride, load, raw);

    __syncthreads();
    // Token n is of the request that ends at the first start above n, if that one
    // begins at or below n and no earlier request begins above it.
    bool fell = false;   // some start is below the one before, or outside [0, N]
    if (a.bt.q_start) {
        int beyond = INT_MAX;   // this thread's first start above all of the block's tokens
        for (int j = tid; j <= a.bt.B; j += kThreads) {
            const int s = a.bt.q_start[j], last = j > 0 ? a.bt.q_start[j - 1] : 0;
            fell |= s < last || s > a.bt.N;
            if (j == 0 || s <= n0) continue;
            if (s >= n0 + nt)
                beyond = min(beyond, j);
            else
                atomicMin(&s_end[s - n0 - 1], j);
        }
        beyond = __reduce_min_sync(0xffffffffu, beyond);
        if ((tid & 31) == 0 && beyond != INT_MAX) atomicMin(&s_end[nt - 1], beyond);
        fell = __syncthreads_or(fell);
        if (fell && blockIdx.x == 0 && tid == 0) set_dev_err(CSLA_DEVERR_INDEX);
    }
    if (tid < nt) {
        const int n = n0 + tid;
        int b = n / max(a.bt.T, 1);
        if (a.bt.q_start) {
            int end = INT_MAX;
            for (int j = tid; j < nt; ++j) end = min(end, s_end[j]);
            b = end - 1;
        }
        long long dst = -1;
        int pos = 0;
        unsigned err = 0;
        if (b < a.bt.B) {
            const KvReq r = kv_request(a.bt, b, 0x7FFFFFFF, 0x7FFFFFFF);
            err = r.err;
            if (fell)
                for (int j = 0; j < b; ++j)
                    if (a.bt.q_start[j] > r.n0) err = CSLA_DEVERR_INDEX;
            if (!err && r.ok && n >= r.n0 && n < r.n0 + r.T) {   // else: a row of no request
                pos = r.L - r.T + (n - r.n0);
                const int page = a.bt.block_table[(long long)r.slot * a.bt.bt_stride + pos / CSLA_PAGE_TOKENS];
                if (page >= 0 && page < a.bt.n_pages)
                    dst = ((long long)page * a.HK * CSLA_PAGE_TOKENS + pos % CSLA_PAGE_TOKENS) * D;
                else
                    err |= CSLA_DEVERR_PAGE;
            }
        }
        if (err) set_dev_err(err);
        s_dst[tid] = dst;
        s_pos[tid] = pos;
    }
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = a.gamma_k ? a.gamma_k[i < 4 ? rl.d0 + i : rl.d1 + i - 4] : 1.f;
    __syncthreads();
    if (tid % (D / 2) < half)
        for (int t = tid / (D / 2); t < nt; t += kThreads / (D / 2))
            s_cs[t][tid % (D / 2)] = kv_cos_sin(s_pos[t], s_turn[tid % (D / 2)]);
    __syncthreads();

    auto store = [&](uint16_t *pool, const RowPos &p, const float (&y)[8]) {
        const long long dst = p.t < nt ? s_dst[p.t] : -1;
        if (dst < 0) return;
        uint16_t *out = pool + dst + p.h * (CSLA_PAGE_TOKENS * D);
        *reinterpret_cast<uint2 *>(out + rl.d0) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
        *reinterpret_cast<uint2 *>(out + rl.d1) = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    };
    const int rows = nt * a.HK;
    // K rows; every lane of a warp takes the norm's shuffles
    RowPos at = start;
    for (int r0 = 0; r0 < rows; r0 += kFly * kRows) {
        if (r0 + kFly * kRows < rows) {
            fetch(a.k_new, a.k_stride, load, ahead);
        } else {
            load = start;
            fetch(a.v_new, a.v_stride, load, ahead);
        }
        float x[kFly][8];
#pragma unroll
        for (int j = 0; j < kFly; ++j) widen8<BF16>(raw[j], x[j]);
        if (a.gamma_k) rows_norm<D>(x, g, a.eps);
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            if (rl.pair >= 0) {
                float2 cs[4];
                const int t = min(at.t, nt - 1);
#pragma unroll
                for (int p = 0; p < 4; ++p) cs[p] = s_cs[t][rl.pair + p];
                row_rope(x[j], a.pairs, cs);
            }
            store(a.k, at, x[j]);
            advance(at, dt, dh, a.HK);
            raw[j] = ahead[j];
        }
    }
    // V rows
    at = start;
    for (int r0 = 0; r0 < rows; r0 += kFly * kRows) {
        if (r0 + kFly * kRows < rows) fetch(a.v_new, a.v_stride, load, ahead);
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            float x[8];
            widen8<BF16>(raw[j], x);
            store(a.v, at, x);
            advance(at, dt, dh, a.HK);
            raw[j] = ahead[j];
        }
    }
}

template <int D>
cudaError_t launch(const KvAppendArgs &a, bool bf16, cudaStream_t s) {
    // As few tokens per block as one round of blocks over the SMs allows: a
    // block's latencies (requests, pages) are what a short call costs, and what a long
    // one pays per round (8192 tokens of 8 heads x 128: 16.2 us in one round, 21.5 in
    // four); up to kPass K rows per thread.
    const int slots = kBlocks * 148, most = kPass * (kThreads * 8 / D) / a.HK;
    int tok = (a.bt.N + slots - 1) / slots;
    tok = tok > most ? most : tok;
    tok = tok < 1 ? 1 : (tok > kMaxTok ? kMaxTok : tok);
    const dim3 grid((a.bt.N + tok - 1) / tok);
    return bf16 ? launch_pdl(kv_append_kernel<D, true>, grid, dim3(kThreads), 0, s, a, tok)
                : launch_pdl(kv_append_kernel<D, false>, grid, dim3(kThreads), 0, s, a, tok);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, bool bf16, cudaStream_t stream) {
    return a.D == 64 ? launch<64>(a, bf16, stream) : launch<128>(a, bf16, stream);
}

}  // namespace csla
