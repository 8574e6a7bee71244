// kv_append.cu -- keys and values of new tokens into the dense layers' pages
// (csla_kv_append).
//
//   K row = bf16(R(p) (k / sqrt(mean(k^2) + eps) * gamma_k)),  V row = bf16(v)
//
// A block takes a few consecutive tokens of the ragged batch.  It finds their
// requests by counting the request starts at or below each token, resolves
// each token's page once, and evaluates the rotation's cosines and sines once
// per token and pair in shared memory; then D/8 lanes move one (token, head)
// row, 16 or 32 bytes per lane, several rows of a thread in flight together.
// The bytes bound it (each row read once and written once); short calls are
// bound by the chain offsets -> slot -> length -> page, which runs while the
// first rows' loads are in flight.
#include "kv.cuh"

namespace csla {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;   // tokens per block
constexpr int kFly = 4;       // rows of a thread in flight

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendArgs a, int tok) {
    CSLA_TL_SCOPE(kTlKvAppend);
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;   // rows per pass
    __shared__ int s_cnt[kMaxTok];
    __shared__ int s_pos[kMaxTok];
    __shared__ long long s_dst[kMaxTok];   // element of the token's row in head 0, -1: skipped
    __shared__ float2 s_cs[kMaxTok][D / 2];
    __shared__ unsigned long long s_turn[D / 2];
    pdl_trigger();
    const int tid = threadIdx.x, c = tid % kLanes;
    const int n0 = blockIdx.x * tok, nt = min(tok, a.bt.N - n0);
    const int rows = nt * 2 * a.HK;   // (token, K or V, head)
    const int half = a.d_rope / 2;
    const RowLane rl = row_lane<D>(c, a.d_rope, a.pairs);
    if (tid < kMaxTok) s_cnt[tid] = 0;
    if (tid < half) s_turn[tid] = a.freq.turn[tid];
    pdl_wait();
    CSLA_TL_WAITED();

    Raw8<BF16> raw[kFly];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const int r = r0 + j * kRows + tid / kLanes;
            if (r < rows) {
                const int t = r / (2 * a.HK), w = r % (2 * a.HK);
                const long long n = n0 + t;
                raw[j] = w < a.HK ? load8<BF16>(a.k_new, n * a.k_stride + (long long)w * D, rl)
                                  : load8<BF16>(a.v_new, n * a.v_stride + (long long)(w - a.HK) * D, rl);
            }
        }
    };
    fetch(0);

    __syncthreads();
    // the request of token n is the number of starts q_start[1..B] at or below n
    if (a.bt.q_start) {
        for (int j = tid + 1; j <= a.bt.B; j += kThreads) {
            const int s = a.bt.q_start[j];
            if (s < n0 + nt) atomicAdd(&s_cnt[max(s - n0, 0)], 1);
        }
        __syncthreads();
    }
    if (tid < nt) {
        const int n = n0 + tid;
        int b = n / max(a.bt.T, 1);
        if (a.bt.q_start) {
            b = 0;
            for (int j = 0; j <= tid; ++j) b += s_cnt[j];
        }
        long long dst = -1;
        int pos = 0;
        unsigned err = 0;
        if (b < a.bt.B) {
            const KvReq r = kv_request(a.bt, b, 0x7FFFFFFF, 0x7FFFFFFF);
            err = r.err;
            if (r.ok && n >= r.n0 && n < r.n0 + r.T) {   // else: a row of no request
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
    __syncthreads();
    for (int i = tid; i < nt * half; i += kThreads) {
        const int t = i / half, p = i % half;
        s_cs[t][p] = kv_cos_sin(s_pos[t], s_turn[p]);
    }
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = a.gamma_k ? a.gamma_k[i < 4 ? rl.d0 + i : rl.d1 + i - 4] : 1.f;
    __syncthreads();

    for (int r0 = 0; r0 < rows; r0 += kFly * kRows) {
        if (r0) fetch(r0);
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const int r = r0 + j * kRows + tid / kLanes;
            if (r0 + j * kRows >= rows) break;   // uniform in the block
            const int rr = min(r, rows - 1);
            const int t = rr / (2 * a.HK), w = rr % (2 * a.HK);
            float x[8];
            widen8<BF16>(raw[j], x);
            // every lane of a warp takes the shuffles; V rows keep their values
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
            if (a.gamma_k) row_norm<D>(y, g, a.eps);
            if (rl.pair >= 0) {
                float2 cs[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) cs[p] = s_cs[t][rl.pair + p];
                row_rope(y, a.pairs, cs);
            }
            const bool is_k = w < a.HK;
            uint2 o[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                o[i] = is_k ? make_uint2(pack_bf16(y[4 * i], y[4 * i + 1]), pack_bf16(y[4 * i + 2], y[4 * i + 3]))
                            : make_uint2(pack_bf16(x[4 * i], x[4 * i + 1]), pack_bf16(x[4 * i + 2], x[4 * i + 3]));
            const long long dst = s_dst[t];
            if (r < rows && dst >= 0) {
                const int h = is_k ? w : w - a.HK;
                uint16_t *out = (is_k ? a.k : a.v) + dst + (long long)h * CSLA_PAGE_TOKENS * D;
                *reinterpret_cast<uint2 *>(out + rl.d0) = o[0];
                *reinterpret_cast<uint2 *>(out + rl.d1) = o[1];
            }
        }
    }
}

template <int D>
cudaError_t launch(const KvAppendArgs &a, bool bf16, cudaStream_t s) {
    // One pass of a block is 2048 / D rows.  Short calls: one token per block, so
    // that all SMs share the latency.  Long ones: enough tokens for kFly rows
    // per thread.
    int tok = 1;
    if (a.bt.N > 4 * 148) {
        tok = kFly * (kThreads * 8 / D) / (2 * a.HK);
        tok = tok < 1 ? 1 : (tok > kMaxTok ? kMaxTok : tok);
    }
    const dim3 grid((a.bt.N + tok - 1) / tok);
    return bf16 ? launch_pdl(kv_append_kernel<D, true>, grid, dim3(kThreads), 0, s, a, tok)
                : launch_pdl(kv_append_kernel<D, false>, grid, dim3(kThreads), 0, s, a, tok);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, bool bf16, cudaStream_t stream) {
    return a.D == 64 ? launch<64>(a, bf16, stream) : launch<128>(a, bf16, stream);
}

}  // namespace csla
