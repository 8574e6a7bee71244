// kernels.h -- launch interfaces between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

namespace csla {

// RoPE inverse frequencies theta^(-2i/d_rope), i < d_rope/2, computed on the
// host in double and passed to the kernels.
struct RopeFreq {
    double inv[32];
};

inline RopeFreq rope_freq(float theta, int d_rope) {
    RopeFreq f{};
    for (int i = 0; i < d_rope / 2 && i < 32; ++i) f.inv[i] = pow((double)theta, -(2.0 * i) / (double)d_rope);
    return f;
}

// Launch with programmatic stream serialization (see pdl_wait in common.cuh).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              Args &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

struct CompressArgs {
    int m, D, d_rope, dI, n_win;
    float theta, eps;
    RopeFreq freq;
    const int32_t *slots;
    int B, T;
    const void *kv_new, *kidx_new;
    const float *gamma_kv, *wg, *gb, *wgi, *gbi;
    uint8_t *win_rows;
    float *win_scales, *tail_kv, *tail_idx;
    int32_t *len;
    uint8_t *rows;
    float *scales;
    void *kidx;           // bf16 keys, or E4M3 codes (key_fmt)
    float *kscale;        // E4M3 keys: per-entry power-of-two scale
    int key_fmt;
    int gate;             // CSLA_GATE_TOKEN or CSLA_GATE_CHANNEL (gb, gbi [m][width])
    const int32_t *block_table;
    int bt_stride, n_pages, n_slots;
    uint8_t *tok_rows;    // optional: window-format row of every new token
    float *tok_scales;    //   token i of request b -> row b * tok_stride + tok_offset + i
    int tok_stride, tok_offset;
};
cudaError_t launch_compress_append(const CompressArgs &a, bool bf16, cudaStream_t stream);

// Ring rows of the last n positions of each request, in position order.
struct WindowRowsArgs {
    const int32_t *slots;
    const int32_t *len;
    int B, n, n_win, n_slots, row_bytes;
    const uint8_t *win_rows;
    const float *win_scales;
    uint8_t *out_rows;
    float *out_scales;
    int stride;
};
cudaError_t launch_window_rows(const WindowRowsArgs &a, cudaStream_t stream);

// Context-parallel entry records (csla_cp_select / csla_cp_place).
struct CpArgs {
    int place;                   // 0: cache -> records (select), 1: records -> cache (place)
    int slot, epp, bt_stride, n_pages;
    const int32_t *block_table;
    uint8_t *rows;
    float *scales;
    uint8_t *kidx;               // CSA keys (bf16 or E4M3 bytes), else null
    float *kscale;               // E4M3 key scales, else null
    int row_bytes, key_bytes, rec_bytes;
    uint8_t *recs;               // [R][E_max][rec_bytes]
    int R, E_max;
    int b_lo[CSLA_CP_MAX_RANKS];  // first block of rank r's run
    int n[CSLA_CP_MAX_RANKS];     // valid records of rank r
};
cudaError_t launch_cp_move(const CpArgs &a, cudaStream_t stream);

// Lightning indexer.  NQ = rows of the bf16 query operand (hi, mid and lo
// terms of every head, zero padding to a multiple of 16).
struct IndexerArgs {
    int m, HI, dI, dc, NQ;
    const int32_t *slots;
    const int32_t *len;
    const int32_t *block_table;
    int bt_stride, n_pages, n_slots;
    int B, tiles_per_req, max_len;
    const void *cq, *W;
    const float *head_w;
    float *scores;
    int scores_stride;
    uint16_t *q_ws;     // [B][NQ][dI] bf16
    int key_fmt;                // CSLA_KEY_BF16 (keys by TMA tensor map) or CSLA_KEY_E4M3:
    const uint8_t *kidx8;       //   E4M3 key codes [n_pages * 32][dI]
    const float *kscale;        //   and per-entry scales [n_pages * 32]
    const int32_t *q_len;   // optional per-row visible length (else len[slot])
    int rows_per_cta;       // 1, or indexer_rows_per_cta(NQ) when all rows share slots[0]
    int range;              // 0: all visible entries; 1: those below len0[b]/m; 2: those from len0[b]/m on
    const int32_t *len0;    // [B] length of row b's request before the step's append (range 1, 2)
    // Streaming selection (csla_indexer_topk); all zero/null for a plain call.
    int page_step;          // > 1 (range 0, sample): the CTA's pages are the request's pages
                            //   (32x + j)*page_step, j < 32, in 8 tiles of 4; entry i of its j-th
                            //   page goes to score column 32*(32x + j) + i
    int persist;            // > 0 (range 0): `persist` CTAs per row group (grid.x) each walk a
                            //   contiguous run of tiles, page ids read per tile; a CTA whose rows
                            //   are all unflagged (row_flag) exits before it sets anything up
    const uint32_t *cand_t0;   // candidate output: entries whose score_key >= cand_t0[b] are appended,
    uint2 *cand;               //   as (key, entry), to sub-list j = (entry/32) % 4 of row b:
    int32_t *cand_cnt;         //   cand[(4b + j) * cand_cap + ..] (any order), cand_cnt[4b + j] counting
    int cand_cap;              //   them all, also past cand_cap (per sub-list); nothing goes to `scores`
    const int32_t *row_flag;   // rows with row_flag[b] == 0 are not scored
};
// len0[b] = len[slots[b]] (0 for a slot outside the pool).
cudaError_t launch_len_snapshot(const int32_t *slots, const int32_t *len, int B, int n_slots, int32_t *len0,
                                cudaStream_t stream);

// Query rows sharing one key tile per MMA when the rows of a call all belong
// to one request: as many as fit the UMMA N limit of 256 columns.
__host__ __device__ constexpr int indexer_rows_per_cta(int NQ) { return 256 / NQ; }
// Tensor maps of the index-query projection on the tensor cores (bf16 cq
// and W_iq): cq [B][dc] in 128-row boxes, W_iq [HI*dI][dc] in boxes of
// iq_gemm_bn(B) rows, 64 columns (128 bytes) per box, 128-byte swizzle.
struct ProjMaps {
    CUtensorMap cq, w;
};
// Output features per CTA of that projection (the W_iq box height).
// (16 for small batches measured slower at decode: 24.5 against 17.6 us per
// indexer call, the extra CTAs each filling a whole 128-row cq tile.)
inline int iq_gemm_bn(int B) {
    (void)B;
    return 64;
}
cudaError_t launch_indexer(const IndexerArgs &a, bool cq_bf16, bool w_bf16, const CUtensorMap &kmap,
                           const CUtensorMap &qmap, int num_sms, cudaStream_t stream, bool project = true,
                           const ProjMaps *pm = nullptr);

struct TopkArgs {
    const float *scores;
    int stride;
    const int32_t *slots;
    const int32_t *len;
    int m, k, B, max_n, n_slots;
    int32_t *idx;
    const int32_t *q_len;   // optional per-row visible length (else len[slot])
    const int32_t *row_flag;   // rows with row_flag[b] == 0 are left alone (their idx untouched)
};
cudaError_t launch_topk(const TopkArgs &a, cudaStream_t stream);

// Streaming selection (csla_indexer_topk), around the indexer's sample and
// candidate passes.  Per row b of a TopkArgs `t`:
//  threshold: cand_t0[b] from the sample scores (32 pages of 32 entries,
//    page_step apart: 1024 columns per row), cand_cnt[b] = 0;
//  select: the top-k from the cand_cnt[b] candidates when k <= cand_cnt[b]
//    <= cand_cap (row_flag[b] = 0), else row_flag[b] = 1 and idx untouched.
constexpr int kCandCap = 8192;        // candidates kept per row (4 sub-lists of 2048)
constexpr int kCandSub = 4;
constexpr int kSampleCols = 1024;     // sample scores per row (32 pages)
constexpr int kPersistSlices = 2;     // CTAs per row group in the stored-score fallback (few: most
                                      // groups have no flagged row and exit at once)
struct CandArgs {
    const float *sample;
    int page_step;
    uint32_t *cand_t0;
    const uint2 *cand;
    int32_t *cand_cnt;
    int32_t *row_flag;
};
cudaError_t launch_cand_threshold(const TopkArgs &t, const CandArgs &c, cudaStream_t stream);
cudaError_t launch_cand_select(const TopkArgs &t, const CandArgs &c, cudaStream_t stream);

// Attention over the canonical row set of each request: compressed entries
// (top-k list or all visible) then the window, reduced in fixed chunks.
struct AttendArgs {
    int m, D, d_rope, H, n_win;
    float theta, eps;
    RopeFreq freq;
    const int32_t *slots;
    const int32_t *len;
    int B;
    const void *q;
    const int32_t *idx;   // CSA top-k list or null (HCA)
    int k;                // CSA list length
    const float *sink, *gamma_q;
    const uint8_t *rows;
    const float *scales;
    const int32_t *block_table;
    int bt_stride, n_pages, n_slots;
    const uint8_t *win_rows;
    const float *win_scales;
    void *out;
    float *part;          // workspace: chunk partials
    int max_chunks;
    int max_len;
    const int32_t *q_len;         // optional per-row visible length (else len[slot])
    const uint8_t *src_rows;      // optional window rows by position:
    const float *src_scales;      //   position p of row b is src row win_base[b] + p
    const int32_t *win_base;
    int n_src;
};

// Visible length of query row b: q_len[b] when given (1 <= q_len[b] <=
// len[slot]), else len[slot].  Returns -1 for a q_len outside that range.
__device__ __forceinline__ int row_visible_len(const int32_t *len, const int32_t *q_len, int slot, int b) {
    const int L = len[slot];
    if (!q_len) return L;
    const int lq = q_len[b];
    return (lq >= 1 && lq <= L) ? lq : -1;
}
cudaError_t launch_attend(const AttendArgs &a, bool q_bf16, bool out_bf16, int variant, int num_sms,
                          cudaStream_t stream);

// Canonical chunk length for a set of n rows (a function of n only):
//   n <= 1024:         64 rows (decode at top-k 512: 10 chunks spread a few
//                      requests over the SMs);
//   1024 < n <= 4096:  320 rows (top-k 1024 + window: 4 chunks, not 18 --
//                      every chunk costs an H*D fp32 partial written and
//                      read back, most of a query row's time when thousands
//                      of rows fill the GPU);
//   n > 4096:          32 * ceil(n / 1024) rows, whole tiles, so that a long
//                      HCA set has close to 32 chunks (8320 rows: 29 chunks
//                      of 288, against 26 of 320 at 64-row granularity).
// A request never has more than 32 chunks.
__host__ __device__ inline int attend_chunk_rows(long long n) {
    if (n <= 1024) return 64;
    if (n <= 4096) return 320;
    return (int)(32 * ((n + 1023) / 1024));
}
__host__ __device__ inline int attend_num_chunks(long long n) {
    const int c = attend_chunk_rows(n);
    return (int)((n + c - 1) / c);
}
// Largest chunk count over all set sizes <= n (never above 32).
__host__ __device__ inline int attend_max_chunks(long long n) {
    const long long c = (n + 63) / 64;
    return (int)(c < 1 ? 1 : (c > 32 ? 32 : c));
}

// ---------------------------------------------------------------- dense paged layers
// Integer division out of line on the device: a divisor that the compiler does
// not know costs some 30 instructions each time it is written, and code that
// runs once per item or launch is paid for by the instruction (it comes from L2).
#ifdef __CUDA_ARCH__
static __device__ __noinline__ int kv_div(int a, int b) { return a / b; }
#else
inline int kv_div(int a, int b) { return a / b; }
#endif

// A kernel's dynamic shared memory beyond the default, allowed once per device.
struct KvSmemOnce {
    std::atomic<unsigned long long> done{0};   // by device
    template <typename... KArgs>
    cudaError_t allow(void (*kernel)(KArgs...), int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

// RoPE frequencies theta^(-2i/d_rope) of a dense layer (d_rope up to 128) as
// turns per position, in units of 2^-64 turn: position times frequency
// modulo one turn is then one 64-bit integer product, exact in the product and
// off by less than pos * 2^-57 turns from the frequency's (64 products of
// extended precision, then cut to a whole number of units).
struct KvFreq {
    unsigned long long turn[64];
};
inline KvFreq kv_freq(float theta, int d_rope) {
    // powers of one ratio in extended precision (64 products: below 2^-57
    // relative), a fraction of what 64 calls of pow cost the host
    KvFreq f{};
    if (d_rope <= 0) return f;
    const long double ratio = expl(-2.0L / d_rope * logl((long double)theta));
    const long double whole = 18446744073709551616.0L;   // 2^64: one turn
    long double x = whole / 6.283185307179586476925286766559L;
    for (int i = 0; i < d_rope / 2 && i < 64; ++i, x *= ratio)
        f.turn[i] = (unsigned long long)(x < whole ? x : fmodl(x, whole));   // (theta below 1: turns of more than one)
    return f;
}

// The ragged batch of a dense layer's call and its paged cache.
struct KvBatch {
    const int32_t *slots;
    const int32_t *q_start;   // [B+1] or null: T new tokens each
    const int32_t *len;
    const int32_t *block_table;
    int B, N, T;
    int bt_stride, n_pages, n_slots;
};

struct KvAppendArgs {
    KvBatch bt;
    int D, HK, d_rope, pairs;
    int inv_hk;                     // 2^16 / HK, rounded up
    float eps;
    KvFreq freq;
    const void *k_new, *v_new;
    long long k_stride, v_stride;   // elements between tokens
    const float *gamma_k;           // null: no norm
    uint16_t *k, *v;                // bf16 pages
};
cudaError_t launch_kv_append(const KvAppendArgs &a, bool bf16, cudaStream_t stream);

struct KvJoin {
    int n0, rows_s;      // the request's first row of out; rows to join per KV head (0: none)
    int parts;           // of each row; 0: by row tile, see T and L
    int T, L, pad;
    long long base;      // first partial row
};
struct KvAttendArgs {
    KvBatch bt;
    int D, HQ, HK, d_rope, pairs, window;
    int inv_g;   // 2^16 / G, rounded up, G = HQ / HK: x * inv_g >> 16 is x / G for x up to 512
    int max_new, max_len;
    float eps, scale;
    KvFreq freq;
    const void *q;
    long long q_stride;
    const float *sink, *gamma_q;    // null: none
    void *out;
    // workspace: what the join needs of each request [B] (null: another kernel of
    // the call writes it), (m, l) and O of the partial rows
    KvJoin *part_req;
    float2 *part_ml;
    float *part_o;
};

// How the attention cuts a request of T new tokens (context L): a function of
// T, L and the layer alone.  rows = T*G rows per KV head.
//   few     up to 16 rows: kv_few_kernel, R = 1;
//   single  up to 128 rows: kv_attend_kernel, R = 1, its two streams take key tiles in turn;
//   paired  more: kv_attend_kernel, R row tiles of 256.
// The keys of row tiles i < Rs are cut into chunks of c tiles, nch at most per
// row tile: all of them when the request has few row tiles for the SMs, else those
// left over from full rounds over the SMs (512 row tiles of all heads on 148
// SMs are 3 rounds and 68 left: cut in two they take half a round, not a whole one).
enum { kKvFew = 0, kKvSingle = 1, kKvPaired = 2 };
struct KvPlan {
    int rows, R, Rs, rows_s, kind, c, nch, T, G, heads_inside;   // rows_s: rows of the cut row tiles
};
constexpr int kKvFewRows = 16;
// items that a long request is cut into (all heads), and the least tiles of a
// chunk, by kind.  An item costs about as much as two pages of 128 dims (its
// Q, its join), so short chunks cost throughput, and long ones the latency of
// a lone short request:
//   few    4 pages of 128 dims (64 ragged requests: 135 us, with 3, 6 and 8 pages
//          136, 137 and 133; one request of 2001 tokens: 15 us, with 6 or 8 pages 19),
//          but 2 in a context of up to 8 (one user, 901 tokens, 8 heads: 13.5 us,
//          with 4 pages 15.5); 8 of 64 dims (32 requests, window of 9 pages, 16
//          heads: 31.7 us whole, 36 in two);
//   single 16 (32 requests of 20 rows: 144 us, with 8 tiles 166), or 12 where
//          half of the items then have 12 to 16 tiles each (a lone request in one
//          round over the SMs: 64 rows of one KV head over 262144 tokens, 147
//          chunks of 14 tiles instead of 128 of 16);
//   paired 8 where the row tiles do not fill the SMs; where they do, only those
//          left over from full rounds are cut, in up to four (kv_plan).
__host__ __device__ constexpr int kv_units(int kind) { return kind == kKvPaired ? 148 : 296; }
__host__ __device__ constexpr int kv_min_tiles(int kind, int D, int nt) {
    return kind == kKvFew ? (D == 64 ? 8 : (nt <= 8 ? 2 : 4)) : (kind == kKvSingle ? 16 : 8);
}

// Key tiles of row tile i: [lo, hi); of its two halves: first half [lo, hi0), second [lo1, hi).
// [k_lo, k_hi): the positions that some row sees.
struct KvRange {
    int lo, hi, hi0, lo1, k_lo, k_hi;
};
__host__ __device__ inline KvRange kv_range(const KvPlan &p, int pos0, int i, int window) {
    KvRange g;
    const int r0 = p.kind == kKvPaired ? 256 * i : 0, rows_left = p.rows - r0;
    const int n = rows_left < 256 ? rows_left : 256;
    const int first = kv_div(r0, p.G), last = kv_div(r0 + n - 1, p.G);
    g.k_lo = window > 0 && pos0 + first - window + 1 > 0 ? pos0 + first - window + 1 : 0;
    g.k_hi = pos0 + last + 1;
    g.lo = g.k_lo / CSLA_PAGE_TOKENS;
    g.hi = (g.k_hi + CSLA_PAGE_TOKENS - 1) / CSLA_PAGE_TOKENS;
    g.hi0 = g.hi;
    g.lo1 = g.lo;
    if (p.kind == kKvPaired) {
        if (n <= 128) {
            g.lo1 = g.hi;
        } else {
            g.hi0 = (pos0 + kv_div(r0 + 127, p.G)) / CSLA_PAGE_TOKENS + 1;
            const int lo = window > 0 ? pos0 + kv_div(r0 + 128, p.G) - window + 1 : 0;
            g.lo1 = lo > 0 ? lo / CSLA_PAGE_TOKENS : 0;
        }
    }
    return g;
}
__host__ __device__ inline KvPlan kv_plan(int T, int L, int G, int HK, int window, int D) {
    KvPlan p;
    p.T = T;
    p.G = G;
    p.rows = T * G;
    p.kind = p.rows <= kKvFewRows ? kKvFew : (p.rows <= 128 ? kKvSingle : kKvPaired);
    p.R = p.kind == kKvPaired ? (p.rows + 255) / 256 : 1;
    // key tiles of the longest row tile (with a window: an upper bound)
    int nt = (L - 1) / CSLA_PAGE_TOKENS + 1;
    if (window > 0 && window < L) {
        const int w = (window - 2 + (p.kind == kKvPaired ? kv_div(256, G) + 1 : T) + CSLA_PAGE_TOKENS) / CSLA_PAGE_TOKENS + 1;
        nt = w < nt ? w : nt;
    }
    // chunks: kv_units items in all at most, kv_min_tiles tiles at least, of even sizes
    // (32-bit divisions only: this runs ahead of every item's first load)
    int n = kv_div(kv_units(p.kind), HK * p.R);
    const int fit = nt / kv_min_tiles(p.kind, D, nt);
    if (p.kind == kKvSingle && n > fit && n / 2 * 12 <= nt && n / 2 > fit)
        n /= 2;   // one round over the SMs with chunks of 12 to 16 tiles rather than less than one
    else
        n = n < fit ? n : fit;
    const bool many = HK * p.R >= kv_units(p.kind);
    int c = n > 1 ? kv_div(nt + n - 1, n) : nt;
    p.Rs = p.kind == kKvSingle || c < nt ? p.R : 0;
    if (p.kind == kKvPaired && many && (window == 0 || window >= L) && L - T >= T) {
        // more row tiles than SMs, all of about nt tiles
        const int sms = kv_units(kKvPaired), left = HK * p.R % sms, cuts = left ? kv_div(sms, left) : 1;
        if (cuts > 1 && nt >= 32 && HK * p.R < 16 * sms) {
            p.Rs = kv_div(left + HK - 1, HK);
            c = kv_div(nt + (cuts < 4 ? cuts : 4) - 1, cuts < 4 ? cuts : 4);
        }
    }
    p.c = c;
    p.nch = p.Rs ? kv_div(nt + c - 1, c) : 1;
    p.rows_s = p.Rs == p.R ? p.rows : 256 * p.Rs;
    // K and V of all heads below half of L2: heads in turn, longest row tiles first
    p.heads_inside = (long long)L * HK * D * 4 <= (64ll << 20);
    return p;
}
// Items of a request: row tiles Rs .. R-1 once per head, the cut ones nch times.
__host__ __device__ inline int kv_items(const KvPlan &p, int HK) { return HK * (p.R - p.Rs + p.Rs * p.nch); }
// Partials of a row of row tile i (keys g): 1 means it is written out at once.
__host__ __device__ inline int kv_parts(const KvPlan &p, const KvRange &g, int i) {
    if (i >= p.Rs) return 1;
    const int nt = g.hi - g.lo, n = kv_div(nt + p.c - 1, p.c);
    return p.kind == kKvSingle && nt > 1 ? 2 * n : n;
}
// Partial rows that a request may need (rows_s of each part and head).
__host__ __device__ inline long long kv_part_rows(const KvPlan &p, int HK) {
    if (p.Rs == 0 || (p.kind == kKvSingle ? p.c == 1 : p.nch == 1)) return 0;
    return (p.kind == kKvSingle ? 2ll : 1ll) * p.nch * p.rows_s * HK;
}
cudaError_t launch_kv_few(const KvAttendArgs &a, bool q_bf16, bool out_bf16, const CUtensorMap &km,
                          const CUtensorMap &vm, int num_sms, long long items, cudaStream_t stream);
// Tokens of a ring stage of kv_few_kernel (the height of its tensor maps' boxes).
inline int kv_few_box(int D) { return D == 128 ? 64 : 128; }
// Reads and clears the device error word of kv_attend.cu's unit (0 where it shares the library's).
cudaError_t kv_attend_dev_err(unsigned int *bits);
cudaError_t launch_kv_attend(const KvAttendArgs &a, bool q_bf16, bool out_bf16, const CUtensorMap &km,
                             const CUtensorMap &vm, int num_sms, long long items, cudaStream_t stream);
cudaError_t launch_kv_join(const KvAttendArgs &a, bool out_bf16, int num_sms, cudaStream_t stream);

}  // namespace csla
