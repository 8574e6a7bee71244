// The batch walk and the bounded wait of the dense attention (kv_walk.cuh) as
// host code: 32 lanes as fibers that meet at every warp intrinsic.  Built by
// test_kv_walk.py.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>
#include <ucontext.h>

#include <algorithm>
#include <functional>
#include <vector>

using std::max;
using std::min;

#include "../include/csla.h"

// ---- a warp
struct Dim {
    int x;
};
static Dim threadIdx, blockIdx, gridDim;
static ucontext_t g_main, g_lane[32];
static bool g_done[32];
static std::function<void()> g_body;
static uint64_t g_box[2][32];
static int g_turn[32];

static void enter(int lane) {
    threadIdx.x = lane;
    g_body();
    g_done[lane] = true;
}
static void run_warp(const std::function<void()> &body) {
    static std::vector<char> stacks(32 * 65536);
    g_body = body;
    for (int i = 0; i < 32; ++i) {
        g_done[i] = false;
        g_turn[i] = 0;
        getcontext(&g_lane[i]);
        g_lane[i].uc_stack.ss_sp = &stacks[i * 65536];
        g_lane[i].uc_stack.ss_size = 65536;
        g_lane[i].uc_link = &g_main;
        makecontext(&g_lane[i], reinterpret_cast<void (*)()>(enter), 1, i);
    }
    for (bool live = true; live;) {
        live = false;
        for (int i = 0; i < 32; ++i)
            if (!g_done[i]) {
                threadIdx.x = i;
                swapcontext(&g_main, &g_lane[i]);
                live = live || !g_done[i];
            }
    }
}
// Every lane's value; two boxes, so that a lane may be one step ahead.
template <typename T>
static const uint64_t *meet(T v) {
    const int lane = threadIdx.x;
    uint64_t *box = g_box[g_turn[lane]++ & 1];
    box[lane] = 0;
    memcpy(&box[lane], &v, sizeof(v));
    swapcontext(&g_lane[lane], &g_main);
    return box;
}
template <typename T>
static T lane_of(const uint64_t *box, int i) {
    T v;
    memcpy(&v, &box[i], sizeof(v));
    return v;
}
template <typename T>
static T __shfl_sync(unsigned, T v, int src) {
    return lane_of<T>(meet(v), src & 31);
}
template <typename T>
static T __shfl_xor_sync(unsigned, T v, int o) {
    const int me = threadIdx.x;
    return lane_of<T>(meet(v), me ^ o);
}
template <typename T>
static T __shfl_up_sync(unsigned, T v, int o) {
    const int me = threadIdx.x;
    return lane_of<T>(meet(v), me >= o ? me - o : me);
}
static unsigned __ballot_sync(unsigned, int p) {
    const uint64_t *box = meet(p);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (lane_of<int>(box, i) != 0) << i;
    return r;
}
static int __any_sync(unsigned m, int p) { return __ballot_sync(m, p) != 0; }
static int __ffs(unsigned x) { return __builtin_ffs(x); }

// ---- a clock, a barrier that completes at a time, the error word
static unsigned g_err;
static uint64_t g_now, g_ready, g_stop_at;
static volatile int g_stop;
static void set_dev_err(unsigned bits) { g_err |= bits; }
static uint64_t globaltimer_ns() { return g_now; }
static bool mbar_try_wait(uint64_t *, uint32_t) {
    g_now += 1000;
    if (g_now >= g_stop_at) g_stop = 1;
    return g_now >= g_ready;
}
namespace csla {
using ::set_dev_err;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
}  // namespace csla

#include "../compressed_sparse_long_append_b200/csrc/kv_walk.cuh"

using namespace csla;

extern "C" {

// Walks the batch as CTA `block` of `grid`.  join [B][6]: n0, rows_s, parts, T, L, base as
// left by CTA 0; out: items taken, error bits, partial rows of the whole batch.
void walk(const int32_t *shape, const int32_t *slots, const int32_t *q_start, const int32_t *len, int B, int N, int T,
          int n_slots, int bt_stride, int max_new, int max_len, int grid, int block, unsigned kinds, int give_up,
          int64_t *join, int64_t *out) {
    KvAttendArgs a{};
    a.D = shape[0]; a.HQ = shape[1]; a.HK = shape[2]; a.window = shape[3];
    a.bt.slots = slots; a.bt.q_start = q_start; a.bt.len = len;
    a.bt.B = B; a.bt.N = N; a.bt.T = T; a.bt.n_slots = n_slots; a.bt.bt_stride = bt_stride;
    a.max_new = max_new; a.max_len = max_len;
    std::vector<KvJoin> req(B);
    memset(req.data(), 0x77, B * sizeof(KvJoin));
    a.part_req = req.data();
    gridDim.x = grid;
    blockIdx.x = block;
    g_err = 0;
    run_warp([&] {
        int n = 0;
        kv_walk(a, kinds, [&](const KvWalk &w, bool more, int, int) {
            if (threadIdx.x == 0 && !more) out[2] = w.part_before;   // (of all requests, at the end)
            return !more || n++ != give_up;
        });
        if (threadIdx.x == 0) out[0] = n;
    });
    out[1] = g_err;
    for (int b = 0; b < B; ++b) {
        const KvJoin &r = req[b];
        const int64_t v[6] = {r.n0, r.rows_s, r.parts, r.T, r.L, (int64_t)r.base};
        memcpy(join + 6 * b, v, sizeof(v));
    }
}

// kv_wait on a barrier that completes after ready_ms (item 1: a wait for the end of an item), of a CTA in which another
// role gives up after abort_ms (0: never).  Returns what it returned, *ms the time it took, *abort the flag it left.
int wait(int64_t ready_ms, int64_t abort_ms, int item, int64_t *ms, int *abort, unsigned *err) {
    uint64_t bar = 0;
    const uint64_t t0 = g_now = 12345;
    g_ready = g_now + ready_ms * 1000000;
    g_stop_at = abort_ms ? g_now + abort_ms * 1000000 : ~0ull;
    g_stop = 0;
    g_err = 0;
    const bool ok = item ? kv_wait(&bar, 0, &g_stop, kItemLimitNs) : kv_wait(&bar, 0, &g_stop);
    *ms = (int64_t)((g_now - t0) / 1000000);
    *abort = g_stop;
    *err = g_err;
    return ok;
}

}  // extern "C"
