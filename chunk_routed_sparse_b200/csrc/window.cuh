// Sliding-window attention with always-visible first keys: the problem, its rows'
// key sets and a query tile's key tiles, shared by the forward, backward and
// few-row kernels.
//
// Row t < m of a sequence of n keys (m = q_len, n = kv_len) is at position
// p = t + n - m. Key u < n is visible to it iff (not causal or u <= p) and
// (u < sinks or p - left <= u <= p + right): the union of [0, s) and [lo, hi)
// with all three ends non-decreasing in p, so that the keys that a run of rows can
// see are the first row's lo, the last row's hi and the last row's s.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moc.h"

namespace moc {

constexpr int kWinOpen = 1 << 30;  // left / right: no limit

struct WinArgs {
    int32_t B, Hq, Hk, group;   // group = Hq / Hk query heads share a key head
    int32_t Lq, Lk;
    int32_t left, right, sinks; // kWinOpen: no limit (left, right); causal: right is 0
    int32_t causal;
    const int32_t* q_len;       // [B] or null: Lq
    const int32_t* kv_len;      // [B] or null: Lk
    float scale;
    int16_t fill;               // rows past the lengths: 0 left as they were, 1 written as empty
    int16_t joined;             // backward: O and lse go over more keys than this call's
};
static_assert(sizeof(WinArgs) == 64, "eight bytes more cost every launch 0.3 us (tiny scene 14.0 -> 14.4 us a call)");

#ifdef __CUDACC__
namespace win {

// Lengths of a batch entry, clamped to the tensors.
struct Seq {
    int n, m, shift;  // keys, query rows, position of row 0
};
__device__ __forceinline__ Seq seq(const WinArgs& a, int b) {
    Seq s;
    s.n = a.kv_len ? min(max(a.kv_len[b], 0), a.Lk) : a.Lk;
    s.m = a.q_len ? min(max(a.q_len[b], 0), a.Lq) : a.Lq;
    s.shift = s.n - s.m;
    return s;
}

// Visible keys of the row at position p: [0, s) and [lo, hi).
struct Row {
    int s, lo, hi;
};
__device__ __forceinline__ Row row(const WinArgs& a, int n, int p) {
    Row r;
    const int end = a.causal ? min(max(p + 1, 0), n) : n;
    r.s = min(a.sinks, end);
    r.lo = max(p - a.left, 0);
    r.hi = min(max(p + a.right + 1, 0), end);
    return r;
}

// Key tiles of rows [t0, t1) (t0 < t1 <= m): na tiles of [0, a1), then nb of [b0, b1).
struct Span {
    int a1, b0, b1, na, nb;
};
constexpr int kTile = 128;
__device__ __forceinline__ Span span(const WinArgs& a, const Seq& q, int t0, int t1) {
    const Row f = row(a, q.n, t0 + q.shift), l = row(a, q.n, t1 - 1 + q.shift);
    Span x;
    if (l.hi <= f.lo) {          // no window keys
        x.a1 = 0;
        x.b0 = 0;
        x.b1 = l.s;
    } else if (f.lo <= l.s) {    // the two runs meet
        x.a1 = 0;
        x.b0 = 0;
        x.b1 = max(l.s, l.hi);
    } else {
        x.a1 = l.s;
        x.b0 = f.lo;
        x.b1 = l.hi;
    }
    x.na = (x.a1 + kTile - 1) / kTile;
    x.nb = (x.b1 - x.b0 + kTile - 1) / kTile;
    return x;
}
// Tile j of a span: first key and end of its keys (at most kTile past it).
__device__ __forceinline__ void tile(const Span& x, int j, int& key0, int& end) {
    if (j < x.na) {
        key0 = j * kTile;
        end = min(key0 + kTile, x.a1);
    } else {
        key0 = x.b0 + (j - x.na) * kTile;
        end = min(key0 + kTile, x.b1);
    }
}
// Whether a run of rows with span y sees any key of [key0, end).
__device__ __forceinline__ bool meets(const Span& y, int key0, int end) {
    return key0 < y.a1 || (key0 < y.b1 && end > y.b0);
}

// A work item of the kernels that own rows: up to `rows_item` consecutive rows of a query
// head. Items of one range of rows lie next to each other over the heads; the last rows
// (the longest spans under an open causal window) come first.
struct Item {
    int b, hq, t0;  // first row
    int rows;       // live rows (<= 0: none)
    Seq seq;
    Span y;         // key tiles
    int tiles;
};
__device__ __forceinline__ void decode(const WinArgs& a, int rows_item, int nqt, int item, Item& x) {
    const int heads = a.B * a.Hq;
    const int qt = nqt - 1 - item / heads, bh = item % heads;
    x.b = bh / a.Hq;
    x.hq = bh - x.b * a.Hq;
    x.t0 = qt * rows_item;
    x.seq = seq(a, x.b);
    x.rows = min(rows_item, x.seq.m - x.t0);
    x.y = Span{0, 0, 0, 0, 0};
    if (x.rows > 0) x.y = span(a, x.seq, x.t0, x.t0 + x.rows);
    x.tiles = x.y.na + x.y.nb;
}
// The k-th item of a CTA: rounds over the grid, every other one backwards, so that
// no CTA gets the longer item of every round.
__device__ __forceinline__ int nth_item(int k) {
    const int g = int(gridDim.x), i = int(blockIdx.x);
    return k * g + ((k & 1) ? g - 1 - i : i);
}

// The tcgen05 kernels' block: two warpgroups that compute and one that loads and issues.
constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168, kRegsCompute = 216, kRegsOther = 72;  // registers a thread: at launch, then by role
static_assert(256 * kRegsCompute + 128 * kRegsOther <= kThreads * kRegsLaunch, "registers of the launch");

// Bits c of [0, 32) with lo <= c < hi.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (hi <= lo) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

}  // namespace win
#endif

// The window kernels' error code and detail on the current device (device memory).
cudaError_t window_error_word(int32_t** word);

// Workspace of the backward pass.
struct WinBwdPlan {
    size_t work = 0;     // int32[64]: work counters of the dQ and the dK / dV kernel
    size_t nl2 = 0;      // fp32 [B Hq][Lq up to a multiple of 4], + 128: minus the log-sum-exp in exp2 units
    size_t nd = 0;       // the same of minus D = - dO . o
    size_t part = 0;     // fp32 [units][2][128][d]: dV, dK parts of the split key tiles
    size_t total = 0;
    int key_tiles = 0;   // of one (b, key head)
    int split_tiles = 0; // leading key tiles whose rows are split over units
    int splits = 1;      // units of such a tile
};
WinBwdPlan plan_window_bwd(const WinArgs& a, int d);
cudaError_t launch_window_bwd(const WinArgs& a, int d, const void* Q, const void* K, const void* V, const void* O,
                              const float* lse, const void* dO, void* dQ, void* dK, void* dV, char* ws,
                              const WinBwdPlan& p, cudaStream_t s);

cudaError_t launch_window_fwd(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                              float* lse, cudaStream_t s);

// The same, one 128-row tile an item: called by launch_window_fwd for few row tiles.
cudaError_t launch_window_tile(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                               float* lse, cudaStream_t s);

// Few rows against a cache: Lq * group <= kWinFewRows, B * Hk <= 65535, Lk > 0.
constexpr int kWinFewRows = 16;
cudaError_t launch_window_few(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                              float* lse, cudaStream_t s);

}  // namespace moc
