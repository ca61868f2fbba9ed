// Sliding-window attention with always-visible first keys, forward, on the
// 5th-generation tensor cores.
//
//   O_t = sum_u softmax_u(scale q_t . k_u) v_u over the row's visible keys
//   (window.cuh), lse_t = log sum_u exp(scale q_t . k_u);
//   a row that sees no key: O = 0, lse = -inf.
//
// One persistent CTA per SM walks work items (up to 256 consecutive rows of a head, two
// 128-row tiles A and B that share one key stream) in a fixed order: no counter in
// memory, so calls on different streams and captured graphs share nothing.
// (Items handed out by the hardware, clusterlaunchcontrol.try_cancel: 658 -> 715 us on the
// clip below. Padded batches, whose items are unlike, take k_window_tile.cu.)
//   warp 8 (one lane): TMA of Q tiles and of 128-key K and V tiles (2-stage rings).
//   warp 9 (one lane): S_q = Q K^T and O_q += P V (P from TMEM), alternating A and
//          B; an item's last PV and the next item's first S are issued back to back.
//   warps 0-3 / 4-7: softmax of tile A / B, one thread a row, running max and sum
//          in fp32, P written over S as bf16 (2^-8 of each weight at most; the sum is of
//          the unrounded weights) in two halves, so that the first half of P V runs
//          under the second half's exponentials (5 %); the epilogue stages O through
//          shared memory into whole 128-byte row pieces.
// Single-shot clip (12 heads, 33,272 tokens, d = 128, 512 first keys and 1,560 on either
// side; 722 GFLOP on visible pairs): 0.66 ms in short runs (1.10 PFLOP/s), 0.77 ms
// once the 1 kW power cap holds the clock. Neither the tensor core nor the exponentials
// are above half busy (45 % each with 4 heads, 53 % each causal over 6,239 keys): each
// tile's chain of product, softmax and product sets the pace; a share of the exponentials
// on the FMA pipe measured slower.
// A tile that one of A, B cannot see is skipped for it; a tile that every row of a
// warp sees whole takes no masking. Keys past a tile's end are other rows' or none:
// their scores become -inf and their V rows are zeroed in shared memory (0 x NaN).
// Every wait is bounded (2 s): a wait that gives up records itself in the error
// word of moc_window_device_error and every role leaves.
#include <atomic>

#include "common.cuh"
#include "pipeline.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace moc {

namespace {

__device__ int32_t g_window_err[64];  // error code and detail of the window kernels on this device

constexpr int kMaxDevices = 64;
std::atomic<int32_t*> g_err_ptr[kMaxDevices];  // its address on each device, looked up once

}  // namespace

cudaError_t window_error_word(int32_t** word) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    *word = g_err_ptr[dev].load(std::memory_order_acquire);
    if (*word) return cudaSuccess;
    void* p = nullptr;
    const cudaError_t st = cudaGetSymbolAddress(&p, g_window_err);
    if (st != cudaSuccess) return st;
    *word = static_cast<int32_t*>(p);
    g_err_ptr[dev].store(*word, std::memory_order_release);
    return cudaSuccess;
}

namespace {

using namespace sm100;

using win::kRegsCompute;
using win::kRegsOther;
using win::kThreads;
constexpr uint32_t kTmemCols = 512;
constexpr int kRowsItem = 256;
constexpr float kLazy = 8.f;  // O is rescaled once the row max grows by more than 2^8

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int oQ = 0;
    static constexpr int oK = oQ + 2 * kTileBytes;
    static constexpr int oV = oK + 2 * kTileBytes;
    static constexpr int oStage = oV + 2 * kTileBytes;  // 8 warps x 32 rows x 128 B
    static constexpr int oBar = oStage + 8 * 4096;
    // + alignment slack; at least 120 KB so that one CTA owns an SM and its TMEM
    static constexpr int kSmem = (oBar + 256 + 1024) > 120 * 1024 ? (oBar + 256 + 1024) : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
};

__device__ __forceinline__ uint32_t col_s(int q) { return q ? 128u : 0u; }
__device__ __forceinline__ uint32_t col_o(int q) { return q ? 384u : 256u; }

enum {
    B_Q_FULL = 0, B_Q_EMPTY = 2, B_K_FULL = 4, B_K_EMPTY = 6, B_V_FULL = 8, B_V_EMPTY = 10, B_S_FULL = 12,
    B_P_FULL = 14, B_PV_DONE = 16, B_MMA_DONE = 18, B_P_HALF = 19, B_COUNT = 21
};
struct Shared {  // at oBar + 176
    uint32_t tmem_base;
    int abort;
};
static_assert(B_COUNT * 8 <= 176, "barriers");

using win::Item;
using win::nth_item;
// One of an item's two row tiles. Each role keeps both in scalars (an index that the
// compiler cannot see through would put them in local memory).
struct QTile {
    int rows;         // live rows
    win::Span y;
    int last;         // the item's last key tile that it sees (-1: none)
    __device__ __forceinline__ bool sees(int key0, int end) const { return last >= 0 && win::meets(y, key0, end); }
};

__device__ __forceinline__ void decode(const WinArgs& a, int item, Item& x) {
    win::decode(a, kRowsItem, (a.Lq + kRowsItem - 1) / kRowsItem, item, x);
}
__device__ __forceinline__ QTile tile_of(const WinArgs& a, const Item& x, int q) {
    QTile t;
    const int r0 = x.t0 + 128 * q, r1 = min(r0 + 128, x.t0 + x.rows);
    t.rows = max(r1 - r0, 0);
    t.y = win::Span{0, 0, 0, 0, 0};
    t.last = -1;
    if (t.rows > 0) {
        t.y = win::span(a, x.seq, r0, r1);
        const int key = max(t.y.a1, t.y.b1) - 1;  // its last key lies in one of the item's runs
        if (key >= 0) t.last = x.y.nb > 0 && key >= x.y.b0 ? x.y.na + (key - x.y.b0) / win::kTile : key / win::kTile;
    }
    return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WinArgs a, int n_items,
                      __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base + C::oQ, sK = base + C::oK, sV = base + C::oV, sBar = base + C::oBar;
    Shared& sh = *reinterpret_cast<Shared*>(gbase + C::oBar + 176);
    volatile int* abort = &sh.abort;
    int32_t* const hdr = g_window_err;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    let_next_kernel_start();

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) mbar_init(bar(x), (x == B_P_FULL || x == B_P_FULL + 1 || x >= B_P_HALF) ? 128 : 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uint32_t(uniform(int(sh.tmem_base)));
    wait_for_previous_kernel();
    const int n_rounds = (n_items + int(gridDim.x) - 1) / int(gridDim.x);

    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == 8 && lane == 0) {
            // ---------------------------------------------------------- loads
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            uint32_t gk = 0, gv = 0, nq[2] = {0, 0};
            bool stop = false;
            for (int k = 0; k < n_rounds && !stop; ++k) {
                const int item = nth_item(k);
                if (item >= n_items) continue;
                Item x;
                decode(a, item, x);
                const QTile qt[2] = {tile_of(a, x, 0), tile_of(a, x, 1)};
                const int qrow = (x.b * a.Hq + x.hq) * a.Lq + x.t0;
                const int krow = (x.b * a.Hk + x.hq / a.group) * a.Lk;
                bool have[2] = {false, false};
                for (int j = 0; j < x.tiles && !stop; ++j) {
                    int key0, end;
                    win::tile(x.y, j, key0, end);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {  // a Q tile arrives with the first key tile that it sees
                        if (have[q] || !qt[q].sees(key0, end)) continue;
                        have[q] = true;
                        if (!wait_bar(bar(B_Q_EMPTY + q), (nq[q] & 1) ^ 1, abort, hdr, 201)) { stop = true; break; }
                        ++nq[q];
                        mbar_expect_tx(bar(B_Q_FULL + q), C::kTileBytes);
#pragma unroll
                        for (int s = 0; s < C::kSlabs; ++s)
                            tma_load_2d(sQ + q * C::kTileBytes + s * C::kSlabBytes, &tmQ, bar(B_Q_FULL + q), 64 * s,
                                        qrow + 128 * q);
                    }
                    if (stop) break;
                    const uint32_t st = gk & 1, sv = gv & 1;
                    if (!wait_bar(bar(B_K_EMPTY + st), ((gk >> 1) & 1) ^ 1, abort, hdr, 202)) { stop = true; break; }
                    mbar_expect_tx(bar(B_K_FULL + st), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sK + st * C::kTileBytes + s * C::kSlabBytes, &tmK, bar(B_K_FULL + st), 64 * s,
                                    krow + key0);
                    ++gk;
                    if (!wait_bar(bar(B_V_EMPTY + sv), ((gv >> 1) & 1) ^ 1, abort, hdr, 203)) { stop = true; break; }
                    mbar_expect_tx(bar(B_V_FULL + sv), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sV + sv * C::kTileBytes + s * C::kSlabBytes, &tmV, bar(B_V_FULL + sv), 64 * s,
                                    krow + key0);
                    ++gv;
                }
            }
            // every issued copy lands before the CTA exits
            for (uint32_t g = gk >= 2 ? gk - 2 : 0; g < gk; ++g) drain_bar(bar(B_K_FULL + (g & 1)), (g >> 1) & 1, hdr, 204);
            for (uint32_t g = gv >= 2 ? gv - 2 : 0; g < gv; ++g) drain_bar(bar(B_V_FULL + (g & 1)), (g >> 1) & 1, hdr, 205);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (nq[q] > 0) drain_bar(bar(B_Q_FULL + q), (nq[q] - 1) & 1, hdr, 206);
        } else if (warp == 9) {
            // ---------------------------------------------------------- MMA issue
            // The whole warp walks the tiles and one elected lane issues, so that addresses
            // and descriptors stay in uniform registers: issued from a divergent lane, a
            // product of eight MMAs took 700 cycles to issue, longer than it runs.
            const bool leader = elect_one();
            uint32_t gt = 0;                 // key tiles
            uint32_t np[2] = {0, 0};         // tiles of A / B (S_FULL, P_FULL, PV_DONE phases)
            uint32_t nq[2] = {0, 0};         // Q tiles
            bool pend[2] = {false, false};   // S issued for the previous key tile, PV outstanding
            bool fresh[2] = {false, false};  // that PV is the item's first
            bool stop = false;
            // O_q += P_q V of the previous key tile
            auto issue_pv = [&](const int q) -> bool {
                if (!wait_bar_warp(bar(B_P_HALF + q), (np[q] - 1) & 1, abort, hdr, 210)) return false;
                tc_fence_after();
                const uint32_t vb = sV + ((gt - 1) & 1) * C::kTileBytes;
                const uint32_t acc = fresh[q] ? 0u : 1u;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_ts(tmem + col_o(q), tmem + col_s(q) + kk * 8, sdesc_sw128(vb + kk * 2048, C::kSlabBytes, 1024),
                                C::kIdescPV, kk > 0 ? 1u : acc);
                }
                __syncwarp();
                if (!wait_bar_warp(bar(B_P_FULL + q), (np[q] - 1) & 1, abort, hdr, 211)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 4; kk < 8; ++kk)
                        umma_ts(tmem + col_o(q), tmem + col_s(q) + kk * 8, sdesc_sw128(vb + kk * 2048, C::kSlabBytes, 1024),
                                C::kIdescPV, kk > 0 ? 1u : acc);
                    umma_commit(bar(B_PV_DONE + q));
                }
                __syncwarp();
                pend[q] = fresh[q] = false;
                return true;
            };
            for (int k = 0; k < n_rounds && !stop; ++k) {
                const int item = nth_item(k);
                if (item >= n_items) continue;
                Item x;
                decode(a, item, x);
                const QTile qt[2] = {tile_of(a, x, 0), tile_of(a, x, 1)};
                const int tiles = uniform(x.tiles);
                bool have[2] = {false, false};
                for (int j = 0; j < tiles; ++j) {
                    int key0, end;
                    win::tile(x.y, j, key0, end);
                    const uint32_t st = gt & 1;
                    if (gt > 0 && !wait_bar_warp(bar(B_V_FULL + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1, abort, hdr, 212)) { stop = true; break; }
                    bool k_ready = false;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (pend[q] && !issue_pv(q)) { stop = true; break; }
                        if (!k_ready) {
                            if (!wait_bar_warp(bar(B_K_FULL + st), (gt >> 1) & 1, abort, hdr, 213)) { stop = true; break; }
                            k_ready = true;
                        }
                        if (!uniform(qt[q].sees(key0, end))) continue;
                        if (!have[q]) {
                            if (!wait_bar_warp(bar(B_Q_FULL + q), nq[q] & 1, abort, hdr, 214)) { stop = true; break; }
                            have[q] = fresh[q] = true;
                            ++nq[q];
                        }
                        tc_fence_after();
                        const uint32_t qb = sQ + q * C::kTileBytes, kb = sK + st * C::kTileBytes;
                        const bool last = uniform(j == qt[q].last);
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                                umma_ss(tmem + col_s(q), sdesc_sw128(qb + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024),
                                        C::kIdescQK, kk > 0);
                            }
                            umma_commit(bar(B_S_FULL + q));
                            if (last) umma_commit(bar(B_Q_EMPTY + q));  // its Q rows may be replaced
                        }
                        __syncwarp();
                        pend[q] = true;
                        ++np[q];
                    }
                    if (stop) break;
                    if (leader) {
                        if (gt > 0) umma_commit(bar(B_V_EMPTY + ((gt - 1) & 1)));
                        umma_commit(bar(B_K_EMPTY + st));
                    }
                    __syncwarp();
                    ++gt;
                }
            }
            if (!stop && gt > 0) {
                if (wait_bar_warp(bar(B_V_FULL + ((gt - 1) & 1)), ((gt - 1) >> 1) & 1, abort, hdr, 215)) {
                    bool ok = !pend[0] || issue_pv(0);
                    if (ok && pend[1]) issue_pv(1);
                }
            }
            if (leader) {
                umma_commit(bar(B_MMA_DONE));  // TMEM is released after every MMA
                drain_bar(bar(B_MMA_DONE), 0, hdr, 216);
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- softmax
        const int q = warp >> 2, row = tid & 127;
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + col_s(q), o_addr = lane_addr + col_o(q);
        const uint32_t stg = base + C::oStage + warp * 4096;
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t gt = 0, np = 0;
        bool stop = false;
        for (int k = 0; k < n_rounds && !stop; ++k) {
            const int item = nth_item(k);
            if (item >= n_items) continue;
            Item x;
            decode(a, item, x);
            const QTile qt = tile_of(a, x, q);
            const int rows_out = qt.rows;  // all rows live: padded batches take the one-tile kernel
            if (rows_out <= 0) {
                gt += x.tiles;
                continue;
            }
            const int t = x.t0 + 128 * q + row;
            const bool live = row < qt.rows;
            const win::Row vis = win::row(a, x.seq.n, t + x.seq.shift);
            float m_used = -INFINITY, l = 0.f;
            bool any = false;
            for (int j = 0; j < x.tiles; ++j, ++gt) {
                int key0, end;
                win::tile(x.y, j, key0, end);
                if (!qt.sees(key0, end)) continue;
                if (!wait_bar_warp(bar(B_S_FULL + q), np & 1, abort, hdr, 221)) { stop = true; break; }
                tc_fence_after();
                const int ns = min(vis.s, end) - key0, lo = vis.lo - key0, hi = min(vis.hi, end) - key0;
                if (!__all_sync(0xffffffffu, !live || ns >= 128 || (lo <= 0 && hi >= 128))) {
                    // masked in TMEM, 64 columns at a time, before the scores are loaded: masking
                    // them among the 128 loaded registers spilled in every tile (1.09 ms against
                    // 0.70 ms on the single-shot clip)
#pragma unroll 1
                    for (int w = 0; w < 128; w += 64) {
                        const uint32_t k0 = win::bits(0, ns - w) | win::bits(lo - w, hi - w);
                        const uint32_t k1 = win::bits(0, ns - w - 32) | win::bits(lo - w - 32, hi - w - 32);
                        if (__all_sync(0xffffffffu, (k0 & k1) == 0xffffffffu)) continue;
                        uint32_t v[64];
                        tmem_ld32(s_addr + w, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                        tmem_ld32(s_addr + w + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                        tmem_wait_ld_regs(v);
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!((c < 32 ? k0 : k1) & (1u << (c & 31)))) v[c] = 0xff800000u;  // -inf
                        tmem_st32(s_addr + w, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
                        tmem_st32(s_addr + w + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
                    }
                    tmem_wait_st();
                }
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
                tmem_wait_ld_regs(s);
                float mv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mv[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
                for (int c = 16; c < 128; c += 16) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mv[i] = max3(mv[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
                }
                const float mx = max3(max3(mv[0], mv[1], mv[2]), max3(mv[3], mv[4], mv[5]), fmaxf(mv[6], mv[7])) * sl2;
                float alpha = 1.f;
                bool rescale = false;
                if (mx > m_used + kLazy) {  // also the first visible key: nothing to rescale then
                    if (m_used > -INFINITY) {
                        alpha = ex2(m_used - mx);
                        rescale = true;
                    }
                    m_used = mx;
                }
                if (__any_sync(0xffffffffu, rescale)) {  // warp-collective TMEM access; alpha = 1 elsewhere
                    if (!wait_bar_warp(bar(B_PV_DONE + q), (np - 1) & 1, abort, hdr, 222)) { stop = true; break; }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + c * 32, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(o_addr + c * 32, o);
                    }
                }
                if (end - key0 < 128) {  // V rows past the tile's keys: zeros, whatever was loaded
                    if (!wait_bar_warp(bar(B_V_FULL + (gt & 1)), (gt >> 1) & 1, abort, hdr, 223)) { stop = true; break; }
                    if (row >= end - key0) {
                        const uint32_t vr = sV + (gt & 1) * C::kTileBytes + row * 128;
#pragma unroll
                        for (int i = 0; i < C::kSlabs * 8; ++i)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vr + (i >> 3) * C::kSlabBytes + (i & 7) * 16),
                                         "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();
                }
                // a row without a visible key so far: its weights are exp2(-inf - 0) = 0
                const float m0 = m_used > -INFINITY ? m_used : 0.f;
                const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m0, -m0);
                uint64_t sum2a = 0, sum2b = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const int e = h * 64 + 2 * c;
                        float x0, x1;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2, nm2), x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        if (c & 1) sum2b = f2_add(sum2b, f2_pack(p0, p1));
                        else sum2a = f2_add(sum2a, f2_pack(p0, p1));
                        pk[c] = pack_bf16(p0, p1);
                    }
                    tmem_st32(s_addr + h * 32, pk);
                    if (h == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(bar(B_P_HALF + q));
                    }
                }
                float r0, r1, r2, r3;
                f2_unpack(sum2a, r0, r1);
                f2_unpack(sum2b, r2, r3);
                l = l * alpha + ((r0 + r1) + (r2 + r3));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_P_FULL + q));
                ++np;
                any = true;
            }
            if (stop) break;
            // ---------------------------------------------------------- epilogue
            const size_t orow = (size_t(x.b) * a.Hq + x.hq) * size_t(a.Lq) + size_t(x.t0 + 128 * q);
            if (any) {
                if (!wait_bar_warp(bar(B_PV_DONE + q), (np - 1) & 1, abort, hdr, 224)) break;
                tc_fence_after();
            }
            const bool seen = live && (l > 0.f || l != l);  // NaN stays NaN
            const float inv = 1.f / l;
            const int w0 = (warp & 3) * 32;
            __nv_bfloat16* out = O + (orow + w0) * D;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t pk[32];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t o[32];
                    if (any) {
                        tmem_ld32(o_addr + c * 64 + hh * 32, o);
                        tmem_wait_ld_regs(o);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[hh * 16 + i] = seen ? pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stg + lane * 128 + ((i ^ (lane & 7)) << 4)),
                                 "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3]) : "memory");
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3), ch = lane & 7;
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(stg + r * 128 + ((ch ^ (r & 7)) << 4)) : "memory");
                    if (w0 + r < rows_out) *reinterpret_cast<uint4*>(out + size_t(r) * D + c * 64 + ch * 8) = v;
                }
                __syncwarp();
            }
            tc_fence_before();
            if (row < rows_out && lse) lse[orow + row] = seen ? (m_used + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch_d(const WinArgs& a, int n_items, int sms, const void* Q, const void* K, const void* V, void* O,
                     float* lse, cudaStream_t s) {
    CUtensorMap tmQ, tmK, tmV;
    const int64_t qrows = int64_t(a.B) * a.Hq * a.Lq, krows = int64_t(a.B) * a.Hk * a.Lk;
    if (!make_tmap(&tmQ, Q, D, qrows)) return cudaErrorInvalidValue;
    if (krows == 0) tmK = tmV = tmQ;  // no key tile is loaded
    else if (!make_tmap(&tmK, K, D, krows) || !make_tmap(&tmV, V, D, krows)) return cudaErrorInvalidValue;
    const int smem = Cfg<D>::kSmem;
    cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(window_fwd_kernel<D>, n_items < sms ? n_items : sms, kThreads, smem, s, tmQ, tmK, tmV, a,
                        n_items, static_cast<__nv_bfloat16*>(O), lse);
}

}  // namespace

cudaError_t launch_window_fwd(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                              float* lse, cudaStream_t s) {
    const int sms = multiprocessors();
    const int n_items = a.B * a.Hq * ((a.Lq + kRowsItem - 1) / kRowsItem);
    // Two row tiles an item keep the tensor core busy and share their keys (the single-shot
    // clip's 1,572 items: 661 against 788 us); up to three items for two SMs the one-tile
    // kernel's shorter chain and finer items end sooner (2,112 tokens, window 256 + 64, d = 64:
    // 18 items 14.9 -> 11.8 us, 81 items 18.5 -> 13.7, 162 items 27.1 -> 20.6, 216 items
    // 35.4 -> 27.9; open and causal, 33 to 34 us: 108 items -> 22.8, 216 items -> 37.4; at 408
    // items the two are level). Padded batches go there whatever their size, as it hands
    // items out by demand and the lengths are on the device. Its time over the two-tile
    // kernel's for 768 to 6,240 items, d = 64 / 128: lengths down to a tenth 0.57 to 1.15 /
    // 0.51 to 1.12, down to a half 0.77 to 1.17 / 0.75 to 1.09, one sequence empty 0.85 to 1.18 /
    // 0.76 to 1.04, within a tenth of full 1.04 to 1.21 / 0.98 to 1.13, all full 1.10 to 1.25 / 0.92 to
    // 1.08 (a batch known to be full is better called without q_len).
    if (a.q_len || n_items <= sms + sms / 2) return launch_window_tile(a, d, Q, K, V, O, lse, s);
    return d == 128 ? launch_d<128>(a, n_items, sms, Q, K, V, O, lse, s)
                    : launch_d<64>(a, n_items, sms, Q, K, V, O, lse, s);
}

}  // namespace moc
