// Sliding-window attention with always-visible first keys, backward, on the
// 5th-generation tensor cores. With p_tu = exp(scale q_t . k_u - lse_t) over the
// row's visible keys (window.cuh), D_t = dO_t . o_t and
// ds_tu = p_tu (dO_t . v_u - D_t):
//   dq_t = scale sum_u ds_tu k_u,
//   dk_u = scale sum_t ds_tu q_t,   dv_u = sum_t p_tu dO_t,
// the sums over t also over the query heads that share u's key head. p and ds are
// rounded to bf16 (2^-8 of each) as operands of the last products; all sums are in
// fp32.
//
// Three launches: D (which also clears the work counters), dQ (a work unit is a
// 128-row tile, it owns its dQ rows) and dK / dV (a unit is a 128-key tile of a key
// head, it owns its dK and dV rows and walks the rows that see it). The first keys
// are seen by every later row: their tiles' rows are split over units that write
// fp32 parts, added in order by a fourth launch. No atomics on results: they do not
// depend on the order of the units, which are handed out longest first by a counter.
#include "common.cuh"
#include "pipeline.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace moc {
namespace {

using namespace sm100;
using win::kTile;

constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

struct Shared {
    int item[2];
    uint32_t tmem_base;
    int abort;
};

// Columns [32 w, 32 w + 32) of a TMEM row: where `keep` has no bit, set `fill`.
__device__ __forceinline__ void mask_cols(uint32_t addr, uint32_t keep, uint32_t fill) {
    uint32_t v[32];
    tmem_ld32(addr, v);
    tmem_wait_ld_regs(v);
#pragma unroll
    for (int c = 0; c < 32; ++c)
        if (!(keep & (1u << c))) v[c] = fill;
    tmem_st32(addr, v);
}
constexpr uint32_t kMinusInf = 0xff800000u;

// ---- D -------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) window_rowdot_kernel(const __grid_constant__ WinArgs a,
                                                            const __nv_bfloat16* __restrict__ O,
                                                            const __nv_bfloat16* __restrict__ dO,
                                                            float* __restrict__ Dsum, int32_t* __restrict__ work) {
    constexpr int LPR = D / 8;  // lanes a row, 16 bytes each
    if (blockIdx.x == 0 && threadIdx.x < 2) work[threadIdx.x] = 0;
    const int64_t rows = int64_t(a.B) * a.Hq * a.Lq;
    const int r = threadIdx.x % LPR;
    for (int64_t row0 = int64_t(blockIdx.x) * (256 / LPR); row0 < rows; row0 += int64_t(gridDim.x) * (256 / LPR)) {
        const int64_t row = row0 + threadIdx.x / LPR;
        float acc = 0.f;
        if (row < rows) {
            const uint4 x = ldg_nc16(O + size_t(row) * D + r * 8), y = ldg_nc16(dO + size_t(row) * D + r * 8);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc = fmaf(bf16lo(xs[i]), bf16lo(ys[i]), acc);
                acc = fmaf(bf16hi(xs[i]), bf16hi(ys[i]), acc);
            }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o, LPR);
        if (r == 0 && row < rows) Dsum[row] = acc;
    }
}

// ---- dQ ------------------------------------------------------------------------
// One CTA per SM, 384 threads. TMEM: two S buffers, dP and the dQ accumulator.
//   warp 8 (one lane): units and TMA: Q and dO tiles, K tiles into a 3-stage ring (a
//          K tile serves S and, two tiles later, dQ), V tiles into a 2-stage ring.
//   warp 9 (one lane): S(j) = Q K(j)^T two tiles ahead, dP(j) = dO V(j)^T, and
//          dQ += dS(j) K(j) with dS from TMEM.
//   warps 0-7: two warpgroups, each half of a tile's keys for all 128 rows (one
//          thread a row): dS in fp32, written as bf16 over its own half of S.
namespace dq {

constexpr int kThreads = 384;
// launched at 168 registers a thread: 2 x 128 x 216 + 128 x 72 = 384 x 168
constexpr int kRegsCompute = 216, kRegsOther = 72;
constexpr uint32_t kColS0 = 0, kColS1 = 128, kColDP = 256, kColDQ = 384;

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int oQ = 0;
    static constexpr int oDO = oQ + kTileBytes;
    static constexpr int oK = oDO + kTileBytes;      // 3 stages
    static constexpr int oV = oK + 3 * kTileBytes;   // 2 stages
    static constexpr int oBar = oV + 2 * kTileBytes;
    static constexpr int kSmem = (oBar + 512 + 1024) > 120 * 1024 ? (oBar + 512 + 1024) : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr uint32_t kIdescSS = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescDQ = idesc_bf16_f32(128, D, 1);
};

enum {
    B_ITEM_FULL = 0, B_ITEM_EMPTY = 2, B_K_FULL = 4, B_K_EMPTY = 7, B_V_FULL = 10, B_V_EMPTY = 12, B_QDO_FULL = 14,
    B_QDO_EMPTY = 15, B_S_FULL = 16, B_DP_FULL = 18, B_DS_FULL = 19, B_DQ_DONE = 20, B_MMA_DONE = 21, B_COUNT = 22
};

__device__ __forceinline__ uint32_t col_s(int b) { return b ? kColS1 : kColS0; }
// column (from a buffer's first) of the bf16 pairs of keys 16 kk .. + 15
__device__ __forceinline__ uint32_t ds_col(int kk) { return 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3); }

struct Unit {
    int b, hq, t0, rows, tiles;
    win::Seq seq;
    win::Span y;
};
// the last rows (the longest spans under an open causal window) first
__device__ __forceinline__ void decode(const WinArgs& a, int nqt, int u, Unit& x) {
    const int heads = a.B * a.Hq;
    const int qt = nqt - 1 - u / heads, bh = u % heads;
    x.b = bh / a.Hq;
    x.hq = bh - x.b * a.Hq;
    x.t0 = qt * kTile;
    x.seq = win::seq(a, x.b);
    x.rows = min(kTile, x.seq.m - x.t0);
    x.y = win::Span{0, 0, 0, 0, 0};
    if (x.rows > 0) x.y = win::span(a, x.seq, x.t0, x.t0 + x.rows);
    x.tiles = x.y.na + x.y.nb;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ WinArgs a, int n_units, int nqt, const float* __restrict__ lse,
                     const float* __restrict__ Dsum, int32_t* __restrict__ work, int32_t* __restrict__ hdr,
                     __nv_bfloat16* __restrict__ dQ) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base + C::oQ, sDO = base + C::oDO, sK = base + C::oK, sV = base + C::oV;
    const uint32_t sBar = base + C::oBar;
    Shared& sh = *reinterpret_cast<Shared*>(gbase + C::oBar + 256);
    volatile int* abort = &sh.abort;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) {
            int n = 1;
            if (x == B_ITEM_EMPTY || x == B_ITEM_EMPTY + 1) n = 1 + 256;
            if (x == B_DS_FULL) n = 256;
            mbar_init(bar(x), n);
        }
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
    const uint32_t tmem = sh.tmem_base;

    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == 8 && lane == 0) {
            // ---------------------------------------------------------- units + loads
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmDO);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            uint32_t gk = 0, gv = 0, nu = 0;
            bool stop = false;
            for (int it = 0; !stop; ++it) {
                const int slot = it & 1;
                if (!wait_bar(bar(B_ITEM_EMPTY + slot), ((it >> 1) & 1) ^ 1, abort, hdr, 231)) break;
                const int u = atomicAdd(work, 1);
                sh.item[slot] = u < n_units ? u : -1;
                mbar_arrive(bar(B_ITEM_FULL + slot));
                if (u >= n_units) break;
                Unit x;
                decode(a, nqt, u, x);
                if (x.tiles == 0) continue;
                const int qrow = (x.b * a.Hq + x.hq) * a.Lq + x.t0, krow = (x.b * a.Hk + x.hq / a.group) * a.Lk;
                // the previous unit's last S and dP have read Q and dO
                if (!wait_bar(bar(B_QDO_EMPTY), (nu & 1) ^ 1, abort, hdr, 232)) break;
                ++nu;
                mbar_expect_tx(bar(B_QDO_FULL), 2 * C::kTileBytes);
#pragma unroll
                for (int s = 0; s < C::kSlabs; ++s) {
                    tma_load_2d(sQ + s * C::kSlabBytes, &tmQ, bar(B_QDO_FULL), 64 * s, qrow);
                    tma_load_2d(sDO + s * C::kSlabBytes, &tmDO, bar(B_QDO_FULL), 64 * s, qrow);
                }
                for (int j = 0; j < x.tiles; ++j) {
                    int key0, end;
                    win::tile(x.y, j, key0, end);
                    const uint32_t ks = gk % 3, vs = gv & 1;
                    if (!wait_bar(bar(B_K_EMPTY + ks), ((gk / 3) & 1) ^ 1, abort, hdr, 233)) { stop = true; break; }
                    mbar_expect_tx(bar(B_K_FULL + ks), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sK + ks * C::kTileBytes + s * C::kSlabBytes, &tmK, bar(B_K_FULL + ks), 64 * s, krow + key0);
                    ++gk;
                    if (!wait_bar(bar(B_V_EMPTY + vs), ((gv >> 1) & 1) ^ 1, abort, hdr, 234)) { stop = true; break; }
                    mbar_expect_tx(bar(B_V_FULL + vs), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sV + vs * C::kTileBytes + s * C::kSlabBytes, &tmV, bar(B_V_FULL + vs), 64 * s, krow + key0);
                    ++gv;
                }
            }
            // every issued copy lands before the CTA exits
            for (uint32_t g = gk >= 3 ? gk - 3 : 0; g < gk; ++g) drain_bar(bar(B_K_FULL + g % 3), (g / 3) & 1, hdr, 235);
            for (uint32_t g = gv >= 2 ? gv - 2 : 0; g < gv; ++g) drain_bar(bar(B_V_FULL + (g & 1)), (g >> 1) & 1, hdr, 236);
            if (nu > 0) drain_bar(bar(B_QDO_FULL), (nu - 1) & 1, hdr, 237);
        } else if (warp == 9 && lane == 0) {
            // ---------------------------------------------------------- MMA issue
            uint32_t gk = 0, gv = 0, gt = 0, nu = 0;
            bool stop = false;
            auto issue_s = [&](uint32_t kt, int b) -> bool {  // S(b) = Q K(kt)^T
                const uint32_t ks = kt % 3;
                if (!wait_bar(bar(B_K_FULL + ks), (kt / 3) & 1, abort, hdr, 241)) return false;
                tc_fence_after();
                const uint32_t kb = sK + ks * C::kTileBytes;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                    umma_ss(tmem + col_s(b), sdesc_sw128(sQ + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024),
                            C::kIdescSS, kk > 0);
                }
                umma_commit(bar(B_S_FULL + b));
                return true;
            };
            auto issue_dp = [&]() -> bool {  // dP = dO V(gv)^T, then V(gv) is free
                const uint32_t vs = gv & 1;
                if (!wait_bar(bar(B_V_FULL + vs), (gv >> 1) & 1, abort, hdr, 242)) return false;
                tc_fence_after();
                const uint32_t vb = sV + vs * C::kTileBytes;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                    umma_ss(tmem + kColDP, sdesc_sw128(sDO + off, 16, 1024), sdesc_sw128(vb + off, 16, 1024),
                            C::kIdescSS, kk > 0);
                }
                umma_commit(bar(B_DP_FULL));
                umma_commit(bar(B_V_EMPTY + vs));
                ++gv;
                return true;
            };
            for (int it = 0; !stop; ++it) {
                const int slot = it & 1;
                if (!wait_bar(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 243)) break;
                const int u = sh.item[slot];
                mbar_arrive(bar(B_ITEM_EMPTY + slot));
                if (u < 0) break;
                Unit x;
                decode(a, nqt, u, x);
                const int T = x.tiles;
                if (T == 0) continue;
                if (!wait_bar(bar(B_QDO_FULL), nu & 1, abort, hdr, 244)) break;
                ++nu;
                tc_fence_after();
                if (!issue_s(gk, 0) || !issue_dp() || (T > 1 && !issue_s(gk + 1, 1))) break;
                if (T == 1) umma_commit(bar(B_QDO_EMPTY));
                for (int j = 0; j < T; ++j) {
                    if (!wait_bar(bar(B_DS_FULL), gt & 1, abort, hdr, 245)) { stop = true; break; }
                    tc_fence_after();
                    ++gt;
                    if (j + 1 < T && !issue_dp()) { stop = true; break; }
                    if (T > 1 && j == T - 2) umma_commit(bar(B_QDO_EMPTY));  // the last S was issued before it
                    const uint32_t ks = (gk + j) % 3, kb = sK + ks * C::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ts(tmem + kColDQ, tmem + col_s(j & 1) + ds_col(kk),
                                sdesc_sw128(kb + kk * 2048, C::kSlabBytes, 1024), C::kIdescDQ, (j > 0 || kk > 0));
                    umma_commit(bar(B_K_EMPTY + ks));
                    if (j + 2 < T && !issue_s(gk + j + 2, j & 1)) { stop = true; break; }
                }
                if (stop) break;
                gk += T;
                umma_commit(bar(B_DQ_DONE));
            }
            umma_commit(bar(B_MMA_DONE));
            drain_bar(bar(B_MMA_DONE), 0, hdr, 246);
        }
        __syncwarp();
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- compute (warps 0-7)
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const float sl2 = a.scale * kLog2e;
        uint32_t gt = 0, nu = 0, ns[2] = {0, 0}, gk = 0;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 251)) break;
            const int u = sh.item[slot];
            mbar_arrive(bar(B_ITEM_EMPTY + slot));
            if (u < 0) break;
            Unit x;
            decode(a, nqt, u, x);
            if (x.rows <= 0) continue;
            const bool live = row < x.rows;
            const size_t rowg = (size_t(x.b) * a.Hq + x.hq) * size_t(a.Lq) + size_t(x.t0) + row;
            // rows past the last, and rows that see no key (lse = -inf): +inf makes every p zero
            float lse2 = INFINITY, drow = 0.f;
            if (live) {
                const float v = __ldg(lse + rowg);
                if (v > -INFINITY || v != v) lse2 = v * kLog2e;
                drow = __ldg(Dsum + rowg);
            }
            const win::Row vis = win::row(a, x.seq.n, x.t0 + row + x.seq.shift);
            bool stop = false;
            for (int j = 0; j < x.tiles; ++j, ++gk) {
                int key0, end;
                win::tile(x.y, j, key0, end);
                const int b = j & 1;
                if (!wait_bar_warp(bar(B_S_FULL + b), (b ? ns[1] : ns[0]) & 1, abort, hdr, 252)) { stop = true; break; }
                if (b) ++ns[1]; else ++ns[0];
                if (!wait_bar_warp(bar(B_DP_FULL), gt & 1, abort, hdr, 253)) { stop = true; break; }
                tc_fence_after();
                const uint32_t s_addr = lane_addr + col_s(b) + 64 * wg, p_addr = lane_addr + kColDP + 64 * wg;
                const int k0 = key0 + 64 * wg;
                const int nsk = min(vis.s, end) - k0, lo = vis.lo - k0, hi = min(vis.hi, end) - k0;
                if (!__all_sync(0xffffffffu, !live || nsk >= 64 || (lo <= 0 && hi >= 64))) {
                    // masked scores and their dP (which a key past the lengths may have made NaN), in TMEM
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t keep = win::bits(0, nsk - 32 * w) | win::bits(lo - 32 * w, hi - 32 * w);
                        mask_cols(s_addr + 32 * w, keep, kMinusInf);
                        mask_cols(p_addr + 32 * w, keep, 0u);
                    }
                    tmem_wait_st();
                }
                uint32_t s[64], p[64];
                tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                tmem_ld32(p_addr, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
                tmem_ld32(p_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&p[32]));
                tmem_wait_ld_regs(s);
                tmem_wait_ld_regs(p);
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float d0 = ex2(fmaf(__uint_as_float(s[2 * c]), sl2, -lse2)) * (__uint_as_float(p[2 * c]) - drow);
                    const float d1 = ex2(fmaf(__uint_as_float(s[2 * c + 1]), sl2, -lse2)) * (__uint_as_float(p[2 * c + 1]) - drow);
                    pk[c] = pack_bf16(d0, d1);
                }
                tmem_st32(s_addr, pk);
                if (end - key0 < 128) {  // K rows past the tile's keys: zeros (S has read them)
                    if (wg == 0 && row >= end - key0) {
                        const uint32_t kr = sK + (gk % 3) * C::kTileBytes + row * 128;
#pragma unroll
                        for (int i = 0; i < C::kSlabs * 8; ++i)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(kr + (i >> 3) * C::kSlabBytes + (i & 7) * 16),
                                         "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_DS_FULL));
                ++gt;
            }
            if (stop) break;
            // dq_t = scale * accumulator; this warpgroup's half of the columns
            if (x.tiles > 0) {
                if (!wait_bar_warp(bar(B_DQ_DONE), nu & 1, abort, hdr, 254)) break;
                ++nu;
                tc_fence_after();
            }
            constexpr int HC = D / 2;
            __nv_bfloat16* dst = dQ + rowg * D + wg * HC;
#pragma unroll
            for (int c0 = 0; c0 < HC; c0 += 32) {
                uint32_t o[32];
                if (x.tiles > 0) {
                    tmem_ld32(lane_addr + kColDQ + wg * HC + c0, o);
                    tmem_wait_ld_regs(o);
                }
                if (live) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = x.tiles > 0 ? pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * a.scale,
                                                           __uint_as_float(o[8 * i + 2 * e + 1]) * a.scale)
                                               : 0u;
                        *reinterpret_cast<uint4*>(dst + c0 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace dq

// ---- dK, dV --------------------------------------------------------------------
// One CTA per SM, 512 threads. TMEM: S^T and dP^T (128 keys x 128 rows) and the dV
// and dK accumulators.
//   warp 12 (one lane): units and TMA of a unit's K and V tiles (loaded once the
//          previous unit's last S^T and dP^T have read theirs).
//   warps 8-11: copy each 128-row tile's Q and dO (16-byte pieces into the swizzled
//          layout, zeros past the last row) and its lse and D into a 2-stage ring.
//   warp 13 (one lane): S^T = K Q^T, dP^T = V dO^T, then dV += P^T dO and
//          dK += dS^T Q with P^T and dS^T from TMEM.
//   warps 0-7: two warpgroups, each 64 of the tile's rows for all 128 keys (one
//          thread a key): P^T and dS^T as bf16 over its own halves of S^T and dP^T.
namespace dkv {

constexpr int kThreads = 512;
// launched at 128 registers a thread: 2 x 128 x 176 + 128 x 104 + 128 x 56 = 512 x 128
constexpr int kRegsCompute = 176, kRegsGather = 104, kRegsOther = 56;
constexpr uint32_t kColST = 0, kColDPT = 128, kColDV = 256, kColDK = 384;

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int oK = 0;
    static constexpr int oV = oK + kTileBytes;
    static constexpr int oQ = oV + kTileBytes;          // 2 stages
    static constexpr int oDO = oQ + 2 * kTileBytes;     // 2 stages
    static constexpr int oStat = oDO + 2 * kTileBytes;  // [2 stages][lse2 | D][128] fp32
    static constexpr int oBar = oStat + 2 * 2 * 128 * 4;
    static constexpr int kSmem = (oBar + 512 + 1024) > 120 * 1024 ? (oBar + 512 + 1024) : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr uint32_t kIdescSS = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, 1);
};

enum {
    B_ITEM_FULL = 0, B_ITEM_EMPTY = 2, B_KV_FULL = 4, B_KV_EMPTY = 5, B_QT_FULL = 6, B_QT_EMPTY = 8, B_ST_FULL = 10,
    B_P_FULL = 11, B_ACC_DONE = 12, B_MMA_DONE = 13, B_COUNT = 14
};

// A unit: a key tile of a (batch, key head), all of its row tiles or one split of them.
struct Unit {
    int b, hk, k0, nk;     // nk <= 0: no keys
    int t_lo, t_hi;        // rows of a query head that may see it
    int per_head;          // their 128-row tiles
    int i0, i1;            // this unit's tiles, counted over the heads of the group
    int part;              // split: index of the fp32 part, else -1
    win::Seq seq;
};

__device__ __forceinline__ void decode(const WinArgs& a, const WinBwdPlan& p, int u, Unit& x) {
    const int heads = a.B * a.Hk, lead = p.split_tiles * p.splits * heads;
    int kt, bh, split = 0;
    x.part = -1;
    if (u < lead) {  // the first keys' tiles: the longest units
        split = u % p.splits;
        bh = (u / p.splits) % heads;
        kt = u / p.splits / heads;
        if (p.splits > 1) x.part = u;
    } else {
        kt = p.split_tiles + (u - lead) / heads;
        bh = (u - lead) % heads;
    }
    x.b = bh / a.Hk;
    x.hk = bh - x.b * a.Hk;
    x.k0 = kt * kTile;
    x.seq = win::seq(a, x.b);
    x.nk = min(kTile, x.seq.n - x.k0);
    x.t_lo = x.t_hi = x.per_head = x.i0 = x.i1 = 0;
    if (x.nk <= 0) return;
    const bool first = x.k0 < a.sinks;
    int p_lo = first ? -(1 << 30) : x.k0 - a.right;
    if (a.causal) p_lo = max(p_lo, x.k0);
    const int p_hi = first ? (1 << 30) : x.k0 + x.nk - 1 + a.left;  // last position
    x.t_lo = max(p_lo - x.seq.shift, 0);
    x.t_hi = min(p_hi - x.seq.shift + 1, x.seq.m);
    if (x.t_hi <= x.t_lo) return;
    x.per_head = (x.t_hi - x.t_lo + kTile - 1) / kTile;
    const int total = x.per_head * a.group;
    const int splits = x.part >= 0 ? p.splits : 1;
    x.i0 = int(int64_t(total) * split / splits);
    x.i1 = int(int64_t(total) * (split + 1) / splits);
}
// Row tile i of a unit: query head, first row, rows.
__device__ __forceinline__ void row_tile(const WinArgs& a, const Unit& x, int i, int& hq, int& t0, int& n) {
    const int g = i / x.per_head;
    hq = x.hk * a.group + g;
    t0 = x.t_lo + (i - g * x.per_head) * kTile;
    n = min(kTile, x.t_hi - t0);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ WinArgs a, const __grid_constant__ WinBwdPlan p, int n_units,
                      const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ dO,
                      const float* __restrict__ lse, const float* __restrict__ Dsum, int32_t* __restrict__ work,
                      int32_t* __restrict__ hdr, float* __restrict__ parts, __nv_bfloat16* __restrict__ dK,
                      __nv_bfloat16* __restrict__ dV) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t sK = base + C::oK, sV = base + C::oV, sQ = base + C::oQ, sDO = base + C::oDO;
    float* stat = reinterpret_cast<float*>(gbase + C::oStat);  // [stage][0: lse2, 1: D][128]
    const uint32_t sBar = base + C::oBar;
    Shared& sh = *reinterpret_cast<Shared*>(gbase + C::oBar + 256);
    volatile int* abort = &sh.abort;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) {
            int n = 1;
            if (x == B_ITEM_EMPTY || x == B_ITEM_EMPTY + 1) n = 1 + 256 + 128;
            if (x == B_QT_FULL || x == B_QT_FULL + 1) n = 128;
            if (x == B_P_FULL) n = 256;
            mbar_init(bar(x), n);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(smem_u32(&sh.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;

    if (warp >= 12) {
        regs_dec<kRegsOther>();
        if (warp == 12 && lane == 0) {
            // ---------------------------------------------------------- units + K/V loads
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            uint32_t nu = 0;
            for (int it = 0;; ++it) {
                const int slot = it & 1;
                if (!wait_bar(bar(B_ITEM_EMPTY + slot), ((it >> 1) & 1) ^ 1, abort, hdr, 261)) break;
                const int u = atomicAdd(work, 1);
                sh.item[slot] = u < n_units ? u : -1;
                mbar_arrive(bar(B_ITEM_FULL + slot));
                if (u >= n_units) break;
                Unit x;
                decode(a, p, u, x);
                if (x.i0 >= x.i1) continue;
                if (!wait_bar(bar(B_KV_EMPTY), (nu & 1) ^ 1, abort, hdr, 262)) break;
                ++nu;
                mbar_expect_tx(bar(B_KV_FULL), 2 * C::kTileBytes);
                const int krow = (x.b * a.Hk + x.hk) * a.Lk + x.k0;
#pragma unroll
                for (int s = 0; s < C::kSlabs; ++s) {
                    tma_load_2d(sK + s * C::kSlabBytes, &tmK, bar(B_KV_FULL), 64 * s, krow);
                    tma_load_2d(sV + s * C::kSlabBytes, &tmV, bar(B_KV_FULL), 64 * s, krow);
                }
            }
            if (nu > 0) drain_bar(bar(B_KV_FULL), (nu - 1) & 1, hdr, 263);
        } else if (warp == 13 && lane == 0) {
            // ---------------------------------------------------------- MMA issue
            uint32_t gq = 0, nu = 0;
            bool stop = false;
            for (int it = 0; !stop; ++it) {
                const int slot = it & 1;
                if (!wait_bar(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 264)) break;
                const int u = sh.item[slot];
                mbar_arrive(bar(B_ITEM_EMPTY + slot));
                if (u < 0) break;
                Unit x;
                decode(a, p, u, x);
                if (x.i0 >= x.i1) continue;
                if (!wait_bar(bar(B_KV_FULL), nu & 1, abort, hdr, 265)) break;
                ++nu;
                tc_fence_after();
                for (int i = x.i0; i < x.i1; ++i, ++gq) {
                    const uint32_t st = gq & 1;
                    if (!wait_bar(bar(B_QT_FULL + st), (gq >> 1) & 1, abort, hdr, 266)) { stop = true; break; }
                    tc_fence_after();
                    const uint32_t qb = sQ + st * C::kTileBytes, gb = sDO + st * C::kTileBytes;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + kColST, sdesc_sw128(sK + off, 16, 1024), sdesc_sw128(qb + off, 16, 1024),
                                C::kIdescSS, kk > 0);
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + kColDPT, sdesc_sw128(sV + off, 16, 1024), sdesc_sw128(gb + off, 16, 1024),
                                C::kIdescSS, kk > 0);
                    }
                    umma_commit(bar(B_ST_FULL));
                    if (i + 1 == x.i1) umma_commit(bar(B_KV_EMPTY));
                    if (!wait_bar(bar(B_P_FULL), gq & 1, abort, hdr, 267)) { stop = true; break; }
                    tc_fence_after();
                    // rows 16 kk .. + 15 of P^T / dS^T: warpgroup kk / 4 wrote its 64 rows over the
                    // first 32 columns of its own half
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t ac = 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3);
                        umma_ts(tmem + kColDV, tmem + kColST + ac, sdesc_sw128(gb + kk * 2048, C::kSlabBytes, 1024),
                                C::kIdescAcc, (i > x.i0 || kk > 0));
                    }
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t ac = 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3);
                        umma_ts(tmem + kColDK, tmem + kColDPT + ac, sdesc_sw128(qb + kk * 2048, C::kSlabBytes, 1024),
                                C::kIdescAcc, (i > x.i0 || kk > 0));
                    }
                    umma_commit(bar(B_QT_EMPTY + st));
                }
                if (stop) break;
                umma_commit(bar(B_ACC_DONE));
            }
            umma_commit(bar(B_MMA_DONE));
            drain_bar(bar(B_MMA_DONE), 0, hdr, 268);
        }
        __syncwarp();
    } else if (warp >= 8) {
        regs_dec<kRegsGather>();
        // -------------------------------------------------------------- row tiles (warps 8-11)
        const int r = tid - 256, wr = (warp - 8) * 32;
        constexpr int CH = D / 8;  // 16-byte pieces a row
        uint32_t gq = 0;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 271)) break;
            const int u = sh.item[slot];
            mbar_arrive(bar(B_ITEM_EMPTY + slot));
            if (u < 0) break;
            Unit x;
            decode(a, p, u, x);
            bool stop = false;
            for (int i = x.i0; i < x.i1; ++i, ++gq) {
                int hq, t0, n;
                row_tile(a, x, i, hq, t0, n);
                const uint32_t st = gq & 1;
                if (!wait_bar_warp(bar(B_QT_EMPTY + st), ((gq >> 1) & 1) ^ 1, abort, hdr, 272)) { stop = true; break; }
                const size_t row0 = (size_t(x.b) * a.Hq + hq) * size_t(a.Lq) + t0;
                float l2 = INFINITY, dd = 0.f;  // +inf: every p of the row is zero
                if (r < n) {
                    const float v = __ldg(lse + row0 + r);
                    if (v > -INFINITY || v != v) l2 = v * kLog2e;
                    dd = __ldg(Dsum + row0 + r);
                }
                stat[(st * 2 + 0) * 128 + r] = l2;
                stat[(st * 2 + 1) * 128 + r] = dd;
#pragma unroll
                for (int i2 = 0; i2 < CH; ++i2) {
                    const int idx = i2 * 32 + lane;
                    const int rr = wr + idx / CH, ch = idx % CH;
                    const uint32_t off = (ch >> 3) * C::kSlabBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
                    const size_t src = (row0 + (rr < n ? rr : 0)) * D + ch * 8;
                    cp_async16(sQ + st * C::kTileBytes + off, Q + src, rr < n ? 16 : 0);
                    cp_async16(sDO + st * C::kTileBytes + off, dO + src, rr < n ? 16 : 0);
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                mbar_arrive(bar(B_QT_FULL + st));
            }
            if (stop) break;
        }
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- compute (warps 0-7)
        const int wg = warp >> 2, row = tid & 127;  // rows [64 wg, + 64) of the tile; key of the tile
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const float sl2 = a.scale * kLog2e;
        uint32_t gq = 0, nu = 0;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 273)) break;
            const int u = sh.item[slot];
            mbar_arrive(bar(B_ITEM_EMPTY + slot));
            if (u < 0) break;
            Unit x;
            decode(a, p, u, x);
            if (x.nk <= 0 && x.part < 0) continue;
            // positions that see this thread's key: [v_lo, v_hi)
            const int key = x.k0 + row;
            int v_lo = key < a.sinks ? -(1 << 30) : key - a.right;
            if (a.causal) v_lo = max(v_lo, key);
            const int v_hi = key < a.sinks ? (1 << 30) : key + a.left + 1;
            bool stop = false;
            for (int i = x.i0; i < x.i1; ++i, ++gq) {
                int hq, t0, n;
                row_tile(a, x, i, hq, t0, n);
                const uint32_t st = gq & 1;
                if (!wait_bar_warp(bar(B_QT_FULL + st), (gq >> 1) & 1, abort, hdr, 274)) { stop = true; break; }
                if (!wait_bar_warp(bar(B_ST_FULL), gq & 1, abort, hdr, 275)) { stop = true; break; }
                tc_fence_after();
                const float* l2 = stat + (st * 2 + 0) * 128 + 64 * wg;
                const float* dd = stat + (st * 2 + 1) * 128 + 64 * wg;
                const uint32_t s_addr = lane_addr + kColST + 64 * wg, g_addr = lane_addr + kColDPT + 64 * wg;
                const int p0 = t0 + x.seq.shift + 64 * wg;
                const int lo = v_lo - p0, hi = v_hi - p0;
                if (!__all_sync(0xffffffffu, row >= x.nk || (lo <= 0 && hi >= 64))) {
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) mask_cols(s_addr + 32 * w, win::bits(lo - 32 * w, hi - 32 * w), kMinusInf);
                    tmem_wait_st();
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t s[32], g[32];
                    tmem_ld32(s_addr + 32 * c, s);
                    tmem_ld32(g_addr + 32 * c, g);
                    tmem_wait_ld_regs(s);
                    tmem_wait_ld_regs(g);
                    uint32_t pp[16], pd[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int q0 = 32 * c + 2 * e;
                        const float p0f = ex2(fmaf(__uint_as_float(s[2 * e]), sl2, -l2[q0]));
                        const float p1f = ex2(fmaf(__uint_as_float(s[2 * e + 1]), sl2, -l2[q0 + 1]));
                        pp[e] = pack_bf16(p0f, p1f);
                        pd[e] = pack_bf16(p0f * (__uint_as_float(g[2 * e]) - dd[q0]), p1f * (__uint_as_float(g[2 * e + 1]) - dd[q0 + 1]));
                    }
                    tmem_st16(s_addr + 16 * c, pp);
                    tmem_st16(g_addr + 16 * c, pd);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_P_FULL));
            }
            if (stop) break;
            // this warpgroup's half of the columns of dV and dK for its key rows
            const bool some = x.i0 < x.i1;
            if (some) {
                if (!wait_bar_warp(bar(B_ACC_DONE), nu & 1, abort, hdr, 276)) break;
                ++nu;
                tc_fence_after();
            }
            constexpr int HC = D / 2;
            const bool valid = row < x.nk;
            const size_t orow = ((size_t(x.b) * a.Hk + x.hk) * size_t(a.Lk) + size_t(x.k0) + row) * D + wg * HC;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                __nv_bfloat16* out = t == 0 ? dV : dK;
                const float mul = t == 0 ? 1.f : a.scale;
#pragma unroll
                for (int c0 = 0; c0 < HC; c0 += 32) {
                    uint32_t o[32];
                    if (some) {
                        tmem_ld32(lane_addr + (t == 0 ? kColDV : kColDK) + wg * HC + c0, o);
                        tmem_wait_ld_regs(o);
                    }
                    if (x.part >= 0) {
                        float* dst = parts + ((size_t(x.part) * 2 + t) * 128 + row) * D + wg * HC + c0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (some && valid)
                                v = make_float4(__uint_as_float(o[4 * i]) * mul, __uint_as_float(o[4 * i + 1]) * mul,
                                                __uint_as_float(o[4 * i + 2]) * mul, __uint_as_float(o[4 * i + 3]) * mul);
                            reinterpret_cast<float4*>(dst)[i] = v;
                        }
                    } else if (valid) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = some ? pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * mul, __uint_as_float(o[8 * i + 2 * e + 1]) * mul) : 0u;
                            *reinterpret_cast<uint4*>(out + orow + c0 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The split tiles' dV and dK: their parts added in order. A thread owns four columns
// of a key.
template <int D>
__global__ void __launch_bounds__(256) window_dkv_join_kernel(const __grid_constant__ WinArgs a,
                                                              const __grid_constant__ WinBwdPlan p,
                                                              const float* __restrict__ parts,
                                                              __nv_bfloat16* __restrict__ dK,
                                                              __nv_bfloat16* __restrict__ dV) {
    constexpr int PER = D / 4;
    const int heads = a.B * a.Hk;
    const int64_t total = int64_t(p.split_tiles) * heads * 2 * 128 * PER;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
        const int c = int(i % PER), r = int(i / PER % 128), t = int(i / PER / 128 % 2);
        const int64_t tile = i / PER / 128 / 2;  // key tile x heads + (batch, key head)
        const int kt = int(tile / heads), bh = int(tile % heads), key = kt * kTile + r;
        if (key >= win::seq(a, bh / a.Hk).n) continue;
        const float4* src = reinterpret_cast<const float4*>(parts + ((tile * p.splits * 2 + t) * 128 + r) * D) + c;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < p.splits; ++k) {
            const float4 v = src[size_t(k) * (2 * 128 * PER)];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        __nv_bfloat16* out = (t == 0 ? dV : dK) + (size_t(bh) * a.Lk + key) * D + c * 4;
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
}

}  // namespace dkv

int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

template <int D>
cudaError_t launch_d(const WinArgs& a, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                     const void* dO, void* dQ, void* dK, void* dV, char* ws, const WinBwdPlan& p, cudaStream_t s) {
    int32_t* hdr = nullptr;
    cudaError_t e = window_error_word(&hdr);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    const int64_t qrows = int64_t(a.B) * a.Hq * a.Lq, krows = int64_t(a.B) * a.Hk * a.Lk;
    int32_t* work = reinterpret_cast<int32_t*>(ws + p.work);
    float* dsum = reinterpret_cast<float*>(ws + p.dsum);
    float* parts = reinterpret_cast<float*>(ws + p.part);
    const auto* q = static_cast<const __nv_bfloat16*>(Q);
    const auto* g = static_cast<const __nv_bfloat16*>(dO);
    const int64_t want = (qrows * (D / 8) + 255) / 256, most = int64_t(sms) * 16;
    window_rowdot_kernel<D><<<int(want < 1 ? 1 : want < most ? want : most), 256, 0, s>>>(
        a, static_cast<const __nv_bfloat16*>(O), g, dsum, work);
    CUtensorMap tmQ, tmDO, tmK, tmV;
    if (krows > 0) {
        if (!make_tmap(&tmK, K, D, krows) || !make_tmap(&tmV, V, D, krows)) return cudaErrorInvalidValue;
    }
    if (qrows > 0) {
        if (!make_tmap(&tmQ, Q, D, qrows) || !make_tmap(&tmDO, dO, D, qrows)) return cudaErrorInvalidValue;
        if (krows == 0) tmK = tmV = tmQ;  // no key tile is loaded
        const int smem = dq::Cfg<D>::kSmem;
        e = cudaFuncSetAttribute(dq::window_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int nqt = (a.Lq + kTile - 1) / kTile, n = a.B * a.Hq * nqt;
        dq::window_dq_kernel<D><<<n < sms ? n : sms, dq::kThreads, smem, s>>>(
            tmQ, tmDO, tmK, tmV, a, n, nqt, lse, dsum, work, hdr, static_cast<__nv_bfloat16*>(dQ));
    }
    if (krows > 0) {
        const int smem = dkv::Cfg<D>::kSmem;
        e = cudaFuncSetAttribute(dkv::window_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int heads = a.B * a.Hk;
        const int n = heads * (p.key_tiles - p.split_tiles + p.split_tiles * p.splits);
        dkv::window_dkv_kernel<D><<<n < sms ? n : sms, dkv::kThreads, smem, s>>>(
            tmK, tmV, a, p, n, q, g, lse, dsum, work + 1, hdr, parts, static_cast<__nv_bfloat16*>(dK),
            static_cast<__nv_bfloat16*>(dV));
        if (p.splits > 1) {
            const int64_t blocks = (int64_t(p.split_tiles) * heads * 2 * 128 * (D / 4) + 255) / 256;
            dkv::window_dkv_join_kernel<D><<<int(blocks < most ? blocks : most), 256, 0, s>>>(
                a, p, parts, static_cast<__nv_bfloat16*>(dK), static_cast<__nv_bfloat16*>(dV));
        }
    }
    return cudaGetLastError();
}

}  // namespace

WinBwdPlan plan_window_bwd(const WinArgs& a, int d) {
    WinBwdPlan p;
    auto align = [](size_t x) { return (x + 255) & ~size_t(255); };
    p.work = 0;
    p.dsum = 256;
    p.part = p.dsum + align(size_t(a.B) * a.Hq * a.Lq * sizeof(float));
    p.key_tiles = (a.Lk + kTile - 1) / kTile;
    const int sink_tiles = (a.sinks + kTile - 1) / kTile;
    p.split_tiles = sink_tiles < p.key_tiles ? sink_tiles : p.key_tiles;
    // The first keys' tiles walk every row, the others the rows of one window. Split
    // into about the others' length, but into no more units than four an SM: a unit
    // costs its fp32 part (128 KB at d = 128, written and read once).
    const int64_t heads = int64_t(a.B) * a.Hk;
    if (p.split_tiles > 0 && heads > 0 && a.Lq > 0) {
        const int64_t all = (a.Lq + kTile - 1) / kTile;
        const int64_t reach = (a.left == kWinOpen ? a.Lq : a.left) + (a.causal ? 0 : a.right == kWinOpen ? a.Lq : a.right);
        const int64_t near = (reach + kTile - 1) / kTile + 1;
        int64_t n = (all + near - 1) / near;
        const int64_t cap = (4 * int64_t(sm_count()) + p.split_tiles * heads - 1) / (p.split_tiles * heads);
        if (n > cap) n = cap;
        p.splits = int(n < 1 ? 1 : n);
    }
    const size_t parts = p.splits > 1 ? size_t(p.split_tiles) * size_t(heads) * p.splits : 0;
    p.total = p.part + align(parts * 2 * 128 * size_t(d) * sizeof(float));
    return p;
}

cudaError_t launch_window_bwd(const WinArgs& a, int d, const void* Q, const void* K, const void* V, const void* O,
                              const float* lse, const void* dO, void* dQ, void* dK, void* dV, char* ws,
                              const WinBwdPlan& p, cudaStream_t s) {
    if (d == 128) return launch_d<128>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s);
    return launch_d<64>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s);
}

}  // namespace moc
