// Sliding-window attention with always-visible first keys, backward, on the
// 5th-generation tensor cores. With p_tu = exp(scale q_t . k_u - lse_t) over the
// row's visible keys (window.cuh), D_t = dO_t . o_t and
// ds_tu = p_tu (dO_t . v_u - D_t):
//   dq_t = scale sum_u ds_tu k_u,
//   dk_u = scale sum_t ds_tu q_t,   dv_u = sum_t p_tu dO_t,
// the sums over t also over the query heads that share u's key head. p and ds are
// rounded to bf16 (2^-8 of each) as operands of the last products; all sums are in
// fp32. Where a query head has no more than kFineRows rows, the rest of p and ds goes
// into the products as a second bf16 (2^-16 of each is lost): few terms average
// nothing out (kFineRows has what was measured).
//
// Launches: one that forms each row's statistics (the log-sum-exp in exp2 units and
// D) and clears the work counters; dQ (a work unit is a 128-row tile, it owns its dQ
// rows); dK / dV (a unit is a 128-key tile of a key head, it owns its dK and dV rows
// and walks the rows that see it). The first keys are seen by every later row: their
// tiles' rows are split over units that write fp32 parts, added in order by a fourth
// launch. No atomics on results: they do not depend on the order of the units, which
// are handed out longest first by a counter.
//
// Training step of the single-shot clip (causal over 6,239 keys and 512 first ones): dQ
// 1.6 ms and dK / dV 2.0 ms, 1.16 and 1.25 PFLOP/s of executed products (6 d and 8 d a
// pair), at the 1 kW power cap.
//
// D from the rounded O is off by what O's rounding carries, which a row of few keys
// feels as much as the roundings of p and ds. As sum_u ds_tu = 0 for the exact D, the
// dQ kernel adds the sum r of its unrounded ds to D for the dK / dV kernel, and walks
// units of at most kProbeKeys keys twice, the first time for r alone (two of their
// three products again; such units are short). That holds where O and lse are those of
// exactly this call's keys: with a.joined they are not, and D is dO . O.
#include <type_traits>

#include "common.cuh"
#include "pipeline.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace moc {
namespace {

using namespace sm100;
using win::kRegsCompute;
using win::kRegsOther;
using win::kThreads;
using win::kTile;

constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kProbeKeys = 384;
// Three products more for 7 in units of few tiles, whose chains hide most of them (8 x 48
// heads of 64 rows and keys: 229 against 212 us; 3 rows of 12 heads: 39 against 36).
// Errors against fp64 over 700 drawn problems, as multiples of the plain form's: up to
// 1.89 at 2 rows, 1.69 at 8, 1.55 at 32, 1.53 at 64, 1.46 at 128 without it; up to 1.02
// with it.
constexpr int kFineRows = 64;

// What two bf16 of a packed pair leave of (x, y), as bf16.
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t pk) {
    return pack_bf16(x - bf16lo(pk), y - bf16hi(pk));
}

// Halves of a packed pair to keep: the low one for bit i of `bits`, the high one for bit i + 1.
__device__ __forceinline__ uint32_t pair_mask(uint32_t bits, int i) {
    uint32_t m;  // bytes 3 of the shifted words, their sign over 16 bits each
    asm("prmt.b32 %0, %1, %2, 0xffbb;" : "=r"(m) : "r"(bits << (31 - i)), "r"(bits << (30 - i)));
    return m;
}

// Row statistics, negated for the sums they enter: - log2 sum exp2 of the scores and
// - D, rows of a head padded to a multiple of four (16-byte copies from any fourth row)
// and 128 more at the end; -inf and 0 where there is no row or the row sees no key, so
// that every p of it is zero.
__host__ __device__ __forceinline__ int64_t stat_rows(int Lq) { return (int64_t(Lq) + 3) & ~int64_t(3); }

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

// ---- row statistics ------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) window_stats_kernel(const __grid_constant__ WinArgs a,
                                                           const __nv_bfloat16* O, const __nv_bfloat16* dO,
                                                           const float* lse, float* nl2, float* nd, int32_t* work) {
    constexpr int LPR = D / 8, RPC = 256 / LPR;  // lanes a row (16 bytes each), rows a step
    let_next_kernel_start();
    wait_for_previous_kernel();
    if (blockIdx.x == 0 && threadIdx.x < 2) work[threadIdx.x] = 0;
    const int per = int(stat_rows(a.Lq));
    const int64_t heads = int64_t(a.B) * a.Hq, total = heads * per + 128;
    const int r = threadIdx.x % LPR;
    for (int64_t i0 = int64_t(blockIdx.x) * RPC; i0 < total; i0 += int64_t(gridDim.x) * RPC) {
        const int64_t i = i0 + threadIdx.x / LPR;
        const int64_t head = per > 0 ? i / per : heads;
        const int t = int(i - head * per);
        float acc = 0.f, l2 = -INFINITY;
        if (head < heads && t < win::seq(a, int(head / a.Hq)).m) {
            const size_t row = size_t(head) * a.Lq + t;
            uint32_t xs[4], ys[4];
            ld16(O + row * D + r * 8, xs);
            ld16(dO + row * D + r * 8, ys);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc = fmaf(bf16lo(xs[k]), bf16lo(ys[k]), acc);
                acc = fmaf(bf16hi(xs[k]), bf16hi(ys[k]), acc);
            }
            const float v = lse[row];
            if (v > -INFINITY || v != v) l2 = -v * kLog2e;
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o, LPR);
        if (r == 0 && i < total) {
            nl2[i] = l2;
            nd[i] = l2 == -INFINITY ? 0.f : -acc;
        }
    }
}

// ---- dQ ------------------------------------------------------------------------
// One CTA per SM, 384 threads. TMEM: two S buffers, dP and the dQ accumulator.
//   warp 8 (one lane): units and TMA: Q and dO tiles, K tiles into a 3-stage ring (a
//          K tile serves S and, two tiles later, dQ), V tiles into a 2-stage ring.
//   warp 9 (one lane): S(j) = Q K(j)^T two tiles ahead, dP(j) = dO V(j)^T, and
//          dQ += dS(j) K(j) with dS from TMEM.
//   warps 0-7: two warpgroups, each half of a tile's keys for all 128 rows (one
//          thread a row): dS in fp32, written as bf16 over its own half of S (32 of the 64
//          columns; Fine: what that leaves of it over the other 32).
namespace dq {

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
    static constexpr int oSum = oV + 2 * kTileBytes;  // fp32 [2 exchanges][2 warpgroups][128]
    static constexpr int oBar = oSum + 2048;
    // the dynamic shared memory of a kernel without static shared memory starts on a
    // 1024-byte boundary (checked at the start): no room for slack at d = 128
    static constexpr int kSmem = oBar + 256 > 120 * 1024 ? oBar + 256 : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr uint32_t kIdescSS = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescDQ = idesc_bf16_f32(128, D, 1);
};

enum {
    B_ITEM_FULL = 0, B_ITEM_EMPTY = 2, B_K_FULL = 4, B_K_EMPTY = 7, B_V_FULL = 10, B_V_EMPTY = 12, B_QDO_FULL = 14,
    B_QDO_EMPTY = 15, B_S_FULL = 16, B_DP_FULL = 18, B_DS_FULL = 19, B_DQ_DONE = 21, B_MMA_DONE = 22, B_SUM = 23, B_DP_READ = 24, B_COUNT = 25
};
static_assert(B_COUNT * 8 + sizeof(Shared) <= 256, "barriers");

__device__ __forceinline__ uint32_t col_s(int b) { return b ? kColS1 : kColS0; }
// column (from a buffer's first) of the bf16 pairs of keys 16 kk .. + 15
__device__ __forceinline__ uint32_t ds_col(int kk) { return 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3); }

struct Unit : win::Item {
    int probe;  // tiles walked first for the sum of ds alone: `tiles` or 0
};
__device__ __forceinline__ void decode(const WinArgs& a, int nqt, int u, Unit& x) {
    win::decode(a, kTile, nqt, u, x);
    x.probe = !a.joined && x.y.a1 + x.y.b1 - x.y.b0 <= kProbeKeys ? x.tiles : 0;
}

template <int D, bool Fine>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ WinArgs a, int n_units, int nqt, const float* nl2, float* nd, int32_t* work,
                     int32_t* hdr, __nv_bfloat16* __restrict__ dQ) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {
        wait_for_previous_kernel();
        if (threadIdx.x == 0) set_error(hdr, ERR_CHECK, 230);
        return;
    }
    const uint32_t sQ = base + C::oQ, sDO = base + C::oDO, sK = base + C::oK, sV = base + C::oV;
    const uint32_t sBar = base + C::oBar;
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + C::oBar + 8 * B_COUNT);
    volatile int* abort = &sh.abort;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    let_next_kernel_start();

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) {
            int n = 1;
            if (x == B_ITEM_EMPTY || x == B_ITEM_EMPTY + 1) n = 1 + 256;
            if (x == B_DS_FULL || x == B_DS_FULL + 1 || x == B_SUM || x == B_DP_READ) n = 256;
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
    const uint32_t tmem = uint32_t(uniform(int(sh.tmem_base)));
    wait_for_previous_kernel();

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
                for (int j = 0; j < x.probe + x.tiles; ++j) {
                    int key0, end;
                    win::tile(x.y, j < x.probe ? j : j - x.probe, key0, end);
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
        } else if (warp == 9) {
            // ---------------------------------------------------------- MMA issue
            // the whole warp walks the tiles, one elected lane issues (uniform descriptors)
            const bool leader = elect_one();
            uint32_t gk = 0, gv = 0, gt = 0, nu = 0;
            bool stop = false;
            auto issue_s = [&](uint32_t kt, int b) -> bool {  // S(b) = Q K(kt)^T
                const uint32_t ks = kt % 3;
                if (!wait_bar_warp(bar(B_K_FULL + ks), (kt / 3) & 1, abort, hdr, 241)) return false;
                tc_fence_after();
                const uint32_t kb = sK + ks * C::kTileBytes;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + col_s(b), sdesc_sw128(sQ + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024),
                                C::kIdescSS, kk > 0);
                    }
                    umma_commit(bar(B_S_FULL + b));
                }
                __syncwarp();
                return true;
            };
            auto issue_dp = [&]() -> bool {  // dP = dO V(gv)^T, then V(gv) is free
                const uint32_t vs = gv & 1;
                if (!wait_bar_warp(bar(B_V_FULL + vs), (gv >> 1) & 1, abort, hdr, 242)) return false;
                tc_fence_after();
                const uint32_t vb = sV + vs * C::kTileBytes;
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + kColDP, sdesc_sw128(sDO + off, 16, 1024), sdesc_sw128(vb + off, 16, 1024),
                                C::kIdescSS, kk > 0);
                    }
                    umma_commit(bar(B_DP_FULL));
                    umma_commit(bar(B_V_EMPTY + vs));
                }
                __syncwarp();
                ++gv;
                return true;
            };
            for (int it = 0; !stop; ++it) {
                const int slot = it & 1;
                if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 243)) break;
                const int u = uniform(sh.item[slot]);
                if (leader) mbar_arrive(bar(B_ITEM_EMPTY + slot));
                __syncwarp();
                if (u < 0) break;
                Unit x;
                decode(a, nqt, u, x);
                const int probe = uniform(x.probe), T = uniform(x.probe + x.tiles);
                if (T == 0) continue;
                if (!wait_bar_warp(bar(B_QDO_FULL), nu & 1, abort, hdr, 244)) break;
                ++nu;
                tc_fence_after();
                if (!issue_s(gk, 0) || !issue_dp() || (T > 1 && !issue_s(gk + 1, 1))) break;
                if (T == 1 && leader) umma_commit(bar(B_QDO_EMPTY));
                __syncwarp();
                for (int j = 0; j < T; ++j) {
                    // dP(j) is in the warps' registers: dP(j + 1) runs while they form dS(j)
                    if (!wait_bar_warp(bar(B_DP_READ), gt & 1, abort, hdr, 247)) { stop = true; break; }
                    tc_fence_after();
                    if (j + 1 < T && !issue_dp()) { stop = true; break; }
                    if (T > 1 && j == T - 2 && leader) umma_commit(bar(B_QDO_EMPTY));  // the last S was issued before it
                    if (!wait_bar_warp(bar(B_DS_FULL + (gt & 1)), (gt >> 1) & 1, abort, hdr, 245)) { stop = true; break; }
                    tc_fence_after();
                    ++gt;
                    const uint32_t ks = (gk + j) % 3, kb = sK + ks * C::kTileBytes;
                    if (leader) {
                        if (j >= probe) {
                            const uint32_t acc = j > probe ? 1u : 0u, sc = tmem + col_s(j & 1);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_ts(tmem + kColDQ, sc + ds_col(kk), sdesc_sw128(kb + kk * 2048, C::kSlabBytes, 1024),
                                        C::kIdescDQ, kk > 0 ? 1u : acc);
                            if constexpr (Fine) {
#pragma unroll
                                for (int kk = 0; kk < 8; ++kk)
                                    umma_ts(tmem + kColDQ, sc + 32 + ds_col(kk), sdesc_sw128(kb + kk * 2048, C::kSlabBytes, 1024),
                                            C::kIdescDQ, 1u);
                            }
                        }
                        umma_commit(bar(B_K_EMPTY + ks));
                    }
                    __syncwarp();
                    if (j + 2 < T && !issue_s(gk + j + 2, j & 1)) { stop = true; break; }
                }
                if (stop) break;
                gk += T;
                if (leader) umma_commit(bar(B_DQ_DONE));
                __syncwarp();
            }
            if (leader) {
                umma_commit(bar(B_MMA_DONE));
                drain_bar(bar(B_MMA_DONE), 0, hdr, 246);
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- compute (warps 0-7)
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const float sl2 = a.scale * kLog2e;
        const uint64_t sc2 = f2_pack(sl2, sl2);
        uint32_t gt = 0, nu = 0, ns[2] = {0, 0}, gk = 0, nx = 0;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 251)) break;
            const int u = sh.item[slot];
            mbar_arrive(bar(B_ITEM_EMPTY + slot));
            if (u < 0) break;
            Unit x;
            decode(a, nqt, u, x);
            const int rows_out = a.fill ? min(kTile, a.Lq - x.t0) : x.rows;  // with those past the last
            if (rows_out <= 0) continue;
            const bool live = row < x.rows;
            const size_t rowg = (size_t(x.b) * a.Hq + x.hq) * size_t(a.Lq) + size_t(x.t0) + row;
            const int64_t srow = (int64_t(x.b) * a.Hq + x.hq) * stat_rows(a.Lq) + x.t0 + row;
            const float l2 = live ? nl2[srow] : -INFINITY;
            float drow = live ? nd[srow] : 0.f;  // - D
            // takes from drow what the two warpgroups have for their halves of the row's keys;
            // exchanges alternate between two buffers, so that one's values are read before
            // the next but one overwrites them
            auto add_both = [&](float v) -> bool {
                float* sums = reinterpret_cast<float*>(smem_raw + C::oSum) + (nx & 1) * 256;
                sums[wg * 128 + row] = v;
                mbar_arrive(bar(B_SUM));
                if (!wait_bar_warp(bar(B_SUM), nx & 1, abort, hdr, 255)) return false;
                ++nx;
                drow -= sums[row] + sums[128 + row];
                return true;
            };
            uint64_t ra = 0, rb = 0;  // packed sums of the unrounded ds
            auto half_sum = [&]() -> float {
                float r0, r1, r2, r3;
                f2_unpack(ra, r0, r1);
                f2_unpack(rb, r2, r3);
                ra = rb = 0;
                return (r0 + r1) + (r2 + r3);
            };
            const win::Row vis = win::row(a, x.seq.n, x.t0 + row + x.seq.shift);
            bool stop = false;
            for (int j = 0; j < x.probe + x.tiles; ++j, ++gk) {
                int key0, end;
                win::tile(x.y, j < x.probe ? j : j - x.probe, key0, end);
                if (j > 0 && j == x.probe && !add_both(half_sum())) { stop = true; break; }
                const int b = j & 1;
                if (!wait_bar_warp(bar(B_S_FULL + b), (b ? ns[1] : ns[0]) & 1, abort, hdr, 252)) { stop = true; break; }
                if (b) ++ns[1]; else ++ns[0];
                tc_fence_after();
                const uint32_t s_addr = lane_addr + col_s(b) + 64 * wg, p_addr = lane_addr + kColDP + 64 * wg;
                const int k0 = key0 + 64 * wg;
                const int nsk = min(vis.s, end) - k0, lo = vis.lo - k0, hi = min(vis.hi, end) - k0;
                const bool masked = !__all_sync(0xffffffffu, !live || nsk >= 64 || (lo <= 0 && hi >= 64));
                if (masked) {
#pragma unroll 1
                    for (int w = 0; w < 2; ++w)
                        mask_cols(s_addr + 32 * w, win::bits(0, nsk - 32 * w) | win::bits(lo - 32 * w, hi - 32 * w), kMinusInf);
                    tmem_wait_st();
                }
                // p while dP is still being formed
                uint32_t s[64];
                tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                tmem_wait_ld_regs(s);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float p0, p1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sc2, f2_pack(l2, l2)), p0, p1);
                    s[2 * c] = __float_as_uint(ex2(p0));
                    s[2 * c + 1] = __float_as_uint(ex2(p1));
                }
                if (!wait_bar_warp(bar(B_DP_FULL), gt & 1, abort, hdr, 253)) { stop = true; break; }
                tc_fence_after();
                if (masked) {  // dP of a key past the lengths may be NaN
#pragma unroll 1
                    for (int w = 0; w < 2; ++w)
                        mask_cols(p_addr + 32 * w, win::bits(0, nsk - 32 * w) | win::bits(lo - 32 * w, hi - 32 * w), 0u);
                    tmem_wait_st();
                }
                uint32_t p[64], pk[32], rest[Fine ? 32 : 1];
                const uint64_t nd2 = f2_pack(drow, drow);
                tmem_ld32(p_addr, *reinterpret_cast<uint32_t(*)[32]>(&p[0]));
                tmem_ld32(p_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&p[32]));
                tmem_wait_ld_regs(p);
                tc_fence_before();
                mbar_arrive(bar(B_DP_READ));
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const uint64_t d = f2_mul(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])),
                                              f2_add(f2_pack(__uint_as_float(p[2 * c]), __uint_as_float(p[2 * c + 1])), nd2));
                    if (c & 1) rb = f2_add(rb, d);
                    else ra = f2_add(ra, d);
                    float d0, d1;
                    f2_unpack(d, d0, d1);
                    pk[c] = pack_bf16(d0, d1);
                    if constexpr (Fine) rest[c] = pack_rest(d0, d1, pk[c]);
                }
                tmem_st32(s_addr, pk);
                if constexpr (Fine) tmem_st32(s_addr + 32, rest);
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
                // a barrier for even tiles and one for odd: a warpgroup may be a tile ahead (its S
                // and dP need nothing of this tile's dS), and must not complete this tile's phase
                mbar_arrive(bar(B_DS_FULL + (gt & 1)));
                ++gt;
            }
            if (stop) break;
            // dq_t = scale * accumulator; this warpgroup's half of the columns
            if (x.tiles > 0) {
                if (!a.joined) {
                    if (!add_both(half_sum())) break;
                    if (wg == 0 && live && l2 != -INFINITY) nd[srow] = drow;
                }
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
                if (row < rows_out) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = x.tiles > 0 && live ? pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * a.scale,
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
// One CTA per SM, 384 threads, 128-row tiles. TMEM is full with S^T, dP^T (128 keys x
// 128 rows) and the dV and dK accumulators, so nothing can be double-buffered; the
// tensor core is kept busy by the order of its products instead:
//     dV(i-1) S^T(i) | dK(i-1) dP^T(i) | dV(i) S^T(i+1) | ...
// S^T(i) runs as soon as dV(i-1) has read P^T(i-1) in its columns, while ds(i-1) is
// formed; the exponentials of tile i run under dK(i-1) and dP^T(i). (All four products
// of a tile in a row, then its math: 2.80 ms on the single-shot training step against
// 1.97 ms; two TMEM buffers of 64 rows each: 3.14 ms, a 64-column product takes as
// long as a 128-column one.)
// At d = 64 the accumulators leave room for a second S^T: it runs a tile ahead (the
// odd padded batch: 43.6 against 45.1 us).
//   warp 8 (one lane): units and TMA: K and V of a unit, Q tiles into a 3-stage ring,
//          dO tiles and row statistics into a 2-stage ring.
//   warp 9 (one lane): the products.
//   warps 0-7: two warpgroups, each 64 of the tile's rows for all 128 keys (one thread
//          a key): P^T, then dS^T, as bf16 over its own halves of S^T and dP^T.
namespace dkv {

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int kQStages = 3, kOStages = 2;
    static constexpr int kStatBytes = kTile * 8;  // 128 of either statistic
    static constexpr int oK = 0;
    static constexpr int oV = oK + kTileBytes;
    static constexpr int oQ = oV + kTileBytes;
    static constexpr int oDO = oQ + kQStages * kTileBytes;
    static constexpr int oStat = oDO + kOStages * kTileBytes;  // [stage][- log-sum-exp | - D][row]
    static constexpr int oBar = oStat + kOStages * kStatBytes;
    // the dynamic shared memory of a kernel without static shared memory starts on a
    // 1024-byte boundary (checked at the start): no room for slack at d = 128
    static constexpr int kSmem = oBar + 256 > 120 * 1024 ? oBar + 256 : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    // TMEM columns. d = 64 leaves room for a second S^T.
    static constexpr bool kTwoS = D == 64;
    static constexpr uint32_t kColDPT = kTwoS ? 256 : 128, kColDV = kTwoS ? 384 : 256, kColDK = kTwoS ? 448 : 384;
    static __device__ __forceinline__ uint32_t col_st(uint32_t g) { return kTwoS && (g & 1) ? 128u : 0u; }
    static constexpr uint32_t kIdescSS = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescAcc = idesc_bf16_f32(128, D, 1);
};

enum {
    B_ITEM_FULL = 0, B_ITEM_EMPTY = 2, B_KV_FULL = 4, B_KV_EMPTY = 5, B_Q_FULL = 6, B_Q_EMPTY = 9, B_O_FULL = 12,
    B_O_EMPTY = 14, B_S_FULL = 16, B_P_FULL = 18, B_P_HALF = 20, B_DP_FULL = 22, B_DS_FULL = 23, B_ACC_DONE = 24,
    B_EPI_DONE = 25, B_MMA_DONE = 26, B_TAIL = 27, B_COUNT = 29
};
// S_FULL, P_HALF and P_FULL: one for even tiles and one for odd. With two S^T a
// warpgroup may be a tile ahead of the other, and must not complete its phase.
static_assert(B_COUNT * 8 + sizeof(Shared) <= 256, "barriers");

// A unit: a key tile of a (batch, key head), all of its row tiles or one split of them.
struct Unit {
    int b, hk, k0, nk;     // nk <= 0: no keys
    int t_lo, t_hi;        // rows of a query head that may see it, from a multiple of four
    int skip;              // rows at t_lo that come before the first that does
    int per_head;          // their tiles
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
    x.t_lo = x.t_hi = x.skip = x.per_head = x.i0 = x.i1 = 0;
    if (x.nk <= 0) return;
    const bool first = x.k0 < a.sinks;
    int p_lo = first ? -(1 << 30) : x.k0 - a.right;
    if (a.causal) p_lo = max(p_lo, x.k0);
    const int p_hi = first ? (1 << 30) : x.k0 + x.nk - 1 + a.left;  // last position
    const int t_first = max(p_lo - x.seq.shift, 0);
    x.t_lo = t_first & ~3;                                          // 16-byte copies of the statistics
    x.skip = t_first - x.t_lo;
    x.t_hi = min(p_hi - x.seq.shift + 1, x.seq.m);
    if (x.t_hi <= x.t_lo) return;
    x.per_head = (x.t_hi - x.t_lo + kTile - 1) / kTile;
    const int total = x.per_head * a.group;
    const int splits = x.part >= 0 ? p.splits : 1;
    x.i0 = int(int64_t(total) * split / splits);
    x.i1 = int(int64_t(total) * (split + 1) / splits);
}
// Walk over a unit's row tiles, the heads of the group one after the other.
struct RowWalk {
    int r, hq, t0;  // tile of the head, query head, first row
    __device__ __forceinline__ RowWalk(const WinArgs& a, const Unit& x) {
        const int g = x.i0 / max(x.per_head, 1);
        r = x.i0 - g * x.per_head;
        hq = x.hk * a.group + g;
        t0 = x.t_lo + r * kTile;
    }
    __device__ __forceinline__ int rows(const Unit& x) const { return min(kTile, x.t_hi - t0); }
    __device__ __forceinline__ void next(const Unit& x) {
        t0 += kTile;
        if (++r == x.per_head) {
            r = 0;
            t0 = x.t_lo;
            ++hq;
        }
    }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int D, bool Fine>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkv_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                      const __grid_constant__ WinArgs a, const __grid_constant__ WinBwdPlan p, int n_units,
                      const float* nl2, const float* nd, int32_t* work, int32_t* hdr, float* parts, __nv_bfloat16* __restrict__ dK, __nv_bfloat16* __restrict__ dV) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {
        wait_for_previous_kernel();
        if (threadIdx.x == 0) set_error(hdr, ERR_CHECK, 260);
        return;
    }
    const uint32_t sK = base + C::oK, sV = base + C::oV, sQ = base + C::oQ, sDO = base + C::oDO;
    const uint32_t sBar = base + C::oBar;
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + C::oBar + 8 * B_COUNT);
    volatile int* abort = &sh.abort;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    let_next_kernel_start();

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) {
            int n = 1;
            if (x == B_ITEM_EMPTY || x == B_ITEM_EMPTY + 1) n = 1 + 256;
            if (x == B_O_EMPTY || x == B_O_EMPTY + 1) n = 1 + 256;  // dV has read dO, the warps the statistics
            if ((x >= B_P_FULL && x < B_P_HALF + 2) || x == B_DS_FULL || x == B_EPI_DONE) n = 256;
            if (x == B_TAIL || x == B_TAIL + 1) n = 128;
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
    const uint32_t tmem = uint32_t(uniform(int(sh.tmem_base)));
    wait_for_previous_kernel();

    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == 8 && lane == 0) {
            // ---------------------------------------------------------- units + loads
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmDO);
            uint32_t nu = 0, g = 0;  // units with tiles, tiles
            bool stop = false;
            for (int it = 0; !stop; ++it) {
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
                RowWalk walk(a, x);
                for (int i = x.i0; i < x.i1; ++i, ++g, walk.next(x)) {
                    const int64_t head = int64_t(x.b) * a.Hq + walk.hq;
                    const int qrow = int(head * a.Lq) + walk.t0;
                    const uint32_t qs = g % 3, os = g & 1;
                    if (!wait_bar(bar(B_Q_EMPTY + qs), ((g / 3) & 1) ^ 1, abort, hdr, 263)) { stop = true; break; }
                    mbar_expect_tx(bar(B_Q_FULL + qs), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sQ + qs * C::kTileBytes + s * C::kSlabBytes, &tmQ, bar(B_Q_FULL + qs), 64 * s, qrow);
                    if (!wait_bar(bar(B_O_EMPTY + os), ((g >> 1) & 1) ^ 1, abort, hdr, 264)) { stop = true; ++g; break; }
                    mbar_expect_tx(bar(B_O_FULL + os), C::kTileBytes + C::kStatBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sDO + os * C::kTileBytes + s * C::kSlabBytes, &tmDO, bar(B_O_FULL + os), 64 * s, qrow);
                    const int64_t srow = head * stat_rows(a.Lq) + walk.t0;
                    bulk_load(base + C::oStat + os * C::kStatBytes, nl2 + srow, C::kStatBytes / 2, bar(B_O_FULL + os));
                    bulk_load(base + C::oStat + os * C::kStatBytes + C::kStatBytes / 2, nd + srow, C::kStatBytes / 2,
                              bar(B_O_FULL + os));
                }
            }
            // every issued copy lands before the CTA exits (after an abort the last dO copy may
            // not have been issued: its wait then runs out)
            if (nu > 0) drain_bar(bar(B_KV_FULL), (nu - 1) & 1, hdr, 265);
            for (uint32_t i = g >= 3 ? g - 3 : 0; i < g; ++i) drain_bar(bar(B_Q_FULL + i % 3), (i / 3) & 1, hdr, 266);
            for (uint32_t i = g >= 2 ? g - 2 : 0; i < g; ++i) drain_bar(bar(B_O_FULL + (i & 1)), (i >> 1) & 1, hdr, 267);
        } else if (warp == 9) {
            // ---------------------------------------------------------- MMA issue
            // the whole warp walks the tiles, one elected lane issues (uniform descriptors)
            const bool leader = elect_one();
            uint32_t g = 0, nu = 0;  // tiles, units with tiles
            bool stop = false;
            // column (from a buffer's first) of the bf16 pairs of rows 16 kk .. + 15: warpgroup
            // kk / 4 wrote its 64 rows over the first 32 columns of its own half
            auto pcol = [](int kk) { return 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3); };
            // Fine: what they leave of P^T in the half's other 32 columns, and of dS^T, whose
            // pairs take 16 of the 32 columns that dP^T of the same rows had, in the other 16
            auto gcol = [&](int kk) { return Fine ? 64u * uint32_t(kk >> 2) + 32u * uint32_t((kk >> 1) & 1) + 8u * uint32_t(kk & 1) : pcol(kk); };
            auto issue_dv = [&](uint32_t t, bool first) -> bool {  // dV += P^T dO of tile t
                const uint32_t gb = sDO + (t & 1) * C::kTileBytes;
                const uint32_t acc = first ? 0u : 1u;
                // the first 32 rows of either warpgroup, then the others
                if (!wait_bar_warp(bar(B_P_HALF + (t & 1)), (t >> 1) & 1, abort, hdr, 277)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if ((kk & 2) == 0) {
                            umma_ts(tmem + C::kColDV, tmem + C::col_st(t) + pcol(kk), sdesc_sw128(gb + kk * 2048, C::kSlabBytes, 1024),
                                    C::kIdescAcc, kk > 0 ? 1u : acc);
                            if constexpr (Fine)
                                umma_ts(tmem + C::kColDV, tmem + C::col_st(t) + 32 + pcol(kk),
                                        sdesc_sw128(gb + kk * 2048, C::kSlabBytes, 1024), C::kIdescAcc, 1u);
                        }
                }
                __syncwarp();
                if (!wait_bar_warp(bar(B_P_FULL + (t & 1)), (t >> 1) & 1, abort, hdr, 268)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if ((kk & 2) != 0) {
                            umma_ts(tmem + C::kColDV, tmem + C::col_st(t) + pcol(kk), sdesc_sw128(gb + kk * 2048, C::kSlabBytes, 1024),
                                    C::kIdescAcc, 1u);
                            if constexpr (Fine)
                                umma_ts(tmem + C::kColDV, tmem + C::col_st(t) + 32 + pcol(kk),
                                        sdesc_sw128(gb + kk * 2048, C::kSlabBytes, 1024), C::kIdescAcc, 1u);
                        }
                    umma_commit(bar(B_O_EMPTY + (t & 1)));
                }
                __syncwarp();
                return true;
            };
            auto issue_dk = [&](uint32_t t, bool first) -> bool {  // dK += dS^T Q of tile t
                if (!wait_bar_warp(bar(B_DS_FULL), t & 1, abort, hdr, 269)) return false;
                tc_fence_after();
                const uint32_t qb = sQ + (t % 3) * C::kTileBytes;
                if (leader) {
                    const uint32_t acc = first ? 0u : 1u;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        umma_ts(tmem + C::kColDK, tmem + C::kColDPT + gcol(kk), sdesc_sw128(qb + kk * 2048, C::kSlabBytes, 1024),
                                C::kIdescAcc, kk > 0 ? 1u : acc);
                        if constexpr (Fine)
                            umma_ts(tmem + C::kColDK, tmem + C::kColDPT + 16 + gcol(kk),
                                    sdesc_sw128(qb + kk * 2048, C::kSlabBytes, 1024), C::kIdescAcc, 1u);
                    }
                    umma_commit(bar(B_Q_EMPTY + t % 3));
                }
                __syncwarp();
                return true;
            };
            // D[col] = A[sA] B[sB]^T over d, then an arrival on `done`
            auto issue_ss = [&](uint32_t col, uint32_t sa, uint32_t sb, uint32_t done) {
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + col, sdesc_sw128(sa + off, 16, 1024), sdesc_sw128(sb + off, 16, 1024), C::kIdescSS, kk > 0);
                    }
                    umma_commit(done);
                }
                __syncwarp();
            };
            for (int it = 0; !stop; ++it) {
                const int slot = it & 1;
                if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 270)) break;
                const int u = uniform(sh.item[slot]);
                if (leader) mbar_arrive(bar(B_ITEM_EMPTY + slot));
                __syncwarp();
                if (u < 0) break;
                Unit x;
                decode(a, p, u, x);
                const int i0 = uniform(x.i0), i1 = uniform(x.i1);
                if (i0 >= i1) continue;
                if (!wait_bar_warp(bar(B_KV_FULL), nu & 1, abort, hdr, 271)) break;
                auto issue_s = [&](uint32_t t) -> bool {  // S^T of tile t
                    if (!wait_bar_warp(bar(B_Q_FULL + t % 3), (t / 3) & 1, abort, hdr, 273)) return false;
                    tc_fence_after();
                    issue_ss(C::col_st(t), sK, sQ + (t % 3) * C::kTileBytes, bar(B_S_FULL + (t & 1)));
                    return true;
                };
                auto issue_dp = [&](uint32_t t) -> bool {  // dP^T of tile t
                    if (!wait_bar_warp(bar(B_O_FULL + (t & 1)), (t >> 1) & 1, abort, hdr, 274)) return false;
                    tc_fence_after();
                    issue_ss(C::kColDPT, sV, sDO + (t & 1) * C::kTileBytes, bar(B_DP_FULL));
                    return true;
                };
                // both warpgroups have read the previous unit's dV and dK
                auto accumulators = [&]() -> bool {
                    return nu == 0 || wait_bar_warp(bar(B_EPI_DONE), (nu - 1) & 1, abort, hdr, 272);
                };
                if constexpr (C::kTwoS) {
                    // S^T a tile ahead: the exponentials never wait for it
                    if (!issue_s(g)) break;
                    for (int i = i0; i < i1; ++i, ++g) {
                        if (!issue_dp(g) || (i + 1 < i1 && !issue_s(g + 1))) { stop = true; break; }
                        if (i + 1 == i1 && leader) umma_commit(bar(B_KV_EMPTY));
                        __syncwarp();
                        if ((i == i0 && !accumulators()) || !issue_dv(g, i == i0) || !issue_dk(g, i == i0)) { stop = true; break; }
                    }
                    if (stop) break;
                } else {
                    for (int i = i0; i < i1; ++i, ++g) {
                        if (i == i0 + 1 && !accumulators()) { stop = true; break; }
                        if (i > i0 && !issue_dv(g - 1, i - 1 == i0)) { stop = true; break; }
                        if (!issue_s(g)) { stop = true; break; }
                        if (i > i0 && !issue_dk(g - 1, i - 1 == i0)) { stop = true; break; }
                        if (!issue_dp(g)) { stop = true; break; }
                    }
                    if (stop) break;
                    if (leader) umma_commit(bar(B_KV_EMPTY));
                    __syncwarp();
                    const bool one = i1 - i0 == 1;
                    if (one && !accumulators()) break;
                    if (!issue_dv(g - 1, one) || !issue_dk(g - 1, one)) break;
                }
                if (leader) umma_commit(bar(B_ACC_DONE));
                __syncwarp();
                ++nu;
            }
            if (leader) {
                umma_commit(bar(B_MMA_DONE));
                drain_bar(bar(B_MMA_DONE), 0, hdr, 276);
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- compute (warps 0-7)
        const int wg = warp >> 2, row = tid & 127;  // rows [64 wg, + 64) of the tiles; key of the unit
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t g_addr = lane_addr + C::kColDPT + 64 * wg;
        const uint64_t sc2 = f2_pack(a.scale * kLog2e, a.scale * kLog2e);
        uint32_t g = 0, nu = 0, nt = 0;
        for (int it = 0;; ++it) {
            const int slot = it & 1;
            if (!wait_bar_warp(bar(B_ITEM_FULL + slot), (it >> 1) & 1, abort, hdr, 281)) break;
            const int u = sh.item[slot];
            mbar_arrive(bar(B_ITEM_EMPTY + slot));
            if (u < 0) break;
            Unit x;
            decode(a, p, u, x);
            const int keys_out = a.fill ? min(kTile, a.Lk - x.k0) : x.nk;  // with those past the last
            if (keys_out <= 0 && x.part < 0) continue;
            // positions that see this thread's key: [v_lo, v_hi)
            const int key = x.k0 + row;
            int v_lo = key < a.sinks ? -(1 << 30) : key - a.right;
            if (a.causal) v_lo = max(v_lo, key);
            const int v_hi = key < a.sinks ? (1 << 30) : key + a.left + 1;
            bool stop = false;
            RowWalk walk(a, x);
            for (int i = x.i0; i < x.i1; ++i, ++g, walk.next(x)) {
                const int t0 = walk.t0, n = walk.rows(x), skip = walk.r == 0 ? x.skip : 0;
                const uint32_t os = g & 1, s_addr = lane_addr + C::col_st(g) + 64 * wg;
                // dO and the statistics (their own barrier makes the copies visible here), S^T
                if (!wait_bar_warp(bar(B_O_FULL + os), (g >> 1) & 1, abort, hdr, 282)) { stop = true; break; }
                if (!wait_bar_warp(bar(B_S_FULL + (g & 1)), (g >> 1) & 1, abort, hdr, 283)) { stop = true; break; }
                tc_fence_after();
                float* stat = reinterpret_cast<float*>(smem_raw + C::oStat + os * C::kStatBytes) + 64 * wg;
                if (n < kTile || skip > 0) {
                    // rows past the last or before the first: nothing of theirs (whatever was loaded)
                    // may reach a product. dP^T may still be reading dO: what it makes of these rows
                    // is masked.
                    if (row >= n || row < skip) {
                        if ((row >> 6) == wg) {
                            stat[row & 63] = -INFINITY;
                            stat[128 + (row & 63)] = 0.f;
                        }
                        const uint32_t dst = (wg == 0 ? sQ + (g % 3) * C::kTileBytes : sDO + os * C::kTileBytes) + row * 128;
#pragma unroll
                        for (int c = 0; c < C::kSlabs * 8; ++c)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst + (c >> 3) * C::kSlabBytes + (c & 7) * 16),
                                         "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(bar(B_TAIL + wg));  // the statistics above are read by the whole warpgroup
                    if (!wait_bar_warp(bar(B_TAIL + wg), nt & 1, abort, hdr, 284)) { stop = true; break; }
                    ++nt;
                }
                const int p0 = t0 + x.seq.shift + 64 * wg;
                const int lo = v_lo - p0, hi = min(v_hi - p0, n - 64 * wg);
                const bool masked = !__all_sync(0xffffffffu, n == kTile && (row >= x.nk || (lo <= 0 && hi >= 64)));
                if (masked) {
#pragma unroll 1
                    for (int w = 0; w < 2; ++w) mask_cols(s_addr + 32 * w, win::bits(lo - 32 * w, hi - 32 * w), kMinusInf);
                    tmem_wait_st();
                }
                uint32_t s[64];
                tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                tmem_wait_ld_regs(s);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[16], rest[Fine ? 16 : 1];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float4 q = *reinterpret_cast<const float4*>(stat + 32 * c + 2 * e);  // four rows
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t& s0 = s[32 * c + 2 * (e + h)];
                            uint32_t& s1 = s[32 * c + 2 * (e + h) + 1];
                            float p0, p1;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(s0), __uint_as_float(s1)), sc2,
                                             h == 0 ? f2_pack(q.x, q.y) : f2_pack(q.z, q.w)), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            pk[e + h] = pack_bf16(p0, p1);
                            if constexpr (Fine) rest[e + h] = pack_rest(p0, p1, pk[e + h]);
                            s0 = __float_as_uint(p0);
                            s1 = __float_as_uint(p1);
                        }
                    }
                    tmem_st16(s_addr + 16 * c, pk);
                    if constexpr (Fine) tmem_st16(s_addr + 32 + 16 * c, rest);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar((c == 0 ? B_P_HALF : B_P_FULL) + int(g & 1)));
                }
                if (!wait_bar_warp(bar(B_DP_FULL), g & 1, abort, hdr, 285)) { stop = true; break; }
                tc_fence_after();
                // ds is zero where the row does not see the key: p is zero there, but dP or D of a
                // value, a gradient or a row past the last that nobody sees may be NaN. (A body
                // of its own for the edge tiles: 8,000 rows, window 256 + 256, 198.5 -> 201.3 us a
                // gradient; in one body for all tiles 202.4, and the long causal step 1 % slower.)
                auto form_ds = [&](auto edge) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t d[32], pk[16], rest[Fine ? 16 : 1];
                        tmem_ld32(g_addr + 32 * c, d);
                        tmem_wait_ld_regs(d);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float4 q = *reinterpret_cast<const float4*>(stat + 128 + 32 * c + 2 * e);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int i0 = 2 * (e + h);
                                float d0, d1;
                                f2_unpack(f2_mul(f2_pack(__uint_as_float(s[32 * c + i0]), __uint_as_float(s[32 * c + i0 + 1])),
                                                 f2_add(f2_pack(__uint_as_float(d[i0]), __uint_as_float(d[i0 + 1])),
                                                        h == 0 ? f2_pack(q.x, q.y) : f2_pack(q.z, q.w))), d0, d1);
                                pk[e + h] = pack_bf16(d0, d1);
                                if constexpr (Fine) rest[e + h] = pack_rest(d0, d1, pk[e + h]);
                            }
                        }
                        if constexpr (decltype(edge)::value) {
                            const uint32_t see = win::bits(lo - 32 * c, hi - 32 * c);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint32_t keep = pair_mask(see, 2 * e);
                                pk[e] &= keep;
                                if constexpr (Fine) rest[e] &= keep;
                            }
                        }
                        tmem_st16(g_addr + (Fine ? 32 : 16) * c, pk);
                        if constexpr (Fine) tmem_st16(g_addr + 32 * c + 16, rest);
                    }
                };
                if (masked) form_ds(std::true_type{});
                else form_ds(std::false_type{});
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_DS_FULL));
                mbar_arrive(bar(B_O_EMPTY + os));
            }
            if (stop) break;
            // this warpgroup's half of the columns of dV and dK for its key rows
            const bool some = x.i0 < x.i1;
            if (some) {
                if (!wait_bar_warp(bar(B_ACC_DONE), nu & 1, abort, hdr, 286)) break;
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
                        tmem_ld32(lane_addr + (t == 0 ? C::kColDV : C::kColDK) + wg * HC + c0, o);
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
                    } else if (row < keys_out) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = some && valid ? pack_bf16(__uint_as_float(o[8 * i + 2 * e]) * mul, __uint_as_float(o[8 * i + 2 * e + 1]) * mul) : 0u;
                            *reinterpret_cast<uint4*>(out + orow + c0 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            tc_fence_before();
            if (some) mbar_arrive(bar(B_EPI_DONE));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The split tiles' dV and dK: their parts added in order. A thread owns four columns
// of a key.
template <int D>
__global__ void __launch_bounds__(256) window_dkv_join_kernel(const __grid_constant__ WinArgs a,
                                                              const __grid_constant__ WinBwdPlan p,
                                                              const float* parts, __nv_bfloat16* dK, __nv_bfloat16* dV) {
    constexpr int PER = D / 4;
    wait_for_previous_kernel();
    const int heads = a.B * a.Hk;
    const int64_t total = int64_t(p.split_tiles) * heads * 2 * 128 * PER;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
        const int c = int(i % PER), r = int(i / PER % 128), t = int(i / PER / 128 % 2);
        const int64_t tile = i / PER / 128 / 2;  // key tile x heads + (batch, key head)
        const int kt = int(tile / heads), bh = int(tile % heads), key = kt * kTile + r;
        if (key >= (a.fill ? a.Lk : win::seq(a, bh / a.Hk).n)) continue;
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

template <int D, bool Fine>
cudaError_t launch_d(const WinArgs& a, const void* Q, const void* K, const void* V, const void* O, const float* lse,
                     const void* dO, void* dQ, void* dK, void* dV, char* ws, const WinBwdPlan& p, cudaStream_t s) {
    int32_t* hdr = nullptr;
    cudaError_t e = window_error_word(&hdr);
    if (e != cudaSuccess) return e;
    const int sms = multiprocessors();
    const int64_t qrows = int64_t(a.B) * a.Hq * a.Lq, krows = int64_t(a.B) * a.Hk * a.Lk;
    int32_t* work = reinterpret_cast<int32_t*>(ws + p.work);
    float* nl2 = reinterpret_cast<float*>(ws + p.nl2);
    float* nd = reinterpret_cast<float*>(ws + p.nd);
    float* parts = reinterpret_cast<float*>(ws + p.part);
    const int64_t want = ((int64_t(a.B) * a.Hq * stat_rows(a.Lq) + 128) * (D / 8) + 255) / 256, most = int64_t(sms) * 16;
    e = launch_after(window_stats_kernel<D>, int(want < most ? want : most), 256, 0, s, a,
                     static_cast<const __nv_bfloat16*>(O), static_cast<const __nv_bfloat16*>(dO), lse, nl2, nd, work);
    if (e != cudaSuccess) return e;
    CUtensorMap tmQ, tmDO, tmK, tmV;
    if (krows > 0) {
        if (!make_tmap(&tmK, K, D, krows) || !make_tmap(&tmV, V, D, krows)) return cudaErrorInvalidValue;
    }
    if (qrows > 0) {
        if (!make_tmap(&tmQ, Q, D, qrows) || !make_tmap(&tmDO, dO, D, qrows)) return cudaErrorInvalidValue;
        if (krows == 0) tmK = tmV = tmQ;  // no key tile is loaded
        const int smem = dq::Cfg<D>::kSmem;
        e = cudaFuncSetAttribute(dq::window_dq_kernel<D, Fine>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int nqt = (a.Lq + kTile - 1) / kTile, n = a.B * a.Hq * nqt;
        e = launch_after(dq::window_dq_kernel<D, Fine>, n < sms ? n : sms, kThreads, smem, s, tmQ, tmDO, tmK, tmV, a, n,
                         nqt, nl2, nd, work, hdr, static_cast<__nv_bfloat16*>(dQ));
        if (e != cudaSuccess) return e;
    }
    if (krows > 0) {
        const int smem = dkv::Cfg<D>::kSmem;
        e = cudaFuncSetAttribute(dkv::window_dkv_kernel<D, Fine>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const int heads = a.B * a.Hk;
        const int n = heads * (p.key_tiles - p.split_tiles + p.split_tiles * p.splits);
        if (qrows == 0) tmQ = tmDO = tmK;  // no row tile is loaded
        e = launch_after(dkv::window_dkv_kernel<D, Fine>, n < sms ? n : sms, kThreads, smem, s, tmK, tmV, tmQ, tmDO, a,
                         p, n, nl2, nd, work + 1, hdr, parts, static_cast<__nv_bfloat16*>(dK), static_cast<__nv_bfloat16*>(dV));
        if (e != cudaSuccess) return e;
        if (p.splits > 1) {
            const int64_t blocks = (int64_t(p.split_tiles) * heads * 2 * 128 * (D / 4) + 255) / 256;
            e = launch_after(dkv::window_dkv_join_kernel<D>, int(blocks < most ? blocks : most), 256, 0, s, a, p, parts,
                             static_cast<__nv_bfloat16*>(dK), static_cast<__nv_bfloat16*>(dV));
            if (e != cudaSuccess) return e;
        }
    }
    return cudaGetLastError();
}

}  // namespace

WinBwdPlan plan_window_bwd(const WinArgs& a, int d) {
    WinBwdPlan p;
    auto align = [](size_t x) { return (x + 255) & ~size_t(255); };
    p.work = 0;
    const size_t stat = align((size_t(a.B) * a.Hq * size_t(stat_rows(a.Lq)) + 128) * sizeof(float));
    p.nl2 = 256;
    p.nd = p.nl2 + stat;
    p.part = p.nd + stat;
    p.key_tiles = (a.Lk + kTile - 1) / kTile;
    const int sink_tiles = (a.sinks + kTile - 1) / kTile;
    p.split_tiles = sink_tiles < p.key_tiles ? sink_tiles : p.key_tiles;
    // The first keys' tiles walk every row, the others the rows of one window. Split
    // into about the others' length, but into no more units than four an SM: a unit
    // costs its fp32 part (128 KB at d = 128, written and read once).
    const int64_t heads = int64_t(a.B) * a.Hk;
    if (p.split_tiles > 0 && heads > 0 && a.Lq > 0) {
        const int64_t all = (a.Lq + kTile - 1) / kTile;
        const int64_t reach = (a.left == kWinOpen ? a.Lq : a.left) + (a.right == kWinOpen ? a.Lq : a.right);
        const int64_t near = (reach + kTile - 1) / kTile + 1;
        int64_t n = (all + near - 1) / near;
        const int64_t cap = (4 * int64_t(multiprocessors()) + p.split_tiles * heads - 1) / (p.split_tiles * heads);
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
    if (a.Lq <= kFineRows)
        return d == 128 ? launch_d<128, true>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s)
                        : launch_d<64, true>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s);
    return d == 128 ? launch_d<128, false>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s)
                    : launch_d<64, false>(a, Q, K, V, O, lse, dO, dQ, dK, dV, ws, p, s);
}

}  // namespace moc
