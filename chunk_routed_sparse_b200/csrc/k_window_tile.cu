// Sliding-window attention with always-visible first keys, forward, one 128-row tile
// per work item: for problems with few row tiles, where each item's chain of product,
// softmax and product sets the time, and for padded batches, whose items are handed out
// as CTAs become free (k_window_fwd.cu: two tiles an item, which share their keys and hide
// one another's chain).
//
// The same mathematics, masking, rounding and bounds as there. Here both softmax
// warpgroups work on the one tile, half of a key tile's columns each (one thread a row
// and half), and exchange their row maxima through shared memory; TMEM holds two S, so
// that S(j+1) is formed under the softmax of S(j). Open and causal over 2,112 tokens (17 key
// tiles at most, 2 heads): 21.9 us at d = 64, against 30.1 with one of the two-tile
// kernel's tiles an item; the tiny scene (window 256 + 64) 11.8 against 14.9. Bound by the
// chain of product, row maximum, exchange, exponentials and product of each key tile.
//   warp 8 (one lane): TMA: Q, a 3-stage ring of K tiles, a 2-stage ring of V tiles.
//   warp 9: S(j+1) = Q K(j+1)^T, then O += P(j) V(j).
//   warps 0-3 / 4-7: keys 0-63 / 64-127 of every tile.
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
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;  // O is rescaled once the row max grows by more than 2^8
constexpr uint32_t kColO = 256;
constexpr int kKSt = 3, kVSt = 2;

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = 128 * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int oQ = 0;
    static constexpr int oK = oQ + kTileBytes;
    static constexpr int oV = oK + kKSt * kTileBytes;
    static constexpr int oStage = oV + kVSt * kTileBytes;  // 8 warps x 32 rows x D bytes
    static constexpr int oEx = oStage + 8 * 32 * D;        // fp32 [2 exchanges][2 warpgroups][128]
    static constexpr int oBar = oEx + 2048;
    // the dynamic shared memory of a kernel without static shared memory starts on a
    // 1024-byte boundary (checked at the start): no room for slack at d = 128
    static constexpr int kSmem = oBar + 256 > 120 * 1024 ? oBar + 256 : 120 * 1024;
    static_assert(kSmem <= 232448, "shared memory per CTA");
    static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0);
    static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
};

__device__ __forceinline__ uint32_t col_s(uint32_t g) { return (g & 1) * 128u; }
// column (from a buffer's first) of the bf16 pairs of keys 16 kk .. + 15
__device__ __forceinline__ uint32_t p_col(int kk) { return 64u * uint32_t(kk >> 2) + 8u * uint32_t(kk & 3); }

enum {
    B_Q_FULL = 0, B_Q_EMPTY = 1, B_K_FULL = 2, B_K_EMPTY = 5, B_V_FULL = 8, B_V_EMPTY = 10, B_S_FULL = 12, B_P_FULL = 14,
    B_PV_DONE = 16, B_EX = 17, B_MMA_DONE = 18, B_ITEM_FULL = 19, B_ITEM_EMPTY = 21, B_COUNT = 23
};
struct Shared {  // at oBar + 240, after two answers of 16 bytes and the barriers
    uint32_t tmem_base;
    int abort;
};
static_assert(32 + B_COUNT * 8 <= 240, "barriers");

using win::Item;
using win::nth_item;
__device__ __forceinline__ void decode(const WinArgs& a, int nqt, int item, Item& x) { win::decode(a, 128, nqt, item, x); }

// Ask: the grid has a CTA for every item, and a running one asks for those that are not
// launched yet; otherwise it has a CTA an SM, and its items are those of nth_item.
template <int D, bool Ask>
__global__ void __launch_bounds__(kThreads, 1)
    window_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ WinArgs a, int n_items, int nqt,
                       int32_t* __restrict__ hdr, __nv_bfloat16* __restrict__ O, float* __restrict__ lse) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    if (base & 1023u) {
        wait_for_previous_kernel();
        if (threadIdx.x == 0) set_error(hdr, ERR_CHECK, 310);
        return;
    }
    const uint32_t sQ = base + C::oQ, sK = base + C::oK, sV = base + C::oV, sBar = base + C::oBar + 32;
    Shared& sh = *reinterpret_cast<Shared*>(smem_raw + C::oBar + 240);
    volatile int* abort = &sh.abort;
    auto bar = [&](int i) { return sBar + 8u * uint32_t(i); };
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    let_next_kernel_start();

    if (tid == 0) {
        for (int x = 0; x < B_COUNT; ++x) {
            int n = x == B_P_FULL || x == B_P_FULL + 1 || x == B_EX ? 256 : 1;
            if (x >= B_ITEM_EMPTY) n = 2 + 256;  // the loading lane, the issuing one, the softmax warps
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
    // Ask: item n > 0 of a CTA is its n-th answer, in slot n & 1, the slot's ((n - 1) / 2)-th.
    auto answer = [&](int n) { return base + C::oBar + 16u * uint32_t(n & 1); };
    auto full = [&](int n) { return bar(B_ITEM_FULL + (n & 1)); };
    auto parity = [](int n) { return uint32_t((n - 1) >> 1) & 1u; };

    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == 8 && lane == 0) {
            // ---------------------------------------------------------- loads
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            uint32_t g = 0, nq = 0;
            bool stop = false;
            int asked = 0;  // the answer that is outstanding
            for (int n = 0, item = int(blockIdx.x); !stop; ++n) {
                if (!Ask && n > 0) {
                    item = nth_item(n);
                    if (item >= n_items) break;
                } else if (n > 0) {
                    // asked for once this CTA's last loads are under way: an item claimed earlier
                    // would wait here while other CTAs have nothing left to do
                    if (!wait_bar(bar(B_ITEM_EMPTY + (n & 1)), parity(n) ^ 1, abort, hdr, 318)) break;
                    mbar_expect_tx(full(n), 16);
                    ask_for_cta(answer(n), full(n));
                    asked = n;
                    if (!wait_bar(full(n), parity(n), abort, hdr, 317)) break;
                    asked = 0;
                    item = asked_cta(answer(n));
                    fence_proxy_async_smem();  // read before the slot's next answer
                    mbar_arrive(bar(B_ITEM_EMPTY + (n & 1)));
                    if (item < 0) break;
                }
                Item x;
                decode(a, nqt, item, x);
                if (x.tiles == 0) continue;
                const int krow = (x.b * a.Hk + x.hq / a.group) * a.Lk;
                if (!wait_bar(bar(B_Q_EMPTY), (nq & 1) ^ 1, abort, hdr, 311)) break;
                ++nq;
                mbar_expect_tx(bar(B_Q_FULL), C::kTileBytes);
#pragma unroll
                for (int s = 0; s < C::kSlabs; ++s)
                    tma_load_2d(sQ + s * C::kSlabBytes, &tmQ, bar(B_Q_FULL), 64 * s, (x.b * a.Hq + x.hq) * a.Lq + x.t0);
                for (int j = 0; j < x.tiles; ++j, ++g) {
                    int key0, end;
                    win::tile(x.y, j, key0, end);
                    const uint32_t ks = g % kKSt, vs = g % kVSt;
                    if (!wait_bar(bar(B_K_EMPTY + ks), ((g / kKSt) & 1) ^ 1, abort, hdr, 312)) { stop = true; break; }
                    mbar_expect_tx(bar(B_K_FULL + ks), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sK + ks * C::kTileBytes + s * C::kSlabBytes, &tmK, bar(B_K_FULL + ks), 64 * s, krow + key0);
                    if (!wait_bar(bar(B_V_EMPTY + vs), ((g / kVSt) & 1) ^ 1, abort, hdr, 313)) { stop = true; ++g; break; }
                    mbar_expect_tx(bar(B_V_FULL + vs), C::kTileBytes);
#pragma unroll
                    for (int s = 0; s < C::kSlabs; ++s)
                        tma_load_2d(sV + vs * C::kTileBytes + s * C::kSlabBytes, &tmV, bar(B_V_FULL + vs), 64 * s, krow + key0);
                }
            }
            if (asked) drain_bar(full(asked), parity(asked), hdr, 319);
            // every issued copy lands before the CTA exits (after an abort the last V copy may
            // not have been issued: its wait then runs out)
            if (nq > 0) drain_bar(bar(B_Q_FULL), (nq - 1) & 1, hdr, 314);
            for (uint32_t i = g >= kKSt ? g - kKSt : 0; i < g; ++i) drain_bar(bar(B_K_FULL + i % kKSt), (i / kKSt) & 1, hdr, 315);
            for (uint32_t i = g >= kVSt ? g - kVSt : 0; i < g; ++i) drain_bar(bar(B_V_FULL + i % kVSt), (i / kVSt) & 1, hdr, 316);
        } else if (warp == 9) {
            // ---------------------------------------------------------- MMA issue
            // (the whole warp walks the tiles, one elected lane issues: uniform descriptors)
            const bool leader = elect_one();
            uint32_t g = 0, nq = 0;
            bool stop = false;
            auto issue_s = [&](uint32_t t, bool last) -> bool {  // S(t) = Q K(t)^T
                const uint32_t ks = t % kKSt, kb = sK + ks * C::kTileBytes;
                if (!wait_bar_warp(bar(B_K_FULL + ks), (t / kKSt) & 1, abort, hdr, 321)) return false;
                tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::kSlabBytes + (kk & 3) * 32;
                        umma_ss(tmem + col_s(t), sdesc_sw128(sQ + off, 16, 1024), sdesc_sw128(kb + off, 16, 1024), C::kIdescQK, kk > 0);
                    }
                    umma_commit(bar(B_S_FULL + (t & 1)));
                    umma_commit(bar(B_K_EMPTY + ks));
                    if (last) umma_commit(bar(B_Q_EMPTY));
                }
                __syncwarp();
                return true;
            };
            for (int n = 0, item = int(blockIdx.x); !stop; ++n) {
                if (!Ask && n > 0) {
                    item = nth_item(n);
                    if (item >= n_items) break;
                } else if (n > 0) {
                    if (!wait_bar_warp(full(n), parity(n), abort, hdr, 326)) break;
                    item = uniform(asked_cta(answer(n)));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (leader) mbar_arrive(bar(B_ITEM_EMPTY + (n & 1)));
                    __syncwarp();
                    if (item < 0) break;
                }
                Item x;
                decode(a, nqt, item, x);
                const int T = uniform(x.tiles);
                if (T == 0) continue;
                if (!wait_bar_warp(bar(B_Q_FULL), nq & 1, abort, hdr, 322)) break;
                ++nq;
                if (!issue_s(g, T == 1)) break;
                for (int j = 0; j < T; ++j, ++g) {
                    if (j + 1 < T && !issue_s(g + 1, j + 2 == T)) { stop = true; break; }
                    const uint32_t vs = g % kVSt, vb = sV + vs * C::kTileBytes;
                    if (!wait_bar_warp(bar(B_V_FULL + vs), (g / kVSt) & 1, abort, hdr, 323)) { stop = true; break; }
                    if (!wait_bar_warp(bar(B_P_FULL + (g & 1)), (g >> 1) & 1, abort, hdr, 324)) { stop = true; break; }
                    tc_fence_after();
                    if (leader) {
                        const uint32_t acc = j > 0 ? 1u : 0u;
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_ts(tmem + kColO, tmem + col_s(g) + p_col(kk), sdesc_sw128(vb + kk * 2048, C::kSlabBytes, 1024),
                                    C::kIdescPV, kk > 0 ? 1u : acc);
                        umma_commit(bar(B_PV_DONE));
                        umma_commit(bar(B_V_EMPTY + vs));
                    }
                    __syncwarp();
                }
            }
            if (leader) {
                umma_commit(bar(B_MMA_DONE));  // TMEM is released after every MMA
                drain_bar(bar(B_MMA_DONE), 0, hdr, 325);
            }
        }
        __syncwarp();
    } else {
        regs_inc<kRegsCompute>();
        // -------------------------------------------------------------- softmax
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t o_addr = lane_addr + kColO + wg * (D / 2);  // this warpgroup's half of O's columns
        const uint32_t stg = base + C::oStage + warp * 32 * D;
        const float sl2 = a.scale * 1.4426950408889634f;
        const uint64_t sc2 = f2_pack(sl2, sl2);
        uint32_t g = 0, nx = 0;
        // What the row's other half has; exchanges alternate between two buffers, so that
        // one's values are read before the next but one overwrites them.
        auto other = [&](float v, float& o) -> bool {
            float* ex = reinterpret_cast<float*>(smem_raw + C::oEx) + (nx & 1) * 256;
            ex[wg * 128 + row] = v;
            mbar_arrive(bar(B_EX));
            if (!wait_bar_warp(bar(B_EX), nx & 1, abort, hdr, 331)) return false;
            ++nx;
            o = ex[(wg ^ 1) * 128 + row];
            return true;
        };
        bool stop = false;
        for (int n = 0, item = int(blockIdx.x); !stop; ++n) {
            if (!Ask && n > 0) {
                item = nth_item(n);
                if (item >= n_items) break;
            } else if (n > 0) {
                if (!wait_bar_warp(full(n), parity(n), abort, hdr, 336)) break;
                item = asked_cta(answer(n));
                fence_proxy_async_smem();
                mbar_arrive(bar(B_ITEM_EMPTY + (n & 1)));
                if (item < 0) break;
            }
            Item x;
            decode(a, nqt, item, x);
            // rows to write: the live ones, and with a.fill those past the last
            const int rows_out = a.fill ? min(128, a.Lq - x.t0) : x.rows;
            if (rows_out <= 0) continue;
            const bool live = row < x.rows;
            const win::Row vis = win::row(a, x.seq.n, x.t0 + row + x.seq.shift);
            float m_used = -INFINITY, l = 0.f;
            for (int j = 0; j < x.tiles; ++j, ++g) {
                int key0, end;
                win::tile(x.y, j, key0, end);
                const uint32_t s_addr = lane_addr + col_s(g) + 64 * wg;
                const int k0 = key0 + 64 * wg;
                const int ns = min(vis.s, end) - k0, lo = vis.lo - k0, hi = min(vis.hi, end) - k0;
                if (!wait_bar_warp(bar(B_S_FULL + (g & 1)), (g >> 1) & 1, abort, hdr, 332)) { stop = true; break; }
                tc_fence_after();
                uint32_t s[64];
                // (the loads inside the branches: a mask after a common load becomes selects that
                // every tile executes)
                if (__all_sync(0xffffffffu, !live || ns >= 64 || (lo <= 0 && hi >= 64))) {
                    tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                    tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                    tmem_wait_ld_regs(s);
                } else {
                    const uint32_t m0 = win::bits(0, ns) | win::bits(lo, hi);
                    const uint32_t m1 = win::bits(0, ns - 32) | win::bits(lo - 32, hi - 32);
                    tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                    tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                    tmem_wait_ld_regs(s);
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!((c < 32 ? m0 : m1) & (1u << (c & 31)))) s[c] = 0xff800000u;  // -inf
                }
                float mv[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mv[i] = fmaxf(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
#pragma unroll
                for (int c = 16; c < 64; c += 16) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mv[i] = max3(mv[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
                }
                const float mh = max3(max3(mv[0], mv[1], mv[2]), max3(mv[3], mv[4], mv[5]), fmaxf(mv[6], mv[7]));
                float mo;
                if (!other(mh, mo)) { stop = true; break; }
                const float mx = fmaxf(mh, mo) * sl2;  // the same in both halves, and all that follows from it
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
                    if (!wait_bar_warp(bar(B_PV_DONE), (g - 1) & 1, abort, hdr, 333)) { stop = true; break; }
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_addr + c * 32, o);
                        tmem_wait_ld_regs(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(o_addr + c * 32, o);
                    }
                }
                // a row without a visible key so far: its weights are exp2(-inf - 0) = 0
                const float m0f = m_used > -INFINITY ? m_used : 0.f;
                const uint64_t nm2 = f2_pack(-m0f, -m0f);
                uint64_t sum2a = 0, sum2b = 0;
                uint32_t pk[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float x0, x1;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sc2, nm2), x0, x1);
                    const float p0 = ex2(x0), p1 = ex2(x1);
                    if (c & 1) sum2b = f2_add(sum2b, f2_pack(p0, p1));
                    else sum2a = f2_add(sum2a, f2_pack(p0, p1));
                    pk[c] = pack_bf16(p0, p1);
                }
                tmem_st32(s_addr, pk);
                float r0, r1, r2, r3;
                f2_unpack(sum2a, r0, r1);
                f2_unpack(sum2b, r2, r3);
                l = l * alpha + ((r0 + r1) + (r2 + r3));
                if (end - key0 < 128) {  // V rows past the tile's keys: zeros, whatever was loaded
                    if (!wait_bar_warp(bar(B_V_FULL + g % kVSt), (g / kVSt) & 1, abort, hdr, 334)) { stop = true; break; }
                    if (row >= end - key0) {
                        const uint32_t vr = sV + (g % kVSt) * C::kTileBytes + row * 128;
#pragma unroll
                        for (int i = 0; i < C::kSlabs * 4; ++i) {  // half of the row's 16-byte pieces
                            const int ch = wg * C::kSlabs * 4 + i;
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vr + (ch >> 3) * C::kSlabBytes + (ch & 7) * 16),
                                         "r"(0u) : "memory");
                        }
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(B_P_FULL + (g & 1)));
            }
            if (stop) break;
            // ---------------------------------------------------------- epilogue
            float lo_half = 0.f;
            if (x.tiles > 0) {
                if (!other(l, lo_half)) break;
                if (!wait_bar_warp(bar(B_PV_DONE), (g - 1) & 1, abort, hdr, 335)) break;
                tc_fence_after();
            }
            l = wg == 0 ? l + lo_half : lo_half + l;
            const size_t orow = (size_t(x.b) * a.Hq + x.hq) * size_t(a.Lq) + size_t(x.t0);
            const bool seen = live && (l > 0.f || l != l);  // NaN stays NaN
            const float inv = 1.f / l;
            const int w0 = (warp & 3) * 32;
            constexpr int PC = D / 16;  // 16-byte pieces of this warpgroup's half row
            uint32_t pk[D / 4];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t o[32];
                if (x.tiles > 0) {
                    tmem_ld32(o_addr + c * 32, o);
                    tmem_wait_ld_regs(o);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    pk[c * 16 + i] = seen ? pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
            }
#pragma unroll
            for (int i = 0; i < PC; ++i)
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stg + lane * D + ((i ^ (lane & (PC - 1))) << 4)),
                             "r"(pk[4 * i]), "r"(pk[4 * i + 1]), "r"(pk[4 * i + 2]), "r"(pk[4 * i + 3]) : "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PC; ++i) {
                const int idx = i * 32 + lane, r = idx / PC, ch = idx % PC;
                uint4 v;
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(stg + r * D + ((ch ^ (r & (PC - 1))) << 4)) : "memory");
                if (w0 + r < rows_out)
                    *reinterpret_cast<uint4*>(O + (orow + w0 + r) * D + wg * (D / 2) + ch * 8) = v;
            }
            __syncwarp();
            tc_fence_before();
            if (wg == 0 && row < rows_out && lse)
                lse[orow + row] = seen ? (m_used + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool Ask>
cudaError_t launch_d(const WinArgs& a, const void* Q, const void* K, const void* V, void* O, float* lse,
                     cudaStream_t s) {
    int32_t* hdr = nullptr;
    cudaError_t e = window_error_word(&hdr);
    if (e != cudaSuccess) return e;
    CUtensorMap tmQ, tmK, tmV;
    const int64_t qrows = int64_t(a.B) * a.Hq * a.Lq, krows = int64_t(a.B) * a.Hk * a.Lk;
    if (!make_tmap(&tmQ, Q, D, qrows)) return cudaErrorInvalidValue;
    if (krows == 0) tmK = tmV = tmQ;  // no key tile is loaded
    else if (!make_tmap(&tmK, K, D, krows) || !make_tmap(&tmV, V, D, krows)) return cudaErrorInvalidValue;
    const int smem = Cfg<D>::kSmem;
    e = cudaFuncSetAttribute(window_tile_kernel<D, Ask>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int nqt = (a.Lq + 127) / 128, n_items = a.B * a.Hq * nqt;
    const int sms = multiprocessors();
    return launch_after(window_tile_kernel<D, Ask>, !Ask && n_items > sms ? sms : n_items, kThreads, smem, s, tmQ, tmK,
                        tmV, a, n_items, nqt, hdr, static_cast<__nv_bfloat16*>(O), lse);
}

}  // namespace

cudaError_t launch_window_tile(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                               float* lse, cudaStream_t s) {
    // Items of equal rows go in rounds: asking costs them up to 13 % (18 heads of 2,112 rows,
    // 256 keys either side: 19.8 against 22.4 us). In a padded batch rounds leave some CTAs
    // the items without rows: three sequences, the last empty, 12 heads, 700 keys back, open
    // and causal at 2,501 rows 43.6 and 57.6 us in rounds, 31.9 and 37.1 asking.
    if (a.q_len)
        return d == 128 ? launch_d<128, true>(a, Q, K, V, O, lse, s) : launch_d<64, true>(a, Q, K, V, O, lse, s);
    return d == 128 ? launch_d<128, false>(a, Q, K, V, O, lse, s) : launch_d<64, false>(a, Q, K, V, O, lse, s);
}

}  // namespace moc
