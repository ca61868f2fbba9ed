// Sliding-window attention of a few rows (new tokens) against a long cache.
//
// The rows of all query heads of a key head (at most 16: Lq x group) form one
// 16-row tile, so the cache is read once: the floor is its visible K and V bytes. A
// thread-block cluster takes one (batch, key head); its CTAs take 64-key tiles in
// turn, and their running maxima, sums and outputs are joined through distributed
// shared memory in the same launch, in CTA order: one launch, no workspace, nothing
// kept between calls.
//   warp 4 (one lane): TMA of K and V tiles (128-byte swizzle) into a 3-stage ring
//          (96 KB at d = 128: two CTAs an SM, 192 KB in flight).
//   warps 0-3: 16 keys of every tile each: S = Q K^T and O += P V with warp-level
//          MMAs (mma.sync; 16 rows fill its M, a 128-row tcgen05 tile would be an
//          eighth used at best, and the bytes bound this kernel either way), running
//          maximum and sum per warp in fp32; joined over the warps at the end.
// One token of eight streams, 24 heads, 8,255 visible keys each (811 MB): 125 us, the
// measured copy bandwidth. A fourth stage (one CTA an SM) takes 202 us; clusters of 1,
// 2, 4 and 8 CTAs 131, 153, 129 and 144 us.
// Rounding and masking as in the many-row kernel: P to bf16 before P V, sums of the
// unrounded weights, keys past a run of visible ones never reach a product. (The rest of P
// as a second operand: errors of O 1.00 instead of 1.35 times its own rounding's, for 2 to
// 6 % of the time, 124.5 -> 127.4 us here. Not taken: a token's O then has the error that
// the many-row kernels and the routed attention give it in a prompt, and not another.)
#include "common.cuh"
#include "pipeline.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace moc {
namespace {

using namespace sm100;

constexpr int kThreads = 160, kWarps = 4, kKeys = 64, kStages = 3, kR = kWinFewRows;
constexpr int kMaxCluster = 8;  // the portable limit

template <int D>
struct Cfg {
    static constexpr int kSlabs = D / 64;
    static constexpr int kSlabBytes = kKeys * 128;
    static constexpr int kTileBytes = kSlabs * kSlabBytes;
    static constexpr int oV = kStages * kTileBytes;
    static constexpr int oBar = 2 * kStages * kTileBytes;
    static constexpr int kSmem = oBar + 128 + 1024;
    // after the last tile the ring holds the join: O [5][16][D + 4], max and sum [5][16]
    static constexpr int kRow = D + 4;
    static_assert((kWarps + 1) * kR * (kRow + 2) * 4 <= oBar, "join");
};

template <int D>
__global__ void __launch_bounds__(kThreads)
    window_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ WinArgs a, const __nv_bfloat16* Q,
                      __nv_bfloat16* __restrict__ O, float* __restrict__ lse, int32_t* __restrict__ hdr) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t sBar = base + C::oBar;
    auto full = [&](int s) { return sBar + 16u * uint32_t(s); };
    auto empty = [&](int s) { return sBar + 16u * uint32_t(s) + 8u; };
    volatile int* abort = reinterpret_cast<volatile int*>(gbase + C::oBar + 96);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    sm100::let_next_kernel_start();
    const int rank = int(cluster_rank()), cs = int(gridDim.x);  // a cluster spans the grid's x
    const int bh = blockIdx.y, b = bh / a.Hk, hk = bh - b * a.Hk;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        *abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    sm100::wait_for_previous_kernel();

    const win::Seq seq = win::seq(a, b);
    win::Span y{0, 0, 0, 0, 0};
    if (seq.m > 0) y = win::span(a, seq, 0, seq.m);
    const int na = (y.a1 + kKeys - 1) / kKeys, nb = (y.b1 - y.b0 + kKeys - 1) / kKeys;
    auto tile = [&](int j, int& key0, int& end) {
        if (j < na) {
            key0 = j * kKeys;
            end = min(key0 + kKeys, y.a1);
        } else {
            key0 = y.b0 + (j - na) * kKeys;
            end = min(key0 + kKeys, y.b1);
        }
    };
    const int mine = (na + nb - rank + cs - 1) / cs;  // tiles rank, rank + cs, ...
    const size_t qrow = (size_t(b) * a.Hq + size_t(hk) * a.group) * a.Lq;  // rows of the group's heads are contiguous
    const int rows = a.group * a.Lq;

    float o[D / 8][4];
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    if (warp == kWarps) {
        if (lane == 0) {
            prefetch_tmap(&tmK);
            prefetch_tmap(&tmV);
            const int krow = bh * a.Lk;
            int i = 0;
            for (; i < mine; ++i) {
                const int s = i % kStages;
                if (!wait_bar(empty(s), ((i / kStages) & 1) ^ 1, abort, hdr, 301)) break;
                int key0, end;
                tile(rank + i * cs, key0, end);
                mbar_expect_tx(full(s), 2 * C::kTileBytes);
#pragma unroll
                for (int x = 0; x < C::kSlabs; ++x) {
                    tma_load_2d(base + s * C::kTileBytes + x * C::kSlabBytes, &tmK, full(s), 64 * x, krow + key0);
                    tma_load_2d(base + C::oV + s * C::kTileBytes + x * C::kSlabBytes, &tmV, full(s), 64 * x, krow + key0);
                }
            }
            // every issued copy lands before the ring is used for the join
            for (int k = i >= kStages ? i - kStages : 0; k < i; ++k) drain_bar(full(k % kStages), (k / kStages) & 1, hdr, 302);
        }
        __syncwarp();
    } else {
        // Q of the 16 rows as MMA A fragments (zeros past the last row)
        const int r0 = lane >> 2, c0 = (lane & 3) * 2;
        uint32_t q[D / 16][4];
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int r = r0 + (h & 1) * 8, c = 16 * k + c0 + (h >> 1) * 8;
                q[k][h] = r < rows ? *reinterpret_cast<const uint32_t*>(Q + (qrow + r) * D + c) : 0u;
            }
        }
        win::Row vis[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = r0 + 8 * h, t = r % a.Lq;
            vis[h] = win::Row{0, 0, 0};
            if (r < rows && t < seq.m) vis[h] = win::row(a, seq.n, t + seq.shift);
        }
        const float sl2 = a.scale * 1.4426950408889634f;
        const int k16 = warp * 16;  // this warp's keys of a tile
        for (int i = 0; i < mine; ++i) {
            const int s = i % kStages;
            int key0, end;
            tile(rank + i * cs, key0, end);
            if (!wait_bar_warp(full(s), (i / kStages) & 1, abort, hdr, 303)) break;
            const uint32_t kb = base + s * C::kTileBytes, vb = base + C::oV + s * C::kTileBytes;
            const int nv = end - key0 - k16;  // visible-run keys among this warp's 16
            if (nv > 0) {
                if (nv < 16) {  // V rows past the run: zeros, whatever was loaded
#pragma unroll
                    for (int x = lane; x < 16 * C::kSlabs * 8; x += 32) {
                        const int r = x / (C::kSlabs * 8), ch = x % (C::kSlabs * 8);
                        if (r >= nv)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                             vb + (ch >> 3) * C::kSlabBytes + (k16 + r) * 128 + (ch & 7) * 16), "r"(0u) : "memory");
                    }
                    fence_proxy_async_smem();  // before the slot's next copy
                    __syncwarp();
                }
                float sc[2][4] = {};
                {
                    const int key = k16 + (lane & 7) + ((lane >> 4) << 3);
                    float s2[2][4] = {};  // two chains over d
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int ch = 2 * k + ((lane >> 3) & 1);
                        uint32_t f0, f1, f2, f3;
                        ldmatrix_x4(kb + (ch >> 3) * C::kSlabBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4), f0, f1, f2, f3);
                        mma_bf16_16816((k & 1) ? s2[0] : sc[0], q[k], f0, f1);
                        mma_bf16_16816((k & 1) ? s2[1] : sc[1], q[k], f2, f3);
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sc[n][e] += s2[n][e];
                }
                // mask, running maximum over the row's 16 keys (four lanes a row)
                bool grow = false;
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float m = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = key0 + k16 + 8 * n + c0 + e;
                            const bool see = key < end && (key < vis[h].s || (key >= vis[h].lo && key < vis[h].hi));
                            float& v = sc[n][2 * h + e];
                            v = see ? v * sl2 : -INFINITY;
                            m = fmaxf(m, v);
                        }
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    alpha[h] = 1.f;
                    if (m > mx[h]) {
                        alpha[h] = mx[h] > -INFINITY ? ex2(mx[h] - m) : 1.f;  // nothing to rescale yet
                        mx[h] = m;
                        grow = true;
                    }
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= alpha[0];
                        o[n][1] *= alpha[0];
                        o[n][2] *= alpha[1];
                        o[n][3] *= alpha[1];
                    }
                }
                uint32_t pa[4];  // P as the A fragment: rows r0, r0 + 8; keys c0, c0 + 8
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float m0 = mx[h] > -INFINITY ? mx[h] : 0.f;
                    float l = 0.f;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = ex2(sc[n][2 * h] - m0), p1 = ex2(sc[n][2 * h + 1] - m0);
                        l += p0 + p1;
                        pa[2 * n + h] = pack_bf16(p0, p1);
                    }
                    sum[h] = sum[h] * alpha[h] + l;
                }
                const int key = k16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    const int ch = 2 * n + (lane >> 4);
                    uint32_t f0, f1, f2, f3;
                    ldmatrix_x4_trans(vb + (ch >> 3) * C::kSlabBytes + key * 128 + (((ch & 7) ^ (key & 7)) << 4), f0, f1, f2, f3);
                    mma_bf16_16816(o[2 * n], pa, f0, f1);
                    mma_bf16_16816(o[2 * n + 1], pa, f2, f3);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
        }
    }
    __syncthreads();  // every tile consumed, every copy landed: the ring is free

    // ---- join: warps, then CTAs -------------------------------------------------
    float* oj = reinterpret_cast<float*>(gbase);               // [warps + 1][16][kRow]
    float* mj = oj + (kWarps + 1) * kR * C::kRow;              // [warps + 1][16]
    float* lj = mj + (kWarps + 1) * kR;
    if (warp < kWarps) {
        const int r0 = lane >> 2, c0 = (lane & 3) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
            const int r = r0 + 8 * h;
            if (r < rows) {
                if ((lane & 3) == 0) {
                    mj[warp * kR + r] = mx[h];
                    lj[warp * kR + r] = sum[h];
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(oj + (warp * kR + r) * C::kRow + 8 * n + c0) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
            }
        }
    }
    __syncthreads();
    for (int x = tid; x < rows * D; x += kThreads) {
        const int r = x / D, c = x % D;
        float m = mj[r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, mj[w * kR + r]);
        const float m0 = m > -INFINITY ? m : 0.f;
        float v = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(mj[w * kR + r] - m0);
            v = fmaf(f, oj[(w * kR + r) * C::kRow + c], v);
            l = fmaf(f, lj[w * kR + r], l);
        }
        oj[(kWarps * kR + r) * C::kRow + c] = v;
        if (c == 0) {
            mj[kWarps * kR + r] = m;
            lj[kWarps * kR + r] = l;
        }
    }
    __syncwarp();
    cluster_sync();
    // each CTA finishes a share of the columns
    const int cols = D / cs;
    for (int x = tid; x < rows * cols; x += kThreads) {
        const int r = x / cols, c = rank * cols + x % cols, t = r % a.Lq;
        float m = -INFINITY, pm[kMaxCluster], pl[kMaxCluster], po[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            if (k >= cs) break;
            auto peer = [&](const float* p) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa(smem_u32(p), uint32_t(k))) : "memory");
                return v;
            };
            pm[k] = peer(mj + kWarps * kR + r);
            pl[k] = peer(lj + kWarps * kR + r);
            po[k] = peer(oj + (kWarps * kR + r) * C::kRow + c);
            m = fmaxf(m, pm[k]);
        }
        const float m0 = m > -INFINITY ? m : 0.f;
        float v = 0.f, l = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            if (k >= cs) break;
            const float f = ex2(pm[k] - m0);
            v = fmaf(f, po[k], v);
            l = fmaf(f, pl[k], l);
        }
        if (t >= seq.m && !a.fill) continue;  // rows past the last stay as they were
        const bool seen = l > 0.f || l != l;  // NaN stays NaN
        O[(qrow + r) * D + c] = __float2bfloat16_rn(seen ? v / l : 0.f);
        if (c == 0 && lse) lse[qrow + r] = seen ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its shared memory is read
}

template <int D>
cudaError_t launch_d(const WinArgs& a, const void* Q, const void* K, const void* V, void* O, float* lse,
                     cudaStream_t s) {
    int32_t* hdr = nullptr;
    cudaError_t e = window_error_word(&hdr);
    if (e != cudaSuccess) return e;
    CUtensorMap tmK, tmV;
    const int64_t krows = int64_t(a.B) * a.Hk * a.Lk;
    if (!make_tmap_box(&tmK, K, D, krows, kKeys) || !make_tmap_box(&tmV, V, D, krows, kKeys)) return cudaErrorInvalidValue;
    const int smem = Cfg<D>::kSmem;
    e = cudaFuncSetAttribute(window_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int sms = multiprocessors();
    // Split the keys over a cluster until there are four CTAs an SM (two are resident;
    // the others even out streams of unlike lengths), while every CTA keeps two tiles.
    const int64_t heads = int64_t(a.B) * a.Hk;
    const int64_t keys = a.left == kWinOpen || a.right == kWinOpen
                             ? a.Lk
                             : int64_t(a.left) + a.right + a.Lq + a.sinks;
    const int64_t tiles = ((keys < a.Lk ? keys : a.Lk) + kKeys - 1) / kKeys;
    int cs = 1;
    while (cs < kMaxCluster && heads * cs < 4 * int64_t(sms) && tiles >= 4 * cs) cs *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(cs), unsigned(heads));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(cs);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // wait_for_previous_kernel
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, window_few_kernel<D>, tmK, tmV, a, static_cast<const __nv_bfloat16*>(Q),
                           static_cast<__nv_bfloat16*>(O), lse, hdr);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_few(const WinArgs& a, int d, const void* Q, const void* K, const void* V, void* O,
                              float* lse, cudaStream_t s) {
    return d == 128 ? launch_d<128>(a, Q, K, V, O, lse, s) : launch_d<64>(a, Q, K, V, O, lse, s);
}

}  // namespace moc
