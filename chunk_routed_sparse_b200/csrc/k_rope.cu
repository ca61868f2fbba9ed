// Row operators in front of the attention: rotary positions, per-head RMS norms
// of queries and keys with the rotation in the same pass, and their gradients.
//
//   norm:     xhat = x r,  r = 1 / sqrt(mean(x^2) + eps),  z = xhat * w
//   rotation: (a, b) -> (a c - b s, a s + b c) on every pair, c = f cos(p w_i),
//             s = f sin(p w_i) for the token's position p on the pair's axis
//   gradient: g = R^T dy,  dw = sum over rows of g * xhat,
//             dx = r (g w - xhat mean(g w xhat))
//
// All of it is memory-bound: the input is read once and the output written once,
// and the re-layout from a projection's token-major rows to the attention's
// head-major ones costs nothing more. A group of d / 8 lanes holds one row, eight
// elements a lane, in registers; a group keeps one token and walks the heads, so
// that the token's cosines and sines are formed once for all of them. Four rows
// are requested before the first is used. Many small CTAs (128 threads: 8 or 16
// tokens, eight an SM) hide the memory's latency: 256 threads cost 9 % on the
// eight-shot projection (1.15 against 1.05 ms), requesting the next rows ahead costs
// more registers than it gives, and addressing every row anew costs 8 % (a third of
// the issue slots are in use). Outputs are streaming stores: nothing here reads them.
// At the measured copy bandwidth: the eight-shot projection (6.65 GB) in 1.03-1.05 ms;
// the single-shot rotation (102 MB in, 102 MB out) in 35 us against 32 us.
//
// Angles: the position times a 64-bit fraction of a turn, modulo 2^64, is exact
// for every 32-bit position (an fp32 product loses 0.01 rad at position 180,000);
// the top 32 bits go to sincospif.
#include <cuda_fp16.h>

#include "common.cuh"
#include "rope.cuh"
#include "sm100.cuh"

namespace moc {
namespace {

constexpr int kThreads = 128;
constexpr int kBwdCtas = 5;  // resident CTAs of the backward kernel an SM
constexpr int kRows = 4;  // rows of one lane group in flight

// ---- eight elements of a row -------------------------------------------------
template <typename T>
struct Raw {
    static constexpr int kWords = 8 * sizeof(T) / 4;
    uint32_t w[kWords];
};

template <typename T, bool AL>
__device__ __forceinline__ void load_raw(const T* p, Raw<T>& r) {
    if constexpr (AL) {  // (not the read-only path: the output may be the input itself)
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; i += 4) ld16(reinterpret_cast<const uint32_t*>(p) + i, r.w + i);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = *reinterpret_cast<const volatile uint32_t*>(p + i);
    } else {
        const volatile uint16_t* q = reinterpret_cast<const volatile uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = uint32_t(q[2 * i]) | (uint32_t(q[2 * i + 1]) << 16);
    }
}

template <typename T, bool AL>
__device__ __forceinline__ void store_raw(T* p, const Raw<T>& r) {
    if constexpr (AL) {
#pragma unroll
        for (int i = 0; i < Raw<T>::kWords; i += 4)
            __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + i),
                   make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            reinterpret_cast<uint16_t*>(p)[2 * i] = uint16_t(r.w[i]);
            reinterpret_cast<uint16_t*>(p)[2 * i + 1] = uint16_t(r.w[i] >> 16);
        }
    }
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16lo(r.w[i]);
            v[2 * i + 1] = bf16hi(r.w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void pack(const float (&v)[8], Raw<T>& r) {  // the one rounding, to nearest even
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = __float_as_uint(v[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
}

template <typename T>
__device__ __forceinline__ float one(const T* p, int i) {
    if constexpr (sizeof(T) == 4) return p[i];
    else if constexpr (std::is_same<T, __half>::value) return __half2float(p[i]);
    else return __bfloat162float(p[i]);
}

template <typename T>
__device__ __forceinline__ float weight(const void* w, int w_fp32, int e) {
    return w == nullptr ? 1.f : w_fp32 ? static_cast<const float*>(w)[e] : one(static_cast<const T*>(w), e);
}

// sum of eight products, on packed fp32 pairs
__device__ __forceinline__ float dot8(const float (&x)[8], const float (&y)[8]) {
    uint64_t s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        s = sm100::f2_fma(sm100::f2_pack(x[2 * j], x[2 * j + 1]), sm100::f2_pack(y[2 * j], y[2 * j + 1]), s);
    float lo, hi;
    sm100::f2_unpack(s, lo, hi);
    return lo + hi;
}

// sum over the LPR lanes of a row
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o, LPR);
    return x;
}

// ---- rotation ----------------------------------------------------------------
// A lane's cosines and sines. Interleaved: four pairs of its own elements. Half:
// one pair an element, the sine signed for the element's side of the pair.
template <bool HALF>
struct Trig {
    static constexpr int kN = HALF ? 8 : 4;
    float c[kN], s[kN];
};

template <bool HALF>
__device__ __forceinline__ void trig(const RowArgs& a, const uint64_t* turn, const uint8_t* axis, int b, int l, int e0,
                                     Trig<HALF>& t) {
    const int n = a.rope.pairs;
#pragma unroll
    for (int j = 0; j < Trig<HALF>::kN; ++j) {
        int i;
        bool hi = false;
        if (HALF) {
            i = e0 + j;
            hi = i >= n;
            if (hi) i -= n;
        } else {
            i = e0 / 2 + j;
        }
        t.c[j] = 1.f;
        t.s[j] = 0.f;
        if (i < n) {
            const int64_t p = a.pos ? int64_t(a.pos[b * a.pos_b + axis[i] * a.pos_a + l]) : int64_t(l);
            const uint64_t turns = uint64_t(p) * turn[i];
            // top 32 bits as a signed fraction of a turn, in half turns [-1, 1)
            const float x = float(int32_t(turns >> 32)) * 4.656612873077393e-10f;
            float s, c;
            sincospif(x, &s, &c);
            t.c[j] = c * a.rope.factor;
            t.s[j] = s * a.rope.factor * ((HALF && !hi) ? -a.sign : a.sign);
        }
    }
}

// Rotate a row in place. Elements past the rotated part keep their values (they
// are not multiplied by one: an infinity in a partner would make that a NaN).
template <int LPR, bool HALF>
__device__ __forceinline__ void rotate(float (&v)[8], const Trig<HALF>& t, int n, int r, int e0) {
    if constexpr (!HALF) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (e0 / 2 + p < n) {
                const float x = v[2 * p], y = v[2 * p + 1];
                v[2 * p] = x * t.c[p] - y * t.s[p];
                v[2 * p + 1] = x * t.s[p] + y * t.c[p];
            }
        }
    } else {
        float o[8];
        const int s = n & 7;
        if (s == 0) {  // a lane's partners are one other lane's elements
            const int src = e0 >= 2 * n ? r : (e0 < n ? r + (n >> 3) : r - (n >> 3));
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(0xffffffffu, v[j], src, LPR);
        } else {
            // partners lie across two lanes: every lane offers its registers turned by
            // s (three select steps), once in each direction
            float up[8], dn[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) up[j] = dn[j] = v[j];
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) {
                float u[8], d[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    u[j] = (s & k) ? up[(j + k) & 7] : up[j];
                    d[j] = (s & k) ? dn[(j - k) & 7] : dn[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) up[j] = u[j], dn[j] = d[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float hi = __shfl_sync(0xffffffffu, up[j], ((e0 + j + n) >> 3) & (LPR - 1), LPR);
                const float lo = __shfl_sync(0xffffffffu, dn[j], ((e0 + j - n + 8 * LPR) >> 3) & (LPR - 1), LPR);
                o[j] = e0 + j < n ? hi : lo;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e0 + j < 2 * n) v[j] = v[j] * t.c[j] + o[j] * t.s[j];
    }
}

__device__ __forceinline__ void tab_to_smem(const RowArgs& a, uint64_t* turn, uint8_t* axis) {
    if (threadIdx.x < kMaxRopePairs && int(threadIdx.x) < a.rope.pairs) {
        turn[threadIdx.x] = a.rope.turn[threadIdx.x];
        axis[threadIdx.x] = a.rope.axis[threadIdx.x];
    }
    __syncthreads();
}

// ---- forward (and the rotation's transpose, with sign = -1) -------------------
template <typename T, int D, bool HALF, bool AL>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(const __grid_constant__ RowArgs a) {
    constexpr int LPR = D / 8, TPC = kThreads / LPR;
    __shared__ uint64_t turn[kMaxRopePairs];
    __shared__ uint8_t axis[kMaxRopePairs];
    const int r = threadIdx.x % LPR, e0 = 8 * r;
    const int64_t tok = int64_t(blockIdx.x) * TPC + threadIdx.x / LPR;
    const bool live = tok < a.tokens;  // lanes past the last token work on it again and store nothing
    const int t = live ? int(tok) : a.tokens - 1;
    const int b = t / a.L, l = t - b * a.L;
    const int h_lo = blockIdx.y * a.heads_per_cta, h_hi = min(h_lo + a.heads_per_cta, a.heads);
    // the CTA's first rows are requested before the angles are formed
    int k0 = 0, base = 0;
    while (h_lo >= base + a.sec[k0].H) base += a.sec[k0++].H;
    sm100::let_next_kernel_start();
    sm100::wait_for_previous_kernel();
    Raw<T> raw[kRows];
    {
        const RowSec& sec = a.sec[k0];
        const T* x = static_cast<const T*>(sec.x) + b * sec.xs[0] + l * sec.xs[2] + e0 + (h_lo - base) * sec.xs[1];
        const int n = min(h_hi - h_lo, sec.H - (h_lo - base));
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (u < n) load_raw<T, AL>(x + u * sec.xs[1], raw[u]);
    }
    tab_to_smem(a, turn, axis);
    Trig<HALF> tr;
    trig<HALF>(a, turn, axis, b, l, e0, tr);
#pragma unroll 1
    for (int k = k0; k < 3; ++k) {
        const RowSec& sec = a.sec[k];
        const int lo = max(h_lo - base, 0), hi = min(h_hi - base, sec.H);
        base += sec.H;
        if (lo >= hi) continue;
        const T* x = static_cast<const T*>(sec.x) + b * sec.xs[0] + l * sec.xs[2] + e0;
        T* y = static_cast<T*>(sec.y) + b * sec.ys[0] + l * sec.ys[2] + e0;
        float w[8];
        if (sec.mode == ROW_NORM) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = weight<T>(sec.w, a.w_fp32, e0 + j);
        }
#pragma unroll 1
        for (int h = lo; h < hi; h += kRows) {
            if (k > k0 || h > lo) {
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (h + u < hi) load_raw<T, AL>(x + (h + u) * sec.xs[1], raw[u]);
            }
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (h + u >= hi) break;
                if (sec.mode != ROW_COPY) {
                    float v[8];
                    unpack<T>(raw[u], v);
                    if (sec.mode == ROW_NORM) {
                        const float rs = rsqrtf(row_sum<LPR>(dot8(v, v)) * (1.f / D) + a.eps);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = v[j] * rs * w[j];
                    }
                    rotate<LPR, HALF>(v, tr, a.rope.pairs, r, e0);
                    pack<T>(v, raw[u]);
                }
                if (live) store_raw<T, AL>(y + (h + u) * sec.ys[1], raw[u]);
            }
        }
    }
}

// ---- backward of norm + rotation ---------------------------------------------
// A persistent CTA strides over token tiles, one tensor after the other (one
// weight's partial gradient in registers at a time); the parts of a CTA are added
// through shared memory in thread order and those of all CTAs by rows_dw_kernel in
// CTA order: no atomics. Rows come in steps of two, copied by cp.async into slots of
// shared memory that belong to the thread that reads them (no barrier), up to three
// steps ahead: loads into registers leave 16 warps an SM idle between their rounds
// (163 us on the single-shot step against 138 us; its bytes take 126 us at the
// measured copy rate). Rows off 16-byte boundaries are loaded when they are used.
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <typename T, int D, bool HALF, bool AL>
__global__ void __launch_bounds__(kThreads, kBwdCtas) rows_bwd_kernel(const __grid_constant__ RowArgs a) {
    constexpr int LPR = D / 8, TPC = kThreads / LPR, RS = 2;
    constexpr int W = sizeof(T) / 2;              // 16-byte words of a lane's eight elements
    constexpr int ST = sizeof(T) == 4 ? 2 : 4;    // steps in the ring
    __shared__ uint64_t turn[kMaxRopePairs];
    __shared__ uint8_t axis[kMaxRopePairs];
    __shared__ __align__(16) float ws[D];
    __shared__ float red[TPC][D];
    __shared__ __align__(16) uint4 ring[AL ? ST * RS * 2 * W * kThreads : 1];
    sm100::let_next_kernel_start();
    tab_to_smem(a, turn, axis);
    sm100::wait_for_previous_kernel();
    const int r = threadIdx.x % LPR, e0 = 8 * r;
    const int h_lo = blockIdx.y * a.heads_per_cta, h_hi = min(h_lo + a.heads_per_cta, a.heads);
    const int64_t step = int64_t(gridDim.x) * TPC, first = int64_t(blockIdx.x) * TPC;
    // slot of (stage, row of the step, tensor): word w of this thread
    const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16;
    auto slot = [&](int st, int u, int x) { return slot0 + uint32_t(((st * RS + u) * 2 + x) * W) * (kThreads * 16); };
    auto at = [&](const int64_t (&st)[3], int64_t t0) -> int64_t {  // a tile's token of this lane group
        const int64_t tok = t0 + threadIdx.x / LPR;
        const int t = tok < a.tokens ? int(tok) : a.tokens - 1;
        const int b = t / a.L;
        return b * st[0] + (t - b * a.L) * st[2] + e0;
    };
    int base = 0;
#pragma unroll 1
    for (int k = 0; k < 3; ++k) {
        const RowSec& sec = a.sec[k];
        const int lo = max(h_lo - base, 0), hi = min(h_hi - base, sec.H);
        base += sec.H;
        if (k == 2) {  // values: the gradient only changes its layout
#pragma unroll 1
            for (int64_t t0 = first; lo < hi && t0 < a.tokens; t0 += step) {
                const T* g = static_cast<const T*>(sec.g) + at(sec.gs, t0);
                T* y = static_cast<T*>(sec.y) + at(sec.ys, t0);
                const bool live = t0 + threadIdx.x / LPR < a.tokens;
#pragma unroll 1
                for (int h = lo; h < hi; h += kRows) {
                    Raw<T> raw[kRows];
#pragma unroll
                    for (int u = 0; u < kRows; ++u)
                        if (h + u < hi) load_raw<T, AL>(g + (h + u) * sec.gs[1], raw[u]);
#pragma unroll
                    for (int u = 0; u < kRows; ++u)
                        if (h + u < hi && live) store_raw<T, AL>(y + (h + u) * sec.ys[1], raw[u]);
                }
            }
            continue;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kThreads) ws[i] = weight<T>(sec.w, a.w_fp32, i);
        __syncthreads();
        float dw[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = 0.f;
        // the next step to request: tile pt, head ph
        int64_t pt = first;
        int ph = lo, pst = 0;
        const T *px = nullptr, *pg = nullptr;
        auto rows_at = [&](int64_t t0) {
            px = static_cast<const T*>(sec.x) + at(sec.xs, t0);
            pg = static_cast<const T*>(sec.g) + at(sec.gs, t0);
        };
        auto request = [&]() {
            if constexpr (AL) {
                if (pt < a.tokens) {
#pragma unroll
                    for (int u = 0; u < RS; ++u) {
                        if (ph + u >= hi) break;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            cp_async16(slot(pst, u, 0) + w * (kThreads * 16), reinterpret_cast<const uint4*>(px + (ph + u) * sec.xs[1]) + w, 16);
                            cp_async16(slot(pst, u, 1) + w * (kThreads * 16), reinterpret_cast<const uint4*>(pg + (ph + u) * sec.gs[1]) + w, 16);
                        }
                    }
                    ph += RS;
                    if (ph >= hi) {
                        ph = lo;
                        pt += step;
                        if (pt < a.tokens) rows_at(pt);
                    }
                }
                cp_async_commit();
                pst = pst + 1 == ST ? 0 : pst + 1;
            }
        };
        if (lo < hi) {
            if (first < a.tokens) rows_at(first);
#pragma unroll
            for (int i = 0; i < ST - 1; ++i) request();
        }
        int st = 0;
#pragma unroll 1
        for (int64_t t0 = first; lo < hi && t0 < a.tokens; t0 += step) {
            const int64_t tok = t0 + threadIdx.x / LPR;
            const bool live = tok < a.tokens;
            const int t = live ? int(tok) : a.tokens - 1;
            const int b = t / a.L, l = t - b * a.L;
            T* y = static_cast<T*>(sec.y) + b * sec.ys[0] + l * sec.ys[2] + e0;
            if (!AL) rows_at(t0);
            Trig<HALF> tr;
            trig<HALF>(a, turn, axis, b, l, e0, tr);
#pragma unroll 1
            for (int h = lo; h < hi; h += RS) {
                Raw<T> rx[RS], rg[RS];
                if constexpr (AL) {
                    request();
                    cp_async_wait<ST - 1>();
#pragma unroll
                    for (int u = 0; u < RS; ++u) {
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const uint4 vx = lds16(slot(st, u, 0) + w * (kThreads * 16)), vg = lds16(slot(st, u, 1) + w * (kThreads * 16));
                            rx[u].w[4 * w] = vx.x, rx[u].w[4 * w + 1] = vx.y, rx[u].w[4 * w + 2] = vx.z, rx[u].w[4 * w + 3] = vx.w;
                            rg[u].w[4 * w] = vg.x, rg[u].w[4 * w + 1] = vg.y, rg[u].w[4 * w + 2] = vg.z, rg[u].w[4 * w + 3] = vg.w;
                        }
                    }
                    st = st + 1 == ST ? 0 : st + 1;
                } else {
#pragma unroll
                    for (int u = 0; u < RS; ++u) {
                        if (h + u < hi) {
                            load_raw<T, AL>(px + (h + u) * sec.xs[1], rx[u]);
                            load_raw<T, AL>(pg + (h + u) * sec.gs[1], rg[u]);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < RS; ++u) {
                    if (h + u >= hi) break;
                    float v[8], q[8], w[8];
                    unpack<T>(rx[u], v);
                    unpack<T>(rg[u], q);
                    rotate<LPR, HALF>(q, tr, a.rope.pairs, r, e0);
                    const float4 wa = *reinterpret_cast<const float4*>(&ws[e0]), wb = *reinterpret_cast<const float4*>(&ws[e0 + 4]);
                    w[0] = wa.x * q[0], w[1] = wa.y * q[1], w[2] = wa.z * q[2], w[3] = wa.w * q[3];  // g w
                    w[4] = wb.x * q[4], w[5] = wb.y * q[5], w[6] = wb.z * q[6], w[7] = wb.w * q[7];
                    const float ss = row_sum<LPR>(dot8(v, v)), sg = row_sum<LPR>(dot8(w, v));
                    const float rs = rsqrtf(ss * (1.f / D) + a.eps);
                    const float m = sg * rs * (1.f / D);  // mean(g w xhat)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float xh = v[j] * rs;
                        if (live) dw[j] = fmaf(q[j], xh, dw[j]);
                        v[j] = rs * (w[j] - xh * m);
                    }
                    Raw<T> ry;
                    pack<T>(v, ry);
                    if (live) store_raw<T, AL>(y + (h + u) * sec.ys[1], ry);
                }
            }
        }
        if constexpr (AL) cp_async_wait<0>();
        if (a.part == nullptr) continue;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) red[threadIdx.x / LPR][e0 + j] = dw[j];
        __syncthreads();
        if (threadIdx.x < D) {  // kThreads >= D
            float s = 0.f;
            for (int i = 0; i < TPC; ++i) s += red[i][threadIdx.x];
            a.part[((size_t(blockIdx.y) * gridDim.x + blockIdx.x) * 2 + k) * D + threadIdx.x] = s;
        }
    }
}

// dw = sum of the CTAs' parts: one CTA per weight and 32 columns, 32 runs of parts
// added in order, then the runs in order.
template <typename W>
__global__ void __launch_bounds__(1024) rows_dw_kernel(int ctas, int D, const float* part, W* dwq, W* dwk) {
    __shared__ float red[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    sm100::wait_for_previous_kernel();
    W* out = blockIdx.y == 0 ? dwq : dwk;
    const int c = blockIdx.x * 32 + tx;
    float s = 0.f;
#pragma unroll 8
    for (int i = ty; i < ctas; i += 32) s += part[(size_t(i) * 2 + blockIdx.y) * D + c];
    red[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && out) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) s += red[i][tx];
        if constexpr (sizeof(W) == 4) out[c] = s;
        else if constexpr (std::is_same<W, __half>::value) out[c] = __float2half_rn(s);
        else out[c] = __float2bfloat16_rn(s);
    }
}

// fn<T, D, HALF, AL>(args...) for the runtime type, width, pair layout and alignment
#define MOC_ROWS_DISPATCH(CALL)                                                     \
    do {                                                                            \
        const bool half = !a.rope.interleaved;                                      \
        if (dtype == MOC_BF16) MOC_ROWS_D(__nv_bfloat16, CALL);                     \
        else if (dtype == MOC_FP16) MOC_ROWS_D(__half, CALL);                       \
        else MOC_ROWS_D(float, CALL);                                               \
    } while (0)
#define MOC_ROWS_D(T, CALL)                                                         \
    do {                                                                            \
        if (d == 128) MOC_ROWS_H(T, 128, CALL); else MOC_ROWS_H(T, 64, CALL);       \
    } while (0)
#define MOC_ROWS_H(T, D, CALL)                                                      \
    do {                                                                            \
        if (half) { if (aligned) CALL(T, D, true, true); else CALL(T, D, true, false); }       \
        else { if (aligned) CALL(T, D, false, true); else CALL(T, D, false, false); }          \
    } while (0)

}  // namespace

// Token tiles on x (at most `most`, CTAs stride over the rest), heads split on y into
// as many shares as keep all CTAs within `want`, one round of resident ones (a second,
// nearly empty round costs the odd padded batch's gradient 10 %: 22.2 against 20.2 us);
// a split forms the token's cosines again.
static dim3 rows_grid(int d, int64_t tokens, int heads, int64_t want, int64_t most, int* heads_per_cta) {
    const int64_t tpc = kThreads * 8 / d;
    int64_t tiles = (tokens + tpc - 1) / tpc;
    int64_t split = tiles >= want ? 1 : want / tiles;
    if (split > heads) split = heads;
    *heads_per_cta = int((heads + split - 1) / split);
    if (tiles > most) tiles = most;
    return dim3(unsigned(tiles), unsigned((heads + *heads_per_cta - 1) / *heads_per_cta));
}

static dim3 rows_bwd_grid(int d, int64_t tokens, int heads, int* heads_per_cta) {
    const int64_t n = kBwdCtas * int64_t(sm100::multiprocessors());
    return rows_grid(d, tokens, heads, n, n, heads_per_cta);
}

cudaError_t launch_rows_fwd(int dtype, int d, bool aligned, const RowArgs& args, cudaStream_t s) {
    RowArgs a = args;
    const dim3 grid = rows_grid(d, a.tokens, a.heads, 8 * int64_t(sm100::multiprocessors()), INT64_MAX, &a.heads_per_cta);
#define MOC_CALL(T, D, HALF, AL) e = sm100::launch_after(rows_fwd_kernel<T, D, HALF, AL>, grid, kThreads, 0, s, a)
    cudaError_t e = cudaSuccess;
    MOC_ROWS_DISPATCH(MOC_CALL);
#undef MOC_CALL
    return e;
}

int rows_bwd_ctas(int d, int64_t tokens, int heads) {
    int per;
    const dim3 g = rows_bwd_grid(d, tokens, heads, &per);
    return int(g.x * g.y);
}

cudaError_t launch_rows_bwd(int dtype, int d, bool aligned, const RowArgs& args, cudaStream_t s) {
    RowArgs a = args;
    const dim3 grid = rows_bwd_grid(d, a.tokens, a.heads, &a.heads_per_cta);
#define MOC_CALL(T, D, HALF, AL) e = sm100::launch_after(rows_bwd_kernel<T, D, HALF, AL>, grid, kThreads, 0, s, a)
    cudaError_t e = cudaSuccess;
    MOC_ROWS_DISPATCH(MOC_CALL);
#undef MOC_CALL
    return e;
}

cudaError_t launch_rows_dw(int dtype, int w_fp32, int d, int ctas, const float* part, void* dwq, void* dwk,
                           cudaStream_t s) {
    const dim3 grid(d / 32, 2);
    if (w_fp32 || dtype == MOC_FP32)
        return sm100::launch_after(rows_dw_kernel<float>, grid, 1024, 0, s, ctas, d, part, static_cast<float*>(dwq),
                                   static_cast<float*>(dwk));
    if (dtype == MOC_FP16)
        return sm100::launch_after(rows_dw_kernel<__half>, grid, 1024, 0, s, ctas, d, part, static_cast<__half*>(dwq),
                                   static_cast<__half*>(dwk));
    return sm100::launch_after(rows_dw_kernel<__nv_bfloat16>, grid, 1024, 0, s, ctas, d, part,
                               static_cast<__nv_bfloat16*>(dwq), static_cast<__nv_bfloat16*>(dwk));
}

}  // namespace moc
