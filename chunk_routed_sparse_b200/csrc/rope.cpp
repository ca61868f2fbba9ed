// Rotary plans and the C entry points of the row operators (rotary positions,
// normalised and rotated queries and keys, and their gradients): argument
// validation and launches.
#include <cmath>
#include <new>

#include "rope.cuh"

namespace {

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

moc_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOC_OK : MOC_ERR_CUDA; }

bool finite_positive(double x) { return std::isfinite(x) && x > 0.0; }

size_t elem_bytes(int dtype) { return dtype == MOC_FP32 ? 4 : 2; }

// Checks of one tensor [B][H][L][d] with strides in elements; clears *al when a row
// of it does not start on a 16-byte boundary.
bool check_tensor(const void* p, const int64_t* st, int dtype, int B, int H, int64_t L, bool written, bool* al) {
    if (!p || !st) return false;
    const size_t eb = elem_bytes(dtype);
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % eb) return false;
    if (a & 15) *al = false;
    const int64_t n[3] = {B, H, L};
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;  // never multiplied by anything but zero
        if (st[i] < 0 || (written && st[i] == 0)) return false;
        if (uint64_t(st[i]) >= (uint64_t(1) << 40)) return false;
        if ((uint64_t(st[i]) * eb) & 15) *al = false;
    }
    return true;
}

void set_strides(int64_t* dst, const int64_t* src, int B, int H, int64_t L) {
    dst[0] = B > 1 ? src[0] : 0;
    dst[1] = H > 1 ? src[1] : 0;
    dst[2] = L > 1 ? src[2] : 0;
}

moc_status check_rows(const moc_rope* rope, int dtype, int B, int64_t heads, int64_t L, int d, const int32_t* pos,
                      int64_t pos_b, int64_t pos_a) {
    if (dtype != MOC_BF16 && dtype != MOC_FP16 && dtype != MOC_FP32) return MOC_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return MOC_ERR_INVALID_ARG;
    if (B < 0 || heads < 0 || L < 0) return MOC_ERR_INVALID_ARG;
    if (rope) {
        if (2 * rope->tab.pairs > d) return MOC_ERR_INVALID_ARG;
        if (!pos && rope->tab.axes != 1) return MOC_ERR_INVALID_ARG;
        if (pos && ((reinterpret_cast<uintptr_t>(pos) & 3) || pos_b < 0 || pos_a < 0)) return MOC_ERR_INVALID_ARG;
    }
    if (heads > 65535 || L > 0x7fffffff || int64_t(B) * L > 0x7fffff00) return MOC_ERR_UNSUPPORTED;
    return MOC_OK;
}

void common_args(moc::RowArgs& a, const moc_rope* rope, int B, int64_t heads, int64_t L, const int32_t* pos,
                 int64_t pos_b, int64_t pos_a, float sign) {
    if (rope) {
        a.rope = rope->tab;
        a.pos = pos;
        a.pos_b = B > 1 ? pos_b : 0;
        a.pos_a = rope->tab.axes > 1 ? pos_a : 0;
    } else {
        a.rope.interleaved = 1;  // no pairs: the norm alone
    }
    a.L = int32_t(L);
    a.tokens = int32_t(B * L);
    a.heads = int32_t(heads);
    a.sign = sign;
}

}  // namespace

extern "C" moc_status moc_build_rope(const moc_rope_desc* d, moc_rope** out) {
    if (!out) return MOC_ERR_INVALID_ARG;
    *out = nullptr;
    if (!d || !d->axis_dim || d->n_axes < 1 || d->n_axes > moc::kMaxRopeAxes) return MOC_ERR_INVALID_ARG;
    if (d->interleaved != 0 && d->interleaved != 1) return MOC_ERR_INVALID_ARG;
    if (!std::isfinite(d->theta) || d->theta <= 1.0) return MOC_ERR_INVALID_ARG;
    if (d->scaling < MOC_ROPE_PLAIN || d->scaling > MOC_ROPE_YARN) return MOC_ERR_INVALID_ARG;
    if (d->scaling != MOC_ROPE_PLAIN && !(std::isfinite(d->factor) && d->factor >= 1.0)) return MOC_ERR_INVALID_ARG;
    if (d->scaling == MOC_ROPE_YARN &&
        (!finite_positive(d->original_length) || !finite_positive(d->alpha) || !std::isfinite(d->beta) ||
         d->beta <= d->alpha || !std::isfinite(d->attention_factor) || d->attention_factor < 0.0))
        return MOC_ERR_INVALID_ARG;
    int total = 0;
    for (int a = 0; a < d->n_axes; ++a) {
        const int n = d->axis_dim[a];
        if (n < 2 || (n & 1) || n > 2 * moc::kMaxRopePairs) return MOC_ERR_INVALID_ARG;
        total += n;
    }
    if (total > 2 * moc::kMaxRopePairs) return MOC_ERR_INVALID_ARG;
    moc_rope* r = new (std::nothrow) moc_rope();
    if (!r) return MOC_ERR_UNSUPPORTED;
    const long double two_pi = 6.283185307179586476925286766559005768L;
    const long double s = d->scaling == MOC_ROPE_PLAIN ? 1.0L : (long double)d->factor;
    int i = 0;
    for (int a = 0; a < d->n_axes; ++a) {
        const int n = d->axis_dim[a];
        long double theta = d->theta;
        if (d->scaling == MOC_ROPE_NTK && n > 2) theta *= powl(s, (long double)n / (n - 2));
        const long double ratio = powl(theta, -2.0L / n);
        long double plain = 1.0L;  // theta^(-2 j / n): 63 products in 64 bits lose nothing that fp64 shows
        for (int j = 0; j < n / 2; ++j, ++i, plain *= ratio) {
            long double w = plain;
            if (d->scaling == MOC_ROPE_LINEAR) w /= s;
            if (d->scaling == MOC_ROPE_YARN) {
                const long double turns = (long double)d->original_length * w / two_pi;
                long double keep = (turns - d->alpha) / ((long double)d->beta - d->alpha);
                keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
                w = keep * w + (1 - keep) * w / s;
            }
            r->freq[i] = double(w);
            r->tab.turn[i] = uint64_t(w / two_pi * 18446744073709551616.0L + 0.5L);  // w <= 1: at most 2^64 / (2 pi)
            r->tab.axis[i] = uint8_t(a);
        }
    }
    r->factor = 1.0;
    if (d->scaling == MOC_ROPE_YARN)
        r->factor = d->attention_factor > 0.0 ? d->attention_factor : 0.1 * std::log(d->factor) + 1.0;
    r->tab.pairs = total / 2;
    r->tab.interleaved = d->interleaved;
    r->tab.axes = d->n_axes;
    r->tab.factor = float(r->factor);
    *out = r;
    return MOC_OK;
}

extern "C" void moc_rope_destroy(moc_rope* rope) { delete rope; }

extern "C" moc_status moc_rope_table(const moc_rope* rope, double* freq, int32_t* axis, int64_t cap, int64_t* count,
                                     double* factor) {
    if (!rope || !count || cap < 0 || (cap > 0 && !freq && !axis)) return MOC_ERR_INVALID_ARG;
    *count = rope->tab.pairs;
    if (factor) *factor = rope->factor;
    for (int64_t i = 0; i < rope->tab.pairs && i < cap; ++i) {
        if (freq) freq[i] = rope->freq[i];
        if (axis) axis[i] = rope->tab.axis[i];
    }
    return MOC_OK;
}

extern "C" moc_status moc_rotary(const moc_rope* rope, int dtype, int B, int H, int64_t L, int d, const void* X,
                                 const int64_t* x_strides, const int32_t* pos, int64_t pos_batch, int64_t pos_axis,
                                 int transpose, void* Y, const int64_t* y_strides, moc_stream_t stream) {
    if (!rope) return MOC_ERR_INVALID_ARG;
    moc_status st = check_rows(rope, dtype, B, H, L, d, pos, pos_batch, pos_axis);
    if (st != MOC_OK) return st;
    if (B == 0 || H == 0 || L == 0) return MOC_OK;
    bool al = true;
    if (!check_tensor(X, x_strides, dtype, B, H, L, false, &al) || !check_tensor(Y, y_strides, dtype, B, H, L, true, &al))
        return MOC_ERR_INVALID_ARG;
    moc::RowArgs a{};
    common_args(a, rope, B, H, L, pos, pos_batch, pos_axis, transpose ? -1.f : 1.f);
    moc::RowSec& s = a.sec[0];
    s.x = X;
    s.y = Y;
    set_strides(s.xs, x_strides, B, H, L);
    set_strides(s.ys, y_strides, B, H, L);
    s.H = H;
    s.mode = moc::ROW_ROPE;
    return cuda_status(moc::launch_rows_fwd(dtype, d, al, a, (cudaStream_t)stream));
}

extern "C" moc_status moc_qk_norm_rope(const moc_rope* rope, int dtype, int B, int Hq, int Hk, int64_t L, int d,
                                       const void* Q, const int64_t* q_strides, const void* K, const int64_t* k_strides,
                                       const void* V, const int64_t* v_strides, const void* wq, const void* wk,
                                       int w_dtype, float eps, const int32_t* pos, int64_t pos_batch, int64_t pos_axis,
                                       void* Qo, const int64_t* qo_strides, void* Ko, const int64_t* ko_strides,
                                       void* Vo, const int64_t* vo_strides, moc_stream_t stream) {
    if (Hq < 0 || Hk < 0) return MOC_ERR_INVALID_ARG;
    const int64_t heads = int64_t(Hq) + Hk + (V ? Hk : 0);
    moc_status st = check_rows(rope, dtype, B, heads, L, d, pos, pos_batch, pos_axis);
    if (st != MOC_OK) return st;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return MOC_ERR_INVALID_ARG;
    if ((wq || wk) && w_dtype != MOC_FP32 && w_dtype != dtype) return MOC_ERR_INVALID_ARG;
    if ((V == nullptr) != (Vo == nullptr)) return MOC_ERR_INVALID_ARG;
    if (B == 0 || L == 0 || heads == 0) return MOC_OK;
    moc::RowArgs a{};
    common_args(a, rope, B, heads, L, pos, pos_batch, pos_axis, 1.f);
    a.eps = eps;
    a.w_fp32 = w_dtype == MOC_FP32;
    const void* x[3] = {Q, K, V};
    const int64_t* xs[3] = {q_strides, k_strides, v_strides};
    void* y[3] = {Qo, Ko, Vo};
    const int64_t* ys[3] = {qo_strides, ko_strides, vo_strides};
    const void* w[3] = {wq, wk, nullptr};
    const int H[3] = {Hq, Hk, V ? Hk : 0};
    bool al = true;
    for (int i = 0; i < 3; ++i) {
        if (H[i] == 0) continue;
        if (!check_tensor(x[i], xs[i], dtype, B, H[i], L, false, &al) ||
            !check_tensor(y[i], ys[i], dtype, B, H[i], L, true, &al))
            return MOC_ERR_INVALID_ARG;
        if (w[i] && reinterpret_cast<uintptr_t>(w[i]) % elem_bytes(w_dtype)) return MOC_ERR_INVALID_ARG;
        moc::RowSec& s = a.sec[i];
        s.x = x[i];
        s.y = y[i];
        set_strides(s.xs, xs[i], B, H[i], L);
        set_strides(s.ys, ys[i], B, H[i], L);
        s.w = w[i];
        s.H = H[i];
        s.mode = i == 2 ? moc::ROW_COPY : moc::ROW_NORM;
    }
    return cuda_status(moc::launch_rows_fwd(dtype, d, al, a, (cudaStream_t)stream));
}

extern "C" size_t moc_qk_norm_rope_bwd_workspace_bytes(int B, int Hq, int Hk, int64_t L, int d) {
    if (B < 0 || Hq < 0 || Hk < 0 || L < 0 || (d != 64 && d != 128)) return 0;
    const int64_t heads = int64_t(Hq) + 2 * int64_t(Hk);
    if (heads > 65535 || L > 0x7fffffff || int64_t(B) * L > 0x7fffff00) return 0;
    if (B == 0 || L == 0 || heads == 0) return 256;
    // with or without values, whichever launch has more CTAs (a partial each)
    int n = moc::rows_bwd_ctas(d, int64_t(B) * L, int(heads));
    if (Hq + Hk > 0) {
        const int m = moc::rows_bwd_ctas(d, int64_t(B) * L, Hq + Hk);
        n = m > n ? m : n;
    }
    return align256(size_t(n) * 2 * d * sizeof(float));
}

extern "C" moc_status moc_qk_norm_rope_bwd(const moc_rope* rope, int dtype, int B, int Hq, int Hk, int64_t L, int d,
                                           const void* Q, const int64_t* q_strides, const void* K,
                                           const int64_t* k_strides, const void* wq, const void* wk, int w_dtype,
                                           float eps, const int32_t* pos, int64_t pos_batch, int64_t pos_axis,
                                           const void* dQo, const int64_t* dqo_strides, const void* dKo,
                                           const int64_t* dko_strides, const void* dVo, const int64_t* dvo_strides,
                                           void* dQ, const int64_t* dq_strides, void* dK, const int64_t* dk_strides,
                                           void* dV, const int64_t* dv_strides, void* dwq, void* dwk, void* ws,
                                           size_t ws_bytes, moc_stream_t stream) {
    if (Hq < 0 || Hk < 0) return MOC_ERR_INVALID_ARG;
    const int64_t heads = int64_t(Hq) + Hk + (dVo ? Hk : 0);
    moc_status st = check_rows(rope, dtype, B, heads, L, d, pos, pos_batch, pos_axis);
    if (st != MOC_OK) return st;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return MOC_ERR_INVALID_ARG;
    if ((wq || wk || dwq || dwk) && w_dtype != MOC_FP32 && w_dtype != dtype) return MOC_ERR_INVALID_ARG;
    if ((dVo == nullptr) != (dV == nullptr)) return MOC_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(wq), static_cast<const void*>(wk), static_cast<const void*>(dwq),
                          static_cast<const void*>(dwk)})
        if (p && reinterpret_cast<uintptr_t>(p) % elem_bytes(w_dtype)) return MOC_ERR_INVALID_ARG;
    const bool want_dw = dwq || dwk;
    cudaStream_t s = (cudaStream_t)stream;
    if (B == 0 || L == 0 || heads == 0) {  // no rows: the weights' gradients are zero
        for (void* p : {dwq, dwk})
            if (p && cudaMemsetAsync(p, 0, size_t(d) * elem_bytes(w_dtype), s) != cudaSuccess) return MOC_ERR_CUDA;
        return MOC_OK;
    }
    moc::RowArgs a{};
    common_args(a, rope, B, heads, L, pos, pos_batch, pos_axis, -1.f);
    a.eps = eps;
    a.w_fp32 = w_dtype == MOC_FP32;
    const int ctas = moc::rows_bwd_ctas(d, a.tokens, a.heads);
    if (want_dw) {
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOC_ERR_INVALID_ARG;
        if (ws_bytes < size_t(ctas) * 2 * d * sizeof(float)) return MOC_ERR_WORKSPACE_TOO_SMALL;
        a.part = static_cast<float*>(ws);
    }
    const void* x[3] = {Q, K, dVo};  // values: only the gradient's layout changes
    const int64_t* xs[3] = {q_strides, k_strides, dvo_strides};
    const void* g[3] = {dQo, dKo, dVo};
    const int64_t* gs[3] = {dqo_strides, dko_strides, dvo_strides};
    void* y[3] = {dQ, dK, dV};
    const int64_t* ys[3] = {dq_strides, dk_strides, dv_strides};
    const void* w[3] = {wq, wk, nullptr};
    const int H[3] = {Hq, Hk, dVo ? Hk : 0};
    bool al = true;
    for (int i = 0; i < 3; ++i) {
        if (H[i] == 0) continue;
        if (!check_tensor(x[i], xs[i], dtype, B, H[i], L, false, &al) ||
            !check_tensor(g[i], gs[i], dtype, B, H[i], L, false, &al) ||
            !check_tensor(y[i], ys[i], dtype, B, H[i], L, true, &al))
            return MOC_ERR_INVALID_ARG;
        moc::RowSec& sc = a.sec[i];
        sc.x = x[i];
        sc.g = g[i];
        sc.y = y[i];
        set_strides(sc.xs, xs[i], B, H[i], L);
        set_strides(sc.gs, gs[i], B, H[i], L);
        set_strides(sc.ys, ys[i], B, H[i], L);
        sc.w = w[i];
        sc.H = H[i];
        sc.mode = i == 2 ? moc::ROW_COPY : moc::ROW_NORM;
    }
    cudaError_t e = moc::launch_rows_bwd(dtype, d, al, a, s);
    if (e == cudaSuccess && want_dw) e = moc::launch_rows_dw(dtype, a.w_fp32, d, ctas, a.part, dwq, dwk, s);
    return cuda_status(e);
}
