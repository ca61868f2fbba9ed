// C entry points of the sliding-window attention: argument validation and launches.
#include <cmath>

#include "window.cuh"

namespace {

moc_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOC_OK : MOC_ERR_CUDA; }

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

struct Range {
    uintptr_t at;
    size_t bytes;
    Range(const void* p, size_t n) : at(reinterpret_cast<uintptr_t>(p)), bytes(p ? n : 0) {}
    bool meets(const Range& o) const { return bytes && o.bytes && at < o.at + o.bytes && o.at < at + bytes; }
};

constexpr int64_t kMaxLen = int64_t(1) << 28;   // positions and their differences with a limit of 2^30 fit 32 bits
// rows of one tensor: a copy's row coordinate, and an item past the last, fit 32 bits
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 65536;

moc_status make_args(moc::WinArgs& a, int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d, int64_t left,
                     int64_t right, int64_t sinks, int causal, const int32_t* q_len, const int32_t* kv_len,
                     int fill, float scale) {
    if (B < 0 || Hq < 0 || Hk < 0 || Lq < 0 || Lk < 0) return MOC_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return MOC_ERR_INVALID_ARG;
    if ((Hk == 0) != (Hq == 0) || (Hk > 0 && Hq % Hk != 0)) return MOC_ERR_INVALID_ARG;
    if (sinks < 0 || !(scale > 0.f) || !std::isfinite(scale)) return MOC_ERR_INVALID_ARG;
    if (!aligned4(q_len) || !aligned4(kv_len)) return MOC_ERR_INVALID_ARG;
    if (Lq >= kMaxLen || Lk >= kMaxLen || Hq > 65535 || B > 65535) return MOC_ERR_UNSUPPORTED;
    if (int64_t(B) * Hq * Lq >= kMaxRows || int64_t(B) * Hk * Lk >= kMaxRows) return MOC_ERR_UNSUPPORTED;
    a.B = B;
    a.Hq = Hq;
    a.Hk = Hk;
    a.group = Hk > 0 ? Hq / Hk : 1;
    a.Lq = int32_t(Lq);
    a.Lk = int32_t(Lk);
    // a limit that reaches every key from every row is none
    a.left = left < 0 || left >= Lq + Lk ? moc::kWinOpen : int32_t(left);
    // (causal: no key lies right of a row, whatever the limit; said once, so that every estimate
    // of a row's reach sees it)
    a.right = causal ? 0 : right < 0 || right >= Lq + Lk ? moc::kWinOpen : int32_t(right);
    a.sinks = int32_t(sinks < Lk ? sinks : Lk);
    a.causal = causal ? 1 : 0;
    a.q_len = q_len;
    a.kv_len = kv_len;
    a.scale = scale;
    a.fill = fill ? 1 : 0;
    return MOC_OK;
}

}  // namespace

extern "C" moc_status moc_window_attention(int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d, const void* Q,
                                           const void* K, const void* V, int64_t left, int64_t right, int64_t sinks,
                                           int causal, const int32_t* q_len, const int32_t* kv_len, int fill_rest,
                                           float softmax_scale, void* O, float* lse, moc_stream_t stream) {
    moc::WinArgs a{};
    const moc_status st = make_args(a, B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, q_len, kv_len, fill_rest,
                                    softmax_scale);
    if (st != MOC_OK) return st;
    if (B == 0 || Hq == 0 || Lq == 0) return MOC_OK;
    if (!aligned16(Q) || !aligned16(O) || (Lk > 0 && (!aligned16(K) || !aligned16(V))) || !aligned4(lse))
        return MOC_ERR_INVALID_ARG;
    const size_t qn = size_t(B) * Hq * Lq, kb = size_t(B) * Hk * Lk * d * 2;
    const Range rq(Q, qn * d * 2), ro(O, qn * d * 2), rl(lse, qn * 4), rk(K, kb), rv(V, kb);
    // an item reads its own Q rows before it writes them; keys and values every item reads
    if (ro.meets(rk) || ro.meets(rv) || (Q != O && ro.meets(rq)) || rl.meets(rq) || rl.meets(rk) || rl.meets(rv) || rl.meets(ro))
        return MOC_ERR_INVALID_ARG;
    // Up to 16 query rows to a key head one CTA cluster reads the cache once for all of them;
    // beyond, the row-tile kernels take a query head's keys in one CTA and the group's heads
    // read them each. Open and causal, d = 128, 1 key head of 22,563 slots: 16 query heads 45 us,
    // 24 192 us; 3 key heads of 60,000 slots, 4 query heads to each: 4 rows 106 us, 7 498 us;
    // 3 heads of 180,512 slots: 16 rows 302 us, 17 and 64 1,481 us.
    if (int64_t(a.group) * Lq <= moc::kWinFewRows && int64_t(B) * Hk <= 65535 && Lk > 0)
        return cuda_status(moc::launch_window_few(a, d, Q, K, V, O, lse, (cudaStream_t)stream));
    return cuda_status(moc::launch_window_fwd(a, d, Q, K, V, O, lse, (cudaStream_t)stream));
}

extern "C" moc_status moc_window_device_error(int32_t* detail, moc_stream_t stream) {
    int32_t* word = nullptr;
    if (moc::window_error_word(&word) != cudaSuccess || !word) return MOC_ERR_CUDA;
    return moc_check_device_error(word, 64 * sizeof(int32_t), detail, stream);
}

extern "C" size_t moc_window_attention_bwd_workspace_bytes(int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d,
                                                           int64_t left, int64_t right, int64_t sinks, int causal) {
    moc::WinArgs a{};
    if (make_args(a, B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, nullptr, nullptr, 0, 1.f) != MOC_OK) return 0;
    return moc::plan_window_bwd(a, d).total;
}

extern "C" moc_status moc_window_attention_bwd(int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d, const void* Q,
                                               const void* K, const void* V, const void* O, const float* lse,
                                               const void* dO, int64_t left, int64_t right, int64_t sinks, int causal,
                                               const int32_t* q_len, const int32_t* kv_len, int flags,
                                               float softmax_scale, void* dQ, void* dK, void* dV, void* ws, size_t ws_bytes,
                                               moc_stream_t stream) {
    if (flags & ~(MOC_WINDOW_FILL_REST | MOC_WINDOW_JOINED)) return MOC_ERR_INVALID_ARG;
    moc::WinArgs a{};
    const moc_status st = make_args(a, B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, q_len, kv_len,
                                    flags & MOC_WINDOW_FILL_REST, softmax_scale);
    if (st != MOC_OK) return st;
    a.joined = flags & MOC_WINDOW_JOINED ? 1 : 0;
    if (B == 0 || Hq == 0 || (Lq == 0 && Lk == 0)) return MOC_OK;
    if (Lq > 0)
        for (const void* t : {Q, O, dO, static_cast<const void*>(dQ)})
            if (!aligned16(t)) return MOC_ERR_INVALID_ARG;
    if (Lk > 0)
        for (const void* t : {K, V, static_cast<const void*>(dK), static_cast<const void*>(dV)})
            if (!aligned16(t)) return MOC_ERR_INVALID_ARG;
    if ((Lq > 0 && !lse) || !aligned4(lse)) return MOC_ERR_INVALID_ARG;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOC_ERR_INVALID_ARG;
    const moc::WinBwdPlan p = moc::plan_window_bwd(a, d);
    if (ws_bytes < p.total) return MOC_ERR_WORKSPACE_TOO_SMALL;
    const size_t qn = size_t(B) * Hq * Lq, qb = qn * d * 2, kb = size_t(B) * Hk * Lk * d * 2;
    const Range out[4] = {{dQ, qb}, {dK, kb}, {dV, kb}, {ws, p.total}}, in[4] = {{Q, qb}, {dO, qb}, {K, kb}, {V, kb}};
    for (int i = 0; i < 4; ++i) {  // (O and lse are read before anything but ws is written)
        for (const Range& r : in)
            if (out[i].meets(r)) return MOC_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (out[i].meets(out[j])) return MOC_ERR_INVALID_ARG;
    }
    if (out[3].meets({O, qb}) || out[3].meets({lse, qn * 4})) return MOC_ERR_INVALID_ARG;
    return cuda_status(moc::launch_window_bwd(a, d, Q, K, V, O, lse, dO, dQ, dK, dV, static_cast<char*>(ws), p,
                                              (cudaStream_t)stream));
}
