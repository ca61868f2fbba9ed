// C entry points of the sliding-window attention: argument validation and launches.
#include <cmath>

#include "window.cuh"

namespace {

moc_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOC_OK : MOC_ERR_CUDA; }

bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

constexpr int64_t kMaxLen = int64_t(1) << 29;   // positions and their sums with a limit stay in 32 bits
constexpr int64_t kMaxRows = int64_t(1) << 31;  // rows of one tensor: a copy's row coordinate is 32 bits

moc_status make_args(moc::WinArgs& a, int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d, int64_t left,
                     int64_t right, int64_t sinks, int causal, const int32_t* q_len, const int32_t* kv_len,
                     float scale) {
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
    a.right = right < 0 || right >= Lq + Lk ? moc::kWinOpen : int32_t(right);
    a.sinks = int32_t(sinks < Lk ? sinks : Lk);
    a.causal = causal ? 1 : 0;
    a.q_len = q_len;
    a.kv_len = kv_len;
    a.scale = scale;
    return MOC_OK;
}

}  // namespace

extern "C" moc_status moc_window_attention(int B, int Hq, int Hk, int64_t Lq, int64_t Lk, int d, const void* Q,
                                           const void* K, const void* V, int64_t left, int64_t right, int64_t sinks,
                                           int causal, const int32_t* q_len, const int32_t* kv_len,
                                           float softmax_scale, void* O, float* lse, moc_stream_t stream) {
    moc::WinArgs a{};
    const moc_status st = make_args(a, B, Hq, Hk, Lq, Lk, d, left, right, sinks, causal, q_len, kv_len, softmax_scale);
    if (st != MOC_OK) return st;
    if (B == 0 || Hq == 0 || Lq == 0) return MOC_OK;
    if (!aligned16(Q) || !aligned16(O) || (Lk > 0 && (!aligned16(K) || !aligned16(V))) || !aligned4(lse))
        return MOC_ERR_INVALID_ARG;
    return cuda_status(moc::launch_window_fwd(a, d, Q, K, V, O, lse, (cudaStream_t)stream));
}
