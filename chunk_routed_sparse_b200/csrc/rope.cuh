// Rotary tables and the row operators' launch parameters, shared by the host
// side (rope.cpp) and the kernels (k_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moc.h"

namespace moc {

constexpr int kMaxRopePairs = 64;  // d <= 128
constexpr int kMaxRopeAxes = 4;

// A rotation by value: it travels in the kernel's parameters, and no device memory
// belongs to it (any device, any stream).
struct RopeTab {
    // angle per position in turns, as a 64-bit fraction: position x turn mod 2^64
    // is the exact fractional turn of any 32-bit position, near or far
    uint64_t turn[kMaxRopePairs];
    uint8_t axis[kMaxRopePairs];
    int32_t pairs;        // rotated pairs (rot_dim / 2)
    int32_t interleaved;  // pairs (2i, 2i + 1), else (i, i + pairs)
    int32_t axes;
    float factor;         // on the rotated part
};
static_assert(sizeof(RopeTab) == 592, "with three tensors' strides well below the 4 KB of a kernel's parameters");

enum { ROW_COPY = 0, ROW_ROPE = 1, ROW_NORM = 2 };  // ROW_NORM: norm, then the rotation

// One tensor of a row operator, [B][H][L][d] with strides in elements (last: 1).
struct RowSec {
    const void* x;   // input
    const void* g;   // upstream gradient (backward only)
    void* y;         // output
    int64_t xs[3], gs[3], ys[3];  // batch, head, token
    const void* w;   // norm weight [d] (null: ones)
    int32_t H;
    int32_t mode;
};

struct RowArgs {
    RowSec sec[3];
    RopeTab rope;
    const int32_t* pos;   // [axes][L] at pos_b per batch, pos_a per axis; null: 0 .. L-1
    int64_t pos_b, pos_a;
    int32_t L;
    int32_t tokens;       // B * L
    int32_t heads;        // over all sections
    int32_t heads_per_cta;
    int32_t w_fp32;       // weights in fp32 (else in the tensors' type)
    float eps;
    float sign;           // +1 rotation, -1 its transpose
    float* part;          // backward: weight gradient partials [cta][2][d]
};

cudaError_t launch_rows_fwd(int dtype, int d, bool aligned, const RowArgs& a, cudaStream_t s);
// CTAs of the backward (the count of weight-gradient partials)
int rows_bwd_ctas(int d, int64_t tokens, int heads);
cudaError_t launch_rows_bwd(int dtype, int d, bool aligned, const RowArgs& a, cudaStream_t s);
cudaError_t launch_rows_dw(int dtype, int w_fp32, int d, int ctas, const float* part, void* dwq, void* dwk,
                           cudaStream_t s);

}  // namespace moc

struct moc_rope {
    moc::RopeTab tab;
    double freq[moc::kMaxRopePairs];  // radians per position
    double factor;
};
