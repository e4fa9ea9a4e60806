// kdn_norm.h -- launch parameters and launchers of the gated norm and of the norm
// of the residual stream.  The C ABI (kdn_norm_abi.cpp) validates arguments and
// fills these.
#pragma once

#include <hip/hip_runtime.h>

#include "kdn.h"

namespace kdn {

constexpr int NORM_DIM = 16384;     // channels of a norm at most

struct GatedNormParams {
    int bf16;
    long tokens;
    int H, d;               // heads of a token, channels of a head
    int per_head;           // weight [H, d], else [d]
    int gate_first;         // kdn_norm_order
    int act;                // kdn_activation
    float eps;
    double inv_d;           // 1 / d
    long x_stride, z_stride;    // elements between tokens
    const void *x, *z;      // z may be null
    const float *weight;
    void *y;                // [tokens, H, d]
    // Gradients.
    const void *d_y;
    void *dx, *dz;
    float *dweight;
    float *ws;              // [parts][segs][heads of weight][d]
    int parts, segs, seg_rounds;    // workgroups; sums of each, over so many rounds of rows
};

struct ResidualNormParams {
    int bf16, stream_bf16;  // types of x and y, of the residual stream
    long tokens;
    int D;
    int scale_n;            // 0, 1 or D
    float eps;
    double inv_d;           // 1 / D
    long x_stride, r_stride;    // elements between tokens
    const void *x, *residual;
    const float *weight, *scale;
    void *y, *h;            // [tokens, D]
    // Gradients (residual holds h).
    const void *d_y, *d_h;  // d_h may be null (zero)
    void *dx, *dresidual;   // dx may be null (not wanted)
    float *dweight, *dscale;    // dscale may be null
    float *ws, *ws_scale;   // [segs][parts][D] of dweight, [segs][parts][D or 1] of dscale
    int parts, segs;        // workgroups of a launch, launches
};

// Parts that the sums over tokens are made in: about as many workgroups as run at once
// (of 256 and of 512 threads).  Half as many, these and twice as many: gated 262144 x 128
// bf16 72, 70 and 71 us, 98304 x 192 float32 by head 93, 80 and 85; residual 2500 x 1543
// bf16 24, 23 and 32, 16384 x 2048 67, 69 and 72.
constexpr int NORM_PARTS = 1024, RESIDUAL_PARTS = 512;
// Rows of a column that a thread adds in float32: behind them a workgroup of the gated norm
// writes its sums and begins anew, and of the residual norm another launch begins (as in the
// gated norm its kernel would take 21.5 us for 2500 x 1543, where it takes 20.2).  (More parts in their place let workgroups that run at once work on rows
// apart from each other: 131072 x 32 heads of 128 bf16, weight by head, 1262 us where it
// is 1177.)
constexpr int SEG_ROUNDS = 256;

// Threads of a row of n elements: one for each 16 bytes, a power of two, up to a
// whole workgroup.
inline int norm_row_threads(int n, bool bf16) {
    const int v = bf16 ? 8 : 4;
    int t = 1;
    while (t < (n + v - 1) / v && t < 1024)
        t *= 2;
    return t;
}

hipError_t launch_gated_norm(const GatedNormParams &P, hipStream_t stream);
hipError_t launch_gated_norm_backward(const GatedNormParams &P, hipStream_t stream);
hipError_t launch_residual_norm(const ResidualNormParams &P, hipStream_t stream);
hipError_t launch_residual_norm_backward(const ResidualNormParams &P, hipStream_t stream);

}  // namespace kdn
