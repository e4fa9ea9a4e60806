// kdn_conv.h -- launch parameters and launchers of the short causal convolution.
// The C ABI (kdn_conv_abi.cpp) validates arguments and fills these.
#pragma once

#include <hip/hip_runtime.h>

#include "kdn.h"

namespace kdn {

constexpr int CONV_TAPS = 4;       // taps at most

struct ConvParams {
    int bf16;
    int N;                  // sequences
    int T;                  // dense: tokens of every sequence
    int C, W;               // channels, taps
    int silu;               // activation
    long tokens;            // rows of x and y
    long x_stride;          // elements between tokens of x
    const void *x;
    const float *weight;    // [C, W]
    const float *bias;      // [C], may be null
    const void *state0;     // [pool, W - 1, C], may be null (zero)
    void *y;                // [tokens, C]
    void *state_out;        // [pool, W - 1, C], may be null (not wanted)
    // blocks of consecutive tokens of one sequence, as in kdn_linear.h
    int block, nblocks;
    const int *blocks, *block_offsets, *slots;
    long pool;
    // Gradients.
    const void *d_y;        // [tokens, C]
    const void *dstate_out; // [pool, W - 1, C], may be null (zero)
    void *dx;               // [tokens, C]
    float *dweight, *dbias; // dbias may be null
    void *dstate0;          // [pool, W - 1, C], may be null
    float *ws;              // [parts][W + 1][C] sums of dweight and dbias
    int parts;
};

struct ConvDecodeParams {
    int bf16;
    int N, C, W, silu;
    long x_stride;
    const void *x;
    const float *weight, *bias;
    const int *slots;       // [N] or null
    long pool;
    void *state;            // [pool, W - 1, C], updated in place
    void *y;                // [N, C]
};

// Tokens of a workgroup's tile in the gradient kernel, whose 64 lanes take 8 bytes
// of a row each.
constexpr int CONV_GRAD_TILE = 64;
inline long conv_tiles(const ConvParams &P, int tile) {
    return P.block_offsets ? (long)P.nblocks * (((long)P.block + tile - 1) / tile)
                           : (long)P.N * (((long)P.T + tile - 1) / tile);
}
inline int conv_chunks(int C, int vec) { return (C + 64 * vec - 1) / (64 * vec); }

hipError_t launch_conv(const ConvParams &P, hipStream_t stream);
hipError_t launch_conv_decode(const ConvDecodeParams &P, hipStream_t stream);
hipError_t launch_conv_backward(const ConvParams &P, hipStream_t stream);

}  // namespace kdn
