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

// Tokens of a workgroup's tile; channels of a lane (16 bytes of a row, gradients 8).
constexpr int CONV_TILE = 64;
inline int conv_vec(bool bf16, bool grad) { return (bf16 ? 8 : 4) / (grad ? 2 : 1); }

// Tiles of a packed batch that are found by their number (kdn_conv.hip): blocks may end
// with a part of a tile, so each adds at most one to the tiles before it.
inline long conv_found_tiles(const ConvParams &P) {
    return P.nblocks > 0 ? P.tokens / CONV_TILE + P.nblocks : 0;
}
// Tiles of a block where each block has room for as many as its length may need.
inline long conv_block_tiles(const ConvParams &P) {
    return ((long)P.block + CONV_TILE - 1) / CONV_TILE;
}
// Tiles of a launch.  `packed`: P.block and P.nblocks are the tables'.  Looking for a tile
// costs a gradient workgroup two loads in front of each of its tiles, a tile without tokens
// a workgroup or a round.  Room in every block and found, bf16, forward and gradients in us:
//     sequences, tokens, channels, block      room / found
//     37 of 590               6144    256         1.05        108  230    109  240
//     256 of 1 to 511, 63569  4096    256         1.35        237  510    203  462
//     256 of 1 to 31, 4225    4096    256         3.2          68  263     28   93
//     37 of 590               6144  21888        34           265  523    105  211
inline long conv_tiles(const ConvParams &P, bool packed) {
    if (!packed)
        return (long)P.N * (((long)P.T + CONV_TILE - 1) / CONV_TILE);
    const long room = P.nblocks * conv_block_tiles(P), found = conv_found_tiles(P);
    return 4 * room <= 5 * found ? room : found;
}
inline int conv_chunks(int C, int vec) { return (C + 64 * vec - 1) / (64 * vec); }

hipError_t launch_conv(const ConvParams &P, hipStream_t stream);
hipError_t launch_conv_decode(const ConvDecodeParams &P, hipStream_t stream);
hipError_t launch_conv_backward(const ConvParams &P, hipStream_t stream);

}  // namespace kdn
