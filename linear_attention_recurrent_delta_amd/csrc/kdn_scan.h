// kdn_scan.h -- launch parameters and launchers of the selective state space scan.
// The C ABI (kdn_scan_abi.cpp) validates arguments and fills these.
#pragma once

#include <hip/hip_runtime.h>

#include "kdn.h"

namespace kdn {

// Tokens of a tile, the unit in which states within a sequence are kept (blocks of
// packed tables are multiples of it): what a workgroup of the gradients holds in
// registers, of 32 states half as many.
__host__ __device__ constexpr int scan_tile(int S) { return S > 16 ? 32 : 64; }
// Channels of a wave: four lanes hold a channel's states.
constexpr int SCAN_CHANNELS = 16;

struct ScanParams {
    int bf16;
    int N;                  // sequences
    int T;                  // dense: tokens of every sequence
    int C, S, G;            // channels, states of a channel, groups that share B and C
    int softplus;
    long tokens;
    long x_stride, d_stride, z_stride, b_stride, c_stride;   // elements between tokens
    const void *x, *delta, *z;      // [tokens, C]; z may be null
    const void *B, *Cm;             // [tokens, G, S]
    const float *A;                 // [C, S]
    const float *D, *bias;          // [C], may be null
    const float *S0;                // [pool, C, S], may be null (zero)
    void *y;                        // [tokens, C]
    float *S_out;                   // [pool, C, S], may be null (not wanted)
    // blocks of consecutive tokens of one sequence, as in kdn_linear.h
    int block, nblocks;
    const int *blocks, *block_offsets, *slots;
    long pool;
    // Sequences of several blocks (gradients: all): each tile's own contribution to the
    // state, replaced by the state at its start, and the sum of its time steps.
    long tile_slots;
    float *ws_state;                // [tile_slots][C][S]
    float *ws_dt;                   // [tile_slots][C]
    // Gradients.
    const void *d_y;                // [tokens, C]
    const float *dS_out;            // [pool, C, S], may be null (zero)
    void *dx, *ddelta, *dz;         // [tokens, C]
    void *dB, *dC;                  // [tokens, G, S]
    float *dA, *dD, *dbias;         // dD, dbias may be null
    float *dS0;                     // may be null
    float *ws_rstate;               // [tile_slots][C][S], the reverse recurrence's
    float *ws_bc;                   // [sets][tokens][G][2][S] of dB and dC
    float *ws_sum;                  // [parts][C][S + 2]: dA, dD, dbias
    int per_set;                    // runs of 16 channels that a workgroup takes
    int parts;                      // workgroups that share a set's tiles
    int classes;                    // workgroups' share of a block: every classes-th tile
};

struct ScanDecodeParams {
    int bf16;
    int N, C, S, G, softplus;
    long x_stride, d_stride, z_stride, b_stride, c_stride;
    const void *x, *delta, *z, *B, *Cm;
    const float *A, *D, *bias;
    const int *slots;               // [N] or null
    long pool;
    float *state;                   // [pool, C, S], updated in place
    void *y;                        // [N, C]
};

// Place of tile j of block b in the workspaces: blocks may end with a part of a
// tile, so each adds at most one to the tiles before it.
__host__ __device__ inline long tile_slot(long b, long first, int j, int S) {
    return first / scan_tile(S) + b + j;
}
inline long tile_slots(long tokens, long blocks, int S) {
    return tokens / scan_tile(S) + blocks + 1;
}

// Runs of 16 channels with the same B and C.
__host__ __device__ inline int scan_groups(int C, int G) {
    return (C / G + SCAN_CHANNELS - 1) / SCAN_CHANNELS;
}
inline long scan_total_blocks(const ScanParams &P) {
    return P.block_offsets ? (long)P.nblocks : (long)P.N * P.nblocks;
}
// Runs of a workgroup of the gradients at most: their sums over tokens lie in LDS.
__host__ __device__ constexpr int scan_per_set(int S) { return S > 16 ? 2 : 8; }
inline int scan_sets(const ScanParams &P) {
    return (scan_groups(P.C, P.G) + P.per_set - 1) / P.per_set;
}

hipError_t launch_scan(const ScanParams &P, bool several, hipStream_t stream);
hipError_t launch_scan_decode(const ScanDecodeParams &P, hipStream_t stream);
hipError_t launch_scan_backward(const ScanParams &P, hipStream_t stream);

// Passes of both directions' calls: the tiles' own contributions to the states (and
// with `reverse` to the reverse recurrence's), and their joins along each sequence.
hipError_t launch_scan_states(const ScanParams &P, bool reverse, hipStream_t stream);

}  // namespace kdn
