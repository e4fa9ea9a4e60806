// kdn_linear.h -- launch parameters and launchers of the linear-attention
// kernels (linear attention with a decay for each head) and of the
// packed-batch tables.  The C ABI (kdn_linear_abi.cpp) validates arguments
// and fills these.
#pragma once

#include <hip/hip_runtime.h>

#include "kdn.h"

namespace kdn {

// Tokens of one chunk of the chunked form: 64 bfloat16 or 32 float32 rows of
// q, k and v (d = 128) are 48 KB, 68 or 55 KB of LDS with their pitch and P, at
// most 80 KB where the state passes through LDS too (d_v = 64), so that two
// workgroups share a CU.
__host__ __device__ constexpr int linear_chunk(bool bf16) { return bf16 ? 64 : 32; }

struct LinearParams {
    int bf16;
    int N;                  // sequences
    int T;                  // dense: tokens of every sequence
    int H, Hq, Hk, Hv, dk, dv;
    int gate;               // kdn_gate
    long tokens;            // rows of q, k, v, o
    long q_stride, k_stride, v_stride;   // elements between tokens
    long o_stride;          // of d_o
    const void *q, *k, *v;
    const void *la;         // log_alpha
    // blocks of consecutive tokens of one sequence, the unit of a workgroup
    int block;              // tokens of a block (a multiple of 64)
    int nblocks;            // dense: blocks of a sequence; packed: rows of `blocks`
    const int *blocks;      // packed: [nblocks][4] first token, tokens, sequence,
                            // index in the sequence
    const int *block_offsets;   // packed: [N + 1] (null: dense)
    const int *slots;       // packed: [N] state of each sequence (null: n)
    long pool;              // states of S0 / S_out
    const float *S0;        // [pool, H, dk, dv], may be null (zero)
    float *S_out;           // [pool, H, dk, dv], may be null (not wanted)
    void *o;                // [tokens, H, dv]
    // Sequences of several blocks: a block's own contribution to the state
    // and its decay, replaced by the state at the block's start.
    float *ws_state;        // [blocks][H][dk * dv]
    float *ws_decay;        // [blocks][H]
    int *ws_order;          // [nblocks] of a packed batch, the order of its blocks in
                            // time (null: as they are)
    // Gradients.
    const void *d_o;        // [tokens, H, dv]
    const float *dS_out;    // [pool, H, dk, dv], may be null (zero)
    void *dq, *dk_, *dv_;   // contiguous [tokens, heads, d], call dtype
    void *dla;              // [tokens, H] or [H], call dtype, may be null
    int dla_f32;            // [H] in float32 whatever the call's dtype
    float *dS0;             // may be null
    float *ws_rstate;       // [blocks][H][dk * dv], the reverse recurrence's
    float *ws_rdecay;       // [blocks][H]
    void *ws_chunk;         // [chunk slots][H][dk * dv] state at every chunk's start,
                            // call dtype, in fragment order (chunk_slot)
    void *ws_chunk_lo;      // what the rounding of ws_chunk leaves, the same way, for
                            // d log_alpha (null: not wanted)
    float *ws_dq, *ws_dk, *ws_dv;   // [tokens, H, d] of shared heads (else null)
    double *ws_dla;         // [blocks][H] sums of d log_alpha (one decay per head)
};

struct LinearDecodeParams {
    int bf16;
    int N, H, Hq, Hk, Hv, dk, dv;
    int gate;
    long q_stride, k_stride, v_stride;
    const void *q, *k, *v, *la;
    const int *slots;       // [N] or null
    long pool;
    float *S;               // [pool, H, dk, dv], updated in place
    void *o;                // [N, H, dv]
};

struct TableParams {
    int N, tokens, block, max_blocks;
    const int *lengths, *slots, *context;
    int *offsets, *block_offsets, *blocks, *slot_map, *positions;
};

// Place of chunk c of block b in ws_chunk: blocks may end with a part of a
// chunk, so each adds at most one to the chunks before it.
__host__ __device__ inline long chunk_slot(long b, long first, int c, int C) {
    return first / C + b + c;
}
inline long chunk_slots(long tokens, long blocks, int C) { return tokens / C + blocks + 1; }

// Blocks of all sequences, for grids and workspaces.
inline long linear_total_blocks(const LinearParams &P) {
    return P.block_offsets ? (long)P.nblocks : (long)P.N * P.nblocks;
}

// Two heads of d_v = 64 in a workgroup, where two neighbours have the same q
// and k and v of their own: q and k are read and q k^T is made once for both,
// and their columns fill the four waves.  Only where single heads would be
// more workgroups than run at once (2 a CU), since one alone takes longer for
// two: B1 H8 T1000 of 128 x 64, bf16, 22 against 19 us; B1 H16 T4000 34
// against 37; B4 H32 T16384 418 against 474 (float32 38 against 31, 70 against
// 79, 1396 against 1598).
inline bool linear_pairs(const LinearParams &P) {
    return P.H > 0 && P.dv == 64 && P.Hv == P.H && P.H / P.Hq % 2 == 0 && P.H / P.Hk % 2 == 0 &&
           linear_total_blocks(P) * P.H >= 512;
}

hipError_t launch_linear_prefill(const LinearParams &P, hipStream_t stream);
hipError_t launch_linear_decode(const LinearDecodeParams &P, hipStream_t stream);
hipError_t launch_linear_backward(const LinearParams &P, hipStream_t stream);
hipError_t launch_sequence_tables(const TableParams &P, hipStream_t stream);

// Passes of the gradient call that are walks of the prefill's kind
// (kdn_linear.hip): the blocks' own contributions to the states of both
// recurrences (ws_state, ws_rstate), and the state at every chunk's start.
hipError_t launch_linear_own(const LinearParams &P, hipStream_t stream);
hipError_t launch_linear_chunk_states(const LinearParams &P, hipStream_t stream);

}  // namespace kdn
