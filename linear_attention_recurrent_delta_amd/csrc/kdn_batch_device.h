// kdn_batch_device.h -- device-side pieces shared by the kernels that take dense
// and packed batches: which tokens of which sequence a workgroup owns.
#pragma once

#include "kdn_device.h"

namespace kdn {

// The wave's number as a scalar: what depends on it are branches of the whole
// wave.  (A vector condition may become an EXEC mask without a branch, which
// an MFMA under it does not heed.)
__device__ __forceinline__ int wave_id() {
    return __builtin_amdgcn_readfirstlane((int)threadIdx.x / WAVE);
}

// Descriptor of `bytes` bytes from `base` (the same in every lane): loads at or past
// their end return 0, stores there are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void *base, unsigned bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                             0x00020000);
}

// ---------------------------------------------------------------------------
// The block of a workgroup.
// ---------------------------------------------------------------------------
struct Block {
    long first;      // first token row
    int count;       // tokens (0: nothing to do)
    int seq;         // sequence
    int index, last; // index in the sequence; 1 if it is the sequence's last
    int single;      // 1: the sequence has this block only
    long slot;       // state of the sequence, -1: the sequence is skipped
};

// Row b of the blocks.  Packed tables are device data that the host cannot
// check: a row that does not fit the call's sizes owns no tokens.
template <typename Params>
__device__ __forceinline__ Block get_block(const Params &P, long b) {
    Block B;
    B.count = 0;
    if (!P.block_offsets) {
        B.seq = (int)(b / P.nblocks);
        B.index = (int)(b - (long)B.seq * P.nblocks);
        const int t0 = B.index * P.block;
        B.first = (long)B.seq * P.T + t0;
        B.count = min(P.block, P.T - t0);
        B.last = B.index + 1 == P.nblocks;
        B.single = P.nblocks == 1;
        B.slot = B.seq;
        return B;
    }
    int4 r = reinterpret_cast<const int4 *>(P.blocks)[b];
    r.x = __builtin_amdgcn_readfirstlane(r.x);      // the same in every lane: scalars
    r.y = __builtin_amdgcn_readfirstlane(r.y);
    r.z = __builtin_amdgcn_readfirstlane(r.z);
    r.w = __builtin_amdgcn_readfirstlane(r.w);
    if (r.z < 0 || r.z >= P.N || r.x < 0 || r.y <= 0 || r.y > P.block ||
        (long)r.x + r.y > P.tokens || r.w < 0)
        return B;
    const int b0 = __builtin_amdgcn_readfirstlane(P.block_offsets[r.z]);
    const int b1 = __builtin_amdgcn_readfirstlane(P.block_offsets[r.z + 1]);
    if (b0 < 0 || b1 > P.nblocks || (long)b0 + r.w != b || b1 <= b)
        return B;
    B.slot = P.slots ? __builtin_amdgcn_readfirstlane(P.slots[r.z]) : r.z;
    if (B.slot >= P.pool)
        B.slot = -1;
    B.first = r.x;
    B.seq = r.z;
    B.index = r.w;
    B.last = b + 1 == b1;
    B.single = b1 - b0 == 1;
    B.count = r.y;
    return B;
}

// Tokens of sequence B.seq from its block B to its end, as the tables have it:
// at least the block's own, and never past the call's rows.
template <typename Params>
__device__ __forceinline__ long tokens_left(const Params &P, const Block &B) {
    if (!P.block_offsets)
        return P.T - (long)B.index * P.block;
    if (B.last)
        return B.count;
    const int b1 = __builtin_amdgcn_readfirstlane(P.block_offsets[B.seq + 1]);
    const int4 r = reinterpret_cast<const int4 *>(P.blocks)[b1 - 1];
    const long end = (long)__builtin_amdgcn_readfirstlane(r.x) +
                     max(__builtin_amdgcn_readfirstlane(r.y), 0);
    return max(min(end, P.tokens) - B.first, (long)B.count);
}

// First row behind the last sequence of a packed batch.
template <typename Params> __device__ __forceinline__ long tail_start(const Params &P) {
    const int nb = P.block_offsets[P.N];
    long end = 0;
    if (nb > 0 && nb <= P.nblocks) {
        const int4 r = reinterpret_cast<const int4 *>(P.blocks)[nb - 1];
        end = (long)r.x + r.y;
    }
    return end < 0 ? P.tokens : min(end, P.tokens);
}

// State of sequence n of a packed batch if the sequence has no tokens, else -1.
template <typename Params> __device__ __forceinline__ long empty_slot(const Params &P, int n) {
    long slot = n;
    if (P.block_offsets) {
        if (P.block_offsets[n + 1] > P.block_offsets[n])
            return -1;
        slot = P.slots ? P.slots[n] : n;
    } else if (P.T > 0) {
        return -1;
    }
    return slot >= 0 && slot < P.pool ? slot : -1;
}

}  // namespace kdn
