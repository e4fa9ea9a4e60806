// kdn_batch.h -- host-side checks of dense and packed batches, shared by the C ABI
// of the convolution and of the selective scan.
#pragma once

#include "kdn_check.h"

#include <limits.h>

namespace kdn {

// Sizes of a batch: N sequences of T tokens, or a packed batch as its tables were
// built.  Fills N, T, tokens, block, nblocks and pool of P (dense: block and
// nblocks are the kernels' own choice).
template <typename Params>
inline kdn_status batch_shape(Params &P, int N, int T, const kdn_packed *packed) {
    if (N < 0 || T < 0)
        return KDN_ERR_SHAPE;
    const long long tokens = packed ? packed->tokens : (long long)N * T;
    if (tokens > INT_MAX)
        return KDN_ERR_SHAPE;
    P.N = N;
    P.T = T;
    P.tokens = tokens;
    P.pool = N;
    if (packed) {
        if (T != 0 || tokens < 0 || packed->pool < 0 || packed->max_blocks < 0 ||
            packed->max_blocks != kdn_sequence_max_blocks(N, packed->tokens, packed->block))
            return KDN_ERR_SHAPE;
        P.block = packed->block;
        P.nblocks = packed->max_blocks;
        P.pool = packed->pool;
    }
    return KDN_OK;
}

// The packed tables' pointers.
template <typename Params> inline kdn_status batch_tables(Params &P, const kdn_packed *packed) {
    if (!packed)
        return KDN_OK;
    if (!packed->block_offsets || (P.nblocks > 0 && !packed->blocks))
        return KDN_ERR_NULL;
    if (!aligned(packed->blocks, 16) || !aligned(packed->block_offsets, 4) ||
        !aligned(packed->slots, 4))
        return KDN_ERR_ALIGN;
    P.blocks = packed->blocks;
    P.block_offsets = packed->block_offsets;
    P.slots = packed->slots;
    return KDN_OK;
}

// Elements between tokens (0: contiguous rows of `row` elements), any number of
// them from `row` to below 2^28 or the kernel's own limit.
inline kdn_status row_stride(long long given, long long row, long *out,
                             long long limit = 1LL << 28) {
    if (given == 0)
        given = row;
    if (given < row || given >= limit)
        return KDN_ERR_SHAPE;
    *out = given;
    return KDN_OK;
}

}  // namespace kdn
