// kdn_tables.hip -- tables of a packed batch from the sequences' lengths
// (gfx950), in one kernel without an exchange between workgroups: every
// workgroup scans all lengths (a tile of TILE at a time, N int32 from the L2)
// and fills its own share of the tokens and of the block rows by binary
// searches in the tile's offsets.  Bound by the launch and the chain of scan,
// search and write: 48 sequences, 8192 tokens 7.7 us with the maps; 8000
// sequences, 2^20 tokens 18 us (8.7 MB written: 2 us of them at the rate of a
// copy, the rest two tiles of scans and searches of 12 steps in LDS).
#include "kdn_device.h"
#include "kdn_linear.h"

namespace kdn {
namespace tab {

constexpr int NT = 1024, PER = 4, TILE = NT * PER, NW = NT / WAVE;

// Exclusive prefix sums of x over the workgroup's threads; *all gets the sum.
template <typename I>
__device__ __forceinline__ I scan(I x, I *waves, I *all, int tid) {
    const int lane = tid & (WAVE - 1), w = tid / WAVE;
    I y = x;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const I z = __shfl_up(y, off, WAVE);
        if (lane >= off)
            y += z;
    }
    __syncthreads();                 // `waves` of the scan before has been read
    if (lane == WAVE - 1)
        waves[w] = y;
    __syncthreads();
    I before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        before += i < w ? waves[i] : 0;
        sum += waves[i];
    }
    *all = sum;
    return before + y - x;
}

// Largest i in [0, n) with start[i] <= x, where start[0] <= x < start[n]:
// of sequences without tokens at x the last, which is the one that has x.
__device__ __forceinline__ int find(const int *start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(NT) void tables_kernel(TableParams P, int tok_share, int row_share) {
    __shared__ int off[TILE + 1], boff[TILE + 1];
    __shared__ long long wsum[NW];
    __shared__ int wblk[NW];
    const int tid = threadIdx.x;
    const bool maps = P.slot_map || P.positions;
    const long t0 = (long)blockIdx.x * tok_share, t1 = min(t0 + tok_share, (long)P.tokens);
    const long r0 = (long)blockIdx.x * row_share, r1 = min(r0 + row_share, (long)P.max_blocks);
    long long sum = 0;               // tokens and blocks before the tile
    int end = 0, blk = 0;
    // by what is left: N + TILE may pass 32 bits
    for (int left = P.N; left > 0; left -= TILE) {
        const int n0 = P.N - left, m = min(TILE, left);
        long long len[PER], own = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int n = tid * PER + i;
            len[i] = n < m ? max(P.lengths[n0 + n], 0) : 0;
            own += len[i];
        }
        long long all;
        long long at = sum + scan<long long>(own, wsum, &all, tid);
        int nb[PER], bown = 0, start[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            start[i] = (int)min(at, (long long)P.tokens);
            at += len[i];
            const int stop = (int)min(at, (long long)P.tokens);
            // (len + block - 1 would pass 32 bits: blocks may be any length)
            nb[i] = stop > start[i] ? (stop - start[i] - 1) / P.block + 1 : 0;
            bown += nb[i];
        }
        int ball;
        int bat = blk + scan<int>(bown, wblk, &ball, tid);
        const long long next = sum + all;
        const int end_next = (int)min(next, (long long)P.tokens);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int n = tid * PER + i;
            if (n < m) {
                off[n] = start[i];
                boff[n] = bat;
                if (blockIdx.x == 0) {
                    P.offsets[n0 + n] = start[i];
                    P.block_offsets[n0 + n] = bat;
                }
            }
            bat += nb[i];
        }
        if (tid == 0) {
            off[m] = end_next;
            boff[m] = blk + ball;
        }
        __syncthreads();
        if (maps)
            for (long t = max(t0, (long)end) + tid; t < min(t1, (long)end_next); t += NT) {
                const int n = find(off, m, (int)t);
                if (P.slot_map)
                    P.slot_map[t] = P.slots ? P.slots[n0 + n] : n0 + n;
                if (P.positions)
                    P.positions[t] = (int)t - off[n] + (P.context ? P.context[n0 + n] : 0);
            }
        for (long r = max(r0, (long)blk) + tid; r < min(r1, (long)blk + ball); r += NT) {
            const int n = find(boff, m, (int)r);
            const int first = off[n] + (int)(r - boff[n]) * P.block;
            reinterpret_cast<int4 *>(P.blocks)[r] =
                make_int4(first, min(off[n + 1] - first, P.block), n0 + n, (int)(r - boff[n]));
        }
        sum = next;
        end = end_next;
        blk += ball;
        __syncthreads();             // the tile's offsets have been read
    }
    if (blockIdx.x == 0 && tid == 0) {
        P.offsets[P.N] = end;
        P.block_offsets[P.N] = blk;
    }
    if (maps)
        for (long t = max(t0, (long)end) + tid; t < t1; t += NT) {
            if (P.slot_map)
                P.slot_map[t] = -1;
            if (P.positions)
                P.positions[t] = 0;
        }
    for (long r = max(r0, (long)blk) + tid; r < r1; r += NT)
        reinterpret_cast<int4 *>(P.blocks)[r] = make_int4(0, 0, -1, 0);
}

}  // namespace tab

hipError_t launch_sequence_tables(const TableParams &P, hipStream_t st) {
    // a few searches per thread; one workgroup per CU at most
    const long most = (P.slot_map || P.positions) ? max(P.tokens, P.max_blocks) : P.max_blocks;
    long wgs = (most + 4 * tab::NT - 1) / (4 * tab::NT);
    wgs = wgs < 1 ? 1 : (wgs > 256 ? 256 : wgs);
    const int tok_share = (int)(((long)P.tokens + wgs - 1) / wgs);
    const int row_share = (int)(((long)P.max_blocks + wgs - 1) / wgs);
    hipLaunchKernelGGL(tab::tables_kernel, dim3((unsigned)wgs), dim3(tab::NT), 0, st, P, tok_share,
                       row_share);
    return hipGetLastError();
}

}  // namespace kdn
