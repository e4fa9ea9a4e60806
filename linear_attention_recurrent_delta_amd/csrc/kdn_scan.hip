// kdn_scan.hip -- the selective state space scan (gfx950), per channel with S states:
//   dt_t = softplus(delta_t + bias),   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,
//   y_t = (C_t . h_t + D x_t) silu(z_t).
// Every token needs an exponential for each channel and state, so the scan is bound
// by the vector units: a product, an exponential (two instructions' time), a product
// and two sums for each state.  No matrix product is in it: the decays differ for
// each channel and state.  A wave has 16 channels, four lanes each, with S / 4 states
// in a lane's registers: a token's 16 values are 32 or 64 bytes of a row, one read from
// LDS brings B and C of a token to all 16 channels, and the sum over states is two steps
// within four lanes.
#include "kdn_scan_device.h"

namespace kdn {
namespace scan {

// Blocks times runs of channels from which each has one wave and not eight: the one
// wave needs three quarters of the work, and there are enough to fill the CUs.  bf16, 16
// states, eight waves and one, in us:
//     tokens    512 runs    1024       2048        4096
//       300     26   35    49   37    95   54    185   89
//      1000     62  114   121  117   229  159
//      4000    221  426   463  430   894  610   1786 1157
constexpr long SCAN_MANY = 1024;
// Workgroups that the pass over tiles' own states is shared out to.  With 1024, 4096
// and 16384: one sequence of 16000 tokens and 1024 channels 213, 207 and 207 us,
// gradients of 11 packed sequences of 518 channels, float32, 211, 205 and 216.
constexpr long SCAN_OWN_WGS = 4096;

// Tokens that a wave takes at a time: their decays and inputs stay in registers
// between the two passes over them.
template <int SPL> constexpr int steps() { return SPL <= 4 ? 16 : 8; }

// Per-token values of a wave's channels: lane 4 k + j has tokens 4 i + j.
template <typename T, int K> struct TokenRows {
    T x[K / 4], d[K / 4], z[K / 4];
    // tokens first .. + K of which `count` are there
    __device__ __forceinline__ void load(const ScanParams &P, const Channels &ch, long first,
                                         int count) {
        const int j = threadIdx.x & 3;
        const Rows<T, K> rx(P.x, first, P.x_stride, P.C, count);
        const Rows<T, K> rd(P.delta, first, P.d_stride, P.C, count);
        const Rows<T, K> rz(P.z, first, P.z_stride, P.C, P.z ? count : 0);
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            x[i] = rx.load(rx.at(4 * i + j, P.x_stride, ch.c, true));
            d[i] = rd.load(rd.at(4 * i + j, P.d_stride, ch.c, true));
            z[i] = rz.load(rz.at(4 * i + j, P.z_stride, ch.c, true));
        }
    }
    // time step of token 4 i + j (0 of one that is not there, which leaves the state as
    // it is)
    template <bool FINE>
    __device__ __forceinline__ float step(const ScanParams &P, float bias, int i,
                                          int count) const {
        const float v = to_f32(d[i]) + bias;
        const float dt = P.softplus ? softplus<FINE>(v) : v;
        return 4 * i + ((int)threadIdx.x & 3) < count ? dt : 0.f;
    }
};

// Block number p of a packed batch by length, the longest first (of equal ones the
// first), for up to 64 blocks: each lane ranks one.
__device__ __forceinline__ int by_length(const ScanParams &P, int p) {
    const int lane = threadIdx.x & (WAVE - 1), n = P.nblocks;
    const int count = lane < n ? P.blocks[4 * lane + 1] : 0;
    int rank = 0;
    for (int k = 0; k < n; ++k) {
        const int other = __builtin_amdgcn_readlane(count, k);
        rank += other > count || (other == count && k < lane);
    }
    return __builtin_ctzll(__ballot(lane < n && rank == p));
}

// ---------------------------------------------------------------------------
// Outputs.  NW waves of a workgroup walk one block, K tokens each at a time: every
// wave scans its tokens from nothing and puts its end and its decay into LDS; the
// lanes, one for each of the run's 16 S states, fold the waves' ends into the states
// in front of their tokens and carry the last on; and every wave goes through its
// tokens again, with their decays and inputs from registers (one more product and sum
// for a state than a walk by one wave, which NW = 1 is).  The chain along a sequence
// is then an eighth as long.  37 packed prompts (22 thousand tokens) of 4096 channels,
// 16 states, bf16: 361 to 370 us with the tables' 6 (420 where each kernel is traced by
// itself), bound by the vector units: six instructions' time for a state are 245, B and C
// from LDS, softplus, gate and sums over states the rest.  The instructions take 1.10 of
// the vector units' time as counted, with two for an exponential; others are issued in its
// second half, and a loop of one exponential and five others reaches 1.06.  2.0 TB/s.  A
// prompt of 190 tokens and 2048 channels: 11 us.
// ---------------------------------------------------------------------------
template <typename T, int SPL, int NW>
__global__ __launch_bounds__(NW == 1 ? 256 : NW *WAVE, 2) void scan_kernel(ScanParams P,
                                                                           int groups,
                                                                           long blocks) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int S = 4 * SPL, K = steps<SPL>(), WAVES = NW == 1 ? 4 : NW;
    __shared__ float bc[WAVES][2][K][S];
    // each wave's decay; its end from nothing, and then the state in front of its tokens
    __shared__ float ends[2][NW][NW == 1 ? 1 : WAVE * SPL];
    constexpr int FOLD = WAVE * SPL / NW;            // states that a wave's lanes fold
    const int lane = threadIdx.x & (WAVE - 1), j = lane & 3, w = wave_id();
    const int seg = NW == 1 ? 0 : w;
    const int runs = groups * P.G, fours = (runs + 3) / 4;
    long b = blockIdx.x / fours;
    int run = (int)(blockIdx.x % fours) * 4 + w;     // NW = 1: one for each wave
    if (NW == 1 ? run >= runs : !four_unit(blockIdx.x, blocks, runs, b, run))
        return;
    // of a packed batch the longest sequences go first
    if (P.block_offsets && P.nblocks <= WAVE)
        b = by_length(P, (int)b);
    const Channels ch(P, run, groups);
    const Block B = get_block(P, b);
    if (B.count <= 0 || B.slot < 0 || (!B.single && !P.ws_state))
        return;
    const long at = (B.slot * P.C + ch.c) * S + j * SPL;
    float A2[SPL], h[SPL];
    load_A<SPL>(P, ch.c, j, A2);
    const float bias = P.bias ? P.bias[ch.c] : 0.f, D = P.D ? P.D[ch.c] : 0.f;
    // the state in front of the block: the lane's own states, or the one that it folds
    const float *from = B.single ? P.S0 : P.ws_state;
    const long from_slot = B.single ? B.slot : tile_slot(b, B.first, 0, S);
    const int per = P.C / P.G, first_c = run % groups * SCAN_CHANNELS;
    const int fold = w * FOLD + lane, channels = min(SCAN_CHANNELS, per - first_c);
    const bool folds = NW > 1 && lane < FOLD && fold < channels * S;
    const long fold_at = ((long)ch.g * per + first_c) * S + fold;
    float carry = 0.f;
#pragma unroll
    for (int s = 0; s < SPL; ++s)
        h[s] = 0.f;
    if (NW > 1 && from && folds)
        carry = from[from_slot * P.C * S + fold_at];
    if (NW == 1 && from)
        load_states<SPL>(from + (from_slot * P.C + ch.c) * S + j * SPL, h);

    TokenRows<T, K> rows;
    GroupRows<T, S, K> group;
    rows.load(P, ch, B.first + seg * K, B.count - seg * K);
    group.load(P, ch.g, B.first + seg * K, B.count - seg * K);
    for (int t0 = 0; t0 < B.count; t0 += NW * K) {
        const int own = t0 + seg * K, count = B.count - own;
        // this round's values; the next round's are requested before the work on them
        const TokenRows<T, K> now = rows;
        group.put(bc[w]);
        if (t0 + NW * K < B.count) {
            rows.load(P, ch, B.first + own + NW * K, count - NW * K);
            group.load(P, ch.g, B.first + own + NW * K, count - NW * K);
        }
        float dt[K / 4], in[K / 4], sum = 0.f;
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            dt[i] = now.template step<FINE>(P, bias, i, count);
            in[i] = dt[i] * to_f32(now.x[i]);
            sum += dt[i];
        }
        // outputs of four tokens at a time, each by the lane that has its x and z
        const Rows<T, K> ry(P.y, B.first + own, P.C, P.C, count);
        float part[4];
        auto output = [&](auto I) {
            constexpr int i = I;
            if constexpr (i % 4 == 3) {
                float out = fmaf(D, to_f32(now.x[i / 4]), quad_sums(part, j));
                if (P.z)
                    out *= silu_f32<FINE>(to_f32(now.z[i / 4]));
                ry.store(from_f32<T>(out), ry.at(i - 3 + j, P.C, ch.c, ch.live));
            }
        };
        if constexpr (NW == 1) {
            unrolled<K>([&](auto I) {
                constexpr int i = I;
                const float d = quad_lane<i % 4>(dt[i / 4]), v = quad_lane<i % 4>(in[i / 4]);
                float Bt[SPL], Ct[SPL], y = 0.f;
                load_states<SPL>(&bc[w][0][i][j * SPL], Bt);
                load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    h[s] = fmaf(__builtin_amdgcn_exp2f(d * A2[s]), h[s], v * Bt[s]);
                    y = fmaf(Ct[s], h[s], y);
                }
                part[i % 4] = y;
                output(I);
            });
        } else {
            float a[K][SPL], u[K][SPL], end[SPL];
#pragma unroll
            for (int s = 0; s < SPL; ++s)
                end[s] = 0.f;
            unrolled<K>([&](auto I) {
                constexpr int i = I;
                const float d = quad_lane<i % 4>(dt[i / 4]), v = quad_lane<i % 4>(in[i / 4]);
                float Bt[SPL];
                load_states<SPL>(&bc[w][0][i][j * SPL], Bt);
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    a[i][s] = __builtin_amdgcn_exp2f(d * A2[s]);
                    u[i][s] = v * Bt[s];
                    end[s] = fmaf(a[i][s], end[s], u[i][s]);
                }
            });
            sum = quad_sum(sum);
            float all[SPL];
#pragma unroll
            for (int s = 0; s < SPL; ++s)
                all[s] = __builtin_amdgcn_exp2f(sum * A2[s]);
            store_states<SPL>(&ends[0][seg][lane * SPL], all);
            store_states<SPL>(&ends[1][seg][lane * SPL], end);
            __syncthreads();
            if (lane < FOLD) {
                float va[NW], ve[NW];
#pragma unroll
                for (int q = 0; q < NW; ++q) {
                    va[q] = ends[0][q][fold];
                    ve[q] = ends[1][q][fold];
                }
#pragma unroll
                for (int q = 0; q < NW; ++q) {
                    ends[1][q][fold] = carry;
                    carry = fmaf(va[q], carry, ve[q]);
                }
            }
            __syncthreads();
            load_states<SPL>(&ends[1][seg][lane * SPL], h);
            unrolled<K>([&](auto I) {
                constexpr int i = I;
                float Ct[SPL], y = 0.f;
                load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    h[s] = fmaf(a[i][s], h[s], u[i][s]);
                    y = fmaf(Ct[s], h[s], y);
                }
                part[i % 4] = y;
                output(I);
            });
        }
    }
    // (where S_out is S0: a state is read and written by the same lane)
    if (P.S_out && B.last) {
        if (NW == 1 && ch.live)
            store_states<SPL>(P.S_out + at, h);
        if (NW > 1 && folds)
            P.S_out[B.slot * P.C * S + fold_at] = carry;
    }
}

// ---------------------------------------------------------------------------
// A tile's own contribution to the state from nothing, U = sum_t (decay behind t)
// dt_t x_t B_t, the sum of its time steps, and with REV what its tokens hand to the
// reverse recurrence, Q = sum_t (decay up to and with t) dy'_t C_t, dy' = dy silu(z).
// A workgroup has a run of 16 channels and a share of a block: its waves take every
// fourth of every `classes`-th four tiles, token by token.  Bound by the vector units
// as the outputs are: B2 T4096, 2048 channels, 16 states, bf16, both ways 88 us.
// ---------------------------------------------------------------------------
constexpr int OWN_WAVES = 4;
template <typename T, int SPL, bool REV>
__global__ __launch_bounds__(OWN_WAVES *WAVE) void scan_own_kernel(ScanParams P, int groups,
                                                                   int classes, long shares) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int S = 4 * SPL, K = steps<SPL>(), TILE = scan_tile(S);
    __shared__ float bc[OWN_WAVES][2][K][S];
    const int lane = threadIdx.x & (WAVE - 1), j = lane & 3, w = wave_id();
    long outer;
    int run;
    if (!four_unit(blockIdx.x, shares, groups * P.G, outer, run))
        return;
    const long b = outer / classes;
    const int share = (int)(outer % classes);
    const Channels ch(P, run, groups);
    const Block B = get_block(P, b);
    if (B.count <= 0 || B.slot < 0 || (!REV && B.single))
        return;
    // the outputs alone do not need the last tile's
    const int stop = !REV && B.last ? (B.count - 1) / TILE * TILE : B.count;
    float A2[SPL];
    load_A<SPL>(P, ch.c, j, A2);
    const float bias = P.bias ? P.bias[ch.c] : 0.f;
    for (int t1 = (share * OWN_WAVES + w) * TILE; t1 < stop; t1 += classes * OWN_WAVES * TILE) {
        const int n = min(TILE, B.count - t1);
        float end[SPL], back[SPL], all[SPL];
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            end[s] = back[s] = 0.f;
            all[s] = 1.f;
        }
        float sum = 0.f;
        for (int t0 = 0; t0 < n; t0 += K) {
            TokenRows<T, K> rows;
            GroupRows<T, S, K> group;
            const long first = B.first + t1 + t0;
            rows.load(P, ch, first, n - t0);
            group.load(P, ch.g, first, n - t0);
            float dt[K / 4], in[K / 4], g[K / 4];
            const Rows<T, K> ry(P.d_y, first, P.C, P.C, REV ? n - t0 : 0);
#pragma unroll
            for (int i = 0; i < K / 4; ++i)
                g[i] = REV ? to_f32(ry.load(ry.at(4 * i + j, P.C, ch.c, true))) : 0.f;
            group.put(bc[w]);
#pragma unroll
            for (int i = 0; i < K / 4; ++i) {
                dt[i] = rows.template step<FINE>(P, bias, i, n - t0);
                in[i] = dt[i] * to_f32(rows.x[i]);
                sum += dt[i];
                if (REV && P.z)
                    g[i] *= silu_f32<FINE>(to_f32(rows.z[i]));
            }
            unrolled<K>([&](auto I) {
                constexpr int i = I;
                const float d = quad_lane<i % 4>(dt[i / 4]), v = quad_lane<i % 4>(in[i / 4]);
                const float e = quad_lane<i % 4>(g[i / 4]);
                float Bt[SPL], Ct[SPL];
                load_states<SPL>(&bc[w][0][i][j * SPL], Bt);
                if constexpr (REV)
                    load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                for (int s = 0; s < SPL; ++s) {
                    const float a = __builtin_amdgcn_exp2f(d * A2[s]);
                    end[s] = fmaf(a, end[s], v * Bt[s]);
                    if constexpr (REV) {
                        all[s] *= a;
                        back[s] = fmaf(all[s], e * Ct[s], back[s]);
                    }
                }
            });
        }
        sum = quad_sum(sum);
        const long slot = tile_slot(b, B.first, t1 / TILE, S) * P.C + ch.c;
        if (ch.live) {
            store_states<SPL>(P.ws_state + slot * S + j * SPL, end);
            if constexpr (REV)
                store_states<SPL>(P.ws_rstate + slot * S + j * SPL, back);
            if (j == 0)
                P.ws_dt[slot] = sum;
        }
    }
}

// ---------------------------------------------------------------------------
// Join of the tiles along each sequence: a tile's own contribution U becomes the
// state at its start, h <- 2^(A2 sum dt) h + U; reverse (tiles last to first): Q
// becomes the reverse state behind its end, and behind the first tile is dS0.  A
// thread holds two states of a channel; the next JOIN tiles are on their way while as
// many are joined (4, 8 and 16: one sequence of 16000 tokens and 1024 channels 211, 207
// and 204 us, gradients of B2 T4096 356, 355 and 355).  Bound by a chain of as many
// loads as there are tiles: 16 us for two of 64 both ways, 2048 channels (27 with one
// state a thread and no tiles on their way).
// ---------------------------------------------------------------------------
constexpr int JOIN = 8, JOIN_NT = 256;
template <bool REV>
__device__ __forceinline__ void join(const ScanParams &P, int seq, long e, bool all) {
    const long size = (long)P.C * P.S;
    long b0 = (long)seq * P.nblocks, b1 = b0 + P.nblocks, slot = seq, first, n;
    if (P.block_offsets) {
        b0 = P.block_offsets[seq];
        b1 = P.block_offsets[seq + 1];
        slot = P.slots ? P.slots[seq] : seq;
        if (b0 < 0 || b1 > P.nblocks || slot < 0 || slot >= P.pool)
            return;
    }
    const float *from = REV ? P.dS_out : P.S0;
    float *pass = REV ? P.dS0 : P.S_out;
    float2 h = make_float2(0.f, 0.f);
    if (from)
        h = *reinterpret_cast<const float2 *>(from + slot * size + e);
    if (b1 <= b0) {                  // no tokens: the state passes on
        if (pass && pass != from)
            *reinterpret_cast<float2 *>(pass + slot * size + e) = h;
        return;
    }
    if (b1 - b0 == 1 && !all)
        return;
    first = (long)seq * P.T;
    n = P.T;
    if (P.block_offsets) {
        const int4 r0 = reinterpret_cast<const int4 *>(P.blocks)[b0];
        const int4 r1 = reinterpret_cast<const int4 *>(P.blocks)[b1 - 1];
        first = r0.x;
        n = (b1 - b0 - 1) * P.block + r1.y;
    }
    const int tile = scan_tile(P.S);
    const long tiles = (n + tile - 1) / tile, per = P.block / tile;
    // blocks but the last are whole tiles: tile i has slot first / tile + b0 + i + i / per
    const long base = first / tile + b0;
    float *ws = REV ? P.ws_rstate : P.ws_state;
    if (!ws || first < 0 || n <= 0 || base + tiles - 1 + (tiles - 1) / per >= P.tile_slots)
        return;
    const float2 A = *reinterpret_cast<const float2 *>(P.A + e);
    const long c = e / P.S;
    // the tiles in the order of the join
    struct Place {
        long slot, in;               // slot, and index in the block
    };
    auto next = [&](Place &p) {
        if (REV ? p.in == 0 : p.in + 1 == per) {
            p.in = REV ? per - 1 : 0;
            p.slot += REV ? -2 : 2;
        } else {
            p.in += REV ? -1 : 1;
            p.slot += REV ? -1 : 1;
        }
    };
    const long t0 = REV ? tiles - 1 : 0;
    Place at{base + t0 + t0 / per, t0 % per}, ahead = at;
    const long need = REV ? tiles : tiles - 1;      // own contributions that are used
    float2 u[JOIN], u1[JOIN];
    float d[JOIN], d1[JOIN];
    auto load = [&](long i, float2(&v)[JOIN], float(&t)[JOIN]) {
#pragma unroll
        for (int k = 0; k < JOIN; ++k)
            if (i + k < need) {
                v[k] = *reinterpret_cast<const float2 *>(ws + ahead.slot * size + e);
                t[k] = P.ws_dt[ahead.slot * P.C + c];
                next(ahead);
            }
    };
    auto step = [&](long i, const float2(&v)[JOIN], const float(&t)[JOIN]) {
#pragma unroll
        for (int k = 0; k < JOIN; ++k)
            if (i + k < tiles) {
                *reinterpret_cast<float2 *>(ws + at.slot * size + e) = h;
                next(at);
                if (i + k < need) {
                    h.x = fmaf(__builtin_amdgcn_exp2f(t[k] * LOG2E * A.x), h.x, v[k].x);
                    h.y = fmaf(__builtin_amdgcn_exp2f(t[k] * LOG2E * A.y), h.y, v[k].y);
                }
            }
    };
    load(0, u, d);
    for (long i = 0; i < tiles; i += 2 * JOIN) {
        load(i + JOIN, u1, d1);
        step(i, u, d);
        load(i + 2 * JOIN, u, d);
        step(i + JOIN, u1, d1);
    }
    if (REV && pass)
        *reinterpret_cast<float2 *>(pass + slot * size + e) = h;
}

template <bool REV>
__global__ __launch_bounds__(JOIN_NT) void scan_join_kernel(ScanParams P, int pieces) {
    long id = blockIdx.x;
    bool reverse = false;
    if (REV) {
        reverse = id & 1;
        id >>= 1;
    }
    const long e = 2 * ((id % pieces) * JOIN_NT + threadIdx.x);
    const int seq = (int)(id / pieces);
    if (e >= (long)P.C * P.S)
        return;
    if (REV && reverse)
        join<true>(P, seq, e, true);
    else
        join<false>(P, seq, e, REV);
}

// ---------------------------------------------------------------------------
// Single tokens.  Bound by one read and one write of the states.  Four lanes a
// channel, as above; no state is read twice, so they pass the caches.  256 sequences,
// 4096 channels, 16 states, bf16: 30 us, 4.8 TB/s.
// ---------------------------------------------------------------------------
template <typename T, int SPL>
__global__ __launch_bounds__(256) void scan_decode_kernel(ScanDecodeParams P, int chunks) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int S = 4 * SPL;
    const int j = threadIdx.x & 3;
    const long n = blockIdx.x / chunks;
    const int in = (int)(blockIdx.x % chunks) * 64 + (threadIdx.x >> 2);
    const long slot = P.slots ? P.slots[n] : n;
    if (slot < 0 || slot >= P.pool)
        return;
    const bool live = in < P.C;
    const int c = live ? in : P.C - 1, g = c / (P.C / P.G);
    float *state = P.state + (slot * P.C + c) * S + j * SPL;
    float h[SPL], A[SPL], y = 0.f;
    typedef float V __attribute__((ext_vector_type(SPL < 4 ? SPL : 4)));
    constexpr int VN = SPL < 4 ? SPL : 4;
#pragma unroll
    for (int s = 0; s < SPL; s += VN) {
        const V v = __builtin_nontemporal_load(reinterpret_cast<const V *>(state + s));
#pragma unroll
        for (int e = 0; e < VN; ++e)
            h[s + e] = v[e];
    }
    load_states<SPL>(P.A + (long)c * S + j * SPL, A);
    const float x = to_f32(static_cast<const T *>(P.x)[n * P.x_stride + c]);
    float dt = to_f32(static_cast<const T *>(P.delta)[n * P.d_stride + c]) +
               (P.bias ? P.bias[c] : 0.f);
    if (P.softplus)
        dt = softplus<FINE>(dt);
    const T *B = static_cast<const T *>(P.B) + n * P.b_stride + (long)g * S + j * SPL;
    const T *Cm = static_cast<const T *>(P.Cm) + n * P.c_stride + (long)g * S + j * SPL;
    Pack<T, SPL> Bt, Ct;
    Bt.load(B);
    Ct.load(Cm);
    const float in_x = dt * x;
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
        h[s] = fmaf(exp_f32<FINE>(dt * A[s]), h[s], in_x * Bt.get(s));
        y = fmaf(Ct.get(s), h[s], y);
    }
    if (live)
#pragma unroll
        for (int s = 0; s < SPL; s += VN) {
            V v;
#pragma unroll
            for (int e = 0; e < VN; ++e)
                v[e] = h[s + e];
            __builtin_nontemporal_store(v, reinterpret_cast<V *>(state + s));
        }
    y = quad_sum(y);
    if (j == 0 && live) {
        y = fmaf(P.D ? P.D[c] : 0.f, x, y);
        if (P.z)
            y *= silu_f32<FINE>(to_f32(static_cast<const T *>(P.z)[n * P.z_stride + c]));
        static_cast<T *>(P.y)[n * P.C + c] = from_f32<T>(y);
    }
}

template <typename T, int SPL>
hipError_t launch_t(const ScanParams &P, hipStream_t st) {
    constexpr int NW = 8;
    const int groups = scan_groups(P.C, P.G);
    const long blocks = scan_total_blocks(P), runs = (long)groups * P.G;
    if (blocks * runs == 0)
        return hipSuccess;
    if (blocks * runs >= SCAN_MANY)
        hipLaunchKernelGGL((scan_kernel<T, SPL, 1>), dim3((unsigned)(blocks * ((runs + 3) / 4))), dim3(256), 0, st, P,
                           groups, blocks);
    else
        hipLaunchKernelGGL((scan_kernel<T, SPL, NW>),
                           dim3((unsigned)four_grid(blocks, runs)), dim3(NW * WAVE), 0, st, P,
                           groups, blocks);
    return hipGetLastError();
}

template <typename T, int SPL>
hipError_t launch_own_t(const ScanParams &P, bool reverse, hipStream_t st) {
    const int groups = scan_groups(P.C, P.G);
    const long blocks = scan_total_blocks(P), runs = (long)groups * P.G;
    if (blocks * runs == 0)
        return hipSuccess;
    // blocks of many tiles are shared out where they are few
    constexpr int FOUR = OWN_WAVES * scan_tile(4 * SPL);
    const long most = min((long)P.block, P.tokens), fours = (most + FOUR - 1) / FOUR;
    const int classes = (int)max(1l, min(fours, (SCAN_OWN_WGS + blocks * runs - 1) / (blocks * runs)));
    const long shares = blocks * classes;
    const dim3 grid((unsigned)four_grid(shares, runs)), block(OWN_WAVES * WAVE);
    if (reverse)
        hipLaunchKernelGGL((scan_own_kernel<T, SPL, true>), grid, block, 0, st, P, groups, classes, shares);
    else
        hipLaunchKernelGGL((scan_own_kernel<T, SPL, false>), grid, block, 0, st, P, groups, classes, shares);
    return hipGetLastError();
}

template <typename T, int SPL>
hipError_t launch_decode_t(const ScanDecodeParams &P, hipStream_t st) {
    const int chunks = (P.C + 63) / 64;
    hipLaunchKernelGGL((scan_decode_kernel<T, SPL>), dim3((unsigned)((long)P.N * chunks)), dim3(256),
                       0, st, P, chunks);
    return hipGetLastError();
}

}  // namespace scan

#define KDN_SCAN(fn, ...)                                        \
    switch (P.S) {                                               \
    case 8: return P.bf16 ? scan::fn<bf16, 2>(__VA_ARGS__)       \
                          : scan::fn<float, 2>(__VA_ARGS__);     \
    case 16: return P.bf16 ? scan::fn<bf16, 4>(__VA_ARGS__)      \
                           : scan::fn<float, 4>(__VA_ARGS__);    \
    default: return P.bf16 ? scan::fn<bf16, 8>(__VA_ARGS__)      \
                           : scan::fn<float, 8>(__VA_ARGS__);    \
    }

static hipError_t outputs(const ScanParams &P, hipStream_t st) { KDN_SCAN(launch_t, P, st) }
static hipError_t own(const ScanParams &P, bool reverse, hipStream_t st) {
    KDN_SCAN(launch_own_t, P, reverse, st)
}

static hipError_t joins(const ScanParams &P, bool reverse, hipStream_t st) {
    if (P.N == 0)
        return hipSuccess;
    const int pieces = (int)(((long)P.C * P.S / 2 + scan::JOIN_NT - 1) / scan::JOIN_NT);
    if (reverse)
        hipLaunchKernelGGL((scan::scan_join_kernel<true>), dim3((unsigned)(2l * P.N * pieces)),
                           dim3(scan::JOIN_NT), 0, st, P, pieces);
    else
        hipLaunchKernelGGL((scan::scan_join_kernel<false>), dim3((unsigned)((long)P.N * pieces)),
                           dim3(scan::JOIN_NT), 0, st, P, pieces);
    return hipGetLastError();
}

hipError_t launch_scan_states(const ScanParams &P, bool reverse, hipStream_t st) {
    const hipError_t e = own(P, reverse, st);
    return e == hipSuccess ? joins(P, reverse, st) : e;
}

hipError_t launch_scan(const ScanParams &P, bool several, hipStream_t st) {
    if (P.C == 0)
        return hipSuccess;
    // sequences of several blocks: their states first; sequences without tokens: the
    // joins pass their state on
    const bool empty = (P.block_offsets || P.T == 0) && P.S_out && P.S_out != P.S0;
    const hipError_t e = several ? launch_scan_states(P, false, st)
                                 : (empty ? joins(P, false, st) : hipSuccess);
    return e == hipSuccess ? outputs(P, st) : e;
}

hipError_t launch_scan_decode(const ScanDecodeParams &P, hipStream_t st) {
    if ((long)P.N * P.C == 0)
        return hipSuccess;
    KDN_SCAN(launch_decode_t, P, st)
}
#undef KDN_SCAN

}  // namespace kdn
