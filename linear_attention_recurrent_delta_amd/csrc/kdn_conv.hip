// kdn_conv.hip -- the short causal convolution in front of a recurrence (gfx950):
//   s_t = bias + sum_j w_j x_{t-W+1+j},   y_t = s_t sigmoid(s_t)   (or s_t),
// per channel, W <= 4 taps.  The rows before a sequence are its state, the last
// W - 1 rows of x, kept in the call's type: they are the inputs themselves.
// Bound by memory: x read and y written once.  A lane owns VEC neighbouring
// channels (16 bytes) of RT consecutive tokens, so that a wave reads whole lines
// and every row is read (RT + W - 1) / RT times, the second time from the caches;
// all rows of a lane are requested before the first is used.  37 packed prompts
// (22 thousand tokens) of 6144 channels, bf16, states in a pool: 112 us, 4.8 TB/s,
// 571 MB moved where 539 have to be.
#include "kdn_act.h"
#include "kdn_batch_device.h"
#include "kdn_conv.h"

#include <initializer_list>

namespace kdn {
namespace conv {

constexpr int NT = 256, NW = NT / WAVE;

// Where a workgroup is: tile of tokens and 64 * VEC channels, or (behind the
// tiles) one sequence.
struct Place {
    long tile;
    int chunk;
};
__device__ __forceinline__ Place place(int chunks) {
    return Place{(long)blockIdx.x / chunks, (int)(blockIdx.x % chunks)};
}

// Tile `id` of a batch: its block, and in t0 the tile's first token in it (a block without
// tokens where there is no such tile).  sub > 0: tile id % sub of block id / sub.  sub 0:
// tile j of block b has the number first / CONV_TILE + b + j, so that there are as many
// numbers as tokens and blocks need, however long a block may be; the block is the last
// whose first number is not behind id, which the wave's 64 lanes look for together (all of
// them have to come here): 37 packed prompts (21830 tokens) of 6144 channels in a table of
// one block a sequence 105 us, as with blocks of 256.
__device__ __forceinline__ Block tile_block(const ConvParams &P, long id, int sub, int &t0) {
    if (sub > 0) {
        t0 = (int)(id % sub) * CONV_TILE;
        return get_block(P, id / sub);
    }
    const int lane = threadIdx.x & (WAVE - 1);
    // rows of the table that hold blocks; device data, so kept within the table
    long lo = 0, hi = min(max(__builtin_amdgcn_readfirstlane(P.block_offsets[P.N]), 0), P.nblocks);
    while (hi - lo > 1) {
        const long step = (hi - lo + WAVE - 1) / WAVE, row = lo + lane * step;
        const bool before = row < hi && P.blocks[4 * row] / CONV_TILE + row <= id;
        const int n = __builtin_popcountll(__ballot(before));
        lo += (n > 1 ? n - 1 : 0) * step;
        hi = min(hi, lo + step);
    }
    Block B = get_block(P, lo);
    const long t = B.count > 0 ? (id - B.first / CONV_TILE - lo) * CONV_TILE : 0;
    t0 = 0;
    if (t < 0 || t >= B.count)
        B.count = 0;
    else
        t0 = (int)t;
    return B;
}

// Rows of VEC channels of a lane, n of them there (the same in every lane).  WHOLE: rows of
// whole pieces on their boundaries, through a descriptor that ends with the last row, so
// that rows behind it read 0 and are not written without a branch; else by the pieces'
// elements.
template <typename T, int VEC, bool WHOLE> struct Lines {
    typedef Pack<T, VEC> V;
    __amdgpu_buffer_rsrc_t d;
    T *p;
    long pitch;
    unsigned lane, step;
    int n, nc;
    // base: the first row (the same in every lane); c, nc: the lane's first channel and
    // how many of its VEC are there
    __device__ __forceinline__ Lines(const void *base, long pitch_, int C, long n_, long c, int nc_) {
        n = (int)(n_ < 0 ? 0 : (n_ > 64 ? 64 : n_));
        nc = nc_;
        pitch = pitch_;
        p = static_cast<T *>(const_cast<void *>(base)) + c;
        if constexpr (WHOLE) {
            step = (unsigned)pitch * sizeof(T);
            lane = (unsigned)c * sizeof(T);
            d = buf_rsrc(base, n > 0 ? (n - 1) * step + (unsigned)C * sizeof(T) : 0u);
        }
    }
    __device__ __forceinline__ void load(V &v, int i) const {
        if constexpr (WHOLE) {
            const int at = (int)(lane + (unsigned)i * step);
            if constexpr (VEC * sizeof(T) == 16)
                v.r = __builtin_bit_cast(typename V::Vec, __builtin_amdgcn_raw_buffer_load_b128(d, at, 0, 0));
            else
                v.r = __builtin_bit_cast(typename V::Vec, __builtin_amdgcn_raw_buffer_load_b64(d, at, 0, 0));
        } else {
            v.zero();
            if (i < n)
                v.load(p + (long)i * pitch, nc);
        }
    }
    __device__ __forceinline__ void store(const V &v, int i) const {
        if constexpr (WHOLE) {
            const int at = (int)(lane + (unsigned)i * step);
            if constexpr (VEC * sizeof(T) == 16)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(__attribute__((ext_vector_type(4))) unsigned, v.r), d, at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b64(
                    __builtin_bit_cast(__attribute__((ext_vector_type(2))) unsigned, v.r), d, at, 0, 0);
        } else {
            if (i < n)
                v.store(p + (long)i * pitch, nc);
        }
    }
};

// Weights of VEC channels, tap j of channel e in w[j][e], and the bias.
template <int VEC, int W>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, long c, int n,
                                             float (&w)[W][VEC], float (&b)[VEC]) {
    Pack<float, W> taps;
    Pack<float, VEC> first;
    first.zero();
    if (bias)
        first.load(bias + c, n);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        taps.zero();
        if (e < n)
            taps.load(weight + (c + e) * W);
#pragma unroll
        for (int j = 0; j < W; ++j)
            w[j][e] = taps.get(j);
        b[e] = first.get(e);
    }
}

template <typename T, int VEC, int W, int RT, bool WHOLE>
__global__ __launch_bounds__(NT) void conv_kernel(ConvParams P, int chunks, int sub, long tiles) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int H = W - 1;
    static_assert(NW * RT == CONV_TILE, "a workgroup's tokens");
    const int lane = threadIdx.x & (WAVE - 1);
    const Place at = place(chunks);
    const long c = ((long)at.chunk * WAVE + lane) * VEC;
    T *state_out = static_cast<T *>(P.state_out);
    const T *state0 = static_cast<const T *>(P.state0);
    const int nc = (int)min((long)VEC, P.C - c);     // channels of this lane
    typedef Pack<T, VEC> V;
    if (at.tile >= tiles) {
        // a sequence without tokens passes its state on
        if (at.chunk > 0 || !state_out || state_out == state0)
            return;
        const long slot = empty_slot(P, (int)(at.tile - tiles));
        if (slot < 0)
            return;
        for (long i = threadIdx.x; i < (long)H * P.C; i += NT)
            state_out[slot * H * P.C + i] = state0 ? state0[slot * H * P.C + i] : from_f32<T>(0.f);
        return;
    }
    int t0;
    const Block B = tile_block(P, at.tile, sub, t0);
    t0 += wave_id() * RT;
    if (t0 >= B.count || B.slot < 0 || c >= P.C)
        return;
    const bool start = B.index == 0 && t0 == 0;
    typedef Lines<T, VEC, WHOLE> L;
    const T *x = static_cast<const T *>(P.x) + B.first * P.x_stride + c;
    const T *x0 = static_cast<const T *>(P.x) + (B.first + t0) * P.x_stride;
    // the tokens' rows and the H before them (of a sequence's start: the state's)
    const L here(x0, P.x_stride, P.C, B.count - t0, c, nc);
    const L before(start ? state0 + B.slot * H * P.C : x0 - H * P.x_stride, start ? P.C : P.x_stride, P.C,
                   start ? (state0 ? H : 0) : (B.first + t0 >= H ? H : 0), c, nc);
    V rows[RT + H];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        here.load(rows[H + i], i);
#pragma unroll
    for (int i = 0; i < H; ++i)
        before.load(rows[i], i);
    if (start) {
        const long at0 = B.slot * H * P.C + c;
        if (state_out) {
            // the last W - 1 of the sequence's rows with its state before them; the
            // state has been read, and no other thread reads or writes it
            const long n = tokens_left(P, B);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                V last;
                last.zero();
                if (n + i >= H)
                    last.load(x + (n + i - H) * P.x_stride, nc);
#pragma unroll
                for (int j = 1; j < H; ++j)
                    if (n + i == j)
                        last = rows[j];
                last.store(state_out + at0 + (long)i * P.C, nc);
            }
        }
    }
    float w[W][VEC], b[VEC];
    load_weights<VEC, W>(P.weight, P.bias, c, nc, w, b);
    const L y(static_cast<T *>(P.y) + (B.first + t0) * P.C, P.C, P.C, B.count - t0, c, nc);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        V out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = b[e];
#pragma unroll
            for (int j = 0; j < W; ++j)
                s = fmaf(w[j][e], rows[i + j].get(e), s);
            out.set(e, P.silu ? silu_f32<FINE>(s) : s);
        }
        y.store(out, i);
    }
}

// ---------------------------------------------------------------------------
// Single tokens: a thread shifts the state of VEC channels of one row, its W rows
// and weights all requested at once.  One wave a workgroup, to spread few rows over
// the CUs.  45 rows of 6144 channels, bf16: 4.4 us, of which 0.9 are for the bytes;
// a call is bound by its launch (8.9 us).
// ---------------------------------------------------------------------------
template <typename T, int VEC, int W>
__global__ __launch_bounds__(WAVE) void conv_decode_kernel(ConvDecodeParams P, int chunks) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int H = W - 1;
    const Place at = place(chunks);
    const long c = ((long)at.chunk * WAVE + threadIdx.x) * VEC;
    const long slot = P.slots ? P.slots[at.tile] : at.tile;
    if (slot < 0 || slot >= P.pool || c >= P.C)
        return;
    T *state = static_cast<T *>(P.state) + slot * H * P.C + c;
    const int nc = (int)min((long)VEC, P.C - c);
    Pack<T, VEC> rows[W];
    rows[H].load(static_cast<const T *>(P.x) + at.tile * P.x_stride + c, nc);
#pragma unroll
    for (int i = 0; i < H; ++i)
        rows[i].load(state + (long)i * P.C, nc);
    float w[W][VEC], b[VEC];
    load_weights<VEC, W>(P.weight, P.bias, c, nc, w, b);
#pragma unroll
    for (int i = 0; i < H; ++i)
        rows[i + 1].store(state + (long)i * P.C, nc);
    Pack<T, VEC> out;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float s = b[e];
#pragma unroll
        for (int j = 0; j < W; ++j)
            s = fmaf(w[j][e], rows[j].get(e), s);
        out.set(e, P.silu ? silu_f32<FINE>(s) : s);
    }
    out.store(static_cast<T *>(P.y) + at.tile * P.C + c, nc);
}

// ---------------------------------------------------------------------------
// Gradients: with ds_t = dy_t act'(s_t) (s made again from x),
//   dx_t = sum_j w_j ds_{t+W-1-j},  dw_j = sum_t ds_t x_{t-W+1+j},  db = sum_t ds_t,
// the same sum for the rows of the state before the sequence, and what reaches
// the state behind it added to its last rows.  Bound by memory: x and dy read, dx
// written.  A lane walks RT tokens and the W - 1 behind them, whose ds it makes
// again, with 8 bytes of each row: 16 would not leave registers for two workgroups a
// CU.  B4 T4096 of 2048 channels, bf16: 52 us, 3.9 TB/s and 66 % of the vector units'
// time (each activation and its slope take an exponential and a division, (RT + W - 1)
// / RT times), and the sums 4.8.  A workgroup keeps the sums of its channels over all its tiles (every
// `parts`-th, 32 at most) in registers and writes them once; a second kernel adds the parts
// in order, in 64 bits.
// ---------------------------------------------------------------------------
template <typename T, int VEC, int W, bool WHOLE>
__global__ __launch_bounds__(NT) void conv_grad_kernel(ConvParams P, int chunks, int sub,
                                                       long tiles) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int H = W - 1, RT = CONV_TILE / NW;
    const int lane = threadIdx.x & (WAVE - 1), wv = wave_id();
    const int chunk = blockIdx.x % chunks, part = blockIdx.x / chunks;
    const long c = ((long)chunk * WAVE + lane) * VEC;
    const bool live = c < P.C;
    const int nc = (int)min((long)VEC, P.C - c);     // channels of this lane
    typedef Pack<T, VEC> V;
    float w[W][VEC], b[VEC], dw[W + 1][VEC];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            dw[j][e] = 0.f;
    if (live)
        load_weights<VEC, W>(P.weight, P.bias, c, nc, w, b);
    for (long tile = part; tile < tiles; tile += P.parts) {
        int t0;
        const Block B = tile_block(P, tile, sub, t0);     // (every lane takes part in it)
        t0 += wv * RT;
        if (t0 >= B.count || !live)
            continue;
        typedef Lines<T, VEC, WHOLE> L;
        const int n = min(RT, B.count - t0);      // own tokens
        const L dx(static_cast<T *>(P.dx) + (B.first + t0) * P.C, P.C, P.C, n, c, nc);
        if (B.slot < 0) {
            V none;
            none.zero();
            for (int i = 0; i < n; ++i)
                dx.store(none, i);
            continue;
        }
        const long left = tokens_left(P, B) - t0;     // tokens to the sequence's end
        const bool start = B.index == 0 && t0 == 0;
        const T *state0 = static_cast<const T *>(P.state0);
        const T *dlast = static_cast<const T *>(P.dstate_out);
        const long at0 = B.slot * H * P.C + c;
        // rows t0 - H .. t0 + RT + H - 1 of x and t0 .. of dy, those of the sequence
        const T *x0 = static_cast<const T *>(P.x) + (B.first + t0) * P.x_stride;
        const L here(x0, P.x_stride, P.C, left, c, nc);
        const L before(start ? state0 + B.slot * H * P.C : x0 - H * P.x_stride,
                       start ? P.C : P.x_stride, P.C,
                       start ? (state0 ? H : 0) : (B.first + t0 >= H ? H : 0), c, nc);
        const L dy(static_cast<const T *>(P.d_y) + (B.first + t0) * P.C, P.C, P.C, left, c, nc);
        V xs[RT + 2 * H], g[RT + H];
#pragma unroll
        for (int i = 0; i < H; ++i)
            before.load(xs[i], i);
#pragma unroll
        for (int i = 0; i < RT + H; ++i) {
            here.load(xs[H + i], i);
            dy.load(g[i], i);
        }
        // near[k] = ds of token i - H + 1 + k
        float near[W][VEC];
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                near[k][e] = 0.f;
#pragma unroll
        for (int i = 0; i < RT + H; ++i) {
            V out;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
#pragma unroll
                for (int k = 0; k < H; ++k)
                    near[k][e] = near[k + 1][e];
                float d = g[i].get(e);
                if (P.silu) {
                    float s = b[e], y, dact;
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        s = fmaf(w[j][e], xs[i + j].get(e), s);
                    silu_grad<FINE>(s, y, dact);
                    d *= dact;
                }
                // tokens behind the sequence have no gradient, whatever s was
                d = i < left ? d : 0.f;
                near[H][e] = d;
                if (i < n) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        dw[j][e] = fmaf(d, xs[i + j].get(e), dw[j][e]);
                    dw[W][e] += d;
                }
                // the row H before: dx_t = sum_k w_{H-k} ds_{t+k}
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    sum = fmaf(w[H - k][e], near[k][e], sum);
                out.set(e, sum);
            }
            // row t0 + i - H, of the sequence or of the state before it
            const int t = i - H;
            if (t >= 0 ? t < n : start && P.dstate0) {
                if (dlast && left - t <= H) {
                    V last;
                    last.load(dlast + at0 + (long)(H + t - left) * P.C, nc);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float sum = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            sum = fmaf(w[H - k][e], near[k][e], sum);
                        out.set(e, sum + last.get(e));
                    }
                }
                if (t >= 0)
                    dx.store(out, t);
                else
                    out.store(static_cast<T *>(P.dstate0) + at0 + (long)i * P.C, nc);
            }
        }
    }
    // sums over the four waves, in order
    __shared__ float sums[NW][W + 1][WAVE * VEC];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            sums[wv][j][lane * VEC + e] = dw[j][e];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * WAVE * VEC; i += NT) {
        const int j = i / (WAVE * VEC), k = i % (WAVE * VEC);
        const long cc = (long)chunk * WAVE * VEC + k;
        if (cc < P.C) {
            float s = sums[0][j][k];
#pragma unroll
            for (int q = 1; q < NW; ++q)
                s += sums[q][j][k];
            P.ws[((long)part * (W + 1) + j) * P.C + cc] = s;
        }
    }
}

// The parts' sums, 16 columns a workgroup; behind those workgroups: zero gradients of
// the rows behind the last sequence, and the states' of sequences without tokens.
constexpr int TAIL_WGS = 64;
template <typename T>
__global__ __launch_bounds__(NT) void conv_sum_kernel(ConvParams P, long wide) {
    const int W = P.W;
    const long id = blockIdx.x;
    if (id < wide) {
        __shared__ double lds[NW][16];
        const long n = (long)(W + 1) * P.C;
        for (long first = id * 16; first < n; first += wide * 16) {
            const long i = first + threadIdx.x;
            const double s = part_sums<NT>(P.ws, n, P.parts, first, lds);
            if (threadIdx.x < 16 && i < n) {
                const long j = i / P.C, c = i - j * P.C;
                if (j < W)
                    P.dweight[c * W + j] = (float)s;
                else if (P.dbias)
                    P.dbias[c] = (float)s;
            }
            __syncthreads();             // the sums have been read
        }
        return;
    }
    const long wg = id - wide;
    if (wg < TAIL_WGS) {
        if (!P.block_offsets)
            return;
        const long first = tail_start(P);
        for (long i = first * P.C + wg * NT + threadIdx.x; i < P.tokens * P.C;
             i += (long)TAIL_WGS * NT)
            static_cast<T *>(P.dx)[i] = from_f32<T>(0.f);
        return;
    }
    if (!P.dstate0)
        return;
    const long slot = empty_slot(P, (int)(wg - TAIL_WGS)), size = (long)(W - 1) * P.C;
    if (slot < 0)
        return;
    const T *dlast = static_cast<const T *>(P.dstate_out);
    for (long i = threadIdx.x; i < size; i += NT)
        static_cast<T *>(P.dstate0)[slot * size + i] = dlast ? dlast[slot * size + i]
                                                             : from_f32<T>(0.f);
}

// Rows of whole pieces of `bytes` bytes on such boundaries, near enough for 32 bits: they
// are read through descriptors (37 packed prompts 111 us, by elements' addresses and
// branches 130; gradients B4 T4096 of 2048 channels 56 and 64).
bool whole(int C, long stride, int es, int bytes, std::initializer_list<const void *> p) {
    bool ok = C * (long)es % bytes == 0 && stride * es % bytes == 0 && stride < (1l << 24);
    for (const void *x : p)
        ok = ok && (reinterpret_cast<uintptr_t>(x) & (bytes - 1)) == 0;
    return ok;
}

// Blocks and tiles of a launch: of a dense batch a block is a tile.
struct Tiles {
    ConvParams P;
    long n;
    int sub;
    explicit Tiles(const ConvParams &P_) : P(P_), n(conv_tiles(P_, P_.block_offsets)), sub(1) {
        if (!P.block_offsets) {
            P.block = CONV_TILE;
            P.nblocks = (int)((P.T + CONV_TILE - 1l) / CONV_TILE);
        } else {
            sub = n == P.nblocks * conv_block_tiles(P) ? (int)conv_block_tiles(P) : 0;
        }
    }
};

template <typename T, int VEC, int W>
hipError_t launch_conv_fwd_t(const ConvParams &P, hipStream_t st) {
    // tokens of a lane (8, 16 and 32: 37 prompts of 590 tokens, C 6144 bf16, 116, 108 and 116 us)
    constexpr int RT = CONV_TILE / NW;
    const int chunks = conv_chunks(P.C, VEC);
    const Tiles q(P);
    const long empty = P.state_out && P.state_out != P.state0 && (P.block_offsets || P.T == 0) ? P.N : 0;
    if (q.n + empty == 0)
        return hipSuccess;
    const dim3 grid((unsigned)((q.n + empty) * chunks)), block(NT);
    if (whole(P.C, P.x_stride, sizeof(T), VEC * sizeof(T), {P.x, P.y, P.state0, P.state_out}))
        hipLaunchKernelGGL((conv_kernel<T, VEC, W, RT, true>), grid, block, 0, st, q.P, chunks, q.sub, q.n);
    else
        hipLaunchKernelGGL((conv_kernel<T, VEC, W, RT, false>), grid, block, 0, st, q.P, chunks, q.sub, q.n);
    return hipGetLastError();
}

template <typename T, int VEC, int W>
hipError_t launch_conv_decode_t(const ConvDecodeParams &P, hipStream_t st) {
    const int chunks = conv_chunks(P.C, VEC);
    hipLaunchKernelGGL((conv_decode_kernel<T, VEC, W>), dim3((unsigned)((long)P.N * chunks)),
                       dim3(WAVE), 0, st, P, chunks);
    return hipGetLastError();
}

template <typename T, int VEC, int W>
hipError_t launch_conv_grad_t(const ConvParams &P, hipStream_t st) {
    const int chunks = conv_chunks(P.C, VEC);
    const Tiles q(P);
    if (P.parts > 0) {
        const dim3 grid((unsigned)(chunks * (long)P.parts)), block(NT);
        if (whole(P.C, P.x_stride, sizeof(T), VEC * sizeof(T), {P.x, P.d_y, P.dx, P.state0}))
            hipLaunchKernelGGL((conv_grad_kernel<T, VEC, W, true>), grid, block, 0, st, q.P, chunks, q.sub, q.n);
        else
            hipLaunchKernelGGL((conv_grad_kernel<T, VEC, W, false>), grid, block, 0, st, q.P, chunks, q.sub, q.n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    const long wide = min(((long)(W + 1) * P.C + 15) / 16, 65536l);
    const long empty = P.dstate0 && (P.block_offsets || P.T == 0) ? P.N : 0;
    hipLaunchKernelGGL((conv_sum_kernel<T>), dim3((unsigned)(wide + TAIL_WGS + empty)),
                       dim3(NT), 0, st, P, wide);
    return hipGetLastError();
}

}  // namespace conv

#define KDN_CONV(fn, T_, V_)                              \
    switch (P.W) {                                        \
    case 2: return conv::fn<T_, V_, 2>(P, stream);        \
    case 3: return conv::fn<T_, V_, 3>(P, stream);        \
    default: return conv::fn<T_, V_, 4>(P, stream);       \
    }

hipError_t launch_conv(const ConvParams &P, hipStream_t stream) {
    if (P.bf16)
        KDN_CONV(launch_conv_fwd_t, bf16, 8)
    KDN_CONV(launch_conv_fwd_t, float, 4)
}

hipError_t launch_conv_decode(const ConvDecodeParams &P, hipStream_t stream) {
    if ((long)P.N * P.C == 0)
        return hipSuccess;
    if (P.bf16)
        KDN_CONV(launch_conv_decode_t, bf16, 8)
    KDN_CONV(launch_conv_decode_t, float, 4)
}

hipError_t launch_conv_backward(const ConvParams &P, hipStream_t stream) {
    if (P.C == 0)
        return hipSuccess;
    if (P.bf16)
        KDN_CONV(launch_conv_grad_t, bf16, 4)
    KDN_CONV(launch_conv_grad_t, float, 2)
}
#undef KDN_CONV

}  // namespace kdn
