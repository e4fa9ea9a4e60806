// kdn_linear_device.h -- device-side pieces shared by the linear-attention
// kernels: which tokens a workgroup owns, MFMA fragments, and the decays of a
// chunk.
#pragma once

#include "kdn_batch_device.h"
#include "kdn_linear.h"

namespace kdn {
namespace lin {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// ---------------------------------------------------------------------------
// Fragments of 32 x 32 tiles: the 8 contraction elements of one lane for a
// step of 16.  For bfloat16 they are the operand of one
// v_mfma_f32_32x32x16_bf16 (half as many operand reads and instructions for
// the same products as 16 x 16 tiles); for float32 element s of every lane is
// the operand of the s-th of eight v_mfma_f32_32x32x2_f32.  Lane l holds row
// (A) or column (B) n = l & 31 and the half h = l >> 5 of the contraction;
// which 8 of the 16 indices those are only has to agree between A and B.
// Accumulator register r of lane l: row 8 (r / 4) + 4 h + r % 4, column n.
// ---------------------------------------------------------------------------
template <typename T> struct Frag;
template <> struct Frag<bf16> { typedef bf16x8 V; };
template <> struct Frag<float> { typedef f32x8 V; };
template <typename T> using FragV = typename Frag<T>::V;
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        z[i] = 0.f;
    return z;
}
__device__ __forceinline__ void mma(f32x16 &acc, bf16x8 a, bf16x8 b) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &acc, f32x8 a, f32x8 b) {
#pragma unroll
    for (int s = 0; s < 8; ++s)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[s], b[s], acc, 0, 0, 0);
}

// 16 x 16 tiles, for products that are shared out among waves in smaller
// pieces: row or column lane & 15, the lane's 8 of 32 contraction elements from
// 8 (lane >> 4); accumulator register r: row 4 (lane >> 4) + r.
__device__ __forceinline__ void mma(f32x4 &acc, bf16x8 a, bf16x8 b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, f32x8 a, f32x8 b) {
#pragma unroll
    for (int s = 0; s < 8; ++s)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
}

// p: this lane's row at its 8 consecutive elements (contraction 8 h + e).
__device__ __forceinline__ bf16x8 frag_row(const bf16 *p) {
    return *reinterpret_cast<const bf16x8 *>(p);
}
__device__ __forceinline__ f32x8 frag_row(const float *p) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Rows 16 b .. + 15 of an accumulator tile, whose row operand was read in the
// order of chan(), as the fragment whose contraction runs over them.
template <typename T> __device__ __forceinline__ FragV<T> frag_acc(const f32x16 &a, int b) {
    FragV<T> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = from_f32<T>(a[8 * b + e]);
    return f;
}

// What that rounding leaves, to T.
template <typename T> __device__ __forceinline__ FragV<T> frag_rest(const f32x16 &a, int b) {
    FragV<T> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = from_f32<T>(a[8 * b + e] - to_f32(from_f32<T>(a[8 * b + e])));
    return f;
}

// Channel of row or column n of a 32-channel tile.  The middle bits of the
// groups of 4 change places, so that accumulator registers 0-7 and 8-15 of a
// lane are 8 consecutive channels each, from 8 h and 16 + 8 h.
__device__ __forceinline__ int chan(int n) {
    const int q = n >> 2;
    return 4 * ((q & 4) | ((q & 1) << 1) | ((q >> 1) & 1)) + (n & 3);
}

// Place of row r of an LDS tile: within each 16 rows the 4 x 4 transpose.  A
// transposed read takes 4 neighbouring rows, 16 banks of each; at the pitches of
// lds_pitch rows 4 places apart are the ones that fill the 64 banks (next to
// each other, half of the read's cycles were conflicts), and 16 neighbouring
// rows at the same column still fall into 16 different groups of 4.
__device__ __forceinline__ int lds_row(int r) {
    return (r & ~15) | ((r & 3) << 2) | ((r >> 2) & 3);
}

// Transposed read of a tile [token][channel], rows as in lds_row: tokens 8 h + e
// of the 16 behind `m`, channel n of the 32 behind `m` (CH: in the order of
// chan()).  bfloat16: ds_read_b64_tr_b16 gives lane i of a group of 16 column i
// of the 4 rows x 16 columns whose 8-byte pieces the lanes point to (lane i: row
// i / 4, columns 4 (i % 4) .. + 3).
template <int PITCH, bool CH>
__device__ __forceinline__ bf16x8 frag_cols(const bf16 *m, int lane) {
    const int i = lane & 15, h = lane >> 5, q = 4 * ((lane >> 4) & 1) + (i & 3);
    const bf16 *p = m + (4 * (i >> 2) + 2 * h) * PITCH + (CH ? chan(4 * q) : 4 * q);
    union { s16x4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + PITCH));
    return u.v;
}
template <int PITCH, bool CH>
__device__ __forceinline__ f32x8 frag_cols(const float *m, int lane) {
    const int n = lane & 31, h = lane >> 5;
    const float *p = m + 2 * h * PITCH + (CH ? chan(n) : n);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = p[(4 * (e % 4) + e / 4) * PITCH];
    return f;
}

// x (.) w as an operand of more bits than T has: bfloat16 as the sum of PARTS
// operands.  Three have 24 significant bits: states that a call returns, and
// what goes into them, stay float32.  Two leave 2^-16 of a term (2.4e-6 of a
// state as measured): for states that are only read rounded to bfloat16,
// within a block or a chunk's saved state (one would show, at 2^-8).  float32
// is one operand.  It is made in 4 PARTS steps, each a part of a pair of
// elements, so that they can stand between MFMAs.
template <typename T, int N> struct Split;
template <int N> struct Split<bf16, N> {
    static constexpr int PARTS = N;
    bf16x8 part[N];                  // low to high
    float y[2];                      // what is left of the pair
    __device__ __forceinline__ void step(int i, bf16x8 x, const float (&w)[8]) {
        const int p = 2 * (i / N), l = i % N;
        if (l == 0) {
            y[0] = to_f32(x[p]) * w[p];
            y[1] = to_f32(x[p + 1]) * w[p + 1];
        } else {
            y[0] -= static_cast<float>(part[N - l][p]);
            y[1] -= static_cast<float>(part[N - l][p + 1]);
        }
        part[N - 1 - l][p] = static_cast<bf16>(y[0]);
        part[N - 1 - l][p + 1] = static_cast<bf16>(y[1]);
    }
};
template <int N> struct Split<float, N> {
    static constexpr int PARTS = 1;
    f32x8 part[1];
    __device__ __forceinline__ void step(int i, f32x8 x, const float (&w)[8]) {
        part[0][2 * i] = x[2 * i] * w[2 * i];
        part[0][2 * i + 1] = x[2 * i + 1] * w[2 * i + 1];
    }
};

// acc[i] += sum over the chunk's tokens of a_i (w (.) b): the update of a state.
// b[s]: the column operand of 16 tokens (s = 0 .. KS - 1), w: the tokens'
// weights in LDS, rows(s, i): the row operand of tile i.  cur and a come with
// the operands of the first step.  Between the MFMAs of a step stand the reads
// and the splitting of the next one and extra(u), u = 0 .. U - 1 the MFMA's
// number (the next chunk's loads), a few instructions behind each MFMA
// (sched_barrier holds them there: left alone the compiler reads, waits,
// splits and multiplies one after the other, and two waves a SIMD cannot hide
// that).
template <typename T, int PARTS, int N, int KS, typename Rows, typename Extra>
__device__ __forceinline__ void update_state(f32x16 (&acc)[N], const FragV<T> (&b)[KS],
                                             const float *w, int hf, Split<T, PARTS> &cur,
                                             FragV<T> (&a)[N], Rows rows, Extra extra) {
    typedef Split<T, PARTS> S;
    constexpr int M = S::PARTS * N, STEPS = 4 * S::PARTS;    // of 16 tokens
    S nxt;
    float wt[8];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const bool more = s + 1 < KS;
        if (more)
            lds_ld8(w + 16 * (s + 1) + 8 * hf, wt);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            mma(acc[m % N], a[m % N], cur.part[m / N]);
            if (more) {
                if (m >= M - N)              // its last use in this step
                    a[m % N] = rows(s + 1, m % N);
#pragma unroll
                for (int i = m * STEPS / M; i < (m + 1) * STEPS / M; ++i)
                    nxt.step(i, b[s + 1], wt);
            }
            extra(s * M + m, KS * M);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (more)
            cur = nxt;
    }
}

// sum over D channels of a tile's rows: acc += A B^T, the rows of lane n at a
// and b (8 h on).  The operands of STEPS steps are read before the first of
// their products, so that their latency is paid once.
template <typename T, int D, int STEPS>
__device__ __forceinline__ void mma_rows(f32x16 &acc, const T *a, const T *b) {
    constexpr int G = sizeof(T) == 4 ? 2 : (STEPS < D / 16 ? STEPS : D / 16);
#pragma unroll
    for (int s0 = 0; s0 < D / 16; s0 += G) {
        FragV<T> x[G], y[G];
#pragma unroll
        for (int s = 0; s < G; ++s) {
            x[s] = frag_row(a + 16 * (s0 + s));
            y[s] = frag_row(b + 16 * (s0 + s));
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < G; ++s)
            mma(acc, x[s], y[s]);
    }
}

// ---------------------------------------------------------------------------
// Decays of a chunk, all in powers of two.  Prefix sums of the log-decays run
// in 64 bits: a difference of two of them must keep its own bits also behind
// strong decays.  A log-decay below -152 (base 2) counts as -152, whose power
// is 0 in float32 as that of -infinity is, so that a reset costs no NaN.
// ---------------------------------------------------------------------------
// Aligned, since it is read 16 bytes at a time and stands in arrays.  Tokens
// behind the end decay by nothing, so the last one's 2^G_i is 2^G_C.
template <int C> struct alignas(16) Decays {
    float hi[C], lo[C];   // prefix sum G_i in two floats
    float in[C];          // 2^G_i: from the chunk's start through token i
    float out[C];         // 2^(G_C - G_j): behind token j to the chunk's end
    __device__ __forceinline__ float all() const { return in[C - 1]; }     // 2^G_C
};
static_assert(sizeof(Decays<32>) == 4 * 32 * sizeof(float) &&
                  sizeof(Decays<64>) == 4 * 64 * sizeof(float),
              "no padding, every element of an array aligned");

constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESET2 = -152.f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ double log2_decay(float la) {
    const float g = la * LOG2E;
    // NaN stays NaN: no fmax
    return g < RESET2 ? (double)RESET2 : (double)la * 1.4426950408889634074;
}

// x + (x of the lane CTRL names, 0 where there is none or the row is not in
// ROWS), in 64 bits by moves of the halves within the registers.
template <int CTRL, int ROWS> __device__ __forceinline__ double add_dpp(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive prefix sums over the lanes, and the value of a lane.
__device__ __forceinline__ double prefix_sum(double x) {
    x = add_dpp<0x111, 0xf>(x);      // the lane before, 2, 4 and 8 before (rows of 16)
    x = add_dpp<0x112, 0xf>(x);
    x = add_dpp<0x114, 0xf>(x);
    x = add_dpp<0x118, 0xf>(x);
    x = add_dpp<0x142, 0xa>(x);      // the end of the row before, to rows 1 and 3
    return add_dpp<0x143, 0xc>(x);   // lane 31, to rows 2 and 3
}
__device__ __forceinline__ double lane_value(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// One wave: lane j < C holds the log-decay (natural) of token j, 0 behind the
// end.  Returns the base-2 sum of the chunk.
template <int C>
__device__ __forceinline__ double chunk_decays(Decays<C> &D, float la, int lane) {
    const double x = prefix_sum(log2_decay(la));
    const double all = lane_value(x, C - 1);
    if (lane < C) {
        const float hi = (float)x;
        D.hi[lane] = hi;
        D.lo[lane] = (float)(x - (double)hi);
        D.in[lane] = exp2_fast((float)x);
        D.out[lane] = exp2_fast((float)(all - x));
    }
    return all;
}

// 2^(G_i - G_j) of N (a multiple of 4) consecutive j, 0 right of the diagonal
// (j > i)
template <typename T, int C, int N>
__device__ __forceinline__ void decay_between(const Decays<C> &D, float hi_i, float lo_i, int i,
                                              int j, float (&d)[N]) {
#pragma unroll
    for (int q = 0; q < N; q += 4) {
        f32x4 x = hi_i - *reinterpret_cast<const f32x4 *>(D.hi + j + q);
        // bfloat16 products: the low parts are 2^-24 of a prefix sum, of at most
        // 64 resets (2^14) 7e-4 of the factor, a sixth of the product's rounding,
        // and of common decays nothing of it
        if (sizeof(T) == 4)
            x += lo_i - *reinterpret_cast<const f32x4 *>(D.lo + j + q);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float y = exp2_fast(x[r]);
            d[q + r] = j + q + r <= i ? y : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// Loads of a chunk's rows through buffer descriptors: rows behind the last
// return 0 without a branch.  (A guarded and an unguarded load path that meet
// make the compiler wait for the loads in flight on each of them.)
// ---------------------------------------------------------------------------

// The log-decays of a chunk, one per lane, on their way: the bits as they were
// loaded, made a float only where they are used.
template <typename T> struct GateReg {
    uint32_t bits = 0;
    // tokens first .. + count - 1 (at most C) of head h; lane j has token j
    template <int C>
    __device__ __forceinline__ void load(const LinearParams &P, long first, int count, int h,
                                         int lane) {
        if (P.gate == KDN_GATE_HEAD)
            return;
        const int rows = min(count, C);
        const auto r = buf_rsrc(static_cast<const T *>(P.la) + first * P.H + h,
                                rows > 0 ? ((rows - 1) * (unsigned)P.H + 1) * sizeof(T) : 0u);
        const int at = (int)(lane * (unsigned)P.H * sizeof(T));
        if constexpr (sizeof(T) == 2)
            bits = __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0);
        else
            bits = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0);
    }
    // head: the head's constant; live: the lane has a token
    __device__ __forceinline__ float value(const LinearParams &P, float head, bool live) const {
        if (P.gate == KDN_GATE_HEAD)
            return live ? head : 0.f;
        return __uint_as_float(sizeof(T) == 2 ? bits << 16 : bits);
    }
};

// Elements between the rows of an LDS tile of D columns.  16 rows at the same
// 16 bytes (frag_row) have to fall into different groups of 4 banks (the pitch
// an odd multiple of 4 of the 64), and the 4 rows of a transposed read, 4 places
// apart (lds_row), 16 banks from each other: 76 and 36 banks for bfloat16, one
// group more than the row for float32.  (Row reads of 16 x 16 tiles lose 4 cycles
// of 12 to conflicts at any such pitch.)
template <typename T> constexpr int lds_pitch(int d) {
    return sizeof(T) == 4 ? d + 4 : (d == 128 ? 152 : d + 8);
}

// A tile [ROWS][COLS] from global memory, held in registers between its load
// and its store to LDS (NT threads, 16-byte pieces); rows behind `count` are
// zero and not read.  The entry points keep ROWS strides below 2^32 bytes.
template <typename T, int ROWS, int COLS, int NT> struct TileRegs {
    static constexpr int VEC = 16 / sizeof(T);
    static constexpr int PER_ROW = COLS / VEC;
    static constexpr int STEP = NT / PER_ROW;          // rows of one pass
    static constexpr int N = ROWS / STEP;
    static_assert(NT % PER_ROW == 0 && ROWS % STEP == 0, "tile shape");
    f32x4 r[N];

    // base: the tile's first row (element pointer), stride in elements
    struct Source {
        __amdgpu_buffer_rsrc_t d;
        unsigned at, pitch;
        __device__ __forceinline__ Source(const T *base, long stride, int count, int tid) {
            pitch = (unsigned)stride * sizeof(T);
            const int rows = min(count, ROWS);
            d = buf_rsrc(base, rows > 0 ? (rows - 1) * pitch + COLS * sizeof(T) : 0u);
            at = (tid / PER_ROW) * pitch + (tid % PER_ROW) * 16;
        }
    };
    __device__ __forceinline__ void load(const Source &s, int i) {
        r[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             s.d, (int)(s.at + i * STEP * s.pitch), 0, 0));
    }
    __device__ __forceinline__ void load(const T *base, long stride, int count, int tid) {
        const Source s(base, stride, count, tid);
#pragma unroll
        for (int i = 0; i < N; ++i)
            load(s, i);
    }
    template <int PITCH> __device__ __forceinline__ void store(T *lds, int tid) const {
        const int row = tid / PER_ROW, c = (tid % PER_ROW) * VEC;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<f32x4 *>(lds + lds_row(row + i * STEP) * PITCH + c) = r[i];
    }
};

// ---------------------------------------------------------------------------
// Join of the blocks along each sequence: block b's own contribution U_b in
// ws_state becomes the state at its start (REV: in ws_rstate, the reverse
// state behind its end, blocks last to first).  One thread holds 4 values of S
// of one (sequence, head); the blocks' values are loaded JOIN ahead (B2 H16, 16
// blocks of 128 x 128: 67 MB in 13 us).  A sequence of one block has nothing to
// join, one without tokens passes its state on.
// ---------------------------------------------------------------------------
constexpr int JOIN = 8, JOIN_NT = 256;

// Workgroups of a (sequence, head).  With many of these, of which most may have
// nothing to join, one takes all of the state (37 sequences of 32 heads, 128 x
// 64: 8 a state 9.9 us, one 8.0).
inline int join_pieces(const LinearParams &P) {
    return (long)P.N * P.H >= 1024 ? 1 : P.dk * P.dv / (4 * JOIN_NT);
}

// Values e .. e + 3 of a thread.
template <bool REV>
__device__ __forceinline__ void join_values(const LinearParams &P, int seq, int h, int e) {
    const long size = (long)P.dk * P.dv;
    long b0 = (long)seq * P.nblocks, b1 = b0 + P.nblocks, slot = seq;
    if (P.block_offsets) {
        b0 = P.block_offsets[seq];
        b1 = P.block_offsets[seq + 1];
        slot = P.slots ? P.slots[seq] : seq;
        if (b0 < 0 || b1 > P.nblocks || slot < 0 || slot >= P.pool)
            return;
    }
    const long nb = b1 - b0;
    if (nb == 1)
        return;
    const float *first = REV ? P.dS_out : P.S0;
    float *pass = REV ? P.dS0 : P.S_out;
    float *ws = REV ? P.ws_rstate : P.ws_state;
    const float *decay = REV ? P.ws_rdecay : P.ws_decay;
    const long at = (slot * P.H + h) * size + e;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (first)
        s = *reinterpret_cast<const f32x4 *>(first + at);
    if (nb <= 0) {
        if (pass && pass != first)
            *reinterpret_cast<f32x4 *>(pass + at) = s;
        return;
    }
    auto block = [&](long i) { return (REV ? b1 - 1 - i : b0 + i) * P.H + h; };
    for (long j = 0; j < nb; j += JOIN) {
        f32x4 u[JOIN];
        float a[JOIN];
#pragma unroll
        for (int i = 0; i < JOIN; ++i)
            if (j + i < nb - 1) {
                u[i] = *reinterpret_cast<const f32x4 *>(ws + block(j + i) * size + e);
                a[i] = decay[block(j + i)];
            }
#pragma unroll
        for (int i = 0; i < JOIN; ++i)
            if (j + i < nb) {
                *reinterpret_cast<f32x4 *>(ws + block(j + i) * size + e) = s;
                if (j + i < nb - 1)
                    s = s * a[i] + u[i];
            }
    }
}

template <bool REV>
__device__ __forceinline__ void join_blocks(const LinearParams &P, long id, int pieces) {
    const int piece = id % pieces;
    const int h = (id / pieces) % P.H;
    const int seq = id / ((long)pieces * P.H);
    if (P.block_offsets && P.block_offsets[seq + 1] - P.block_offsets[seq] == 1)
        return;
    for (int e = (piece * JOIN_NT + threadIdx.x) * 4; e < P.dk * P.dv; e += pieces * JOIN_NT * 4)
        join_values<REV>(P, seq, h, e);
}

// Order of a packed batch's blocks in time: the longest first, so that the
// workgroups that start last are short ones.  Worth it where there are more
// workgroups than run at once; with very many blocks the differences even out
// (and one workgroup sorts).  37 sequences of 700 tokens at the mean, bf16,
// the prefill: H32 of 128 x 64 in blocks of 1664 149 -> 140 us, H16 of 128 x 128
// in blocks of 832 205 -> 187 us.
constexpr int ORDER_BINS = 512, ORDER_MAX = 4096;
inline bool ordered(const LinearParams &P) {
    return P.ws_order && P.nblocks <= ORDER_MAX && (long)P.nblocks * P.H > 256;
}
// By one workgroup of JOIN_NT threads: a counting sort by length.  Which of two
// blocks of about the same length is first may change, results do not.
__device__ __forceinline__ void order_blocks(const LinearParams &P) {
    static_assert(ORDER_BINS == 2 * JOIN_NT, "two bins a thread");
    __shared__ int count[ORDER_BINS], wave[JOIN_NT / WAVE];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    count[tid] = count[tid + JOIN_NT] = 0;
    __syncthreads();
    // bin 0: the longest
    auto bin = [&](int b) {
        const int n = min(max(P.blocks[4l * b + 1], 0), P.block);
        return ORDER_BINS - 1 - (int)((long)n * (ORDER_BINS - 1) / P.block);
    };
    for (int b = tid; b < P.nblocks; b += JOIN_NT)
        atomicAdd(&count[bin(b)], 1);
    __syncthreads();
    const int x = count[2 * tid], y = count[2 * tid + 1];
    int sum = x + y;
    for (int off = 1; off < WAVE; off *= 2) {
        const int below = __shfl_up(sum, off, WAVE);
        sum += lane >= off ? below : 0;
    }
    if (lane == WAVE - 1)
        wave[tid / WAVE] = sum;
    __syncthreads();
    for (int i = 0; i < tid / WAVE; ++i)
        sum += wave[i];
    count[2 * tid] = sum - x - y;
    count[2 * tid + 1] = sum - y;
    __syncthreads();
    for (int b = tid; b < P.nblocks; b += JOIN_NT)
        P.ws_order[atomicAdd(&count[bin(b)], 1)] = b;
}
// The block of the i-th place.
__device__ __forceinline__ long block_at(const LinearParams &P, long i) {
    return P.ws_order ? __builtin_amdgcn_readfirstlane(P.ws_order[i]) : i;
}

}  // namespace lin
}  // namespace kdn
