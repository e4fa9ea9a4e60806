// kdn_linear_device.h -- device-side pieces shared by the linear-attention
// kernels: which tokens a workgroup owns, MFMA fragments, and the decays of a
// chunk.
#pragma once

#include "kdn_device.h"
#include "kdn_linear.h"

namespace kdn {
namespace lin {

typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

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
__device__ __forceinline__ Block get_block(const LinearParams &P, long b) {
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
    const int4 r = reinterpret_cast<const int4 *>(P.blocks)[b];
    if (r.z < 0 || r.z >= P.N || r.x < 0 || r.y <= 0 || r.y > P.block ||
        (long)r.x + r.y > P.tokens || r.w < 0)
        return B;
    const int b0 = P.block_offsets[r.z], b1 = P.block_offsets[r.z + 1];
    if (b0 < 0 || b1 > P.nblocks || (long)b0 + r.w != b || b1 <= b)
        return B;
    B.slot = P.slots ? P.slots[r.z] : r.z;
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

// ---------------------------------------------------------------------------
// Fragments: the 8 contraction elements of one lane for a step of 32.  For
// bfloat16 they are the operand of one v_mfma_f32_16x16x32_bf16; for float32
// element s of every lane is the operand of the s-th of eight
// v_mfma_f32_16x16x4_f32.  Lane l holds row (A) or column (B) l & 15; which
// 8 of the 32 contraction indices it holds only has to agree between A and B.
// ---------------------------------------------------------------------------
template <typename T> struct Frag;
template <> struct Frag<bf16> { typedef bf16x8 V; };
template <> struct Frag<float> { typedef f32x8 V; };
template <typename T> using FragV = typename Frag<T>::V;

__device__ __forceinline__ void mma(f32x4 &acc, bf16x8 a, bf16x8 b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x4 &acc, f32x8 a, f32x8 b) {
#pragma unroll
    for (int s = 0; s < 8; ++s)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], acc, 0, 0, 0);
}

// p: this lane's row at its 8 consecutive elements (contraction 8 g + e).
__device__ __forceinline__ bf16x8 frag_row(const bf16 *p) {
    return *reinterpret_cast<const bf16x8 *>(p);
}
__device__ __forceinline__ f32x8 frag_row(const float *p) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// p: this lane's row at 4 g; elements 4 g .. + 3 and 16 + 4 g .. + 3, the
// order of two accumulator tiles (frag_acc).
__device__ __forceinline__ bf16x8 frag_row_perm(const bf16 *p) {
    const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p);
    const bf16x4 b = *reinterpret_cast<const bf16x4 *>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x8 frag_row_perm(const float *p) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Two accumulator tiles (rows 16 t + 4 g + r and 16 (t + 1) + 4 g + r) as the
// fragment whose contraction runs over their 32 rows.
template <typename T> __device__ __forceinline__ FragV<T> frag_acc(f32x4 a, f32x4 b) {
    FragV<T> f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[e] = from_f32<T>(a[e]);
        f[4 + e] = from_f32<T>(b[e]);
    }
    return f;
}

// Transposed read of a tile [token][column]: tokens 8 g + e of the 32 behind
// `m`, at the 16 columns c(n) = c0 + cs * (n / 4) + n % 4 of lane n = l & 15.
// bfloat16: ds_read_b64_tr_b16 gives lane n of a group of 16 column n of the
// 4 rows x 16 columns whose 8-byte pieces the lanes point to (lane i: row
// i / 4, columns 4 (i % 4) .. + 3).
template <int PITCH>
__device__ __forceinline__ bf16x8 frag_cols(const bf16 *m, int c0, int cs, int lane) {
    const int g = lane >> 4, i = lane & 15;
    const bf16 *p = m + (8 * g + i / 4) * PITCH + c0 + cs * (i & 3);
    union { s16x4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * PITCH));
    return u.v;
}
template <int PITCH>
__device__ __forceinline__ f32x8 frag_cols(const float *m, int c0, int cs, int lane) {
    const int g = lane >> 4, n = lane & 15;
    const float *p = m + 8 * g * PITCH + c0 + cs * (n >> 2) + (n & 3);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = p[e * PITCH];
    return f;
}

// As frag_cols, rows 4 g .. + 3 and 16 + 4 g .. + 3 (the order of frag_acc).
template <int PITCH>
__device__ __forceinline__ bf16x8 frag_cols_perm(const bf16 *m, int c0, int cs, int lane) {
    const int g = lane >> 4, i = lane & 15;
    const bf16 *p = m + (4 * g + i / 4) * PITCH + c0 + cs * (i & 3);
    union { s16x4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * PITCH));
    return u.v;
}
template <int PITCH>
__device__ __forceinline__ f32x8 frag_cols_perm(const float *m, int c0, int cs, int lane) {
    const int g = lane >> 4, n = lane & 15;
    const float *p = m + 4 * g * PITCH + c0 + cs * (n >> 2) + (n & 3);
    f32x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = p[(e + (e & 4 ? 12 : 0)) * PITCH];
    return f;
}

// x (.) w as an operand that keeps 32-bit products: bfloat16 as the sum of two
// operands (16 significant bits; a single one would leave 2^-9 in a float32
// state), float32 as one.
template <typename T> struct Split;
template <> struct Split<bf16> {
    bf16x8 hi, lo;
    __device__ __forceinline__ Split(bf16x8 x, const float (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = to_f32(x[e]) * w[e];
            hi[e] = static_cast<bf16>(y);
            lo[e] = static_cast<bf16>(y - static_cast<float>(hi[e]));
        }
    }
    __device__ __forceinline__ void mma_a(f32x4 &acc, bf16x8 a) const {
        mma(acc, a, lo);
        mma(acc, a, hi);
    }
};
template <> struct Split<float> {
    f32x8 f;
    __device__ __forceinline__ Split(f32x8 x, const float (&w)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = x[e] * w[e];
    }
    __device__ __forceinline__ void mma_a(f32x4 &acc, f32x8 a) const { mma(acc, a, f); }
};

// ---------------------------------------------------------------------------
// Decays of a chunk, all in powers of two.  Prefix sums of the log-decays run
// in 64 bits: a difference of two of them must keep its own bits also behind
// strong decays.  A log-decay below -152 (base 2) counts as -152, whose power
// is 0 in float32 as that of -infinity is, so that a reset costs no NaN.
// ---------------------------------------------------------------------------
template <int C> struct Decays {
    float hi[C], lo[C];   // prefix sum G_i in two floats
    float in[C];          // 2^G_i: from the chunk's start through token i
    float out[C];         // 2^(G_C - G_j): behind token j to the chunk's end
    float all;            // 2^G_C
};

constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESET2 = -152.f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ double log2_decay(float la) {
    const float g = la * LOG2E;
    // NaN stays NaN: no fmax
    return g < RESET2 ? (double)RESET2 : (double)la * 1.4426950408889634074;
}

// One wave: lane j < C holds the log-decay (natural) of token j, 0 behind the
// end.  Returns the base-2 prefix sum of the chunk.
template <int C>
__device__ __forceinline__ double chunk_decays(Decays<C> &D, float la, int lane) {
    double x = log2_decay(la);
#pragma unroll
    for (int off = 1; off < C; off <<= 1) {
        const double y = __shfl_up(x, off, WAVE);
        if (lane >= off)
            x += y;
    }
    const double all = __shfl(x, C - 1, WAVE);
    if (lane < C) {
        const float hi = (float)x;
        D.hi[lane] = hi;
        D.lo[lane] = (float)(x - (double)hi);
        D.in[lane] = exp2_fast((float)x);
        D.out[lane] = exp2_fast((float)(all - x));
        if (lane == 0)
            D.all = exp2_fast((float)all);
    }
    return all;
}

// 2^(G_i - G_j)
template <typename T, int C>
__device__ __forceinline__ float decay_between(const Decays<C> &D, float hi_i, float lo_i, int j) {
    float x = hi_i - D.hi[j];
    // bfloat16 products: the low parts (2^-24 of a prefix sum) are far below
    // their rounding
    if (sizeof(T) == 4)
        x += lo_i - D.lo[j];
    return exp2_fast(x);
}

// log-decay of token row `row`, head h
template <typename T>
__device__ __forceinline__ float load_gate(const LinearParams &P, long row, int h) {
    if (P.gate == KDN_GATE_HEAD)
        return static_cast<const float *>(P.la)[h];
    return to_f32(static_cast<const T *>(P.la)[row * P.H + h]);
}

// ---------------------------------------------------------------------------
// A tile [ROWS][COLS] from global memory, held in registers between its load
// and its store to LDS (NT threads, 16-byte pieces); rows behind `count` are
// zero and not read.
// ---------------------------------------------------------------------------
template <typename T, int ROWS, int COLS, int NT> struct TileRegs {
    static constexpr int VEC = 16 / sizeof(T);
    static constexpr int PER_ROW = COLS / VEC;
    static constexpr int STEP = NT / PER_ROW;          // rows of one pass
    static constexpr int N = ROWS / STEP;
    static_assert(NT % PER_ROW == 0 && ROWS % STEP == 0, "tile shape");
    uint4 r[N];

    // base: the tile's first row (element pointer), stride in elements
    __device__ __forceinline__ void load(const T *base, long stride, int count, int tid) {
        const int row = tid / PER_ROW, c = (tid % PER_ROW) * VEC;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int rr = row + i * STEP;
            r[i] = make_uint4(0, 0, 0, 0);
            if (rr < count)
                r[i] = *reinterpret_cast<const uint4 *>(base + rr * stride + c);
        }
    }
    template <int PITCH> __device__ __forceinline__ void store(T *lds, int tid) const {
        const int row = tid / PER_ROW, c = (tid % PER_ROW) * VEC;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<uint4 *>(lds + (row + i * STEP) * PITCH + c) = r[i];
    }
};

}  // namespace lin
}  // namespace kdn
