// kdn_linear.hip -- chunked linear attention with a decay for each head
// (gfx950): o_t = S_t^T q_t, S_t = e^{g_t} S_{t-1} + k_t v_t^T.
//
// Within a chunk of C tokens, with G_i the prefix sum of g and S the state at
// the chunk's start,
//   o_i = e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j,
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T.
// A workgroup walks the chunks of one block (consecutive tokens of a sequence)
// for one head.  A sequence of one block is one pass.  Longer sequences are
// cut so that few heads still fill the chip: every block but the last first
// sums its own contribution from a zero state (k and v only), a join carries
// the states along the sequence, and the walk then starts every block from its
// own state.  The cut costs one more read of k and v.
//
// Four waves work on 32 x 32 tiles.  With d_v = 128 wave w keeps 32 columns of
// S in MFMA accumulators (float32) for the whole block; all products are
// computed transposed (o^T = S^T q^T + v^T P^T), so that the accumulators of S
// are the A operand of S^T q^T as they are.  With d_v = 64 two waves share 32
// columns: each keeps half of the rows of S and computes half of the tokens
// of o, and S passes between them through LDS in the operand type.  P = D (.)
// q k^T is computed once, a tile per wave, and shared through LDS.  q, k and v
// of the next chunk are in flight (in registers) while one is worked on, and
// two workgroups share a CU.
//
// Tiles are 32 x 32 because the operands come from LDS: 16 x 16 tiles read
// every operand twice as often for the same products.
//
// Measured (bf16, 128 x 128): B2 H16 T16384 in blocks of 1024, constant decays,
// 207 us a call (own states 68-88 us, join 12, outputs 120-153: the clock falls
// in long runs).  It moves 924 MB where 539 are needed (k and v twice, and the
// blocks' states), at 4.4 TB/s, 91 % of the rate of a large copy.  In the outputs
// LDS is busy for 23 % of the time, VALU 32, MFMA 29, and 29 % is waiting.  B1
// H16 T190 takes 13.7 us, three chunks one after the other.
#include "kdn_linear_device.h"

namespace kdn {
namespace lin {

// OWN: a block's own contribution to the state; ROWN: to the state of the
// reverse recurrence R <- e^{G_C} R + sum_i e^{G_i} q_i do_i^T, chunks last to
// first (q and do in the places of k and v); OUT: outputs; CHUNKS: the state
// at every chunk's start, transposed (k and v change places, so that a lane
// holds runs of d_v and stores whole fragments).
enum Mode { OWN = 0, OUT = 1, CHUNKS = 2, ROWN = 3 };

constexpr int NT = 256;

// NH heads of DV / NH columns share a workgroup.
template <typename T, int DK, int DV, int NH = 1> struct Shape {
    static constexpr int HD = DV / NH;         // d_v
    static constexpr int C = linear_chunk(sizeof(T) == 2);
    static constexpr int PK = lds_pitch<T>(DK), PV = lds_pitch<T>(DV), PP = lds_pitch<T>(C);
    static constexpr int NCT = DV / 32;        // column tiles
    static constexpr int TW = NT / WAVE / NCT; // waves that share a column tile
    static constexpr int TK = DK / 32 / TW;    // row tiles of S in a wave
    static constexpr int IT = C / 32;          // token tiles
    static constexpr int OT = (IT + TW - 1) / TW;   // token tiles of o in a wave
    static constexpr int KS = C / 16;          // contraction steps over tokens

    template <int MODE> struct Lds {
        static constexpr bool SHARED = MODE == OUT && TW > 1;    // S passes through LDS
        __attribute__((aligned(16))) T Ks[C * PK];
        __attribute__((aligned(16))) T Vs[C * PV];
        __attribute__((aligned(16))) T Qs[MODE == OUT ? C * PK : 1];
        __attribute__((aligned(16))) T Ps[NH][MODE == OUT ? C * PP : 1];
        __attribute__((aligned(16))) T Ss[SHARED ? DV * PK : 1];
        Decays<C> D[2][NH];
    };
};

// The part of the state of one wave: row tiles t TK .. + TK - 1 of column tile
// ct (t = w / NCT, ct = w % NCT), rows and columns in the order of chan(): a lane
// has one column and of each 32 rows twice 8 neighbours.
template <typename T, int DK, int DV, int NH> struct StateAcc {
    using SH = Shape<T, DK, DV, NH>;
    f32x16 t[SH::TK];
    int row0, col;                             // of this lane

    __device__ __forceinline__ StateAcc(int w, int lane) {
        row0 = w / SH::NCT * SH::TK * 32 + 8 * (lane >> 5);
        col = w % SH::NCT * 32 + chan(lane & 31);
    }
    __device__ __forceinline__ int row(int i, int r) const {
        return row0 + 32 * i + 16 * (r / 8) + r % 8;
    }
    // element (row, col) of the heads' matrices [NH][DK][HD]
    __device__ __forceinline__ int at(int i, int r) const {
        return col / SH::HD * (DK * SH::HD) + row(i, r) * SH::HD + col % SH::HD;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
            t[i] = zero16();
    }
    __device__ __forceinline__ void load(const float *S) {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                t[i][r] = S[at(i, r)];
    }
    // from the transposed matrix [DV][DK]
    __device__ __forceinline__ void load_t(const float *S) {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(S + col * DK + row(i, 4 * j));
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    t[i][4 * j + r] = x[r];
            }
    }
    __device__ __forceinline__ void store(float *S) const {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                S[at(i, r)] = t[i][r];
    }
    // operand fragments [column tile][16 rows][lane], rounded to T: the
    // products that read them round the same state in the prefill.  `rest`: what
    // the rounding leaves, where wanted.
    __device__ __forceinline__ void store_frags(T *S, T *rest, int w, int lane) const {
        const int first = (w % SH::NCT * (DK / 32) + w / SH::NCT * SH::TK) * 2;
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                reinterpret_cast<FragV<T> *>(S)[(first + 2 * i + b) * WAVE + lane] =
                    frag_acc<T>(t[i], b);
        if (sizeof(T) == 2 && rest) {
#pragma unroll
            for (int i = 0; i < SH::TK; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    reinterpret_cast<FragV<T> *>(rest)[(first + 2 * i + b) * WAVE + lane] =
                        frag_rest<T>(t[i], b);
        }
    }
    // to LDS, transposed [DV][pitch], in the operand type
    __device__ __forceinline__ void share(T *Ss, int pitch) const {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    f[r] = t[i][8 * j + r];
                lds_st8(Ss + col * pitch + row(i, 8 * j), f);
            }
    }
};

// PARTS: of the split operands in the update of S (Split).
template <typename T, int DK, int DV, int NH, int MODE, int PARTS>
__device__ __forceinline__ void linear_walk(
    const LinearParams &P, const Block &B, long b, int h,
    typename Shape<T, DK, DV, NH>::template Lds<MODE> &L) {
    using SH = Shape<T, DK, DV, NH>;
    constexpr int C = SH::C, TK = SH::TK, KS = SH::KS, IT = SH::IT, OT = SH::OT, TW = SH::TW;
    constexpr int NCT = SH::NCT, PK = SH::PK, PV = SH::PV, PP = SH::PP;
    constexpr bool SHARED = SH::template Lds<MODE>::SHARED;

    T *const Ks = L.Ks, *const Vs = L.Vs, *const Qs = L.Qs, *const Ss = L.Ss;
    auto &D = L.D;
    constexpr int HD = SH::HD;

    const int tid = threadIdx.x, lane = tid & (WAVE - 1), w = wave_id();
    const int hf = lane >> 5, n = lane & 31, cn = chan(n);
    const int rn = lds_row(n), rcn = lds_row(cn);   // their places in a tile
    const int ct = w % NCT, tw = w / NCT;
    const int eh = ct / (NCT / NH);     // head of this wave's columns
    T *const Ps = L.Ps[eh];
    constexpr int HK = MODE == CHUNKS ? DV : DK, HV = MODE == CHUNKS ? DK : HD;
    const T *q = static_cast<const T *>(P.q) + B.first * P.q_stride + (h / (P.H / P.Hq)) * HK;
    const T *k = static_cast<const T *>(P.k) + B.first * P.k_stride + (h / (P.H / P.Hk)) * HK;
    const T *v = static_cast<const T *>(P.v) + B.first * P.v_stride + (h / (P.H / P.Hv)) * HV;
    long ks = P.k_stride, vs = P.v_stride;
    if (MODE == CHUNKS) {
        const T *x = k;
        k = v;
        v = x;
        ks = P.v_stride;
        vs = P.k_stride;
    }
    if (MODE == ROWN) {
        k = q;
        ks = P.q_stride;
        vs = P.o_stride;
        v = static_cast<const T *>(P.d_o) + B.first * vs + h * HD;
    }

    TileRegs<T, C, DK, NT> qr, kr;
    TileRegs<T, C, DV, NT> vr;
    const int nchunk = (B.count + C - 1) / C;
    // the wave that sums the decays: not one of those with a tile of P
    constexpr int GW = NT / WAVE - 1;
    float head[NH];
    GateReg<T> la[NH];              // this lane's token of the next chunk
    auto gate = [&](int c) {
#pragma unroll
        for (int e = 0; e < NH; ++e)
            la[e].template load<C>(P, B.first + (long)c * C, B.count - c * C, h + e, lane);
    };
    double total[NH];               // base-2 log of the block's decay (wave GW)
    auto decays = [&](int c, int buffer) {
#pragma unroll
        for (int e = 0; e < NH; ++e)
            total[e] += chunk_decays<C>(
                D[buffer][e], la[e].value(P, head[e], lane < C && c * C + lane < B.count), lane);
    };
#pragma unroll
    for (int e = 0; e < NH; ++e) {
        head[e] = P.gate == KDN_GATE_HEAD ? static_cast<const float *>(P.la)[h + e] : 0.f;
        total[e] = 0.;
    }
    typedef TileRegs<T, C, DK, NT> KT;
    typedef TileRegs<T, C, DV, NT> VT;
    // part i of n of chunk c's loads of k and v, and its loads of q (a chunk
    // behind the last: nothing is read)
    auto tokens_of = [&](int c) { return c < nchunk && c >= 0 ? B.count - c * C : 0; };
    auto load_kv = [&](int c, int i, int n) {
        const typename KT::Source sk(k + (long)c * C * ks, ks, tokens_of(c), tid);
        const typename VT::Source sv(v + (long)c * C * vs, vs, tokens_of(c), tid);
        constexpr int ALL = KT::N + VT::N;
#pragma unroll
        for (int j = i * ALL / n; j < (i + 1) * ALL / n; ++j) {
            if (j < KT::N)
                kr.load(sk, j);
            else
                vr.load(sv, j - KT::N);
        }
    };
    auto load_q = [&](int c) {
        if (MODE == OUT)
            qr.load(q + (long)c * C * P.q_stride, P.q_stride, tokens_of(c), tid);
    };
    // the chunk of step i
    auto chunk = [&](int i) { return MODE == ROWN ? nchunk - 1 - i : i; };
    if (w == GW)
        gate(chunk(0));
    load_kv(chunk(0), 0, 1);
    load_q(chunk(0));

    StateAcc<T, DK, DV, NH> S(w, lane);
    const long sidx = (b * P.H + h) * (long)(DK * HD);
    const float *start = B.single ? P.S0 : P.ws_state;
    if (start)
        start += B.single ? (B.slot * P.H + h) * (long)(DK * HD) : sidx;
    if (MODE == OWN || MODE == ROWN || !start)
        S.zero();
    else if (MODE == CHUNKS)
        S.load_t(start);
    else
        S.load(start);

    if (w == GW) {
        decays(chunk(0), 0);
        if (nchunk > 1)
            gate(chunk(1));
    }
    if (SHARED)
        S.share(Ss, PK);

    for (int step = 0; step < nchunk; ++step) {
        const int c = chunk(step);
        const Decays<C> &dc = D[step & 1][eh];
        const int cnt = B.count - c * C;       // tokens from here on
        kr.template store<PK>(Ks, tid);
        vr.template store<PV>(Vs, tid);
        if (MODE == OUT)
            qr.template store<PK>(Qs, tid);
        __syncthreads();
        if (MODE != OUT)                // OUT: later, its registers are taken here
            load_kv(chunk(step + 1), 0, 1);

        if (MODE == CHUNKS) {
            const long at = (chunk_slot(b, B.first, c, C) * P.H + h) * (long)(DK * HD);
            T *const rest = static_cast<T *>(P.ws_chunk_lo);
            S.store_frags(static_cast<T *>(P.ws_chunk) + at, rest ? rest + at : nullptr, w, lane);
        }

        if (MODE == OUT && w < IT * (IT + 1) / 2) {
            // tiles of P^T on and below the diagonal: lane n has query
            // i = 32 it + n, registers 0-7 and 8-15 eight keys each
            const int it = w > 0, jt = w > 1;
            const int i = 32 * it + n;
            f32x16 p = zero16();
            float d[NH][2][8];
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Decays<C> &de = D[step & 1][e];
                    decay_between<T>(de, de.hi[i], de.lo[i], i, 32 * jt + 16 * u + 8 * hf, d[e][u]);
                }
            mma_rows<T, DK, 8>(p, Ks + (32 * jt + rcn) * PK + 8 * hf,
                               Qs + (32 * it + rn) * PK + 8 * hf);
#pragma unroll
            for (int e = 0; e < NH; ++e)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // rounded to the operand type: P feeds one product whose
                    // result is rounded to the same type
                    float x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        x[r] = p[8 * u + r] * d[e][u][r];
                    lds_st8(L.Ps[e] + i * PP + 32 * jt + 16 * u + 8 * hf, x);
                }
        }

        // operands of the state's update, S <- all S + k^T (out (.) v)
        const float all = dc.all();
        const float *weight = MODE == ROWN ? dc.in : dc.out;
        auto rows = [&](int s, int i) {
            return frag_cols<PK, true>(Ks + 16 * s * PK + 32 * (tw * TK + i), lane);
        };
        FragV<T> vf[KS], kf[TK];
        Split<T, PARTS> split;
        constexpr int STEPS = 4 * Split<T, PARTS>::PARTS;
        float wt[8];
        lds_ld8(weight + 8 * hf, wt);
#pragma unroll
        for (int s = 0; s < KS; ++s)
            vf[s] = frag_cols<PV, true>(Vs + 16 * s * PV + 32 * ct, lane);
        f32x16 o[OT];
        if constexpr (MODE == OUT) {
            // o^T = S^T q^T, scaled to each token.  Between the MFMAs: the
            // operands of the steps that follow, the state's decay and the first
            // operands of its update
            constexpr int NS = DK / 16, U = NS * OT;
            auto read_q = [&](int s, int t) {
                const int i = 32 * (t * TW + (IT >= TW ? tw : 0)) + rn;
                return frag_row(Qs + i * PK + 16 * s + 8 * hf);
            };
            auto read_s = [&](int s) {
                if constexpr (SHARED)
                    return frag_row(Ss + (32 * ct + cn) * PK + 16 * s + 8 * hf);
                else
                    return frag_acc<T>(S.t[s / 2], s % 2);
            };
            FragV<T> qf[2][OT], sf[2];
#pragma unroll
            for (int t = 0; t < OT; ++t) {
                o[t] = zero16();
                qf[0][t] = read_q(0, t);
                qf[1][t] = read_q(1, t);
            }
            sf[0] = read_s(0);
            if (SHARED)
                sf[1] = read_s(1);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    const int u = s * OT + t;
                    mma(o[t], sf[s & 1], qf[s & 1][t]);
                    if (s + 2 < NS)
                        qf[s & 1][t] = read_q(s + 2, t);
                    if (!SHARED && t == 0 && s + 1 < NS)
                        sf[(s + 1) & 1] = read_s(s + 1);
                    if (SHARED) {       // the state's registers are not read here
#pragma unroll
                        for (int e = u * 16 * TK / U; e < (u + 1) * 16 * TK / U; ++e)
                            S.t[e / 16][e % 16] *= all;
                    } else if (s % 2) { // tile s / 2 has been read
#pragma unroll
                        for (int e = t * 16 / OT; e < (t + 1) * 16 / OT; ++e)
                            S.t[s / 2][e] *= all;
                    }
#pragma unroll
                    for (int i = u * STEPS / U; i < (u + 1) * STEPS / U; ++i)
                        split.step(i, vf[0], wt);
#pragma unroll
                    for (int i = 0; i < TK; ++i)
                        if (u == U - TK + i || (U < TK && u == 0))
                            kf[i] = rows(0, i);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (SHARED && s + 2 < NS)
                    sf[s & 1] = read_s(s + 2);
            }
#pragma unroll
            for (int t = 0; t < OT; ++t)
                o[t] *= dc.in[32 * (t * TW + (IT >= TW ? tw : 0)) + n];
        } else {
#pragma unroll
            for (int i = 0; i < TK; ++i) {
                kf[i] = rows(0, i);
                S.t[i] *= all;
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                split.step(i, vf[0], wt);
        }
        update_state<T, PARTS>(S.t, vf, weight, hf, split, kf, rows, [&](int u, int U) {
            if (MODE == OUT && u < U / 2)
                load_kv(chunk(step + 1), u, U / 2);
        });
        if (w == GW) {              // the next chunk's decays
            if (step + 1 < nchunk)
                decays(chunk(step + 1), (step + 1) & 1);
            if (step + 2 < nchunk)
                gate(chunk(step + 2));
        }
        // P is whole, and q, k and v have been read: what follows reads P and
        // registers only, and the next chunk's tiles may be stored
        __syncthreads();

        if (MODE == OUT) {
            load_q(chunk(step + 1));
            // o^T += v^T P^T (right of the diagonal Ps holds nothing)
            FragV<T> pf[OT][KS];
#pragma unroll
            for (int t = 0; t < OT; ++t) {
                const int it = t * TW + (IT >= TW ? tw : 0);
#pragma unroll
                for (int s = 0; s < KS; ++s)
                    if (s / 2 <= (TW > 1 ? IT : t))
                        pf[t][s] = frag_row(Ps + (32 * it + n) * PP + 16 * s + 8 * hf);
            }
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int t = 0; t < OT; ++t)
                    if (s / 2 <= t * TW + (IT >= TW ? tw : 0))
                        mma(o[t], vf[s], pf[t][s]);
#pragma unroll
            for (int t = 0; t < OT; ++t) {
                const int it = t * TW + tw, i = 32 * it + n;
                if (it < IT && i < cnt) {
                    T *dst = static_cast<T *>(P.o) + ((B.first + (long)c * C) * P.H + h) * HD +
                             (unsigned)i * (unsigned)(P.H * HD) + (unsigned)(32 * ct + 8 * hf);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            x[r] = o[t][8 * u + r];
                        lds_st8(dst + 16 * u, x);
                    }
                }
            }
        }
        if (SHARED)
            S.share(Ss, PK);
    }
    if (MODE == OWN || MODE == ROWN) {
        S.store((MODE == OWN ? P.ws_state : P.ws_rstate) + sidx);
        if (w == GW && lane == 0) {
#pragma unroll
            for (int e = 0; e < NH; ++e)
                (MODE == OWN ? P.ws_decay : P.ws_rdecay)[b * P.H + h + e] =
                    exp2_fast((float)total[e]);
        }
    }
    if (MODE == OUT && B.last && P.S_out)
        S.store(P.S_out + (B.slot * P.H + h) * (long)(DK * HD));
}

// One block and NH heads of a mode.  Three parts for a state that is returned
// and for what goes into one: the last block's in the prefill and the blocks'
// own (the forward ones of the gradient call excepted, which are only read
// rounded).
template <typename T, int DK, int DV, int NH, int MODE, bool GRAD>
__device__ __forceinline__ void linear_block_heads(
    const LinearParams &P, long id, typename Shape<T, DK, DV, NH>::template Lds<MODE> &L) {
    const int groups = P.H / NH;
    // the order is made with the joins, which the blocks' own states precede
    const long b = MODE == OUT || MODE == CHUNKS ? block_at(P, id / groups) : id / groups;
    const int h = id % groups * NH;
    const Block B = get_block(P, b);
    if (B.count == 0 || B.slot < 0 || (MODE == OWN && B.last) || (MODE == ROWN && B.index == 0))
        return;
    if (MODE == OUT ? B.last : MODE == ROWN || (MODE == OWN && !GRAD))
        linear_walk<T, DK, DV, NH, MODE, 3>(P, B, b, h, L);
    else if (MODE == OUT || MODE == CHUNKS || GRAD)
        linear_walk<T, DK, DV, NH, MODE, 2>(P, B, b, h, L);
}

template <typename T, int DK, int DV, int NH, int MODE>
__global__ __launch_bounds__(NT, 2) void linear_kernel(LinearParams P) {
    __shared__ typename Shape<T, DK, DV, NH>::template Lds<MODE> L;
    static_assert(sizeof(L) <= 80 * 1024, "two workgroups share a CU");
    linear_block_heads<T, DK, DV, NH, MODE, false>(P, blockIdx.x, L);
}

// The blocks' own contributions to both recurrences of the gradient call, in
// one launch: forward ones in the even workgroups, reverse ones in the odd.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(NT, 2) void linear_own_kernel(LinearParams P) {
    __shared__ union U {
        typename Shape<T, DK, DV>::template Lds<OWN> f;
        typename Shape<T, DK, DV>::template Lds<ROWN> r;
    } L;
    if (blockIdx.x & 1)
        linear_block_heads<T, DK, DV, 1, ROWN, true>(P, blockIdx.x >> 1, L.r);
    else
        linear_block_heads<T, DK, DV, 1, OWN, true>(P, blockIdx.x >> 1, L.f);
}

__global__ __launch_bounds__(JOIN_NT) void linear_join_kernel(LinearParams P, int pieces) {
    if (blockIdx.x == (unsigned long)P.N * P.H * pieces)
        order_blocks(P);
    else
        join_blocks<false>(P, blockIdx.x, pieces);
}

#define KDN_LINEAR_SIZES(rows, cols, CASE)         \
    if (rows == 64 && cols == 64) { CASE(64, 64) } \
    if (rows == 64 && cols == 128) { CASE(64, 128) } \
    if (rows == 128 && cols == 64) { CASE(128, 64) } \
    if (rows == 128 && cols == 128) { CASE(128, 128) }

template <typename T, int MODE>
static hipError_t launch_mode(const LinearParams &P, hipStream_t st) {
    const dim3 grid((unsigned)(linear_total_blocks(P) * P.H)), block(NT);
    // rows and columns of the state the mode works on
    const int rows = MODE == CHUNKS ? P.dv : P.dk, cols = MODE == CHUNKS ? P.dk : P.dv;
#define KDN_CASE(DK_, DV_)                                                         \
    hipLaunchKernelGGL((linear_kernel<T, DK_, DV_, 1, MODE>), grid, block, 0, st, P); \
    return hipGetLastError();
    KDN_LINEAR_SIZES(rows, cols, KDN_CASE)
#undef KDN_CASE
    return hipErrorInvalidValue;
}

template <typename T, int MODE>
static hipError_t launch_prefill_mode(const LinearParams &P, hipStream_t st) {
    if (!linear_pairs(P))
        return launch_mode<T, MODE>(P, st);
    const dim3 grid((unsigned)(linear_total_blocks(P) * (P.H / 2))), block(NT);
    if (P.dk == 64)
        hipLaunchKernelGGL((linear_kernel<T, 64, 128, 2, MODE>), grid, block, 0, st, P);
    else
        hipLaunchKernelGGL((linear_kernel<T, 128, 128, 2, MODE>), grid, block, 0, st, P);
    return hipGetLastError();
}

template <typename T> static hipError_t launch_own(const LinearParams &P, hipStream_t st) {
    const dim3 grid((unsigned)(linear_total_blocks(P) * P.H * 2)), block(NT);
#define KDN_CASE(DK_, DV_)                                                       \
    hipLaunchKernelGGL((linear_own_kernel<T, DK_, DV_>), grid, block, 0, st, P); \
    return hipGetLastError();
    KDN_LINEAR_SIZES(P.dk, P.dv, KDN_CASE)
#undef KDN_CASE
    return hipErrorInvalidValue;
}

}  // namespace lin

hipError_t launch_linear_own(const LinearParams &P, hipStream_t st) {
    return P.bf16 ? lin::launch_own<bf16>(P, st) : lin::launch_own<float>(P, st);
}

hipError_t launch_linear_chunk_states(const LinearParams &P, hipStream_t st) {
    return P.bf16 ? lin::launch_mode<bf16, lin::CHUNKS>(P, st)
                  : lin::launch_mode<float, lin::CHUNKS>(P, st);
}

hipError_t launch_linear_prefill(const LinearParams &call, hipStream_t st) {
    LinearParams P = call;
    if (P.N == 0 || P.H == 0)
        return hipSuccess;
    const bool any = linear_total_blocks(P) > 0, sort = lin::ordered(P);
    if (!sort)
        P.ws_order = nullptr;
    hipError_t e = hipSuccess;
    if (P.block_offsets || P.nblocks != 1) {
        // the blocks' own contributions and their join, where a sequence may
        // have more than one; the join also passes on the states of empty ones
        if (any)
            e = P.bf16 ? lin::launch_prefill_mode<bf16, lin::OWN>(P, st)
                       : lin::launch_prefill_mode<float, lin::OWN>(P, st);
        if (e == hipSuccess) {
            const int pieces = lin::join_pieces(P);
            hipLaunchKernelGGL(lin::linear_join_kernel, dim3((unsigned)((long)P.N * P.H * pieces + sort)),
                               dim3(lin::JOIN_NT), 0, st, P, pieces);
            e = hipGetLastError();
        }
    }
    if (e != hipSuccess || !any)
        return e;
    return P.bf16 ? lin::launch_prefill_mode<bf16, lin::OUT>(P, st)
                  : lin::launch_prefill_mode<float, lin::OUT>(P, st);
}

}  // namespace kdn
