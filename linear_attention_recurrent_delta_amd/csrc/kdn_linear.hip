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
// Four waves split the d_v columns; wave w keeps its columns of S in MFMA
// accumulators (float32) for the whole block.  All products are computed
// transposed (o^T = S^T q^T + v^T P^T), so that the accumulator tiles of S
// are the A operand of S^T q^T as they are and a lane ends with 8 consecutive
// values of o.  P = D (.) q k^T is computed once, one 16-row strip per wave,
// and shared through LDS.  q, k and v of the next chunk are in flight while
// one is worked on.
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

template <typename T, int DK, int DV> struct Shape {
    static constexpr int C = linear_chunk(sizeof(T) == 2);
    static constexpr int PAD = 16 / sizeof(T);
    static constexpr int PK = DK + PAD, PV = DV + PAD, PP = C + PAD;   // LDS pitches
    static constexpr int NC = DV / 64;         // 16-column tiles of a wave
    static constexpr int TK = DK / 16;         // 16-row tiles of S
    static constexpr int KS = C / 32;          // contraction steps over tokens
    static constexpr int IT = C / 16;          // 16-token tiles
};

template <typename T, int DK, int DV>
struct StateAcc {
    using SH = Shape<T, DK, DV>;
    f32x4 t[SH::TK][SH::NC];

    // column of accumulator column n of tile c in wave w
    __device__ __forceinline__ static int col(int w, int c, int n) {
        return w * 16 * SH::NC + 4 * SH::NC * (n >> 2) + 4 * c + (n & 3);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int c = 0; c < SH::NC; ++c)
                t[i][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void load(const float *S, int w, int lane) {
        const int g = lane >> 4, n = lane & 15;
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int c = 0; c < SH::NC; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    t[i][c][r] = S[(16 * i + 4 * g + r) * DV + col(w, c, n)];
    }
    // from the transposed matrix [DV][DK]
    __device__ __forceinline__ void load_t(const float *S, int w, int lane) {
        const int g = lane >> 4, n = lane & 15;
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int c = 0; c < SH::NC; ++c)
                t[i][c] = *reinterpret_cast<const f32x4 *>(S + col(w, c, n) * DK + 16 * i + 4 * g);
    }
    __device__ __forceinline__ void store(float *S, int w, int lane) const {
        const int g = lane >> 4, n = lane & 15;
#pragma unroll
        for (int i = 0; i < SH::TK; ++i)
#pragma unroll
            for (int c = 0; c < SH::NC; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S[(16 * i + 4 * g + r) * DV + col(w, c, n)] = t[i][c][r];
    }
    // operand fragments [column tile][32 rows][lane], rounded to T: the
    // products that read them round the same state in the prefill
    __device__ __forceinline__ void store_frags(T *S, int w, int lane) const {
#pragma unroll
        for (int c = 0; c < SH::NC; ++c)
#pragma unroll
            for (int s = 0; s < DK / 32; ++s)
                reinterpret_cast<FragV<T> *>(S)[((w * SH::NC + c) * (DK / 32) + s) * WAVE + lane] =
                    frag_acc<T>(t[2 * s][c], t[2 * s + 1][c]);
    }
};

template <typename T, int DK, int DV, int MODE>
__global__ __launch_bounds__(NT, 2) void linear_kernel(LinearParams P) {
    using SH = Shape<T, DK, DV>;
    constexpr int C = SH::C, NC = SH::NC, TK = SH::TK, KS = SH::KS, IT = SH::IT;
    constexpr int PK = SH::PK, PV = SH::PV, PP = SH::PP;

    __shared__ __attribute__((aligned(16))) T Ks[C * PK];
    __shared__ __attribute__((aligned(16))) T Vs[C * PV];
    __shared__ __attribute__((aligned(16))) T Qs[MODE == OUT ? C * PK : 1];
    __shared__ __attribute__((aligned(16))) T Ps[MODE == OUT ? C * PP : 1];
    __shared__ __attribute__((aligned(16))) Decays<C> D[2];

    const int tid = threadIdx.x, lane = tid & (WAVE - 1), w = tid / WAVE;
    const int g = lane >> 4, n = lane & 15;
    const long b = blockIdx.x / P.H;
    const int h = blockIdx.x % P.H;
    const Block B = get_block(P, b);
    if (B.count == 0 || B.slot < 0 || (MODE == OWN && B.last) || (MODE == ROWN && B.index == 0))
        return;

    constexpr int HK = MODE == CHUNKS ? DV : DK, HV = MODE == CHUNKS ? DK : DV;
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
        vs = (long)P.H * DV;
        v = static_cast<const T *>(P.d_o) + B.first * vs + h * DV;
    }

    TileRegs<T, C, DK, NT> qr, kr;
    TileRegs<T, C, DV, NT> vr;
    const int nchunk = (B.count + C - 1) / C;
    auto gate = [&](int c) {        // wave 0: log-decay of this lane's token
        const int i = c * C + lane;
        return (lane < C && i < B.count) ? load_gate<T>(P, B.first + i, h) : 0.f;
    };
    auto load_chunk = [&](int c) {
        const int cnt = B.count - c * C;
        kr.load(k + (long)c * C * ks, ks, cnt, tid);
        vr.load(v + (long)c * C * vs, vs, cnt, tid);
        if (MODE == OUT)
            qr.load(q + (long)c * C * P.q_stride, P.q_stride, cnt, tid);
    };
    // the chunk of step i
    auto chunk = [&](int i) { return MODE == ROWN ? nchunk - 1 - i : i; };
    load_chunk(chunk(0));
    float la0 = 0.f, la1 = 0.f;
    if (w == 0) {
        la0 = gate(chunk(0));
        la1 = nchunk > 1 ? gate(chunk(1)) : 0.f;
    }

    StateAcc<T, DK, DV> S;
    const long sidx = (b * P.H + h) * (long)(DK * DV);
    const float *start = B.single ? P.S0 : P.ws_state;
    if (start)
        start += B.single ? (B.slot * P.H + h) * (long)(DK * DV) : sidx;
    if (MODE == OWN || MODE == ROWN || !start)
        S.zero();
    else if (MODE == CHUNKS)
        S.load_t(start, w, lane);
    else
        S.load(start, w, lane);

    if (MODE == OUT) {
        // the 16 x 16 tiles right of the diagonal inside a step of 32 tokens
        // are read and never written again
        for (int i = tid; i < C * PP; i += NT)
            Ps[i] = from_f32<T>(0.f);
    }
    double total = 0.;              // base-2 log of the block's decay (wave 0)
    if (w == 0)
        total = chunk_decays<C>(D[0], la0, lane);

    for (int step = 0; step < nchunk; ++step) {
        const int c = chunk(step);
        const Decays<C> &dc = D[step & 1];
        const int cnt = B.count - c * C;       // tokens from here on
        kr.template store<PK>(Ks, tid);
        vr.template store<PV>(Vs, tid);
        if (MODE == OUT)
            qr.template store<PK>(Qs, tid);
        __syncthreads();
        if (step + 1 < nchunk)
            load_chunk(chunk(step + 1));

        if (MODE == CHUNKS)
            S.store_frags(static_cast<T *>(P.ws_chunk) +
                              (chunk_slot(b, B.first, c, C) * P.H + h) * (long)(DK * DV),
                          w, lane);

        f32x4 o[IT][NC];
        if (MODE == OUT) {
            // P^T strip of 16 query rows: D[j][i], lane holds i = n, j = 4 g + r
            if (w < IT && 16 * w < cnt) {
                const int i = 16 * w + n;
                FragV<T> qf[DK / 32];
#pragma unroll
                for (int s = 0; s < DK / 32; ++s)
                    qf[s] = frag_row(Qs + i * PK + 32 * s + 8 * g);
                const float hi = dc.hi[i], lo = dc.lo[i];
#pragma unroll
                for (int jt = 0; jt < IT; ++jt) {
                    if (jt > w)
                        break;
                    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = 0; s < DK / 32; ++s)
                        mma(p, frag_row(Ks + (16 * jt + n) * PK + 32 * s + 8 * g), qf[s]);
                    float x[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * jt + 4 * g + r;
                        x[r] = j <= i ? p[r] * decay_between<T, C>(dc, hi, lo, j) : 0.f;
                    }
                    // rounded to the operand type: P feeds one product whose
                    // result is rounded to the same type
                    lds_stn<4>(Ps + i * PP + 16 * jt + 4 * g, x);
                }
            }
            // o^T = S^T q^T, scaled to each token
            FragV<T> sf[NC];
#pragma unroll
            for (int it = 0; it < IT; ++it)
#pragma unroll
                for (int cc = 0; cc < NC; ++cc)
                    o[it][cc] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) {
#pragma unroll
                for (int cc = 0; cc < NC; ++cc)
                    sf[cc] = frag_acc<T>(S.t[2 * s][cc], S.t[2 * s + 1][cc]);
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    const FragV<T> qf = frag_row_perm(Qs + (16 * it + n) * PK + 32 * s + 4 * g);
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc)
                        mma(o[it][cc], sf[cc], qf);
                }
            }
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const float a = dc.in[16 * it + n];
#pragma unroll
                for (int cc = 0; cc < NC; ++cc)
                    o[it][cc] *= a;
            }
        }
        if (w == 0) {               // the next chunk's decays
            if (step + 1 < nchunk)
                total += chunk_decays<C>(D[(step + 1) & 1], la1, lane);
            la1 = step + 2 < nchunk ? gate(chunk(step + 2)) : 0.f;
        }
        if (MODE == OUT)
            __syncthreads();        // P

        // v^T P^T, and the state: S <- all S + k^T (out (.) v)
        const float all = dc.all;
#pragma unroll
        for (int i = 0; i < TK; ++i)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
                S.t[i][cc] *= all;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            FragV<T> vf[NC];
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
                vf[cc] = frag_cols<PV>(Vs + 32 * s * PV, w * 16 * NC + 4 * cc, 4 * NC, lane);
            if (MODE == OUT) {
#pragma unroll
                for (int it = 2 * s; it < IT; ++it) {
                    const FragV<T> pf = frag_row(Ps + (16 * it + n) * PP + 32 * s + 8 * g);
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc)
                        mma(o[it][cc], vf[cc], pf);
                }
            }
            float wt[8];
            lds_ld8((MODE == ROWN ? dc.in : dc.out) + 32 * s + 8 * g, wt);
            const Split<T> v0(vf[0], wt);
            const Split<T> v1(vf[NC - 1], wt);
#pragma unroll
            for (int i = 0; i < TK; ++i) {
                const FragV<T> kf = frag_cols<PK>(Ks + 32 * s * PK, 16 * i, 4, lane);
                v0.mma_a(S.t[i][0], kf);
                if (NC == 2)
                    v1.mma_a(S.t[i][NC - 1], kf);
            }
        }
        if (MODE == OUT) {
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = 16 * it + n;
                if (i < cnt) {
                    T *dst = static_cast<T *>(P.o) +
                             ((B.first + (long)c * C + i) * P.H + h) * DV + w * 16 * NC + 4 * NC * g;
                    float x[4 * NC];
#pragma unroll
                    for (int cc = 0; cc < NC; ++cc)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            x[4 * cc + r] = o[it][cc][r];
                    if constexpr (NC == 2)
                        lds_st8(dst, x);
                    else
                        lds_stn<4>(dst, x);
                }
            }
        }
        __syncthreads();            // the chunk's tiles have been read
    }
    if (MODE == OWN || MODE == ROWN) {
        S.store((MODE == OWN ? P.ws_state : P.ws_rstate) + sidx, w, lane);
        if (tid == 0)
            (MODE == OWN ? P.ws_decay : P.ws_rdecay)[b * P.H + h] = exp2_fast((float)total);
    }
    if (MODE == OUT && B.last && P.S_out)
        S.store(P.S_out + (B.slot * P.H + h) * (long)(DK * DV), w, lane);
}

// ---------------------------------------------------------------------------
// Join of the blocks along each sequence: block b's own contribution U_b in
// ws_state becomes the state at its start (REV: in ws_rstate, the reverse
// state behind its end, blocks last to first).  One thread holds 4 values of S
// of one (sequence, head); the blocks' values are loaded JOIN ahead.  A
// sequence of one block has nothing to join, one without tokens passes its
// state on.
// ---------------------------------------------------------------------------
constexpr int JOIN = 8;

template <bool REV>
__global__ __launch_bounds__(NT) void linear_join_kernel(LinearParams P, int pieces) {
    const long id = blockIdx.x;
    const int piece = id % pieces;
    const int h = (id / pieces) % P.H;
    const int seq = id / ((long)pieces * P.H);
    const int e = (piece * NT + threadIdx.x) * 4;
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

template <typename T, int MODE>
static hipError_t launch_mode(const LinearParams &P, hipStream_t st) {
    const dim3 grid((unsigned)(linear_total_blocks(P) * P.H)), block(NT);
    // rows and columns of the state the mode works on
    const int rows = MODE == CHUNKS ? P.dv : P.dk, cols = MODE == CHUNKS ? P.dk : P.dv;
#define KDN_LIN(DK_, DV_)                                                              \
    if (rows == DK_ && cols == DV_) {                                                  \
        hipLaunchKernelGGL((linear_kernel<T, DK_, DV_, MODE>), grid, block, 0, st, P); \
        return hipGetLastError();                                                      \
    }
    KDN_LIN(64, 64)
    KDN_LIN(64, 128)
    KDN_LIN(128, 64)
    KDN_LIN(128, 128)
#undef KDN_LIN
    return hipErrorInvalidValue;
}

// The blocks' own contributions and their join, where a sequence may have more
// than one block; the join also passes on the states of empty sequences.
template <bool REV> static hipError_t launch_states(const LinearParams &P, hipStream_t st) {
    constexpr int MODE = REV ? ROWN : OWN;
    hipError_t e = hipSuccess;
    if (!P.block_offsets && P.nblocks == 1)
        return e;
    if (linear_total_blocks(P) > 0)
        e = P.bf16 ? launch_mode<bf16, MODE>(P, st) : launch_mode<float, MODE>(P, st);
    if (e != hipSuccess)
        return e;
    const int pieces = P.dk * P.dv / (4 * NT);
    const dim3 grid((unsigned)((long)P.N * P.H * pieces)), block(NT);
    hipLaunchKernelGGL((linear_join_kernel<REV>), grid, block, 0, st, P, pieces);
    return hipGetLastError();
}

}  // namespace lin

hipError_t launch_linear_states(const LinearParams &P, hipStream_t st) {
    return lin::launch_states<false>(P, st);
}

hipError_t launch_linear_reverse_states(const LinearParams &P, hipStream_t st) {
    return lin::launch_states<true>(P, st);
}

hipError_t launch_linear_chunk_states(const LinearParams &P, hipStream_t st) {
    return P.bf16 ? lin::launch_mode<bf16, lin::CHUNKS>(P, st)
                  : lin::launch_mode<float, lin::CHUNKS>(P, st);
}

hipError_t launch_linear_prefill(const LinearParams &P, hipStream_t st) {
    if (P.N == 0 || P.H == 0)
        return hipSuccess;
    const hipError_t e = launch_linear_states(P, st);
    if (e != hipSuccess || linear_total_blocks(P) == 0)
        return e;
    return P.bf16 ? lin::launch_mode<bf16, lin::OUT>(P, st) : lin::launch_mode<float, lin::OUT>(P, st);
}

}  // namespace kdn
