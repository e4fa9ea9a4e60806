// kdn_linear_backward.hip -- gradients of the chunked linear attention with a
// decay for each head (gfx950).
//
// With R the state of the reverse recurrence behind a chunk (of the block's
// end; R_T = dS_out) and S the state at its start, D_ij = e^{G_i - G_j}
// (j <= i), P = D (.) q k^T and Y = D (.) do v^T,
//   dq_i = sum_j Y_ij k_j + e^{G_i} S do_i
//   dk_j = sum_i Y_ij q_i + e^{G_C - G_j} R v_j
//   dv_j = sum_i P_ij do_i + e^{G_C - G_j} R^T k_j
//   R   <- e^{G_C} R + sum_i e^{G_i} q_i do_i^T        (dS0 = R at the start)
// and the gradient of a log-decay is everything that flows past its token:
//   dg_s = sum_{i >= s > j} X_ij + sum_{i >= s} x_i + sum_{j < s} y_j + z,
//   X = P (.) do v^T,  x_i = q_i . e^{G_i} S do_i,  y_j = k_j . e^{G_C-G_j} R v_j,
//   z = e^{G_C} <S, R>.
// The rows and columns of the same X are summed, so the terms of i < s cancel
// to float32; sums that ran on to the sequence's end would gather the rounding
// of every later token.
//
// The forward pass re-runs with a state at every chunk's start in memory
// (CHUNKS, in the call's type: the precision its product reads it in); the
// blocks' reverse states are joined as the forward ones are.  A workgroup then
// walks the chunks of one block backwards for one head, with R in MFMA
// accumulators (float32) and, in the operand type, in LDS; each wave has one
// 32 x 32 tile (channels x tokens) of dq, dk and dv and its tiles of R.  All
// products are computed transposed, so that a lane ends with runs of 8
// consecutive channels of a token.
//
// P, Y, S and R are read rounded to the operand type, once each: bfloat16
// gradients carry about one such rounding beside their own; sums over tokens are
// float32, of log-decays 64 bits.
//
// With one decay per head the sum of d log_alpha over all tokens cancels while
// these roundings add up (B3 H3 T186 with states: 1.2e-2 of the sum, computed in
// float32 7e-4, its own rounding).  FINE keeps both out of it: what the rounding
// of S leaves is saved beside it and multiplied too, what that of R leaves is
// multiplied from the accumulators (x and y to 2^-16 of a term), and <S, R> is a
// product only at the block's last chunk: from there on it is the sum of the x
// and y that it passes, exact enough for a sum over all tokens, not for a token's
// own value where later ones are far larger.  B4 H16 T4096 of 128 x 128 378 us
// against 302 with decays per token, B2 H16 T4096 of 64 x 64 94 against 87.
// Sequences of one chunk with states take it with decays per token as well: of
// few tokens x, y and z are most of d log_alpha, there is no sum over chunks, and
// the errors were up to twice those of a sum in float32.
//
// Measured (bf16, 128 x 128): B4 H16 T4096 302 us a call: own states of both
// directions 66-79 us, joins 14, states at the chunks' starts 60-71 (290 MB), the
// walk below 167-196.  It moves 1231 MB where 483 are needed, at 4.1 TB/s, 83 % of
// the rate of a large copy.  One workgroup has a CU: 512 threads of 256 registers
// each fill its registers, and q, k, v, do, P, Y and R of a chunk are 141 KB of
// LDS.  (64 x 64 has 4 waves and 70 KB, so that two fit.)  The walk's phases (P and
// Y; dq, dk, dv; R; d log_alpha) follow one another behind barriers: LDS is busy
// 27 % of the time, VALU 30, MFMA 18, 42 % is waiting; of its LDS cycles 18 % are
// bank conflicts, the row reads of the 16 x 16 tiles.  about 200 scalars are
// spilled to lanes of vector registers (strides, addresses and descriptors live
// over the loop).  The walk of the chunks' states split into two workgroups of 64
// columns each took 71 us for 68.  B1 H4 T333 of 64 x 64 float32: 33 us of
// kernels, the walk 17 (22 with dq and dk in the same waves).
#include <type_traits>

#include "kdn_linear_device.h"

namespace kdn {
namespace lin {

// FINE: what the roundings of S and R leave goes into d log_alpha.
template <typename T, int DK, int DV, bool FINE = false> struct GradShape {
    static constexpr int C = linear_chunk(sizeof(T) == 2);
    static constexpr int W = (DK > DV ? DK : DV) / 16;     // waves
    static constexpr int NT = W * WAVE;
    static constexpr int IT = C / 32;          // token tiles
    static constexpr int KT = DK / 32, VT = DV / 32;       // channel tiles
    static constexpr int TR = KT * VT / W;     // row tiles of R in a wave
    static constexpr int KS = C / 16;          // steps, and 16-token tiles
    static constexpr int PK = lds_pitch<T>(DK), PV = lds_pitch<T>(DV), PP = lds_pitch<T>(C);

    struct Lds {
        __attribute__((aligned(16))) T Qs[C * PK];
        __attribute__((aligned(16))) T Ks[C * PK];
        __attribute__((aligned(16))) T Vs[C * PV];
        __attribute__((aligned(16))) T Os[C * PV];
        __attribute__((aligned(16))) T Ps[C * PP];
        __attribute__((aligned(16))) T Ys[C * PP];
        __attribute__((aligned(16))) T Rs[DV * PK];      // R^T
        Decays<C> D[2];
        // sums of X over a tile's keys, and over a tile's queries
        __attribute__((aligned(16))) float rowx[KS][C], colx[KS][C];
        float xs[KT][C], ys[KT][C], zs[KT];
        float ylo[FINE ? W : 1][C];         // a wave's part of y from the rest of R
        double flow[FINE ? W : 1];          // and of <S, R> at the block's last chunk
    };
};

// Store of channels of a token to the gradient (call dtype) or to the float32
// partial of a shared head.
template <typename T>
__device__ __forceinline__ void store8(void *out, float *part, long at, const float (&f)[8]) {
    if (part)
        lds_st8(part + at, f);
    else
        lds_st8(static_cast<T *>(out) + at, f);
}
template <typename T>
__device__ __forceinline__ void store4(void *out, float *part, long at, f32x4 x) {
    const float f[4] = {x[0], x[1], x[2], x[3]};
    if (part)
        lds_stn<4>(part + at, f);
    else
        lds_stn<4>(static_cast<T *>(out) + at, f);
}

// PARTS: of the split operands in the update of R (Split).
template <typename T, int DK, int DV, int PARTS, bool FINE>
__device__ __forceinline__ void grad_walk(const LinearParams &P, const Block &B, long b, int h,
                                          typename GradShape<T, DK, DV, FINE>::Lds &L) {
    using SH = GradShape<T, DK, DV, FINE>;
    constexpr int C = SH::C, W = SH::W, NT = SH::NT, TR = SH::TR, KT = SH::KT, VT = SH::VT;
    constexpr int IT = SH::IT, KS = SH::KS, PK = SH::PK, PV = SH::PV, PP = SH::PP;

    T *const Qs = L.Qs, *const Ks = L.Ks, *const Vs = L.Vs, *const Os = L.Os;
    T *const Ps = L.Ps, *const Ys = L.Ys, *const Rs = L.Rs;
    auto &D = L.D;
    auto &rowx = L.rowx;
    auto &colx = L.colx;
    auto &xs = L.xs, &ys = L.ys;
    auto &zs = L.zs;

    const int tid = threadIdx.x, lane = tid & (WAVE - 1), w = wave_id();
    const int hf = lane >> 5, n = lane & 31, cn = chan(n);
    const int rn = lds_row(n), rcn = lds_row(cn);   // their places in a tile
    // channel and token tile of dq and dk; where there are waves for both (float32,
    // and d_k < d_v), dq and dk have waves of their own, and so has <S, R>
    constexpr int ROLES = W / KT / IT;
    constexpr bool APART = ROLES >= 2;
    const int qc = w % KT, qt = w / KT % IT, role = w / KT / IT;
    const bool do_q = role == 0, do_k = role == (APART ? 1 : 0);
    constexpr int ZROLE = ROLES > 2 ? 2 : ROLES - 1;
    const bool do_z = role == ZROLE && qt == 0;
    const int vc = w % VT, vt = w / VT;     // of dv; and column tile and row group of R
    const int hq = h / (P.H / P.Hq), hk = h / (P.H / P.Hk), hv = h / (P.H / P.Hv);
    // outputs: rows of the shared heads' partials have all H heads
    const long qrow = P.ws_dq ? (long)P.H * DK : (long)P.Hq * DK;
    const long krow = P.ws_dk ? (long)P.H * DK : (long)P.Hk * DK;
    const long vrow = P.ws_dv ? (long)P.H * DV : (long)P.Hv * DV;
    const long qat = B.first * qrow + (P.ws_dq ? h : hq) * DK;
    const long kat = B.first * krow + (P.ws_dk ? h : hk) * DK;
    const long vat = B.first * vrow + (P.ws_dv ? h : hv) * DV;
    T *dla = static_cast<T *>(P.gate == KDN_GATE_TOKEN ? P.dla : nullptr);
    if (B.slot < 0) {               // a skipped sequence: zero
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        // 64 bits: a block may have 2^26 tokens and more
        for (long i = tid; i < (long)B.count * (DK / 4); i += NT) {
            const long r = i / (DK / 4), c = i % (DK / 4) * 4;
            store4<T>(P.dq, P.ws_dq, qat + r * qrow + c, zero);
            store4<T>(P.dk_, P.ws_dk, kat + r * krow + c, zero);
        }
        for (long i = tid; i < (long)B.count * (DV / 4); i += NT)
            store4<T>(P.dv_, P.ws_dv, vat + i / (DV / 4) * vrow + i % (DV / 4) * 4, zero);
        if (dla)
            for (long i = tid; i < B.count; i += NT)
                dla[(B.first + i) * P.H + h] = from_f32<T>(0.f);
        return;
    }

    const T *q = static_cast<const T *>(P.q) + B.first * P.q_stride + hq * DK;
    const T *k = static_cast<const T *>(P.k) + B.first * P.k_stride + hk * DK;
    const T *v = static_cast<const T *>(P.v) + B.first * P.v_stride + hv * DV;
    const long ostride = P.o_stride;
    const T *od = static_cast<const T *>(P.d_o) + B.first * ostride + h * DV;

    TileRegs<T, C, DK, NT> qr, kr;
    TileRegs<T, C, DV, NT> vr, orr;
    const int nchunk = (B.count + C - 1) / C;
    const float head = P.gate == KDN_GATE_HEAD ? static_cast<const float *>(P.la)[h] : 0.f;
    GateReg<T> la0, la1;            // wave GW: this lane's token, this chunk and the next
    auto gate = [&](GateReg<T> &x, int c) {
        x.template load<C>(P, B.first + (long)c * C, B.count - c * C, h, lane);
    };
    auto gate_value = [&](const GateReg<T> &x, int c) {
        return x.value(P, head, lane < C && c * C + lane < B.count);
    };
    auto load_chunk = [&](int c) {
        const int cnt = B.count - c * C;
        qr.load(q + (long)c * C * P.q_stride, P.q_stride, cnt, tid);
        kr.load(k + (long)c * C * P.k_stride, P.k_stride, cnt, tid);
        vr.load(v + (long)c * C * P.v_stride, P.v_stride, cnt, tid);
        orr.load(od + (long)c * C * ostride, ostride, cnt, tid);
    };
    constexpr int GW = W - 1;       // the wave of the decays: the fewest tiles of P
    if (w == GW) {
        gate(la0, nchunk - 1);
        if (nchunk > 1)
            gate(la1, nchunk - 2);
    }
    load_chunk(nchunk - 1);

    // R: rows row(i, r), column col of this lane
    f32x16 R[TR];
    const int col = 32 * vc + cn, row0 = vt * TR * 32 + 8 * hf;
    auto row = [&](int i, int r) { return row0 + 32 * i + 16 * (r / 8) + r % 8; };
    auto share_state = [&]() {
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    f[r] = R[i][8 * j + r];
                lds_st8(Rs + (32 * vc + rcn) * PK + row(i, 8 * j), f);
            }
    };
    const long hs = (long)DK * DV;
    const float *rstart = B.single ? P.dS_out : P.ws_rstate;
    if (rstart)
        rstart += B.single ? (B.slot * P.H + h) * hs : (b * P.H + h) * hs;
#pragma unroll
    for (int i = 0; i < TR; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            R[i][r] = rstart ? rstart[row(i, r) * DV + col] : 0.f;
    FragV<T> sf[DV / 16];           // rows of S of this wave, a chunk ahead
    auto state_of = [&](const void *ws, int c) {
        return reinterpret_cast<const FragV<T> *>(
            static_cast<const T *>(ws) + (chunk_slot(b, B.first, c, C) * P.H + h) * hs);
    };
    auto load_state = [&](const void *ws, int c) {
        const FragV<T> *src = state_of(ws, c);
#pragma unroll
        for (int s = 0; s < DV / 16; ++s)
            sf[s] = src[(qc * (DV / 16) + s) * WAVE + lane];
    };
    if (do_q || (do_z && !FINE))
        load_state(P.ws_chunk, nchunk - 1);
    if constexpr (FINE) {
        // <S, R> of the block's last chunk, R as it is and S in both its parts:
        // a piece is 8 neighbours of a row of S
        float z = 0.f;
        if (rstart) {
            const FragV<T> *hi = state_of(P.ws_chunk, nchunk - 1);
            const FragV<T> *lo = state_of(P.ws_chunk_lo, nchunk - 1);
            for (int i = tid; i < DK * DV / 8; i += NT) {
                const int l = i % WAVE, s = i / WAVE % (DV / 16), t = i / WAVE / (DV / 16);
                const float *r = rstart + (32 * t + chan(l & 31)) * DV + 16 * s + 8 * (l >> 5);
                const FragV<T> x = hi[i], y = lo[i];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    z += (to_f32(x[e]) + to_f32(y[e])) * r[e];
            }
        }
        z = wave_sum(z);
        if (lane == 0)
            L.flow[w] = z;
    }
    if (w == GW)
        chunk_decays<C>(D[0], gate_value(la0, nchunk - 1), lane);
    share_state();
    // P and Y right of the diagonal inside the 32 x 32 tiles: never written
    for (int i = tid; i < C * PP; i += NT) {
        Ps[i] = from_f32<T>(0.f);
        Ys[i] = from_f32<T>(0.f);
    }
    double gsum = 0.;               // wave GW: sum of the block's d log_alpha (this lane's)
    double flow = 0.;               // FINE: <S, R> between two chunks

    for (int step = 0; step < nchunk; ++step) {
        const int c = nchunk - 1 - step;
        const Decays<C> &dc = D[step & 1];
        const int cnt = B.count - c * C;
        qr.template store<PK>(Qs, tid);
        kr.template store<PK>(Ks, tid);
        vr.template store<PV>(Vs, tid);
        orr.template store<PV>(Os, tid);
        __syncthreads();

        // 16 x 16 tiles of P^T and Y^T on and below the diagonal (small ones:
        // 10 tiles keep 8 waves busy, 3 of 32 x 32 would not), and X's sums.
        // Lane m has query i = 16 it + m and 4 keys.
        for (int t = w; t < KS * (KS + 1) / 2; t += W) {
            int it = 0, jt = t;
            while (jt > it)
                jt -= ++it;
            const int m = lane & 15, g = lane >> 4;
            const int i = 16 * it + m, j = 16 * jt + 4 * g;
            const int ri = lds_row(i), rk = 16 * jt + lds_row(m);
            f32x4 p = {0.f, 0.f, 0.f, 0.f}, y = p;
            {
                FragV<T> a[DK / 32], x[DK / 32];
#pragma unroll
                for (int s = 0; s < DK / 32; ++s) {
                    a[s] = frag_row(Ks + rk * PK + 32 * s + 8 * g);
                    x[s] = frag_row(Qs + ri * PK + 32 * s + 8 * g);
                }
                FragV<T> e[DV / 32], f[DV / 32];
#pragma unroll
                for (int s = 0; s < DV / 32; ++s) {
                    e[s] = frag_row(Vs + rk * PV + 32 * s + 8 * g);
                    f[s] = frag_row(Os + ri * PV + 32 * s + 8 * g);
                }
                if (sizeof(T) == 2)
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < DK / 32; ++s)
                    mma(p, a[s], x[s]);
#pragma unroll
                for (int s = 0; s < DV / 32; ++s)
                    mma(y, e[s], f[s]);
            }
            float d[4], pf[4], yf[4], row = 0.f;
            decay_between<T>(dc, dc.hi[i], dc.lo[i], i, j, d);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                pf[r] = p[r] * d[r];
                yf[r] = y[r] * d[r];
                // X without its diagonal, which no log-decay is between
                float x = j + r < i ? pf[r] * y[r] : 0.f;
                row += x;
                x = row16_sum_last(x);
                if (m == 15)
                    colx[it][j + r] = x;
            }
            lds_stn<4>(Ps + ri * PP + j, pf);
            lds_stn<4>(Ys + ri * PP + j, yf);
            row += __shfl_xor(row, 16, WAVE);
            row += __shfl_xor(row, 32, WAVE);
            if (g == 0)
                rowx[jt][i] = row;
        }

        // What comes from S and R, scaled to each token.  Operands are read a
        // few steps at a time, so that their latency is paid once for all.
        // (sched_barrier: what a phase reads is not read in the phase before,
        // whose registers it would need.)
        __builtin_amdgcn_sched_barrier(0);
        // as the registers allow
        constexpr int G = DK + DV < 256 ? (sizeof(T) == 2 ? 4 : 2) : (sizeof(T) == 2 ? 2 : 1);
        f32x16 aq = zero16(), ak = zero16(), av = zero16();
        auto channels = [&](auto dq, auto dk, auto dz) {    // which of them: compile-time
            constexpr bool Q = decltype(dq)::value, K = decltype(dk)::value, Z = decltype(dz)::value;
            const int i = 32 * qt + n, ri = 32 * qt + rn;
            const bool want_z = Z && P.dla && do_z;
            f32x16 z = zero16();         // S R^T of this wave's channels: its diagonal
#pragma unroll
            for (int s0 = 0; s0 < DV / 16; s0 += G) {
                FragV<T> rf[G], of[G], vf[G];
#pragma unroll
                for (int s = 0; s < G; ++s) {
                    if constexpr (K || Z)
                        rf[s] = frag_cols<PK, true>(Rs + 16 * (s0 + s) * PK + 32 * qc, lane);
                    if constexpr (Q)
                        of[s] = frag_row(Os + ri * PV + 16 * (s0 + s) + 8 * hf);
                    if constexpr (K)
                        vf[s] = frag_row(Vs + ri * PV + 16 * (s0 + s) + 8 * hf);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < G; ++s) {
                    if constexpr (Q)
                        mma(aq, sf[s0 + s], of[s]);
                    if constexpr (K)
                        mma(ak, rf[s], vf[s]);
                }
                if constexpr (Z)
                    if (want_z) {
#pragma unroll
                        for (int s = 0; s < G; ++s)
                            mma(z, sf[s0 + s], rf[s]);
                    }
            }
            if constexpr (Q)
                aq *= dc.in[i];
            if constexpr (K)
                ak *= dc.out[i];
            if (P.dla) {
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float qx[8], kx[8];
                    if constexpr (Q)
                        lds_ld8(Qs + ri * PK + 32 * qc + 16 * u + 8 * hf, qx);
                    if constexpr (K)
                        lds_ld8(Ks + ri * PK + 32 * qc + 16 * u + 8 * hf, kx);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if constexpr (Q)
                            x += aq[8 * u + r] * qx[r];
                        if constexpr (K)
                            y += ak[8 * u + r] * kx[r];
                    }
                }
                if constexpr (Q)
                    x += __shfl_xor(x, 32, WAVE);
                if constexpr (K)
                    y += __shfl_xor(y, 32, WAVE);
                if (hf == 0) {
                    if constexpr (Q)
                        xs[qc][i] = x;
                    if constexpr (K)
                        ys[qc][i] = y;
                }
                if (want_z) {
                    float zd = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        zd += 8 * (r / 4) + 4 * hf + r % 4 == n ? z[r] : 0.f;
                    zd = wave_sum(zd);
                    if (lane == 0)
                        zs[qc] = zd;
                }
            }
        };
        typedef std::true_type Yes;
        typedef std::false_type No;
        if constexpr (!APART) {
            if (do_q)
                channels(Yes{}, Yes{}, std::bool_constant<!FINE>{});
        } else {
            if (do_q)
                channels(Yes{}, No{}, No{});
            else if (do_k)
                channels(No{}, Yes{}, std::bool_constant<ZROLE == 1 && !FINE>{});
            else if (ZROLE == 2 && do_z && !FINE)
                channels(No{}, No{}, Yes{});
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (FINE) {
            if (do_q)
                load_state(P.ws_chunk_lo, c);
        } else if ((do_q || do_z) && step + 1 < nchunk)
            load_state(P.ws_chunk, c - 1);
        if (vt < IT) {
            const int i = 32 * vt + n;
#pragma unroll
            for (int s0 = 0; s0 < DK / 16; s0 += G) {
                FragV<T> rf[G], kf[G];
#pragma unroll
                for (int s = 0; s < G; ++s) {
                    rf[s] = frag_row(Rs + (32 * vc + rcn) * PK + 16 * (s0 + s) + 8 * hf);
                    kf[s] = frag_row(Ks + (32 * vt + rn) * PK + 16 * (s0 + s) + 8 * hf);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < G; ++s)
                    mma(av, rf[s], kf[s]);
            }
            av *= dc.out[i];
        }
        if constexpr (FINE) {
            // what the roundings of R and S leave of y and x: this wave's tiles of
            // R, as they are in its registers, on all tokens (y_j = v_j . R^T k_j),
            // and the rest of its channels of S
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                const int i = 32 * it + n, ri = 32 * it + rn;
                f32x16 a = zero16();
#pragma unroll
                for (int s = 0; s < 2 * TR; ++s)
                    mma(a, frag_rest<T>(R[s / 2], s % 2),
                        frag_row(Ks + ri * PK + 32 * vt * TR + 16 * s + 8 * hf));
                float y = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float vx[8];
                    lds_ld8(Vs + ri * PV + 32 * vc + 16 * u + 8 * hf, vx);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        y += a[8 * u + r] * vx[r];
                }
                y += __shfl_xor(y, 32, WAVE);
                if (hf == 0)
                    L.ylo[w][i] = y * dc.out[i];
                __builtin_amdgcn_sched_barrier(0);
            }
            if (do_q) {
                const int i = 32 * qt + n, ri = 32 * qt + rn;
                f32x16 a = zero16();
#pragma unroll
                for (int s = 0; s < DV / 16; ++s)
                    mma(a, sf[s], frag_row(Os + ri * PV + 16 * s + 8 * hf));
                float x = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float qx[8];
                    lds_ld8(Qs + ri * PK + 32 * qc + 16 * u + 8 * hf, qx);
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        x += a[8 * u + r] * qx[r];
                }
                x += __shfl_xor(x, 32, WAVE);
                if (hf == 0)
                    xs[qc][i] += x * dc.in[i];      // which this lane wrote
                __builtin_amdgcn_sched_barrier(0);
                if (step + 1 < nchunk)
                    load_state(P.ws_chunk, c - 1);
            }
        }
        const float la = gate_value(la0, c);      // wave GW: this chunk's log-decays
        if (w == GW) {
            if (step + 1 < nchunk)
                chunk_decays<C>(D[(step + 1) & 1], gate_value(la1, c - 1), lane);
            la0 = la1;
            if (step + 2 < nchunk)
                gate(la1, c - 2);
        }
        __syncthreads();            // P, Y and the sums

        if (w == GW && P.dla) {
            // opaque: the addresses below are made here, not held over the loop
            int tok = lane;
            asm volatile("" : "+v"(tok));
            const bool live = tok < C && tok < cnt;
            float u = 0.f, x = 0.f, y = 0.f, zz = 0.f;
            if (tok < C) {
                const int t = tok / 16;
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    u += (j <= t ? rowx[j][tok] : 0.f) - (j >= t ? colx[j][tok] : 0.f);
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    x += xs[i][tok];
                    y += ys[i][tok];
                }
                if constexpr (FINE)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        y += L.ylo[i][tok];
                u += x;
                u -= y;
            }
            if (!FINE) {
#pragma unroll
                for (int i = 0; i < KT; ++i)
                    zz += zs[i];
            }
            // with u = row - col + x - y: sum_{i >= s} (u_i + y_i) + sum_{j < s} y_j
            // is all of y and what of u is not before s
            const double past = prefix_sum((double)u);
            const double ally = lane_value(prefix_sum((double)y), WAVE - 1);
            double dg = lane_value(past, WAVE - 1) - past + (double)u + ally;
            if constexpr (FINE) {
                // <S, R> at the chunk's end is z and all of y, at its start z and all
                // of x: only the last chunk's is a product
                double z = flow - ally;
                if (step == 0) {
                    z = 0.;
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        z += L.flow[i];
                    z *= (double)dc.all();
                }
                flow = z + lane_value(prefix_sum((double)x), WAVE - 1);
                dg += z;
            } else {
                dg = (float)dg + dc.all() * zz;
            }
            if (log2_decay(la) <= (double)RESET2)
                dg = 0.;            // a reset lets nothing past
            if (live) {
                if (dla)
                    dla[(B.first + (long)c * C + tok) * P.H + h] = from_f32<T>((float)dg);
                gsum += dg;
            }
        }

        __builtin_amdgcn_sched_barrier(0);
        // what comes from the chunk's own tokens: operands first
        auto own_q = [&]() {
            FragV<T> x[KS], y[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 <= qt) {      // dq_i: j <= i
                    x[s] = frag_cols<PK, true>(Ks + 16 * s * PK + 32 * qc, lane);
                    y[s] = frag_row(Ys + (32 * qt + rn) * PP + 16 * s + 8 * hf);
                }
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 <= qt)
                    mma(aq, x[s], y[s]);
        };
        auto own_k = [&]() {
            FragV<T> x[KS], y[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 >= qt) {      // dk_j: i >= j
                    x[s] = frag_cols<PK, true>(Qs + 16 * s * PK + 32 * qc, lane);
                    y[s] = frag_cols<PP, false>(Ys + 16 * s * PP + 32 * qt, lane);
                }
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 >= qt)
                    mma(ak, x[s], y[s]);
        };
        auto store_channels = [&](const f32x16 &a, void *out, float *part, long at, long pitch) {
            if (32 * qt + n >= cnt)
                return;
            const long t0 = (long)c * C + 32 * qt + n;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    x[r] = a[8 * u + r];
                store8<T>(out, part, at + t0 * pitch + 32 * qc + 16 * u + 8 * hf, x);
            }
        };
        if (do_q) {
            own_q();
            if constexpr (!APART) {
                __builtin_amdgcn_sched_barrier(0);
                own_k();
                __builtin_amdgcn_sched_barrier(0);
                store_channels(ak, P.dk_, P.ws_dk, kat, krow);
            }
            store_channels(aq, P.dq, P.ws_dq, qat, qrow);
        } else if (APART && do_k) {
            own_k();
            store_channels(ak, P.dk_, P.ws_dk, kat, krow);
        }
        __builtin_amdgcn_sched_barrier(0);
        FragV<T> of[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s)
            of[s] = frag_cols<PV, true>(Os + 16 * s * PV + 32 * vc, lane);
        if (step + 1 < nchunk)
            load_chunk(c - 1);
        if (vt < IT) {
            FragV<T> pc[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 >= vt)
                    pc[s] = frag_cols<PP, false>(Ps + 16 * s * PP + 32 * vt, lane);
#pragma unroll
            for (int s = 0; s < KS; ++s)
                if (s / 2 >= vt)
                    mma(av, of[s], pc[s]);
            if (32 * vt + n < cnt) {
                const long t0 = (long)c * C + 32 * vt + n;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        x[r] = av[8 * u + r];
                    store8<T>(P.dv_, P.ws_dv, vat + t0 * vrow + 32 * vc + 16 * u + 8 * hf, x);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // R <- all R + q^T (in (.) do)
        auto rows = [&](int s, int i) {
            return frag_cols<PK, true>(Qs + 16 * s * PK + 32 * (vt * TR + i), lane);
        };
        FragV<T> rq[TR];
        Split<T, PARTS> split;
        float wt[8];
        lds_ld8(dc.in + 8 * hf, wt);
#pragma unroll
        for (int i = 0; i < TR; ++i)
            rq[i] = rows(0, i);
        const float all = dc.all();
#pragma unroll
        for (int i = 0; i < TR; ++i)
            R[i] *= all;
#pragma unroll
        for (int i = 0; i < 4 * Split<T, PARTS>::PARTS; ++i)
            split.step(i, of[0], wt);
        update_state<T, PARTS>(R, of, dc.in, hf, split, rq, rows, [](int, int) {});
        share_state();              // Rs was read before the barrier above
        __syncthreads();            // the chunk's tiles have been read
    }
    if (B.index == 0 && P.dS0) {
        float *dst = P.dS0 + (B.slot * P.H + h) * hs;
#pragma unroll
        for (int i = 0; i < TR; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                dst[row(i, r) * DV + col] = R[i][r];
    }
    if (P.ws_dla && w == GW) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            gsum += __shfl_xor(gsum, off, WAVE);
        if (lane == 0)
            P.ws_dla[b * P.H + h] = gsum;
    }
}

template <typename T, int DK, int DV, bool FINE>
__global__ __launch_bounds__((GradShape<T, DK, DV>::NT)) void linear_grad_kernel(LinearParams P) {
    const long b = block_at(P, blockIdx.x / P.H);
    const int h = blockIdx.x % P.H;
    const Block B = get_block(P, b);
    if (P.ws_dla && (B.count == 0 || B.slot < 0) && threadIdx.x == 0)
        P.ws_dla[b * P.H + h] = 0.;
    if (B.count == 0)
        return;
    __shared__ typename GradShape<T, DK, DV, FINE>::Lds L;
    // three parts where R ends as dS0
    if (B.index == 0)
        grad_walk<T, DK, DV, 3, FINE>(P, B, b, h, L);
    else
        grad_walk<T, DK, DV, 2, FINE>(P, B, b, h, L);
}

// Joins of the forward and of the reverse states, zero gradients for the rows
// behind the last sequence of a packed batch, and the order of its blocks, by
// the workgroups' numbers.
constexpr int TNT = 256, TAIL_WGS = 64;
template <typename T>
__device__ __forceinline__ void clear_tail(const LinearParams &P, long wg) {
    const int nb = P.block_offsets[P.N];
    long end = 0;
    if (nb > 0 && nb <= P.nblocks) {
        const int4 r = reinterpret_cast<const int4 *>(P.blocks)[nb - 1];
        end = (long)r.x + r.y;
    }
    if (end < 0 || end >= P.tokens)
        return;
    const long rows = P.tokens - end, stride = (long)TAIL_WGS * TNT;
    const long id = wg * TNT + threadIdx.x;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    auto clear = [&](void *out, float *part, int heads, int d) {
        const long row = (long)(part ? P.H : heads) * d;
        for (long i = id; i < rows * row / 4; i += stride)
            store4<T>(out, part, end * row + 4 * i, zero);
    };
    clear(P.dq, P.ws_dq, P.Hq, P.dk);
    clear(P.dk_, P.ws_dk, P.Hk, P.dk);
    clear(P.dv_, P.ws_dv, P.Hv, P.dv);
    if (P.dla && P.gate == KDN_GATE_TOKEN)
        for (long i = id; i < rows * P.H; i += stride)
            static_cast<T *>(P.dla)[end * P.H + i] = from_f32<T>(0.f);
}

template <typename T>
__global__ __launch_bounds__(TNT) void linear_grad_join_kernel(LinearParams P, int pieces,
                                                               long joins, long tail) {
    static_assert(TNT == JOIN_NT, "one launch for both");
    const long id = blockIdx.x;
    if (id >= 2 * joins + tail)
        order_blocks(P);
    else if (id >= 2 * joins)
        clear_tail<T>(P, id - 2 * joins);
    else if (id & 1)
        join_blocks<true>(P, id >> 1, pieces);
    else
        join_blocks<false>(P, id >> 1, pieces);
}

// Gradient of a shared head: the sum over the states that read it, in order.
// n groups of 4 values of `out`, `row` values of a token in it.
template <typename T> struct Share {
    const float *part;
    T *out;
    long n;
    int row, d, group;
    __device__ __forceinline__ void sum(long g) const {
        const long i = g * 4, t = i / row;
        const int c = i % row, hh = c / d;
        const float *p = part + t * row * group + (long)hh * group * d + c % d;
        f32x4 x = *reinterpret_cast<const f32x4 *>(p);
        for (int j = 1; j < group; ++j)
            x += *reinterpret_cast<const f32x4 *>(p + (long)j * d);
        store4<T>(out, nullptr, i, x);
    }
};
template <typename T>
__global__ __launch_bounds__(TNT) void linear_share_kernel(Share<T> q, Share<T> k, Share<T> v) {
    long i = (long)blockIdx.x * TNT + threadIdx.x;
    if (i < q.n)
        return q.sum(i);
    if ((i -= q.n) < k.n)
        return k.sum(i);
    if ((i -= k.n) < v.n)
        v.sum(i);
}

// One decay per head: the sum over the blocks, in 64 bits in a fixed order.
template <typename T>
__global__ __launch_bounds__(WAVE) void linear_gate_sum_kernel(LinearParams P, long blocks) {
    const int h = blockIdx.x, lane = threadIdx.x;
    double x = 0.;
    for (long b = lane; b < blocks; b += WAVE)
        x += P.ws_dla[b * P.H + h];
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1)
        x += __shfl_xor(x, off, WAVE);
    if (lane == 0) {
        if (P.dla_f32)
            static_cast<float *>(P.dla)[h] = (float)x;
        else
            static_cast<T *>(P.dla)[h] = from_f32<T>((float)x);
    }
}

template <typename T>
static Share<T> share(const LinearParams &P, const float *part, void *out, int heads, int d) {
    return Share<T>{part, static_cast<T *>(out), part ? P.tokens * heads * d / 4 : 0, heads * d, d,
                    P.H / (heads ? heads : 1)};
}

template <typename T> static hipError_t launch_grad(const LinearParams &call, hipStream_t st) {
    LinearParams P = call;
    const long blocks = linear_total_blocks(P);
    const bool sort = ordered(P);
    if (!sort)
        P.ws_order = nullptr;
    hipError_t e = hipSuccess;
    const bool several = P.block_offsets || P.nblocks != 1;     // blocks in a sequence, or none
    if (several && blocks > 0)
        e = launch_linear_own(P, st);
    const int pieces = join_pieces(P);
    const long joins = several ? (long)P.N * P.H * pieces : 0;
    const long tail = P.block_offsets && P.tokens > 0 ? TAIL_WGS : 0;
    if (e == hipSuccess && joins + tail + sort > 0) {
        hipLaunchKernelGGL(linear_grad_join_kernel<T>, 
                           dim3((unsigned)(2 * joins + tail + sort)), dim3(TNT), 0, st, P, pieces,
                           joins, tail);
        e = hipGetLastError();
    }
    if (e == hipSuccess && blocks > 0)
        e = launch_linear_chunk_states(P, st);
    if (e == hipSuccess && blocks > 0) {
        const dim3 grid((unsigned)(blocks * P.H));
        auto walk = [&](auto fine) {
#define KDN_LGRAD(DK_, DV_)                                                                  \
            if (P.dk == DK_ && P.dv == DV_)                                                  \
                hipLaunchKernelGGL((linear_grad_kernel<T, DK_, DV_, decltype(fine)::value>), \
                                   grid, dim3(GradShape<T, DK_, DV_>::NT), 0, st, P);
            KDN_LGRAD(64, 64)
            KDN_LGRAD(64, 128)
            KDN_LGRAD(128, 64)
            KDN_LGRAD(128, 128)
#undef KDN_LGRAD
        };
        if constexpr (sizeof(T) == 2) {
            if (P.ws_chunk_lo)
                walk(std::true_type{});
            else
                walk(std::false_type{});
        } else {
            walk(std::false_type{});
        }
        e = hipGetLastError();
    }
    const Share<T> q = share<T>(P, P.ws_dq, P.dq, P.Hq, P.dk);
    const Share<T> k = share<T>(P, P.ws_dk, P.dk_, P.Hk, P.dk);
    const Share<T> v = share<T>(P, P.ws_dv, P.dv_, P.Hv, P.dv);
    const long n = q.n + k.n + v.n;
    if (e == hipSuccess && n > 0) {
        hipLaunchKernelGGL(linear_share_kernel<T>, dim3((unsigned)((n + TNT - 1) / TNT)), dim3(TNT),
                           0, st, q, k, v);
        e = hipGetLastError();
    }
    if (e == hipSuccess && P.dla && P.gate == KDN_GATE_HEAD) {
        hipLaunchKernelGGL(linear_gate_sum_kernel<T>, dim3((unsigned)P.H), dim3(WAVE), 0, st, P,
                           blocks);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace lin

hipError_t launch_linear_backward(const LinearParams &P, hipStream_t st) {
    if (P.H == 0)
        return hipSuccess;
    return P.bf16 ? lin::launch_grad<bf16>(P, st) : lin::launch_grad<float>(P, st);
}

}  // namespace kdn
