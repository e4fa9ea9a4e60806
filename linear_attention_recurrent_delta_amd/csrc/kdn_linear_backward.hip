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
// accumulators, each wave the rows of dq and dk and the columns of dv and R
// that follow from its number.  All products are computed transposed (a lane
// ends with consecutive channels of a token).
#include "kdn_linear_device.h"

namespace kdn {
namespace lin {

template <typename T, int DK, int DV> struct GradShape {
    static constexpr int C = linear_chunk(sizeof(T) == 2);
    static constexpr int W = (DK < DV ? DK : DV) / 16;     // waves
    static constexpr int NT = W * WAVE;
    static constexpr int NC = DV / 16 / W;     // column tiles of R and dv of a wave
    static constexpr int TR = DK / 16 / W;     // row tiles of dq and dk of a wave
    static constexpr int TK = DK / 16;         // row tiles of R
    static constexpr int IT = C / 16, KS = C / 32;
    static constexpr int PAD = 16 / sizeof(T);
    static constexpr int PK = DK + PAD, PV = DV + PAD, PP = C + PAD;
};

// First channel and the step between groups of 4 of 16-channel tile t of D
// channels: tiles share runs of 4 D / 64 channels, as the accumulators of
// kdn_linear.hip do (the saved states are in that order).
template <int D> __device__ __forceinline__ int tile_first(int t) {
    return t / (D / 64) * (D / 4) + 4 * (t % (D / 64));
}
template <int D> constexpr int tile_step() { return 4 * (D / 64); }

// Store of 4 channels of a token to the gradient (call dtype) or to the
// float32 partial of a shared head.
template <typename T>
__device__ __forceinline__ void store4(void *out, float *part, long at, f32x4 x) {
    const float f[4] = {x[0], x[1], x[2], x[3]};
    if (part)
        lds_stn<4>(part + at, f);
    else
        lds_stn<4>(static_cast<T *>(out) + at, f);
}

template <typename T, int DK, int DV>
__global__ __launch_bounds__((GradShape<T, DK, DV>::NT)) void linear_grad_kernel(LinearParams P) {
    using SH = GradShape<T, DK, DV>;
    constexpr int C = SH::C, W = SH::W, NT = SH::NT, NC = SH::NC, TR = SH::TR, TK = SH::TK;
    constexpr int IT = SH::IT, KS = SH::KS, PK = SH::PK, PV = SH::PV, PP = SH::PP;

    __shared__ __attribute__((aligned(16))) T Qs[C * PK];
    __shared__ __attribute__((aligned(16))) T Ks[C * PK];
    __shared__ __attribute__((aligned(16))) T Vs[C * PV];
    __shared__ __attribute__((aligned(16))) T Os[C * PV];
    __shared__ __attribute__((aligned(16))) T Ps[C * PP];
    __shared__ __attribute__((aligned(16))) T Ys[C * PP];
    __shared__ __attribute__((aligned(16))) T Rs[DV * PK];      // R^T
    __shared__ __attribute__((aligned(16))) Decays<C> D[2];
    __shared__ float rowx[IT][C], colx[IT][C];   // sums of X over a tile's columns / rows
    __shared__ float xs[W][C], ys[W][C], zs[W];

    const int tid = threadIdx.x, lane = tid & (WAVE - 1), w = tid / WAVE;
    const int g = lane >> 4, n = lane & 15;
    const long b = blockIdx.x / P.H;
    const int h = blockIdx.x % P.H;
    const Block B = get_block(P, b);
    if (P.ws_dla && (B.count == 0 || B.slot < 0) && tid == 0)
        P.ws_dla[b * P.H + h] = 0.;
    if (B.count == 0)
        return;

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
        for (int i = tid; i < B.count * (DK / 4); i += NT) {
            const int r = i / (DK / 4), c = i % (DK / 4) * 4;
            store4<T>(P.dq, P.ws_dq, qat + r * qrow + c, zero);
            store4<T>(P.dk_, P.ws_dk, kat + r * krow + c, zero);
        }
        for (int i = tid; i < B.count * (DV / 4); i += NT)
            store4<T>(P.dv_, P.ws_dv, vat + i / (DV / 4) * vrow + i % (DV / 4) * 4, zero);
        if (dla)
            for (int i = tid; i < B.count; i += NT)
                dla[(B.first + i) * P.H + h] = from_f32<T>(0.f);
        return;
    }

    const T *q = static_cast<const T *>(P.q) + B.first * P.q_stride + hq * DK;
    const T *k = static_cast<const T *>(P.k) + B.first * P.k_stride + hk * DK;
    const T *v = static_cast<const T *>(P.v) + B.first * P.v_stride + hv * DV;
    const long ostride = (long)P.H * DV;
    const T *od = static_cast<const T *>(P.d_o) + B.first * ostride + h * DV;

    TileRegs<T, C, DK, NT> qr, kr;
    TileRegs<T, C, DV, NT> vr, orr;
    const int nchunk = (B.count + C - 1) / C;
    auto gate = [&](int c) {
        const int i = c * C + lane;
        return (lane < C && i < B.count) ? load_gate<T>(P, B.first + i, h) : 0.f;
    };
    auto load_chunk = [&](int c) {
        const int cnt = B.count - c * C;
        qr.load(q + (long)c * C * P.q_stride, P.q_stride, cnt, tid);
        kr.load(k + (long)c * C * P.k_stride, P.k_stride, cnt, tid);
        vr.load(v + (long)c * C * P.v_stride, P.v_stride, cnt, tid);
        orr.load(od + (long)c * C * ostride, ostride, cnt, tid);
    };
    load_chunk(nchunk - 1);
    float la0 = 0.f, la1 = 0.f;     // wave 0: log-decays of this chunk and the next
    if (w == 0) {
        la0 = gate(nchunk - 1);
        la1 = nchunk > 1 ? gate(nchunk - 2) : 0.f;
    }

    // R: rows 16 i + 4 g + r, column vcol(c) of this lane
    f32x4 R[TK][NC];
    auto vcol = [&](int c) {
        return tile_first<DV>(w * NC + c) + tile_step<DV>() * (n >> 2) + (n & 3);
    };
    const long hs = (long)DK * DV;
    const float *rstart = B.single ? P.dS_out : P.ws_rstate;
    if (rstart)
        rstart += B.single ? (B.slot * P.H + h) * hs : (b * P.H + h) * hs;
#pragma unroll
    for (int i = 0; i < TK; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                R[i][c][r] = rstart ? rstart[(16 * i + 4 * g + r) * DV + vcol(c)] : 0.f;

    for (int i = tid; i < C * PP; i += NT) {     // right of the diagonal: never written
        Ps[i] = from_f32<T>(0.f);
        Ys[i] = from_f32<T>(0.f);
    }
    if (w == 0)
        chunk_decays<C>(D[0], la0, lane);
    double gsum = 0.;               // wave 0: sum of the block's d log_alpha (this lane's)

    for (int step = 0; step < nchunk; ++step) {
        const int c = nchunk - 1 - step;
        const Decays<C> &dc = D[step & 1];
        const int cnt = B.count - c * C;
        qr.template store<PK>(Qs, tid);
        kr.template store<PK>(Ks, tid);
        vr.template store<PV>(Vs, tid);
        orr.template store<PV>(Os, tid);
#pragma unroll
        for (int i = 0; i < TK; ++i)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                const float f[4] = {R[i][cc][0], R[i][cc][1], R[i][cc][2], R[i][cc][3]};
                lds_stn<4>(Rs + vcol(cc) * PK + 16 * i + 4 * g, f);
            }
        FragV<T> sf[TR][DV / 32];
        {
            const FragV<T> *src = reinterpret_cast<const FragV<T> *>(
                static_cast<const T *>(P.ws_chunk) +
                (chunk_slot(b, B.first, c, C) * P.H + h) * hs);
#pragma unroll
            for (int t = 0; t < TR; ++t)
#pragma unroll
                for (int s = 0; s < DV / 32; ++s)
                    sf[t][s] = src[((w * TR + t) * (DV / 32) + s) * WAVE + lane];
        }
        __syncthreads();
        if (step + 1 < nchunk)
            load_chunk(c - 1);

        // 16 x 16 tiles of P and Y on and below the diagonal, and of X's sums
        for (int t = w; t < IT * (IT + 1) / 2; t += W) {
            int it = 0, jt = t;
            while (jt > it)
                jt -= ++it;
            const int i = 16 * it + n;
            f32x4 p = {0.f, 0.f, 0.f, 0.f}, y = p;
#pragma unroll
            for (int s = 0; s < DK / 32; ++s)
                mma(p, frag_row(Ks + (16 * jt + n) * PK + 32 * s + 8 * g),
                    frag_row(Qs + i * PK + 32 * s + 8 * g));
#pragma unroll
            for (int s = 0; s < DV / 32; ++s)
                mma(y, frag_row(Vs + (16 * jt + n) * PV + 32 * s + 8 * g),
                    frag_row(Os + i * PV + 32 * s + 8 * g));
            const float hi = dc.hi[i], lo = dc.lo[i];
            float pf[4], yf[4], row = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * jt + 4 * g + r;
                const float d = j <= i ? decay_between<T, C>(dc, hi, lo, j) : 0.f;
                pf[r] = j <= i ? p[r] * d : 0.f;
                yf[r] = j <= i ? y[r] * d : 0.f;
                // X without its diagonal, which no log-decay is between
                float x = j < i ? pf[r] * y[r] : 0.f;
                row += x;
                x = row16_sum_last(x);
                if (n == 15)
                    colx[it][j] = x;
            }
            lds_stn<4>(Ps + i * PP + 16 * jt + 4 * g, pf);
            lds_stn<4>(Ys + i * PP + 16 * jt + 4 * g, yf);
            row += __shfl_xor(row, 16, WAVE);
            row += __shfl_xor(row, 32, WAVE);
            if (g == 0)
                rowx[jt][i] = row;
        }

        // what comes from S and R, scaled to each token
        f32x4 aq[TR][IT], ak[TR][IT], av[NC][IT];
        float z = 0.f;
#pragma unroll
        for (int t = 0; t < TR; ++t) {
            const int c0 = tile_first<DK>(w * TR + t);
#pragma unroll
            for (int it = 0; it < IT; ++it) {
                aq[t][it] = f32x4{0.f, 0.f, 0.f, 0.f};
                ak[t][it] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
#pragma unroll
            for (int s = 0; s < DV / 32; ++s) {
                const FragV<T> rf = frag_cols_perm<PK>(Rs + 32 * s * PK, c0, tile_step<DK>(), lane);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    z += to_f32(sf[t][s][e]) * to_f32(rf[e]);
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    mma(aq[t][it], sf[t][s],
                        frag_row_perm(Os + (16 * it + n) * PV + 32 * s + 4 * g));
                    mma(ak[t][it], rf, frag_row_perm(Vs + (16 * it + n) * PV + 32 * s + 4 * g));
                }
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int i = 16 * it + n;
            const float in = dc.in[i], out = dc.out[i];
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int t = 0; t < TR; ++t) {
                const int c0 = tile_first<DK>(w * TR + t) + tile_step<DK>() * g;
                aq[t][it] *= in;
                ak[t][it] *= out;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x += aq[t][it][r] * to_f32(Qs[i * PK + c0 + r]);
                    y += ak[t][it][r] * to_f32(Ks[i * PK + c0 + r]);
                }
            }
            x += __shfl_xor(x, 16, WAVE);
            x += __shfl_xor(x, 32, WAVE);
            y += __shfl_xor(y, 16, WAVE);
            y += __shfl_xor(y, 32, WAVE);
            if (g == 0) {
                xs[w][i] = x;
                ys[w][i] = y;
            }
        }
        z = wave_sum(z);
        if (lane == 0)
            zs[w] = z;
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
#pragma unroll
            for (int it = 0; it < IT; ++it)
                av[cc][it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < DK / 32; ++s) {
                const FragV<T> rf = frag_acc<T>(R[2 * s][cc], R[2 * s + 1][cc]);
#pragma unroll
                for (int it = 0; it < IT; ++it)
                    mma(av[cc][it], rf, frag_row_perm(Ks + (16 * it + n) * PK + 32 * s + 4 * g));
            }
#pragma unroll
            for (int it = 0; it < IT; ++it)
                av[cc][it] *= dc.out[16 * it + n];
        }
        const float la = la0;       // wave 0: this chunk's log-decays
        if (w == 0) {
            if (step + 1 < nchunk)
                chunk_decays<C>(D[(step + 1) & 1], la1, lane);
            la0 = la1;
            la1 = step + 2 < nchunk ? gate(c - 2) : 0.f;
        }
        __syncthreads();            // P, Y and the sums

        if (w == 0 && P.dla) {
            const bool live = lane < C && lane < cnt;
            float u = 0.f, y = 0.f, zz = 0.f;
            if (live) {
                const int t = lane / 16;
                for (int j = 0; j <= t; ++j)
                    u += rowx[j][lane];
                for (int i = t; i < IT; ++i)
                    if (16 * i < cnt)
                        u -= colx[i][lane];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    u += xs[i][lane];
                    y += ys[i][lane];
                }
            }
#pragma unroll
            for (int i = 0; i < W; ++i)
                zz += zs[i];
            // suffix sums of u, prefix sums of y before the token
            float before = y;
#pragma unroll
            for (int off = 1; off < C; off <<= 1) {
                const float a = __shfl_down(u, off, WAVE), bb = __shfl_up(before, off, WAVE);
                if (lane + off < C)
                    u += a;
                if (lane >= off)
                    before += bb;
            }
            before -= y;
            float dg = u + before + dc.all * zz;
            if (log2_decay(la) <= (double)RESET2)
                dg = 0.f;           // a reset lets nothing past
            if (live) {
                if (dla)
                    dla[(B.first + (long)c * C + lane) * P.H + h] = from_f32<T>(dg);
                gsum += dg;
            }
        }

        // what comes from the chunk's own tokens, and R <- all R + q^T (in (.) do)
        const float all = dc.all;
#pragma unroll
        for (int i = 0; i < TK; ++i)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
                R[i][cc] *= all;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int t = 0; t < TR; ++t) {
                const int c0 = tile_first<DK>(w * TR + t);
                const FragV<T> kf = frag_cols<PK>(Ks + 32 * s * PK, c0, tile_step<DK>(), lane);
                const FragV<T> qf = frag_cols<PK>(Qs + 32 * s * PK, c0, tile_step<DK>(), lane);
#pragma unroll
                for (int it = 0; it < IT; ++it) {
                    if (it >= 2 * s)        // dq_i: j <= i
                        mma(aq[t][it], kf, frag_row(Ys + (16 * it + n) * PP + 32 * s + 8 * g));
                    if (it < 2 * s + 2)     // dk_j: i >= j
                        mma(ak[t][it], qf, frag_cols<PP>(Ys + 32 * s * PP, 16 * it, 4, lane));
                }
            }
            float wt[8];
            lds_ld8(dc.in + 32 * s + 8 * g, wt);
#pragma unroll
            for (int cc = 0; cc < NC; ++cc) {
                const FragV<T> of = frag_cols<PV>(Os + 32 * s * PV, tile_first<DV>(w * NC + cc),
                                                  tile_step<DV>(), lane);
#pragma unroll
                for (int it = 0; it < IT; ++it)
                    if (it < 2 * s + 2)
                        mma(av[cc][it], of, frag_cols<PP>(Ps + 32 * s * PP, 16 * it, 4, lane));
                const Split<T> os(of, wt);
#pragma unroll
                for (int i = 0; i < TK; ++i)
                    os.mma_a(R[i][cc], frag_cols<PK>(Qs + 32 * s * PK, 16 * i, 4, lane));
            }
        }
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int i = 16 * it + n;
            if (i < cnt) {
                const long t0 = (long)c * C + i;
#pragma unroll
                for (int t = 0; t < TR; ++t) {
                    const int c0 = tile_first<DK>(w * TR + t) + tile_step<DK>() * g;
                    store4<T>(P.dq, P.ws_dq, qat + t0 * qrow + c0, aq[t][it]);
                    store4<T>(P.dk_, P.ws_dk, kat + t0 * krow + c0, ak[t][it]);
                }
#pragma unroll
                for (int cc = 0; cc < NC; ++cc)
                    store4<T>(P.dv_, P.ws_dv,
                              vat + t0 * vrow + tile_first<DV>(w * NC + cc) + tile_step<DV>() * g,
                              av[cc][it]);
            }
        }
        __syncthreads();            // the chunk's tiles have been read
    }
    if (B.index == 0 && P.dS0) {
        float *dst = P.dS0 + (B.slot * P.H + h) * hs;
#pragma unroll
        for (int i = 0; i < TK; ++i)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    dst[(16 * i + 4 * g + r) * DV + vcol(c)] = R[i][c][r];
    }
    if (P.ws_dla && w == 0) {
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            gsum += __shfl_xor(gsum, off, WAVE);
        if (lane == 0)
            P.ws_dla[b * P.H + h] = gsum;
    }
}

// Rows behind the last sequence of a packed batch: zero gradients.
constexpr int TNT = 256;
template <typename T> __global__ __launch_bounds__(TNT) void linear_tail_kernel(LinearParams P) {
    const int nb = P.block_offsets[P.N];
    long end = 0;
    if (nb > 0 && nb <= P.nblocks) {
        const int4 r = reinterpret_cast<const int4 *>(P.blocks)[nb - 1];
        end = (long)r.x + r.y;
    }
    if (end < 0 || end >= P.tokens)
        return;
    const long rows = P.tokens - end, stride = (long)gridDim.x * TNT;
    const long id = (long)blockIdx.x * TNT + threadIdx.x;
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

// Gradient of a shared head: the sum over the states that read it, in order.
template <typename T>
__global__ __launch_bounds__(TNT) void linear_share_kernel(const float *part, T *out, long n,
                                                           int row, int d, int group) {
    // n: groups of 4 values of `out`; row: values of a token in `out`
    const long i = ((long)blockIdx.x * TNT + threadIdx.x) * 4;
    if (i >= n * 4)
        return;
    const long t = i / row;
    const int c = i % row, hh = c / d;
    const float *p = part + t * row * group + (long)hh * group * d + c % d;
    f32x4 x = *reinterpret_cast<const f32x4 *>(p);
    for (int j = 1; j < group; ++j)
        x += *reinterpret_cast<const f32x4 *>(p + (long)j * d);
    store4<T>(out, nullptr, i, x);
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
    if (lane == 0)
        static_cast<T *>(P.dla)[h] = from_f32<T>((float)x);
}

template <typename T>
static hipError_t share(const float *part, void *out, long tokens, int H, int heads, int d,
                        hipStream_t st) {
    const long n = tokens * heads * d / 4;
    if (!part || n == 0)
        return hipSuccess;
    hipLaunchKernelGGL(linear_share_kernel<T>, dim3((unsigned)((n + TNT - 1) / TNT)), dim3(TNT), 0,
                       st, part, static_cast<T *>(out), n, heads * d, d, H / heads);
    return hipGetLastError();
}

template <typename T> static hipError_t launch_grad(const LinearParams &P, hipStream_t st) {
    const long blocks = linear_total_blocks(P);
    hipError_t e = hipSuccess;
    if (blocks > 0) {
        const dim3 grid((unsigned)(blocks * P.H));
#define KDN_LGRAD(DK_, DV_)                                                                  \
        if (P.dk == DK_ && P.dv == DV_)                                                      \
            hipLaunchKernelGGL((linear_grad_kernel<T, DK_, DV_>), grid,                      \
                               dim3(GradShape<T, DK_, DV_>::NT), 0, st, P);
        KDN_LGRAD(64, 64)
        KDN_LGRAD(64, 128)
        KDN_LGRAD(128, 64)
        KDN_LGRAD(128, 128)
#undef KDN_LGRAD
        e = hipGetLastError();
    }
    if (e == hipSuccess && P.block_offsets && P.tokens > 0) {
        hipLaunchKernelGGL(linear_tail_kernel<T>, dim3(256), dim3(TNT), 0, st, P);
        e = hipGetLastError();
    }
    if (e == hipSuccess)
        e = share<T>(P.ws_dq, P.dq, P.tokens, P.H, P.Hq, P.dk, st);
    if (e == hipSuccess)
        e = share<T>(P.ws_dk, P.dk_, P.tokens, P.H, P.Hk, P.dk, st);
    if (e == hipSuccess)
        e = share<T>(P.ws_dv, P.dv_, P.tokens, P.H, P.Hv, P.dv, st);
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
    hipError_t e = hipSuccess;
    if (P.N > 0) {
        if (linear_total_blocks(P) > 0)
            e = launch_linear_states(P, st);
        if (e == hipSuccess)
            e = launch_linear_reverse_states(P, st);
        if (e == hipSuccess && linear_total_blocks(P) > 0)
            e = launch_linear_chunk_states(P, st);
    }
    if (e != hipSuccess)
        return e;
    return P.bf16 ? lin::launch_grad<bf16>(P, st) : lin::launch_grad<float>(P, st);
}

}  // namespace kdn
