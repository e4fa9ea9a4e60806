// kdn_norm.hip -- RMS norms around a block (gfx950), r(u) = (mean(u^2) + eps)^(-1/2):
// of a recurrence's outputs with their gate, each head by itself,
//   y = x r(x) w act(z)   or   u = x act(z), y = u r(u) w,
// and of the residual stream before the next block,
//   h = residual + scale x,   y = h r(h) w;
// with their gradients: for u, n = u r and t = dn w,
//   du = r (t - n mean(t n)),   dw = sum over rows of dn n.
// Bound by memory: every row is read and written once, from and to registers.
// A row is TPR threads (a power of two, as few as hold it in IT pieces of VEC
// elements each), so that short heads share a wave and long rows a workgroup.
// The sum of squares is kept in 64 bits: two instructions for each element, which
// memory hides, and no row of finite values is lost to an overflow.
//
// Measured: residual stream and norm of 16384 x 4096 (bf16, stream float32) 146 us,
// 5.5 TB/s; gradients of the gated norm of 262144 x 128 bf16 69 us, 4.9 TB/s, and the
// parts' sums 5 (calls: with the gate's kind and whole rows known to the compiler 69 us,
// whole rows alone 79, the kind alone 72, neither 85);
// of the residual norm of 2500 x 1543 bf16 20 us and 4, where rows start on no boundary
// and a row takes 256 threads of which 193 work; one token of 16 heads of 128 2 us of
// the call's 9, which binding and launch take.
#include "kdn_act.h"
#include "kdn_norm.h"

#include <type_traits>

namespace kdn {
namespace norm {

constexpr int NT = 256, NT_MAX = 1024;

// The value of the lane that CTRL names, in 64 bits.
template <int CTRL> __device__ __forceinline__ double dpp64(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xf, 0xf, true);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// x + that of the lane 16 (or 32) away.
template <bool FAR> __device__ __forceinline__ double swap64(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = (unsigned)b, hi = (unsigned)(b >> 32);
    const auto l = FAR ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false)
                       : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto h = FAR ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false)
                       : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    return __builtin_bit_cast(double, (uint64_t)h[0] << 32 | l[0]) +
           __builtin_bit_cast(double, (uint64_t)h[1] << 32 | l[1]);
}
// Sum over groups of tpr lanes (a power of two up to 64) within the registers; every
// lane gets it.  A mirror is as good as an exchange once the lanes of each half agree.
__device__ __forceinline__ double lane_sum(double x, int tpr) {
    if (tpr > 1)
        x += dpp64<0xB1>(x);             // the neighbour
    if (tpr > 2)
        x += dpp64<0x4E>(x);             // two away
    if (tpr > 4)
        x += dpp64<0x141>(x);            // the mirror of 8
    if (tpr > 8)
        x += dpp64<0x140>(x);            // the mirror of 16
    if (tpr > 16)
        x = swap64<false>(x);
    if (tpr > 32)
        x = swap64<true>(x);
    return x;
}

// Sums of N values over the TPR threads of a row; every thread gets them.  Rows of
// several waves meet in LDS, so that all threads of the workgroup have to come here;
// calls that follow each other take the two buffers in turn.
template <int N>
__device__ __forceinline__ void row_sums(double (&x)[N], int tpr, double (*lds)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
        x[n] = lane_sum(x[n], tpr);
    if (tpr <= WAVE)
        return;
    if ((threadIdx.x & (WAVE - 1)) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n)
            lds[threadIdx.x / WAVE][n] = x[n];
    __syncthreads();
    const int first = threadIdx.x / tpr * (tpr / WAVE);
#pragma unroll
    for (int n = 0; n < N; ++n)
        x[n] = lds[first][n];
    for (int i = 1; i < tpr / WAVE; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n)
            x[n] += lds[first + i][n];
}

// (m)^(-1/2) of a positive m in float32's range of roots: m is brought near 1 by
// an even power of two, for v_rsq_f32 (an ulp); float32 calls add a Newton step.
template <bool FINE> __device__ __forceinline__ float inv_sqrt(double m) {
    const int k = __builtin_amdgcn_frexp_exp(m) >> 1;
    const double s = __builtin_amdgcn_ldexp(m, -2 * k);
    float r = __builtin_amdgcn_rsqf((float)s);
    if constexpr (FINE) {
        const double y = r;
        if (r > 0.f && r < 3e38f)
            r = (float)(y * (1.5 - 0.5 * s * y * y));
    }
    return __builtin_amdgcn_ldexpf(r, -k);
}

template <bool FINE> __device__ __forceinline__ float act_f32(int act, float z) {
    if (act == KDN_ACT_NONE)
        return z;
    const float g = sigmoid_f32<FINE>(z);
    return act == KDN_ACT_SILU ? z * g : g;
}
template <bool FINE>
__device__ __forceinline__ void act_grad(int act, float z, float &y, float &dy) {
    float g, rest;
    if (act == KDN_ACT_NONE) {
        y = z;
        dy = 1.f;
        return;
    }
    sigmoid2<FINE>(z, g, rest);
    y = act == KDN_ACT_SILU ? z * g : g;
    dy = act == KDN_ACT_SILU ? fmaf(y, rest, g) : g * rest;
}

// Where a thread is: its row's slot in the workgroup, its first element of piece i.
struct Lane {
    int tpr, slot, lane;
    __device__ __forceinline__ Lane(int tpr_) : tpr(tpr_) {
        slot = threadIdx.x / tpr;
        lane = threadIdx.x % tpr;
    }
};

// Piece i of a thread: VEC elements of a row of d from `at` on, of which those from `skip`
// on are its own; none where `there` is false.  A row's last piece ends with the row and
// has elements of the piece before it in front (a load of fewer elements would be waited
// for at once); a row shorter than a piece is loaded by its elements.  FULL: rows are
// whole pieces.
template <int VEC, bool FULL> struct Piece {
    int at, skip, n;
    bool there, whole;
    __device__ __forceinline__ Piece(const Lane &L, int i, int d) {
        at = (i * L.tpr + L.lane) * VEC;
        skip = 0;
        there = at < d;
        n = VEC;
        whole = true;
        if constexpr (!FULL) {
            if (there && at + VEC > d) {
                n = d - at;
                whole = d >= VEC;
                skip = whole ? VEC - n : 0;
                at = whole ? d - VEC : at;
            }
        }
    }
    __device__ __forceinline__ bool own(int e) const { return FULL || e >= skip; }
    template <typename T> __device__ __forceinline__ void load(Pack<T, VEC> &v, const T *row) const {
        if (FULL || whole)
            v.load(row + at);
        else
            v.load(row + at, n);
    }
    template <typename T> __device__ __forceinline__ void store(const Pack<T, VEC> &v, T *row) const {
        if (FULL || n == VEC) {
            v.store(row + at);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (e >= skip && e < skip + n)
                    row[at + e] = v.r[e];
        }
    }
};

// What a gated norm's kernel knows of its gate: silu in either order, or nothing
// (gradients of 262144 x 128: 69 us where it knows, 79 where it asks; with a sigmoid, for
// which it asks, 75, without a gate 43).
enum Kind { NORM_SILU, SILU_NORM, ANY };
template <Kind KIND> struct Gate {
    bool there, first;
    int act;
    __device__ __forceinline__ Gate(const GatedNormParams &P)
        : there(KIND != ANY || P.z), first(KIND == ANY ? P.z && P.gate_first : KIND == SILU_NORM),
          act(KIND == ANY ? P.act : (int)KDN_ACT_SILU) {}
};

template <typename T, int VEC, int IT, bool FULL, Kind KIND>
__global__ __launch_bounds__(NT_MAX) void gated_norm_kernel(GatedNormParams P, int tpr) {
    constexpr bool FINE = sizeof(T) == 4;
    __shared__ double lds[NT_MAX / WAVE][1];
    const Lane L(tpr);
    const Gate<KIND> gate(P);
    const long row = (long)blockIdx.x * (blockDim.x / tpr) + L.slot, rows = P.tokens * P.H;
    const bool in = row < rows;
    const unsigned at_row = in ? (unsigned)row : 0u, t = at_row / (unsigned)P.H, h = at_row - t * P.H;
    const T *x = static_cast<const T *>(P.x) + t * P.x_stride + (long)h * P.d;
    const T *z = static_cast<const T *>(P.z) + t * P.z_stride + (long)h * P.d;
    const float *w = P.weight + (P.per_head ? (long)h * P.d : 0);
    Pack<T, VEC> xs[IT], zs[IT];
    Pack<float, VEC> ws[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.d);
        xs[i].zero();
        zs[i].zero();
        ws[i].zero();
        if (in && piece.there) {
            piece.load(xs[i], x);
            if (gate.there)
                piece.load(zs[i], z);
            piece.load(ws[i], w);
        }
    }
    float u[IT][VEC];
    double sum[1] = {0.};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            u[i][e] = xs[i].get(e);
            if (gate.first)
                u[i][e] *= act_f32<FINE>(gate.act, zs[i].get(e));
            const float own = piece.own(e) ? u[i][e] : 0.f;
            sum[0] = fma((double)own, (double)own, sum[0]);
        }
    }
    row_sums(sum, tpr, lds);
    const float r = inv_sqrt<FINE>(sum[0] * P.inv_d + (double)P.eps);
    T *y = static_cast<T *>(P.y) + row * P.d;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        Pack<T, VEC> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float v = u[i][e] * r * ws[i].get(e);
            if (gate.there && !gate.first)
                v *= act_f32<FINE>(gate.act, zs[i].get(e));
            out.set(e, v);
        }
        const Piece<VEC, FULL> piece(L, i, P.d);
        if (in && piece.there)
            piece.store(out, y);
    }
}

// A workgroup's sums of the values of each column over its rows, in the order of the
// rows' slots, into out[column].
template <int VEC, int IT, bool FULL>
__device__ __forceinline__ void column_sums(const float (&v)[IT][VEC], const Lane &L, int d,
                                            float *lds, float *out) {
    const int slots = blockDim.x / L.tpr;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = v[i][e];
            if (slots > 1) {
                __syncthreads();
                lds[threadIdx.x] = s;
                __syncthreads();
                if (L.slot == 0)
                    for (int q = 1; q < slots; ++q)
                        s += lds[q * L.tpr + L.lane];
            }
            if (L.slot == 0 && piece.there && piece.own(e) && piece.at + e < d)
                out[piece.at + e] = s;
        }
    }
}

template <typename T, int VEC, int IT, bool FULL, Kind KIND>
__global__ __launch_bounds__(NT_MAX) void gated_norm_grad_kernel(GatedNormParams P, int tpr) {
    constexpr bool FINE = sizeof(T) == 4;
    __shared__ double lds[2][NT_MAX / WAVE][2];
    __shared__ float cols[NT_MAX];
    const Lane L(tpr);
    const Gate<KIND> gate(P);
    const int slots = blockDim.x / tpr;
    // weight by head: a workgroup has one head's rows; else rows of all heads
    const unsigned head = P.per_head ? blockIdx.y : 0, heads = P.per_head ? 1 : P.H;
    const unsigned rows = (unsigned)(P.tokens * heads), step = (unsigned)P.parts * slots;
    const float *w = P.weight + (long)head * P.d;
    Pack<float, VEC> ws[IT];
    float dw[IT][VEC];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.d);
        ws[i].zero();
        if (piece.there)
            piece.load(ws[i], w);
    }
    // the row's token and head, and the steps of both (a division once a row would cost a
    // tenth of the row's work)
    unsigned row = blockIdx.x * slots + L.slot, t = row / heads, h = row - t * heads;
    const unsigned dt = step / heads, dh = step - dt * heads;
    int buf = 0;
    long first = (long)blockIdx.x * slots;
    for (int seg = 0; seg < P.segs; ++seg) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                dw[i][e] = 0.f;
        // the same number of rounds for every thread: they meet in row_sums
        for (int k = 0; k < P.seg_rounds && first < rows; ++k, first += step, buf ^= 1) {
            const bool in = row < rows;
            const T *x = static_cast<const T *>(P.x) + t * P.x_stride + (long)(head + h) * P.d;
            const T *z = static_cast<const T *>(P.z) + t * P.z_stride + (long)(head + h) * P.d;
            const long out = ((long)t * P.H + head + h) * P.d;
            const T *dy = static_cast<const T *>(P.d_y) + out;
            Pack<T, VEC> xs[IT], zs[IT], gs[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const Piece<VEC, FULL> piece(L, i, P.d);
                xs[i].zero();
                zs[i].zero();
                gs[i].zero();
                if (in && piece.there) {
                    piece.load(xs[i], x);
                    piece.load(gs[i], dy);
                    if (gate.there)
                        piece.load(zs[i], z);
                }
            }
            double sums[2] = {0., 0.};       // of u^2 and of t u
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const Piece<VEC, FULL> piece(L, i, P.d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float u = xs[i].get(e), dn = gs[i].get(e);
                    if (gate.there) {
                        const float a = act_f32<FINE>(gate.act, zs[i].get(e));
                        u = gate.first ? u * a : u;
                        dn = gate.first ? dn : dn * a;
                    }
                    u = piece.own(e) ? u : 0.f;
                    dn = piece.own(e) ? dn * ws[i].get(e) : 0.f;
                    sums[0] = fma((double)u, (double)u, sums[0]);
                    sums[1] = fma((double)dn, (double)u, sums[1]);
                }
            }
            row_sums(sums, tpr, lds[buf]);
            const float r = inv_sqrt<FINE>(sums[0] * P.inv_d + (double)P.eps);
            // mean(t n)
            const float m = (float)(sums[1] * (double)r * P.inv_d);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                Pack<T, VEC> dx, dz;
                const Piece<VEC, FULL> piece(L, i, P.d);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xe = xs[i].get(e), ge = gs[i].get(e), we = ws[i].get(e);
                    float a = 1.f, da = 0.f;
                    if (gate.there)
                        act_grad<FINE>(gate.act, zs[i].get(e), a, da);
                    const float n = (gate.first ? xe * a : xe) * r;
                    const float dn = gate.first ? ge : ge * a;
                    const float du = r * (dn * we - n * m);
                    // (what lies behind the rows and the row is zero; a piece's elements that are not
                    // its own are left out of the columns' sums)
                    dw[i][e] = fmaf(dn, n, dw[i][e]);
                    dx.set(e, gate.first ? du * a : du);
                    dz.set(e, gate.first ? du * xe * da : ge * n * we * da);
                }
                if (in && piece.there) {
                    piece.store(dx, static_cast<T *>(P.dx) + out);
                    if (gate.there)
                        piece.store(dz, static_cast<T *>(P.dz) + out);
                }
            }
            row += step;
            t += dt;
            h += dh;
            if (h >= heads) {
                h -= heads;
                ++t;
            }
        }
        column_sums<VEC, IT, FULL>(dw, L, P.d, cols,
                             P.ws + (((long)blockIdx.x * P.segs + seg) * gridDim.y + head) * P.d);
    }
}

template <typename T, typename S, int VEC, int IT, bool FULL>
__global__ __launch_bounds__(NT_MAX) void residual_norm_kernel(ResidualNormParams P, int tpr) {
    constexpr bool FINE = sizeof(T) == 4;
    __shared__ double lds[NT_MAX / WAVE][1];
    const Lane L(tpr);
    const long row = (long)blockIdx.x * (blockDim.x / tpr) + L.slot;
    const bool in = row < P.tokens;
    const T *x = static_cast<const T *>(P.x) + (in ? row : 0) * P.x_stride;
    const S *res = static_cast<const S *>(P.residual) + (in ? row : 0) * P.r_stride;
    Pack<T, VEC> xs[IT];
    Pack<S, VEC> rs[IT];
    Pack<float, VEC> ws[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.D);
        xs[i].zero();
        rs[i].zero();
        ws[i].zero();
        if (in && piece.there) {
            piece.load(xs[i], x);
            piece.load(rs[i], res);
            piece.load(ws[i], P.weight);
        }
    }
    float h[IT][VEC];
    double sum[1] = {0.};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.D);
        Pack<float, VEC> sc;
        sc.zero();
        if (P.scale_n > 1 && piece.there)
            piece.load(sc, P.scale);
        Pack<S, VEC> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float s = P.scale_n == 0 ? 1.f : (P.scale_n == 1 ? P.scale[0] : sc.get(e));
            h[i][e] = fmaf(s, xs[i].get(e), rs[i].get(e));
            const float own = piece.own(e) ? h[i][e] : 0.f;
            sum[0] = fma((double)own, (double)own, sum[0]);
            out.set(e, h[i][e]);
        }
        if (in && piece.there)
            piece.store(out, static_cast<S *>(P.h) + row * P.D);
    }
    row_sums(sum, tpr, lds);
    const float r = inv_sqrt<FINE>(sum[0] * P.inv_d + (double)P.eps);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.D);
        Pack<T, VEC> out;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            out.set(e, h[i][e] * r * ws[i].get(e));
        if (in && piece.there)
            piece.store(out, static_cast<T *>(P.y) + row * P.D);
    }
}

template <typename T, typename S, int VEC, int IT, bool FULL>
__global__ __launch_bounds__(NT_MAX) void residual_norm_grad_kernel(ResidualNormParams P, int tpr) {
    constexpr bool FINE = sizeof(T) == 4;
    __shared__ double lds[2][NT_MAX / WAVE][2];
    __shared__ float cols[NT_MAX];
    const Lane L(tpr);
    const int slots = blockDim.x / tpr;
    Pack<float, VEC> ws[IT], sc[IT];
    float dw[IT][VEC], ds[IT][VEC];
    const float one = P.scale_n == 1 ? P.scale[0] : 1.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.D);
        ws[i].zero();
        sc[i].zero();
        if (piece.there) {
            piece.load(ws[i], P.weight);
            if (P.scale_n > 1)
                piece.load(sc[i], P.scale);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            dw[i][e] = ds[i][e] = 0.f;
    }
    // a row's values, requested while the row before is worked on
    Pack<S, VEC> h1[IT], dh1[IT];
    Pack<T, VEC> g1[IT], x1[IT];
    auto load = [&](long row) {
        const bool in = row < P.tokens;
        const S *hrow = static_cast<const S *>(P.residual) + (in ? row : 0) * P.r_stride;
        const T *x = static_cast<const T *>(P.x) + (in ? row : 0) * P.x_stride;
        const long out = (in ? row : 0) * P.D;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const Piece<VEC, FULL> piece(L, i, P.D);
            h1[i].zero();
            dh1[i].zero();
            g1[i].zero();
            x1[i].zero();
            if (in && piece.there) {
                piece.load(h1[i], hrow);
                piece.load(g1[i], static_cast<const T *>(P.d_y) + out);
                if (P.d_h)
                    piece.load(dh1[i], static_cast<const S *>(P.d_h) + out);
                if (P.dscale)
                    piece.load(x1[i], x);
            }
        }
    };
    load((long)blockIdx.x * slots + L.slot);
    int buf = 0;
    for (long first = (long)blockIdx.x * slots; first < P.tokens;
         first += (long)P.parts * slots, buf ^= 1) {
        const long row = first + L.slot;
        const bool in = row < P.tokens;
        const long out = (in ? row : 0) * P.D;
        Pack<S, VEC> hs[IT], dh[IT];
        Pack<T, VEC> gs[IT], xs[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            hs[i] = h1[i];
            dh[i] = dh1[i];
            gs[i] = g1[i];
            xs[i] = x1[i];
        }
        load(row + (long)P.parts * slots);
        double sums[2] = {0., 0.};       // of u^2 and of t u
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const Piece<VEC, FULL> piece(L, i, P.D);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const double u = piece.own(e) ? hs[i].get(e) : 0.f;
                const float t = piece.own(e) ? gs[i].get(e) * ws[i].get(e) : 0.f;
                sums[0] = fma(u, u, sums[0]);
                sums[1] = fma((double)t, u, sums[1]);
            }
        }
        row_sums(sums, tpr, lds[buf]);
        const float r = inv_sqrt<FINE>(sums[0] * P.inv_d + (double)P.eps);
        const float m = (float)(sums[1] * (double)r * P.inv_d);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            Pack<S, VEC> dres;
            Pack<T, VEC> dx;
            const Piece<VEC, FULL> piece(L, i, P.D);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float g = gs[i].get(e), n = hs[i].get(e) * r;
                const float d = fmaf(r, g * ws[i].get(e) - n * m, dh[i].get(e));
                dw[i][e] = fmaf(g, n, dw[i][e]);
                ds[i][e] = fmaf(d, xs[i].get(e), ds[i][e]);
                dres.set(e, d);
                dx.set(e, d * (P.scale_n > 1 ? sc[i].get(e) : one));
            }
            if (in && piece.there) {
                piece.store(dres, static_cast<S *>(P.dresidual) + out);
                if (P.dx)
                    piece.store(dx, static_cast<T *>(P.dx) + out);
            }
        }
    }
    column_sums<VEC, IT, FULL>(dw, L, P.D, cols, P.ws + (long)blockIdx.x * P.D);
    if (!P.dscale)
        return;
    float *part = P.ws_scale;
    if (P.scale_n > 1) {
        column_sums<VEC, IT, FULL>(ds, L, P.D, cols, part + (long)blockIdx.x * P.D);
        return;
    }
    // one scale: its sum over the workgroup's columns and rows
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const Piece<VEC, FULL> piece(L, i, P.D);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            s += piece.own(e) ? ds[i][e] : 0.f;
    }
    __syncthreads();
    cols[threadIdx.x] = s;
    __syncthreads();
    for (int n = blockDim.x / 2; n >= 1; n >>= 1) {
        if ((int)threadIdx.x < n)
            cols[threadIdx.x] += cols[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        part[blockIdx.x] = cols[0];
}

// out[c] = sum over parts of ws[part][c], 16 columns a workgroup.  Two arrays in one
// launch: those of ws2 behind those of ws.
struct Sums {
    const float *ws, *ws2;
    float *out, *out2;
    long n, n2;
    int parts;
};
__global__ __launch_bounds__(NT_MAX) void sum_parts_kernel(Sums S) {
    __shared__ double lds[NT_MAX / WAVE][16];
    const long wide = (S.n + 15) / 16;
    const bool second = blockIdx.x >= wide;
    const long n = second ? S.n2 : S.n, first = ((long)blockIdx.x - (second ? wide : 0)) * 16;
    const double s = part_sums<NT_MAX>(second ? S.ws2 : S.ws, n, S.parts, first, lds);
    if (threadIdx.x < 16 && first + threadIdx.x < n)
        (second ? S.out2 : S.out)[first + threadIdx.x] = (float)s;
}

hipError_t sum_parts(const Sums &S, hipStream_t st) {
    const long wgs = (S.n + 15) / 16 + (S.n2 + 15) / 16;
    if (wgs == 0)
        return hipSuccess;
    hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)wgs), dim3(NT_MAX), 0, st, S);
    return hipGetLastError();
}

}  // namespace norm

// FN(IT) for a row of `width` elements in pieces of V.
#define KDN_NORM_IT(FN, width)                                                         \
    {                                                                                  \
        const int pieces = (width + V - 1) / V, tpr = norm_row_threads(width, V == 8);\
        const int threads = tpr < norm::NT ? norm::NT : tpr;                           \
        const int it = (pieces + tpr - 1) / tpr;                                       \
        if (it <= 1)                                                                   \
            FN(1)                                                                      \
        if (it <= 2)                                                                   \
            FN(2)                                                                      \
        if constexpr (V < 8)                                                           \
            FN(4)                                                                      \
    }

// Rounds of a segment: `step` rows a round for all workgroups together.
static int seg_rounds(long rows, long step, int segs) {
    const long rounds = (rows + step - 1) / step;
    return (int)((rounds + segs - 1) / segs);
}

template <typename T, bool FULL, norm::Kind KIND>
static hipError_t gated_norm_k(const GatedNormParams &P, hipStream_t st, bool back) {
    constexpr int V = 16 / sizeof(T);
#define KDN_GATED(IT_)                                                                      \
    {                                                                                           \
        const long slots = threads / tpr, rows = P.tokens * P.H;                                \
        const dim3 grid = back ? dim3((unsigned)P.parts, P.per_head ? P.H : 1)                  \
                               : dim3((unsigned)((rows + slots - 1) / slots));                  \
        GatedNormParams Q = P;                                                                  \
        if (back)                                                                               \
            Q.seg_rounds = seg_rounds(P.per_head ? P.tokens : rows, P.parts * slots, P.segs);   \
        auto kernel = back ? norm::gated_norm_grad_kernel<T, V, IT_, FULL, KIND>                \
                           : norm::gated_norm_kernel<T, V, IT_, FULL, KIND>;                    \
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, Q, tpr);                         \
        return hipGetLastError();                                                               \
    }
    KDN_NORM_IT(KDN_GATED, P.d)
#undef KDN_GATED
    return hipErrorInvalidValue;
}

template <typename T, typename S, bool FULL>
static hipError_t residual_norm_k(const ResidualNormParams &P, hipStream_t st, bool back) {
    constexpr int V = 16 / sizeof(T);
#define KDN_RESIDUAL(IT_)                                                                   \
    {                                                                                           \
        /* gradients: wider workgroups, so that there are fewer parts to write and to add */ \
        const int wide = back && threads < 512 ? 512 : threads;                                 \
        const long slots = wide / tpr;                                                          \
        const dim3 grid((unsigned)(back ? P.parts : (P.tokens + slots - 1) / slots));           \
        auto kernel = back ? norm::residual_norm_grad_kernel<T, S, V, IT_, FULL>                \
                           : norm::residual_norm_kernel<T, S, V, IT_, FULL>;                    \
        hipLaunchKernelGGL(kernel, grid, dim3(wide), 0, st, P, tpr);                         \
        return hipGetLastError();                                                               \
    }
    KDN_NORM_IT(KDN_RESIDUAL, P.D)
#undef KDN_RESIDUAL
    return hipErrorInvalidValue;
}
#undef KDN_NORM_IT

template <typename T, bool FULL>
static hipError_t gated_norm_f(const GatedNormParams &P, hipStream_t st, bool back) {
    if (!P.z || P.act != KDN_ACT_SILU)
        return gated_norm_k<T, FULL, norm::ANY>(P, st, back);
    return P.gate_first ? gated_norm_k<T, FULL, norm::SILU_NORM>(P, st, back)
                        : gated_norm_k<T, FULL, norm::NORM_SILU>(P, st, back);
}
template <typename T>
static hipError_t gated_norm_t(const GatedNormParams &P, hipStream_t st, bool back) {
    return P.d % (16 / sizeof(T)) == 0 ? gated_norm_f<T, true>(P, st, back)
                                       : gated_norm_f<T, false>(P, st, back);
}
template <typename T, typename S>
static hipError_t residual_norm_t(const ResidualNormParams &P, hipStream_t st, bool back) {
    return P.D % (16 / sizeof(T)) == 0 ? residual_norm_k<T, S, true>(P, st, back)
                                       : residual_norm_k<T, S, false>(P, st, back);
}

hipError_t launch_gated_norm(const GatedNormParams &P, hipStream_t st) {
    if (P.tokens * P.H * P.d == 0)
        return hipSuccess;
    return P.bf16 ? gated_norm_t<bf16>(P, st, false) : gated_norm_t<float>(P, st, false);
}

hipError_t launch_gated_norm_backward(const GatedNormParams &P, hipStream_t st) {
    if (P.parts > 0) {
        const hipError_t e = P.bf16 ? gated_norm_t<bf16>(P, st, true) : gated_norm_t<float>(P, st, true);
        if (e != hipSuccess)
            return e;
    }
    const long n = (long)(P.per_head ? P.H : 1) * P.d;
    return norm::sum_parts(norm::Sums{P.ws, nullptr, P.dweight, nullptr, n, 0, P.parts * P.segs}, st);
}

static hipError_t residual(const ResidualNormParams &P, hipStream_t st, bool back) {
    if (P.bf16)
        return P.stream_bf16 ? residual_norm_t<bf16, bf16>(P, st, back)
                             : residual_norm_t<bf16, float>(P, st, back);
    return residual_norm_t<float, float>(P, st, back);
}

hipError_t launch_residual_norm(const ResidualNormParams &P, hipStream_t st) {
    return P.tokens * P.D == 0 ? hipSuccess : residual(P, st, false);
}

// Rows `first` .. + tokens of a call.
static ResidualNormParams rows_of(const ResidualNormParams &P, long first, long tokens) {
    ResidualNormParams Q = P;
    const long es = P.bf16 ? 2 : 4, rs = P.stream_bf16 ? 2 : 4;
    auto at = [](auto *p, long bytes) {
        typedef std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(p)>>, const char, char> Byte;
        return p ? static_cast<decltype(p)>(static_cast<Byte *>(p) + bytes) : p;
    };
    Q.tokens = tokens;
    Q.x = at(P.x, first * P.x_stride * es);
    Q.residual = at(P.residual, first * P.r_stride * rs);
    Q.d_y = at(P.d_y, first * P.D * es);
    Q.d_h = at(P.d_h, first * P.D * rs);
    Q.dx = at(P.dx, first * P.D * es);
    Q.dresidual = at(P.dresidual, first * P.D * rs);
    return Q;
}

hipError_t launch_residual_norm_backward(const ResidualNormParams &P, hipStream_t st) {
    if (P.D == 0)
        return hipSuccess;
    const long parts = (long)P.parts * P.segs, n_scale = P.dscale ? P.scale_n : 0;
    float *scales = P.ws + parts * P.D;
    const long rows = parts > 0 ? (P.tokens + P.segs - 1) / P.segs : 0;
    for (int seg = 0; parts > 0 && seg < P.segs; ++seg) {
        const long first = min(seg * rows, P.tokens);
        ResidualNormParams Q = rows_of(P, first, min(rows, P.tokens - first));
        Q.ws = P.ws + seg * P.parts * (long)P.D;
        Q.ws_scale = scales + seg * P.parts * n_scale;
        const hipError_t e = residual(Q, st, true);
        if (e != hipSuccess)
            return e;
    }
    return norm::sum_parts(norm::Sums{P.ws, scales, P.dweight, P.dscale, P.D, n_scale, (int)parts}, st);
}

}  // namespace kdn
