// kdn_scan_backward.hip -- gradients of the selective scan (gfx950).  With p_t = C_t .
// h_t + D x_t, dp_t = dy_t silu(z_t) and the reverse recurrence from dS
//     g_t = R_t + dp_t C_t,   R_{t-1} = a_t g_t   (a_t = exp(dt_t A)),
// and w_t = R_{t-1} h_{t-1}:
//     dx = D dp + dt sum_n g B,        ddt = sum_n w A + x sum_n g B,
//     dA = sum_t w dt,                 dB = sum_c dt x g,      dC = sum_c dp h,
//     dD = sum_t dp x,  dz = dy p silu'(z),  ddelta = ddt sigmoid(delta + bias).
// The states of both recurrences at every tile's ends come from the tiles' own
// contributions and their joins (kdn_scan.hip).  A workgroup then takes a tile, its
// waves K tokens each, and for each of its runs of 16 channels scans both ways as the
// outputs do: every wave its tokens from nothing, a fold through LDS, and again with
// the decays and the states in registers.  Bound by the vector units: 18 instructions'
// time for each token, channel and state, an exponential's two among them (140 us for
// B2 T4096, 2048 channels, 16 states), and as much again for B and C from LDS, the
// exchanges between lanes and the tokens' own functions.  That call, bf16: 353 us; traced,
// one by one, 89 + 17 + 290 + 8, of which this kernel is the 290, with 82 % of the vector
// units' time, two waves a SIMD by their registers; the call moves 608 MB, where its inputs and gradients are 236.  Softplus, the gate and their slopes are
// made once, in front, and take fewer registers than the inputs that they replace (made
// again behind the scans: 323 us, with 20 registers spilled).
// dB and dC are sums over channels: a lane adds those of its runs in registers, so
// that only their sum goes through the exchanges between lanes, once for each set of
// runs; the sets' sums are added by another kernel.
#include "kdn_scan_device.h"

namespace kdn {
namespace scan {

// Tokens of a wave, and waves: registers hold two values and two sums for each state
// and token.
template <int SPL> constexpr int grad_steps() { return SPL <= 4 ? 8 : 4; }
template <int SPL> constexpr int grad_waves() { return scan_tile(4 * SPL) / grad_steps<SPL>(); }

// A wave's tokens of one run of channels, requested while it works on another.
template <typename T, int K> struct Run {
    T x[K / 4], d[K / 4], z[K / 4], g[K / 4];
    __device__ __forceinline__ void load(const ScanParams &P, const Channels &ch, long first,
                                         int count) {
        // the rows' offsets are made again for every run: kept over the runs they would
        // not fit the registers, and a reload waits for all loads before it
        int j = threadIdx.x & 3;
        asm volatile("" : "+v"(j));
        const Rows<T, K> rx(P.x, first, P.x_stride, P.C, count);
        const Rows<T, K> rd(P.delta, first, P.d_stride, P.C, count);
        const Rows<T, K> rz(P.z, first, P.z_stride, P.C, P.z ? count : 0);
        const Rows<T, K> rg(P.d_y, first, P.C, P.C, count);
#pragma unroll
        for (int i = 0; i < K / 4; ++i) {
            // lanes behind the last channel: x = dy = 0, nothing of them in dB and dC
            const int t = 4 * i + j;
            x[i] = rx.load(rx.at(t, P.x_stride, ch.c, ch.live));
            d[i] = rd.load(rd.at(t, P.d_stride, ch.c, ch.live));
            z[i] = rz.load(rz.at(t, P.z_stride, ch.c, ch.live));
            g[i] = rg.load(rg.at(t, P.C, ch.c, ch.live));
        }
    }
};

__device__ __forceinline__ float swap_add(float a, float b, bool half) {
    const auto p = half ? __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false)
                        : __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Sums over the 16 channels of a wave of M = 16 V values f: lane 4 k + j gets in v the
// sums over lanes j of f[V x .. + V], x = 4 (k & 3) + 2 ((k >> 2) & 1) + (k >> 3).  Two
// steps swap halves of registers (each leaves half as many), two add within 16 lanes.
template <int V>
__device__ __forceinline__ void channel_sums(const float (&f)[16 * V], float (&v)[V]) {
    float a[8 * V], b[4 * V];
#pragma unroll
    for (int m = 0; m < 8 * V; ++m) {
        // places 2 m and 2 m + 1 of the order 4 V q + 4 i + e, f index V (4 q + e) + i
        const int p0 = 2 * m, p1 = p0 + 1;
        const int f0 = V * (4 * (p0 / (4 * V)) + p0 % 4) + p0 % (4 * V) / 4;
        const int f1 = V * (4 * (p1 / (4 * V)) + p1 % 4) + p1 % (4 * V) / 4;
        a[m] = swap_add(f[f0], f[f1], true);
    }
#pragma unroll
    for (int m = 0; m < 4 * V; ++m) {
        b[m] = swap_add(a[2 * m], a[2 * m + 1], false);
        b[m] += dpp<0x128>(b[m]);            // row_ror:8
        b[m] += dpp<0x124>(b[m]);            // row_ror:4
    }
    const int q = (threadIdx.x >> 2) & 3;
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = q & 2 ? (q & 1 ? b[3 * V + i] : b[2 * V + i]) : (q & 1 ? b[V + i] : b[i]);
}

template <typename T, int SPL>
__global__ __launch_bounds__(grad_waves<SPL>() * WAVE, 2) void scan_grad_kernel(ScanParams P,
                                                                              int groups,
                                                                              int sets,
                                                                              long blocks) {
    constexpr bool FINE = sizeof(T) == 4;
    constexpr int S = 4 * SPL, K = grad_steps<SPL>(), NW = grad_waves<SPL>(), TILE = NW * K;
    constexpr int M = 2 * K * SPL, V = M / 16;     // sums of a lane, and after the exchange
    __shared__ float bc[NW][2][K][S];
    // each wave's decay, and its ends of both recurrences from nothing, which the fold
    // makes the states in front of its tokens and behind them
    __shared__ float ends[3][NW][WAVE * SPL];
    constexpr int ITEMS = 2 * WAVE * SPL / NW, ROUNDS = (ITEMS + WAVE - 1) / WAVE;
    __shared__ float sum_A[scan_per_set(S)][NW][WAVE * SPL];
    __shared__ float sum_D[scan_per_set(S)][2][NW][SCAN_CHANNELS];
    __shared__ float par_A[scan_per_set(S)][WAVE * SPL], par[scan_per_set(S)][2][SCAN_CHANNELS];
    const int lane = threadIdx.x & (WAVE - 1), j = lane & 3, w = wave_id();
    const int set = blockIdx.x % sets, g = (int)(blockIdx.x / sets) % P.G;
    const int part = (int)(blockIdx.x / sets) / P.G;
    const int run0 = set * P.per_set, runs = min(P.per_set, groups - run0), per = P.C / P.G;
    for (int k = 0; k < runs; ++k) {         // a wave's own place: no barrier
        const float zero[SPL] = {};
        store_states<SPL>(&sum_A[k][w][lane * SPL], zero);
        sum_D[k][j & 1][w][lane >> 2] = 0.f;
        if (k % NW == w) {                   // A, delta's bias and D, for all waves
            const Channels ch(P, g * groups + run0 + k, groups);
            float A2[SPL];
            load_A<SPL>(P, ch.c, j, A2);
            store_states<SPL>(&par_A[k][lane * SPL], A2);
            const float *from = j & 1 ? P.D : P.bias;
            par[k][j & 1][lane >> 2] = from ? from[ch.c] : 0.f;
        }
    }
    __syncthreads();
    for (long u = part; u < blocks * P.classes; u += P.parts) {
        const long b = u / P.classes;
        const Block B = get_block(P, b);
        for (int t1 = (int)(u % P.classes) * TILE; t1 < B.count; t1 += P.classes * TILE) {
            const int count = B.count - t1 - w * K;          // of the wave's tokens
            const long first = B.first + t1 + w * K;
            float *rows_bc = P.ws_bc + ((set * P.tokens + first) * P.G + g) * (2 * S);
            float acc[M];
#pragma unroll
            for (int i = 0; i < M; ++i)
                acc[i] = 0.f;
            if (B.slot < 0) {
                // a skipped sequence has no gradients
                for (int k = 0; k < runs; ++k) {
                    const Channels ch(P, g * groups + run0 + k, groups);
                    for (int t = j; t < min(K, count); t += 4)
                        if (ch.live) {
                            const long at = (first + t) * P.C + ch.c;
                            static_cast<T *>(P.dx)[at] = from_f32<T>(0.f);
                            static_cast<T *>(P.ddelta)[at] = from_f32<T>(0.f);
                            if (P.z)
                                static_cast<T *>(P.dz)[at] = from_f32<T>(0.f);
                        }
                }
            } else {
                const long slot = tile_slot(b, B.first, t1 / TILE, S);
                GroupRows<T, S, K> group;
                Run<T, K> next;
                group.load(P, g, first, count);
                next.load(P, Channels(P, g * groups + run0, groups), first, count);
                group.put(bc[w]);
                for (int k = 0; k < runs; ++k) {
                    const Channels ch(P, g * groups + run0 + k, groups);
                    const Run<T, K> now = next;
                    float A2[SPL], hs[SPL], r[SPL];
                    // the tile's states that this lane folds: its waves have 1 / NW of
                    // the run's 16 S each, forward ones and then reverse ones
                    float state[ROUNDS];
                    const long run_at = (slot * P.C + (long)g * per + (run0 + k) * SCAN_CHANNELS) * S;
#pragma unroll
                    for (int n = 0; n < ROUNDS; ++n) {
                        int it = lane + n * WAVE;
                        if constexpr (SPL == 4)
                            asm volatile("" : "+v"(it));
                        const int e = w * (ITEMS / 2) + it % (ITEMS / 2);
                        const int behind = (per - (run0 + k) * SCAN_CHANNELS) * S - 1;
                        state[n] = 0.f;
                        if (it < ITEMS)
                            state[n] = (it < ITEMS / 2 ? P.ws_state : P.ws_rstate)[run_at + min(e, behind)];
                    }
                    // behind the last run nothing is read, but without a branch, behind
                    // which all loads would be waited for
                    next.load(P, Channels(P, g * groups + run0 + min(k + 1, runs - 1), groups),
                              first, k + 1 < runs ? count : 0);
                    load_states<SPL>(&par_A[k][lane * SPL], A2);
                    const float bias = par[k][0][lane >> 2], D = par[k][1][lane >> 2];
                    // slope: of softplus; dz: dy silu'(z), the gate's gradient without its p
                    float dt[K / 4], in[K / 4], dp[K / 4], slope[K / 4], dz[K / 4], sum = 0.f;
#pragma unroll
                    for (int i = 0; i < K / 4; ++i) {
                        dt[i] = to_f32(now.d[i]) + bias;
                        slope[i] = 1.f;
                        if (P.softplus)
                            softplus_grad<FINE>(dt[i], dt[i], slope[i]);
                        dt[i] = 4 * i + j < count ? dt[i] : 0.f;
                        in[i] = dt[i] * to_f32(now.x[i]);
                        dp[i] = dz[i] = to_f32(now.g[i]);
                        if (P.z) {
                            float act, dact;
                            silu_grad<FINE>(to_f32(now.z[i]), act, dact);
                            dp[i] *= act;
                            dz[i] *= dact;
                        }
                        sum += dt[i];
                    }
                    float a[K][SPL], h[K][SPL], end[SPL], back[SPL], all[SPL];
#pragma unroll
                    for (int s = 0; s < SPL; ++s)
                        end[s] = back[s] = 0.f;
                    unrolled<K>([&](auto I) {
                        constexpr int i = I;
                        const float d = quad_lane<i % 4>(dt[i / 4]), v = quad_lane<i % 4>(in[i / 4]);
                        float Bt[SPL];
                        load_states<SPL>(&bc[w][0][i][j * SPL], Bt);
#pragma unroll
                        for (int s = 0; s < SPL; ++s) {
                            a[i][s] = __builtin_amdgcn_exp2f(d * A2[s]);
                            h[i][s] = v * Bt[s];
                            end[s] = fmaf(a[i][s], end[s], h[i][s]);
                        }
                    });
                    unrolled<K>([&](auto I) {
                        constexpr int i = K - 1 - I;
                        const float e = quad_lane<i % 4>(dp[i / 4]);
                        float Ct[SPL];
                        load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                        for (int s = 0; s < SPL; ++s)
                            back[s] = a[i][s] * fmaf(e, Ct[s], back[s]);
                    });
                    sum = quad_sum(sum);
#pragma unroll
                    for (int s = 0; s < SPL; ++s)
                        all[s] = __builtin_amdgcn_exp2f(sum * A2[s]);
                    store_states<SPL>(&ends[0][w][lane * SPL], all);
                    store_states<SPL>(&ends[1][w][lane * SPL], end);
                    store_states<SPL>(&ends[2][w][lane * SPL], back);
                    __syncthreads();
#pragma unroll
                    for (int n = 0; n < ROUNDS; ++n) {
                        // (where registers are short, places are made again, as the rows' offsets)
                        int it = lane + n * WAVE;
                        if constexpr (SPL == 4)
                            asm volatile("" : "+v"(it));
                        const int e = w * (ITEMS / 2) + it % (ITEMS / 2);
                        if (it < ITEMS) {
                            // the waves in their order, or from the last one
                            const bool rev = it >= ITEMS / 2;
                            const int step = rev ? -WAVE * SPL : WAVE * SPL;
                            const float *pa = &ends[0][rev ? NW - 1 : 0][e];
                            float *pe = &ends[rev ? 2 : 1][rev ? NW - 1 : 0][e];
                            // behind the last channel nothing, so that its last state, which was
                            // read without a branch, does not get into other states' sums
                            const int behind = (per - (run0 + k) * SCAN_CHANNELS) * S - 1;
                            float va[NW], ve[NW], v = e > behind ? 0.f : state[n];
#pragma unroll
                            for (int q = 0; q < NW; ++q) {
                                va[q] = pa[q * step];
                                ve[q] = pe[q * step];
                            }
#pragma unroll
                            for (int q = 0; q < NW; ++q) {
                                pe[q * step] = v;
                                v = fmaf(va[q], v, ve[q]);
                            }
                        }
                    }
                    __syncthreads();
                    load_states<SPL>(&ends[1][w][lane * SPL], hs);
                    load_states<SPL>(&ends[2][w][lane * SPL], r);
                    // forwards: h[i] becomes the state before token i
                    float part[4], y[K / 4];
                    unrolled<K>([&](auto I) {
                        constexpr int i = I;
                        const float e = quad_lane<i % 4>(dp[i / 4]);
                        float Ct[SPL], sum_y = 0.f;
                        load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                        for (int s = 0; s < SPL; ++s) {
                            const float before = hs[s];
                            hs[s] = fmaf(a[i][s], before, h[i][s]);
                            h[i][s] = before;
                            acc[(2 * i + 1) * SPL + s] = fmaf(e, hs[s], acc[(2 * i + 1) * SPL + s]);
                            sum_y = fmaf(Ct[s], hs[s], sum_y);
                        }
                        part[i % 4] = sum_y;
                        if constexpr (i % 4 == 3)
                            y[i / 4] = quad_sums(part, j);
                    });
                    // backwards
                    float dA[SPL], part_A[4], sum_B[K / 4], sum_w[K / 4];
#pragma unroll
                    for (int s = 0; s < SPL; ++s)
                        dA[s] = 0.f;
                    unrolled<K>([&](auto I) {
                        constexpr int i = K - 1 - I;
                        const float e = quad_lane<i % 4>(dp[i / 4]), v = quad_lane<i % 4>(in[i / 4]);
                        const float d = quad_lane<i % 4>(dt[i / 4]);
                        float Bt[SPL], Ct[SPL], gb = 0.f, wa = 0.f;
                        load_states<SPL>(&bc[w][0][i][j * SPL], Bt);
                        load_states<SPL>(&bc[w][1][i][j * SPL], Ct);
#pragma unroll
                        for (int s = 0; s < SPL; ++s) {
                            const float gs = fmaf(e, Ct[s], r[s]);
                            acc[2 * i * SPL + s] = fmaf(v, gs, acc[2 * i * SPL + s]);
                            gb = fmaf(gs, Bt[s], gb);
                            r[s] = a[i][s] * gs;
                            const float ws = r[s] * h[i][s];
                            wa = fmaf(ws, A2[s], wa);
                            dA[s] = fmaf(ws, d, dA[s]);
                        }
                        part[i % 4] = gb;
                        part_A[i % 4] = wa;
                        if constexpr (i % 4 == 0) {
                            sum_B[i / 4] = quad_sums(part, j);
                            sum_w[i / 4] = quad_sums(part_A, j);
                        }
                    });
                    float dD = 0.f, dbias = 0.f;
                    int j1 = j;
                    asm volatile("" : "+v"(j1));
                    const Rows<T, K> rx(P.dx, first, P.C, P.C, count);
                    const Rows<T, K> rd(P.ddelta, first, P.C, P.C, count);
                    const Rows<T, K> rz(P.dz, first, P.C, P.C, P.z ? count : 0);
#pragma unroll
                    for (int i = 0; i < K / 4; ++i) {
                        const float x = to_f32(now.x[i]);
                        const float dx = fmaf(dt[i], sum_B[i], D * dp[i]);
                        const float dd = slope[i] * fmaf(x, sum_B[i], sum_w[i] * (1.f / LOG2E));
                        if (4 * i + j < count) {
                            dD = fmaf(dp[i], x, dD);
                            dbias += dd;
                        }
                        const int at = rx.at(4 * i + j1, P.C, ch.c, ch.live);
                        rx.store(from_f32<T>(dx), at);
                        rd.store(from_f32<T>(dd), at);
                        rz.store(from_f32<T>(dz[i] * fmaf(D, x, y[i])), at);
                    }
                    float old[SPL];
                    load_states<SPL>(&sum_A[k][w][lane * SPL], old);
#pragma unroll
                    for (int s = 0; s < SPL; ++s)
                        old[s] += dA[s];
                    store_states<SPL>(&sum_A[k][w][lane * SPL], old);
                    dD = quad_sum(dD);
                    dbias = quad_sum(dbias);
                    if (j < 2)
                        sum_D[k][j][w][lane >> 2] += j ? dbias : dD;
                }
            }
            float v[V];
            channel_sums<V>(acc, v);
            const int x = 4 * ((lane >> 2) & 3) + 2 * ((lane >> 4) & 1) + (lane >> 5);
            const int t = V * x / (2 * SPL), rest = V * x % (2 * SPL);   // token; tensor and state
            if (t < count)
                store_states<V>(rows_bc + (long)t * P.G * (2 * S) + rest / SPL * S + j * SPL + rest % SPL, v);
        }
    }
    // the waves' sums, in order
    __syncthreads();
    for (int k = 0; k < runs; ++k) {
        const int in0 = (run0 + k) * SCAN_CHANNELS;
        for (int i = threadIdx.x; i < SCAN_CHANNELS * (S + 2); i += NW * WAVE) {
            const int cl = i / (S + 2), n = i % (S + 2);
            if (in0 + cl >= per)
                continue;
            float s = 0.f;
            for (int q = 0; q < NW; ++q) {
                if (n < S) {
                    s += sum_A[k][q][(4 * cl + n / SPL) * SPL + n % SPL];
                } else {
                    s += sum_D[k][n - S][q][cl];
                }
            }
            P.ws_sum[((long)part * P.C + (long)g * per + in0 + cl) * (S + 2) + n] = s;
        }
    }
}

// Sums of the parts (64 bits, in order) and of the sets; zero gradients of the rows
// behind the last sequence.
constexpr int NT = 256, TAIL_WGS = 64;
template <typename T>
__global__ __launch_bounds__(NT) void scan_sum_kernel(ScanParams P, int sets, long wide, long bc) {
    const long id = blockIdx.x;
    if (id < wide) {
        const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE;
        const long i = id * WAVE + lane, n = (long)P.C * (P.S + 2);
        double s = 0.;
        if (i < n)
            for (int p = wv; p < P.parts; p += NT / WAVE)
                s += (double)P.ws_sum[p * n + i];
        __shared__ double sums[NT / WAVE][WAVE];
        sums[wv][lane] = s;
        __syncthreads();
        if (wv > 0 || i >= n)
            return;
        for (int q = 1; q < NT / WAVE; ++q)
            s += sums[q][lane];
        const long c = i / (P.S + 2);
        const int k = (int)(i % (P.S + 2));
        if (k < P.S)
            P.dA[c * P.S + k] = (float)s;
        else if (k == P.S && P.dD)
            P.dD[c] = (float)s;
        else if (k > P.S && P.dbias)
            P.dbias[c] = (float)s;
        return;
    }
    const long end = P.block_offsets ? tail_start(P) : P.tokens;
    const long wg = id - wide;
    if (wg < bc) {
        const long row = (long)P.G * 2 * P.S, i = wg * NT + threadIdx.x;
        if (i >= P.tokens * row)
            return;
        const long t = i / row;
        float s = 0.f;
        if (t < end)
            for (int q = 0; q < sets; ++q)
                s += P.ws_bc[q * P.tokens * row + i];
        const int in = (int)(i % row), grp = in / (2 * P.S), which = in / P.S % 2, n = in % P.S;
        T *to = static_cast<T *>(which ? P.dC : P.dB);
        to[(t * P.G + grp) * P.S + n] = from_f32<T>(s);
        return;
    }
    for (long i = end * P.C + (wg - bc) * NT + threadIdx.x; i < P.tokens * P.C;
         i += (long)TAIL_WGS * NT) {
        static_cast<T *>(P.dx)[i] = from_f32<T>(0.f);
        static_cast<T *>(P.ddelta)[i] = from_f32<T>(0.f);
        if (P.z)
            static_cast<T *>(P.dz)[i] = from_f32<T>(0.f);
    }
}

template <typename T, int SPL> hipError_t launch_grad_t(const ScanParams &P, hipStream_t st) {
    constexpr int NW = grad_waves<SPL>();
    const int groups = scan_groups(P.C, P.G), sets = scan_sets(P);
    const long blocks = scan_total_blocks(P);
    if (P.parts > 0) {
        hipLaunchKernelGGL((scan_grad_kernel<T, SPL>), dim3((unsigned)((long)P.parts * sets * P.G)),
                           dim3(NW * WAVE), 0, st, P, groups, sets, blocks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    const long wide = ((long)P.C * (P.S + 2) + WAVE - 1) / WAVE;
    const long bc = P.dB ? (P.tokens * P.G * 2 * P.S + NT - 1) / NT : 0;
    if (wide + bc == 0)
        return hipSuccess;
    hipLaunchKernelGGL((scan_sum_kernel<T>), dim3((unsigned)(wide + bc + (P.block_offsets ? TAIL_WGS : 0))),
                       dim3(NT), 0, st, P, sets, wide, bc);
    return hipGetLastError();
}

}  // namespace scan

hipError_t launch_scan_backward(const ScanParams &P, hipStream_t st) {
    // (without channels what is left are zeros in dB and dC)
    const hipError_t e = P.C > 0 ? launch_scan_states(P, true, st) : hipSuccess;
    if (e != hipSuccess)
        return e;
    switch (P.S) {
    case 8: return P.bf16 ? scan::launch_grad_t<bf16, 2>(P, st) : scan::launch_grad_t<float, 2>(P, st);
    case 16: return P.bf16 ? scan::launch_grad_t<bf16, 4>(P, st) : scan::launch_grad_t<float, 4>(P, st);
    default: return P.bf16 ? scan::launch_grad_t<bf16, 8>(P, st) : scan::launch_grad_t<float, 8>(P, st);
    }
}

}  // namespace kdn
