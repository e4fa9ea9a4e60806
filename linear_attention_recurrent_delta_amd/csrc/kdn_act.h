// kdn_act.h -- device-side activations (silu, sigmoid) and element packs of a
// chosen width, shared by the convolution, norm and scan kernels.
#pragma once

#include "kdn_device.h"

namespace kdn {

// e^x.  v_exp_f32 is off by an ulp; the rounding of x log2(e) adds |x| 2^-24 to it
// (with the constant's own rounding as much again), which float32 calls (FINE)
// take back by the part that the product lost.
template <bool FINE> __device__ __forceinline__ float exp_f32(float x) {
    constexpr float L = 1.44269504f, L_LO = 1.92596299e-8f;
    const float t = x * L;
    float e = __builtin_amdgcn_exp2f(t);
    if constexpr (FINE) {
        const float lo = fmaf(x, L, -t) + x * L_LO;
        // past the ends of float32 e is 0 or infinite and stays so
        if (fabsf(t) < 126.f)
            e = fmaf(e, lo * 0.693147181f, e);
    }
    return e;
}

// sigmoid(x) and 1 - sigmoid(x), both without cancellation (and where e^-x is
// infinite, with g zero).
template <bool FINE>
__device__ __forceinline__ void sigmoid2(float x, float &g, float &rest) {
    const float e = exp_f32<FINE>(-x);
    g = FINE ? 1.f / (1.f + e) : fast_rcp(1.f + e);
    rest = e > 1e37f ? 1.f : e * g;       // NaN stays NaN
}
template <bool FINE> __device__ __forceinline__ float sigmoid_f32(float x) {
    float g, rest;
    sigmoid2<FINE>(x, g, rest);
    return g;
}
template <bool FINE> __device__ __forceinline__ float silu_f32(float x) {
    return x * sigmoid_f32<FINE>(x);
}
// silu(x) and its derivative
template <bool FINE>
__device__ __forceinline__ void silu_grad(float x, float &y, float &dy) {
    float g, rest;
    sigmoid2<FINE>(x, g, rest);
    y = x * g;
    dy = fmaf(y, rest, g);
}

// V consecutive elements as they lie in memory, on any element's boundary (global
// memory takes wide accesses there), of which the first n are there.
template <typename T, int V> struct Pack {
    typedef T Vec __attribute__((ext_vector_type(V)));
    typedef Vec Raw __attribute__((aligned(sizeof(T))));
    Vec r;
    __device__ __forceinline__ void zero() { r = (Vec)(T)0.f; }
    __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const Raw *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Raw *>(p) = r; }
    // elements past n (1 at least): zero (the last one is read in their place, so that
    // all loads are on their way together), not written
    __device__ __forceinline__ void load(const T *p, int n) {
        if (n >= V) {
            load(p);
        } else {
            T v[V - 1];
#pragma unroll
            for (int i = 0; i < V - 1; ++i)
                v[i] = p[i < n ? i : n - 1];
            zero();
#pragma unroll
            for (int i = 0; i < V - 1; ++i)
                r[i] = i < n ? v[i] : r[i];
        }
    }
    __device__ __forceinline__ void store(T *p, int n) const {
        if (n >= V) {
            store(p);
        } else {
#pragma unroll
            for (int i = 0; i < V - 1; ++i)
                if (i < n)
                    p[i] = r[i];
        }
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(r[i]); }
    __device__ __forceinline__ void set(int i, float x) { r[i] = from_f32<T>(x); }
};

// Sums over `parts` rows of 16 columns of ws [parts][n], in 64 bits in a fixed order, by a
// workgroup of NT threads: thread r * 16 + c adds every NT / 16-th row of column c, many
// loads at once; the first 16 threads get the sums of columns first .. + 16.
template <int NT>
__device__ __forceinline__ double part_sums(const float *ws, long n, int parts, long first,
                                            double (*lds)[16]) {
    constexpr int STEP = NT / 16, AHEAD = 8;
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const bool live = first + c < n;
    double s = 0.;
    for (int p = r; p < parts; p += AHEAD * STEP) {
        float v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            v[i] = 0.f;
            if (live && p + i * STEP < parts)
                v[i] = ws[(long)(p + i * STEP) * n + first + c];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            s += (double)v[i];
    }
    s += __shfl_xor(s, 16, WAVE);
    s += __shfl_xor(s, 32, WAVE);
    if ((threadIdx.x & (WAVE - 1)) < 16)
        lds[threadIdx.x / WAVE][c] = s;
    __syncthreads();
    s = lds[0][c];
#pragma unroll
    for (int i = 1; i < NT / WAVE; ++i)
        s += lds[i][c];
    return s;
}

}  // namespace kdn
