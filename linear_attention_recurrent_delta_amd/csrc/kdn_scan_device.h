// kdn_scan_device.h -- device-side pieces shared by the kernels of the selective
// scan: a wave's channels and tokens, time steps, and exchanges within four lanes.
//
// A wave holds 16 channels.  Lane 4 k + j has the states j SPL .. + SPL of channel k
// (S = 4 SPL), and of the per-token values of channel k those of every fourth
// token, t = 4 i + j: loads of a row are 16 neighbouring channels, each value is
// loaded and each time step made once, and the other three lanes get it by a DPP
// broadcast within the four.
#pragma once

#include "kdn_act.h"
#include "kdn_batch_device.h"
#include "kdn_scan.h"

#include <utility>

namespace kdn {
namespace scan {

constexpr float LOG2E = 1.44269504f;

// f(0), f(1), .. f(N - 1) with constants.
template <int... I, typename F>
__device__ __forceinline__ void for_seq(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void unrolled(F f) {
    for_seq(std::make_integer_sequence<int, N>{}, f);
}

template <int CTRL> __device__ __forceinline__ float dpp(float x) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// The value of lane J of the four; of the lane one or two away.
template <int J> __device__ __forceinline__ float quad_lane(float x) { return dpp<J * 0x55>(x); }
__device__ __forceinline__ float quad_xor1(float x) { return dpp<0xB1>(x); }
__device__ __forceinline__ float quad_xor2(float x) { return dpp<0x4E>(x); }
__device__ __forceinline__ float quad_sum(float x) {
    x += quad_xor1(x);
    return x + quad_xor2(x);
}
// Lane j gets the sum over the four lanes of their v[j].
__device__ __forceinline__ float quad_sums(const float (&v)[4], int j) {
    const float a = (j & 1 ? v[1] : v[0]) + quad_xor1(j & 1 ? v[0] : v[1]);
    const float b = (j & 1 ? v[3] : v[2]) + quad_xor1(j & 1 ? v[2] : v[3]);
    return (j & 2 ? b : a) + quad_xor2(j & 2 ? a : b);
}

// log(1 + e^x) = max(x, 0) + log(1 + w), w = e^-|x| <= 1, by
// log(1 + w) = 2 (s + s^3 / 3 + s^5 / 5 ..), s = w / (2 + w) <= 1/3: no cancellation,
// so that small time steps keep their relative precision.  The terms left out are
// below 2^-18 of the sum in bfloat16 calls, 2^-26 in float32 ones.
template <bool FINE> __device__ __forceinline__ float softplus(float x, float w) {
    const float s = FINE ? w / (2.f + w) : w * fast_rcp(2.f + w);
    const float q = s * s;
    float p;
    if constexpr (FINE) {
        p = fmaf(q, 1.f / 15.f, 1.f / 13.f);
        p = fmaf(p, q, 1.f / 11.f);
        p = fmaf(p, q, 1.f / 9.f);
    } else {
        p = 1.f / 9.f;
    }
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p * q, s, s);
    // NaN stays NaN: no fmaxf
    return fmaf(2.f, p, x < 0.f ? 0.f : x);
}
template <bool FINE> __device__ __forceinline__ float softplus(float x) {
    return softplus<FINE>(x, exp_f32<FINE>(-fabsf(x)));
}
// softplus(x) and its derivative, 1 / (1 + e^-x), from the same exponential
template <bool FINE>
__device__ __forceinline__ void softplus_grad(float x, float &y, float &dy) {
    const float w = exp_f32<FINE>(-fabsf(x)), n = x < 0.f ? w : 1.f;
    y = softplus<FINE>(x, w);
    dy = FINE ? n / (1.f + w) : n * fast_rcp(1.f + w);
}

constexpr int XCDS = 8;

// Workgroup `id` of a grid over (outer, run of channels): four runs share the lines of
// a row and are neighbours on an XCD; fours go over the XCDs in turn, so that each has
// its part of every sequence (2048 channels of packed prompts of 100, 200, 400 and 3000
// tokens: 90 us, and 181 where an XCD has consecutive units).
__host__ __device__ __forceinline__ long four_grid(long outers, long runs) {
    return (outers * ((runs + 3) / 4) + XCDS - 1) / XCDS * XCDS * 4;
}
__device__ __forceinline__ bool four_unit(long id, long outers, int runs, long &outer, int &run) {
    const int fours = (runs + 3) / 4;
    const long k = id / XCDS, four = k / 4 * XCDS + id % XCDS;
    outer = four / fours;
    run = (int)(four % fours * 4 + k % 4);
    return outer < outers && run < runs;
}

// A wave's 16 channels: run k of the channels of group g.
struct Channels {
    int g, c;       // group; the lane's channel (of a lane behind the last: the last)
    bool live;
    __device__ __forceinline__ Channels(const ScanParams &P, int run, int groups) {
        const int per = P.C / P.G, k = run % groups;
        g = run / groups;
        const int in = k * SCAN_CHANNELS + ((threadIdx.x & (WAVE - 1)) >> 2);
        live = in < per;
        c = g * per + (live ? in : per - 1);
    }
};

// Rows of a per-token tensor of C channels, K of them at a time through a descriptor
// that ends with the last that is there: rows behind it read 0 and are not written,
// without a branch.  Strides are below 2^25 elements, K rows below 2^32 bytes.
template <typename T, int K> struct Rows {
    __amdgpu_buffer_rsrc_t d;
    // rows first .. of which `count` are there (the same in every lane)
    __device__ __forceinline__ Rows(const void *p, long first, long stride, int C, int count) {
        const int rows = min(count, K);
        d = buf_rsrc(static_cast<const T *>(p) + first * stride,
                     rows > 0 ? ((rows - 1) * (unsigned)stride + (unsigned)C) * (unsigned)sizeof(T) : 0u);
    }
    // row t, channel c, for lanes that take part in it
    __device__ __forceinline__ static int at(int t, long stride, int c, bool live) {
        return live ? (int)(((unsigned)t * (unsigned)stride + (unsigned)c) * (unsigned)sizeof(T)) : -1;
    }
    __device__ __forceinline__ T load(int at) const {
        if constexpr (sizeof(T) == 2)
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(d, at, 0, 0));
        else
            return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(d, at, 0, 0));
    }
    __device__ __forceinline__ void store(T x, int at) const {
        if constexpr (sizeof(T) == 2)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, x), d, at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, x), d, at, 0, 0);
    }
};

// B and C of K consecutive tokens of a group, float32 in LDS, written and read by one
// wave.
template <typename T, int S, int K> struct GroupRows {
    static constexpr int EPL = 2 * K * S / WAVE;      // elements of a lane
    Pack<T, EPL> r;
    bool there;
    // rows first .. + K of which `count` are there (none or less: first + count is the
    // end of the rows): in the place of one behind them the last is read
    __device__ __forceinline__ void load(const ScanParams &P, int g, long first, int count) {
        const int lane = threadIdx.x & (WAVE - 1), e = (lane & 31) * EPL;
        const int row = min(e / S, count - 1), col = e % S;
        there = e / S < count;
        const T *p = lane < 32 ? static_cast<const T *>(P.B) + (first + row) * P.b_stride
                               : static_cast<const T *>(P.Cm) + (first + row) * P.c_stride;
        r.load(p + (long)g * S + col);
    }
    __device__ __forceinline__ float get(int i) const { return there ? r.get(i) : 0.f; }
    // to[0]: B, to[1]: C
    __device__ __forceinline__ void put(float (*to)[K][S]) const {
        const int lane = threadIdx.x & (WAVE - 1), e = (lane & 31) * EPL;
        float *p = &to[lane >> 5][0][0] + e;
        order();
        if constexpr (EPL == 2) {
            *reinterpret_cast<float2 *>(p) = make_float2(get(0), get(1));
        } else {
#pragma unroll
            for (int i = 0; i < EPL; i += 4)
                *reinterpret_cast<f32x4 *>(p + i) =
                    f32x4{get(i), get(i + 1), get(i + 2), get(i + 3)};
        }
        order();
    }
    // what a wave's lanes read from each other through LDS stays in order
    __device__ __forceinline__ static void order() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
};

// SPL consecutive floats, 8-byte aligned at least.
template <int SPL> __device__ __forceinline__ void load_states(const float *p, float (&v)[SPL]) {
    if constexpr (SPL == 2) {
        const float2 a = *reinterpret_cast<const float2 *>(p);
        v[0] = a.x; v[1] = a.y;
    } else {
#pragma unroll
        for (int i = 0; i < SPL; i += 4) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p + i);
            v[i] = a[0]; v[i + 1] = a[1]; v[i + 2] = a[2]; v[i + 3] = a[3];
        }
    }
}
template <int SPL>
__device__ __forceinline__ void store_states(float *p, const float (&v)[SPL]) {
    if constexpr (SPL == 2) {
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < SPL; i += 4)
            *reinterpret_cast<f32x4 *>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    }
}

// A with -inf (states that forget at once) as the lowest number, so that a token that is
// not there, of time step 0, leaves the state as it is: 0 (-inf) would be NaN.
__device__ __forceinline__ float finite_A(float a) {
    constexpr float LOWEST = -3.40282347e38f;
    return a < LOWEST ? LOWEST : a;      // NaN stays NaN
}
// A's row of the lane's channel times log2(e): a = 2^(dt A2).
template <int SPL>
__device__ __forceinline__ void load_A(const ScanParams &P, int c, int j, float (&A2)[SPL]) {
    load_states<SPL>(P.A + (long)c * (4 * SPL) + j * SPL, A2);
#pragma unroll
    for (int s = 0; s < SPL; ++s)
        A2[s] = finite_A(A2[s] * LOG2E);
}

}  // namespace scan
}  // namespace kdn
