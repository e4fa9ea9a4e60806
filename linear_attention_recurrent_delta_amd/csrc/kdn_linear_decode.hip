// kdn_linear_decode.hip -- one token of linear attention with a decay for
// each head for every row of a batch (gfx950):
//   S <- e^g S + k v^T,   o = S^T q.
// Bound by one read and one write of S: 8192 states of 128 x 128 (1.07 GB) in
// 192 us, 5.6 TB/s, above what a large copy reaches (4.9); a step of a few
// states by the launch and the latency of one load and one store, 3.3 us.  S
// passes the caches (non-temporal): nothing of it is read twice in a step.
// The columns of S are independent, so a workgroup of 256 threads owns CW of
// the d_v columns of one (row, head); thread (rg, cg) holds rows
// [rg * RPT, + RPT) of 4 columns in registers, and the partial outputs of the
// row groups are summed by lane exchanges, then across the waves in LDS (a
// fixed order: results are the same every time).
#include "kdn_linear_device.h"

namespace kdn {
namespace lin {

constexpr int DNT = 256;

template <typename T, int DK, int DV, int CW>
__global__ __launch_bounds__(DNT) void linear_decode_kernel(LinearDecodeParams P) {
    constexpr int CG = CW / 4, RG = DNT / CG, RPT = DK / RG, SPL = DV / CW;
    static_assert(RPT * RG == DK && RPT >= 1, "decode tiling");
    const int tid = threadIdx.x, lane = tid & (WAVE - 1), w = tid / WAVE;
    const int cg = tid % CG, rg = tid / CG;
    const long id = blockIdx.x;
    const int c0 = (int)(id % SPL) * CW + 4 * cg;
    const int h = (id / SPL) % P.H;
    const long n = id / SPL / P.H;
    const long slot = P.slots ? P.slots[n] : n;
    if (slot < 0 || slot >= P.pool)
        return;

    float *S = P.S + (slot * P.H + h) * (long)(DK * DV) + rg * RPT * DV + c0;
    const T *q = static_cast<const T *>(P.q) + n * P.q_stride + (h / (P.H / P.Hq)) * DK + rg * RPT;
    const T *k = static_cast<const T *>(P.k) + n * P.k_stride + (h / (P.H / P.Hk)) * DK + rg * RPT;
    const T *v = static_cast<const T *>(P.v) + n * P.v_stride + (h / (P.H / P.Hv)) * DV + c0;

    f32x4 s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        s[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(S + m * DV));
    const float la = P.gate == KDN_GATE_HEAD ? static_cast<const float *>(P.la)[h]
                                             : to_f32(static_cast<const T *>(P.la)[n * P.H + h]);
    const float a = exp2_fast((float)log2_decay(la));
    f32x4 x, acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x[e] = to_f32(v[e]);
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        const float ki = to_f32(k[m]), qi = to_f32(q[m]);
        s[m] = s[m] * a + x * ki;
        acc += s[m] * qi;
        __builtin_nontemporal_store(s[m], reinterpret_cast<f32x4 *>(S + m * DV));
    }
    // row groups of this wave, then the waves
#pragma unroll
    for (int off = CG; off < WAVE; off <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] += __shfl_xor(acc[e], off, WAVE);
    __shared__ f32x4 part[DNT / WAVE][CG];
    if (lane < CG)
        part[w][lane] = acc;
    __syncthreads();
    if (tid < CG) {
        f32x4 y = part[0][tid];
#pragma unroll
        for (int i = 1; i < DNT / WAVE; ++i)
            y += part[i][tid];
        T *o = static_cast<T *>(P.o) + (n * P.H + h) * DV + c0;
        const float f[4] = {y[0], y[1], y[2], y[3]};
        lds_stn<4>(o, f);
    }
}

template <typename T>
static hipError_t launch_decode_t(const LinearDecodeParams &P, hipStream_t st) {
    const long nh = (long)P.N * P.H;
#define KDN_LDEC(DK_, DV_, CW_)                                                             \
    if (P.dk == DK_ && P.dv == DV_) {                                                       \
        hipLaunchKernelGGL((linear_decode_kernel<T, DK_, DV_, CW_>),                        \
                           dim3((unsigned)(nh * (DV_ / CW_))), dim3(DNT), 0, st, P);        \
        return hipGetLastError();                                                           \
    }
    // No more states than CUs: 32 columns (whole cache lines) each, so that more
    // CUs share a state.  bf16, us, split against whole: 8 states of 128 x 128
    // 3.3 / 5.6, 256 7.2 / 8.0, 512 14.0 / 13.2; 256 of 128 x 64 4.8 / 5.2, 512
    // 7.1 / 7.1; 256 of 64 x 64 3.8 / 3.9.
    if (nh <= 256) {
        KDN_LDEC(64, 64, 32)
        KDN_LDEC(64, 128, 32)
        KDN_LDEC(128, 64, 32)
        KDN_LDEC(128, 128, 32)
    }
    KDN_LDEC(64, 64, 64)
    KDN_LDEC(64, 128, 128)
    KDN_LDEC(128, 64, 64)
    KDN_LDEC(128, 128, 128)
#undef KDN_LDEC
    return hipErrorInvalidValue;
}

}  // namespace lin

hipError_t launch_linear_decode(const LinearDecodeParams &P, hipStream_t st) {
    if ((long)P.N * P.H == 0)
        return hipSuccess;
    return P.bf16 ? lin::launch_decode_t<bf16>(P, st) : lin::launch_decode_t<float>(P, st);
}

}  // namespace kdn
