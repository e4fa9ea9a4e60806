// kdn_norm_abi.cpp -- C ABI of the gated norm and of the norm of the residual
// stream: host-side validation of every argument (before any HIP call), then the
// launches on the caller's stream.
#include "kdn.h"
#include "kdn_batch.h"
#include "kdn_norm.h"

#include <algorithm>
#include <math.h>

using kdn::aligned;
using kdn::clash;
using kdn::Range;
using kdn::span;

namespace {

bool valid_eps(float eps) { return eps > 0.f && eps < INFINITY; }

kdn_status gated_shape(kdn::GatedNormParams &P, int dtype, int tokens, int H, int d, int order,
                       int act, int per_head, float eps, long long x_stride, long long z_stride) {
    if (!kdn::valid_dtype(dtype) || (order != KDN_NORM_GATE && order != KDN_GATE_NORM) ||
        act < KDN_ACT_NONE || act > KDN_ACT_SIGMOID || !valid_eps(eps))
        return KDN_ERR_UNSUPPORTED;
    if (tokens < 0 || H < 0 || d < 0 || H >= (1 << 16) || (long long)tokens * H > INT_MAX)
        return KDN_ERR_SHAPE;
    if (d < 1 || d > kdn::NORM_DIM)
        return KDN_ERR_UNSUPPORTED;
    P = kdn::GatedNormParams{};
    P.bf16 = dtype == KDN_BF16;
    P.tokens = tokens; P.H = H; P.d = d;
    P.per_head = per_head != 0; P.gate_first = order == KDN_GATE_NORM; P.act = act; P.eps = eps; P.inv_d = 1. / d;
    if (kdn_status st = kdn::row_stride(x_stride, (long long)H * d, &P.x_stride)) return st;
    if (kdn_status st = kdn::row_stride(z_stride, (long long)H * d, &P.z_stride)) return st;
    return KDN_OK;
}

// Rows as a norm's outputs are launched: threads of a row as it has 16-byte pieces, in
// workgroups of 256 or of one row.
bool rows_launchable(long long rows, int d, bool bf16) {
    const int tpr = kdn::norm_row_threads(d, bf16);
    const int per = std::max(1, 256 / tpr);
    return kdn::launchable((rows + per - 1) / per, std::max(256, tpr));
}
// Gradients' workgroups, of up to 1024 threads, and those that sum up 16 columns each.
bool parts_launchable(long long parts, int d, long long columns) {
    return kdn::launchable(parts, std::max(512, kdn::norm_row_threads(d, false))) &&
           kdn::launchable((columns + 15) / 16, 1024);
}

int gated_parts(int tokens, int H, int per_head) {
    const long long rows = per_head ? tokens : (long long)tokens * H;
    const int most = per_head ? std::max(1, kdn::NORM_PARTS / std::max(1, H)) : kdn::NORM_PARTS;
    return (int)std::min(rows, (long long)most);
}

// Sums over `rows` rows that a workgroup of `parts` writes: its threads hold as many float32
// rows of d values at once as fit, and of bf16 rows twice as many.
int norm_segs(long long rows, int d, int threads, int parts) {
    const long long held = std::max(1, threads / kdn::norm_row_threads(d, false));
    return (int)std::max(1LL, (rows - 1) / (std::max(1, parts) * held * kdn::SEG_ROUNDS) + 1);
}
int gated_segs(int tokens, int H, int d, int per_head) {
    return norm_segs(per_head ? tokens : (long long)tokens * H, d, 256, gated_parts(tokens, H, per_head));
}

bool gated_launchable(int tokens, int H, int d, int per_head) {
    return parts_launchable((long long)gated_parts(tokens, H, per_head) * (per_head ? H : 1), d,
                            (long long)(per_head ? H : 1) * d);
}

kdn_status residual_shape(kdn::ResidualNormParams &P, int dtype, int stream_dtype, int tokens,
                          int D, int scale_n, float eps, long long x_stride, long long r_stride) {
    if (!kdn::valid_dtype(dtype) || (stream_dtype != dtype && stream_dtype != KDN_F32) ||
        !valid_eps(eps))
        return KDN_ERR_UNSUPPORTED;
    if (tokens < 0 || D < 0 || (scale_n != 0 && scale_n != 1 && scale_n != D))
        return KDN_ERR_SHAPE;
    if (D < 1 || D > kdn::NORM_DIM)
        return KDN_ERR_UNSUPPORTED;
    P = kdn::ResidualNormParams{};
    P.bf16 = dtype == KDN_BF16; P.stream_bf16 = stream_dtype == KDN_BF16;
    P.tokens = tokens; P.D = D; P.scale_n = scale_n; P.eps = eps; P.inv_d = 1. / D;
    if (kdn_status st = kdn::row_stride(x_stride, D, &P.x_stride)) return st;
    if (kdn_status st = kdn::row_stride(r_stride, D, &P.r_stride)) return st;
    return KDN_OK;
}

int residual_parts(int tokens) { return std::min(tokens, kdn::RESIDUAL_PARTS); }
int residual_segs(int tokens, int D) { return norm_segs(tokens, D, 512, residual_parts(tokens)); }

// The workspace's checks, against all other arguments.
kdn_status workspace_ok(void *workspace, unsigned long long bytes, long long need,
                        const Range *ins, int ni, const Range *outs, int no) {
    if (need <= 0)
        return KDN_OK;
    if (!workspace || bytes < (unsigned long long)need)
        return KDN_ERR_WORKSPACE;
    if (!aligned(workspace, 256))
        return KDN_ERR_ALIGN;
    const Range ws[] = {{workspace, need}};
    return clash(ws, 1, ins, ni) || clash(ws, 1, outs, no) ? KDN_ERR_ALIAS : KDN_OK;
}

kdn_status done(hipError_t e) { return e == hipSuccess ? KDN_OK : KDN_ERR_HIP; }

}  // namespace

extern "C" {

kdn_status kdn_gated_norm(kdn_dtype dtype, int tokens, int H, int d, kdn_norm_order order,
                          kdn_activation act, int per_head, float eps, long long x_stride,
                          long long z_stride, const void *x, const float *weight, const void *z,
                          void *y, void *stream) {
    kdn::GatedNormParams P;
    if (kdn_status st = gated_shape(P, dtype, tokens, H, d, order, act, per_head, eps, x_stride,
                                    z_stride))
        return st;
    if (!rows_launchable((long long)tokens * H, d, P.bf16))
        return KDN_ERR_SHAPE;
    const long long es = P.bf16 ? 2 : 4, row = (long long)H * d;
    if (tokens * row > 0 && (!x || !weight || !y))
        return KDN_ERR_NULL;
    if (!aligned(x, es) || !aligned(z, es) || !aligned(y, es) || !aligned(weight, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{x, span(tokens, P.x_stride, row, es)},
                         {z, span(tokens, P.z_stride, row, es)},
                         {weight, 4LL * (per_head ? row : d)}};
    const Range outs[] = {{y, tokens * row * es}};
    if (clash(outs, 1, ins, 3))
        return KDN_ERR_ALIAS;
    P.x = x; P.z = z; P.weight = weight; P.y = y;
    return done(kdn::launch_gated_norm(P, static_cast<hipStream_t>(stream)));
}

unsigned long long kdn_gated_norm_backward_workspace_size(int tokens, int H, int d, int per_head,
                                                          kdn_status *status) {
    kdn::GatedNormParams P;
    kdn_status st = gated_shape(P, KDN_F32, tokens, H, d, KDN_NORM_GATE, KDN_ACT_SILU, per_head, 1.f,
                                0, 0);
    if (st == KDN_OK && !gated_launchable(tokens, H, d, per_head))
        st = KDN_ERR_SHAPE;
    if (status)
        *status = st;
    return st == KDN_OK ? 4ull * gated_parts(tokens, H, per_head) * gated_segs(tokens, H, d, per_head) *
                                (per_head ? H : 1) * d : 0;
}

kdn_status kdn_gated_norm_backward(kdn_dtype dtype, int tokens, int H, int d,
                                   kdn_norm_order order, kdn_activation act, int per_head,
                                   float eps, long long x_stride, long long z_stride,
                                   const void *x, const float *weight, const void *z,
                                   const void *d_y, void *dx, void *dz, float *dweight,
                                   void *workspace, unsigned long long workspace_bytes,
                                   void *stream) {
    kdn::GatedNormParams P;
    if (kdn_status st = gated_shape(P, dtype, tokens, H, d, order, act, per_head, eps, x_stride,
                                    z_stride))
        return st;
    if (!gated_launchable(tokens, H, d, per_head))
        return KDN_ERR_SHAPE;
    const long long es = P.bf16 ? 2 : 4, row = (long long)H * d, n_w = per_head ? row : d;
    if ((tokens * row > 0 && (!x || !weight || !d_y || !dx || (z && !dz))) || (n_w > 0 && !dweight) ||
        (!z && dz))
        return KDN_ERR_NULL;
    for (const void *p : {x, z, d_y, (const void *)dx, (const void *)dz})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    if (!aligned(weight, 4) || !aligned(dweight, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{x, span(tokens, P.x_stride, row, es)},
                         {z, span(tokens, P.z_stride, row, es)},
                         {weight, 4 * n_w},
                         {d_y, tokens * row * es}};
    const Range outs[] = {{dx, tokens * row * es}, {dz, tokens * row * es}, {dweight, 4 * n_w}};
    if (clash(outs, 3, ins, 4))
        return KDN_ERR_ALIAS;
    P.parts = H > 0 ? gated_parts(tokens, H, per_head) : 0;
    P.segs = gated_segs(tokens, H, d, per_head);
    if (kdn_status st = workspace_ok(workspace, workspace_bytes, 4LL * P.parts * P.segs * n_w, ins, 4, outs, 3))
        return st;
    P.x = x; P.z = z; P.weight = weight; P.d_y = d_y;
    P.dx = dx; P.dz = dz; P.dweight = dweight; P.ws = static_cast<float *>(workspace);
    return done(kdn::launch_gated_norm_backward(P, static_cast<hipStream_t>(stream)));
}

kdn_status kdn_residual_norm(kdn_dtype dtype, kdn_dtype stream_dtype, int tokens, int D,
                             int scale_n, float eps, long long x_stride, long long residual_stride,
                             const void *x, const void *residual, const float *weight,
                             const float *scale, void *y, void *h, void *stream) {
    kdn::ResidualNormParams P;
    if (kdn_status st = residual_shape(P, dtype, stream_dtype, tokens, D, scale_n, eps, x_stride,
                                       residual_stride))
        return st;
    if (!rows_launchable(tokens, D, P.bf16))
        return KDN_ERR_SHAPE;
    const long long es = P.bf16 ? 2 : 4, rs = P.stream_bf16 ? 2 : 4, n = (long long)tokens * D;
    if (n > 0 && (!x || !residual || !weight || !y || !h))
        return KDN_ERR_NULL;
    if ((scale_n > 0) != (scale != nullptr))
        return KDN_ERR_NULL;
    if (!aligned(x, es) || !aligned(y, es) || !aligned(residual, rs) || !aligned(h, rs) ||
        !aligned(weight, 4) || !aligned(scale, 4))
        return KDN_ERR_ALIGN;
    const bool in_place = h == residual && P.r_stride == D;
    const Range ins[] = {{x, span(tokens, P.x_stride, D, es)},
                         {in_place ? nullptr : residual, span(tokens, P.r_stride, D, rs)},
                         {weight, 4LL * D},
                         {scale, 4LL * scale_n}};
    const Range outs[] = {{y, n * es}, {h, n * rs}};
    if (clash(outs, 2, ins, 4))
        return KDN_ERR_ALIAS;
    P.x = x; P.residual = residual; P.weight = weight; P.scale = scale; P.y = y; P.h = h;
    return done(kdn::launch_residual_norm(P, static_cast<hipStream_t>(stream)));
}

unsigned long long kdn_residual_norm_backward_workspace_size(int tokens, int D, int scale_n,
                                                             kdn_status *status) {
    kdn::ResidualNormParams P;
    const kdn_status st = residual_shape(P, KDN_F32, KDN_F32, tokens, D, scale_n, 1.f, 0, 0);
    if (status)
        *status = st;
    return st == KDN_OK ? 4ull * residual_parts(tokens) * residual_segs(tokens, D) * (D + scale_n) : 0;
}

kdn_status kdn_residual_norm_backward(kdn_dtype dtype, kdn_dtype stream_dtype, int tokens, int D,
                                      int scale_n, float eps, long long x_stride,
                                      long long h_stride, const void *x, const void *h,
                                      const float *weight, const float *scale, const void *d_y,
                                      const void *d_h, void *dx, void *dresidual, float *dweight,
                                      float *dscale, void *workspace,
                                      unsigned long long workspace_bytes, void *stream) {
    kdn::ResidualNormParams P;
    if (kdn_status st = residual_shape(P, dtype, stream_dtype, tokens, D, scale_n, eps, x_stride,
                                       h_stride))
        return st;
    const long long es = P.bf16 ? 2 : 4, rs = P.stream_bf16 ? 2 : 4, n = (long long)tokens * D;
    if ((n > 0 && (!h || !weight || !d_y || !dresidual || (dscale && !x))) || !dweight ||
        (scale_n > 0) != (scale != nullptr) || (dscale && !scale))
        return KDN_ERR_NULL;
    if (!aligned(x, es) || !aligned(d_y, es) || !aligned(dx, es) || !aligned(h, rs) ||
        !aligned(d_h, rs) || !aligned(dresidual, rs) || !aligned(weight, 4) || !aligned(scale, 4) ||
        !aligned(dweight, 4) || !aligned(dscale, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{x, span(tokens, P.x_stride, D, es)},
                         {h, span(tokens, P.r_stride, D, rs)},
                         {weight, 4LL * D},
                         {scale, 4LL * scale_n},
                         {d_y, n * es},
                         {d_h, n * rs}};
    const Range outs[] = {{dx, n * es}, {dresidual, n * rs}, {dweight, 4LL * D}, {dscale, 4LL * scale_n}};
    if (clash(outs, 4, ins, 6))
        return KDN_ERR_ALIAS;
    P.parts = residual_parts(tokens);
    P.segs = residual_segs(tokens, D);
    const long long n_ws = 4LL * P.parts * P.segs * (D + (dscale ? scale_n : 0));
    if (kdn_status st = workspace_ok(workspace, workspace_bytes, n_ws, ins, 6, outs, 4))
        return st;
    P.x = x; P.residual = h; P.weight = weight; P.scale = scale; P.d_y = d_y; P.d_h = d_h;
    P.dx = dx; P.dresidual = dresidual; P.dweight = dweight; P.dscale = dscale;
    P.ws = static_cast<float *>(workspace);
    return done(kdn::launch_residual_norm_backward(P, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
