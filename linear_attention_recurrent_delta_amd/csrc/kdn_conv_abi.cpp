// kdn_conv_abi.cpp -- C ABI of the short causal convolution: host-side validation
// of every argument (before any HIP call), then the launches on the caller's
// stream.
#include "kdn.h"
#include "kdn_batch.h"
#include "kdn_conv.h"

#include <algorithm>

using kdn::aligned;
using kdn::clash;
using kdn::launchable;
using kdn::overlap;
using kdn::Range;
using kdn::span;

namespace {

kdn_status conv_shape(kdn::ConvParams &P, int dtype, int N, int T, int C, int W, int act,
                      long long x_stride, const kdn_packed *packed) {
    if (!kdn::valid_dtype(dtype) || (act != KDN_ACT_NONE && act != KDN_ACT_SILU))
        return KDN_ERR_UNSUPPORTED;
    if (C < 0 || W < 0)
        return KDN_ERR_SHAPE;
    if (W < 2 || W > kdn::CONV_TAPS)
        return KDN_ERR_UNSUPPORTED;
    P = kdn::ConvParams{};
    if (kdn_status st = kdn::batch_shape(P, N, T, packed))
        return st;
    P.bf16 = dtype == KDN_BF16;
    P.C = C; P.W = W; P.silu = act == KDN_ACT_SILU;
    if (kdn_status st = kdn::row_stride(x_stride, C, &P.x_stride))
        return st;
    if (C >= (1 << 26) || P.pool * (W - 1) >= (1LL << 32))
        return KDN_ERR_SHAPE;
    return KDN_OK;
}

// Parts that the sums over tokens are made in: as many workgroups as run at once
// (two a CU, by their registers), each over all the tiles it takes.  With 256, 512 and
// 1024 of them: B4 T4096 C2048 bf16 73, 56 and 59 us, 11 packed sequences of 1030
// channels in float32 48, 49 and 48.  A lane adds 16 tokens of a tile in float32: from
// PART_TILES tiles a part on there are twice, three times .. as many parts, so that no sum
// is a chain of more than 512 of them, however long the sequences are.
constexpr int GRAD_WGS = 512, PART_TILES = 32;
long long grad_parts(const kdn::ConvParams &P, bool packed) {
    const long long tiles = kdn::conv_tiles(P, packed);
    const int chunks = std::max(1, kdn::conv_chunks(P.C, kdn::conv_vec(P.bf16, true)));
    const long long once = std::max(1, GRAD_WGS / chunks);
    return std::min(tiles, once * std::max(1LL, (tiles - 1) / (once * PART_TILES) + 1));
}
// The gradients' launches: the parts' and the sums' with what follows them.
bool grad_launchable(const kdn::ConvParams &P, bool packed) {
    return launchable(grad_parts(P, packed) * kdn::conv_chunks(P.C, kdn::conv_vec(P.bf16, true)), 256) &&
           launchable(65536LL + 64 + P.N, 256);
}

}  // namespace

extern "C" {

kdn_status kdn_causal_conv(kdn_dtype dtype, int N, int T, int C, int W, kdn_activation act,
                           long long x_stride, const void *x, const float *weight,
                           const float *bias, const void *state0, void *y, void *state_out,
                           const kdn_packed *packed, void *stream) {
    kdn::ConvParams P;
    if (kdn_status st = conv_shape(P, dtype, N, T, C, W, act, x_stride, packed))
        return st;
    // tiles and, behind them, sequences
    if (!launchable((kdn::conv_tiles(P, packed != nullptr) + N) *
                    kdn::conv_chunks(C, kdn::conv_vec(P.bf16, false)), 256))
        return KDN_ERR_SHAPE;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens;
    if (tok * C > 0 && (!x || !weight || !y))
        return KDN_ERR_NULL;
    if (kdn_status st = kdn::batch_tables(P, packed))
        return st;
    for (const void *p : {x, state0, (const void *)y, (const void *)state_out})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    if (!aligned(weight, 4) || !aligned(bias, 4))
        return KDN_ERR_ALIGN;
    const long long n_s = P.pool * (W - 1) * C * es;
    const Range ins[] = {{x, span(tok, P.x_stride, C, es)},
                         {weight, 4LL * C * W},
                         {bias, 4LL * C},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {state0 == state_out ? nullptr : state0, n_s}};
    const Range outs[] = {{y, tok * C * es}, {state_out, n_s}};
    if (clash(outs, 2, ins, 7))
        return KDN_ERR_ALIAS;
    if (C == 0)
        return KDN_OK;
    P.x = x; P.weight = weight; P.bias = bias; P.state0 = state0;
    P.y = y; P.state_out = state_out;
    const hipError_t e = kdn::launch_conv(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

kdn_status kdn_causal_conv_decode(kdn_dtype dtype, int N, int C, int W, kdn_activation act,
                                  long long x_stride, const void *x, const float *weight,
                                  const float *bias, const int *slots, int pool, void *state,
                                  void *y, void *stream) {
    kdn::ConvParams L;
    if (kdn_status st = conv_shape(L, dtype, N, 1, C, W, act, x_stride, nullptr))
        return st;
    if (pool < 0 || (!slots && pool < N) || (long long)pool * (W - 1) >= (1LL << 32) ||
        !launchable((long long)N * kdn::conv_chunks(C, kdn::conv_vec(L.bf16, false)), 64))
        return KDN_ERR_SHAPE;
    const long long es = L.bf16 ? 2 : 4, n = (long long)N * C;
    if (n > 0 && (!x || !weight || !y || (pool > 0 && !state)))
        return KDN_ERR_NULL;
    for (const void *p : {x, (const void *)state, (const void *)y})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(slots, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{x, span(N, L.x_stride, C, es)},
                         {weight, 4LL * C * W},
                         {bias, 4LL * C},
                         {slots, 4LL * N}};
    const Range outs[] = {{y, n * es}, {state, (long long)pool * (W - 1) * C * es}};
    if (clash(outs, 2, ins, 4))
        return KDN_ERR_ALIAS;
    kdn::ConvDecodeParams P;
    P.bf16 = L.bf16;
    P.N = N; P.C = C; P.W = W; P.silu = L.silu;
    P.x_stride = L.x_stride;
    P.x = x; P.weight = weight; P.bias = bias;
    P.slots = slots; P.pool = pool; P.state = state; P.y = y;
    const hipError_t e = kdn::launch_conv_decode(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

unsigned long long kdn_causal_conv_backward_workspace_size(kdn_dtype dtype, int N, int T, int C,
                                                           int W, const kdn_packed *packed,
                                                           kdn_status *status) {
    kdn::ConvParams P;
    kdn_status st = conv_shape(P, dtype, N, T, C, W, KDN_ACT_SILU, 0, packed);
    if (st == KDN_OK && !grad_launchable(P, packed != nullptr))
        st = KDN_ERR_SHAPE;
    if (status)
        *status = st;
    return st == KDN_OK ? 4ull * (unsigned long long)grad_parts(P, packed != nullptr) * (W + 1) * C : 0;
}

kdn_status kdn_causal_conv_backward(kdn_dtype dtype, int N, int T, int C, int W,
                                    kdn_activation act, long long x_stride, const void *x,
                                    const float *weight, const float *bias, const void *state0,
                                    const void *d_y, const void *dstate_out, void *dx,
                                    float *dweight, float *dbias, void *dstate0,
                                    const kdn_packed *packed, void *workspace,
                                    unsigned long long workspace_bytes, void *stream) {
    kdn::ConvParams P;
    if (kdn_status st = conv_shape(P, dtype, N, T, C, W, act, x_stride, packed))
        return st;
    if (!grad_launchable(P, packed != nullptr))
        return KDN_ERR_SHAPE;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens;
    if ((tok * C > 0 && (!x || !d_y || !dx)) || (C > 0 && (!weight || !dweight)))
        return KDN_ERR_NULL;
    if (kdn_status st = kdn::batch_tables(P, packed))
        return st;
    for (const void *p : {x, state0, d_y, dstate_out, (const void *)dx, (const void *)dstate0})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    for (const void *p : {weight, bias, (const float *)dweight, (const float *)dbias})
        if (!aligned(p, 4))
            return KDN_ERR_ALIGN;
    const long long n_s = P.pool * (W - 1) * C * es;
    const Range ins[] = {{x, span(tok, P.x_stride, C, es)},
                         {weight, 4LL * C * W},
                         {bias, 4LL * C},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {state0, n_s},
                         {d_y, tok * C * es},
                         {dstate_out, n_s}};
    const Range outs[] = {{dx, tok * C * es},
                          {dweight, 4LL * C * W},
                          {dbias, 4LL * C},
                          {dstate0, n_s}};
    if (clash(outs, 4, ins, 9))
        return KDN_ERR_ALIAS;
    P.parts = (int)grad_parts(P, packed != nullptr);
    const long long n_ws = 4LL * P.parts * (W + 1) * C;
    if (n_ws > 0) {
        if (!workspace || workspace_bytes < (unsigned long long)n_ws)
            return KDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return KDN_ERR_ALIGN;
        const Range ws[] = {{workspace, n_ws}};
        if (clash(ws, 1, ins, 9) || clash(ws, 1, outs, 4))
            return KDN_ERR_ALIAS;
        P.ws = static_cast<float *>(workspace);
    }
    P.x = x; P.weight = weight; P.bias = bias; P.state0 = state0;
    P.d_y = d_y; P.dstate_out = dstate_out;
    P.dx = dx; P.dweight = dweight; P.dbias = dbias; P.dstate0 = dstate0;
    const hipError_t e = kdn::launch_conv_backward(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
