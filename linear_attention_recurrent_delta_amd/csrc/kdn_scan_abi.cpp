// kdn_scan_abi.cpp -- C ABI of the selective state space scan: host-side validation
// of every argument (before any HIP call), then the launches on the caller's stream.
#include "kdn.h"
#include "kdn_batch.h"
#include "kdn_scan.h"

#include <algorithm>

using kdn::aligned;
using kdn::clash;
using kdn::launchable;
using kdn::Range;
using kdn::span;
using kdn::up256;

namespace {

// Workgroups of the outputs' kernel that run at once: one a CU, by its registers.
constexpr int SCAN_WGS = 256;
// Tokens that a workgroup of the outputs' kernel takes at a time.
constexpr int SCAN_STEP = 128;

// Tokens of a block.  A workgroup walks a block for 16 channels, and sequences are cut
// into as many blocks as run at once, where the walk becomes shorter by more than the
// price: another pass of half the work and two launches, together some 4 steps.  bf16,
// 16 states, whole and cut, in us:
//     tokens   16 runs of channels    64          128
//      1000     30    22               29   24     31   34
//      4000    100    31              110   61    112   99
//     16000    390    90              415  204    418  357
int scan_block(long long tokens, int N, int C) {
    const long long runs = (C + kdn::SCAN_CHANNELS - 1) / kdn::SCAN_CHANNELS;
    long long block = tokens;
    const long long len = N > 0 ? (tokens + N - 1) / N : 0;
    const long long blocks = runs * N > 0 ? SCAN_WGS / (runs * N) : 1;
    if (blocks >= 2 && len * (2 * blocks - 3) > 8 * SCAN_STEP * blocks)
        block = std::max((len + blocks - 1) / blocks, (long long)SCAN_STEP);
    block = (std::max(block, 1LL) + 63) / 64 * 64;
    return (int)std::min(block, 1LL << 30);
}

struct Strides {
    long long x, delta, z, B, C;
};

// Elements of a row: 16 rows are below 2^32 bytes.
constexpr long long ROW = 1LL << 25;

kdn_status scan_shape(kdn::ScanParams &P, int dtype, int N, int T, int C, int S, int G,
                      const Strides &st, const kdn_packed *packed) {
    if (!kdn::valid_dtype(dtype))
        return KDN_ERR_UNSUPPORTED;
    if (C < 0 || S < 0 || G < 0 || (C > 0 && (G == 0 || C % G != 0)) || C >= (1 << 24))
        return KDN_ERR_SHAPE;
    if (S != 8 && S != 16 && S != 32)
        return KDN_ERR_UNSUPPORTED;
    P = kdn::ScanParams{};
    if (kdn_status e = kdn::batch_shape(P, N, T, packed))
        return e;
    P.bf16 = dtype == KDN_BF16;
    P.C = C; P.S = S; P.G = std::max(G, 1);
    if (kdn_status e = kdn::row_stride(st.x, C, &P.x_stride, ROW)) return e;
    if (kdn_status e = kdn::row_stride(st.delta, C, &P.d_stride, ROW)) return e;
    if (kdn_status e = kdn::row_stride(st.z, C, &P.z_stride, ROW)) return e;
    if (kdn_status e = kdn::row_stride(st.B, (long long)G * S, &P.b_stride, ROW)) return e;
    if (kdn_status e = kdn::row_stride(st.C, (long long)G * S, &P.c_stride, ROW)) return e;
    if (P.pool * C >= (1LL << 40))
        return KDN_ERR_SHAPE;
    return KDN_OK;
}

// Sequences of several blocks, or of what a packed batch may have.
bool several(const kdn::ScanParams &P, bool packed) {
    return packed ? P.block < P.tokens : P.nblocks > 1;
}

// Blocks of a dense call, and what follows from the blocks' number: the launches of the
// outputs, of the tiles' own states (sequences of several blocks, and the gradients) and of
// the joins.
kdn_status scan_blocks(kdn::ScanParams &P, bool packed, int block, bool back) {
    if (!packed) {
        P.block = block;
        P.nblocks = P.T == 0 ? 0 : (P.T - 1) / block + 1;
    }
    const long long blocks = packed ? P.nblocks : (long long)P.N * P.nblocks;
    P.tile_slots = kdn::tile_slots(P.tokens, blocks, P.S);
    if (blocks >= (1LL << 32) || P.tile_slots * P.C >= (1LL << 40))
        return KDN_ERR_SHAPE;
    // grids have fours of runs: a wave each of the outputs, a workgroup each of the own
    // states, with a few thousand workgroups more where there are less
    const long long runs = P.C > 0 ? (long long)kdn::scan_groups(P.C, P.G) * P.G : 0;
    const long long fours = blocks * ((runs + 3) / 4);
    const long long pieces = ((long long)P.C * P.S / 2 + 255) / 256;
    if (!launchable(fours + 1024, 256) || !launchable((back ? 2LL : 1LL) * P.N * pieces, 256) ||
        ((back || several(P, packed)) && !launchable(4 * fours + (1 << 15), 256)))
        return KDN_ERR_SHAPE;
    return KDN_OK;
}

// Workspace of the tiles' states and sums of time steps.
long long state_bytes(const kdn::ScanParams &P) { return up256(P.tile_slots * P.C * P.S * 4); }
long long dt_bytes(const kdn::ScanParams &P) { return up256(P.tile_slots * P.C * 4); }

// Blocks of the gradients: a wave a tile in the pass over the tiles' own states.  Of 128,
// 256 and 512 tokens: B2 T4096 C2048 bf16 366, 354 and 351 us, 11 packed sequences of 518
// channels in float32 207, 205 and 207.
constexpr int GRAD_BLOCK = 256;
// Workgroups of the gradients' kernel that run at once: one a CU (with two of them shared
// out B2 T4096 C2048 is 360 us where it is 354, B1 T1000 C1024 68 where it is 52).
constexpr int GRAD_WGS = 256;
// Tiles whose sums over tokens a wave of a workgroup adds in float32 (on average, where a
// packed batch is uneven).
constexpr int PART_TILES = 256;

// How the gradients' work is shared out: runs of 16 channels for a workgroup, as many
// as leave two workgroups a CU, since the sums over channels cost each set of runs the
// same; then workgroups for the tiles of a set, as many as run at once, and whole times
// that many of long batches, so that no float32 sum is a chain that grows with the tokens.
void grad_shares(kdn::ScanParams &P, bool packed) {
    const int tile = kdn::scan_tile(P.S);
    const long long blocks = packed ? P.nblocks : (long long)P.N * P.nblocks;
    const long long tiles = P.tokens / tile + (packed ? std::min<long long>(P.N, P.tokens) : P.N);
    const int groups = P.C > 0 ? kdn::scan_groups(P.C, P.G) : 0;
    P.per_set = kdn::scan_per_set(P.S);
    while (P.per_set > 1 &&
           (groups + P.per_set - 1LL) / P.per_set * P.G * tiles < 2 * GRAD_WGS)
        P.per_set /= 2;
    const long long sets = groups > 0 ? (long long)kdn::scan_sets(P) * P.G : 0;
    const long long in_block = std::min<long long>(P.block, std::max<long long>(P.tokens, 1));
    const long long per_block = (in_block + tile - 1) / tile;
    const long long once = sets > 0 ? std::max(1LL, GRAD_WGS / sets) : 0;
    const long long parts = once * std::max(1LL, once > 0 ? (tiles - 1) / (once * PART_TILES) + 1 : 0);
    P.classes = (int)std::min(per_block, blocks > 0 ? (4 * parts + blocks - 1) / blocks : 1);
    P.parts = (int)std::min(parts, blocks * P.classes);
}

struct GradWs {
    long long state, rstate, dt, bc, sum, total;
};
GradWs grad_ws(const kdn::ScanParams &P) {
    GradWs w{};
    if (P.parts == 0)
        return w;
    long long o = 0;
    auto take = [&](long long n) {
        const long long at = o;
        o += up256(n);
        return at;
    };
    w.state = take(state_bytes(P));
    w.rstate = take(state_bytes(P));
    w.dt = take(dt_bytes(P));
    w.bc = take(4LL * kdn::scan_sets(P) * P.tokens * P.G * 2 * P.S);
    w.sum = take(4LL * P.parts * P.C * (P.S + 2));
    w.total = o;
    return w;
}

kdn_status done(hipError_t e) { return e == hipSuccess ? KDN_OK : KDN_ERR_HIP; }

}  // namespace

extern "C" {

int kdn_selective_block(int tokens, int N, int C, int S) {
    if (tokens < 0 || N < 0 || C < 0 || S < 0)
        return -1;
    return scan_block(tokens, N, C);
}

unsigned long long kdn_selective_scan_workspace_size(kdn_dtype dtype, int N, int T, int C, int S,
                                                     int G, const kdn_packed *packed,
                                                     kdn_status *status) {
    kdn::ScanParams P;
    kdn_status st = scan_shape(P, dtype, N, T, C, S, G, Strides{}, packed);
    if (st == KDN_OK)
        st = scan_blocks(P, packed != nullptr, scan_block(P.tokens, N, C), false);
    if (status)
        *status = st;
    return st == KDN_OK && C > 0 && several(P, packed != nullptr)
               ? (unsigned long long)(state_bytes(P) + dt_bytes(P)) : 0;
}

kdn_status kdn_selective_scan(kdn_dtype dtype, int N, int T, int C, int S, int G, int softplus,
                              long long x_stride, long long delta_stride, long long z_stride,
                              long long B_stride, long long C_stride, const void *x,
                              const void *delta, const float *A, const void *B, const void *Cm,
                              const float *D, const void *z, const float *delta_bias,
                              const float *S0, void *y, float *S_out, const kdn_packed *packed,
                              void *workspace, unsigned long long workspace_bytes, void *stream) {
    kdn::ScanParams P;
    if (kdn_status st = scan_shape(P, dtype, N, T, C, S, G,
                                   Strides{x_stride, delta_stride, z_stride, B_stride, C_stride}, packed))
        return st;
    if (kdn_status st = scan_blocks(P, packed != nullptr, scan_block(P.tokens, N, C), false))
        return st;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens, gs = (long long)G * S;
    if (tok * C > 0 && (!x || !delta || !A || !B || !Cm || !y))
        return KDN_ERR_NULL;
    if (kdn_status st = kdn::batch_tables(P, packed))
        return st;
    for (const void *p : {x, delta, z, B, Cm, (const void *)y})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    if (!aligned(A, 16) || !aligned(S0, 16) || !aligned(S_out, 16) || !aligned(D, 4) ||
        !aligned(delta_bias, 4))
        return KDN_ERR_ALIGN;
    const long long n_S = P.pool * C * S * 4;
    const Range ins[] = {{x, span(tok, P.x_stride, C, es)},
                         {delta, span(tok, P.d_stride, C, es)},
                         {z, span(tok, P.z_stride, C, es)},
                         {B, span(tok, P.b_stride, gs, es)},
                         {Cm, span(tok, P.c_stride, gs, es)},
                         {A, 4LL * C * S},
                         {D, 4LL * C},
                         {delta_bias, 4LL * C},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {S0 == S_out ? nullptr : S0, n_S}};
    const Range outs[] = {{y, tok * C * es}, {S_out, n_S}};
    if (clash(outs, 2, ins, 12))
        return KDN_ERR_ALIAS;
    const bool many = several(P, packed != nullptr);
    const long long n_ws = many && C > 0 ? state_bytes(P) + dt_bytes(P) : 0;
    if (n_ws > 0) {
        if (!workspace || workspace_bytes < (unsigned long long)n_ws)
            return KDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return KDN_ERR_ALIGN;
        const Range ws[] = {{workspace, n_ws}};
        if (clash(ws, 1, ins, 12) || clash(ws, 1, outs, 2) || kdn::overlap(workspace, n_ws, S0, n_S))
            return KDN_ERR_ALIAS;
        P.ws_state = static_cast<float *>(workspace);
        P.ws_dt = reinterpret_cast<float *>(static_cast<char *>(workspace) + state_bytes(P));
    }
    P.softplus = softplus != 0;
    P.x = x; P.delta = delta; P.z = z; P.B = B; P.Cm = Cm; P.A = A; P.D = D; P.bias = delta_bias;
    P.S0 = S0; P.y = y; P.S_out = S_out;
    return done(kdn::launch_scan(P, many, static_cast<hipStream_t>(stream)));
}

kdn_status kdn_selective_decode(kdn_dtype dtype, int N, int C, int S, int G, int softplus,
                                long long x_stride, long long delta_stride, long long z_stride,
                                long long B_stride, long long C_stride, const void *x,
                                const void *delta, const float *A, const void *B, const void *Cm,
                                const float *D, const void *z, const float *delta_bias,
                                const int *slots, int pool, float *state, void *y, void *stream) {
    kdn::ScanParams L;
    if (kdn_status st = scan_shape(L, dtype, N, 1, C, S, G,
                                   Strides{x_stride, delta_stride, z_stride, B_stride, C_stride}, nullptr))
        return st;
    if (pool < 0 || (!slots && pool < N) || (long long)pool * C >= (1LL << 40) ||
        !launchable((long long)N * ((C + 63) / 64), 256))
        return KDN_ERR_SHAPE;
    const long long es = L.bf16 ? 2 : 4, n = (long long)N * C, gs = (long long)G * S;
    if (n > 0 && (!x || !delta || !A || !B || !Cm || !y || (pool > 0 && !state)))
        return KDN_ERR_NULL;
    for (const void *p : {x, delta, z, B, Cm, (const void *)y})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    if (!aligned(A, 16) || !aligned(state, 16) || !aligned(D, 4) || !aligned(delta_bias, 4) ||
        !aligned(slots, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{x, span(N, L.x_stride, C, es)},
                         {delta, span(N, L.d_stride, C, es)},
                         {z, span(N, L.z_stride, C, es)},
                         {B, span(N, L.b_stride, gs, es)},
                         {Cm, span(N, L.c_stride, gs, es)},
                         {A, 4LL * C * S},
                         {D, 4LL * C},
                         {delta_bias, 4LL * C},
                         {slots, 4LL * N}};
    const Range outs[] = {{y, n * es}, {state, (long long)pool * C * S * 4}};
    if (clash(outs, 2, ins, 9))
        return KDN_ERR_ALIAS;
    kdn::ScanDecodeParams P;
    P.bf16 = L.bf16;
    P.N = N; P.C = C; P.S = S; P.G = L.G; P.softplus = softplus != 0;
    P.x_stride = L.x_stride; P.d_stride = L.d_stride; P.z_stride = L.z_stride;
    P.b_stride = L.b_stride; P.c_stride = L.c_stride;
    P.x = x; P.delta = delta; P.z = z; P.B = B; P.Cm = Cm; P.A = A; P.D = D; P.bias = delta_bias;
    P.slots = slots; P.pool = pool; P.state = state; P.y = y;
    return done(kdn::launch_scan_decode(P, static_cast<hipStream_t>(stream)));
}

unsigned long long kdn_selective_scan_backward_workspace_size(kdn_dtype dtype, int N, int T, int C,
                                                              int S, int G,
                                                              const kdn_packed *packed,
                                                              kdn_status *status) {
    kdn::ScanParams P;
    kdn_status st = scan_shape(P, dtype, N, T, C, S, G, Strides{}, packed);
    if (st == KDN_OK)
        st = scan_blocks(P, packed != nullptr, GRAD_BLOCK, true);
    if (status)
        *status = st;
    if (st != KDN_OK)
        return 0;
    grad_shares(P, packed != nullptr);
    return (unsigned long long)grad_ws(P).total;
}

kdn_status kdn_selective_scan_backward(kdn_dtype dtype, int N, int T, int C, int S, int G,
                                       int softplus, long long x_stride, long long delta_stride,
                                       long long z_stride, long long B_stride, long long C_stride,
                                       const void *x, const void *delta, const float *A,
                                       const void *B, const void *Cm, const float *D,
                                       const void *z, const float *delta_bias, const float *S0,
                                       const void *d_y, const float *dS_out, void *dx,
                                       void *ddelta, float *dA, void *dB, void *dC, float *dD,
                                       void *dz, float *ddelta_bias, float *dS0,
                                       const kdn_packed *packed, void *workspace,
                                       unsigned long long workspace_bytes, void *stream) {
    kdn::ScanParams P;
    if (kdn_status st = scan_shape(P, dtype, N, T, C, S, G,
                                   Strides{x_stride, delta_stride, z_stride, B_stride, C_stride}, packed))
        return st;
    if (kdn_status st = scan_blocks(P, packed != nullptr, GRAD_BLOCK, true))
        return st;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens, gs = (long long)G * S;
    if (!launchable(((long long)C * (S + 2) + 63) / 64 + (tok * gs * 2 + 255) / 256 + 64, 256))
        return KDN_ERR_SHAPE;
    if ((tok * C > 0 && (!x || !delta || !B || !Cm || !d_y || !dx || !ddelta || (z && !dz))) ||
        (tok * gs > 0 && (!dB || !dC)) || (C > 0 && (!A || !dA)) || (!z && dz))
        return KDN_ERR_NULL;
    if (kdn_status st = kdn::batch_tables(P, packed))
        return st;
    for (const void *p : {x, delta, z, B, Cm, d_y, (const void *)dx, (const void *)ddelta,
                          (const void *)dB, (const void *)dC, (const void *)dz})
        if (!aligned(p, es))
            return KDN_ERR_ALIGN;
    for (const void *p : {(const void *)A, (const void *)S0, (const void *)dS_out, (const void *)dS0})
        if (!aligned(p, 16))
            return KDN_ERR_ALIGN;
    for (const float *p : {D, delta_bias, (const float *)dA, (const float *)dD,
                           (const float *)ddelta_bias})
        if (!aligned(p, 4))
            return KDN_ERR_ALIGN;
    const long long n_S = P.pool * C * S * 4;
    const Range ins[] = {{x, span(tok, P.x_stride, C, es)},
                         {delta, span(tok, P.d_stride, C, es)},
                         {z, span(tok, P.z_stride, C, es)},
                         {B, span(tok, P.b_stride, gs, es)},
                         {Cm, span(tok, P.c_stride, gs, es)},
                         {A, 4LL * C * S},
                         {D, 4LL * C},
                         {delta_bias, 4LL * C},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {S0, n_S},
                         {d_y, tok * C * es},
                         {dS_out, n_S}};
    const Range outs[] = {{dx, tok * C * es}, {ddelta, tok * C * es}, {dA, 4LL * C * S},
                          {dB, tok * gs * es}, {dC, tok * gs * es}, {dD, 4LL * C},
                          {dz, tok * C * es}, {ddelta_bias, 4LL * C}, {dS0, n_S}};
    if (clash(outs, 9, ins, 14))
        return KDN_ERR_ALIAS;
    grad_shares(P, packed != nullptr);
    if (!launchable((long long)P.parts * kdn::scan_sets(P) * P.G, 512))
        return KDN_ERR_SHAPE;
    const GradWs w = grad_ws(P);
    if (w.total > 0) {
        if (!workspace || workspace_bytes < (unsigned long long)w.total)
            return KDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return KDN_ERR_ALIGN;
        const Range ws[] = {{workspace, w.total}};
        if (clash(ws, 1, ins, 14) || clash(ws, 1, outs, 9))
            return KDN_ERR_ALIAS;
        auto f32 = [&](long long at) {
            return reinterpret_cast<float *>(static_cast<char *>(workspace) + at);
        };
        P.ws_state = f32(w.state);
        P.ws_rstate = f32(w.rstate);
        P.ws_dt = f32(w.dt);
        P.ws_bc = f32(w.bc);
        P.ws_sum = f32(w.sum);
    }
    P.softplus = softplus != 0;
    P.x = x; P.delta = delta; P.z = z; P.B = B; P.Cm = Cm; P.A = A; P.D = D; P.bias = delta_bias;
    P.S0 = S0; P.d_y = d_y; P.dS_out = dS_out;
    P.dx = dx; P.ddelta = ddelta; P.dA = dA;
    P.dB = gs > 0 ? dB : nullptr; P.dC = dC; P.dD = dD; P.dz = dz;
    P.dbias = ddelta_bias; P.dS0 = dS0;
    return done(kdn::launch_scan_backward(P, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
