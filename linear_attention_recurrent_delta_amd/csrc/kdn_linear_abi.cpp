// kdn_linear_abi.cpp -- C ABI of the linear-attention entry points and of the
// packed-batch tables: host-side validation of every argument (before any HIP
// call), then the launches on the caller's stream.
#include "kdn.h"
#include "kdn_check.h"
#include "kdn_linear.h"

#include <initializer_list>
#include <limits.h>

using kdn::aligned;
using kdn::overlap;

namespace {

struct Range {
    const void *p;
    long long n;
};

long long up256(long long n) { return (n + 255) / 256 * 256; }

// Workgroups that dense blocks are cut for: the 256 CUs hold two each of the
// prefill's kernels (LDS), and one of the gradients' walk (of 128 x 128 registers
// and LDS; of 64 x 64 two would fit).
constexpr int PREFILL_WGS = 512, GRAD_WGS = 256;

// Tokens of a block: as many blocks as workgroups run at once.  Below that the
// longest chain counts: the chunks of a block twice (its own state and its
// outputs, 3.5 us a chunk of 64 each) and the join over the sequence's blocks
// (1.5 us for 8), least at a block of about sqrt(2 tokens); up to 256 tokens a
// bfloat16 prefill is as quick in one block as in three launches.
// The rule is the bfloat16 prefill's.  us a call of 256 tokens (one block) and of
// 257 (blocks of 64), H4, 64 x 64 / 128 x 128: bf16 prefill 11.2 / 16.2 and 16.9 /
// 17.3; float32 prefill, in chunks of 32, 32 / 62 and 20 / 32; gradients bf16 33 /
// 43 and 35 / 35, float32 66 / 153 and 35 / 62.  float32 calls would be quicker cut
// from about 128 tokens on, bf16 gradients from about 192.
int dense_block(int tokens, int N, int H, int wgs) {
    const long long full = ((long long)tokens * H + wgs - 1) / wgs;
    const long long len = N > 0 ? tokens / N : 0;
    long long chain = 64;
    while (chain * chain < 2 * len)
        chain += 64;
    if (len <= 256)
        chain = 256;
    const long long block = ((full > chain ? full : chain) + 63) / 64 * 64;
    return (int)(block > (1 << 30) ? (1 << 30) : block);
}

// Sizes common to the prefill and its gradients; fills the sizes of P.  `wgs`: the
// workgroups that dense blocks are cut for.
kdn_status linear_shape(kdn::LinearParams &P, int dtype, int N, int T, int H, int Hq, int Hk,
                        int Hv, int d_k, int d_v, int gate, const kdn_packed *packed, int wgs) {
    if (!kdn::valid_dtype(dtype) || (gate != KDN_GATE_TOKEN && gate != KDN_GATE_HEAD))
        return KDN_ERR_UNSUPPORTED;
    if (N < 0 || T < 0 || H < 0 || Hq < 0 || Hk < 0 || Hv < 0 || d_k <= 0 || d_v <= 0)
        return KDN_ERR_SHAPE;
    for (int x : {Hq, Hk, Hv})
        if (H > 0 && (x == 0 || H % x != 0))
            return KDN_ERR_SHAPE;
    const long long tokens = packed ? packed->tokens : (long long)N * T;
    if (tokens > INT_MAX)
        return KDN_ERR_SHAPE;
    P = kdn::LinearParams{};
    if (packed) {
        if (T != 0 || tokens < 0 || packed->pool < 0 || packed->max_blocks < 0 ||
            packed->max_blocks != kdn_sequence_max_blocks(N, packed->tokens, packed->block))
            return KDN_ERR_SHAPE;
        P.block = packed->block;
        P.nblocks = packed->max_blocks;
        P.pool = packed->pool;
    } else {
        P.block = dense_block((int)tokens, N, H, wgs);
        P.nblocks = T == 0 ? 0 : (T - 1) / P.block + 1;
        P.pool = N;
    }
    const long long blocks = packed ? P.nblocks : (long long)N * P.nblocks;
    if (tokens * H * (d_k > d_v ? d_k : d_v) >= (1LL << 40) || 2 * blocks * H > INT_MAX ||
        (long long)N * H > INT_MAX / 64 || P.pool * H >= (1LL << 40))
        return KDN_ERR_SHAPE;
    if (!kdn::valid_dim(d_k) || !kdn::valid_dim(d_v))
        return KDN_ERR_UNSUPPORTED;
    P.bf16 = dtype == KDN_BF16;
    P.N = N; P.T = T; P.H = H; P.Hq = Hq; P.Hk = Hk; P.Hv = Hv; P.dk = d_k; P.dv = d_v;
    P.gate = gate;
    P.tokens = tokens;
    return KDN_OK;
}

// A launch has less than 2^32 work-items: of more the runtime starts what their
// low 32 bits say, and reports no error.
bool launchable(long long workgroups, int threads) { return workgroups * threads < (1LL << 32); }

// Elements between tokens (0: contiguous), or an error.
kdn_status token_stride(long long given, long long row, long long es, long *out) {
    if (given == 0)
        given = row;
    // the rows of a chunk (64 bfloat16, 32 float32) lie within 2^32 bytes
    if (given < row || given * es >= (1LL << 26))
        return KDN_ERR_SHAPE;
    if (given * es % 16 != 0)
        return KDN_ERR_ALIGN;
    *out = given;
    return KDN_OK;
}

// Bytes from the first to the last element of `rows` strided rows.
long long span(long long rows, long stride, long long row, long long es) {
    return rows > 0 ? ((rows - 1) * stride + row) * es : 0;
}

// Workspace sections: states at the blocks' starts, and the blocks' decays with
// a packed batch's order behind them; nothing where every sequence is known to
// be one block.
long long state_sections(const kdn::LinearParams &P, bool packed, long long *decay) {
    const long long blocks = packed ? P.nblocks : (long long)P.N * P.nblocks;
    if (!packed && P.nblocks <= 1)
        return 0;
    const long long n = up256(blocks * P.H * P.dk * P.dv * 4);
    *decay = n;
    return n + up256(blocks * (P.H + packed) * 4);
}

// Outputs overlap no input and no other output.
bool clash(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return true;
    }
    return false;
}

// The packed tables' pointers.
kdn_status packed_tables(kdn::LinearParams &P, const kdn_packed *packed) {
    if (!packed)
        return KDN_OK;
    if (P.N + P.tokens > 0 && !packed->block_offsets)
        return KDN_ERR_NULL;
    if (P.nblocks > 0 && !packed->blocks)
        return KDN_ERR_NULL;
    if (!aligned(packed->blocks, 16) || !aligned(packed->block_offsets, 4) ||
        !aligned(packed->slots, 4))
        return KDN_ERR_ALIGN;
    P.blocks = packed->blocks;
    P.block_offsets = packed->block_offsets;
    P.slots = packed->slots;
    return KDN_OK;
}

}  // namespace

extern "C" {

int kdn_sequence_max_blocks(int N, int tokens, int block) {
    if (N < 0 || tokens < 0 || block <= 0 || block % 64 != 0)
        return -1;
    if (N == 0)
        return 0;
    // sum of ceil(len / block) over N lengths that sum to tokens at most
    const long long n = (long long)tokens / block + N;
    return (int)(n < tokens ? n : tokens);
}

int kdn_linear_block(int tokens, int N, int H) {
    if (tokens < 0 || N < 0 || H < 0)
        return -1;
    return dense_block(tokens, N, H, PREFILL_WGS);
}

kdn_status kdn_sequence_tables(int N, int tokens, int block, int max_blocks, const int *lengths,
                               const int *slots, const int *context, int *offsets,
                               int *block_offsets, int *blocks, int *slot_map, int *positions,
                               void *stream) {
    if (N < 0 || tokens < 0 || block <= 0 || block % 64 != 0 ||
        max_blocks != kdn_sequence_max_blocks(N, tokens, block))
        return KDN_ERR_SHAPE;
    if (!offsets || !block_offsets || (N > 0 && !lengths) || (max_blocks > 0 && !blocks))
        return KDN_ERR_NULL;
    for (const void *x : {(const void *)lengths, (const void *)slots, (const void *)context,
                          (const void *)offsets, (const void *)block_offsets,
                          (const void *)slot_map, (const void *)positions})
        if (!aligned(x, 4))
            return KDN_ERR_ALIGN;
    if (!aligned(blocks, 16))
        return KDN_ERR_ALIGN;
    const long long n = 4LL * N;
    const Range ins[] = {{lengths, n}, {slots, n}, {context, n}};
    const Range outs[] = {{offsets, n + 4}, {block_offsets, n + 4}, {blocks, 16LL * max_blocks},
                          {slot_map, 4LL * tokens}, {positions, 4LL * tokens}};
    if (clash(outs, 5, ins, 3))
        return KDN_ERR_ALIAS;
    kdn::TableParams P;
    P.N = N; P.tokens = tokens; P.block = block; P.max_blocks = max_blocks;
    P.lengths = lengths; P.slots = slots; P.context = context;
    P.offsets = offsets; P.block_offsets = block_offsets; P.blocks = blocks;
    P.slot_map = slot_map; P.positions = positions;
    const hipError_t e = kdn::launch_sequence_tables(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

unsigned long long kdn_linear_prefill_workspace_size(kdn_dtype dtype, int N, int T, int H,
                                                     int d_k, int d_v, const kdn_packed *packed,
                                                     kdn_status *status) {
    kdn::LinearParams P;
    const kdn_status st = linear_shape(P, dtype, N, T, H, H, H, H, d_k, d_v, KDN_GATE_TOKEN, packed,
                                       PREFILL_WGS);
    if (status)
        *status = st;
    long long decay;
    return st == KDN_OK ? (unsigned long long)state_sections(P, packed != nullptr, &decay) : 0;
}

kdn_status kdn_linear_prefill(kdn_dtype dtype, int N, int T, int H, int Hq, int Hk, int Hv,
                              int d_k, int d_v, kdn_gate gate, long long q_stride,
                              long long k_stride, long long v_stride, const void *q,
                              const void *k, const void *v, const void *log_alpha,
                              const float *S0, void *o, float *S_out, const kdn_packed *packed,
                              void *workspace, unsigned long long workspace_bytes,
                              void *stream) {
    kdn::LinearParams P;
    if (kdn_status st = linear_shape(P, dtype, N, T, H, Hq, Hk, Hv, d_k, d_v, gate, packed,
                                         PREFILL_WGS))
        return st;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens;
    if (kdn_status st = token_stride(q_stride, (long long)Hq * d_k, es, &P.q_stride)) return st;
    if (kdn_status st = token_stride(k_stride, (long long)Hk * d_k, es, &P.k_stride)) return st;
    if (kdn_status st = token_stride(v_stride, (long long)Hv * d_v, es, &P.v_stride)) return st;
    if (kdn_status st = token_stride(0, (long long)H * d_v, es, &P.o_stride)) return st;
    if (tok * H > 0 && (!q || !k || !v || !log_alpha || !o))
        return KDN_ERR_NULL;
    if (kdn_status st = packed_tables(P, packed))
        return st;
    // the walks; sequences of several blocks (or none): the joins
    const bool several = packed || P.nblocks != 1;
    const long long wgs = kdn::linear_total_blocks(P) * H / (kdn::linear_pairs(P) ? 2 : 1);
    if (!launchable(wgs, 256) || (several && !launchable((long long)N * H + 1, 256)))
        return KDN_ERR_SHAPE;
    for (const void *x : {q, k, v, (const void *)S0, (const void *)o, (const void *)S_out})
        if (!aligned(x, 16))
            return KDN_ERR_ALIGN;
    if (!aligned(log_alpha, gate == KDN_GATE_HEAD ? 4 : es))
        return KDN_ERR_ALIGN;
    const long long n_S = P.pool * H * d_k * d_v * 4;
    const Range ins[] = {{q, span(tok, P.q_stride, (long long)Hq * d_k, es)},
                         {k, span(tok, P.k_stride, (long long)Hk * d_k, es)},
                         {v, span(tok, P.v_stride, (long long)Hv * d_v, es)},
                         {log_alpha, gate == KDN_GATE_HEAD ? 4LL * H : tok * H * es},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {S0 == S_out ? nullptr : S0, n_S}};
    const Range outs[] = {{o, tok * H * d_v * es}, {S_out, n_S}};
    if (clash(outs, 2, ins, 8))
        return KDN_ERR_ALIAS;
    long long decay = 0;
    const long long n_ws = state_sections(P, packed != nullptr, &decay);
    if (n_ws > 0) {
        if (!workspace || workspace_bytes < (unsigned long long)n_ws)
            return KDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return KDN_ERR_ALIGN;
        const Range ws[] = {{workspace, n_ws}};
        if (clash(ws, 1, ins, 8) || clash(ws, 1, outs, 2) || overlap(workspace, n_ws, S0, n_S))
            return KDN_ERR_ALIAS;
        P.ws_state = static_cast<float *>(workspace);
        P.ws_decay = reinterpret_cast<float *>(static_cast<char *>(workspace) + decay);
        if (packed)
            P.ws_order = reinterpret_cast<int *>(P.ws_decay + (long)P.nblocks * H);
    }
    P.q = q; P.k = k; P.v = v; P.la = log_alpha;
    P.S0 = S0; P.o = o; P.S_out = S_out;
    const hipError_t e = kdn::launch_linear_prefill(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

kdn_status kdn_linear_decode(kdn_dtype dtype, int N, int H, int Hq, int Hk, int Hv, int d_k,
                             int d_v, kdn_gate gate, long long q_stride, long long k_stride,
                             long long v_stride, const void *q, const void *k, const void *v,
                             const void *log_alpha, const int *slots, int pool, float *S,
                             void *o, void *stream) {
    kdn::LinearParams L;
    if (kdn_status st = linear_shape(L, dtype, N, 1, H, Hq, Hk, Hv, d_k, d_v, gate, nullptr,
                                         PREFILL_WGS))
        return st;
    const long long es = L.bf16 ? 2 : 4, nh = (long long)N * H;
    if (pool < 0 || (!slots && pool < N) || (long long)pool * H >= (1LL << 40) ||
        !launchable(nh, 256))
        return KDN_ERR_SHAPE;
    if (kdn_status st = token_stride(q_stride, (long long)Hq * d_k, es, &L.q_stride)) return st;
    if (kdn_status st = token_stride(k_stride, (long long)Hk * d_k, es, &L.k_stride)) return st;
    if (kdn_status st = token_stride(v_stride, (long long)Hv * d_v, es, &L.v_stride)) return st;
    if (nh > 0 && (!q || !k || !v || !log_alpha || !o || (pool > 0 && !S)))
        return KDN_ERR_NULL;
    for (const void *x : {q, k, v, (const void *)S, (const void *)o})
        if (!aligned(x, 16))
            return KDN_ERR_ALIGN;
    if (!aligned(log_alpha, gate == KDN_GATE_HEAD ? 4 : es) || !aligned(slots, 4))
        return KDN_ERR_ALIGN;
    const Range ins[] = {{q, span(N, L.q_stride, (long long)Hq * d_k, es)},
                         {k, span(N, L.k_stride, (long long)Hk * d_k, es)},
                         {v, span(N, L.v_stride, (long long)Hv * d_v, es)},
                         {log_alpha, gate == KDN_GATE_HEAD ? 4LL * H : nh * es},
                         {slots, 4LL * N}};
    const Range outs[] = {{o, nh * d_v * es}, {S, (long long)pool * H * d_k * d_v * 4}};
    if (clash(outs, 2, ins, 5))
        return KDN_ERR_ALIAS;
    kdn::LinearDecodeParams P;
    P.bf16 = L.bf16;
    P.N = N; P.H = H; P.Hq = Hq; P.Hk = Hk; P.Hv = Hv; P.dk = d_k; P.dv = d_v; P.gate = gate;
    P.q_stride = L.q_stride; P.k_stride = L.k_stride; P.v_stride = L.v_stride;
    P.q = q; P.k = k; P.v = v; P.la = log_alpha;
    P.slots = slots; P.pool = pool; P.S = S; P.o = o;
    const hipError_t e = kdn::launch_linear_decode(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

// ---------------------------------------------------------------------------
// Gradients.
// ---------------------------------------------------------------------------
namespace {
// Workspace, sections 256-byte aligned: the forward and the reverse states at
// the blocks' ends with the blocks' decays (sequences of several blocks; a
// packed batch's order behind the decays), the state at every chunk's start
// (where `fine`: what its rounding leaves, too), float32 gradients of shared
// heads before their sum, and for one decay per head each block's sum.
//
// fine: d log_alpha of a bfloat16 call beyond its operands' rounding, for the sum
// over tokens of one decay per head and for dense sequences of one chunk
// (kdn_linear_backward.hip).
bool fine(const kdn::LinearParams &P, bool packed) {
    return P.bf16 && (P.gate == KDN_GATE_HEAD || (!packed && P.T <= kdn::linear_chunk(true)));
}
struct GradWs {
    long long state, decay, rstate, rdecay, chunk, chunk_lo, dq, dk, dv, dla, total;
};
GradWs grad_ws(const kdn::LinearParams &P, bool packed) {
    GradWs w{};
    const long long blocks = packed ? P.nblocks : (long long)P.N * P.nblocks;
    if (blocks * P.H == 0)
        return w;
    const long long n_S = (long long)P.dk * P.dv, es = P.bf16 ? 2 : 4;
    long long o = 0;
    auto take = [&](long long n) {
        const long long at = o;
        o += up256(n);
        return at;
    };
    if (packed || P.nblocks > 1) {
        w.state = take(blocks * P.H * n_S * 4);
        w.decay = take(blocks * (P.H + packed) * 4);
        w.rstate = take(blocks * P.H * n_S * 4);
        w.rdecay = take(blocks * P.H * 4);
    }
    const long long n_chunk =
        kdn::chunk_slots(P.tokens, blocks, kdn::linear_chunk(P.bf16)) * P.H * n_S * es;
    w.chunk = take(n_chunk);
    if (fine(P, packed))
        w.chunk_lo = take(n_chunk);
    if (P.Hq != P.H)
        w.dq = take(P.tokens * P.H * P.dk * 4);
    if (P.Hk != P.H)
        w.dk = take(P.tokens * P.H * P.dk * 4);
    if (P.Hv != P.H)
        w.dv = take(P.tokens * P.H * P.dv * 4);
    if (P.gate == KDN_GATE_HEAD)
        w.dla = take(blocks * P.H * 8);
    w.total = o;
    return w;
}
}  // namespace

unsigned long long kdn_linear_prefill_backward_workspace_size(
    kdn_dtype dtype, int N, int T, int H, int Hq, int Hk, int Hv, int d_k, int d_v, kdn_gate gate,
    const kdn_packed *packed, kdn_status *status) {
    if (gate == KDN_GATE_HEAD_F32)
        gate = KDN_GATE_HEAD;
    kdn::LinearParams P;
    const kdn_status st = linear_shape(P, dtype, N, T, H, Hq, Hk, Hv, d_k, d_v, gate, packed,
                                         GRAD_WGS);
    if (status)
        *status = st;
    return st == KDN_OK ? (unsigned long long)grad_ws(P, packed != nullptr).total : 0;
}

kdn_status kdn_linear_prefill_backward(kdn_dtype dtype, int N, int T, int H, int Hq, int Hk,
                                       int Hv, int d_k, int d_v, kdn_gate gate,
                                       long long q_stride, long long k_stride,
                                       long long v_stride, const void *q, const void *k,
                                       const void *v, const void *log_alpha, const float *S0,
                                       const void *d_o, const float *dS_out, void *dq, void *dk,
                                       void *dv, void *dlog_alpha, float *dS0,
                                       const kdn_packed *packed, void *workspace,
                                       unsigned long long workspace_bytes, void *stream) {
    const bool dla_f32 = gate == KDN_GATE_HEAD_F32;
    if (dla_f32)
        gate = KDN_GATE_HEAD;
    kdn::LinearParams P;
    if (kdn_status st = linear_shape(P, dtype, N, T, H, Hq, Hk, Hv, d_k, d_v, gate, packed,
                                         GRAD_WGS))
        return st;
    const long long es = P.bf16 ? 2 : 4, tok = P.tokens;
    if (kdn_status st = token_stride(q_stride, (long long)Hq * d_k, es, &P.q_stride)) return st;
    if (kdn_status st = token_stride(k_stride, (long long)Hk * d_k, es, &P.k_stride)) return st;
    if (kdn_status st = token_stride(v_stride, (long long)Hv * d_v, es, &P.v_stride)) return st;
    if (kdn_status st = token_stride(0, (long long)H * d_v, es, &P.o_stride)) return st;
    if (tok * H > 0 && (!q || !k || !v || !log_alpha || !d_o || !dq || !dk || !dv))
        return KDN_ERR_NULL;
    if (kdn_status st = packed_tables(P, packed))
        return st;
    // the walk; sequences of several blocks (or none): the blocks' own states and
    // the joins, both directions, with the packed tail; the shared heads' sums
    const long long wgs = kdn::linear_total_blocks(P) * H;
    const bool several = packed || P.nblocks != 1;
    const long long shared = tok * ((Hq != H ? (long long)Hq * d_k : 0) +
                                    (Hk != H ? (long long)Hk * d_k : 0) +
                                    (Hv != H ? (long long)Hv * d_v : 0)) / 4;
    if (!launchable(wgs, 4 * (d_k > d_v ? d_k : d_v)) || (several && !launchable(2 * wgs, 256)) ||
        (several && !launchable(2LL * N * H + 128, 256)) || !launchable(shared / 256 + 1, 256))
        return KDN_ERR_SHAPE;
    for (const void *x : {q, k, v, (const void *)S0, d_o, (const void *)dS_out, (const void *)dq,
                          (const void *)dk, (const void *)dv, (const void *)dS0})
        if (!aligned(x, 16))
            return KDN_ERR_ALIGN;
    if (!aligned(log_alpha, gate == KDN_GATE_HEAD ? 4 : es) ||
        !aligned(dlog_alpha, dla_f32 ? 4 : es))
        return KDN_ERR_ALIGN;
    const long long n_S = P.pool * H * d_k * d_v * 4;
    const long long n_la = gate == KDN_GATE_HEAD ? 4LL * H : tok * H * es;
    const Range ins[] = {{q, span(tok, P.q_stride, (long long)Hq * d_k, es)},
                         {k, span(tok, P.k_stride, (long long)Hk * d_k, es)},
                         {v, span(tok, P.v_stride, (long long)Hv * d_v, es)},
                         {log_alpha, n_la},
                         {P.blocks, packed ? 16LL * P.nblocks : 0},
                         {P.block_offsets, packed ? 4LL * (N + 1) : 0},
                         {P.slots, packed ? 4LL * N : 0},
                         {S0, n_S},
                         {d_o, tok * H * d_v * es},
                         {dS_out, n_S}};
    const Range outs[] = {{dq, tok * Hq * d_k * es},
                          {dk, tok * Hk * d_k * es},
                          {dv, tok * Hv * d_v * es},
                          {dlog_alpha, gate == KDN_GATE_HEAD ? H * (dla_f32 ? 4 : es) : tok * H * es},
                          {dS0, n_S}};
    if (clash(outs, 5, ins, 10))
        return KDN_ERR_ALIAS;
    const GradWs w = grad_ws(P, packed != nullptr);
    if (w.total > 0) {
        if (!workspace || workspace_bytes < (unsigned long long)w.total)
            return KDN_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return KDN_ERR_ALIGN;
        const Range ws[] = {{workspace, w.total}};
        if (clash(ws, 1, ins, 10) || clash(ws, 1, outs, 5))
            return KDN_ERR_ALIAS;
        char *base = static_cast<char *>(workspace);
        auto f32 = [&](long long at) { return reinterpret_cast<float *>(base + at); };
        if (packed || P.nblocks > 1) {
            P.ws_state = f32(w.state);
            P.ws_decay = f32(w.decay);
            P.ws_rstate = f32(w.rstate);
            P.ws_rdecay = f32(w.rdecay);
            if (packed)
                P.ws_order = reinterpret_cast<int *>(P.ws_decay + (long)P.nblocks * H);
        }
        P.ws_chunk = base + w.chunk;
        // without states a single chunk has neither x nor y nor z
        if (w.chunk_lo && dlog_alpha && (gate == KDN_GATE_HEAD || S0 || dS_out))
            P.ws_chunk_lo = base + w.chunk_lo;
        P.ws_dq = Hq != H ? f32(w.dq) : nullptr;
        P.ws_dk = Hk != H ? f32(w.dk) : nullptr;
        P.ws_dv = Hv != H ? f32(w.dv) : nullptr;
        P.ws_dla = gate == KDN_GATE_HEAD ? reinterpret_cast<double *>(base + w.dla) : nullptr;
    }
    P.q = q; P.k = k; P.v = v; P.la = log_alpha;
    P.S0 = S0; P.d_o = d_o; P.dS_out = dS_out;
    P.dq = dq; P.dk_ = dk; P.dv_ = dv; P.dla = dlog_alpha; P.dla_f32 = dla_f32; P.dS0 = dS0;
    const hipError_t e = kdn::launch_linear_backward(P, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? KDN_OK : KDN_ERR_HIP;
}

}  // extern "C"
