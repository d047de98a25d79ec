// C ABI entry points of the gated delta rule (include/ssd.h): argument validation, workspace
// carving and the choice of the kernels.
#include "api.cuh"
#include "delta.cuh"

namespace ssd {
namespace {

// The kernels of a forward pass.  Below kChunkTokens the token recurrence, one launch, is as fast as
// the chunked kernels.  Of these the warp-level ones (16 state rows to a warp) are ahead while each
// warp has an SM to itself, by 6 us for short sequences and as fast for long ones (8 heads of 64, N 128,
// us: 129 tokens 18 against 25, 2048 tokens 104 against 105; 37 heads 19 against 25, 115 against 113), and
// for sequences of up to 64 tokens (8 x 80 heads: 37 against 47; of 128 tokens 61 against 62); with more
// to do the tcgen05 ones are (80 heads, 2048 tokens: 131 against 209; 8 x 80 heads 456 against 699).
constexpr int kChunkTokens = 24, kTcTokens = 64;
constexpr int64_t kTcRows = 148 * 16;

enum class Path { kRecurrent, kChunk, kTc };

Path forward_path(const ssd_shape *s, int64_t nseq)
{
    const bool is_bf16 = s->dtype == SSD_BF16;
    if (s->seqlen < kChunkTokens ||
        !delta_chunk_supported(is_bf16, (int)s->headdim, (int)s->dstate)) return Path::kRecurrent;
    const int64_t tokens = s->batch * s->seqlen;   // over all sequences
    return delta_tc_supported((int)s->headdim, (int)s->dstate) && tokens > nseq * kTcTokens &&
                   nseq * s->nheads * s->headdim > kTcRows
               ? Path::kTc : Path::kChunk;
}

int64_t chunks_of(const ssd_shape *s, int tokens) { return (s->seqlen + tokens - 1) / tokens; }

// Tokens of a forward chunk, and the bytes of `chunks` of them over all heads.
int path_tokens(Path p) { return p == Path::kTc ? kDeltaTcChunk : kDeltaChunk; }
size_t items_bytes(const ssd_shape *s, Path p, int64_t chunks)
{
    const size_t items = (size_t)(s->batch * chunks * s->nheads);
    return p == Path::kTc ? items * kDeltaTcItem
                          : p == Path::kChunk ? items * DeltaItem::kBytes : 0;
}

ssd_status check_delta(const ssd_shape *s, const ssd_delta_options *o, bool need_seq)
{
    ssd_status st = api_check_shape(s, need_seq);
    if (st != SSD_OK) return st;
    if (!delta_recurrent_supported((int)s->dstate))
        return api_fail(SSD_ERR_UNSUPPORTED, "the delta rule needs dstate 32, 64, 128 or 256 "
                        "(got %lld)", (long long)s->dstate);
    if (o && o->qk_l2norm != 0 && o->qk_l2norm != 1)
        return api_fail(SSD_ERR_INVALID_ARG, "qk_l2norm must be 0 or 1");
    const int64_t blocks = (s->headdim + 15) / 16;   // of the launch grid, per batch row and head
    const int64_t seqlen = need_seq ? s->seqlen : 1;
    if (s->batch * s->nheads * blocks > 0x7fffffffLL || seqlen > (int64_t)1 << 34 ||
        s->batch * s->nheads * (seqlen / 32 + 1) > (int64_t)1 << 36)
        return api_fail(SSD_ERR_UNSUPPORTED, "problem too large for one launch grid");
    return SSD_OK;
}

DeltaArgs delta_args(const ssd_shape *s, const ssd_delta_options *o, const void *q,
                     const void *k, const void *v, const float *g, const float *beta)
{
    DeltaArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.batch = s->batch;
    a.L = s->seqlen;
    a.H = (int)s->nheads;
    a.G = (int)s->ngroups;
    a.P = (int)s->headdim;
    a.N = (int)s->dstate;
    a.scale = o->scale;
    a.l2norm = o->qk_l2norm;
    return a;
}

struct VarlenWs {
    size_t status, tab, cstart, items, total;
    int64_t slots;
};

VarlenWs varlen_ws(const ssd_shape *s, int nseq)
{
    VarlenWs w;
    const Path path = forward_path(s, nseq);
    w.slots = s->seqlen / path_tokens(path) + nseq;
    w.status = 0;
    w.tab = 256;
    w.cstart = w.tab + api_round256((size_t)w.slots * sizeof(int2));
    w.items = w.cstart + api_round256((size_t)(nseq + 1) * sizeof(int32_t));
    w.total = w.items + items_bytes(s, path, w.slots);
    return w;
}

ssd_status check_delta_varlen(const ssd_shape *s, int nseq, const ssd_delta_options *o)
{
    ssd_status st = check_delta(s, o, true);
    if (st != SSD_OK) return st;
    if (s->batch != 1)
        return api_fail(SSD_ERR_INVALID_ARG, "variable-length input is packed: batch must be 1 "
                        "(got %lld)", (long long)s->batch);
    if (nseq < 1) return api_fail(SSD_ERR_INVALID_ARG, "nseq must be >= 1 (got %d)", nseq);
    if (s->seqlen > 0x7fffffffLL - 256)
        return api_fail(SSD_ERR_UNSUPPORTED, "packed token count must fit int32 cu_seqlens");
    if ((int64_t)nseq * s->nheads * 8 > 0x7fffffffLL)
        return api_fail(SSD_ERR_UNSUPPORTED, "problem too large for one launch grid");
    return SSD_OK;
}

// The backward's workspace: the items, then what the chains hand to the gradients' kernels.
struct BwdWs {
    size_t items, states, dstates, wfrag, dot_oo, dot_vv, dot_vw, dot_ss, dq, dk, total;
    int64_t chunks, spans;
    int runs, run_heads;
};

BwdWs bwd_ws(const ssd_shape *s)
{
    BwdWs w;
    w.chunks = chunks_of(s, kDeltaChunk);
    w.spans = (s->seqlen + 63) / 64;
    const size_t H = (size_t)s->nheads, PN = (size_t)(s->headdim * s->dstate);
    const size_t items = (size_t)(s->batch * w.chunks) * H, spans = (size_t)(s->batch * w.spans) * H;
    const size_t tiles = (size_t)s->headdim / 16, tokens = (size_t)(s->batch * s->seqlen);
    // heads of a group per CTA of the gradients' kernel, whose sums stay in registers: what takes the
    // fewest turns of a head (one more for a CTA's start) on 148 SMs with one or two CTAs each
    const int64_t hpg = s->nheads / s->ngroups, slots = s->headdim <= 64 ? 296 : 148;
    const int64_t spans_groups = s->batch * w.spans * s->ngroups;
    int64_t best = 0;
    w.run_heads = 1;
    for (int64_t n = 1; n <= 8 && n <= hpg; ++n) {
        const int64_t ctas = spans_groups * ((hpg + n - 1) / n);
        const int64_t turns = (ctas + slots - 1) / slots * (n + 1);
        if (n == 1 || turns <= best) {
            best = turns;
            w.run_heads = (int)n;
        }
    }
    w.runs = (int)((hpg + w.run_heads - 1) / w.run_heads);
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += api_round256(bytes);
        return here;
    };
    w.items = take(items * DeltaItem::kBytes);
    w.states = take((spans + (size_t)s->batch * H) * PN * 4);
    w.dstates = take(spans * PN * 2);
    w.wfrag = take(items * (size_t)s->headdim * kDeltaChunk * 4);
    w.dot_oo = take(items * tiles * kDeltaChunk * 4);
    w.dot_vv = take(items * tiles * kDeltaChunk * 4);
    w.dot_vw = take(items * tiles * kDeltaChunk * 4);
    w.dot_ss = take((spans + (size_t)s->batch * H) * tiles * 4);
    w.dq = take(tokens * (size_t)(s->ngroups * w.runs) * (size_t)s->dstate * 4);
    w.dk = take(tokens * (size_t)(s->ngroups * w.runs) * (size_t)s->dstate * 4);
    w.total = at;
    return w;
}

ssd_status check_delta_bwd(const ssd_shape *s, const ssd_delta_options *o)
{
    ssd_status st = check_delta(s, o, true);
    if (st != SSD_OK) return st;
    if (!delta_chunk_supported(s->dtype == SSD_BF16, (int)s->headdim, (int)s->dstate))
        return api_fail(SSD_ERR_UNSUPPORTED, "the delta rule's backward needs bf16, headdim a "
                        "multiple of 16 and dstate 64 or 128");
    return SSD_OK;
}

ssd_status check_pointers(const DeltaArgs &a, const void *workspace)
{
    if (!a.q || !a.k || !a.v || !a.beta || !a.o || !workspace)
        return api_fail(SSD_ERR_INVALID_ARG,
                        "q, k, v, beta, o and workspace must be non-NULL");
    if (!api_aligned(a.q, 16) || !api_aligned(a.k, 16) || !api_aligned(a.v, 16) ||
        !api_aligned(a.o, 16))
        return api_fail(SSD_ERR_INVALID_ARG, "q, k, v and o must be 16-byte aligned");
    if (!api_aligned(workspace, 256))
        return api_fail(SSD_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    return SSD_OK;
}

ssd_status check_states(const float *init, const float *final_state)
{
    if (!api_aligned(init, 16) || !api_aligned(final_state, 16))
        return api_fail(SSD_ERR_INVALID_ARG, "initial and final states must be 16-byte aligned");
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_delta_rule_workspace_size(const ssd_shape *shape)
{
    if (check_delta(shape, nullptr, true) != SSD_OK) return 0;
    const Path path = forward_path(shape, shape->batch);
    return 256 + items_bytes(shape, path, chunks_of(shape, path_tokens(path)));
}

ssd_status ssd_delta_rule_fwd(const ssd_shape *shape, const void *q, const void *k,
                              const void *v, const float *g, const float *beta,
                              const ssd_delta_options *options, const float *init_state, void *o,
                              float *final_state, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    if (!options) return api_fail(SSD_ERR_INVALID_ARG, "options is NULL");
    ssd_status st = check_delta(shape, options, true);
    if (st == SSD_OK) st = check_states(init_state, final_state);
    if (st != SSD_OK) return st;
    const ssd_shape s = *shape;
    cudaStream_t cst = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (s.batch == 0) return SSD_OK;
    if (s.seqlen == 0) {
        if (!final_state) return SSD_OK;
        e = launch_fill_final(init_state, final_state,
                              s.batch * s.nheads * s.headdim * s.dstate, cst);
        return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "fill final state");
    }
    DeltaArgs a = delta_args(&s, options, q, k, v, g, beta);
    a.init = init_state;
    a.o = o;
    a.final_state = final_state;
    st = check_pointers(a, workspace);
    if (st != SSD_OK) return st;
    const size_t need = ssd_delta_rule_workspace_size(shape);
    if (workspace_bytes < need)
        return api_fail(SSD_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu", need,
                        workspace_bytes);
    a.clear = static_cast<int *>(workspace);
    const Path path = forward_path(&s, s.batch);
    char *items = static_cast<char *>(workspace) + 256;
    const int64_t chunks = chunks_of(&s, path_tokens(path));
    if (path == Path::kTc) {
        e = launch_delta_tc(a, items, chunks, nullptr, nullptr, static_cast<int *>(workspace), cst);
    } else if (path == Path::kChunk) {
        e = launch_delta_prep(a, items, false, chunks, nullptr, cst);
        if (e == cudaSuccess)
            e = launch_delta_chain(a, nullptr, items, chunks, nullptr, nullptr, nullptr, cst);
    } else {
        e = launch_delta_recurrent(a, s.dtype == SSD_BF16, nullptr, cst);
    }
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "delta rule launch");
}

size_t ssd_delta_rule_varlen_workspace_size(const ssd_shape *shape, int nseq)
{
    if (check_delta_varlen(shape, nseq, nullptr) != SSD_OK) return 0;
    return varlen_ws(shape, nseq).total;
}

ssd_status ssd_delta_rule_varlen_fwd(const ssd_shape *shape, const void *q, const void *k,
                                     const void *v, const float *g, const float *beta,
                                     const ssd_delta_options *options, const int32_t *cu_seqlens,
                                     int nseq, const float *init_states, void *o,
                                     float *final_states, void *workspace,
                                     size_t workspace_bytes, void *stream)
{
    if (!options) return api_fail(SSD_ERR_INVALID_ARG, "options is NULL");
    ssd_status st = check_delta_varlen(shape, nseq, options);
    if (st == SSD_OK) st = check_states(init_states, final_states);
    if (st != SSD_OK) return st;
    if (!cu_seqlens) return api_fail(SSD_ERR_INVALID_ARG, "cu_seqlens must be non-NULL");
    DeltaArgs a = delta_args(shape, options, q, k, v, g, beta);
    a.init = init_states;
    a.o = o;
    a.final_state = final_states;
    a.cu = cu_seqlens;
    a.nseq = nseq;
    if (a.L > 0) {
        st = check_pointers(a, workspace);
        if (st != SSD_OK) return st;
    }
    const VarlenWs w = varlen_ws(shape, nseq);
    if (!workspace || !api_aligned(workspace, 256) || workspace_bytes < w.total)
        return api_fail(SSD_ERR_INVALID_ARG, "workspace too small or unaligned: need %zu bytes, "
                        "got %zu", w.total, workspace_bytes);
    cudaStream_t cst = static_cast<cudaStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    int *status = reinterpret_cast<int *>(ws + w.status);
    int2 *tab = reinterpret_cast<int2 *>(ws + w.tab);
    int32_t *cstart = reinterpret_cast<int32_t *>(ws + w.cstart);
    const Path path = forward_path(shape, nseq);
    cudaError_t e = launch_build_chunk_table(cu_seqlens, nseq, a.L, path_tokens(path), w.slots, tab,
                                             cstart, status, cst);
    if (e == cudaSuccess && path == Path::kTc) {
        e = launch_delta_tc(a, ws + w.items, w.slots, tab, cstart, status, cst);
    } else if (e == cudaSuccess && path == Path::kChunk) {
        e = launch_delta_prep(a, ws + w.items, false, w.slots, tab, cst);
        if (e == cudaSuccess)
            e = launch_delta_chain(a, nullptr, ws + w.items, w.slots, tab, cstart, status, cst);
    } else if (e == cudaSuccess) {
        e = launch_delta_recurrent(a, shape->dtype == SSD_BF16, status, cst);
    }
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "delta rule launch");
}

size_t ssd_delta_rule_bwd_workspace_size(const ssd_shape *shape)
{
    if (check_delta_bwd(shape, nullptr) != SSD_OK) return 0;
    return bwd_ws(shape).total;
}

ssd_status ssd_delta_rule_bwd(const ssd_shape *shape, const void *q, const void *k, const void *v,
                              const float *g, const float *beta,
                              const ssd_delta_options *options, const float *init_state,
                              const void *dout, const float *dfinal, void *dq, void *dk, void *dv,
                              float *dg, float *dbeta, float *dinit, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    if (!options) return api_fail(SSD_ERR_INVALID_ARG, "options is NULL");
    ssd_status st = check_delta_bwd(shape, options);
    if (st == SSD_OK) st = check_states(init_state, nullptr);
    if (st == SSD_OK) st = check_states(dfinal, dinit);
    if (st != SSD_OK) return st;
    const ssd_shape s = *shape;
    cudaStream_t cst = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (s.batch == 0) return SSD_OK;
    if (s.seqlen == 0) {   // the final state is the initial one
        if (!dinit) return SSD_OK;
        e = launch_fill_final(dfinal, dinit, s.batch * s.nheads * s.headdim * s.dstate, cst);
        return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "fill dinit");
    }
    DeltaArgs a = delta_args(&s, options, q, k, v, g, beta);
    a.init = init_state;
    a.o = dv;   // checked like the forward's output
    st = check_pointers(a, workspace);
    if (st != SSD_OK) return st;
    a.o = nullptr;
    if (!dout || !dq || !dk || !dbeta || (g != nullptr) != (dg != nullptr))
        return api_fail(SSD_ERR_INVALID_ARG,
                        "dout, dq, dk and dbeta must be non-NULL, and dg go with g");
    if (!api_aligned(dout, 16) || !api_aligned(dq, 16) || !api_aligned(dk, 16))
        return api_fail(SSD_ERR_INVALID_ARG, "dout, dq and dk must be 16-byte aligned");
    const BwdWs l = bwd_ws(&s);
    if (workspace_bytes < l.total)
        return api_fail(SSD_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu",
                        l.total, workspace_bytes);
    a.clear = static_cast<int *>(workspace);
    char *ws = static_cast<char *>(workspace);
    auto f32 = [&](size_t at) { return reinterpret_cast<float *>(ws + at); };
    DeltaBwd w = {};
    w.dout = static_cast<const bf16 *>(dout);
    w.dfinal = dfinal;
    w.n64 = l.spans;
    w.states = f32(l.states);
    w.dstates = reinterpret_cast<bf16 *>(ws + l.dstates);
    w.wfrag = f32(l.wfrag);
    w.dot_oo = f32(l.dot_oo);
    w.dot_vv = f32(l.dot_vv);
    w.dot_vw = f32(l.dot_vw);
    w.dot_ss = f32(l.dot_ss);
    w.dq_part = f32(l.dq);
    w.dk_part = f32(l.dk);
    w.runs = l.runs;
    w.run_heads = l.run_heads;
    w.dq = static_cast<bf16 *>(dq);
    w.dk = static_cast<bf16 *>(dk);
    w.dv = static_cast<bf16 *>(dv);
    w.dg = dg;
    w.dbeta = dbeta;
    w.dinit = dinit;
    char *items = ws + l.items;
    e = launch_delta_prep(a, items, true, l.chunks, nullptr, cst);
    if (e == cudaSuccess)
        e = launch_delta_chain(a, &w, items, l.chunks, nullptr, nullptr, nullptr, cst);
    if (e == cudaSuccess) e = launch_delta_adjoint(a, w, items, l.chunks, cst);
    if (e == cudaSuccess) e = launch_delta_grads(a, w, l.chunks, cst);
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "delta rule backward launch");
}

ssd_status ssd_delta_rule_update(const ssd_shape *shape, float *state, const void *q,
                                 const void *k, const void *v, const float *g,
                                 const float *beta, const ssd_delta_options *options, void *o,
                                 void *stream)
{
    if (!options) return api_fail(SSD_ERR_INVALID_ARG, "options is NULL");
    ssd_status st = check_delta(shape, options, false);
    if (st != SSD_OK) return st;
    if (shape->batch == 0) return SSD_OK;
    ssd_shape s = *shape;
    s.seqlen = 1;
    DeltaArgs a = delta_args(&s, options, q, k, v, g, beta);
    a.init = state;
    a.final_state = state;
    a.o = o;
    if (!state || !q || !k || !v || !beta || !o)
        return api_fail(SSD_ERR_INVALID_ARG, "state, q, k, v, beta and o must be non-NULL");
    if (!api_aligned(state, 16) || !api_aligned(q, 16) || !api_aligned(k, 16))
        return api_fail(SSD_ERR_INVALID_ARG, "state, q and k must be 16-byte aligned");
    cudaError_t e = launch_delta_recurrent(a, s.dtype == SSD_BF16, nullptr,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SSD_OK : api_cuda_fail(e, "delta rule update launch");
}

}  // extern "C"
