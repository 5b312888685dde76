// api_lm.hip -- C ABI of the operators around the recurrence (embedding,
// token log probabilities, linear attention): argument checks, workspace
// sizes and the launches (lm.h).
#include "../../include/rnn355.h"
#include "host.h"
#include "lm.h"

using namespace rnn355;
using namespace rnn355::host;

namespace {

size_t elt(rnn_dtype dt) { return dt == RNN_BF16 ? 2 : 4; }

// A view starts at a whole element.
bool view_ok(const void *p, size_t e) { return p && (uintptr_t)p % e == 0; }

bool itype_ok(rnn_itype t) { return t == RNN_I32 || t == RNN_I64; }

bool ids_ok(const rnn_ids *i) {
    return i && itype_ok(i->type) && view_ok(i->data, i->type == RNN_I64 ? 8 : 4);
}

bool embed_dims_ok(int T, int B, int V, int D) {
    return T > 0 && B > 0 && V > 0 && D > 0 && (long)T * B <= (1L << 30) && V <= (1 << 30) &&
           D <= (1 << 20);
}

lm::Ids ids_of(const rnn_ids *i, int T, int B) {
    return lm::Ids{i->data, i->stride_t, i->stride_b, T, B, i->type == RNN_I64};
}

bool logp_dims_ok(int M, int V) { return M > 0 && V > 0; }

bool lin_dims_ok(const rnn_lin_dims *d) {
    return d && d->T > 0 && d->B > 0 && d->NH > 0 && d->NKV > 0 && d->Dk > 0 && d->Dv > 0 &&
           d->NH % d->NKV == 0 && (long)d->T * d->B <= (1L << 30) && (long)d->B * d->NH <= (1L << 24);
}

bool lin_depths_ok(const rnn_lin_dims *d) { return d->Dk <= 256 && d->Dv <= 256; }

// Calls that walk the rows, the backward of one token among them: 16 rows of a
// sequence stay within 32 bits of each other (4-byte values).
bool lin_rows_ok(const rnn_lin_dims *d) {
    return lin_depths_ok(d) && (long)d->B * d->NH * (d->Dk > d->Dv ? d->Dk : d->Dv) < (1L << 26);
}

// The forward of one token runs as a step, which has no such distances.
bool lin_fwd_ok(const rnn_lin_dims *d) { return d->T == 1 ? lin_depths_ok(d) : lin_rows_ok(d); }

lm::LinDims lin_dims(const rnn_lin_dims *d) {
    return lm::LinDims{d->T, d->B, d->NH, d->NKV, d->Dk, d->Dv};
}

lm::LinSeq seq_of(const rnn_seq *s) { return lm::LinSeq{s->data, s->stride_t, s->stride_b}; }

bool seq_ok(const rnn_seq *s, rnn_dtype dt) { return s && view_ok(s->data, elt(dt)); }

rnn_status done(hipError_t e) { return e == hipSuccess ? RNN_OK : RNN_ERR_HIP; }

}  // namespace

extern "C" {

rnn_status rnn_embed_fwd(int T, int B, int V, int D, rnn_dtype dt, const rnn_ids *ids,
                         const void *table, int64_t ld, float scale, void *x,
                         hipStream_t stream) {
    if (!embed_dims_ok(T, B, V, D) || !dtype_ok(dt) || !ids_ok(ids)) return RNN_ERR_INVALID_ARG;
    if (!view_ok(table, elt(dt)) || ld < D || !x || !aligned16(x)) return RNN_ERR_INVALID_ARG;
    if (!lm::embed_fwd_grid_ok(T * B, D, dt == RNN_BF16, table, ld)) return RNN_ERR_UNSUPPORTED;
    return done(lm::launch_embed_fwd(ids_of(ids, T, B), V, D, dt == RNN_BF16, table, ld, scale, x,
                                     stream));
}

size_t rnn_workspace_size_embed_bwd(int T, int B, int V, int D) {
    return embed_dims_ok(T, B, V, D) ? lm::embed_bwd_bytes(T * B, V, D) : 0;
}

rnn_status rnn_embed_bwd(int T, int B, int V, int D, rnn_dtype dt, const rnn_ids *ids,
                         const void *dx, float scale, float *dtable, void *ws, size_t ws_bytes,
                         hipStream_t stream) {
    if (!embed_dims_ok(T, B, V, D) || !dtype_ok(dt) || !ids_ok(ids)) return RNN_ERR_INVALID_ARG;
    if (!dx || !dtable || !aligned16(dx) || !aligned16(dtable) || !aligned16(ws))
        return RNN_ERR_INVALID_ARG;
    if (!lm::embed_bwd_grid_ok(T * B, V, D)) return RNN_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < lm::embed_bwd_bytes(T * B, V, D)) return RNN_ERR_WORKSPACE;
    return done(lm::launch_embed_bwd(ids_of(ids, T, B), V, D, dt == RNN_BF16, dx, scale, dtable, ws,
                                     stream));
}

size_t rnn_workspace_size_logprobs(int M, int V, int K) {
    if (!logp_dims_ok(M, V) || V > lm::kMaxVocab || K < 0 || K > V || K > lm::kMaxTop) return 0;
    return lm::logp_bytes(M, V, K);
}

rnn_status rnn_token_logprobs(int M, int V, rnn_dtype dt, const void *logits, int64_t ld,
                              const void *tok, rnn_itype it, int K, float *logp, float *entropy,
                              float *lse, float *top_logp, int *top_id, void *ws,
                              size_t ws_bytes, hipStream_t stream) {
    if (!logp_dims_ok(M, V) || !dtype_ok(dt) || !itype_ok(it) || K < 0 || K > V || ld < V)
        return RNN_ERR_INVALID_ARG;
    if (!view_ok(logits, elt(dt)) || !view_ok(tok, it == RNN_I64 ? 8 : 4) || !logp)
        return RNN_ERR_INVALID_ARG;
    if (K > 0 && (!top_logp || !top_id)) return RNN_ERR_INVALID_ARG;
    const void *ps[] = {logp, entropy, lse, top_logp, top_id};
    for (const void *p : ps)
        if (p && !view_ok(p, 4)) return RNN_ERR_INVALID_ARG;
    if (!aligned16(ws)) return RNN_ERR_INVALID_ARG;
    if (V > lm::kMaxVocab || K > lm::kMaxTop || !lm::logp_grid_ok(M, V, dt == RNN_BF16))
        return RNN_ERR_UNSUPPORTED;
    const size_t need = lm::logp_bytes(M, V, K);
    if (need && (!ws || ws_bytes < need)) return RNN_ERR_WORKSPACE;
    lm::LogpArgs a{M, V, K, logits, ld, tok, it == RNN_I64, logp, entropy, lse, top_logp, top_id, ws};
    return done(lm::launch_logp(a, dt == RNN_BF16, stream));
}

rnn_status rnn_token_logprobs_bwd(int M, int V, rnn_dtype dt, const void *logits, int64_t ld,
                                  const void *tok, rnn_itype it, const float *lse,
                                  const float *entropy, const float *dlogp,
                                  const float *dentropy, void *dlogits, int64_t ldd,
                                  hipStream_t stream) {
    if (!logp_dims_ok(M, V) || !dtype_ok(dt) || !itype_ok(it) || ld < V || ldd < V)
        return RNN_ERR_INVALID_ARG;
    if (!view_ok(logits, elt(dt)) || !view_ok(dlogits, elt(dt)) ||
        !view_ok(tok, it == RNN_I64 ? 8 : 4) || !lse || (dentropy && !entropy))
        return RNN_ERR_INVALID_ARG;
    const void *ps[] = {lse, entropy, dlogp, dentropy};
    for (const void *p : ps)
        if (p && !view_ok(p, 4)) return RNN_ERR_INVALID_ARG;
    if (V > lm::kMaxVocab || !lm::logp_bwd_grid_ok(M, V, dt == RNN_BF16)) return RNN_ERR_UNSUPPORTED;
    lm::LogpBwdArgs a{M, V, logits, ld, tok, it == RNN_I64, lse, entropy, dlogp, dentropy, dlogits, ldd};
    return done(lm::launch_logp_bwd(a, dt == RNN_BF16, stream));
}

size_t rnn_workspace_size_linattn(rnn_lin_op op, const rnn_lin_dims *d, rnn_dtype dt) {
    if (!lin_dims_ok(d) || !dtype_ok(dt)) return 0;
    if (op == RNN_OP_LIN_FWD && lin_fwd_ok(d)) return lm::lin_fwd_bytes(lin_dims(d), dt == RNN_BF16);
    if (op == RNN_OP_LIN_BWD && lin_rows_ok(d)) return lm::lin_bwd_bytes(lin_dims(d), dt == RNN_BF16);
    return 0;
}

rnn_status rnn_linattn_fwd(const rnn_lin_dims *d, rnn_dtype dt, const rnn_seq *q,
                           const rnn_seq *k, const rnn_seq *v, const float *g, float scale,
                           const float *S0, void *o, float *ST, void *ws, size_t ws_bytes,
                           hipStream_t stream) {
    if (!lin_dims_ok(d) || !dtype_ok(dt)) return RNN_ERR_INVALID_ARG;
    if (!seq_ok(q, dt) || !seq_ok(k, dt) || !seq_ok(v, dt) || !g || !o) return RNN_ERR_INVALID_ARG;
    const void *ps[] = {g, S0, o, ST, ws};
    for (const void *p : ps)
        if (!aligned16(p)) return RNN_ERR_INVALID_ARG;
    const lm::LinDims n = lin_dims(d);
    if (!lin_fwd_ok(d) || !lm::lin_fwd_grid_ok(n, dt == RNN_BF16)) return RNN_ERR_UNSUPPORTED;
    const size_t need = lm::lin_fwd_bytes(n, dt == RNN_BF16);
    if (need && (!ws || ws_bytes < need)) return RNN_ERR_WORKSPACE;
    return done(lm::launch_lin_fwd(n, dt == RNN_BF16, seq_of(q), seq_of(k), seq_of(v), g, scale, S0,
                                   o, ST, ws, stream));
}

rnn_status rnn_linattn_step(const rnn_lin_dims *d, rnn_dtype dt, const rnn_seq *q,
                            const rnn_seq *k, const rnn_seq *v, const float *g, float scale,
                            const float *S, void *o, float *S_out, hipStream_t stream) {
    if (!lin_dims_ok(d) || !dtype_ok(dt) || d->T != 1) return RNN_ERR_INVALID_ARG;
    if (!seq_ok(q, dt) || !seq_ok(k, dt) || !seq_ok(v, dt) || !g || !o || !S || !S_out)
        return RNN_ERR_INVALID_ARG;
    const void *ps[] = {g, S, o, S_out};
    for (const void *p : ps)
        if (!aligned16(p)) return RNN_ERR_INVALID_ARG;
    if (!lin_depths_ok(d) || !lm::lin_step_grid_ok(lin_dims(d))) return RNN_ERR_UNSUPPORTED;
    return done(lm::launch_lin_step(lin_dims(d), dt == RNN_BF16, seq_of(q), seq_of(k), seq_of(v), g,
                                    scale, S, o, S_out, stream));
}

rnn_status rnn_linattn_bwd(const rnn_lin_dims *d, rnn_dtype dt, const rnn_seq *q,
                           const rnn_seq *k, const rnn_seq *v, const float *g, float scale,
                           const float *S0, const rnn_seq *dO, const float *dST, void *dq,
                           void *dk, void *dv, float *dS0, void *ws, size_t ws_bytes,
                           hipStream_t stream) {
    if (!lin_dims_ok(d) || !dtype_ok(dt)) return RNN_ERR_INVALID_ARG;
    if (!seq_ok(q, dt) || !seq_ok(k, dt) || !seq_ok(v, dt) || !seq_ok(dO, dt) || !g || !dq || !dk ||
        !dv)
        return RNN_ERR_INVALID_ARG;
    const void *ps[] = {g, S0, dST, dq, dk, dv, dS0, ws};
    for (const void *p : ps)
        if (!aligned16(p)) return RNN_ERR_INVALID_ARG;
    const lm::LinDims n = lin_dims(d);
    if (!lin_rows_ok(d) || !lm::lin_bwd_grid_ok(n, dt == RNN_BF16)) return RNN_ERR_UNSUPPORTED;
    const size_t need = lm::lin_bwd_bytes(n, dt == RNN_BF16);
    if (need && (!ws || ws_bytes < need)) return RNN_ERR_WORKSPACE;
    return done(lm::launch_lin_bwd(n, dt == RNN_BF16, seq_of(q), seq_of(k), seq_of(v), g, scale, S0,
                                   seq_of(dO), dST, dq, dk, dv, dS0, ws, stream));
}

}  // extern "C"
