// C-ABI entry points of the ragged prefill: argument validation on the host,
// then the launches on the caller's stream.
#include <math.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "rs.h"
#include "rs_internal.h"

using namespace rs;

namespace {

constexpr int64_t kMaxRows = 1ll << 30;
constexpr int64_t kMaxGrid = (1ll << 31) - 1;
constexpr int64_t kMaxStride = 1ll << 31;  // rows x stride stays far inside 64 bits

inline bool aligned(const void *p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }

#define RS_TRY(expr)                \
    do {                            \
        rs_status _s = (expr);      \
        if (_s != RS_OK) return _s; \
    } while (0)

rs_status check_ragged(const rs_ragged_desc *rd) {
    if (!rd) return RS_ERR_INVALID_ARG;
    if (rd->R < 1 || rd->R > 65535 || rd->tokens_cap < 1 || rd->tokens_cap > kMaxRows) return RS_ERR_INVALID_ARG;
    if (rd->block < 0 || rd->block > kMaxRows / 2 || rd->block % RS_CHUNK || rd->n_free < 0) return RS_ERR_INVALID_ARG;
    if (rd->block && (rd->max_blocks < 1 || (int64_t)rd->R * rd->max_blocks > kMaxRows)) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

rs_status check_plan(const rs_ragged_desc *rd, const rs_ragged *rg) {
    if (!rg) return RS_ERR_INVALID_ARG;
    if (!aligned(rg->cu_tokens, 4) || !aligned(rg->cu_chunks, 4) || !aligned(rg->cu_blocks, 4) ||
        !aligned(rg->token_req, 16) || !aligned(rg->token_pos, 16) || !aligned(rg->chunks, 16) ||
        !aligned(rg->counts, 4))
        return RS_ERR_INVALID_ARG;
    if (rd->block && !aligned(rg->block_table, 4)) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

// A packed array's row stride: whole 16-byte pieces, at least one row.
bool stride_ok(int64_t ld, int64_t row) { return ld >= row && ld % 8 == 0 && ld <= kMaxStride; }

rs_status check_prefill(const rs_layer_desc *d, const rs_ragged_desc *rd, int max_len) {
    RS_TRY(check_desc(d));
    if (d->kind != RS_GDN) return RS_ERR_UNSUPPORTED;
    RS_TRY(check_ragged(rd));
    if (max_len < 0) return RS_ERR_INVALID_ARG;
    // launch grids: chunks x key heads, requests x value heads x at most 8 column groups
    if ((int64_t)ragged_chunks_cap(*rd) * d->H + (int64_t)rd->R * d->H * 8 > kMaxGrid)
        return RS_ERR_INVALID_ARG;
    return RS_OK;
}

}  // namespace

extern "C" {

rs_status rs_ragged_bytes_for(const rs_ragged_desc *rd, rs_ragged_bytes *o) {
    RS_TRY(check_ragged(rd));
    if (!o) return RS_ERR_INVALID_ARG;
    o->cu_tokens = o->cu_chunks = o->cu_blocks = ((size_t)rd->R + 1) * 4;
    o->token_req = o->token_pos = (size_t)rd->tokens_cap * 4;
    o->chunks = (size_t)ragged_chunks_cap(*rd) * 16;
    o->block_table = rd->block ? (size_t)rd->R * rd->max_blocks * 4 : 0;
    o->counts = 16;
    return RS_OK;
}

rs_status rs_ragged_plan(const rs_ragged_desc *rd, const int32_t *lengths, const int32_t *context,
                         const int32_t *free_blocks, const rs_ragged *rg, uint32_t *status, void *stream) {
    RS_TRY(check_ragged(rd));
    RS_TRY(check_plan(rd, rg));
    if (!aligned(lengths, 4) || (context && !aligned(context, 4)) || !aligned(status, 4)) return RS_ERR_INVALID_ARG;
    if (rd->block && rd->n_free && !aligned(free_blocks, 4)) return RS_ERR_INVALID_ARG;
    return cuda_status(ragged_plan_launch(*rd, lengths, context, free_blocks, *rg, status, (cudaStream_t)stream));
}

rs_status rs_qk_norm(const rs_qk_desc *d, const uint16_t *q, const uint16_t *k, const uint16_t *wq,
                     const uint16_t *wk, const float *inv_freq, const int32_t *positions, uint16_t *q_out,
                     uint16_t *k_out, void *stream) {
    if (!d) return RS_ERR_INVALID_ARG;
    if (d->T < 0 || d->T > kMaxRows || d->Hq < 0 || d->Hk < 0 || d->Hq > 65535 || d->Hk > 65535 || d->Hq + d->Hk < 1)
        return RS_ERR_INVALID_ARG;
    if (d->D != 64 && d->D != 128 && d->D != 256) return RS_ERR_UNSUPPORTED;
    if (d->norm < RS_NORM_NONE || d->norm > RS_NORM_RMS) return RS_ERR_INVALID_ARG;
    if (d->rot < 0 || d->rot > d->D) return RS_ERR_INVALID_ARG;
    if (d->rot % 16) return RS_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || !isfinite(d->eps)) return RS_ERR_INVALID_ARG;
    if (d->T == 0) return RS_OK;  // whose arrays may have no address
    if (d->rot && (!aligned(inv_freq, 4) || !aligned(positions, 4))) return RS_ERR_INVALID_ARG;
    if (d->Hq && (!aligned(q, 16) || !aligned(q_out, 16) || !stride_ok(d->ld_q, (int64_t)d->Hq * d->D) ||
                  !stride_ok(d->ld_qo, (int64_t)d->Hq * d->D)))
        return RS_ERR_INVALID_ARG;
    if (d->Hk && (!aligned(k, 16) || !aligned(k_out, 16) || !stride_ok(d->ld_k, (int64_t)d->Hk * d->D) ||
                  !stride_ok(d->ld_ko, (int64_t)d->Hk * d->D)))
        return RS_ERR_INVALID_ARG;
    if ((wq && !aligned(wq, 16)) || (wk && !aligned(wk, 16))) return RS_ERR_INVALID_ARG;
    return cuda_status(qk_norm_launch(*d, q, k, wq, wk, inv_freq, positions, q_out, k_out, (cudaStream_t)stream));
}

rs_status rs_prefill_bytes_for(const rs_layer_desc *desc, const rs_ragged_desc *rd, int32_t max_len, size_t *out) {
    RS_TRY(check_prefill(desc, rd, max_len));
    if (!out) return RS_ERR_INVALID_ARG;
    *out = prefill_bytes(*desc, *rd, max_len);
    return RS_OK;
}

rs_status rs_prefill_gdn(const rs_layer_desc *d, const rs_state *st, const rs_ragged_desc *rd, const rs_ragged *rg,
                         const rs_prefill *in, uint16_t *y, void *work, void *stream) {
    if (!in) return RS_ERR_INVALID_ARG;
    RS_TRY(check_prefill(d, rd, in->max_len));
    RS_TRY(check_state(d, st));
    RS_TRY(check_plan(rd, rg));
    if (!aligned(in->q, 16) || !aligned(in->k, 16) || !aligned(in->v, 16) || !aligned(in->alpha, 4) ||
        !aligned(in->beta, 4) || !aligned(y, 16))
        return RS_ERR_INVALID_ARG;
    if (!stride_ok(in->ld_q, (int64_t)d->G * d->N) || !stride_ok(in->ld_k, (int64_t)d->G * d->N) ||
        !stride_ok(in->ld_v, (int64_t)d->H * d->P))
        return RS_ERR_INVALID_ARG;
    if ((in->rows && !aligned(in->rows, 4)) || (in->start && !aligned(in->start, 4))) return RS_ERR_INVALID_ARG;
    if (!in->rows && rd->R > d->B) return RS_ERR_INVALID_ARG;
    if (in->n_pool < 0 || (in->n_pool > 0) != (in->pool != nullptr) || (in->pool && !aligned(in->pool, 16)))
        return RS_ERR_INVALID_ARG;
    if (prefill_bytes(*d, *rd, in->max_len) && !aligned(work, 128)) return RS_ERR_INVALID_ARG;
    return cuda_status(prefill_launch(*d, *st, *rd, *rg, *in, y, work, (cudaStream_t)stream));
}

}  // extern "C"
