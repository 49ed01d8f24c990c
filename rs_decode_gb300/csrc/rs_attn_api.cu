// C-ABI entry points of the attention over a paged cache: argument validation on
// the host, the tensor maps of a call's copies, then the launches on the
// caller's stream.
#include <math.h>

#include "rs_attn.cuh"

using namespace rs;
using namespace rs::attn;

namespace {

constexpr int64_t kMaxRows = 1ll << 30;
constexpr int64_t kMaxStride = 1ll << 31;
constexpr float kLog2e = 1.44269504088896341f;

inline bool aligned(const void *p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool stride_ok(int64_t ld, int64_t row) { return ld >= row && ld % 8 == 0 && ld <= kMaxStride; }

#define RS_TRY(expr)                \
    do {                            \
        rs_status _s = (expr);      \
        if (_s != RS_OK) return _s; \
    } while (0)

rs_status check_kv_desc(const rs_kv_desc *d) {
    if (!d) return RS_ERR_INVALID_ARG;
    if (d->Hq < 1 || d->Hq > 65535 || d->Hk < 1 || d->Hq % d->Hk) return RS_ERR_INVALID_ARG;
    if (d->type != RS_KV_BF16 && d->type != RS_KV_E4M3) return RS_ERR_INVALID_ARG;
    if (d->page < 1 || d->n_pages < 1 || d->max_pages < 1) return RS_ERR_INVALID_ARG;
    if ((int64_t)d->n_pages * d->Hk >= 1ll << 31 || (int64_t)d->max_pages * d->page > kMaxRows) return RS_ERR_INVALID_ARG;
    if (d->D != 64 && d->D != 128) return RS_ERR_UNSUPPORTED;
    if (d->page < 16 || d->page > 256 || (d->page & (d->page - 1))) return RS_ERR_UNSUPPORTED;
    if (d->Hq / d->Hk > kTileRows) return RS_ERR_UNSUPPORTED;
    return RS_OK;
}

rs_status check_kv(const rs_kv_desc *d, const rs_kv *kv) {
    if (!kv || !aligned(kv->k, 16) || !aligned(kv->v, 16)) return RS_ERR_INVALID_ARG;
    const bool scales = d->type == RS_KV_E4M3;
    if (scales != (kv->ks != nullptr) || scales != (kv->vs != nullptr)) return RS_ERR_INVALID_ARG;
    if (scales && (!aligned(kv->ks, 16) || !aligned(kv->vs, 16))) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

rs_status check_batch(const rs_kv_desc *d, const rs_ragged_desc *rd) {
    rs_ragged_bytes b;
    RS_TRY(rs_ragged_bytes_for(rd, &b));
    if ((int64_t)rd->R * d->max_pages > 1ll << 31) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

rs_status check_rows(const rs_ragged *rg) {
    if (!rg || !aligned(rg->cu_tokens, 4) || !aligned(rg->token_req, 16) || !aligned(rg->token_pos, 16)) return RS_ERR_INVALID_ARG;
    return RS_OK;
}

// cuTensorMapEncodeTiled, from the driver through the runtime (no link-time
// dependency on the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                   const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// A 3-D map whose copies are box[0] x box[1] x box[2] elements, swizzled.
bool encode(CUtensorMap *map, const void *base, bool bytes, const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
            const cuuint32_t (&box)[3], bool narrow) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint32_t one[3] = {1, 1, 1};
    return fn(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Copies of up to 64 keys of a page and key head, 128 bytes (64 of narrow 8-bit heads) of each.
bool encode_cache(CUtensorMap *map, const void *base, const rs_kv_desc &d) {
    const bool bytes = d.type == RS_KV_E4M3;
    const cuuint64_t esz = bytes ? 1 : 2, row = d.D * esz;
    return encode(map, base, bytes, {(cuuint64_t)d.D, (cuuint64_t)d.page, (cuuint64_t)d.n_pages * d.Hk}, {row, row * d.page},
                  {(cuuint32_t)(row < 128 ? d.D : 128 / esz), (cuuint32_t)(d.page < kKeys ? d.page : kKeys), 1}, row < 128);
}

// Copies of the heads of one group of consecutive tokens, 64 channels of each.
bool encode_queries(CUtensorMap *map, const rs_attn &in, const rs_kv_desc &d, int cap) {
    const int g = d.Hq / d.Hk;
    return encode(map, in.q, false, {(cuuint64_t)d.D, (cuuint64_t)d.Hq, (cuuint64_t)cap}, {(cuuint64_t)d.D * 2, (cuuint64_t)in.ld_q * 2},
                  {64, (cuuint32_t)g, (cuuint32_t)tile_tokens(g)}, false);
}

size_t short_floats(const rs_kv_desc &d, const Form &f) { return f.short_rows ? 2 * kCtas * part_floats(f.short_rows, d.D) : 0; }
size_t long_floats(const rs_kv_desc &d, const Form &f) { return f.any_long ? 2 * kCtas * part_floats(2 * kTileRows, d.D) : 0; }

}  // namespace

extern "C" {

rs_status rs_kv_bytes_for(const rs_kv_desc *d, rs_kv_bytes *o) {
    RS_TRY(check_kv_desc(d));
    if (!o) return RS_ERR_INVALID_ARG;
    const size_t heads = (size_t)d->n_pages * d->Hk * d->page, scales = d->type == RS_KV_E4M3;
    o->k = o->v = heads * d->D * (scales ? 1 : 2);
    o->ks = o->vs = scales ? heads : 0;
    return RS_OK;
}

rs_status rs_kv_write(const rs_kv_desc *d, const rs_kv *kv, const rs_ragged_desc *rd, const rs_ragged *rg, const int32_t *pages,
                      const uint16_t *k, const uint16_t *v, int64_t ld_k, int64_t ld_v, uint32_t *status, void *stream) {
    RS_TRY(check_kv_desc(d));
    RS_TRY(check_batch(d, rd));
    RS_TRY(check_kv(d, kv));
    RS_TRY(check_rows(rg));
    if (!aligned(pages, 4) || !aligned(k, 16) || !aligned(v, 16) || !aligned(status, 4)) return RS_ERR_INVALID_ARG;
    if (!stride_ok(ld_k, (int64_t)d->Hk * d->D) || !stride_ok(ld_v, (int64_t)d->Hk * d->D)) return RS_ERR_INVALID_ARG;
    return cuda_status(kv_write_launch(*d, *kv, *rd, *rg, pages, k, v, ld_k, ld_v, status, (cudaStream_t)stream));
}

rs_status rs_kv_read(const rs_kv_desc *d, const rs_kv *kv, const rs_ragged_desc *rd, const rs_ragged *rg, const int32_t *pages,
                     uint16_t *k, uint16_t *v, uint32_t *status, void *stream) {
    RS_TRY(check_kv_desc(d));
    RS_TRY(check_batch(d, rd));
    RS_TRY(check_kv(d, kv));
    RS_TRY(check_rows(rg));
    if (!aligned(pages, 4) || !aligned(k, 16) || !aligned(v, 16) || !aligned(status, 4)) return RS_ERR_INVALID_ARG;
    return cuda_status(kv_read_launch(*d, *kv, *rd, *rg, pages, k, v, status, (cudaStream_t)stream));
}

rs_status rs_attn_bytes_for(const rs_kv_desc *d, const rs_ragged_desc *rd, int32_t max_len, rs_attn_bytes *o) {
    RS_TRY(check_kv_desc(d));
    RS_TRY(check_batch(d, rd));
    if (max_len < 1 || !o) return RS_ERR_INVALID_ARG;
    const Form f = form_of(d->Hq / d->Hk, max_len, d->type == RS_KV_E4M3);
    o->plan = plan_bytes(rd->R, kCtas);
    o->work = (short_floats(*d, f) + long_floats(*d, f)) * 4;
    return RS_OK;
}

rs_status rs_attn_plan(const rs_kv_desc *d, const rs_ragged_desc *rd, const rs_ragged *rg, int32_t max_len, void *plan,
                       uint32_t *status, void *stream) {
    RS_TRY(check_kv_desc(d));
    RS_TRY(check_batch(d, rd));
    RS_TRY(check_rows(rg));
    if (max_len < 1 || !aligned(plan, 128) || !aligned(status, 4)) return RS_ERR_INVALID_ARG;
    return cuda_status(
        plan_launch(*d, *rd, *rg, max_len, kCtas, form_of(d->Hq / d->Hk, max_len, d->type == RS_KV_E4M3), plan, status, (cudaStream_t)stream));
}

rs_status rs_attend(const rs_kv_desc *d, const rs_kv *kv, const rs_ragged_desc *rd, const rs_ragged *rg, const rs_attn *in,
                    const void *plan, uint16_t *y, void *work, uint32_t *status, void *stream) {
    RS_TRY(check_kv_desc(d));
    RS_TRY(check_batch(d, rd));
    RS_TRY(check_kv(d, kv));
    RS_TRY(check_rows(rg));
    if (!in || in->max_len < 1 || !(in->scale > 0.f) || !isfinite(in->scale * kLog2e) || !aligned(in->q, 16) || !aligned(in->pages, 4)) return RS_ERR_INVALID_ARG;
    if (!stride_ok(in->ld_q, (int64_t)d->Hq * d->D)) return RS_ERR_INVALID_ARG;
    if (!aligned(plan, 128) || !aligned(y, 16) || !aligned(work, 128) || !aligned(status, 4)) return RS_ERR_INVALID_ARG;
    const int g = d->Hq / d->Hk;
    const Form f = form_of(g, in->max_len, d->type == RS_KV_E4M3);
    Params p = {};
    p.Hq = d->Hq, p.Hk = d->Hk, p.g = g, p.type = d->type, p.page = d->page, p.page_log = ilog2(d->page);
    p.n_pages = d->n_pages, p.max_pages = d->max_pages, p.R = rd->R, p.cap = rd->tokens_cap;
    p.ctas = kCtas, p.max_len = in->max_len, p.short_rows = f.short_rows;
    p.pages = in->pages, p.q = in->q, p.ld_q = in->ld_q;
    p.c = in->scale * kLog2e;
    p.y = y, p.plan = const_cast<void *>(plan), p.ks = kv->ks, p.vs = kv->vs, p.status = status;
    p.short_parts = static_cast<float *>(work), p.long_parts = p.short_parts + short_floats(*d, f);
    const bool e4m3 = d->type == RS_KV_E4M3;
    const cudaStream_t s = (cudaStream_t)stream;
    CUtensorMap km, vm, qm;
    if (!encode_cache(&km, kv->k, *d) || !encode_cache(&vm, kv->v, *d)) return cuda_status(cudaErrorInvalidValue);
    cudaError_t e = cudaSuccess;
    if (f.any_long) {
        if (!encode_queries(&qm, *in, *d, rd->tokens_cap)) return cuda_status(cudaErrorInvalidValue);
        e = long_launch(p, d->D, e4m3, qm, km, vm, s);
    }
    if (e == cudaSuccess && f.short_rows) e = short_launch(p, d->D, e4m3, km, vm, f.any_long, s);
    if (e == cudaSuccess) e = join_launch(p, d->D, e4m3, f.any_long, s);
    return cuda_status(e);
}

}  // extern "C"
