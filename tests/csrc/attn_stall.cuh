// Host side of the kernels in attn_stall_short.cu and attn_stall_long.cu: the launch
// parameters and the tensor maps of a call of rs_attend, from the same arguments.
#pragma once
#include "rs_attn.cuh"

struct StallCall {
    rs::attn::Params p;
    CUtensorMap q, k, v;
};

inline bool stall_map(CUtensorMap *map, const void *base, bool bytes, cuuint64_t d0, cuuint64_t d1, cuuint64_t d2, cuuint64_t s1, cuuint64_t s2,
                      cuuint32_t b0, cuuint32_t b1, cuuint32_t b2, bool narrow) {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess || !f) return false;
    const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
    const cuuint32_t box[3] = {b0, b1, b2}, one[3] = {1, 1, 1};
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f)(
               map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool stall_call(StallCall *c, const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_attn &in, void *plan, uint16_t *y,
                       void *work, uint32_t *status) {
    using namespace rs::attn;
    const bool bytes = d.type == RS_KV_E4M3;
    const int g = d.Hq / d.Hk;
    const Form f = form_of(g, in.max_len, bytes);
    Params &p = c->p = {};
    p.Hq = d.Hq, p.Hk = d.Hk, p.g = g, p.type = d.type, p.page = d.page, p.page_log = rs::ilog2(d.page);
    p.n_pages = d.n_pages, p.max_pages = d.max_pages, p.R = rd.R, p.cap = rd.tokens_cap;
    p.ctas = kCtas, p.max_len = in.max_len, p.short_rows = f.short_rows;
    p.pages = in.pages, p.q = in.q, p.ld_q = in.ld_q, p.c = in.scale * 1.44269504f;
    p.y = y, p.plan = plan, p.ks = kv.ks, p.vs = kv.vs, p.status = status;
    p.short_parts = static_cast<float *>(work);
    p.long_parts = p.short_parts + (f.short_rows ? 2 * kCtas * part_floats(f.short_rows, d.D) : 0);
    const cuuint64_t row = d.D * (bytes ? 1 : 2), slabs = (cuuint64_t)d.n_pages * d.Hk;
    const cuuint32_t width = row < 128 ? d.D : 128 / (bytes ? 1 : 2), keys = d.page < kKeys ? d.page : kKeys;
    return stall_map(&c->k, kv.k, bytes, d.D, d.page, slabs, row, row * d.page, width, keys, 1, row < 128) &&
           stall_map(&c->v, kv.v, bytes, d.D, d.page, slabs, row, row * d.page, width, keys, 1, row < 128) &&
           stall_map(&c->q, in.q, false, d.D, d.Hq, rd.tokens_cap, d.D * 2, in.ld_q * 2, 64, g, tile_tokens(g), false);
}
