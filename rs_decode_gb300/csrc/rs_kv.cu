// Keys and values into the pages of a cache and out of them again.
//
// A head is D / 8 lanes of eight channels each.  As bf16 it is copied.  With
// 8 bits it is held as e4m3 codes times a power of two of its own: the least
// 2^e with which its largest magnitude is at most 448, e4m3's largest value.  A
// power of two costs no accuracy (codes are floating point: a smaller scale
// would only move the end where they lose bits), makes the division exact, so
// that a code depends on nothing but the value, and makes code times scale
// exact in bf16: reading back adds no rounding.
//
// Each value is read once and written once, so HBM bounds a batch of prompts,
// and a launch's latency a step of single tokens.
//
// Measured: 29,871 rows of 4 + 4 heads of 128 into a bf16 cache 21.6 us, 5.7 TB/s, 0.84 of the copy peak (17.9 where the
// caches hold part of it); 39,602 such rows out of an 8-bit cache 27.7 us, 4.4 TB/s, out of a bf16 one 29.8, 5.4 TB/s;
// 256 rows 2.5 us, a launch.  Two or four heads a lane, to have more look-ups in flight: no faster (21.6 to 23.7, 27.7 to 30.8).
#include <cuda_fp16.h>

#include "rs_attn.cuh"

namespace rs {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMinScale = 67;   // byte of the least scale, 2^-60
constexpr uint32_t kMaxScale = 246;  // of the largest: 448 * 2^119 is still finite in bf16
constexpr uint32_t kBadScale = 255;  // of a head that is not finite

struct KvParams {
    int Hk, page, page_log, n_pages, max_pages, cap, R;
    const int32_t *req, *pos, *pages;
    uint32_t *status;
    void *ck, *cv;
    uint8_t *ks, *vs;
    uint16_t *k, *v;  // the packed rows
    long long ld_k, ld_v;
};

// The head's place in the cache (in heads), -1 if there is none.
__device__ __forceinline__ long long place(const KvParams &p, int row, int head) {
    const int r = p.req[row], at = p.pos[row];
    if (r < 0) return -1;  // past the batch's rows
    const int j = at >> p.page_log;
    if (r >= p.R || at < 0 || j >= p.max_pages) {
        atomicOr(p.status, RS_DEV_LENGTH);
        return -1;
    }
    const int n = p.pages[(size_t)r * p.max_pages + j];
    if (n < 0 || n >= p.n_pages) {
        atomicOr(p.status, RS_DEV_SLOT);
        return -1;
    }
    return (((long long)n * p.Hk + head) << p.page_log) + (at & (p.page - 1));
}

__device__ __forceinline__ uint32_t two_codes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Eight channels of a head, LPH lanes of the warp to the head.
template <int LPH>
__device__ __forceinline__ void store_codes(uint4 x, long long to, int lane, void *codes, uint8_t *scales) {
    uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);  // patterns of magnitudes order as the magnitudes do, NaN above infinity
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (to < 0) return;
    uint2 out = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);  // NaN
    uint32_t byte = kBadScale;
    if (m < 0x7f80u) {
        byte = min(max((int)(m >> 7) - 8 + ((m & 0x7fu) > 0x60u), (int)kMinScale), (int)kMaxScale);
        const float down = __uint_as_float((254 - byte) << 23);
        float f[8];
        unpack<uint16_t, 8>(x, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= down;
        out.x = two_codes(f[0], f[1]) | two_codes(f[2], f[3]) << 16;
        out.y = two_codes(f[4], f[5]) | two_codes(f[6], f[7]) << 16;
    }
    static_cast<uint2 *>(codes)[to * LPH + lane] = out;
    if (lane == 0) scales[to] = (uint8_t)byte;
}

__device__ __forceinline__ uint4 load_codes(uint2 c, uint32_t byte) {
    const float up = pow2_of(byte);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i < 2 ? c.x : c.y;
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(i & 1 ? w >> 16 : w)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        o[i] = pack_bf2(f.x * up, f.y * up);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int LPH, bool E4M3, bool WRITE>
__global__ void __launch_bounds__(kThreads) kv_kernel(const __grid_constant__ KvParams p) {
    constexpr int D = LPH * 8;
    const long long units = (long long)p.cap * p.Hk;
    const int lane = threadIdx.x % LPH;
    // whole warps go round together: their shuffles need every lane
    for (long long base = (long long)blockIdx.x * (kThreads / LPH); base < units; base += (long long)gridDim.x * (kThreads / LPH)) {
        const long long u = base + threadIdx.x / LPH;
        const bool in = u < units;
        const int row = in ? (int)(u / p.Hk) : 0, head = in ? (int)(u % p.Hk) : 0;
        uint16_t *const kr = p.k + row * p.ld_k + head * D + lane * 8, *const vr = p.v + row * p.ld_v + head * D + lane * 8;
        uint4 k, v;
        if (WRITE) k = ld_stream(kr), v = ld_stream(vr);
        const long long to = in ? place(p, row, head) : -1;
        if (WRITE && E4M3) {
            store_codes<LPH>(k, to, lane, p.ck, p.ks);
            store_codes<LPH>(v, to, lane, p.cv, p.vs);
        } else if (to >= 0) {
            if (WRITE) {
                static_cast<uint4 *>(p.ck)[to * LPH + lane] = k;
                static_cast<uint4 *>(p.cv)[to * LPH + lane] = v;
            } else if (E4M3) {
                const uint2 kc = static_cast<const uint2 *>(p.ck)[to * LPH + lane], vc = static_cast<const uint2 *>(p.cv)[to * LPH + lane];
                const uint32_t ke = p.ks[to], ve = p.vs[to];
                st_stream(kr, load_codes(kc, ke));
                st_stream(vr, load_codes(vc, ve));
            } else {
                k = static_cast<const uint4 *>(p.ck)[to * LPH + lane], v = static_cast<const uint4 *>(p.cv)[to * LPH + lane];
                st_stream(kr, k);
                st_stream(vr, v);
            }
        }
    }
}

template <bool WRITE>
cudaError_t kv_launch(const KvParams &p, int D, bool e4m3, cudaStream_t s) {
    const int lph = D / 8;
    const long long ctas = ((long long)p.cap * p.Hk * lph + kThreads - 1) / kThreads;
    const int grid = (int)(ctas < 152 * 8 ? ctas : 152 * 8);
    if (D == 64)
        e4m3 ? kv_kernel<8, true, WRITE><<<grid, kThreads, 0, s>>>(p) : kv_kernel<8, false, WRITE><<<grid, kThreads, 0, s>>>(p);
    else
        e4m3 ? kv_kernel<16, true, WRITE><<<grid, kThreads, 0, s>>>(p) : kv_kernel<16, false, WRITE><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

KvParams kv_params(const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_ragged &rg,
                   const int32_t *pages, uint32_t *status) {
    return {d.Hk, d.page, ilog2(d.page), d.n_pages, d.max_pages, rd.tokens_cap, rd.R, rg.token_req, rg.token_pos, pages, status,
            kv.k, kv.v, kv.ks, kv.vs, nullptr, nullptr, 0, 0};
}

}  // namespace

cudaError_t kv_write_launch(const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_ragged &rg,
                            const int32_t *pages, const uint16_t *k, const uint16_t *v, long long ld_k, long long ld_v,
                            uint32_t *status, cudaStream_t s) {
    KvParams p = kv_params(d, kv, rd, rg, pages, status);
    p.k = const_cast<uint16_t *>(k), p.v = const_cast<uint16_t *>(v), p.ld_k = ld_k, p.ld_v = ld_v;
    return kv_launch<true>(p, d.D, d.type == RS_KV_E4M3, s);
}

cudaError_t kv_read_launch(const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_ragged &rg,
                           const int32_t *pages, uint16_t *k, uint16_t *v, uint32_t *status, cudaStream_t s) {
    KvParams p = kv_params(d, kv, rd, rg, pages, status);
    p.k = k, p.v = v, p.ld_k = p.ld_v = (long long)d.Hk * d.D;
    return kv_launch<false>(p, d.D, d.type == RS_KV_E4M3, s);
}

}  // namespace attn
}  // namespace rs
