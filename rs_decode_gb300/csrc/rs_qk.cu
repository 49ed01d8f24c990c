// Norms of the query and key heads, with the rotation by position in the same
// pass.
//
// Each head is read once and written once (4 bytes a channel), so the kernel
// is bound by HBM; the arithmetic only has to stay out of the way.  A head is
// D / 8 lanes of 16 bytes each, its sum of squares a shuffle over those lanes.
// A warp takes a token's heads, or every hs-th group of them where tokens alone
// are too few warps, four heads in flight per lane.  The cosines and sines of
// a lane's pairs depend on the token alone: computed once, all its heads use
// them, from registers.  Where channel i turns with i + rot/2, a lane of the
// rotated part holds four channels of either half (8 bytes each), so that its
// pairs are its own and no lane needs another's channels.
//
// The angle positions * inv_freq is reduced exactly: inv_freq / (2 pi) is held
// as a 64-bit fraction of a turn, so the product with an integer position
// modulo 2^64 is the fraction of a turn without any rounding of the product.
// Its error is the position times 2^-64, where an fp32 product would be off by
// 2^-25 of the angle (0.004 radians at position 100,000).  The reduced angle,
// within half a turn, is what the fast sine and cosine are accurate for (2^-20
// absolute, against the 2^-9 of a bf16 result).
//
// Measured: 32,768 rows of 32 heads of 128 in 84 us, 6.36 TB/s, 0.94 of the copy
// peak, and 64 heads of 64 the same; 8,192 rows of 32 heads of 256 52 us, 5.2 TB/s.
// 8,191 rows of 36 heads of 128 with weights and 64 rotated channels 37 us, 4.1 TB/s
// (interleaved pairs 35; heads of 64 58 us for 32,768 rows of 32, heads of 256 60 us for
// 8,192): there one wave and two thirds of warps, and the rotation's arithmetic between
// a warp's loads, are what is left.  Every form spills 8 to 32 bytes a thread at its
// 48 or 64 registers.
#include "rs_common.cuh"
#include "rs_internal.h"

namespace rs {
namespace {

constexpr int kThreads = 256;

enum Rot { ROT_NONE = 0, ROT_HALVES = 1, ROT_PAIRS = 2 };

struct QkParams {
    int T, Hq, Hk, norm, rot, hs;
    float eps, inv_eps, w0, scale_q, scale_k;
    long long ld_q, ld_k, ld_qo, ld_ko;
    const uint16_t *q, *k, *wq, *wk;
    const float *inv_freq;
    const int32_t *positions;
    uint16_t *q_out, *k_out;
};

// Turns per position as a 64-bit fraction: |f| / (2 pi) 2^64, from f's 24-bit
// significand m and exponent: f = m 2^(e - 150), 1 / (2 pi) = c 2^-66.
__device__ __forceinline__ unsigned long long turns(float f) {
    constexpr unsigned long long c = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
    const uint32_t bits = __float_as_uint(f);
    const int e = (bits >> 23) & 255, s = 152 - e;  // s >= 23 for |f| < 2 pi
    const unsigned long long m = e ? (bits & 0x7fffffu) | 0x800000u : 0;
    // m c = hi 2^32 + (low word of lo), 88 bits; shifted right by s
    const unsigned long long lo = m * (uint32_t)c, hi = m * (uint32_t)(c >> 32) + (lo >> 32);
    const unsigned long long v = s < 32 ? hi << (32 - s) | (uint32_t)lo >> s : s < 96 ? hi >> (s - 32) : 0;
    return bits >> 31 ? 0 - v : v;
}

template <int D, int ROT>
__global__ void __launch_bounds__(kThreads, ROT == ROT_NONE ? 5 : 4) qk_kernel(const __grid_constant__ QkParams p) {
    constexpr int kRows = 4;  // heads that a lane has in flight
    constexpr int LPH = D / 8;       // lanes of a head
    constexpr int SLOTS = 32 / LPH;  // heads that a warp takes at once
    const int lane = threadIdx.x & 31, sub = lane % LPH;
    const int heads = p.Hq + p.Hk;
    const bool turning = ROT != ROT_NONE && sub < p.rot / 8;
    // the lane's channels: ch..ch+3 and ch+up..ch+up+3
    const int ch = ROT == ROT_HALVES && turning ? sub * 4 : sub * 8, up = ROT == ROT_HALVES && turning ? p.rot / 2 : 4;
    unsigned long long freq[4];
    if (ROT != ROT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) freq[i] = turning ? turns(p.inv_freq[sub * 4 + i]) : 0;
    }
    auto load8 = [&](const uint16_t *src) {
        if (ROT != ROT_HALVES) return ld_stream(src);
        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(src)), b = __ldcs(reinterpret_cast<const uint2 *>(src + up));
        return make_uint4(a.x, a.y, b.x, b.y);
    };
    const int step = SLOTS * p.hs;
    const long long units = (long long)p.T * p.hs, warps = (long long)gridDim.x * (kThreads / 32);
    for (long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int t = p.hs == 1 ? (int)u : (int)(u / p.hs), part = p.hs == 1 ? 0 : (int)(u - (long long)t * p.hs);
        const uint16_t *qs = p.q + t * p.ld_q + ch, *ks = p.k + t * p.ld_k + ch;
        uint16_t *qd = p.q_out + t * p.ld_qo + ch, *kd = p.k_out + t * p.ld_ko + ch;
        float cs[4], sn[4];
        bool have = false;
        for (int h0 = part * SLOTS + lane / LPH; h0 - lane / LPH < heads; h0 += step * kRows) {
            uint4 raw[kRows];
#pragma unroll
            for (int e = 0; e < kRows; ++e) {
                const int h = h0 + e * step;
                raw[e] = make_uint4(0, 0, 0, 0);
                if (h < heads) raw[e] = load8(h < p.Hq ? qs + (long long)h * D : ks + (long long)(h - p.Hq) * D);
            }
            if (ROT != ROT_NONE && !have) {  // behind the first loads
                have = true;
                const uint32_t pos = (uint32_t)p.positions[t];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t flo = (uint32_t)freq[i], fhi = (uint32_t)(freq[i] >> 32);
                    const uint32_t ph = __umulhi(flo, pos) + fhi * pos - ((int)pos < 0 ? flo : 0);
                    const float a = (float)(int)ph * 1.46291807926715968e-9f;  // 2 pi 2^-32
                    cs[i] = __cosf(a), sn[i] = __sinf(a);
                }
            }
#pragma unroll
            for (int e = 0; e < kRows; ++e) {
                const int h = h0 + e * step;
                if (h - lane / LPH >= heads) break;  // the whole warp
                const bool is_q = h < p.Hq;
                float x[8];
                unpack<uint16_t, 8>(raw[e], x);
                float m = is_q ? p.scale_q : p.scale_k;
                if (p.norm != RS_NORM_NONE) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                    if (p.norm == RS_NORM_L2) {
                        const float r = rsqrtf(ss);
                        m *= r > p.inv_eps ? p.inv_eps : r;  // x / max(|x|, eps); a NaN norm stays one
                    } else {
                        m *= rsqrtf(ss * (1.f / D) + p.eps);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= m;
                const uint16_t *w = is_q ? p.wq : p.wk;
                if (w) {
                    float wf[8];
                    const uint2 wa = *reinterpret_cast<const uint2 *>(w + ch), wb = *reinterpret_cast<const uint2 *>(w + ch + up);
                    unpack<uint16_t, 8>(make_uint4(wa.x, wa.y, wb.x, wb.y), wf);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] *= wf[i] + p.w0;
                }
                if (ROT != ROT_NONE && turning) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ia = ROT == ROT_PAIRS ? 2 * i : i, ib = ROT == ROT_PAIRS ? 2 * i + 1 : i + 4;
                        const float a = x[ia], b = x[ib];
                        x[ia] = a * cs[i] - b * sn[i];
                        x[ib] = b * cs[i] + a * sn[i];
                    }
                }
                if (h < heads) {
                    uint16_t *dst = is_q ? qd + (long long)h * D : kd + (long long)(h - p.Hq) * D;
                    if (ROT == ROT_HALVES) {
                        st_stream2(dst, make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3])));
                        st_stream2(dst + up, make_uint2(pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7])));
                    } else {
                        store_bf16<8>(dst, x);
                    }
                }
            }
        }
    }
}

template <int D>
cudaError_t launch(QkParams &p, int interleaved, cudaStream_t s) {
    // Where the tokens alone are fewer than 24 warps an SM, several warps a token
    const int most = (p.Hq + p.Hk + 32 / (D / 8) - 1) / (32 / (D / 8));  // groups of heads of a token
    p.hs = 1;
    while (p.hs * 2 <= most && (long long)p.T * p.hs < 152 * 24) p.hs *= 2;
    const long long ctas = ((long long)p.T * p.hs + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = (int)(ctas < 152 * 16 ? ctas : 152 * 16);
    if (!p.rot)
        qk_kernel<D, ROT_NONE><<<grid, kThreads, 0, s>>>(p);
    else if (interleaved)
        qk_kernel<D, ROT_PAIRS><<<grid, kThreads, 0, s>>>(p);
    else
        qk_kernel<D, ROT_HALVES><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t qk_norm_launch(const rs_qk_desc &d, const uint16_t *q, const uint16_t *k, const uint16_t *wq,
                           const uint16_t *wk, const float *inv_freq, const int32_t *positions, uint16_t *q_out,
                           uint16_t *k_out, cudaStream_t s) {
    // below 2^-75 a head's squares vanish in fp32, so a smaller eps than 2^-100 decides
    // nothing but heads of zero, which its reciprocal must not turn into 0 times infinity
    const float inv_eps = d.eps > 0x1p-100f ? 1.f / d.eps : 0x1p100f;
    QkParams p = {d.T, d.Hq, d.Hk, d.norm, d.rot, 1, d.eps, inv_eps, d.weight_offset, d.scale_q, d.scale_k,
                  d.ld_q, d.ld_k, d.ld_qo, d.ld_ko, q, k, wq, wk, inv_freq, positions, q_out, k_out};
    switch (d.D) {
        case 64: return launch<64>(p, d.interleaved, s);
        case 128: return launch<128>(p, d.interleaved, s);
        default: return launch<256>(p, d.interleaved, s);
    }
}

}  // namespace rs
