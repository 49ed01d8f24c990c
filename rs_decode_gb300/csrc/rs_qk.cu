// Norms of the query and key heads, with the rotation by position in the same
// pass.
//
// Each head is read once and written once (4 bytes a channel), so the kernel
// is bound by HBM; the arithmetic only has to stay out of the way.  A head is
// D / 8 lanes of 16 bytes each, its sum of squares a shuffle over those lanes,
// and a thread has kRows heads in flight to cover the memory latency.  The
// rotation's cosines and sines depend on the token and the pair alone: a CTA
// computes them once for its tokens into shared memory and all their heads
// read them.
//
// The angle positions * inv_freq is reduced exactly: inv_freq / (2 pi) is held
// as a 64-bit fraction of a turn, so the product with an integer position
// modulo 2^64 is the fraction of a turn without any rounding of the product.
// Its error is the position times 2^-54, where an fp32 product would be off by
// 2^-25 of the angle (0.004 radians at position 100,000).
#include "rs_common.cuh"
#include "rs_internal.h"

namespace rs {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;       // heads that a thread has in flight
constexpr int kMaxTokens = 16;  // tokens of one CTA

struct QkParams {
    int T, Hq, Hk, norm, rot, interleaved, tokens;
    float eps, w0, scale_q, scale_k;
    long long ld_q, ld_k, ld_qo, ld_ko;
    const uint16_t *q, *k, *wq, *wk;
    const float *inv_freq;
    const int32_t *positions;
    uint16_t *q_out, *k_out;
};

template <int D>
__global__ void __launch_bounds__(kThreads) qk_kernel(const __grid_constant__ QkParams p) {
    constexpr int LPH = D / 8;             // lanes of a head
    constexpr int SLOTS = kThreads / LPH;  // heads that the CTA takes at once
    extern __shared__ float2 turn[];       // [tokens][rot / 2] cosine and sine
    const int heads = p.Hq + p.Hk;
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int half = p.rot >> 1;
    if (half) {
        for (int i = threadIdx.x; i < nt * half; i += kThreads) {
            const int t = i / half, j = i - t * half;
            // turns per position as a 64-bit fraction; |inv_freq| < 2 pi keeps it below one turn
            const double f = (double)p.inv_freq[j] * 0.15915494309189533577;
            const long long frac = __double2ll_rn(f * 9223372036854775808.0);  // in 2^-63 turns
            const unsigned long long ph = (unsigned long long)frac * 2ull *
                                          (unsigned long long)(long long)p.positions[t0 + t];
            float s, c;
            sincospif((float)(int)(ph >> 32) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half turns
            turn[i] = make_float2(c, s);
        }
        __syncthreads();
    }
    const int lane = threadIdx.x % LPH, slot = threadIdx.x / LPH;
    const int ch = lane * 8;
    const int total = nt * heads;
    for (int r0 = slot; r0 < total + slot; r0 += SLOTS * kRows) {
        uint4 raw[kRows];
        int tok[kRows], head[kRows];
#pragma unroll
        for (int e = 0; e < kRows; ++e) {
            const int r = r0 + e * SLOTS;
            tok[e] = r / heads;
            head[e] = r - tok[e] * heads;
            raw[e] = make_uint4(0, 0, 0, 0);
            if (r < total) {
                const long long t = t0 + tok[e];
                const uint16_t *src = head[e] < p.Hq ? p.q + t * p.ld_q + (long long)head[e] * D
                                                     : p.k + t * p.ld_k + (long long)(head[e] - p.Hq) * D;
                raw[e] = ld_stream(src + ch);
            }
        }
#pragma unroll
        for (int e = 0; e < kRows; ++e) {
            const int r = r0 + e * SLOTS;
            const bool is_q = head[e] < p.Hq;
            float x[8];
            unpack<uint16_t, 8>(raw[e], x);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
            float m = is_q ? p.scale_q : p.scale_k;
            if (p.norm == RS_NORM_L2) {
                const float n = sqrtf(ss);
                m /= n < p.eps ? p.eps : n;  // a NaN norm stays one
            } else if (p.norm == RS_NORM_RMS) {
                m /= sqrtf(ss * (1.f / D) + p.eps);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= m;
            const uint16_t *w = is_q ? p.wq : p.wk;
            if (w) {
                float wf[8];
                unpack<uint16_t, 8>(ld_u4(w + ch), wf);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= wf[i] + p.w0;
            }
            if (half) {
                if (p.interleaved) {
                    if (ch < p.rot) {
                        const float2 *cs = turn + (r < total ? tok[e] : 0) * half + ch / 2;
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float2 z = cs[i / 2];
                            const float a = x[i], b = x[i + 1];
                            x[i] = a * z.x - b * z.y;
                            x[i + 1] = b * z.x + a * z.y;
                        }
                    }
                } else {
                    // lanes of the first and second half exchange their channels
                    const bool lower = ch < half;
                    const int other = lower ? lane + half / 8 : lane - half / 8;
                    const float2 *cs = turn + (r < total ? tok[e] : 0) * half + (lower ? ch : ch - half);
                    const int src = (threadIdx.x & 31) - lane + (ch < p.rot ? other : lane);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float y = __shfl_sync(~0u, x[i], src);
                        if (ch < p.rot) {
                            const float2 z = cs[i];
                            x[i] = lower ? x[i] * z.x - y * z.y : x[i] * z.x + y * z.y;
                        }
                    }
                }
            }
            if (r < total) {
                const long long t = t0 + tok[e];
                uint16_t *dst = is_q ? p.q_out + t * p.ld_qo + (long long)head[e] * D
                                     : p.k_out + t * p.ld_ko + (long long)(head[e] - p.Hq) * D;
                store_bf16<8>(dst + ch, x);
            }
        }
    }
}

}  // namespace

cudaError_t qk_norm_launch(const rs_qk_desc &d, const uint16_t *q, const uint16_t *k, const uint16_t *wq,
                           const uint16_t *wk, const float *inv_freq, const int32_t *positions, uint16_t *q_out,
                           uint16_t *k_out, cudaStream_t s) {
    QkParams p = {d.T, d.Hq, d.Hk, d.norm, d.rot, d.interleaved, 1, d.eps, d.weight_offset, d.scale_q, d.scale_k,
                  d.ld_q, d.ld_k, d.ld_qo, d.ld_ko, q, k, wq, wk, inv_freq, positions, q_out, k_out};
    // Tokens of a CTA: enough heads for one pass of all threads, as long as the grid still covers the SMs
    const int slots = kThreads / (d.D / 8), heads = d.Hq + d.Hk;
    while (p.tokens < kMaxTokens && p.tokens * heads < slots * kRows && d.T > p.tokens * 152 * 2) p.tokens *= 2;
    const int grid = (d.T + p.tokens - 1) / p.tokens;
    const size_t smem = (size_t)p.tokens * (d.rot / 2) * sizeof(float2);
    switch (d.D) {
        case 64: qk_kernel<64><<<grid, kThreads, smem, s>>>(p); break;
        case 128: qk_kernel<128><<<grid, kThreads, smem, s>>>(p); break;
        default: qk_kernel<256><<<grid, kThreads, smem, s>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace rs
