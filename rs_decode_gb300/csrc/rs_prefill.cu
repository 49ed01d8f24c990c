// The gated delta rule over a ragged batch of prompts (rs_prefill_gdn).
//
// Per request and value head, with state S [key n][value p] and rows t:
//   u_t = beta_t (v_t - alpha_t S k_t),  S <- alpha_t S + u_t k_t^T,  y_t = S q_t.
//
// Chunked form.  Over the C = 64 rows of a chunk, with G_i the sum of
// log alpha up to row i, the rows' u solve a unit lower triangular system and
// everything else is a product:
//   (I + A) u = diag(beta) R,  A_ij = beta_i e^(G_i - G_j) k_i.k_j  (j < i),
//   R_i = v_i - e^(G_i) S k_i,
//   y_i = e^(G_i) S q_i + sum_{j <= i} P_ij u_j,  P_ij = e^(G_i - G_j) q_i.k_j,
//   S'  = e^(G_C) S + sum_j e^(G_C - G_j) u_j k_j^T.
//
// T = (I + A)^-1 diag(beta) and P do not depend on the state, so
//   chunk_cta     computes them for all chunks and heads at once, and
//   the scans     carry S through a request's chunks: 128-wide heads on the
//                 tcgen05 tensor cores (rs_prefill_tc.cu), 64-wide ones here.
// Where few chains would leave the GPU idle, a request's chunks are cut into
// segments (rs_prefill.cuh).  Requests of at most kShort rows go through step_cta
// instead, which runs the recurrence row by row beside one read and one write of
// the state.
//
// Measured on a GB300 with 32 value and 16 key heads of 128 (copy peak 6.78 TB/s):
// 256 cached requests of one row 166 us (6.5 TB/s, the states' bytes); 16 prompts
// of 26,458 rows 496 us (chunk matrices 166, scan 335); one request of 32,768 rows
// 1078 us (chunk matrices 198, states and maps of 9 segments 469, joining them 39,
// scan 374).  Besides the 0.79 GB that the prompts cannot do without, the chunk
// matrices leave 0.60 GB (26 to 34 KiB a chunk and head, 32 KiB a chunk and key head)
// which the scan reads again: together 2.6 times the necessary bytes, at 0.65 and 0.48
// of the copy peak in the two kernels, one after the other.  Those bytes and the
// latency within a chunk (rs_prefill_tc.cu) bound them.
//
// Decays enter as differences G_i - G_j only, so nothing overflows however
// long a chunk's decay is; alpha = 0 is a decay of 2^-160, which is 0 in fp32.
// Growth (alpha > 1) by more than 2^6 within a chunk would pass fp16's range in P and
// leave R and u too few bits in rows before it: it is reported.
//
// Precision.  The tensor cores multiply fp16 operands into fp32 sums.  Keys
// and queries (bf16) enter as one fp16 term, each row scaled by a power of two to
// a largest value in [1, 2) (queries [64, 128)): exact down to 2^-17 of that value,
// and off by at most 2^-25 of it below.  Everything else (S, R, T, P, u) enters as the
// sum of two fp16 terms, 22 bits, scaled by a power of two likewise, so that states and
// outputs come out at fp32 accuracy (bf16 terms would leave 16 bits at the same cost),
// as those of the recurrence for short requests do; y is rounded once, to bf16.
// The rows of a chunk share a scale for R and u in each value column, from its largest
// magnitude, and P has a fixed one; their low terms reach 2^-39 and 2^-40 below those,
// so that what replaces a far larger state within one chunk keeps fewer bits in the end.
// A state 2^k times the values, forgotten at row 20 of 64: the new one is 3.3e-7 off up
// to k = 20, 4.1e-6 at 24, 2.2e-4 at 28; fading over 8 to 30 rows, 1.2e-6 at most up to
// 20, 4.6e-6 at 24.  On the way down y is off, beside the terms that it is the sum of,
// by 5e-6 at k = 12, 6e-5 at 14, 1e-3 at 18, and passes its own rounding from 2^20 on.
#include "rs_prefill.cuh"

namespace rs {

using namespace prefill;

namespace {

// ---------------------------------------------------------------- warp matrix products
// mma.sync m16n8k16: lane = 4 g + t.  A: rows g, g+8, columns 2t..2t+1 and
// 2t+8..2t+9; B: rows (k) the same, column g; C: rows g, g+8, columns 2t..2t+1.
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3) : "memory");
}
// 16-byte copy global -> shared; zeros where `ok` is false (nothing is read).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
// The A fragment of 16 x 16 values held as two accumulator tiles, rows g and
// g + 8 scaled by s0 and s1.
__device__ __forceinline__ void split(const float (&c0)[4], const float (&c1)[4], float s0, float s1,
                                      uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c0[0] * s0, c0[1] * s0, hi[0], lo[0]);
    split2(c0[2] * s1, c0[3] * s1, hi[1], lo[1]);
    split2(c1[0] * s0, c1[1] * s0, hi[2], lo[2]);
    split2(c1[2] * s1, c1[3] * s1, hi[3], lo[3]);
}
// Largest magnitudes of rows g and g + 8 over N accumulator tiles.
template <int N>
__device__ __forceinline__ void row_max(const float (&c)[N][4], float &m0, float &m1) {
    m0 = m1 = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        m0 = fmaxf(m0, fmaxf(fabsf(c[i][0]), fabsf(c[i][1])));
        m1 = fmaxf(m1, fmaxf(fabsf(c[i][2]), fabsf(c[i][3])));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, o));
    }
}

// Copies a chunk's 64 rows of D channels, zeros past the n rows it has.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const uint16_t *src, long long ld, int n, int tid, int nt) {
    constexpr int PIECES = D / 8;
    for (int i = tid; i < C * PIECES; i += nt) {
        const int r = i / PIECES, c = i % PIECES;
        cp16(dst + piece(r, c), src + (r < n ? r : 0) * ld + c * 8, r < n);
    }
}

// ---------------------------------------------------------------- chunk matrices
// One CTA per chunk and key head: the products K K^T and Q K^T are shared by
// the key head's value heads, whose decays and betas differ and which are
// served two at a time, 64 threads each.  The triangular inverse is fp32 and
// in place: four 16 x 16 diagonal blocks by substitution (a column per thread),
// then twice  [[a,0],[c,b]]^-1 = [[a',0],[-b' c a', b']]  with the product c a'
// waiting in the unused block above the diagonal.  Substitution over the whole
// 64 rows would be one dependent chain of 2016 steps; the products run on the
// tensor cores with operands split to 22 bits, since every u of the chunk
// inherits T's accuracy.
// 26,458 rows of 32 value and 16 key heads: 166 us at four CTAs an SM, with half of the
// issue slots, 0.65 of shared memory's bandwidth and 0.65 of the copy peak (its records
// and tiles, 0.60 GB, and 0.2 GB of rows) in use: its writes and the latency of shared
// memory and of the barriers between its short phases bound it together.  (Before P had
// two terms: 163 us, and 171 at five CTAs an SM with 96 registers.)
constexpr int kChunkThreads = 128;
// fp32 matrices in shared memory: 16-byte rows, banks shifted by 12.  Rows 0, 2, 4, 6
// and rows 1, 3, 5, 7 then start 8 banks apart, so a fragment whose 8 rows are taken in
// the order of row_of() and whose columns go in pairs meets no bank twice.
constexpr int LDM = C + 12;
__device__ __forceinline__ int row_of(int g) { return (g & 3) << 1 | (g >> 2 & 1); }
constexpr int kMat = C * LDM;

template <int D>
struct ChunkSmem {
    static constexpr int TILES = 2 * C * D * 2;
    static constexpr int MATS = 2 * kMat * 4;
    static constexpr int VECS = TILES > MATS ? TILES : MATS;  // after the tiles, or the matrices in their place
    static constexpr int BYTES = VECS + (2 + 2 * 3) * C * 4 + 16;
};

// Sum of (value, error) pairs: the sum's rounding error goes into the error.
__device__ __forceinline__ void add2(float &h, float &l, float h2, float l2) {
    const float s = h + h2, b = s - h;
    l = l + l2 + ((h - (s - b)) + (h2 - b));
    h = s;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Products of fp32 blocks on the tensor cores: tf32 operands hold 11 bits, so an
// operand enters as hi (cut to 11 bits) plus lo (what is left, which the
// hardware cuts likewise) and a product takes three terms: 22 bits, without a
// scale, since tf32 has fp32's exponent.
// mma.sync m16n8k8: lane = 4 g + t.  A: rows g, g+8, columns t, t+4; B: rows (k)
// t, t+4, column g; C: rows g, g+8, columns 2t, 2t+1.  Row g holds row_of(g) here, and
// t, t+4 hold the k of 2t, 2t+1, for A and B alike.
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <int N>
__device__ __forceinline__ void cut(const float (&x)[N], uint32_t (&hi)[N], uint32_t (&lo)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        hi[i] = __float_as_uint(x[i]) & 0xffffe000u;
        lo[i] = __float_as_uint(x[i] - __uint_as_float(hi[i]));
    }
}
// a, x: a block's first element, rows LDM apart
__device__ __forceinline__ void frag_a(const float *a, int lane, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    const float *p = a + row_of(lane >> 2) * LDM + (lane & 3) * 2;
    const float2 x = *reinterpret_cast<const float2 *>(p), y = *reinterpret_cast<const float2 *>(p + 8 * LDM);
    const float v[4] = {x.x, y.x, x.y, y.y};
    cut(v, hi, lo);
}
__device__ __forceinline__ void frag_b(const float *x, int lane, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
    const float *p = x + (lane & 3) * 2 * LDM + (lane >> 2);
    const float v[2] = {p[0], p[LDM]};
    cut(v, hi, lo);
}
__device__ __forceinline__ void mma3(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[2],
                                     const uint32_t (&bl)[2]) {
    mma_tf32(c, al, bh);
    mma_tf32(c, ah, bl);
    mma_tf32(c, ah, bh);
}
__device__ __forceinline__ void put_c(float *out, int lane, const float (&c)[4], float sign) {
    float *p = out + row_of(lane >> 2) * LDM + (lane & 3) * 2;
    *reinterpret_cast<float2 *>(p) = make_float2(sign * c[0], sign * c[1]);
    *reinterpret_cast<float2 *>(p + 8 * LDM) = make_float2(sign * c[2], sign * c[3]);
}
// out = sign a x for 16 x 16 blocks, by one warp
__device__ __forceinline__ void product16(const float *a, const float *x, float *out, int lane, float sign) {
    float c[2][4] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t ah[4], al[4], bh[2], bl[2];
        frag_a(a + 8 * k, lane, ah, al);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            frag_b(x + 8 * k * LDM + 8 * n, lane, bh, bl);
            mma3(c[n], ah, al, bh, bl);
        }
    }
    put_c(out, lane, c[0], sign);
    put_c(out + 8, lane, c[1], sign);
}

__device__ __forceinline__ void group_sync(int grp) {  // the 64 threads of one head
    if (grp == 0)
        asm volatile("bar.sync 1, 64;" ::: "memory");
    else
        asm volatile("bar.sync 2, 64;" ::: "memory");
}

// By a warp, two rows a lane: reports a chunk whose summed log2 alpha stands more than 6
// above the least before it, below which P stays under 4 D 2^6.
__device__ __noinline__ void report_growth(float x0, float x1, uint32_t *status) {
    const int lane = threadIdx.x & 31;
    x0 = fmaxf(log2f(x0), -160.f), x1 = fmaxf(log2f(x1), -160.f) + x0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(~0u, x1, o);
        if (lane >= o) x0 += x, x1 += x;
    }
    float low = fminf(x0, x1);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(~0u, low, o);
        if (lane >= o) low = fminf(low, x);
    }
    low = __shfl_up_sync(~0u, low, 1);
    low = lane == 0 ? 0.f : fminf(low, 0.f);
    if (fmaxf(x0 - low, x1 - fminf(low, x0)) > 6.f) atomicOr(status, RS_DEV_GATE);
}

template <int D>
__device__ __forceinline__ void chunk_cta(const PrefillParams &p, int cta, unsigned char *smem) {
    const int chunk = cta / p.G, g = cta - chunk * p.G;
    if (chunk >= min(p.rg.counts[1], p.ccap)) return;
    const int4 e = reinterpret_cast<const int4 *>(p.rg.chunks)[chunk];
    const int n = e.z;
    if (e.x < 0 || e.x >= p.R || n < 1 || n > C || e.y < 0 || e.y > p.cap - n) return;  // the scan reports it
    if (p.rg.cu_tokens[e.x + 1] - p.rg.cu_tokens[e.x] <= kShort) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t sK = smem_u32(smem), sQ = sK + C * D * 2;
    load_tile<D>(sK, p.k + (long long)e.y * p.ld_k + g * D, p.ld_k, n, tid, kChunkThreads);
    load_tile<D>(sQ, p.q + (long long)e.y * p.ld_q + g * D, p.ld_q, n, tid, kChunkThreads);
    asm volatile("cp.async.commit_group;" ::: "memory");

    float *sk = reinterpret_cast<float *>(smem + ChunkSmem<D>::VECS), *sq = sk + C;
    float *vec = sq + C;                               // per head of a pair: gh, gl, beta
    int *grows = reinterpret_cast<int *>(vec + 2 * 3 * C);  // an alpha above 1 in the odd heads, in the even ones
    // the first pair's decays are summed while the tiles are on their way
    float h[2], l[2], cgh, cgl;
    auto decays = [&](int hv, float *v) {
        // two rows a lane; sums of log2 alpha as (value, error) pairs, so that
        // differences of large sums keep their low bits
        float *gh = v, *gl = gh + C, *be = gl + C;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const bool in = t < n;
            const float a = in ? p.alpha[(long long)(e.y + t) * p.H + hv] : 1.f;
            be[t] = in ? p.beta[(long long)(e.y + t) * p.H + hv] : 0.f;
            const float x = log2f(a);
            h[i] = x < -160.f ? -160.f : x;
        }
        add2(h[1], l[1], h[0], l[0]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float xh = __shfl_up_sync(~0u, h[1], o), xl = __shfl_up_sync(~0u, l[1], o);
            if (lane >= o) add2(h[1], l[1], xh, xl);
        }
        float ph = __shfl_up_sync(~0u, h[1], 1), pl = __shfl_up_sync(~0u, l[1], 1);
        if (lane == 0) ph = pl = 0.f;
        add2(h[0], l[0], ph, pl);
        cgh = __shfl_sync(~0u, h[1], 31), cgl = __shfl_sync(~0u, l[1], 31);
        gh[2 * lane] = h[0], gl[2 * lane] = l[0], gh[2 * lane + 1] = h[1], gl[2 * lane + 1] = l[1];
    };
    if (warp < 2) {
        if (warp < p.rep) decays(g * p.rep + warp, vec + warp * 3 * C);
    } else {  // the other two look whether any alpha of the key head's is above 1
        bool any = false;
        for (int r = warp - 2; r < p.rep; r += 2) {
            const float *a = p.alpha + (long long)e.y * p.H + g * p.rep + r;
            const float a0 = 2 * lane < n ? a[(long long)(2 * lane) * p.H] : 1.f;
            const float a1 = 2 * lane + 1 < n ? a[(long long)(2 * lane + 1) * p.H] : 1.f;
            if (__any_sync(~0u, fmaxf(a0, a1) > 1.f)) report_growth(a0, a1, p.status), any = true;
        }
        if (lane == 0) grows[warp - 2] = any;
    }
    cp_async_wait_all();
    __syncthreads();

    // bf16 -> fp16 in place, two threads a row: each row scaled to [1, 2), and queries to
    // [64, 128) where no alpha is above 1: P, which has no scale of its own, is then below
    // 2^15, and what a decay leaves of it keeps more bits, as u may be large.  A thread's
    // pieces go by four, so that eight threads meet eight places of a 128-byte row.
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int row = tid >> 1, c0 = (tid & 1) * 4;
        uint4 v[D / 16];
        __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            v[c] = *reinterpret_cast<const uint4 *>(smem + w * (C * D * 2) + piece(row, c0 | (c & 3)) + (c >> 2) * (C * 128));
#pragma unroll
            for (uint32_t x : {v[c].x, v[c].y, v[c].z, v[c].w}) {
                const uint32_t mag = x & 0x7fff7fffu;
                m2 = __hmax2(m2, *reinterpret_cast<const __nv_bfloat162 *>(&mag));
            }
        }
        float m = fmaxf(__low2float(m2), __high2float(m2));
        m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
        float up, down;
        row_scale(w && !(grows[0] | grows[1]) ? 6 : 0, m, up, down);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            auto half2 = [&](uint32_t x) {
                return pack_h2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
            };
            *reinterpret_cast<uint4 *>(smem + w * (C * D * 2) + piece(row, c0 | (c & 3)) + (c >> 2) * (C * 128)) =
                make_uint4(half2(v[c].x), half2(v[c].y), half2(v[c].z), half2(v[c].w));
        }
        if ((tid & 1) == 0) (w ? sq : sk)[row] = down;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {  // both tiles, as they are, to the workspace
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                         p.tiles + ((size_t)chunk * p.G + g) * (2 * C * D * 2)),
                     "r"(sK), "r"(2 * C * D * 2)
                     : "memory");
    }

    // K K^T and Q K^T in 16 x 16 tiles up to the diagonal, three or two a warp: rows 3,
    // 2 and 1 of the tiles from the left, and the corners (0, 0) and (3, 3).  The shares
    // go around the warps (and with them the schedulers) from CTA to CTA.
    const int share = (warp + cta) & 3, tiles = share < 2 ? 3 : 2, corners = share == 3;
    auto tile_row = [&](int s) { return corners ? 3 * s : 3 - share; };
    auto tile_col = [&](int s) { return corners ? 3 * s : s; };
    float kk[3][2][4] = {}, qk[3][2][4] = {};
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
        uint32_t a[4], b[4], w[4];
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            if (s < tiles) {
                if (s == 0 || (s == 1 && corners)) {
                    const int ar = tile_row(s) * 16 + (lane & 8) + row_of(lane), ac = 2 * x + (lane >> 4);
                    ldsm4(a, sK + piece(ar, ac));
                    ldsm4(b, sQ + piece(ar, ac));
                }
                ldsm4(w, sK + piece(16 * tile_col(s) + (lane & 7) + ((lane & 16) >> 1), 2 * x + ((lane >> 3) & 1)));
                mma_f16(kk[s][0], a, w[0], w[1]);
                mma_f16(kk[s][1], a, w[2], w[3]);
                mma_f16(qk[s][0], b, w[0], w[1]);
                mma_f16(qk[s][1], b, w[2], w[3]);
            }
        }
    }
    // keys' powers of two into K K^T
    const int i0 = row_of(lane >> 2), j0 = (lane & 3) * 2;
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        if (s == 2 && tiles == 2) break;
        const int i = tile_row(s) * 16 + i0;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const float2 sj = *reinterpret_cast<const float2 *>(sk + tile_col(s) * 16 + nt * 8 + j0);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                kk[s][nt][2 * hf] *= sj.x * sk[i + 8 * hf];
                kk[s][nt][2 * hf + 1] *= sj.y * sk[i + 8 * hf];
            }
        }
    }
    if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();  // the tiles' place is the matrices' from here

    float *mats = reinterpret_cast<float *>(smem);
    for (int r0 = 0; r0 < p.rep; r0 += 2) {
        const int heads = min(2, p.rep - r0);
        if (warp < heads) {
            float *v = vec + warp * 3 * C;
            if (r0 > 0) decays(g * p.rep + r0 + warp, v);
            Record &out = p.rec[(size_t)chunk * p.H + g * p.rep + r0 + warp];
            const float e0 = exp2f(h[0] + l[0]), e1 = exp2f(h[1] + l[1]);
            const float k0 = exp2f((cgh - h[0]) + (cgl - l[0])), k1 = exp2f((cgh - h[1]) + (cgl - l[1]));
            const float2 skl = *reinterpret_cast<const float2 *>(sk + 2 * lane), sql = *reinterpret_cast<const float2 *>(sq + 2 * lane);
            *reinterpret_cast<float2 *>(out.egk + 2 * lane) = make_float2(e0 * skl.x, e1 * skl.y);
            *reinterpret_cast<float2 *>(out.eg + 2 * lane) = make_float2(e0, e1);
            *reinterpret_cast<float2 *>(out.sq + 2 * lane) = sql;
            *reinterpret_cast<float2 *>(out.ke + 2 * lane) = make_float2(k0, k1);
            if (lane == 31) out.all = e1;
        }
        __syncthreads();
        // this warp's tiles of A and P
        for (int r = 0; r < heads; ++r) {
            const float *gh = vec + r * 3 * C, *gl = gh + C, *be = gl + C;
            float *A = mats + r * kMat;
            unsigned char *pout = reinterpret_cast<unsigned char *>(p.rec[(size_t)chunk * p.H + g * p.rep + r0 + r].p_hi);
            using f2 = unsigned long long;
            f2 hi[2], lo[2], bi[2];
            const f2 one = f2_pack(1.f, 1.f), minus = f2_pack(-1.f, -1.f);
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                if (s == 2 && tiles == 2) break;
                if (s == 0 || (s == 1 && corners)) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int i = tile_row(s) * 16 + i0 + 8 * hf;
                        hi[hf] = f2_pack(gh[i], gh[i]), lo[hf] = f2_pack(gl[i], gl[i]), bi[hf] = f2_pack(be[i], be[i]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int j = tile_col(s) * 16 + nt * 8 + j0;
                    const f2 hj = *reinterpret_cast<const f2 *>(gh + j), lj = *reinterpret_cast<const f2 *>(gl + j);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int i = tile_row(s) * 16 + i0 + 8 * hf;
                        float x0, x1;
                        f2_unpack(f2_fma(f2_fma(hj, minus, hi[hf]), one, f2_fma(lj, minus, lo[hf])), x0, x1);
                        const f2 d = f2_pack(exp2_fast(x0), exp2_fast(x1));
                        float p0, p1, a0, a1;
                        f2_unpack(f2_mul(d, f2_pack(qk[s][nt][2 * hf], qk[s][nt][2 * hf + 1])), p0, p1);
                        f2_unpack(f2_mul(f2_mul(d, bi[hf]), f2_pack(kk[s][nt][2 * hf], kk[s][nt][2 * hf + 1])), a0, a1);
                        if (tile_row(s) == tile_col(s)) {
                            if (j > i) p0 = 0.f;
                            if (j + 1 > i) p1 = 0.f;
                            if (j >= i) a0 = 0.f;
                            if (j + 1 >= i) a1 = 0.f;
                        }
                        *reinterpret_cast<float2 *>(A + i * LDM + j) = make_float2(a0, a1);
                        uint32_t ph, pl;
                        split_cut(p0, p1, ph, pl);
                        unsigned char *at = pout + piece(i, j >> 3) + (lane & 3) * 4;
                        *reinterpret_cast<uint32_t *>(at) = ph;
                        *reinterpret_cast<uint32_t *>(at + C * C * 2) = pl;  // p_lo
                    }
                }
            }
        }
        __syncthreads();
        const int grp = tid >> 6, t = tid & 63;
        if (grp < heads) {
            float *A = mats + grp * kMat;
            {  // diagonal blocks: column t of block t / 16
                const int b = t & ~15, col = t & 15;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float s0 = i == col ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
                    for (int m = 0; m < i; m += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(A + (b + i) * LDM + b + m);
                        s0 = fmaf(-v.x, x[m], s0);
                        if (m + 1 < i) s1 = fmaf(-v.y, x[m + 1], s1);
                        if (m + 2 < i) s0 = fmaf(-v.z, x[m + 2], s0);
                        if (m + 3 < i) s1 = fmaf(-v.w, x[m + 3], s1);
                    }
                    x[i] = s0 + s1;
                }
                __syncwarp();  // a block's columns are one warp's: all of A's block is read
#pragma unroll
                for (int i = 0; i < 16; ++i) A[(b + i) * LDM + b + col] = x[i];
                __syncwarp();
            }
            {  // the two 32 x 32 blocks, one a warp
                float *X = A + (32 * (warp & 1)) * (LDM + 1);
                product16(X + 16 * LDM, X, X + 16, lane, 1.f);
                __syncwarp();
                product16(X + 16 * LDM + 16, X + 16, X + 16 * LDM, lane, -1.f);
            }
            group_sync(grp);
            {  // the 64 x 64 block; zero tiles of the triangular factors are skipped
                const int w = warp & 1;
                {  // c a': 16 rows a warp
                    float c[4][4] = {};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t ah[4], al[4], bh[2], bl[2];
                        frag_a(A + (32 + 16 * w) * LDM + 8 * k, lane, ah, al);
#pragma unroll
                        for (int n = 0; n <= k; ++n) {
                            frag_b(A + 8 * k * LDM + 8 * n, lane, bh, bl);
                            mma3(c[n], ah, al, bh, bl);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n) put_c(A + 16 * w * LDM + 32 + 8 * n, lane, c[n], 1.f);
                }
                group_sync(grp);
                {  // -b' (c a'): 16 columns a warp
                    float c[2][2][4] = {};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t ah[4], al[4], bh[2][2], bl[2][2];
#pragma unroll
                        for (int n = 0; n < 2; ++n) frag_b(A + 8 * k * LDM + 32 + 16 * w + 8 * n, lane, bh[n], bl[n]);
#pragma unroll
                        for (int m = k / 2; m < 2; ++m) {
                            frag_a(A + (32 + 16 * m) * LDM + 32 + 8 * k, lane, ah, al);
                            mma3(c[m][0], ah, al, bh[0], bl[0]);
                            mma3(c[m][1], ah, al, bh[1], bl[1]);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < 2; ++n) put_c(A + (32 + 16 * m) * LDM + 16 * w + 8 * n, lane, c[m][n], -1.f);
                }
            }
            group_sync(grp);
            // T = X diag(beta), each row scaled and split in two; 8 threads a row, and in
            // every eight lanes halves of two rows, which lie on different banks
            Record &out = p.rec[(size_t)chunk * p.H + g * p.rep + r0 + grp];
            const float *be = vec + grp * 3 * C + 2 * C;
            const int c = (t & 3) | (t >> 1 & 4), rl = (t >> 2 & 1) | (t >> 3 & 6);
            const ulonglong2 b0 = *reinterpret_cast<const ulonglong2 *>(be + c * 8), b1 = *reinterpret_cast<const ulonglong2 *>(be + c * 8 + 4);
            const unsigned long long bj[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll 2
            for (int i = 0; i < 8; ++i) {
                const int row = i * 8 + rl;
                // the row's sum of magnitudes sizes its scale: no element passes 2^15, and those
                // that a decay has made small keep their bits, as what they multiply may be large
                using f2 = unsigned long long;
                ulonglong2 v0 = make_ulonglong2(0, 0), v1 = v0;
                if (c / 2 <= i / 2) {  // right of the diagonal's block another block has waited
                    v0 = *reinterpret_cast<const ulonglong2 *>(A + row * LDM + c * 8);
                    v1 = *reinterpret_cast<const ulonglong2 *>(A + row * LDM + c * 8 + 4);
                }
                const f2 w[4] = {f2_mul(v0.x, bj[0]), f2_mul(v0.y, bj[1]), f2_mul(v1.x, bj[2]), f2_mul(v1.y, bj[3])};
                float v[8], sum = 0.f, up, down;
#pragma unroll
                for (int x = 0; x < 4; ++x) f2_unpack(w[x], v[2 * x], v[2 * x + 1]);
#pragma unroll
                for (int x = 0; x < 8; ++x) sum += fabsf(v[x]);
#pragma unroll
                for (int o : {1, 2, 8}) sum += __shfl_xor_sync(~0u, sum, o);
                row_scale<14>(sum, up, down);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) split_cut(v[2 * x] * up, v[2 * x + 1] * up, hi[x], lo[x]);
                *reinterpret_cast<uint4 *>(reinterpret_cast<unsigned char *>(out.t_hi) + piece(row, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(reinterpret_cast<unsigned char *>(out.t_lo) + piece(row, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (c == 0) out.su[row] = down * sk[row];
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- short requests
// The recurrence for requests of a few rows.  A warp owns 16 value columns of
// a head: lane = 4 rg + cg holds keys D/8 rg .. and values 4 cg .. of them in
// registers, so that the state is read and written once, in 64-byte segments
// with 8 KiB in flight per warp, and no warp waits for another.  One row's
// S k, S q and k.q are summed over the lanes together; S_new q follows as
// alpha S q + (k.q) u.  256 cached requests of 32 heads of 128: 166 us for one row,
// 0.95 of the copy peak in the states' bytes (two-precision checkpoints 204 us, 0.97;
// bf16 135, 0.59: its loads and stores are 8 bytes a lane), and 28 us more for each
// further row, which is issue time.
constexpr int kStepThreads = 128;

template <int D>
constexpr int kStepSplit = D / 16 / (kStepThreads / 32);  // CTAs of a head

template <int D>
__device__ __forceinline__ void step_cta(const PrefillParams &p, int cta) {
    constexpr int ROWS = D / 8;  // key rows of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = cta % kStepSplit<D>, hr = cta / kStepSplit<D>;
    const int h = hr % p.H, r = hr / p.H;
    const bool lead = h == 0 && part == 0 && threadIdx.x == 0;
    // longer requests are the scan's, where it runs at all
    if (p.max_len > kShort && p.rg.cu_tokens[r + 1] - p.rg.cu_tokens[r] > kShort) return;
    const Request rq = load_request(p, r, lead);
    if (!rq.ok) return;
    const int g = h / p.rep;
    const int col = (part * (kStepThreads / 32) + warp) * 16 + (lane & 3) * 4, row0 = (lane >> 2) * ROWS;

    // later rows' inputs on their way to the cache, a line or two a lane: rows
    // follow one another too closely to wait for memory in between
    for (int i = lane; i < (rq.n - 1) * 8; i += 32) {
        const long long row = rq.row0 + 1 + (i >> 3);
        const int w = i & 7;
        const void *at = w < 2   ? (const void *)(p.k + row * p.ld_k + g * D + (w & 1) * (D / 2))
                         : w < 4 ? (const void *)(p.q + row * p.ld_q + g * D + (w & 1) * (D / 2))
                         : w < 5 ? (const void *)(p.v + row * p.ld_v + h * D + col)
                         : w < 6 ? (const void *)(p.alpha + row * p.H + h)
                                 : (const void *)(p.beta + row * p.H + h);
        asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
    }
    float4 S[ROWS];
    {
        const bool cont = rq.start == -2;
        const size_t slab = ((size_t)(cont ? rq.srow : max(rq.start, 0)) * p.H + h) * D * D + (size_t)row0 * D + col;
        if (rq.start == -1) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else if (p.prec == RS_PREC_SHARED_BF16) {
            const uint16_t *b = (cont ? p.lp : static_cast<const uint16_t *>(p.pool)) + slab;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(b + (size_t)i * D));
                S[i] = make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                   __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
            }
        } else {
            const float *f = (cont ? p.hp : static_cast<const float *>(p.pool)) + slab;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) S[i] = __ldcs(reinterpret_cast<const float4 *>(f + (size_t)i * D));
        }
    }
    auto store_state = [&](float *f, uint16_t *b, size_t slab) {
        slab += (size_t)row0 * D + col;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (f) __stcs(reinterpret_cast<float4 *>(f + slab + (size_t)i * D), S[i]);
            if (b) st_stream2(b + slab + (size_t)i * D, make_uint2(pack_bf2(S[i].x, S[i].y), pack_bf2(S[i].z, S[i].w)));
        }
    };
    for (int t = 0; t < rq.n; ++t) {
        const long long row = rq.row0 + t;
        const uint4 *kp = reinterpret_cast<const uint4 *>(p.k + row * p.ld_k + g * D + row0);
        const uint4 *qp = reinterpret_cast<const uint4 *>(p.q + row * p.ld_q + g * D + row0);
        const uint2 vp = *reinterpret_cast<const uint2 *>(p.v + row * p.ld_v + h * D + col);
        const float alpha = p.alpha[row * p.H + h], beta = p.beta[row * p.H + h];
        float k[ROWS];
        float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
        float kq = 0.f;
#pragma unroll
        for (int c = 0; c < ROWS / 8; ++c) {
            float kk[8], qq[8];
            unpack<uint16_t, 8>(kp[c], kk);
            unpack<uint16_t, 8>(qp[c], qq);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 s = S[c * 8 + i];
                sk.x = fmaf(kk[i], s.x, sk.x), sk.y = fmaf(kk[i], s.y, sk.y);
                sk.z = fmaf(kk[i], s.z, sk.z), sk.w = fmaf(kk[i], s.w, sk.w);
                sq.x = fmaf(qq[i], s.x, sq.x), sq.y = fmaf(qq[i], s.y, sq.y);
                sq.z = fmaf(qq[i], s.z, sq.z), sq.w = fmaf(qq[i], s.w, sq.w);
                kq = fmaf(kk[i], qq[i], kq);
                k[c * 8 + i] = kk[i];
            }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            sk.x += __shfl_xor_sync(~0u, sk.x, o), sk.y += __shfl_xor_sync(~0u, sk.y, o);
            sk.z += __shfl_xor_sync(~0u, sk.z, o), sk.w += __shfl_xor_sync(~0u, sk.w, o);
            sq.x += __shfl_xor_sync(~0u, sq.x, o), sq.y += __shfl_xor_sync(~0u, sq.y, o);
            sq.z += __shfl_xor_sync(~0u, sq.z, o), sq.w += __shfl_xor_sync(~0u, sq.w, o);
            kq += __shfl_xor_sync(~0u, kq, o);
        }
        float4 u;
        u.x = beta * (__uint_as_float(vp.x << 16) - alpha * sk.x);
        u.y = beta * (__uint_as_float(vp.x & 0xffff0000u) - alpha * sk.y);
        u.z = beta * (__uint_as_float(vp.y << 16) - alpha * sk.z);
        u.w = beta * (__uint_as_float(vp.y & 0xffff0000u) - alpha * sk.w);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            S[i].x = fmaf(k[i], u.x, alpha * S[i].x), S[i].y = fmaf(k[i], u.y, alpha * S[i].y);
            S[i].z = fmaf(k[i], u.z, alpha * S[i].z), S[i].w = fmaf(k[i], u.w, alpha * S[i].w);
        }
        if (lane < 4)
            *reinterpret_cast<uint2 *>(p.y + (row * p.H + h) * D + col) =
                make_uint2(pack_bf2(fmaf(kq, u.x, alpha * sq.x), fmaf(kq, u.y, alpha * sq.y)),
                           pack_bf2(fmaf(kq, u.z, alpha * sq.z), fmaf(kq, u.w, alpha * sq.w)));
        const int slot = block_slot(p, r, rq.ctx + t + 1, lead);
        if (slot >= 0) {
            const size_t slab = ((size_t)slot * p.H + h) * D * D;
            if (p.prec == RS_PREC_SHARED_BF16)
                store_state(nullptr, static_cast<uint16_t *>(p.pool), slab);
            else
                store_state(static_cast<float *>(p.pool), nullptr, slab);
        }
    }
    store_state(p.hp, p.lp, ((size_t)rq.srow * p.H + h) * D * D);
    if (rq.start != -2 && lead) p.base[rq.srow] = p.h[rq.srow] = p.nd[rq.srow] = 0;
}

template <int D>
__global__ void __launch_bounds__(kStepThreads, 4) step_kernel(const __grid_constant__ PrefillParams p) {
    step_cta<D>(p, blockIdx.x);
}

// ---------------------------------------------------------------- front kernel
// What comes before the scan: the short requests' rows, bound by memory
// latency, beside the long requests' chunk matrices, bound by issue.
static_assert(kStepThreads == kChunkThreads, "one launch runs both");
template <int D>
__global__ void __launch_bounds__(kChunkThreads, 4) front_kernel(const __grid_constant__ PrefillParams p, int steps) {
    extern __shared__ __align__(128) unsigned char smem[];
    let_next_launch();
    if ((int)blockIdx.x < steps)
        step_cta<D>(p, blockIdx.x);
    else
        chunk_cta<D>(p, blockIdx.x - steps, smem);
}

// ---------------------------------------------------------------- scan kernel
// A warp owns 16 value columns of a head's state and carries them through the
// request's chunks on its own: S^T (16 x D) lives in the accumulators of
// m16n8k16 products, whose register layout is also that of their A operand, so
//   S^T K^T, S^T Q^T  ->  R^T  ->  u^T = R^T T^T  ->  y^T += u^T P^T,  S^T += u^T K
// pass from product to product without leaving the registers or meeting
// another warp.  K, Q, T and V come through two shared-memory stages; P, needed last,
// through one, so that two CTAs fit an SM.
// It serves 64-wide heads, whose 64 rows would fill half of a tcgen05 product.
// 24 requests with 2,419 rows in all, 8 heads of 64: 68 us, 2.7 us a chunk of the longest
// chain (4.9 for each of two CTAs on an SM); the warp's own products (312 of m16n8k16 a
// chunk, 8 clocks each) are about half of that.
template <int D>
struct ScanSmem {
    static constexpr int NW = D / 16;  // warps of a head
    static constexpr int TILE = C * D * 2;
    static constexpr int VT = NW * C * 32;  // per warp: 64 rows of its 16 columns
    static constexpr int T = 2 * TILE + VT;
    static constexpr int VEC = T + 2 * C * C * 2;
    static constexpr int STAGE = VEC + kRecVecs;
    static constexpr int P = 2 * STAGE;  // one buffer: hi, lo
    static constexpr int BYTES = P + 2 * C * C * 2;
};

template <int D, bool OUT>
__global__ void __launch_bounds__(2 * D) scan_kernel(const __grid_constant__ PrefillParams p, int units) {
    using M = ScanSmem<D>;
    constexpr int NW = M::NW, NT = NW * 32;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hr = blockIdx.x;
    if (blockIdx.x == 0) wait_for_launch();  // so that this launch does not end before the one it overlaps
    int q;
    const int h = hr % p.H, r = cta_request(p, hr / p.H, units, q);
    if (r < 0) return;
    const Request rq = load_request(p, r, h == 0 && q == 0 && tid == 0);
    if (!rq.ok) return;
    const Unit un = scan_unit<OUT>(p, hr, rq, r, q);
    if (!un.ok) return;
    const int g = h / p.rep;
    const int col0 = warp * 16;
    const uint32_t s0 = smem_u32(smem);

    // chunk i of the request: its first row and row count
    const int head_rows = min(rq.n, C - rq.ctx % C);
    auto first_row = [&](int i) { return i == 0 ? 0 : head_rows + (i - 1) * C; };
    auto fetch = [&](int i, uint32_t st) {
        const int at = first_row(i), n = min(i == 0 ? head_rows : C, rq.n - at);
        const long long row = rq.row0 + at;
        const unsigned char *kq = p.tiles + ((size_t)(rq.chunk0 + i) * p.G + g) * (2 * M::TILE);
        for (int x = tid; x < 2 * M::TILE / 16; x += NT) cp16(st + x * 16, kq + x * 16, true);
        const uint16_t *v = p.v + row * p.ld_v + h * D;
        for (int x = tid; x < C * NW * 2; x += NT) {
            const int t = x / (NW * 2), c = x % (NW * 2);
            cp16(st + 2 * M::TILE + (c >> 1) * (C * 32) + t * 32 + (((c & 1) ^ ((t >> 2) & 1)) << 4),
                 v + (t < n ? t : 0) * p.ld_v + c * 8, t < n && !un.map);
        }
        const Record *rec = p.rec + (size_t)(rq.chunk0 + i) * p.H + h;
        const unsigned char *t = reinterpret_cast<const unsigned char *>(rec->t_hi), *vec = reinterpret_cast<const unsigned char *>(rec->egk);
        for (int x = tid; x < 2 * C * C * 2 / 16; x += NT) cp16(st + M::T + x * 16, t + x * 16, true);
        for (int x = tid; x < kRecVecs / 16; x += NT) cp16(st + M::VEC + x * 16, vec + x * 16, true);
    };
    auto fetch_p = [&](int i) {
        const unsigned char *src = reinterpret_cast<const unsigned char *>(p.rec[(size_t)(rq.chunk0 + i) * p.H + h].p_hi);
        for (int x = tid; x < 2 * C * C * 2 / 16; x += NT) cp16(s0 + M::P + x * 16, src + x * 16, true);
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

    // the starting state: S^T[p][n], rows p = col0 + gr (+8), columns n = 8 nt + 2 tq (+1)
    const int gr = lane >> 2, tq = lane & 3;
    float S[D / 8][4];
    {
        const StateSource from = unit_start<OUT, D>(p, rq, un);
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int k = nt * 8 + tq * 2 + (x & 1), c = col0 + gr + 8 * (x >> 1);
                S[nt][x] = from.kind == 0 ? 0.f : from.kind == 1 ? (k == c ? 1.f : 0.f) : from.kind == 2 ? from.f[k * D + c] : bf2f(from.b[k * D + c]);
            }
    }
    auto store_state = [&](float *f, uint16_t *b, size_t slab) {
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const size_t o = slab + (size_t)(nt * 8 + tq * 2 + (x & 1)) * D + col0 + gr + 8 * (x >> 1);
                if (f) f[o] = S[nt][x];
                if (b) b[o] = (uint16_t)f2bf(S[nt][x]);
            }
    };

    wait_for_launch();  // for the chunks' records
    fetch(un.c0, s0);
    commit();
    if (!OUT && un.seg == 0) store_state(p.segs, nullptr, seg_slab(p, un, 0, D * D));  // for the second pass

    for (int i = un.c0; i < un.c1; ++i) {
        const int odd = (i - un.c0) & 1;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // this chunk's stage has landed, and every warp is done with the other one
        const uint32_t st = s0 + odd * M::STAGE;
        if (OUT) {
            fetch_p(i);  // the last chunk's are used up as well
            commit();
        }
        if (i + 1 < un.c1) fetch(i + 1, s0 + (odd ^ 1) * M::STAGE);
        commit();
        const uint32_t sK = st, sQ = st + M::TILE, sV = st + 2 * M::TILE + warp * (C * 32);
        const uint32_t sTh = st + M::T, sTl = sTh + C * C * 2, sPh = s0 + M::P, sPl = sPh + C * C * 2;
        const Vecs *rec = reinterpret_cast<const Vecs *>(smem + odd * M::STAGE + M::VEC);

        // S^T K^T and S^T Q^T: columns are the chunk's rows
        float X[8][4] = {}, Z[8][4] = {};
        float ms0, ms1, su0, su1, sd0, sd1;
        row_max(S, ms0, ms1);
        row_scale<14>(ms0, su0, sd0);
        row_scale<14>(ms1, su1, sd1);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t hi[4], lo[4], b[4];
            split(S[2 * x], S[2 * x + 1], su0, su1, hi, lo);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t o = piece(16 * j + (lane & 7) + ((lane & 16) >> 1), 2 * x + ((lane >> 3) & 1));
                ldsm4(b, sK + o);
                mma_f16(X[2 * j], hi, b[0], b[1]);
                mma_f16(X[2 * j + 1], hi, b[2], b[3]);
                mma_f16(X[2 * j], lo, b[0], b[1]);
                mma_f16(X[2 * j + 1], lo, b[2], b[3]);
                if (OUT) {
                    ldsm4(b, sQ + o);
                    mma_f16(Z[2 * j], hi, b[0], b[1]);
                    mma_f16(Z[2 * j + 1], hi, b[2], b[3]);
                    mma_f16(Z[2 * j], lo, b[0], b[1]);
                    mma_f16(Z[2 * j + 1], lo, b[2], b[3]);
                }
            }
        }
        // R^T = V^T - e^G S^T K^T, and the state's part of y
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t v[4];
            const int t = 16 * j + (lane & 7) + ((lane & 16) >> 1), c = (lane >> 3) & 1;
            ldsm4t(v, sV + t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int nt = 2 * j + hf;
                const float2 ek = *reinterpret_cast<const float2 *>(rec->egk + nt * 8 + tq * 2);
                const float2 eg = *reinterpret_cast<const float2 *>(rec->eg + nt * 8 + tq * 2);
                // the vectors' powers of two and the rows' first: their product is near 1, the sums alone may not fit
                X[nt][0] = __uint_as_float(v[2 * hf] << 16) - ek.x * sd0 * X[nt][0];
                X[nt][1] = __uint_as_float(v[2 * hf] & 0xffff0000u) - ek.y * sd0 * X[nt][1];
                X[nt][2] = __uint_as_float(v[2 * hf + 1] << 16) - ek.x * sd1 * X[nt][2];
                X[nt][3] = __uint_as_float(v[2 * hf + 1] & 0xffff0000u) - ek.y * sd1 * X[nt][3];
                const float2 sq = *reinterpret_cast<const float2 *>(rec->sq + nt * 8 + tq * 2);
                Z[nt][0] *= eg.x * sq.x * sd0, Z[nt][1] *= eg.y * sq.y * sd0;
                Z[nt][2] *= eg.x * sq.x * sd1, Z[nt][3] *= eg.y * sq.y * sd1;
            }
        }
        // u^T = R^T T^T; T is lower triangular.  u carries its key's power of two.
        float U[8][4] = {};
        {
            float m0, m1, u0, u1, d0, d1;
            row_max(X, m0, m1);
            row_scale<14>(m0, u0, d0);
            row_scale<14>(m1, u1, d1);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t hi[4], lo[4], b[4];
                split(X[2 * x], X[2 * x + 1], u0, u1, hi, lo);
#pragma unroll
                for (int j = x; j < 4; ++j) {
                    const uint32_t o = piece(16 * j + (lane & 7) + ((lane & 16) >> 1), 2 * x + ((lane >> 3) & 1));
                    ldsm4(b, sTh + o);
                    mma_f16(U[2 * j], hi, b[0], b[1]);
                    mma_f16(U[2 * j + 1], hi, b[2], b[3]);
                    mma_f16(U[2 * j], lo, b[0], b[1]);
                    mma_f16(U[2 * j + 1], lo, b[2], b[3]);
                    ldsm4(b, sTl + o);
                    mma_f16(U[2 * j], hi, b[0], b[1]);
                    mma_f16(U[2 * j + 1], hi, b[2], b[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 su = *reinterpret_cast<const float2 *>(rec->su + nt * 8 + tq * 2);
                U[nt][0] *= su.x * d0, U[nt][1] *= su.y * d0, U[nt][2] *= su.x * d1, U[nt][3] *= su.y * d1;
            }
        }
        // y^T = (e^G S^T Q^T + u^T P^T) with the queries' powers of two
        if (OUT) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();  // P has landed
            float m0, m1, u0, u1, d0, d1;
            row_max(U, m0, m1);
            row_scale<14>(m0, u0, d0);
            row_scale<14>(m1, u1, d1);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) X[nt][0] = X[nt][1] = X[nt][2] = X[nt][3] = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t hi[4], lo[4], b[4];
                split(U[2 * x], U[2 * x + 1], u0, u1, hi, lo);
#pragma unroll
                for (int j = x; j < 4; ++j) {
                    const uint32_t o = piece(16 * j + (lane & 7) + ((lane & 16) >> 1), 2 * x + ((lane >> 3) & 1));
                    ldsm4(b, sPh + o);
                    mma_f16(X[2 * j], hi, b[0], b[1]);
                    mma_f16(X[2 * j + 1], hi, b[2], b[3]);
                    mma_f16(X[2 * j], lo, b[0], b[1]);
                    mma_f16(X[2 * j + 1], lo, b[2], b[3]);
                    ldsm4(b, sPl + o);
                    mma_f16(X[2 * j], hi, b[0], b[1]);
                    mma_f16(X[2 * j + 1], hi, b[2], b[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 sq = *reinterpret_cast<const float2 *>(rec->sq + nt * 8 + tq * 2);
                Z[nt][0] += d0 * sq.x * X[nt][0], Z[nt][1] += d0 * sq.y * X[nt][1];
                Z[nt][2] += d1 * sq.x * X[nt][2], Z[nt][3] += d1 * sq.y * X[nt][3];
            }
        }
        // S^T = e^(G_C) S^T + (e^(G_C - G) u)^T K, summed at u's row scale.  Where u is
        // below 2^-30 of the row's state, the state's size sets the scale: at u's own
        // the sum could overflow, and u's lost bits are far below the state's last one.
        {
            const float all = rec->all;
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 ke = *reinterpret_cast<const float2 *>(rec->ke + nt * 8 + tq * 2);
                U[nt][0] *= ke.x, U[nt][1] *= ke.y, U[nt][2] *= ke.x, U[nt][3] *= ke.y;
            }
            float m0, m1, u0, u1, d0, d1;
            row_max(U, m0, m1);
            row_scale<14>(fmaxf(m0, all * ms0 * 9.31322574615478515625e-10f), u0, d0);
            row_scale<14>(fmaxf(m1, all * ms1 * 9.31322574615478515625e-10f), u1, d1);
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt) {
                S[nt][0] *= all * u0, S[nt][1] *= all * u0, S[nt][2] *= all * u1, S[nt][3] *= all * u1;
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t hi[4], lo[4], b[4];
                split(U[2 * x], U[2 * x + 1], u0, u1, hi, lo);
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    ldsm4t(b, sK + piece(16 * x + (lane & 15), 2 * j + (lane >> 4)));
                    mma_f16(S[2 * j], hi, b[0], b[1]);
                    mma_f16(S[2 * j + 1], hi, b[2], b[3]);
                    mma_f16(S[2 * j], lo, b[0], b[1]);
                    mma_f16(S[2 * j + 1], lo, b[2], b[3]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < D / 8; ++nt) S[nt][0] *= d0, S[nt][1] *= d0, S[nt][2] *= d1, S[nt][3] *= d1;
        }
        if (!OUT) continue;
        // y through the warp's own V rows, to whole sectors
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 16 * j + (lane & 7) + ((lane & 16) >> 1), c = (lane >> 3) & 1;
            stsm4t(sV + t * 32 + ((c ^ ((t >> 2) & 1)) << 4), pack_bf2(Z[2 * j][0], Z[2 * j][1]),
                   pack_bf2(Z[2 * j][2], Z[2 * j][3]), pack_bf2(Z[2 * j + 1][0], Z[2 * j + 1][1]),
                   pack_bf2(Z[2 * j + 1][2], Z[2 * j + 1][3]));
        }
        __syncwarp();
        const int at = first_row(i), n = min(i == 0 ? head_rows : C, rq.n - at);
        uint16_t *y = p.y + ((long long)(rq.row0 + at) * p.H + h) * D + col0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int t = x * 16 + (lane >> 1), c = lane & 1;
            if (t < n) {
                const uint4 w = *reinterpret_cast<const uint4 *>(smem + (sV - s0) + t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
                *reinterpret_cast<uint4 *>(y + (long long)t * p.H * D + c * 8) = w;
            }
        }
        const int slot = block_slot(p, r, rq.ctx + at + n, h == 0 && tid == 0);
        if (slot >= 0) {
            const size_t slab = ((size_t)slot * p.H + h) * D * D;
            if (p.prec == RS_PREC_SHARED_BF16)
                store_state(nullptr, static_cast<uint16_t *>(p.pool), slab);
            else
                store_state(static_cast<float *>(p.pool), nullptr, slab);
        }
    }
    if (!OUT) {
        if (un.map)
            store_state(p.maps, nullptr, seg_slab(p, un, un.seg, D * D));
        else
            store_state(p.segs, nullptr, seg_slab(p, un, un.seg + 1, D * D));
        return;
    }
    if (un.seg < un.nsegs - 1) return;
    store_state(p.hp, p.lp, ((size_t)rq.srow * p.H + h) * D * D);
    // a fresh start drops what the row had buffered (a continued row has nothing)
    if (rq.start != -2 && h == 0 && tid == 0) p.base[rq.srow] = p.h[rq.srow] = p.nd[rq.srow] = 0;
}

// ---------------------------------------------------------------- combine kernel
// S_(s+1) = M_s S_s + B_s over a request's segments, in order: per head and W
// value columns one CTA, which keeps S_s's columns in shared memory while the
// next M_s and B_s are on their way.  fp32 throughout.  A step reads a 64 KiB
// map for few columns: narrow CTAs shorten the step, wide ones read the map
// less often.  8 heads of 128, 31 segments: 8 columns a CTA took the whole call from
// 326 us (32 columns) to 243.
template <int D, int W>
struct CombineSmem {
    static constexpr int LD = D + 4;
    static constexpr int MAP = D * LD * 4;
    static constexpr int BYTES = 2 * MAP + 2 * D * W * 4;
};

template <int D, int W>
__global__ void __launch_bounds__(2 * D) combine_kernel(const __grid_constant__ PrefillParams p) {
    using M = CombineSmem<D, W>;
    using f2 = unsigned long long;
    constexpr int NR = W / 8;  // rows of a thread, four columns each
    extern __shared__ __align__(128) unsigned char smem[];
    const int part = blockIdx.x % (D / W), hr = blockIdx.x / (D / W);
    const int tid = threadIdx.x;
    Unit u;
    u.h = hr % p.H, u.r = hr / p.H;
    if (p.rg.cu_tokens[u.r + 1] - p.rg.cu_tokens[u.r] <= kShort) return;
    const Request rq = load_request(p, u.r, false);
    if (!rq.ok) return;
    const int last = (rq.nch + p.seglen - 1) / p.seglen - 1;  // steps 1 .. last - 1
    if (last < 2) return;
    const uint32_t s0 = smem_u32(smem);
    float *X = reinterpret_cast<float *>(smem + 2 * M::MAP);  // two buffers [D][W]
    auto fetch = [&](int s) {
        const float *src = p.maps + seg_slab(p, u, s, D * D);
        const uint32_t dst = s0 + (s & 1) * M::MAP;
        for (int i = tid; i < D * D / 4; i += 2 * D) cp16(dst + (i / (D / 4)) * (M::LD * 4) + (i % (D / 4)) * 16, src + i * 4, true);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(1);
    const int n = tid / (W / 4) * NR, c = tid % (W / 4) * 4;  // rows n.., columns c..c + 3
    auto slab = [&](int s) { return p.segs + seg_slab(p, u, s, D * D) + (size_t)n * D + part * W + c; };
    f2 next[NR][2];
    auto load_b = [&](int s) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(slab(s) + i * D);
            next[i][0] = v.x, next[i][1] = v.y;
        }
    };
#pragma unroll
    for (int i = 0; i < NR; ++i)
        *reinterpret_cast<float4 *>(X + (n + i) * W + c) = *reinterpret_cast<const float4 *>(slab(1) + i * D);
    load_b(2);
    for (int s = 1; s < last; ++s) {
        f2 acc[NR][2];
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[i][0] = next[i][0], acc[i][1] = next[i][1];
        if (s + 1 < last) {
            fetch(s + 1);
            load_b(s + 2);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const float *m = reinterpret_cast<const float *>(smem + (s & 1) * M::MAP) + n * M::LD;
        const float *x = X + ((s - 1) & 1) * (D * W) + c;
#pragma unroll 4
        for (int k = 0; k < D; k += 4) {
            float w[NR][4];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(m + i * M::LD + k);
                w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w;
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(x + (k + kk) * W);
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const f2 a = f2_pack(w[i][kk], w[i][kk]);
                    acc[i][0] = f2_fma(a, v.x, acc[i][0]), acc[i][1] = f2_fma(a, v.y, acc[i][1]);
                }
            }
        }
        float *y = X + (s & 1) * (D * W) + c;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const ulonglong2 v = make_ulonglong2(acc[i][0], acc[i][1]);
            *reinterpret_cast<ulonglong2 *>(slab(s + 1) + i * D) = v;
            *reinterpret_cast<ulonglong2 *>(y + (n + i) * W) = v;
        }
        __syncthreads();  // the next columns are complete, and this map's place is free
    }
}

template <int D, int W>
cudaError_t combine_launch(const PrefillParams &p, cudaStream_t s) {
    static SmemGrants grants;
    const cudaError_t e = grant_smem(reinterpret_cast<const void *>(&combine_kernel<D, W>), CombineSmem<D, W>::BYTES, grants);
    if (e != cudaSuccess) return e;
    combine_kernel<D, W><<<p.R * p.H * (D / W), 2 * D, CombineSmem<D, W>::BYTES, s>>>(p);
    return cudaGetLastError();
}

template <int D, bool OUT>
cudaError_t scans(const PrefillParams &p, cudaStream_t s) {
    if constexpr (D == 128) {
        return scan_tc_launch<OUT>(p, s);
    } else {
        static SmemGrants grants;
        const cudaError_t e = grant_smem(reinterpret_cast<const void *>(&scan_kernel<D, OUT>), ScanSmem<D>::BYTES, grants);
        if (e != cudaSuccess) return e;
        const int units = scan_units<OUT>(p);
        return launch_after(scan_kernel<D, OUT>, p.classes * p.R * p.H * units, 2 * D, ScanSmem<D>::BYTES, s, start_early(p), p, units);
    }
}

template <int D>
cudaError_t launch(const PrefillParams &p, cudaStream_t s) {
    const int steps = p.R * p.H * kStepSplit<D>;
    if (p.max_len <= kShort) {
        step_kernel<D><<<steps, kStepThreads, 0, s>>>(p);
        return cudaGetLastError();
    }
    static SmemGrants grants;
    cudaError_t e = grant_smem(reinterpret_cast<const void *>(&front_kernel<D>), ChunkSmem<D>::BYTES, grants);
    if (e != cudaSuccess) return e;
    front_kernel<D><<<steps + p.ccap * p.G, kChunkThreads, ChunkSmem<D>::BYTES, s>>>(p, steps);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.nseg > 1) {
        e = scans<D, false>(p, s);
        if (e != cudaSuccess) return e;
        // the narrowest columns that still run in one wave of a CTA an SM (32 heads of 128,
        // 9 segments: 50 us at 32 columns, 63 at 16 in two waves)
        const int slabs = p.R * p.H * D;
        e = slabs / 8 <= 152 ? combine_launch<D, 8>(p, s) : slabs / 16 <= 152 ? combine_launch<D, 16>(p, s) : combine_launch<D, 32>(p, s);
        if (e != cudaSuccess) return e;
    }
    return scans<D, true>(p, s);
}

// Segments of a request (1: none), from what the host knows: the chains alone,
// requests x heads, against the 304 CTAs that the GPU holds at once; a segment is
// eight chunks at least, or it would spend its time on starting up.  Segmented
// against one chain each, requests of 16,384 rows and 128-wide heads (us): 9
// segments (32 chains) 579 and 1,244, 5 (60) 918 and 1,322, 4 (76) 1,117 and 1,365,
// 3 (96) 1,229 and 1,422, 2 (128) 1,744 and 1,513; of 64-wide heads 425 and 770, 660
// and 843, 811 and 882, 919 and 928, 1,301 and 1,008.  They start at five, where
// requests of 4,096 rows gain a tenth and more too (4: 335 and 358, 237 and 233).  Short
// requests beside a long one count as chains as well: the host does not know them.
void plan_segments(const rs_layer_desc &d, const rs_ragged_desc &rd, int max_len, int &nseg, int &seglen) {
    const int chunks = (max_len < rd.tokens_cap ? max_len : rd.tokens_cap) / C + 2;
    const long long chains = (long long)rd.R * d.H;
    long long want = chains < 304 ? 304 / chains : 1;
    if (want > chunks / 8) want = chunks / 8;
    nseg = want >= 5 ? (int)want : 1;
    seglen = (chunks + nseg - 1) / nseg;
}

}  // namespace

// The workspace: records, fp16 keys and queries, segments' states and maps.
size_t prefill_bytes(const rs_layer_desc &d, const rs_ragged_desc &rd, int max_len) {
    if (max_len <= kShort) return 0;
    int nseg, seglen;
    plan_segments(d, rd, max_len, nseg, seglen);
    return (size_t)ragged_chunks_cap(rd) * (d.H * sizeof(Record) + (size_t)d.G * 2 * C * d.N * 2) +
           (nseg > 1 ? 2 * (size_t)rd.R * d.H * nseg * d.N * d.P * 4 : 0);
}

cudaError_t prefill_launch(const rs_layer_desc &d, const rs_state &st, const rs_ragged_desc &rd, const rs_ragged &rg,
                           const rs_prefill &in, uint16_t *y, void *work, cudaStream_t s) {
    PrefillParams p = {};
    p.H = d.H, p.G = d.G, p.rep = d.H / d.G, p.prec = d.precision & ~RS_U_BF16, p.B = d.B;
    p.R = rd.R, p.cap = rd.tokens_cap, p.ccap = ragged_chunks_cap(rd), p.block = rd.block, p.max_blocks = rd.max_blocks;
    p.n_pool = in.n_pool, p.max_len = in.max_len;
    p.hp = st.ckpt_hp, p.lp = st.ckpt_lp, p.base = st.base, p.h = st.h, p.nd = st.nd, p.status = st.status;
    p.rg = rg;
    p.q = in.q, p.k = in.k, p.v = in.v, p.alpha = in.alpha, p.beta = in.beta;
    p.ld_q = in.ld_q, p.ld_k = in.ld_k, p.ld_v = in.ld_v;
    p.rows = in.rows, p.start = in.start, p.pool = in.pool, p.y = y, p.rec = static_cast<Record *>(work);
    p.tiles = static_cast<unsigned char *>(work) + (size_t)p.ccap * d.H * sizeof(Record);
    plan_segments(d, rd, in.max_len, p.nseg, p.seglen);
    // Passes over the requests, longest first, where the chains fill the GPU, but not so
    // often that the last one does not show.  Prompts of 300 to 4,000 rows, four passes
    // against one (us): 512 chains of 128-wide heads 483 and 547, 1,952 chains 1,727 and
    // 1,833; 1,024 of 64-wide heads 684 and 807.  Below 304 they only move chains together
    // on some SMs: 128 chains 332 and 315, of 64-wide heads 230 and 207.  A pass costs a
    // CTA for each chain that leaves at once: 4,096 chains of 1 to 900 rows 516 and 507.
    p.maxch = (in.max_len < rd.tokens_cap ? in.max_len : rd.tokens_cap) / C + 2;
    p.classes = p.nseg == 1 && p.R > 1 && p.maxch > 4 && fills_gpu(p) && (long long)p.R * p.H <= 2048 ? 4 : 1;
    p.segs = reinterpret_cast<float *>(p.tiles + (size_t)p.ccap * d.G * 2 * C * d.N * 2);
    p.maps = p.segs + (size_t)rd.R * d.H * p.nseg * d.N * d.P;
    return d.P == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace rs
