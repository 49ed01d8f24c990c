// What the kernels of the ragged delta rule share: the chunk records, the
// launch parameters, a request's facts, and the scaling of fp16 operands.
#pragma once

#include <cuda_fp16.h>

#include "rs_common.cuh"
#include "rs_internal.h"

namespace rs {
namespace prefill {

constexpr int C = RS_CHUNK;
// Rows of the longest request that the recurrence serves.  256 cached requests of
// 32 heads of 128 (us): recurrence 166 (1 row), 247 (4), 362 (8), 471 (12), 597 (16),
// chunks 474 from 13 rows on; with a bf16 state 135, 232, 358, 475 (12), chunks 424.  4 requests
// of 8 heads: recurrence 8.4 (9 rows), 13 (16), chunks 20.
constexpr int kShort = 12;

// What chunk_cta leaves for the scans.  All tiles have rows of 64 fp16
// (128 bytes) with their 16-byte pieces in the order that shared-memory reads
// want: piece c of row r at c ^ (r & 7).
//
// Per chunk and key head: keys, then queries, D / 64 tiles of 64 rows each.
// Per chunk and value head:
struct Record {
    uint16_t t_hi[C * C], t_lo[C * C];  // T, row i scaled by 1 / (its power of two)
    uint16_t p_hi[C * C], p_lo[C * C];  // P without the queries' powers of two; nothing above the diagonal's 16 x 16 blocks
    float egk[C];  // e^(G_i) times key i's power of two
    float eg[C];   // e^(G_i)
    float su[C];   // T's and key i's powers of two: (T R)_i su_i = u_i times key i's power
    float sq[C];   // query i's power of two
    float ke[C];  // e^(G_C - G_i)
    float all;     // e^(G_C)
    float pad[31];
};
constexpr int kRecMats = 4 * C * C * 2;                   // bytes of the matrices, then
constexpr int kRecVecs = (int)sizeof(Record) - kRecMats;  // of the vectors
static_assert(sizeof(Record) == 34176, "records are copied in 16-byte pieces");
struct Vecs {  // the vectors of a Record
    float egk[C], eg[C], su[C], sq[C], ke[C], all, pad[31];
};
static_assert(sizeof(Vecs) == kRecVecs, "");

struct PrefillParams {
    int H, G, rep, prec;  // rep: value heads of a key head
    int R, cap, ccap, block, max_blocks, n_pool, max_len, B;
    float *hp;
    uint16_t *lp;
    int32_t *base, *h, *nd;
    uint32_t *status;
    rs_ragged rg;
    const uint16_t *q, *k, *v;
    const float *alpha, *beta;
    long long ld_q, ld_k, ld_v;
    const int32_t *rows, *start;
    void *pool;
    uint16_t *y;
    Record *rec;  // [ccap][H]
    unsigned char *tiles;  // [ccap][G] keys and queries of a chunk, fp16
    int nseg, seglen;      // segments of a request at most, chunks of a segment
    int classes, maxch;    // length classes of the scan's CTAs, chunks of the longest request
    float *segs, *maps;    // [R][H][nseg][N][P] segments' starting states and transition maps
};

// ---------------------------------------------------------------- fp16 operands
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

// The power of two that brings a row whose largest magnitude is m into
// [2^K, 2^(K+1)), and its inverse.  A bound that is no longer finite counts as 2^128,
// which no finite value reaches; a value that is not finite stays so at any scale.
__device__ __forceinline__ void row_scale(int K, float m, float &up, float &down) {
    const int e = (int)(__float_as_uint(m) >> 23) & 255;
    const int u = min(254 + K - e, 253);  // biased exponent; its inverse is 254 - u >= 1
    up = __uint_as_float((uint32_t)max(u, 1) << 23);
    down = __uint_as_float((uint32_t)(254 - max(u, 1)) << 23);
}
template <int K>
__device__ __forceinline__ void row_scale(float m, float &up, float &down) { row_scale(K, m, up, down); }

// Two values as hi + lo: hi their fp16 rounding, lo the rounding of the rest.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack_h2(x, y);
    const float2 h = unpack_h2(hi);
    lo = pack_h2(x - h.x, y - h.y);
}
// The same with hi cut instead of rounded, its difference taken by mixed-precision
// subtraction: fewer instructions, 22 bits as well.
__device__ __forceinline__ void split_cut(float x, float y, uint32_t &hi, uint32_t &lo) {
    float c, d;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
    asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; sub.f32.f16 %0, l, %3; sub.f32.f16 %1, h, %4;}"
        : "=f"(c), "=f"(d)
        : "r"(hi), "f"(x), "f"(y));
    lo = pack_h2(-c, -d);
}
// Byte offset of 16-byte piece c (8 channels) of row r in 64-row tiles of 64 channels.
__device__ __forceinline__ uint32_t piece(int r, int c) {
    return (uint32_t)((c >> 3) * (C * 128) + r * 128 + (((c ^ r) & 7) << 4));
}

// ---------------------------------------------------------------- requests
struct Request {
    int n, row0, ctx, chunk0, nch, srow, start;
    bool ok;
};

// A request's facts, checked; bits of what is wrong go to the status word.
__device__ __forceinline__ Request load_request(const PrefillParams &p, int r, bool report) {
    Request q = {};
    // two rounds of independent loads
    const int a = p.rg.cu_tokens[r], b = p.rg.cu_tokens[r + 1];
    const int c0 = p.rg.cu_chunks[r], c1 = p.rg.cu_chunks[r + 1];
    const int srow = p.rows ? p.rows[r] : r, start = p.start ? p.start[r] : -2;
    const bool in_cap = a >= 0 && b > a && b <= p.cap, in_rows = srow >= 0 && srow < p.B;
    q.n = b - a;
    if (q.n == 0) return q;
    q.ctx = in_cap ? p.rg.token_pos[a] : -1;
    const int pending = in_rows ? p.h[srow] | p.nd[srow] : 0;
    q.row0 = a, q.chunk0 = c0, q.nch = c1 - c0, q.srow = srow, q.start = start;
    unsigned bits = 0;
    if (!in_cap || q.n > p.max_len || q.ctx < 0 || q.ctx > (1 << 30) || c0 < 0 || c1 > p.ccap ||
        q.nch != (q.ctx + q.n + C - 1) / C - q.ctx / C)
        bits = RS_DEV_LENGTH;
    if (!in_rows || start < -2 || start >= p.n_pool)
        bits |= RS_DEV_SLOT;
    else if (start == -2 && pending != 0)
        bits |= RS_DEV_RECORDS;
    q.ok = bits == 0;
    if (bits && report) atomicOr(p.status, bits);
    return q;
}

// Pool slot of the state after the request's rows up to `end` (a position,
// context included); -1 if it is not to be kept.
__device__ __forceinline__ int block_slot(const PrefillParams &p, int r, int end, bool report) {
    if (!p.block || !p.pool || end % p.block) return -1;
    const int j = end / p.block - 1;
    const int slot = j < p.max_blocks ? p.rg.block_table[(size_t)r * p.max_blocks + j] : -1;
    if (slot >= 0 && slot < p.n_pool) return slot;
    if (slot != -1 && report) atomicOr(p.status, RS_DEV_SLOT);
    return -1;
}

// A scan's CTAs may start while the launch before it still runs (launch_after):
// they fetch their starting state first and wait here for what that launch writes.
__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next launch's CTAs start once all of this launch's have.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... KArgs, class... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), int grid, int block, int smem, cudaStream_t s, bool early, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block), cfg.dynamicSmemBytes = smem, cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Requests and heads alone make a chain for each place on the GPU, two an SM.
inline bool fills_gpu(const PrefillParams &p) { return (long long)p.R * p.H >= 304; }

// CTAs that start early are placed around what still runs, so two may share an SM
// while others stay empty: only where the chains fill the GPU anyway (192 chains of
// 64-wide heads, 100 to 900 rows: 92 us early, 84 after the launch before; 320 of
// 128-wide heads 119 and 124, 1,952 of 1 to 200 rows 145 and 151).
inline bool start_early(const PrefillParams &p) { return p.nseg == 1 && fills_gpu(p); }

// ---------------------------------------------------------------- segments
// A request's chunks form one chain per head.  Where requests and heads alone
// leave most of the GPU idle, the chain is cut into segments.  A segment's final
// state is linear in its starting state, S_out = M S_in + B (M acts on the key
// index), so the segments run twice:
//   first without outputs, from zero (giving B) and, with V = 0, from the
//   identity (giving M), all at once; the first one runs from the request's
//   starting state instead;
//   then S_(s+1) = M_s S_s + B_s in order (combine_kernel), a small product a step;
//   and again, with outputs, from those states.
// That is a little over twice the work on a chain shorter by the number of
// segments.
// Without segments the CTAs come in up to four passes over the requests, longest
// first: a CTA whose request is of another class leaves at once.  Started in the
// requests' own order, a long chain that comes last would run alone at the end.
__device__ __forceinline__ int length_class(const PrefillParams &p, int nch) {
    return nch > p.maxch >> 1 ? 0 : nch > p.maxch >> 2 ? 1 : nch > p.maxch >> 3 ? 2 : 3;
}
// The request of a CTA (already without its head and part), -1 if it has nothing to do; q: its unit.
__device__ __forceinline__ int cta_request(const PrefillParams &p, int cta, int units, int &q) {
    q = cta % units;
    const int cr = cta / units, r = cr % p.R;
    if (p.rg.cu_tokens[r + 1] - p.rg.cu_tokens[r] <= kShort) return -1;
    if (p.classes > 1 && length_class(p, p.rg.cu_chunks[r + 1] - p.rg.cu_chunks[r]) != cr / p.R) return -1;
    return r;
}

struct Unit {          // what one CTA of a scan runs
    int r, h, seg;
    bool map;          // from the identity, without V
    int c0, c1, nsegs;  // its chunks, and the request's segments
    bool ok;
};

// The unit of a CTA (CTAs count heads first); OUT: the pass with outputs.
template <bool OUT>
__device__ __forceinline__ Unit scan_unit(const PrefillParams &p, int cta, const Request &rq, int r, int q) {
    Unit u;
    u.r = r;
    u.h = cta % p.H;
    u.seg = OUT ? q : q >> 1;
    u.map = !OUT && (q & 1);
    u.nsegs = p.nseg > 1 ? (rq.nch + p.seglen - 1) / p.seglen : 1;
    u.c0 = u.seg * p.seglen;
    u.c1 = min(u.c0 + p.seglen, rq.nch);
    // the last segment's final state is the second pass's; the first needs no map
    u.ok = OUT ? u.seg < u.nsegs : u.seg < u.nsegs - 1 && !(u.map && u.seg == 0);
    return u;
}
template <bool OUT>
inline int scan_units(const PrefillParams &p) { return OUT ? p.nseg : 2 * (p.nseg - 1); }

__device__ __forceinline__ size_t seg_slab(const PrefillParams &p, const Unit &u, int seg, int n) {
    return (((size_t)u.r * p.H + u.h) * p.nseg + seg) * n;
}

// Where a unit's state starts: kind 0 zeros, 1 the identity, 2 fp32, 3 bf16.
struct StateSource {
    int kind;
    const float *f;
    const uint16_t *b;
};
template <bool OUT, int D>
__device__ __forceinline__ StateSource unit_start(const PrefillParams &p, const Request &rq, const Unit &u) {
    StateSource s = {0, nullptr, nullptr};
    if (u.map) {
        s.kind = 1;
    } else if (OUT ? u.nsegs > 1 : u.seg > 0) {
        if (OUT) s.kind = 2, s.f = p.segs + seg_slab(p, u, u.seg, D * D);
    } else if (rq.start != -1) {
        const bool cont = rq.start == -2;
        const size_t slab = ((size_t)(cont ? rq.srow : rq.start) * p.H + u.h) * D * D;
        if (p.prec == RS_PREC_SHARED_BF16)
            s.kind = 3, s.b = (cont ? p.lp : static_cast<const uint16_t *>(p.pool)) + slab;
        else
            s.kind = 2, s.f = (cont ? p.hp : static_cast<const float *>(p.pool)) + slab;
    }
    return s;
}

// The scan of 128-wide heads on the fifth-generation tensor cores (rs_prefill_tc.cu).
template <bool OUT>
cudaError_t scan_tc_launch(const PrefillParams &p, cudaStream_t s);

}  // namespace prefill
}  // namespace rs
