// Attention of few rows over a paged cache (one new token a request, or a few
// drafts), and the kernel that joins the parts of heads that several CTAs shared.
//
// For each row x of a request's group of heads on a key head, over its keys j:
//   s_j = c q.k_j,  m = max s_j,  y = sum 2^(s_j - m) v_j / sum 2^(s_j - m)
// with c = scale log2(e).  Every key and value is read once for 16 or 32 rows, so HBM
// bounds it: 2 D bytes of K and of V a key are 4 g D operations, a few tens a byte.
//
// A CTA an SM walks its share of the batch's blocks of 64 keys.  Copying
// warps bring them by TMA into a ring (128-byte swizzle), as far ahead as shared memory
// allows, and each piece's queries: the copies of the next head or request are under way while
// the last one's sums are joined.  Eight warps in groups take the blocks in turns, a warp 32
// keys of a block, each for itself: its own running maximum, sum of weights and sums of
// values in registers, so that no barrier falls between blocks.
// The matrix instructions (mma.sync, 16 rows x 8 x 16) are as many rows as a
// token has heads on a key head; tcgen05's 128 rows would be mostly empty.  The reference
// that weights are relative to follows the maximum only when it is 2^8 behind (2^1 with
// 8 bits), since a step of it costs a pass over the sums.
//
// From a bf16 cache the weights are rounded to bf16 for their product with the values,
// which the product's types ask for: 2^-8 of each weight at most, as y's own rounding,
// and on average less.  (What is left of them as a second bf16 term would leave y's own rounding alone, but four drafts of
// 64 requests take 99 us with it against 85, 256 tokens 318 against 313.)  From an 8-bit cache the codes become fp16, exactly, and so
// queries (scaled row by row by a power of two: bf16's 8 bits fit) and weights: relative to
// m' = max(s_j + e_j), with e_j the exponent of value j's scale, and times 2^14, so that
// the weight times 2^e_j uses fp16's whole range: what lies 2^-28 below the
// largest loses bits.  The sum of weights itself stays fp32 and unrounded in both.  With 8 bits it is of
// 2^(s_j - m' + 25), since e_j is -60 to 119: the largest of them is then 2^-94 to 2^86, and what is 2^-32 of
// the largest still counts.  (Of 2^(s_j - m') those a little below the largest vanished beside values of 2^119.)
// Where such sums are joined they are logarithms relative to their m', which may be far apart.  (A maximum of the scores
// alone, kept beside m', as their reference: four drafts of 64 requests 125 us against 109, 256 tokens 196 against 185.)
//
// Measured (32 query heads on 4 key heads of 128): 256 tokens behind 20 to 8,000 keys each, 2.1 GB of bf16 cache,
// 312 us, 6.8 TB/s, the copy peak; from an 8-bit cache 193 us, 5.6 TB/s, where the conversion and
// the products' own chain bound it (0.43 us a block of 64 keys against 0.37 at the copy's rate); four drafts of 64
// requests 85 us, 4.9 TB/s, on 8 bits 109.  One token behind 131,071 keys 54 us and four behind 50 to 900 each 10 us: there
// the launches, a start of dependent loads, and the joining of parts.
#include "rs_attn.cuh"

namespace rs {
namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kCopiers = 4;  // warps
constexpr int kThreads = (kWarps + kCopiers) * 32;
constexpr int kPass = 32;        // channels joined at a time
constexpr int kPitch = kPass + 8;  // floats between rows of the joining area: conflict-free pairs

template <int D_, bool E4M3_, int MT_>
struct Cfg {
    static constexpr int D = D_, MT = MT_, ROWS = 16 * MT;
    // A warp takes 32 keys of a block: with 16 its chain of products, maximum and exponentials is longer
    // for what it does (256 tokens on an 8-bit cache 243 us against 218, on a bf16 one 321 against 315).  With 32 rows two
    // warps take the same keys and half of the channels of their values each, since a warp's registers hold
    // the sums of 16 rows.  As many warps as a block needs are a group; groups take the blocks in turns.
    static constexpr int NT = 4;   // tiles of eight keys of a warp
    static constexpr int SLICES = kKeys / (8 * NT), PARTS = MT, GROUPS = kWarps / (SLICES * PARTS);
    static constexpr int N = D / 8 / PARTS;               // tiles of eight channels of a warp
    static constexpr bool E4M3 = E4M3_;
    static constexpr int ROWB = D * (E4M3 ? 1 : 2);           // bytes of a key
    static constexpr int HALVES = ROWB > 128 ? 2 : 1;         // tiles of 128-byte rows side by side
    static constexpr int TILE = kKeys * ROWB;
    // whole rounds of all groups of warps: a stage always meets the same group, which
    // then waits on its barriers in every round
    static constexpr int STAGES = 2 * TILE >= 32768 ? 4 : 12;  // 128 KiB and more
    static constexpr int COPIERS = kCopiers;              // copying warps, each every fourth block
    static constexpr int SCALES = STAGES * 2 * TILE;          // [STAGES][2][kKeys]
    static constexpr int JOIN = SCALES + (E4M3 ? STAGES * 2 * kKeys : 0);
    static constexpr int ML = JOIN + kWarps * 16 * kPitch * 4;  // [kWarps][ROWS] (maximum, sum)
    static constexpr int Q = ML + kWarps * ROWS * 8;            // [ROWS] queries of a piece
    static constexpr int QROW = 2 * D + 16;                     // their pitch: conflict-free
    static constexpr int BARS = Q + ROWS * QROW;
    static constexpr int BYTES = BARS + (2 * STAGES + 2) * 8 + 32 + 1024;  // and room to align
    static_assert(BYTES <= 227 * 1024 && STAGES % GROUPS == 0 && STAGES % COPIERS == 0, "");
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool E4M3>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (E4M3)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_h(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t two_halves(uint32_t codes16) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes16));
    return r;
}
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Byte of 16-byte piece c of key r in a tile as the copies leave it.
template <class C>
__device__ __forceinline__ uint32_t piece(int r, int c) {
    if constexpr (C::ROWB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * (kKeys * 128) + r * 128 + (((c ^ r) & 7) << 4);
}

// Where a lane finds the keys (and the values) of its warp's slice of 16 in a tile.  Pieces further
// along a row, and rows further down, are exclusive-ors and sums of constants away, see compute().
template <class C>
__device__ __forceinline__ uint32_t key_place(int slice) {
    const int lane = threadIdx.x & 31;
    return C::E4M3 ? piece<C>(slice + (lane >> 2), lane & 3) : piece<C>(slice + (lane & 7), lane >> 3);
}
template <class C>
__device__ __forceinline__ uint32_t value_place(int slice, int part) {
    const int lane = threadIdx.x & 31;
    if constexpr (!C::E4M3) return piece<C>(slice + (lane & 15), part * C::N + (lane >> 4));
    const int at = (lane >> 2) * (C::D / 8) + part * C::N;  // byte in the row
    return piece<C>(slice + 2 * (lane & 3), at >> 4) + (at & 15);
}

// A CTA's walk over its share: piece after piece.
struct Walk {
    Start at, end;
    int n, Hk;
    const int4 *list;
    int4 q, next;  // the request (index, first row, rows, context), and the one after it
    int keys, blocks, last;
    __device__ __forceinline__ void begin(const Params &p, const PlanView &v) {
        at = v.short_start[blockIdx.x], end = v.short_start[blockIdx.x + 1];
        n = v.head->n_short, list = v.shorts, Hk = p.Hk;
        if (at.idx < n) q = list[at.idx];
        if (at.idx + 1 < n) next = list[at.idx + 1];
    }
    __device__ __forceinline__ bool piece() {
        if (at.idx >= n || (at.idx == end.idx && at.head == end.head && at.part == end.part)) return false;
        keys = q.z + q.w;
        blocks = (keys + kKeys - 1) / kKeys;
        last = at.idx == end.idx && at.head == end.head ? end.part : blocks;
        return true;
    }
    __device__ __forceinline__ void step() {
        if (at.idx == end.idx && at.head == end.head) {  // the share ends within this head
            at = end;
            return;
        }
        at.part = 0;
        if (++at.head < Hk) return;
        at.head = 0, ++at.idx;
        q = next;
        if (at.idx + 1 < n) next = list[at.idx + 1];
    }
};

// ---------------------------------------------------------------- copies
template <class C>
__device__ __forceinline__ void produce(const Params &p, const PlanView &v, const CUtensorMap *km, const CUtensorMap *vm,
                                        uint32_t sm, uint64_t *full, uint64_t *empty, volatile uint32_t *abort) {
    const int lane = threadIdx.x & 31, role = (threadIdx.x >> 5) - kWarps;
    if (role >= C::COPIERS) return;
    volatile uint32_t *const begun = abort + 1 + role;  // blocks, for drain()
    // A block is one warp's: one that issues every copy of every block would take longer than the copies.  A lane
    // to a copy: keys or values, half of the channels, up to 64 keys; then (8 bits) scales of as many keys.
    const int rows = min(p.page, kKeys), boxes = kKeys / rows;
    const bool scales = C::E4M3 && lane >= 16 && lane < 16 + 2 * boxes, is_v = lane & 1;
    const bool tiles = lane < 2 * C::HALVES * boxes;
    const int half = scales ? 0 : (lane >> 1) % C::HALVES, box = scales ? (lane - 16) >> 1 : min((lane >> 1) / C::HALVES, boxes - 1);
    uint64_t *const q_full = empty + C::STAGES, *const q_empty = q_full + 1;
    const bool queries = role == C::COPIERS - 1;  // this warp brings the pieces' queries too, a row a lane
    unsigned q_parity = 0;
    Ring ring;
    ring.at = role;
    bool first_round = true, first_piece = true;
    int skip = role;  // blocks until this warp's next
    PageWindow pages;
    Walk w;
    w.begin(p, v);
    for (; w.piece(); w.step()) {
        if (queries) {
            if (!first_piece) {
                if (!wait_ready(q_empty, q_parity, abort, p.status)) return;
                q_parity ^= 1;
            }
            const int rows = w.q.z * p.g, token = lane / p.g;
            if (lane == 0) {
                abort[1 + kCopiers] += 1;
                mbar_arrive_expect_tx(q_full, rows * 2 * C::D);
            }
            __syncwarp();
            if (lane < rows)
                bulk_load(sm + C::Q + lane * C::QROW, p.q + (long long)(w.q.y + token) * p.ld_q + (w.at.head * p.g + lane - token * p.g) * C::D,
                          2 * C::D, q_full);
            first_piece = false;
        }
        const int entries = min((w.keys + p.page - 1) >> p.page_log, p.max_pages);
        int b = w.at.part + skip;
        for (; b < w.last; b += C::COPIERS) {
            const int key = b * kKeys + box * rows, row = key & (p.page - 1);
            pages.at(p, w.q.x, entries, (b * kKeys) >> p.page_log);
            const int page = pages.page(p, key >> p.page_log, (tiles || scales) && key < w.keys);
            if (!first_round && !wait_ready(empty + ring.at, ring.parity ^ 1, abort, p.status)) return;
            const unsigned there = __ballot_sync(~0u, scales && page >= 0);
            if (lane == 0) {
                *begun += 1;
                mbar_arrive_expect_tx(full + ring.at, 2 * C::TILE + __popc(there) * rows);
            }
            __syncwarp();
            if (tiles) {  // a coordinate past the cache fills in zeros
                const int slab = page >= 0 ? page * p.Hk + w.at.head : p.n_pages * p.Hk;
                const uint32_t to = sm + ring.at * 2 * C::TILE + half * (kKeys * 128) + box * rows * min(C::ROWB, 128);
                if (is_v)
                    tma_load_3d(to + C::TILE, vm, half * 64, row, slab, full + ring.at);
                else
                    tma_load_3d(to, km, half * 64, row, slab, full + ring.at);
            } else if (scales && page >= 0) {
                bulk_load(sm + C::SCALES + (ring.at * 2 + is_v) * kKeys + box * rows,
                          (is_v ? p.vs : p.ks) + (((size_t)page * p.Hk + w.at.head) << p.page_log) + row, rows, full + ring.at);
            }
#pragma unroll
            for (int i = 0; i < C::COPIERS; ++i) ring.step(C::STAGES);
            if (ring.at == role) first_round = false;
        }
        skip = b - w.last;
    }
}

// After giving up: wait (with a limit) for the copies still in flight.
template <class C>
__device__ __forceinline__ void drain(uint64_t *full, const volatile uint32_t *begun) {
    constexpr int PLACES = C::STAGES / C::COPIERS;  // a warp's
    for (int s = 0; s < C::STAGES; ++s) {
        const int n = (int)begun[s % C::COPIERS], first = s / C::COPIERS;
        if (n > first) mbar_wait(full + s, ((n - first + PLACES - 1) / PLACES - 1) & 1);
    }
    if (begun[kCopiers]) mbar_wait(full + 2 * C::STAGES, (begun[kCopiers] - 1) & 1);
}

// ---------------------------------------------------------------- arithmetic
template <class C>
struct Sums {
    float o[C::MT][C::N][4];  // 16 rows x (D or half of it), as the products leave them
    float m[C::MT][2], l[C::MT][2];
};
// 8 bits: exponents of values' scales are held less 16, so that m' of scores far from 0, where it can only be rounded (up),
// is a score itself for values up to 2^25: the products' weights then lose range, not their meaning.
constexpr float kBias = 127.f + 16.f;
constexpr float kUp = 9.f;  // while keys are gone over, l is of weights times 2^kUp, 2^25 without that 16

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 8 bits: a part's (m', logarithm of its sum of weights), the latter relative to another m'.  A part without
// keys has -inf for both; what is not a number stays one.
__device__ __forceinline__ float log_sum_at(float2 part, float m) { return part.x == -INFINITY ? part.y : part.y + (part.x - m); }

// The queries of a piece as operands; with 8 bits scaled to fp16, and c times what undoes it in cq.
// Rows that the piece does not have are zeros.
template <class C>
__device__ __forceinline__ void load_queries(const Params &p, int rows, uint32_t from, uint32_t (&q)[C::MT][C::D / 16][4],
                                             float (&cq)[C::MT][2]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
        if constexpr (!C::E4M3) {
#pragma unroll
            for (int k = 0; k < C::D / 16; ++k) ldmatrix4(q[mt][k], from + (mt * 16 + (lane & 15)) * C::QROW + (2 * k + (lane >> 4)) * 16);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int row = mt * 16 + hf * 8 + (lane >> 2);
            const bool in = row < rows;
            cq[mt][hf] = p.c;
            if constexpr (!C::E4M3) {
#pragma unroll
                for (int k = 0; k < C::D / 16; ++k) {
                    if (!in) q[mt][k][hf] = q[mt][k][2 + hf] = 0;
                }
            } else {
                // a lane's channels are those of its 16 bytes of codes: 16 t, and 64 + 16 t
                uint32_t x[C::D / 8];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < C::D / 64; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 u = lds128(from + row * C::QROW + (k * 64 + t * 16 + e * 8) * 2);
                        x[8 * k + 4 * e] = in ? u.x : 0, x[8 * k + 4 * e + 1] = in ? u.y : 0;
                        x[8 * k + 4 * e + 2] = in ? u.z : 0, x[8 * k + 4 * e + 3] = in ? u.w : 0;
                    }
#pragma unroll
                for (int i = 0; i < C::D / 8; ++i) top = __vmaxu2(top, x[i] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                // the power of two that brings the row's largest magnitude to [2^14, 2^15)
                const int up = min(max(254 + 14 - (int)(top >> 7), 1), 253);
                const float fu = __uint_as_float((uint32_t)up << 23);
                cq[mt][hf] = p.c * __uint_as_float((uint32_t)(254 - up) << 23);
#pragma unroll
                for (int s = 0; s < C::D / 16; ++s)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t u = x[2 * s + e];
                        q[mt][s][2 * e + hf] = pack_h(bf2f(u & 0xffffu) * fu, __uint_as_float(u & 0xffff0000u) * fu);
                    }
            }
        }
    }
}

// One warp's 8 NT keys of a staged block.  key0: position of the first; limit: the
// last key that each of the lane's rows sees.
template <class C>
__device__ __forceinline__ void compute(Sums<C> &a, const uint32_t (&q)[C::MT][C::D / 16][4], const float (&cq)[C::MT][2],
                                        uint32_t k_at, uint32_t v_at, uint32_t v_tile, uint32_t scales, int slice, int key0, int keys,
                                        int seen, const int (&limit)[C::MT][2], int part) {
    constexpr int MT = C::MT, D = C::D, N = C::N, NT = C::NT;
    const int lane = threadIdx.x & 31, t = lane & 3;
    float s[MT][NT][4] = {};
    if constexpr (!C::E4M3) {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            uint32_t b[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ldmatrix4(b[nt], (k_at ^ (kk & 1) << 6) + (kk >> 1) * (kKeys * 128) + nt * 1024);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma<false>(s[mt][nt], q[mt][2 * kk], b[nt][0], b[nt][1]);
                    mma<false>(s[mt][nt], q[mt][2 * kk + 1], b[nt][2], b[nt][3]);
                }
        }
    } else {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            uint4 b[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) b[nt] = lds128((k_at ^ h << 6) + nt * 8 * C::ROWB);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint32_t w = k == 0 ? b[nt].x : k == 1 ? b[nt].y : k == 2 ? b[nt].z : b[nt].w;
                    const uint32_t b0 = two_halves(w), b1 = two_halves(w >> 16);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma<true>(s[mt][nt], q[mt][4 * h + k], b0, b1);
                }
        }
    }
    // scores in units of log2; with 8 bits ev is the power of two of each key's values
    float ev[NT][2];
    if constexpr (C::E4M3) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const uint32_t kb = lds_u16(scales + slice + nt * 8 + 2 * t), vb = lds_u16(scales + kKeys + slice + nt * 8 + 2 * t);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float up = __uint_as_float(e ? (kb & 0xff00u) << 15 : (kb & 0xffu) << 23);
                ev[nt][e] = (float)(e ? vb >> 8 : vb & 0xffu) - kBias;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    s[mt][nt][e] *= up * cq[mt][0];
                    s[mt][nt][2 + e] *= up * cq[mt][1];
                }
            }
        }
    } else {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][nt][e] *= cq[mt][e >> 1];
    }
    const bool masked = key0 + 8 * NT - 1 > seen;  // some row does not see all of them
    if (masked) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key0 + nt * 8 + 2 * t + (e & 1) > limit[mt][e >> 1]) s[mt][nt][e] = -INFINITY;
        // What lies behind the last key is not part of the cache: as zeros it meets its zero weights
        if (!C::E4M3 && key0 + 8 * NT > keys) {
            for (int i = lane; i < (8 * NT - max(keys - key0, 0)) * N; i += 32) {
                const int r = slice + 8 * NT - 1 - i / N, c = part * N + i % N;
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(v_tile + piece<C>(r, c)), "r"(0) : "memory");
            }
            __syncwarp();
        }
    }
    // the largest score so far; the reference follows it only when far behind
    constexpr float kBehind = C::E4M3 ? 1.f : 8.f;
    bool behind = false;
    float top[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float x = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                x = C::E4M3 ? fmaxf(x, fmaxf(__fadd_ru(s[mt][nt][2 * hf], ev[nt][0]), __fadd_ru(s[mt][nt][2 * hf + 1], ev[nt][1])))
                            : fmaxf(x, fmaxf(s[mt][nt][2 * hf], s[mt][nt][2 * hf + 1]));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 1));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 2));
            top[mt][hf] = x;
            behind = behind || x - a.m[mt][hf] > kBehind;
        }
    if (__any_sync(~0u, behind)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float m = fmaxf(a.m[mt][hf], top[mt][hf]);
                const float f = m == -INFINITY ? 1.f : ex2(a.m[mt][hf] - m);
                if constexpr (C::E4M3) {  // m' may move by more than one factor's range
                    const float root = m == -INFINITY ? 1.f : ex2(0.5f * (a.m[mt][hf] - m));
                    a.l[mt][hf] = a.l[mt][hf] * root * root;
                } else {
                    a.l[mt][hf] *= f;
                }
                a.m[mt][hf] = m;
#pragma unroll
                for (int n = 0; n < N; ++n) a.o[mt][n][2 * hf] *= f, a.o[mt][n][2 * hf + 1] *= f;
            }
    }
    uint32_t w[NT / 2][MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x[NT][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            // a row that has seen no key yet has no weights
            const float m = a.m[mt][hf] == -INFINITY ? 0.f : a.m[mt][hf];
            if constexpr (!C::E4M3) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 2 * hf; e < 2 * hf + 2; ++e) {
                        x[nt][e] = ex2(s[mt][nt][e] - m);
                        a.l[mt][hf] += x[nt][e];
                    }
            } else {
                f2 sum = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const f2 below = f2_add(f2_pack(s[mt][nt][2 * hf], s[mt][nt][2 * hf + 1]), f2_pack(-m, -m));
                    float lo, hi;
                    f2_unpack(f2_add(below, f2_pack(kUp, kUp)), lo, hi);
                    sum = f2_add(sum, f2_pack(ex2(lo), ex2(hi)));
                    // at most 2^15: the reference may be 2^1 behind
                    f2_unpack(f2_add(below, f2_pack(ev[nt][0] + 14.f, ev[nt][1] + 14.f)), lo, hi);
                    x[nt][2 * hf] = ex2(lo), x[nt][2 * hf + 1] = ex2(hi);
                }
                float lo, hi;
                f2_unpack(sum, lo, hi);
                a.l[mt][hf] += lo + hi;
            }
        }
#pragma unroll
        for (int kk = 0; kk < NT / 2; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // rows g and g + 8 of the first eight keys, then of the others
                const float lo = x[2 * kk + (i >> 1)][2 * (i & 1)], hi = x[2 * kk + (i >> 1)][2 * (i & 1) + 1];
                w[kk][mt][i] = C::E4M3 ? pack_h(lo, hi) : pack_bf(lo, hi);
            }
    }
#pragma unroll
    for (int kk = 0; kk < NT / 2; ++kk)
    if constexpr (!C::E4M3) {
#pragma unroll
        for (int n = 0; n < N / 2; ++n) {
            uint32_t b[4];
            ldmatrix4_trans(b, (v_at ^ (n & 3) << 5) + (n >> 2) * (kKeys * 128) + kk * 2048);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                mma<false>(a.o[mt][2 * n], w[kk][mt], b[0], b[1]);
                mma<false>(a.o[mt][2 * n + 1], w[kk][mt], b[2], b[3]);
            }
        }
    } else {
        // a lane's N channels from four keys, of the D / 8 that begin at (D / 8) g: bytes of two keys side by side are one operand
        uint32_t r[4][N / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t from = (D == 128 ? (v_at + (i & 1) * 128) ^ (i & 1) << 4 : v_at + (i & 1) * 64) + ((i >> 1) + 2 * kk) * 8 * C::ROWB;
            if constexpr (N == 16) {
                const uint4 u = lds128(from);
                r[i][0] = u.x, r[i][1] = u.y, r[i][2] = u.z, r[i][3] = u.w;
            } else if constexpr (N == 8) {
                const uint2 u = lds64(from);
                r[i][0] = u.x, r[i][1] = u.y;
            } else {
                r[i][0] = lds32(from);
            }
            if (masked && key0 + 16 * kk + 2 * t + (i & 1) + 8 * (i >> 1) >= keys)
#pragma unroll
                for (int e = 0; e < N / 4; ++e) r[i][e] = 0;
        }
#pragma unroll
        for (int e = 0; e < N / 4; ++e)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = __byte_perm(r[0][e], r[1][e], h ? 0x7362 : 0x5140);
                const uint32_t y = __byte_perm(r[2][e], r[3][e], h ? 0x7362 : 0x5140);
                const uint32_t x0 = two_halves(x), x1 = two_halves(x >> 16), y0 = two_halves(y), y1 = two_halves(y >> 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma<true>(a.o[mt][4 * e + 2 * h], w[kk][mt], x0, y0);
                    mma<true>(a.o[mt][4 * e + 2 * h + 1], w[kk][mt], x1, y1);
                }
            }
    }
}

// The eight warps' sums of a piece, joined; whole heads go to y, parts to the workspace.
template <class C>
__device__ __forceinline__ void finish(const Params &p, Sums<C> &a, const int4 &rq, int head, bool whole, int slot, int place,
                                       unsigned char *smem) {
    constexpr int MT = C::MT, D = C::D, SUMS = kWarps / C::PARTS;  // warps whose sums of a channel are joined
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float2 *const ml = reinterpret_cast<float2 *>(smem + C::ML);
    float *const area = reinterpret_cast<float *>(smem + C::JOIN);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float l = a.l[mt][hf];
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            if constexpr (C::E4M3) l = lg2(l) - kUp;
            // two warps of the same keys have the same
            if (t == 0 && place < SUMS) ml[place * C::ROWS + mt * 16 + hf * 8 + g] = make_float2(a.m[mt][hf], l);
        }
    consumers_sync();
    const int rows = rq.z * p.g;
    float *const to_parts = p.short_parts + (size_t)(2 * blockIdx.x + slot) * part_floats(C::ROWS, D);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        // weights of this warp's two rows
        float f[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < SUMS; ++w) m = fmaxf(m, ml[w * C::ROWS + mt * 16 + hf * 8 + g].x);
            f[hf] = a.m[mt][hf] == -INFINITY ? 0.f : ex2(a.m[mt][hf] - m);
            if (C::E4M3) f[hf] *= 4.f;  // 2^16 of the values' exponents, 2^-14 of the weights
        }
        // a thread's row and pair of channels of what is joined
        const int row = threadIdx.x >> 4, col = (threadIdx.x & 15) * 2, x = mt * 16 + row;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < SUMS; ++w) m = fmaxf(m, ml[w * C::ROWS + x].x);
        float most = -INFINITY;  // 8 bits: the largest logarithm, which l is relative to
        if constexpr (C::E4M3) {
#pragma unroll
            for (int w = 0; w < SUMS; ++w) most = fmaxf(most, log_sum_at(ml[w * C::ROWS + x], m));
            if (most == -INFINITY) most = 0.f;  // no weights: a sum of 0, not of what -inf less -inf is
        }
#pragma unroll
        for (int w = 0; w < SUMS; ++w) {
            const float2 v = ml[w * C::ROWS + x];
            // a sum that is not a number stays one
            if constexpr (C::E4M3)
                l += ex2(log_sum_at(v, m) - most);
            else
                l += v.x == -INFINITY ? v.y : v.y * ex2(v.x - m);
        }
        const float inv = 1.f / l, back = C::E4M3 ? ex2(-most) : 1.f;
        if constexpr (C::E4M3) l = lg2(l) + most;
        const int token = x / p.g, in_group = x - token * p.g;
        uint16_t *const y = p.y + ((long long)(rq.y + token) * p.Hq + head * p.g + in_group) * D;
        if (!whole && col == 0 && x < rows) reinterpret_cast<float2 *>(to_parts + (size_t)C::ROWS * D)[x] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < C::N / 4; ++c) {  // 32 channels of each part of the channels at a time
            float *const to = area + (place * 16 + g) * kPitch;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        // 8 bits: sums n of a lane are channels (D / 8) (2 t + k) + part N + n
                        const float2 v = C::E4M3 ? make_float2(a.o[mt][4 * c + 2 * i][2 * hf + k] * f[hf], a.o[mt][4 * c + 2 * i + 1][2 * hf + k] * f[hf])
                                                 : make_float2(a.o[mt][4 * c + 2 * i + k][2 * hf] * f[hf], a.o[mt][4 * c + 2 * i + k][2 * hf + 1] * f[hf]);
                        const int at = C::E4M3 ? (2 * t + k) * 4 + 2 * i : (2 * i + k) * 8 + 2 * t;
                        *reinterpret_cast<float2 *>(to + hf * 8 * kPitch + at) = v;
                    }
            consumers_sync();
#pragma unroll
            for (int part = 0; part < C::PARTS; ++part) {
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < SUMS; ++w) {
                    const float2 v = *reinterpret_cast<const float2 *>(area + ((part * SUMS + w) * 16 + row) * kPitch + col);
                    sum.x += v.x, sum.y += v.y;
                }
                const int d = C::E4M3 ? (D / 8) * (col >> 2) + part * C::N + 4 * c + (col & 3) : part * (D / C::PARTS) + c * kPass + col;
                if (x < rows) {
                    if (whole)
                        *reinterpret_cast<uint32_t *>(y + d) = pack_bf(sum.x * inv * back, sum.y * inv * back);
                    else
                        *reinterpret_cast<float2 *>(to_parts + (size_t)x * D + d) = sum;
                }
            }
            consumers_sync();
        }
    }
}

template <class C>
__device__ __forceinline__ void consume(const Params &p, const PlanView &v, unsigned char *smem, uint64_t *full, uint64_t *empty,
                                        volatile uint32_t *abort) {
    constexpr int MT = C::MT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / (C::SLICES * C::PARTS), part = warp / C::SLICES % C::PARTS, slice = warp % C::SLICES * (8 * C::NT);
    const int place = part * (kWarps / C::PARTS) + group * C::SLICES + warp % C::SLICES;  // among the sums to be joined
    const uint32_t sm = smem_u32(smem);
    const uint32_t k_at = sm + key_place<C>(slice), v_at = sm + C::TILE + value_place<C>(slice, part);
    Ring ring;
    ring.at = group;
    bool ok = true;
    Walk w;
    w.begin(p, v);
    int turn = 0;  // the group that takes the next block
    unsigned q_parity = 0;
    for (; w.piece(); w.step()) {
        uint32_t q[MT][C::D / 16][4];
        float cq[MT][2];
        ok = wait_ready(empty + C::STAGES, q_parity, abort, p.status) && ok;
        q_parity ^= 1;
        if (ok) load_queries<C>(p, w.q.z * p.g, sm + C::Q, q, cq);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + C::STAGES + 1);
        int limit[MT][2];
        const int rows = w.q.z * p.g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) limit[mt][hf] = w.q.w + min(mt * 16 + hf * 8 + (lane >> 2), rows - 1) / p.g;
        Sums<C> a;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) a.m[mt][hf] = -INFINITY, a.l[mt][hf] = 0.f;
#pragma unroll
            for (int n = 0; n < C::N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[mt][n][e] = 0.f;
        }
        for (int b = w.at.part; b < w.last; ++b, turn = (turn + 1) % C::GROUPS) {
            if (turn != group || !ok) continue;
            ok = wait_ready(full + ring.at, ring.parity, abort, p.status);
            const int key0 = b * kKeys + slice;
            if (ok && key0 < w.keys) {
                const uint32_t stage = ring.at * 2 * C::TILE;
                compute<C>(a, q, cq, k_at + stage, v_at + stage, sm + stage + C::TILE, sm + C::SCALES + ring.at * 2 * kKeys, slice, key0, w.keys, w.q.w, limit, part);
                if (!C::E4M3 && key0 + 8 * C::NT > w.keys) fence_proxy_async_smem();  // zeros written before the next copy
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + ring.at);
#pragma unroll
            for (int i = 0; i < C::GROUPS; ++i) ring.step(C::STAGES);
        }
        if (named_sync_or(2, kWarps * 32, !ok)) return;
        finish<C>(p, a, w.q, w.at.head, w.at.part == 0 && w.last == w.blocks, w.at.part > 0 ? 0 : 1, place, smem);
    }
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
short_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm) {
    extern __shared__ unsigned char raw[];
    let_next_launch();
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BARS), *empty = full + C::STAGES;
    uint64_t *q_full = empty + C::STAGES, *q_empty = q_full + 1;
    uint32_t *abort = reinterpret_cast<uint32_t *>(q_empty + 1);  // and what was begun: blocks by warp, queries
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    const bool mine = plan_fits(*v.head, p);
    if (threadIdx.x == 0) {
        if (!mine && blockIdx.x == 0) atomicOr(p.status, RS_DEV_LENGTH);
        for (int i = 0; i < C::STAGES; ++i) mbar_init(full + i, 1), mbar_init(empty + i, kWarps / C::GROUPS);
        mbar_init(q_full, 1), mbar_init(q_empty, kWarps);
        for (int i = 0; i < 2 + kCopiers; ++i) abort[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (mine) {
        // registers of the launch's 168 a thread: the copying warps leave most of theirs to the others
        if (threadIdx.x >= kWarps * 32) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
            produce<C>(p, v, &km, &vm, smem_u32(smem), full, empty, abort);
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
            consume<C>(p, v, smem, full, empty, abort);
        }
    }
    // Every block that was copied has been waited for, but for a wait that gave up
    if (__syncthreads_or(*reinterpret_cast<volatile uint32_t *>(abort)) && threadIdx.x == 0)
        drain<C>(full, abort + 1);
    if (blockIdx.x == 0) wait_for_launch();  // this launch does not end before the one that it overlaps
}

// ---------------------------------------------------------------- parts of a head
constexpr int kJoinWarps = 8;
constexpr int kShortBlocks = 2, kLongBlocks = 16;  // CTAs to a head's 32 rows, or an item's 256

// Rows x0, x0 + dx .. (NR of them, those with y) of a head that CTA c - 1's share ends with and the
// shares c, c + 1 .. begin with: n parts in the order of its keys, stride floats from CTA to CTA.  A warp's
// work, D / 32 channels a lane, the sums of U parts in flight, the first of them with the maxima.
// LOG: with logarithms of the sums of weights (the short form's with 8 bits).
template <int D, int NR, int U, bool LOG>
__device__ __forceinline__ void join_rows(const float *parts, size_t stride, int c, int n, int rows, int x0, int dx, uint16_t *const (&y)[NR]) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    auto part = [&](int k) { return parts + (size_t)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c + k - 1)) * stride; };
    float o[NR][U][V];
    auto load = [&](int k) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < V; ++i) o[r][u][i] = 0.f;
                if (k + u < n && y[r]) {
                    const float *at = part(k + u) + (size_t)(x0 + r * dx) * D + lane * V;
                    if constexpr (V == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(at);
                        o[r][u][0] = v.x, o[r][u][1] = v.y, o[r][u][2] = v.z, o[r][u][3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2 *>(at);
                        o[r][u][0] = v.x, o[r][u][1] = v.y;
                    }
                }
            }
    };
    auto max_sum = [&](int k, int r) {
        return k < n && y[r] ? reinterpret_cast<const float2 *>(part(k) + (size_t)rows * D)[x0 + r * dx] : make_float2(-INFINITY, LOG ? -INFINITY : 0.f);
    };
    // most: the logarithm that l is relative to
    auto put = [&](float (&sum)[V], float l, float most, uint16_t *to) {
        const float inv = 1.f / l, back = LOG ? ex2(-most) : 1.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] = sum[i] * inv * back;
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(to + lane * 4) = make_uint2(pack_bf(sum[0], sum[1]), pack_bf(sum[2], sum[3]));
        else
            *reinterpret_cast<uint32_t *>(to + lane * 2) = pack_bf(sum[0], sum[1]);
    };
    if (n <= U) {  // most heads: every lane reads all maxima
        float2 ml[NR][U];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) ml[r][u] = max_sum(u, r);
        load(0);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float m = -INFINITY, most = -INFINITY, l = 0.f, sum[V] = {};
#pragma unroll
            for (int u = 0; u < U; ++u) m = fmaxf(m, ml[r][u].x);
            if constexpr (LOG) {
#pragma unroll
                for (int u = 0; u < U; ++u) most = fmaxf(most, log_sum_at(ml[r][u], m));
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float f = ml[r][u].x == -INFINITY ? 1.f : ex2(ml[r][u].x - m);
                if constexpr (LOG)
                    l += ex2(log_sum_at(ml[r][u], m) - most);
                else
                    l = fmaf(ml[r][u].y, f, l);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] = fmaf(f, o[r][u][i], sum[i]);
            }
            if (y[r]) put(sum, l, most, y[r]);
        }
        return;
    }
    float2 ml[NR];
    float m[NR], most[NR], l[NR], sum[NR][V];
#pragma unroll
    for (int r = 0; r < NR; ++r) ml[r] = max_sum(lane, r);
    load(0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = ml[r].x, l[r] = 0.f;
        for (int k = 32 + lane; k < n; k += 32) m[r] = fmaxf(m[r], max_sum(k, r).x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m[r] = fmaxf(m[r], __shfl_xor_sync(~0u, m[r], d));
        most[r] = -INFINITY;
        if constexpr (LOG) {
            for (int k = lane; k < n; k += 32) most[r] = fmaxf(most[r], log_sum_at(k < 32 ? ml[r] : max_sum(k, r), m[r]));
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) most[r] = fmaxf(most[r], __shfl_xor_sync(~0u, most[r], d));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) sum[r][i] = 0.f;
    }
    for (int k0 = 0; k0 < n; k0 += 32) {
        float f[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            if (k0) ml[r] = max_sum(k0 + lane, r);
            // a part without keys that the row sees has sums of zero
            f[r] = k0 + lane >= n ? 0.f : ml[r].x == -INFINITY ? 1.f : ex2(ml[r].x - m[r]);
            if constexpr (LOG)
                l[r] += k0 + lane >= n ? 0.f : ex2(log_sum_at(ml[r], m[r]) - most[r]);
            else
                l[r] += ml[r].y * f[r];
        }
        for (int k = k0; k < min(k0 + 32, n); k += U) {
            if (k) load(k);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float fu = __shfl_sync(~0u, f[r], (k + u) & 31);
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[r][i] = fmaf(fu, o[r][u][i], sum[r][i]);
                }
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l[r] += __shfl_xor_sync(~0u, l[r], d);
        if (y[r]) put(sum[r], l[r], most[r], y[r]);
    }
}

// A CTA to a boundary between two shares, and to some of its head's rows.  Latency bounds it: two looks
// into the plan, beside the launch before, then the maxima and the first sums.  151 items of 256 rows, two parts each, take 11 us
// on a cold L2; four parts of one row in flight, two of each of a long form's two rows (64 registers)
// against 16 of one row (124): 16 prompts 417 against 437 us.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ Params p) {
    const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, shorts = p.short_rows ? kShortBlocks : 0;
    const bool lng = blockIdx.y >= shorts;
    if (blockIdx.x == 0 && blockIdx.y == 0) wait_for_launch();  // this launch does not end before the one that it overlaps
    // the plan was there before the launch that this one waits for
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    if (!plan_fits(*v.head, p)) return;  // the lists lie where this call's R says: a smaller plan ends before them
    const Join j = (lng ? v.long_join : v.short_join)[c];
    if (j.n == 0) return;
    const int tile_toks = tile_tokens(p.g);
    // row `in` of query tile t
    auto row = [&](int t, int in) -> uint16_t * {
        const int i = in / p.g, token = t * tile_toks + i;
        const bool live = token < j.tokens && (!lng || i < tile_toks);
        return live ? p.y + ((long long)(j.row + token) * p.Hq + j.head * p.g + in - i * p.g) * D : nullptr;
    };
    wait_for_launch();
    if (lng) {
        for (int x = (blockIdx.y - shorts) * kJoinWarps + warp; x < kTileRows; x += kLongBlocks * kJoinWarps) {
            uint16_t *const y[2] = {row(0, x), row(1, x)};
            if (y[0]) join_rows<D, 2, 2, false>(p.long_parts, part_floats(2 * kTileRows, D), c, j.n, 2 * kTileRows, x, kTileRows, y);
        }
    } else {
        for (int x = blockIdx.y * kJoinWarps + warp; x < p.short_rows; x += kShortBlocks * kJoinWarps) {
            uint16_t *const y[1] = {row(0, x)};
            if (y[0]) join_rows<D, 1, 4, E4M3>(p.short_parts, part_floats(p.short_rows, D), c, j.n, p.short_rows, x, 0, y);
        }
    }
}

template <class C>
cudaError_t launch_cfg(const Params &p, const CUtensorMap &k, const CUtensorMap &v, bool early, cudaStream_t s) {
    static SmemGrants grants;
    const cudaError_t e = grant_smem(reinterpret_cast<const void *>(&short_kernel<C>), C::BYTES, grants);
    if (e != cudaSuccess) return e;
    return launch(short_kernel<C>, p.ctas, kThreads, C::BYTES, s, early, p, k, v);
}

template <int D, bool E4M3>
cudaError_t launch_rows(const Params &p, const CUtensorMap &k, const CUtensorMap &v, bool early, cudaStream_t s) {
    return p.short_rows == 16 ? launch_cfg<Cfg<D, E4M3, 1>>(p, k, v, early, s) : launch_cfg<Cfg<D, E4M3, 2>>(p, k, v, early, s);
}

}  // namespace

cudaError_t short_launch(const Params &p, int D, bool e4m3, const CUtensorMap &k, const CUtensorMap &v, bool early,
                         cudaStream_t s) {
    if (D == 64) return e4m3 ? launch_rows<64, true>(p, k, v, early, s) : launch_rows<64, false>(p, k, v, early, s);
    return e4m3 ? launch_rows<128, true>(p, k, v, early, s) : launch_rows<128, false>(p, k, v, early, s);
}

cudaError_t join_launch(const Params &p, int D, bool e4m3, bool any_long, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.ctas - 1, (p.short_rows ? kShortBlocks : 0) + (any_long ? kLongBlocks : 0)), cfg.blockDim = dim3(kJoinWarps * 32), cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    if (D == 64) return cudaLaunchKernelEx(&cfg, e4m3 ? join_kernel<64, true> : join_kernel<64, false>, p);
    return cudaLaunchKernelEx(&cfg, e4m3 ? join_kernel<128, true> : join_kernel<128, false>, p);
}

}  // namespace attn
}  // namespace rs
