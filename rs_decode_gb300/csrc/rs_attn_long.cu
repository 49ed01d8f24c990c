// Attention of many rows over a paged cache on the fifth-generation tensor
// cores: prompts, and turns behind a cached context.
//
// The rows of a product are tokens x the query heads of one key head, token after
// token, so that a tile of 128 rows reads each key and value once for all heads of the
// group, and a causal edge is 128 / g tokens wide.  A CTA holds two such tiles:
//   S_i = Q_i K_j^T                128 x 128, fp32 in TMEM     (i = 0, 1: the tile)
//   P_i = 2^(c (S_i - m))          bf16, in S's place, by a thread a row
//   O_i (+)= P_i V_j               128 x D, fp32 in TMEM
// The tensor cores work on one tile while the threads work on the other: the order of
// products is P_0 V, Q_0 K, P_1 V, Q_1 K.  A step of a tile is 8 D x 128 x 128 / 2 operations
// to 128 x 128 exponentials, so at D = 128 the products bound it as long as a tile's
// register work hides behind the other tile's two products.
//
// The weights are relative to a reference that follows a row's maximum only when it is
// 2^8 behind: then the row's O is read, scaled and written back before the next product
// (otherwise O never leaves TMEM before the end).  Weights are rounded to bf16, which the product with bf16 values
// asks for: 2^-8 of each at most, no more than y's own rounding and on average less.  Their
// sum is that of the unrounded weights, fp32.
//
// Warps: 0-3 and 4-7 a thread a row of either tile; 8 issues the products; 9 and 10 the copies
// (TMA, 128-byte swizzle, keys and values by turns in one ring); 12-15 take O out at the end of a piece,
// while the next one's first products and weights are under way.  From an 8-bit cache the codes are
// copied, and warps 12-15 turn them into bf16 tiles, code times power of two, exactly.
// A piece of a single query tile (few tokens) takes its key tiles by turns as tile 0 and tile 1,
// with sums and references of their own, which its end puts together.
//
// TMEM columns: S_0 [0, 128), S_1 [128, 256), O_0 [256, 256 + D), O_1 after it.
//
// Measured (D = 128): a prompt of 32,768 tokens, 16 query heads on 2 key heads, 2.74 to 2.82 ms, 1,560 to 1,600 TFLOP/s, 0.80 to
// 0.82 of the measured product rate; 16 prompts of 27,711 tokens in all, 32 on 4 heads, 434 to 455 us, 1,170 to 1,230 TFLOP/s
// (both go with the card's power; about 4 us of each item of 32 tokens and a key head are its start and end).  A key tile
// of two query tiles takes 2,900 clocks: the products 2,600 of them (34 clocks for each 64 columns, 50 where both operands are in shared memory), the rest the
// product warp's waits and commits.  A row's register work is 1,500 clocks a tile.  Where one query tile is all, 1.7 us a key
// tile of 64 KiB from HBM (1.4 at the copy's rate); from an 8-bit cache 2.0, which the conversion takes.
#include "rs_attn.cuh"

namespace rs {
namespace attn {
namespace {

constexpr int kThreads = 512;

template <int D_, bool E4M3_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr bool E4M3 = E4M3_;
    static constexpr int HALF = 128 * 128;                 // 128 rows of 128 bytes
    static constexpr int TILE = (D / 64) * HALF;           // 128 rows of Q, K or V
    static constexpr int QS = E4M3 ? 2 : 3;                // places for query tiles
    static constexpr int STAGES = D == 64 ? 8 : E4M3 ? 3 : 4;
    static constexpr int RAWS = E4M3 ? 4 : 0;              // tiles of codes
    static constexpr int RAW = 128 * D;
    static constexpr int Q = 0;
    static constexpr int RING = QS * TILE;
    static constexpr int CODES = RING + STAGES * TILE;
    static constexpr int TILES = CODES + RAWS * RAW;       // bytes of all tiles, from a multiple of 1024 on
    static constexpr int SMALL = 3 * 1024;                 // what lies before them
    static constexpr int BYTES = SMALL + TILES;
    static_assert(BYTES <= 227 * 1024, "");
    // Registers a thread by role, out of the launch's 128 each
    static constexpr int ROW_REGS = 176, ISSUE_REGS = 56, HELP_REGS = 104;
    static_assert(256 * ROW_REGS + 128 * ISSUE_REGS + 128 * HELP_REGS <= kThreads * 128, "");
};

constexpr int kMaxStages = 8, kMaxRaws = 4, kMaxQs = 3;
struct Shared {
    float2 ml[2][kTileRows];                              // a piece's largest scores (in log2) and sums of weights
    uint8_t scales[kMaxRaws][kTileKeys];
    uint64_t full[kMaxStages], empty[kMaxStages];         // tiles of keys and values
    uint64_t raw_full[kMaxRaws], raw_empty[kMaxRaws];     // tiles of codes
    uint64_t q_full[kMaxQs], q_empty[kMaxQs];
    uint64_t s_full[2], p_ready[2], pv_done[2], o_full[2], o_free[2], end;
    uint32_t tmem, abort, ended, begun[2], begun_q[kMaxQs];  // ended: no product in flight; begun: tiles of keys, of values, of codes or not
};
static_assert(sizeof(Shared) <= 3 * 1024, "");

// ---------------------------------------------------------------- tensor cores
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Tiles are 128-byte-swizzled: rows of 128 bytes, groups of 8 rows 1024 bytes apart; LBO: from
// one half of 64 columns to the next, where a tile is read MN-major.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
// D[tmem] (+)= A[smem] B[smem], and A[tmem] below, by the lane of a converged warp that lead is set in.  The
// operands are the same in all lanes and stay in uniform registers: in a branch that one lane takes,
// moving them there took 45 clocks a product, and a tile's 16 of them longer than the products.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 ad, bd;\n\tmov.b64 ad, {%1, %3};\n\tmov.b64 bd, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 bd;\n\tmov.b64 bd, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
// A value that is the same in all lanes, as a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(~0u, x); }

#define RS_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define RS_U8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
#define RS_32 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}"
// 32 columns of the warp's 32 lanes; complete after ld_done()
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " RS_32 ", [%32];"
                 : RS_R8(v, 0), RS_R8(v, 8), RS_R8(v, 16), RS_R8(v, 24)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ld_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st32(uint32_t addr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " RS_32 ";" ::RS_U8(v, 0), RS_U8(v, 8), RS_U8(v, 16), RS_U8(v, 24),
                 "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#undef RS_R8
#undef RS_U8
#undef RS_32

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---------------------------------------------------------------- a CTA's walk over its share
struct Walk {
    Start at, end;
    int n, Hk, tokens;  // tokens of a query tile
    const int4 *list;
    int4 q, next;
    int items, t0, tn;      // the request's items; the piece's first token and tokens
    int keys;               // of the whole request
    int tiles, last;        // key tiles that the item sees, the piece's end among them
    int need0;              // key tiles that the first query tile sees
    bool one;               // a single query tile
    __device__ __forceinline__ void begin(const Params &p, const PlanView &v) {
        at = v.long_start[blockIdx.x], end = v.long_start[blockIdx.x + 1];
        n = v.head->n_long, list = v.longs, Hk = p.Hk, tokens = tile_tokens(p.g);
        if (at.idx < n) q = list[at.idx];
        if (at.idx + 1 < n) next = list[at.idx + 1];
    }
    __device__ __forceinline__ bool piece() {
        const bool same = at.idx == end.idx && at.item == end.item && at.head == end.head;
        if (at.idx >= n || (same && at.part == end.part)) return false;
        items = (q.z + 2 * tokens - 1) / (2 * tokens);
        t0 = at.item * 2 * tokens, tn = min(2 * tokens, q.z - t0);
        keys = q.z + q.w;
        need0 = (q.w + t0 + min(tn, tokens) + kTileKeys - 1) / kTileKeys;
        tiles = (q.w + t0 + tn + kTileKeys - 1) / kTileKeys;
        one = tn <= tokens;
        last = same ? end.part : tiles;
        return true;
    }
    // The key tiles of place i: first(i), first(i) + stride() .. below end_of(i)
    __device__ __forceinline__ int first(int i) const { return at.part + (one ? i : 0); }
    __device__ __forceinline__ int end_of(int i) const { return one || i ? last : min(last, need0); }
    __device__ __forceinline__ int stride() const { return one ? 2 : 1; }
    __device__ __forceinline__ bool whole() const { return at.part == 0 && last == tiles; }
    __device__ __forceinline__ void step() {
        if (at.idx == end.idx && at.item == end.item && at.head == end.head) {  // the share ends within this head
            at = end;
            return;
        }
        at.part = 0;
        if (++at.head < Hk) return;
        at.head = 0;
        if (++at.item < items) return;
        at.item = 0, ++at.idx;
        q = next;
        if (at.idx + 1 < n) next = list[at.idx + 1];
    }
};

// ---------------------------------------------------------------- copies
// One warp copies the queries and the keys, another the values.  Keys and values take the
// places of one ring by turns; their number is even, so that a place always meets the same
// warp, which then waits on its barriers in every round.
template <class C>
__device__ __forceinline__ void copy_role(const Params &p, const PlanView &v, const CUtensorMap *qm, const CUtensorMap *km,
                                          const CUtensorMap *vm, uint32_t sm, Shared *b, int is_v) {
    constexpr int ROWB = C::E4M3 ? C::D : C::D * 2, HALVES = ROWB > 128 ? 2 : 1;
    constexpr int UNIT = C::E4M3 ? C::RAW : C::TILE, UNITS = C::E4M3 ? C::RAWS : C::STAGES;
    static_assert(UNITS % 2 == 0, "");
    uint64_t *const full = C::E4M3 ? b->raw_full : b->full, *const empty = C::E4M3 ? b->raw_empty : b->empty;
    const int lane = threadIdx.x & 31;
    const int rows = min(p.page, 64), boxes = kTileKeys / rows;
    // lane -> one copy: 64 channels of a box; then (8 bits) a box's scales
    const bool scales = C::E4M3 && lane >= 16 && lane < 16 + boxes;
    const bool copier = lane < boxes * HALVES;
    const int half = scales ? 0 : lane % HALVES, box = scales ? lane - 16 : min(lane / HALVES, boxes - 1);
    Ring ring, qs;
    ring.at = is_v;
    bool first_round = true, first_q = true;
    PageWindow pages;
    Walk w;
    w.begin(p, v);
    for (; w.piece(); w.step()) {
        auto queries = [&](int i) {
            if (!first_q && !wait_warp(b->q_empty + qs.at, qs.parity ^ 1, &b->abort, p.status)) return false;
            if (lane == 0) {
                ++*const_cast<volatile uint32_t *>(b->begun_q + qs.at);
                mbar_arrive_expect_tx(b->q_full + qs.at, (C::D / 64) * w.tokens * p.g * 128);
                for (int h = 0; h < C::D / 64; ++h)
                    tma_load_3d(sm + C::Q + qs.at * C::TILE + h * C::HALF, qm, h * 64, w.at.head * p.g, w.q.y + w.t0 + i * w.tokens,
                                b->q_full + qs.at);
            }
            __syncwarp();
            qs.step(C::QS);
            if (qs.at == 0) first_q = false;
            return true;
        };
        if (!is_v && !queries(0)) return;
        const int entries = min((w.keys + p.page - 1) >> p.page_log, p.max_pages);
        for (int j = w.at.part; j < w.last; ++j) {
            const int key = j * kTileKeys + box * rows, row = key & (p.page - 1);
            pages.at(p, w.q.x, entries, (j * kTileKeys) >> p.page_log);
            const int page = pages.page(p, key >> p.page_log, (copier || scales) && key < w.keys);
            const unsigned with_scales = __ballot_sync(~0u, scales && page >= 0);
            const int slab = page >= 0 ? page * p.Hk + w.at.head : p.n_pages * p.Hk;  // past the cache: zeros
            if (!first_round && !wait_warp(empty + ring.at, ring.parity ^ 1, &b->abort, p.status)) return;
            if (lane == 0) {
                ++*const_cast<volatile uint32_t *>(b->begun + is_v);
                mbar_arrive_expect_tx(full + ring.at, UNIT + __popc(with_scales) * rows);
            }
            __syncwarp();
            const uint32_t to = sm + (C::E4M3 ? C::CODES : C::RING) + ring.at * UNIT + half * C::HALF + box * rows * min(ROWB, 128);
            if (copier) {
                if (is_v)
                    tma_load_3d(to, vm, half * 64, row, slab, full + ring.at);
                else
                    tma_load_3d(to, km, half * 64, row, slab, full + ring.at);
            } else if (scales && page >= 0) {
                bulk_load(smem_u32(b->scales[ring.at % kMaxRaws]) + box * rows,
                          (is_v ? p.vs : p.ks) + (((size_t)page * p.Hk + w.at.head) << p.page_log) + row, rows, full + ring.at);
            }
            ring.step(UNITS), ring.step(UNITS);
            if (ring.at == is_v) first_round = false;
            // the second query tile behind the first keys: its place is free last
            if (!is_v && j == w.at.part && !w.one && !queries(1)) return;
        }
    }
    // the last arrivals on the barriers that this warp waits on
    if (!is_v)
        for (int i = 0; i < C::QS; ++i)
            if (!first_q || i < qs.at) wait_warp(b->q_empty + i, first_q ? 0 : i < qs.at ? qs.parity : qs.parity ^ 1, &b->abort, p.status);
    for (int i = is_v; i < UNITS; i += 2)
        if (!first_round || i < ring.at) wait_warp(empty + i, first_round ? 0 : i < ring.at ? ring.parity : ring.parity ^ 1, &b->abort, p.status);
}

// After giving up: wait (with a limit) for the copies still in flight.
template <class C>
__device__ __forceinline__ void drain(Shared *b) {
    constexpr int UNITS = C::E4M3 ? C::RAWS : C::STAGES;
    uint64_t *const full = C::E4M3 ? b->raw_full : b->full;
    for (int s = 0; s < UNITS; ++s) {
        const int begun = 2 * *const_cast<volatile uint32_t *>(b->begun + (s & 1)) + (s & 1);  // past the warp's last place
        const int rounds = begun > s ? (begun - s + UNITS - 1) / UNITS : 0;
        if (rounds) mbar_wait(full + s, (rounds - 1) & 1);
    }
    for (int i = 0; i < C::QS; ++i) {
        const int q = *const_cast<volatile uint32_t *>(b->begun_q + i);
        if (q) mbar_wait(b->q_full + i, (q - 1) & 1);
    }
}

// ---------------------------------------------------------------- conversion, and the end of a piece
// A tile of codes into a bf16 tile, a thread a key; rows behind the last key become zeros.  Code times
// power of two is exact in bf16.  (The codes' bits moved to bf16's places and multiplied by powers of two
// in bf16, a tenth more instructions on the pipe of the integers: a prompt of 8,192 rows 558 us against 512.)
template <class C>
__device__ __forceinline__ void convert_tile(uint32_t from, uint32_t to, uint32_t byte, int row, bool live) {
    const float up = live ? pow2_of(byte) : 0.f;
    const f2 up2 = f2_pack(up, up);
    if (!live)  // whatever lies there; not by a choice at each store below, which cost a seventh of the kernel's time
        for (int c = 0; c < C::D / 16; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(from + row * C::D + c * 16), "r"(0) : "memory");
    uint32_t x[C::D / 16][4];
#pragma unroll
    for (int c = 0; c < C::D / 16; ++c) {
        const uint32_t at = C::D == 64 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : row * 128 + ((c ^ (row & 7)) << 4);
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x[c][0]), "=r"(x[c][1]), "=r"(x[c][2]), "=r"(x[c][3]) : "r"(from + at) : "memory");
    }
#pragma unroll
    for (int piece = 0; piece < C::D / 8; ++piece) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t h;
            float lo, hi;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(x[piece >> 1][2 * (piece & 1) + (e >> 1)] >> (16 * (e & 1)))));
            asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(h));
            f2_unpack(f2_mul(f2_pack(lo, hi), up2), lo, hi);
            o[e] = pack_bf(lo, hi);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to + (piece >> 3) * C::HALF + row * 128 + (((piece ^ row) & 7) << 4)),
                     "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                     : "memory");
    }
}

// The end of a piece, a thread a row: O out of TMEM, to y or to the workspace.  The next piece's
// scores and weights go on meanwhile.
template <class C>
__device__ __forceinline__ bool end_piece(const Params &p, const Walk &w, Shared *b, unsigned (&parity)[2]) {
    constexpr int D = C::D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const uint32_t t_o = b->tmem + ((uint32_t)(warp & 3) << 21) + 256;
    const int token_in = row / p.g, head_in = row - token_in * p.g;
    const bool whole = w.whole();
    float *const part = p.long_parts + (size_t)(2 * blockIdx.x + (w.at.part > 0 ? 0 : 1)) * part_floats(2 * kTileRows, D);
#pragma unroll 1
    for (int i = 0; i < (w.one ? 1 : 2); ++i) {
        const int token = w.t0 + i * w.tokens + token_in;
        const bool real = token_in < w.tokens && token < w.q.z;
        // the places whose sums these rows have: 0 and 1 both where one tile took both
        const int places = w.one ? (w.first(1) < w.end_of(1) ? 2 : 1) : w.first(i) < w.end_of(i) ? 1 : 0;
        float2 v = make_float2(-INFINITY, 0.f), v1 = v;
        if (places) {
            if (!wait_warp(b->o_full + i, i ? parity[1] : parity[0], &b->abort, p.status)) return false;
            if (places == 2 && !wait_warp(b->o_full + 1, parity[1], &b->abort, p.status)) return false;
            if (i || places == 2) parity[1] ^= 1;
            if (!i) parity[0] ^= 1;
            tc_fence_after_sync();
            v = b->ml[i][row];
            if (places == 2) v1 = b->ml[1][row];
        }
        const float m = fmaxf(v.x, v1.x);
        // a row that has seen no key in a place: sums of zero there
        const float f0 = v.x == -INFINITY ? 1.f : ex2(v.x - m), f1 = v1.x == -INFINITY ? 1.f : ex2(v1.x - m);
        const float l = v.y * f0 + v1.y * f1;
        const float s0 = whole ? f0 / l : f0, s1 = whole ? f1 / l : f1;
        uint16_t *const y = p.y + ((long long)(w.q.y + token) * p.Hq + w.at.head * p.g + head_in) * D;
        const int x = i * kTileRows + row;
        if (!whole && real) reinterpret_cast<float2 *>(part + (size_t)2 * kTileRows * D)[x] = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (places) {
                ld32(t_o + i * D + c, o);
                ld_done();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s0);
            if (places == 2) {
                uint32_t o1[32];
                ld32(t_o + D + c, o1);
                ld_done();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), s1, __uint_as_float(o[e])));
            }
            if (c + 32 == D && places) {  // O is free
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(b->o_free + i);
                    if (places == 2) mbar_arrive(b->o_free + 1);
                }
            }
            if (!real) continue;
            if (whole) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint4 u;
                    u.x = pack_bf(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
                    u.y = pack_bf(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                    u.z = pack_bf(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]));
                    u.w = pack_bf(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7]));
                    *reinterpret_cast<uint4 *>(y + c + e) = u;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4 *>(part + (size_t)x * D + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
    }
    return true;
}

// Tiles of codes become bf16 tiles, pieces are ended.  With codes, a piece is ended when the next
// one's first tiles are there, as many as the ring holds: the products need those first.
template <class C>
__device__ __forceinline__ void help_role(const Params &p, const PlanView &v, uint32_t sm, Shared *b) {
    const int lane = threadIdx.x & 31, row = threadIdx.x & 127;
    unsigned parity[2] = {0, 0};
    Walk w;
    w.begin(p, v);
    if constexpr (!C::E4M3) {
        for (; w.piece(); w.step())
            if (!end_piece<C>(p, w, b, parity)) return;
    } else {
        Ring ring, raw;
        bool first_round = true, to_end = false;
        Walk before = w;
        for (; w.piece(); w.step()) {
            const int units = 2 * (w.last - w.at.part);
#pragma unroll 1
            for (int u = 0; u < units || to_end; ++u) {
                if (to_end && (u == C::STAGES || u == units)) {
                    if (!end_piece<C>(p, before, b, parity)) return;
                    to_end = false;
                    if (u == units) break;
                }
                const int j = w.at.part + (u >> 1);
                if (!wait_warp(b->raw_full + raw.at, raw.parity, &b->abort, p.status)) return;
                if (!first_round && !wait_warp(b->empty + ring.at, ring.parity ^ 1, &b->abort, p.status)) return;
                convert_tile<C>(sm + C::CODES + raw.at * C::RAW, sm + C::RING + ring.at * C::TILE, b->scales[raw.at][row], row,
                                j * kTileKeys + row < w.keys);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(b->full + ring.at), mbar_arrive(b->raw_empty + raw.at);
                raw.step(C::RAWS);
                ring.step(C::STAGES);
                if (ring.at == 0) first_round = false;
            }
            before = w, to_end = true;
        }
        if (to_end && !end_piece<C>(p, before, b, parity)) return;
        for (int i = 0; i < C::STAGES; ++i)
            if (!first_round || i < ring.at)
                wait_warp(b->empty + i, first_round ? 0 : i < ring.at ? ring.parity : ring.parity ^ 1, &b->abort, p.status);
    }
}

// ---------------------------------------------------------------- products
template <class C>
__device__ __forceinline__ bool product_role(const Params &p, const PlanView &v, uint32_t sm, Shared *b) {
    constexpr int D = C::D;
    constexpr uint32_t kIdescS = umma_idesc_bf16(128, 128, false, false), kIdescO = umma_idesc_bf16(128, D, false, true);
    const int lane = threadIdx.x & 31;
    const uint32_t tmem = uniform(b->tmem), lead = elect_one();
    const uint32_t q_desc = uniform(desc_lo(sm + C::Q, 16)), k_desc = uniform(desc_lo(sm + C::RING, 16)), v_desc = uniform(desc_lo(sm + C::RING, C::HALF));
    constexpr uint32_t kStep = C::TILE >> 4;  // from place to place, in descriptors
    Ring ring, qs;
    unsigned p_parity = 0, o_parity = 0, o_used = 0;  // a bit for each place
    // The products' pace is this warp's: operands are worked out before the waits.
    auto wait = [&](uint64_t *bar, unsigned parity) {
        const bool ok = wait_warp(bar, parity, &b->abort, p.status);
        tc_fence_after_sync();
        return ok;
    };
    // S_i = Q K^T; q, k: descriptors
    auto scores = [&](int i, uint32_t q, uint32_t k) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            const uint32_t at = (x >> 2) * (C::HALF >> 4) + (x & 3) * 2;
            mma_ss(tmem + i * 128, q + at, k + at, kIdescS, x > 0, lead);
        }
        commit(b->s_full + i, lead);
    };
    // O_i (+)= P_i V; first: of the piece, when the last one's O_i has to be out of its place
    auto values = [&](int i, uint32_t vd, bool first, bool last) {
        if (first) {
            if (o_used >> i & 1) {
                if (!wait(b->o_free + i, o_parity >> i & 1)) return false;
                o_parity ^= 1u << i;
            }
            o_used |= 1u << i;
        }
        if (!wait(b->p_ready + i, p_parity >> i & 1)) return false;
        p_parity ^= 1u << i;
        mma_ts(tmem + 256 + i * D, tmem + i * 128, vd, kIdescO, !first, lead);
#pragma unroll
        for (int x = 1; x < kTileKeys / 16; ++x) mma_ts(tmem + 256 + i * D, tmem + i * 128 + x * 8, vd + x * 128, kIdescO, true, lead);
        commit(b->pv_done + i, lead);
        if (last) commit(b->o_full + i, lead);
        return true;
    };
    auto release = [&](uint64_t *bar) { commit(bar, lead); };
    // What lies in the tile behind the request's last key is not part of the cache: zeros
    // meet its zero weights.  (8-bit tiles are written so.)
    auto clear = [&](int stage, int from) {
        if (C::E4M3 || from >= kTileKeys) return;
        const int rows = min(p.page, 64), to = (from + rows - 1) / rows * rows;  // copies past the last page's are zeros already
        for (int i = lane; i < (to - from) * (D / 8); i += 32) {
            const int r = from + i / (D / 8), c = i % (D / 8);
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(sm + C::RING + stage * C::TILE + (c >> 3) * C::HALF + r * 128 + (((c ^ r) & 7) << 4)),
                         "r"(0)
                         : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
    };
    Walk w;
    w.begin(p, v);
    for (; w.piece(); w.step()) {
        const int q0 = qs.at;
        const uint32_t q0_desc = q_desc + uniform(q0) * kStep;
        if (!wait(b->q_full + q0, qs.parity)) return false;
        qs.step(C::QS);
        if (w.one) {
            // a single query tile: key tiles by turns in both places, so that the products of one
            // run beside the register work of the other
            int v0 = 0, v1 = 0;  // the places' values
            for (int j = w.at.part; j < w.last + 2; ++j) {
                const int i = uniform((j - w.at.part) & 1), stage = i ? v1 : v0, k_stage = ring.at;
                const uint32_t vd = v_desc + uniform(stage) * kStep, kd = k_desc + uniform(k_stage) * kStep;
                if (j - 2 >= w.at.part) {
                    if (!values(i, vd, j - 2 < w.at.part + 2, j >= w.last)) return false;
                    release(b->empty + stage);
                }
                if (j >= w.last) continue;
                if (!wait(b->full + k_stage, ring.parity)) return false;
                ring.step(C::STAGES);
                scores(i, q0_desc, kd);
                release(b->empty + k_stage);
                if (j == w.last - 1) release(b->q_empty + q0);
                const int next = ring.at;
                if (!wait(b->full + next, ring.parity)) return false;
                ring.step(C::STAGES);
                clear(next, w.keys - j * kTileKeys);
                if (i) v1 = next; else v0 = next;
            }
            continue;
        }
        const int q1 = qs.at;
        const uint32_t q1_desc = q_desc + uniform(q1) * kStep;
        const unsigned q1_parity = qs.parity;
        qs.step(C::QS);
        int v_stage = 0;
        const int end0 = w.end_of(0);
        if (end0 <= w.at.part) release(b->q_empty + q0);  // the first tile's rows see none of these keys
        for (int j = w.at.part; j <= w.last; ++j) {
            // K_j at the ring's place, V_j behind it; V_(j-1) at v_stage
            const int k_stage = ring.at;
            const uint32_t kd = k_desc + uniform(k_stage) * kStep, vd = v_desc + uniform(v_stage) * kStep;
            if (j < w.last) {
                if (!wait(b->full + k_stage, ring.parity)) return false;
                ring.step(C::STAGES);
            }
            if (j > w.at.part && j <= end0 && !values(0, vd, j - 1 == w.at.part, j == end0)) return false;
            if (j < end0) {
                scores(0, q0_desc, kd);
                if (j == end0 - 1) release(b->q_empty + q0);
            }
            if (j > w.at.part) {
                if (!values(1, vd, j - 1 == w.at.part, j == w.last)) return false;
                release(b->empty + v_stage);
            }
            if (j < w.last) {
                if (j == w.at.part && !wait(b->q_full + q1, q1_parity)) return false;
                scores(1, q1_desc, kd);
                release(b->empty + k_stage);
                if (j == w.last - 1) release(b->q_empty + q1);
                v_stage = ring.at;
                if (!wait(b->full + v_stage, ring.parity)) return false;
                ring.step(C::STAGES);
                clear(v_stage, w.keys - j * kTileKeys);
            }
        }
    }
    return true;
}

// ---------------------------------------------------------------- a thread a row
// A row's weights are 2^(c s - M) with m its reference and M = c m rounded up, so that m's own is 1 at most, and all of
// them are relative to the M that there is.  From here on the rounding could leave nothing of it.  But there scores that are
// not equal lie 2^6 and more apart (2^-24 of themselves), so that m is the largest: with c rounded down to a power of two
// c m is exact, the largest weight is 1, and others are 2^-32 at most.
constexpr float kFar = 1073741824.f;  // 2^30
template <class C>
__device__ __forceinline__ bool row_role(const Params &p, const PlanView &v, int i, Shared *b) {
    constexpr int D = C::D;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = b->tmem + lanes + i * 128, t_o = b->tmem + lanes + 256 + i * D;
    auto is_far = [&](float m) { return fabsf(m) * p.c >= kFar; };
    unsigned count = 0, ended = 0;  // key tiles of this place so far, pieces
    Walk w;
    w.begin(p, v);
    const int token_in = row / p.g;
    for (; w.piece(); w.step()) {
        const int t0 = w.t0 + (w.one ? 0 : i * w.tokens), token = t0 + token_in;
        const int first = w.q.w + t0, limit = w.q.w + min(token, w.q.z - 1);  // last keys that the tile's first row and this one see
        const int begin = w.first(i), end = w.end_of(i), stride = w.stride();
        float m = -INFINITY;
        f2 l2 = 0;
        for (int j = begin; j < end; j += stride, ++count) {
            if (!wait_warp(b->s_full + i, count & 1, &b->abort, p.status)) return false;
            tc_fence_after_sync();
            uint32_t s[128];
#pragma unroll
            for (int c = 0; c < 128; c += 32) ld32(t_s + c, s + c);
            ld_done();
            const bool masked = j * kTileKeys + kTileKeys - 1 > first;
            const int seen = limit - j * kTileKeys;
            if (masked) {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (c > seen) s[c] = 0xff800000u;
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) top[c] = __uint_as_float(s[c]);
#pragma unroll
            for (int c = 4; c < 124; c += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[e] = max3(top[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(s[124 + e]));
            const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]);
            if (j == begin) {
                m = most;
            } else {
                const bool behind = (most - m) * p.c > 8.f;
                if (__any_sync(~0u, behind)) {
                    // O waits for its last product, then takes the new reference
                    if (!wait_warp(b->pv_done + i, (count - 1) & 1, &b->abort, p.status)) return false;
                    tc_fence_after_sync();
                    const float by = is_far(m) || is_far(most) ? (m - most) * p.c : __fmul_ru(m, p.c) - __fmul_ru(most, p.c);
                    const float f = behind ? ex2(by) : 1.f;
                    if (behind) m = most;
                    const f2 ff = f2_pack(f, f);
                    l2 = f2_mul(l2, ff);
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        ld32(t_o + c, o);
                        ld_done();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        st32(t_o + c, o);
                    }
                }
            }
            // a row that has seen no key yet has no weights
            const float cr = is_far(m) ? __uint_as_float(__float_as_uint(p.c) & 0x7f800000u) : p.c;
            const float mc = m == -INFINITY ? 0.f : -__fmul_ru(m, cr);
            const f2 c2 = f2_pack(cr, cr), mc2 = f2_pack(mc, mc);
            f2 sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
                if (c) {  // the second half again: its registers held the first half's weights
                    ld32(t_s + 64, s + 64);
                    ld32(t_s + 96, s + 96);
                    ld_done();
                    if (masked) {
#pragma unroll
                        for (int k = 64; k < 128; ++k)
                            if (k > seen) s[k] = 0xff800000u;
                    }
                }
                uint32_t w32[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const f2 x = f2_fma((f2)s[c + e + 1] << 32 | s[c + e], c2, mc2);
                    float lo, hi;
                    f2_unpack(x, lo, hi);
                    lo = ex2(lo), hi = ex2(hi);
                    sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2_pack(lo, hi));
                    w32[e / 2] = pack_bf(lo, hi);
                }
                st32(t_s + c / 2, w32);
            }
            l2 = f2_add(l2, f2_add(sum[0], sum[1]));
            if (j + stride >= end) {
                // the last piece's are read when its O is out (a piece may have one key tile)
                if (ended > 0 && !wait_warp(b->o_free + i, (ended - 1) & 1, &b->abort, p.status)) return false;
                ++ended;
                float l, l_hi;
                f2_unpack(l2, l, l_hi);
                b->ml[i][row] = make_float2(__fmul_ru(m, p.c), l + l_hi);
            }
            st_done();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(b->p_ready + i);
        }
    }
    return true;
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
long_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
            const __grid_constant__ CUtensorMap vm) {
    extern __shared__ __align__(1024) unsigned char raw[];
    let_next_launch();
    // the tiles begin on a multiple of 1024 bytes, the swizzle's period
    const uint32_t sm = (smem_u32(raw) + (uint32_t)sizeof(Shared) + 1023) & ~1023u;
    Shared *b = reinterpret_cast<Shared *>(raw);
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    const bool mine = sm + C::TILES <= smem_u32(raw) + C::BYTES && plan_fits(*v.head, p);
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
    if (warp == 8) {
        tmem_alloc(&b->tmem, 512);
        if ((threadIdx.x & 31) == 0) {
            if (!mine && blockIdx.x == 0) atomicOr(p.status, RS_DEV_LENGTH);
            for (int i = 0; i < C::STAGES; ++i) mbar_init(b->full + i, C::E4M3 ? 4 : 1), mbar_init(b->empty + i, 1);
            for (int i = 0; i < C::RAWS; ++i) mbar_init(b->raw_full + i, 1), mbar_init(b->raw_empty + i, 4);
            for (int i = 0; i < C::QS; ++i) mbar_init(b->q_full + i, 1), mbar_init(b->q_empty + i, 1), b->begun_q[i] = 0;
            for (int i = 0; i < 2; ++i) mbar_init(b->s_full + i, 1), mbar_init(b->p_ready + i, 4), mbar_init(b->pv_done + i, 1);
            for (int i = 0; i < 2; ++i) mbar_init(b->o_full + i, 1), mbar_init(b->o_free + i, 4);
            mbar_init(&b->end, 1);
            b->abort = b->begun[0] = b->begun[1] = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tc_fence_before_sync();
    }
    __syncthreads();
    tc_fence_after_sync();
    if (mine) {
        bool ok = true;
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::ROW_REGS));
            row_role<C>(p, v, warp >> 2, b);
        } else if (warp < 12) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::ISSUE_REGS));
            if (warp == 8) ok = product_role<C>(p, v, sm, b);
            if (warp == 9 || warp == 10) copy_role<C>(p, v, &qm, &km, &vm, sm, b, warp - 9);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::HELP_REGS));
            help_role<C>(p, v, sm, b);
        }
        if (warp == 8 && !ok) {  // products still in flight; elect_one() names the lane that issued them
            commit(&b->end, elect_one());
            mbar_wait(&b->end, 0);
        }
        if (warp == 8) b->ended = !ok;  // (with the wait for all of them behind the barrier the product role spills: 16 prompts 487 us)
    }
    tc_fence_before_sync();
    if (__syncthreads_or(*const_cast<volatile uint32_t *>(&b->abort))) {
        if (warp == 8 && !b->ended) {  // another warp gave up: the last products may be in flight all the same
            commit(&b->end, elect_one());
            mbar_wait(&b->end, 0);
        }
        if (threadIdx.x == 0) drain<C>(b);
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 8) tmem_dealloc(b->tmem, 512);
}

template <class C>
cudaError_t launch_cfg(const Params &p, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t s) {
    static SmemGrants grants;
    const cudaError_t e = grant_smem(reinterpret_cast<const void *>(&long_kernel<C>), C::BYTES, grants);
    if (e != cudaSuccess) return e;
    return launch(long_kernel<C>, p.ctas, kThreads, C::BYTES, s, false, p, q, k, v);
}

}  // namespace

cudaError_t long_launch(const Params &p, int D, bool e4m3, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                        cudaStream_t s) {
    if (D == 64) return e4m3 ? launch_cfg<Cfg<64, true>>(p, q, k, v, s) : launch_cfg<Cfg<64, false>>(p, q, k, v, s);
    return e4m3 ? launch_cfg<Cfg<128, true>>(p, q, k, v, s) : launch_cfg<Cfg<128, false>>(p, q, k, v, s);
}

}  // namespace attn
}  // namespace rs
