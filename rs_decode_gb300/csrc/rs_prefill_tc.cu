// The chunk scan of the gated delta rule for 128-wide heads on the
// fifth-generation tensor cores (tcgen05.mma, fp16 operands, fp32 sums in TMEM).
//
// A CTA carries one head of one request.  Everything is transposed so that the
// M = 128 rows of every product are the head's value columns and a TMEM lane,
// hence two of the CTA's 256 threads, own one of them (one thread the keys
// 0..63 and the chunk's rows 0..31, the other the rest):
//   X = S^T K^T, Z = S^T Q^T     A = S  (hi, lo in TMEM)  B = keys, queries
//   R = V^T - e^G X              (threads)
//   U = R T^T                    A = R  (hi, lo in TMEM)  B = T hi, lo; lower triangular
//   D = (e^(G_C - G) u)^T K      A = u  (hi, lo in TMEM)  B = keys, the same tile read MN-major
//   Y = e^G Z + u^T P^T          A = u  (hi, lo in shared memory)  B = P hi, lo; lower triangular
//   S <- e^(G_C) S + D, y = Y    (threads)
// The state itself stays fp32 in the threads' registers, 64 keys each.
//
// A chunk is a chain of four products with register work between them, so one
// head alone leaves the tensor cores idle half of the time: two CTAs share an
// SM.  That fixes the budget: 256 TMEM columns (below), 128 registers, 102 KiB
// of shared memory, in which only the keys and the vectors are double-buffered
// (they are needed up to the chunk's end; everything else is refilled while
// the chunk goes on).  Two threads a row, not one: the register work is
// straight-line code of thousands of instructions, and two warps that run it
// together on a scheduler share its fetches.
//
// TMEM columns, by phase of a chunk:
//   [0, 64)     S lo  -> U sums -> u hi, lo
//   [64, 128)   X sums -> R hi, lo -> Y sums, starting from e^G Z
//   [128, 192)  Z sums -> D sums, keys 0..63
//   [192, 256)  S hi  -> D sums, keys 64..127
// R and u take the place of the sums that they are made of, 16 rows of the chunk at a
// time: 8 columns of hi and 8 of lo, a step of the product that reads them.
//
// y is held to fp32's accuracy like the state, not to bf16's: where a query meets
// little of a large state, or small values overwrite large ones, the terms of y
// cancel, and what is rounded off them would be left in it.
//
// Measured: 4.46 us a chunk for a CTA alone on its SM, 6.29 for each of two.  The
// tensor cores are at work for 1.3 us of it (34 clocks for each 128 x 64 x 16 product,
// 50 where both operands are in shared memory); the rest is register work, about 1,700
// instructions a warp and chunk at half of the issue slots, waiting on TMEM and
// shared-memory latency and on the barriers between phases.  At 128 registers 12 bytes
// a thread spill, 32 in the form with outputs.  Scales of R and u from bounds that are
// known before their values (4.25 and 5.95 us) cost small values their bits.  Tried in
// the first form, with those and y's operands as single terms (3.9 and 5.8 us), and
// slower: warps specialised into a state chain and outputs (4.8 us a chunk alone: one
// warp a scheduler hides no latency), y of a chunk deferred behind the next one's X
// (4.9 us: Z then waits for it).  Against the register-resident form of the 64-wide
// scan at 128 columns: 16 prompts 0.31 ms instead of 0.58.
#include "rs_prefill.cuh"

namespace rs {

using namespace prefill;

namespace {

constexpr int D = 128;
constexpr int kThreads = 256;
constexpr int kTile = C * D * 2;      // keys or queries of a chunk
constexpr int kHalf = C * 128;        // one 64 x 64 fp16 tile
constexpr int kTmem = 256;

// Shared memory: tiles on 1024-byte boundaries (the swizzle's period).
struct Smem {
    static constexpr int K = 0;                      // two buffers
    static constexpr int Q = K + 2 * kTile;          // queries, then u hi
    static constexpr int T = Q + kTile;              // hi, lo, then u lo
    static constexpr int P = T + 2 * kHalf;          // hi, lo
    static constexpr int V = P + 2 * kHalf;          // [64][128] bf16
    static constexpr int VEC = V + C * D * 2;        // two buffers
    static constexpr int MAX = VEC + 2 * kRecVecs;   // [2][2][128] row maxima of the state and of V
    static constexpr int BAR = MAX + 4 * D * 4;
    static constexpr int BYTES = BAR + 256 + 1024;   // and room to align
};

using f2 = unsigned long long;  // two fp32 values, the operand of paired arithmetic

struct Bars {
    uint64_t full_k[2], full_q, full_t, full_p;  // copies have landed
    uint64_t mx, mz, mu, md, my, mend;                   // products are complete
    uint32_t tmem, abort;
    int nk, nq, nt;                                      // loads begun
    const unsigned char *tiles;                          // the request's keys and queries of this head
    unsigned long long tile_step;
    const Record *rec;                                   // the request's records of this head, p.H apart
};
static_assert(sizeof(Bars) <= 256, "");

__device__ __forceinline__ bool wait_bar(uint64_t *bar, unsigned parity, Bars *b, uint32_t *status) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    volatile uint32_t *abort = &b->abort;
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(status, RS_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The same for a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, unsigned parity, Bars *b, uint32_t *status) {
    return __all_sync(~0u, wait_bar(bar, parity, b, status));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
        "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// Operands in shared memory are 128-byte-swizzled tiles: rows of 128 bytes,
// 8-row groups 1024 bytes apart.  A descriptor's high word is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return (addr >> 4) | ((1024u >> 4) << 16); }
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 bd;\n\tmov.b64 bd, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\tmov.b64 ad, {%1, %3};\n\tmov.b64 bd, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// fp16 A and B, fp32 sums, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

#define R16(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), \
    "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]), "=r"(v[o + 11]),          \
    "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15])
// 16 columns of the warp's 32 lanes, complete on return
__device__ __forceinline__ void ld16(uint32_t addr, f2 (&f)[8]) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : R16(v, 0)
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (f2)v[2 * i + 1] << 32 | v[2 * i];
}
#undef R16
__device__ __forceinline__ void st8(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void st16(uint32_t addr, const f2 (&f)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"((uint32_t)f[0]), "r"((uint32_t)(f[0] >> 32)), "r"((uint32_t)f[1]), "r"((uint32_t)(f[1] >> 32)),
        "r"((uint32_t)f[2]), "r"((uint32_t)(f[2] >> 32)), "r"((uint32_t)f[3]), "r"((uint32_t)(f[3] >> 32)),
        "r"((uint32_t)f[4]), "r"((uint32_t)(f[4] >> 32)), "r"((uint32_t)f[5]), "r"((uint32_t)(f[5] >> 32)),
        "r"((uint32_t)f[6]), "r"((uint32_t)(f[6] >> 32)), "r"((uint32_t)f[7]), "r"((uint32_t)(f[7] >> 32))
        : "memory");
}
__device__ __forceinline__ void st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 values of a row, scaled, as 8 packed hi and 8 packed lo columns.  hi is
// the value cut to 11 bits, lo the fp16 rounding of the rest: 22 bits in all.
__device__ __forceinline__ void put_split(uint32_t hi_addr, uint32_t lo_addr, const f2 *x, f2 up) {
    uint32_t hi[8], lo[8];
    const f2 minus = f2_pack(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f2 v = f2_mul(x[i], up);
        float a, b;
        f2_unpack(v, a, b);
        split_cut(a, b, hi[i], lo[i]);
    }
    st8(hi_addr, hi);
    st8(lo_addr, lo);
}
// The largest magnitude of three.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_b2(f2 v) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float((uint32_t)(v >> 32))), "f"(__uint_as_float((uint32_t)v)));
    return r;
}

struct Work {  // one request's head, as both sides see it
    int n, head_rows;
    __device__ int first(int i) const { return i == 0 ? 0 : head_rows + (i - 1) * C; }
    __device__ int rows(int i) const { return min(i == 0 ? head_rows : C, n - first(i)); }
};

// The copies and products of a chunk are issued by one warp each (X warp 0, U 1,
// D 2, Y 3, Z 4, keys 5, queries and P 6, T 7): an issuing warp falls behind by
// about 40 clocks an instruction, and the others wait for it at the next barrier.
//
// Copies of one head's chunks into shared memory.  Each buffer has one warp
// that refills it, once something that all threads waited for implies that the
// buffer's readers are done.
// (V's rows have the caller's stride: all threads copy them, 16 bytes each; one
// bulk copy a row would hold up its warp for 45 clocks a copy.)
// Where they come from, and how many were begun, is kept beside the barriers.
__device__ __forceinline__ void load_k(Bars *b, uint32_t sm, int i, int heads) {
    if (elect_one()) {
        uint64_t *bar = b->full_k + (i & 1);
        ++b->nk;
        mbar_arrive_expect_tx(bar, kTile + kRecVecs);
        bulk_load(sm + Smem::K + (i & 1) * kTile, b->tiles + (size_t)i * b->tile_step, kTile, bar);
        bulk_load(sm + Smem::VEC + (i & 1) * kRecVecs,
                  reinterpret_cast<const unsigned char *>(b->rec + (size_t)i * heads) + kRecMats, kRecVecs, bar);
    }
    __syncwarp();
}
__device__ __forceinline__ void load_qp(Bars *b, uint32_t sm, int i, int heads) {
    if (elect_one()) {
        ++b->nq;
        mbar_arrive_expect_tx(&b->full_q, kTile);
        bulk_load(sm + Smem::Q, b->tiles + (size_t)i * b->tile_step + kTile, kTile, &b->full_q);
        mbar_arrive_expect_tx(&b->full_p, 2 * kHalf);
        bulk_load(sm + Smem::P, b->rec[(size_t)i * heads].p_hi, 2 * kHalf, &b->full_p);
    }
    __syncwarp();
}
__device__ __forceinline__ void load_t(Bars *b, uint32_t sm, int i, int heads) {
    if (elect_one()) {
        ++b->nt;
        mbar_arrive_expect_tx(&b->full_t, 2 * kHalf);
        bulk_load(sm + Smem::T, b->rec[(size_t)i * heads].t_hi, 2 * kHalf, &b->full_t);
    }
    __syncwarp();
}
// After giving up: wait (with a limit) for what is still in flight.
__device__ __forceinline__ void drain(Bars *b) {
    const int nk = b->nk, nq = b->nq, nt = b->nt;
    for (int c = 0; c < 2; ++c)
        if (nk > c) mbar_wait(b->full_k + c, ((nk + 1 - c) / 2 - 1) & 1);
    if (nq) mbar_wait(&b->full_q, (nq - 1) & 1), mbar_wait(&b->full_p, (nq - 1) & 1);
    if (nt) mbar_wait(&b->full_t, (nt - 1) & 1);
}

// Products, issued by one thread; k, q, t, u, pm: descriptors' low words.
// Steps of 16 in a product's inner dimension are 32 bytes along a row (2 in a
// descriptor), or 16 rows (128) where the tile is read MN-major.
constexpr uint32_t kHalfD = kHalf >> 4;
constexpr uint32_t kHalfStride = ((kHalf >> 4) - (1024 >> 4)) << 16;  // leading offset: from one 64-wide tile to the next
__device__ __forceinline__ void issue_x(uint32_t tm, uint32_t k, Bars *b) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
        mma_ts(tm + 64, tm + 192 + 8 * x, k + (x >> 2) * kHalfD + (x & 3) * 2, idesc_f16(64, false), x > 0);
#pragma unroll
    for (int x = 0; x < 8; ++x)
        mma_ts(tm + 64, tm + 8 * x, k + (x >> 2) * kHalfD + (x & 3) * 2, idesc_f16(64, false), true);
    umma_commit(&b->mx);
}
__device__ __forceinline__ void issue_z(uint32_t tm, uint32_t q, Bars *b) {
#pragma unroll
    for (int x = 0; x < 8; ++x)
        mma_ts(tm + 128, tm + 192 + 8 * x, q + (x >> 2) * kHalfD + (x & 3) * 2, idesc_f16(64, false), x > 0);
#pragma unroll
    for (int x = 0; x < 8; ++x)
        mma_ts(tm + 128, tm + 8 * x, q + (x >> 2) * kHalfD + (x & 3) * 2, idesc_f16(64, false), true);
    umma_commit(&b->mz);
}
__device__ __forceinline__ void issue_u(uint32_t tm, uint32_t t, Bars *b) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // T is lower triangular: rows 16 x and on of its columns 16 x..
        mma_ts(tm + 16 * x, tm + 64 + 16 * x, t + x * 130, idesc_f16(64 - 16 * x, false), x > 0);
        mma_ts(tm + 16 * x, tm + 64 + 16 * x + 8, t + x * 130, idesc_f16(64 - 16 * x, false), true);
        mma_ts(tm + 16 * x, tm + 64 + 16 * x, t + kHalfD + x * 130, idesc_f16(64 - 16 * x, false), true);
    }
    umma_commit(&b->mu);
}
__device__ __forceinline__ void issue_d(uint32_t tm, uint32_t k, Bars *b) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // 16 rows of the chunk a step; two tiles of 64 keys side by side
        mma_ts(tm + 128, tm + 16 * x, k + x * 128 + kHalfStride, idesc_f16(128, true), x > 0);
        mma_ts(tm + 128, tm + 16 * x + 8, k + x * 128 + kHalfStride, idesc_f16(128, true), true);
    }
    umma_commit(&b->md);
}
__device__ __forceinline__ void issue_y(uint32_t tm, uint32_t uh, uint32_t ul, uint32_t pm, Bars *b) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {  // onto e^G Z
        mma_ss(tm + 64 + 16 * x, uh + x * 2, pm + x * 130, idesc_f16(64 - 16 * x, false), true);
        mma_ss(tm + 64 + 16 * x, ul + x * 2, pm + x * 130, idesc_f16(64 - 16 * x, false), true);
        mma_ss(tm + 64 + 16 * x, uh + x * 2, pm + kHalfD + x * 130, idesc_f16(64 - 16 * x, false), true);
    }
    umma_commit(&b->my);
}

// A barrier of a row's two threads (warps w and w + 4), and the larger of their values.
__device__ __forceinline__ void pair_sync(int warp) {
    switch (warp & 3) {
        case 0: asm volatile("bar.sync 1, 64;" ::: "memory"); break;
        case 1: asm volatile("bar.sync 2, 64;" ::: "memory"); break;
        case 2: asm volatile("bar.sync 3, 64;" ::: "memory"); break;
        default: asm volatile("bar.sync 4, 64;" ::: "memory"); break;
    }
}
__device__ __forceinline__ float pair_max(float *m, int hf, int row, int warp, float x) {
    m[hf * D + row] = x;
    pair_sync(warp);
    return fmaxf(x, m[(hf ^ 1) * D + row]);
}

// A head of a request.  Every wait gives up after its time limit; the threads
// learn of it together at the next barrier and leave.
// OUT: with y (otherwise the state alone).
template <bool OUT>
__device__ __forceinline__ void scan_head(const PrefillParams &p, const Request &rq, const Unit &u, unsigned char *smem,
                                          Bars *b) {
    constexpr int DH = D / 2, CH = C / 2;
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), hf = warp >> 2;
    const int row = threadIdx.x & 127;  // value column of the head
    const uint32_t base = __reduce_or_sync(~0u, b->tmem), sm = smem_u32(smem);  // the reduction makes it a uniform register
    const uint32_t lanes = base + ((uint32_t)(warp & 3) << 21);
    const uint32_t t_shi = lanes + 192 + 32 * hf, t_slo = lanes + 32 * hf;          // state
    const uint32_t t_u = lanes + 32 * hf, t_r = lanes + 64 + 32 * hf;  // sums of U; of X and Y
    const uint32_t t_z = lanes + 128 + 32 * hf, t_d = lanes + 128 + 64 * hf;
    Work w;
    w.n = rq.n;
    w.head_rows = min(rq.n, C - rq.ctx % C);
    const int nch = u.c1 - u.c0, h = u.h, r = u.r;
    const int vt = threadIdx.x >> 4, vc = threadIdx.x & 15;  // V: row vt + 16 j, 16-byte piece vc
    const uint16_t *vsrc = p.v + ((long long)rq.row0 + vt) * p.ld_v + h * D + vc * 8;
    auto load_v = [&](int i) {
        if (i < nch && !u.map) {
            const int n = w.rows(u.c0 + i);
            const uint16_t *src = vsrc + (long long)w.first(u.c0 + i) * p.ld_v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = vt + 16 * j < n;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm + Smem::V + (vt + 16 * j) * (D * 2) + vc * 16),
                             "l"(in ? src + 16 * j * p.ld_v : p.v), "r"(in ? 16 : 0)
                             : "memory");
            }
        }
    };
    f2 S[DH / 2];
    {
        const StateSource from = unit_start<OUT, D>(p, rq, u);
        const int o = hf * DH * D + row;
        if (from.kind == 2) {
#pragma unroll
            for (int n = 0; n < DH / 2; ++n) S[n] = f2_pack(from.f[o + 2 * n * D], from.f[o + (2 * n + 1) * D]);
        } else if (from.kind == 3) {
#pragma unroll
            for (int n = 0; n < DH / 2; ++n) S[n] = f2_pack(bf2f(from.b[o + 2 * n * D]), bf2f(from.b[o + (2 * n + 1) * D]));
        } else {
#pragma unroll
            for (int n = 0; n < DH / 2; ++n) {
                const int k = hf * DH + 2 * n;
                S[n] = f2_pack(from.kind == 1 && k == row ? 1.f : 0.f, from.kind == 1 && k + 1 == row ? 1.f : 0.f);
            }
        }
    }
    wait_for_launch();  // for the chunks' records
    if (warp == 5) {
        load_k(b, sm, 0, p.H);
        if (nch > 1) load_k(b, sm, 1, p.H);
    }
    if (OUT && warp == 6) load_qp(b, sm, 0, p.H);
    if (warp == 7) load_t(b, sm, 0, p.H);
    load_v(0);
    auto store_state = [&](float *f, uint16_t *q, size_t slab) {
        slab += hf * DH * D + row;
        if (f) {
#pragma unroll
            for (int n = 0; n < DH / 2; ++n) {
                float lo, hi;
                f2_unpack(S[n], lo, hi);
                f[slab + 2 * n * D] = lo, f[slab + (2 * n + 1) * D] = hi;
            }
        }
        if (q) {
#pragma unroll
            for (int n = 0; n < DH / 2; ++n) {
                float lo, hi;
                f2_unpack(S[n], lo, hi);
                q[slab + 2 * n * D] = (uint16_t)f2bf(lo), q[slab + (2 * n + 1) * D] = (uint16_t)f2bf(hi);
            }
        }
    };

    if (!OUT && u.seg == 0) store_state(p.segs, nullptr, seg_slab(p, u, 0, D * D));  // for the second pass

    const long long ystep = (long long)p.H * D;
    uint16_t *y = p.y + ((long long)rq.row0 * p.H + h) * D + (row & ~1) + (hf * CH + 16 * (row & 1)) * ystep;
    float *rowmax = reinterpret_cast<float *>(smem + Smem::MAX);
    // the first position after the unit's start where a state is to be kept
    int block_end = p.block && p.pool ? ((rq.ctx + w.first(u.c0)) / p.block + 1) * p.block : -1;
    bool ok = true;
    for (int i = 0; i < nch; ++i) {
        const unsigned ph = i & 1, kph = (i >> 1) & 1;
        const int n = w.rows(u.c0 + i);
        const uint32_t sk = desc_lo(sm + Smem::K + (i & 1) * kTile);
        const Vecs &vec = *reinterpret_cast<const Vecs *>(smem + Smem::VEC + (i & 1) * kRecVecs);
        // the state as an operand, its row scaled to fp16's range: the row's
        // two threads agree on its largest magnitude
        float smax = 0.f;
#pragma unroll
        for (int k = 0; k < DH / 2; ++k) {
            float lo, hi;
            f2_unpack(S[k], lo, hi);
            smax = max_abs3(smax, lo, hi);
        }
        smax = pair_max(rowmax, hf, row, warp, smax);
        float sup, sdown;
        row_scale<14>(smax, sup, sdown);
#pragma unroll
        for (int k = 0; k < DH; k += 16) put_split(t_shi + k / 2, t_slo + k / 2, S + k / 2, f2_pack(sup, sup));
        st_done();
        asm volatile("cp.async.wait_all;" ::: "memory");  // this thread's part of V
        tc_fence_before_sync();
        if (__syncthreads_or(!ok)) break;
        if (i > 0 && i + 1 < nch && warp == 5) load_k(b, sm, i + 1, p.H);  // the last chunk's are free: its y is done
        ok = wait_warp(b->full_k + (i & 1), kph, b, p.status) && ok;
        if (warp == 0) {
            tc_fence_after_sync();
            if (elect_one()) issue_x(base, sk, b);
            __syncwarp();
        }
        // V's column, while X is computed
        uint32_t v[CH / 2];
        if (u.map) {
#pragma unroll
            for (int t = 0; t < CH / 2; ++t) v[t] = 0;
        } else {
            const uint16_t *src = reinterpret_cast<const uint16_t *>(smem + Smem::V) + hf * CH * D + row;
#pragma unroll
            for (int t = 0; t < CH; t += 2) v[t / 2] = __byte_perm(src[t * D], src[t * D + D], 0x5410);
        }
        if (OUT && warp == 4) {  // Z, behind X
            ok = wait_warp(&b->full_q, ph, b, p.status) && ok;
            tc_fence_after_sync();
            if (elect_one()) issue_z(base, desc_lo(sm + Smem::Q), b);
            __syncwarp();
        }
        ok = wait_warp(&b->mx, ph, b, p.status) && ok;
        tc_fence_after_sync();
        // R, at a scale from its own largest magnitude: a bound from |S| and |k| is 2^6 and more
        // above it, and a small R behind a large one would lose those bits
        const unsigned long long nsdown = f2_pack(-sdown, -sdown);
        f2 R[CH / 2];
        float rmax = 0.f;
#pragma unroll
        for (int t = 0; t < CH; t += 16) {
            f2 x[8];
            ld16(t_r + t, x);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const ulonglong2 ek = *reinterpret_cast<const ulonglong2 *>(vec.egk + hf * CH + t + 2 * e);
                const uint32_t v0 = v[t / 2 + e], v1 = v[t / 2 + e + 1];
                R[t / 2 + e] = f2_fma(x[e], f2_mul(ek.x, nsdown), (f2)(v0 & 0xffff0000u) << 32 | v0 << 16);
                R[t / 2 + e + 1] = f2_fma(x[e + 1], f2_mul(ek.y, nsdown), (f2)(v1 & 0xffff0000u) << 32 | v1 << 16);
                float a, c;
                f2_unpack(R[t / 2 + e], a, c);
                rmax = max_abs3(rmax, a, c);
                f2_unpack(R[t / 2 + e + 1], a, c);
                rmax = max_abs3(rmax, a, c);
            }
        }
        rmax = pair_max(rowmax + 2 * D, hf, row, warp, rmax);
        float rup, rdown;
        row_scale<14>(rmax, rup, rdown);
#pragma unroll
        for (int t = 0; t < CH; t += 16) put_split(t_r + t, t_r + t + 8, R + t / 2, f2_pack(rup, rup));
        st_done();
        tc_fence_before_sync();
        if (__syncthreads_or(!ok)) { ok = false; break; }
        load_v(i + 1);
        if (warp == 1) {
            ok = wait_warp(&b->full_t, ph, b, p.status) && ok;
            if (OUT) ok = wait_warp(&b->mz, ph, b, p.status) && ok;  // Z reads S lo, where U goes
            tc_fence_after_sync();
            if (elect_one()) issue_u(base, desc_lo(sm + Smem::T), b);
            __syncwarp();
        }
        ok = wait_warp(&b->mu, ph, b, p.status) && ok;
        if (OUT) ok = wait_warp(&b->mz, ph, b, p.status) && ok;
        tc_fence_after_sync();
        // u, with its key's power of two: for y, and with e^(G_C - G) for the state, each at a
        // scale from its own largest magnitude, as R
        f2 U[CH / 2];
        float umax = 0.f, kmax = 0.f;
#pragma unroll
        for (int t = 0; t < CH; t += 16) {
            f2 x[8];
            ld16(t_u + t, x);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const ulonglong2 su = *reinterpret_cast<const ulonglong2 *>(vec.su + hf * CH + t + 2 * e);
                const ulonglong2 ke = *reinterpret_cast<const ulonglong2 *>(vec.ke + hf * CH + t + 2 * e);
                const f2 u0 = U[t / 2 + e] = f2_mul(x[e], su.x), u1 = U[t / 2 + e + 1] = f2_mul(x[e + 1], su.y);
                float a, c;
                if (OUT) {
                    f2_unpack(u0, a, c);
                    umax = max_abs3(umax, a, c);
                    f2_unpack(u1, a, c);
                    umax = max_abs3(umax, a, c);
                }
                f2_unpack(f2_mul(u0, ke.x), a, c);
                kmax = max_abs3(kmax, a, c);
                f2_unpack(f2_mul(u1, ke.y), a, c);
                kmax = max_abs3(kmax, a, c);
            }
        }
        // (the state's and R's maxima are read by now, by all threads)
        if (OUT) rowmax[hf * D + row] = umax;
        kmax = pair_max(rowmax + 2 * D, hf, row, warp, kmax);
        if (OUT) umax = fmaxf(umax, rowmax[(hf ^ 1) * D + row]);
        // Where nothing is written u is 0: a least bound keeps the quotients of the scales
        // in range.  Y's sums start from e^G Z at u's scale: where u is below 2^-30 of the
        // state, the state's size sets it, so that they stay in range too.
        const float least = rmax * 7.88860905221011805411728565283e-31f;  // 2^-100
        float uup, udown, kup, kdown;
        row_scale<14>(fmaxf(umax * rdown, fmaxf(least, smax * 9.31322574615478515625e-10f)), uup, udown);
        row_scale<14>(fmaxf(kmax * rdown, least), kup, kdown);
        const float uups = uup * rdown, kups = kup * rdown;  // from R's scale to u's
        const f2 uup2 = f2_pack(uups, uups);
        if (!OUT && i + 1 < nch && warp == 7) load_t(b, sm, i + 1, p.H);
        // u for Y takes the places of the queries and of T, whose products are complete
        unsigned char *const urow = smem + Smem::Q + row * 128;
        static_assert(Smem::T == Smem::Q + kTile, "u lo lies behind u hi");
#pragma unroll
        for (int t = 0; t < CH; t += 16) {
            f2 *const x = U + t / 2;
            if (OUT) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a, d;
                        f2_unpack(f2_mul(x[4 * c + e], uup2), a, d);
                        split_cut(a, d, hi[e], lo[e]);
                    }
                    unsigned char *const at = urow + (((4 * hf + t / 8 + c) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(at + kTile) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const ulonglong2 ke = *reinterpret_cast<const ulonglong2 *>(vec.ke + hf * CH + t + e);
                x[e / 2] = f2_mul(x[e / 2], ke.x), x[e / 2 + 1] = f2_mul(x[e / 2 + 1], ke.y);
            }
            put_split(t_u + t, t_u + t + 8, x, f2_pack(kups, kups));
        }
        if (OUT) {
            const float zs = sdown * uup;
            const f2 zs2 = f2_pack(zs, zs);
#pragma unroll
            for (int t = 0; t < CH; t += 16) {
                f2 x[8];
                ld16(t_z + t, x);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const ulonglong2 eg = *reinterpret_cast<const ulonglong2 *>(vec.eg + hf * CH + t + e);
                    x[e / 2] = f2_mul(x[e / 2], f2_mul(eg.x, zs2)), x[e / 2 + 1] = f2_mul(x[e / 2 + 1], f2_mul(eg.y, zs2));
                }
                st16(t_r + t, x);
            }
            fence_proxy_async_smem();
        }
        st_done();
        tc_fence_before_sync();
        if (__syncthreads_or(!ok)) { ok = false; break; }
        if (warp == 2) {
            tc_fence_after_sync();
            if (elect_one()) issue_d(base, sk, b);
            __syncwarp();
        }
        if (OUT && warp == 3) {
            ok = wait_warp(&b->full_p, ph, b, p.status) && ok;
            tc_fence_after_sync();
            if (elect_one()) issue_y(base, desc_lo(sm + Smem::Q), desc_lo(sm + Smem::T), desc_lo(sm + Smem::P), b);
            __syncwarp();
        }
        // S <- e^(G_C) S + D
        ok = wait_warp(&b->md, ph, b, p.status) && ok;
        tc_fence_after_sync();
        {
            const unsigned long long all = f2_pack(vec.all, vec.all), kd2 = f2_pack(kdown, kdown);
#pragma unroll
            for (int k = 0; k < DH; k += 16) {
                f2 x[8];
                ld16(t_d + k, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) S[k / 2 + e] = f2_fma(all, S[k / 2 + e], f2_mul(x[e], kd2));
            }
        }
        if (!OUT) continue;
        // y = Y with the query's power of two
        ok = wait_warp(&b->my, ph, b, p.status) && ok;
        tc_fence_after_sync();
        if (i + 1 < nch && warp == 6) load_qp(b, sm, i + 1, p.H);
        if (i + 1 < nch && warp == 7) load_t(b, sm, i + 1, p.H);
        const f2 ud2 = f2_pack(udown, udown);
        uint32_t z[CH / 2];
#pragma unroll
        for (int t = 0; t < CH; t += 16) {
            f2 x[8];
            ld16(t_r + t, x);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const ulonglong2 sq = *reinterpret_cast<const ulonglong2 *>(vec.sq + hf * CH + t + e);
                z[(t + e) / 2] = pack_b2(f2_mul(x[e / 2], f2_mul(sq.x, ud2)));
                z[(t + e) / 2 + 1] = pack_b2(f2_mul(x[e / 2 + 1], f2_mul(sq.y, ud2)));
            }
        }
        // Neighbouring lanes swap halves: an even lane stores its and its neighbour's
        // columns of the first 16 of the thread's 32 rows, an odd lane those of the rest
        {
            const bool odd = row & 1;
            const uint32_t sel0 = odd ? 0x1054 : 0x5410, sel1 = odd ? 0x3276 : 0x7632;
            uint16_t *yc = y + w.first(u.c0 + i) * ystep;
            const int m = n - hf * CH - 16 * odd;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t keep = odd ? z[8 + e] : z[e];
                const uint32_t got = __shfl_xor_sync(~0u, odd ? z[e] : z[8 + e], 1);
                z[e] = __byte_perm(keep, got, sel0);
                z[8 + e] = __byte_perm(keep, got, sel1);
            }
            if (n == C) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    *reinterpret_cast<uint32_t *>(yc) = z[e];
                    yc += ystep;
                    *reinterpret_cast<uint32_t *>(yc) = z[8 + e];
                    yc += ystep;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (2 * e < m) *reinterpret_cast<uint32_t *>(yc) = z[e];
                    yc += ystep;
                    if (2 * e + 1 < m) *reinterpret_cast<uint32_t *>(yc) = z[8 + e];
                    yc += ystep;
                }
            }
        }
        const int end = rq.ctx + w.first(u.c0 + i) + n;
        if (end != block_end) continue;
        block_end += p.block;
        const int slot = block_slot(p, r, end, h == 0 && threadIdx.x == 0);
        if (slot >= 0) {
            const size_t slab = ((size_t)slot * p.H + h) * D * D;
            if (p.prec == RS_PREC_SHARED_BF16)
                store_state(nullptr, static_cast<uint16_t *>(p.pool), slab);
            else
                store_state(static_cast<float *>(p.pool), nullptr, slab);
        }
    }
    if (__syncthreads_or(!ok)) {
        drain(b);
        if (warp < 5) {  // elect_one() names the same lane each time: the one that issued the products
            if (elect_one()) umma_commit(&b->mend);
            __syncwarp();
            mbar_wait(&b->mend, 0);
        }
        return;
    }
    if (!OUT) {
        if (u.map)
            store_state(p.maps, nullptr, seg_slab(p, u, u.seg, D * D));
        else
            store_state(p.segs, nullptr, seg_slab(p, u, u.seg + 1, D * D));
        return;
    }
    if (u.seg < u.nsegs - 1) return;
    store_state(p.hp, p.lp, ((size_t)rq.srow * p.H + h) * D * D);
    if (rq.start != -2 && h == 0 && threadIdx.x == 0) p.base[rq.srow] = p.h[rq.srow] = p.nd[rq.srow] = 0;
}

template <bool OUT>
__global__ void __launch_bounds__(kThreads, 2) scan_tc_kernel(const __grid_constant__ PrefillParams p, int units) {
    extern __shared__ unsigned char raw[];
    if (blockIdx.x == 0) wait_for_launch();  // so that this launch does not end before the one it overlaps
    int q;
    const int h = blockIdx.x % p.H, r = cta_request(p, blockIdx.x / p.H, units, q);
    if (r < 0) return;
    const Request rq = load_request(p, r, h == 0 && q == 0 && threadIdx.x == 0);
    if (!rq.ok) return;
    const Unit u = scan_unit<OUT>(p, blockIdx.x, rq, r, q);
    if (!u.ok) return;
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    Bars *b = reinterpret_cast<Bars *>(smem + Smem::BAR);
    if (threadIdx.x < 32) {
        tmem_alloc(&b->tmem, kTmem);
        if (threadIdx.x == 0) {
            for (uint64_t *x : {b->full_k, b->full_k + 1, &b->full_q, &b->full_t, &b->full_p, &b->mx, &b->mz,
                                &b->mu, &b->md, &b->my})
                mbar_init(x, 1);
            mbar_init(&b->mend, 5);
            b->abort = 0;
            b->nk = b->nq = b->nt = 0;
            b->tiles = p.tiles + ((size_t)(rq.chunk0 + u.c0) * p.G + h / p.rep) * (2 * kTile);
            b->tile_step = (unsigned long long)p.G * (2 * kTile);
            b->rec = p.rec + (size_t)(rq.chunk0 + u.c0) * p.H + h;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tc_fence_before_sync();
    }
    __syncthreads();
    tc_fence_after_sync();
    scan_head<OUT>(p, rq, u, smem, b);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (threadIdx.x < 32) tmem_dealloc(b->tmem, kTmem);
}

}  // namespace

namespace prefill {

template <bool OUT>
cudaError_t scan_tc_launch(const PrefillParams &p, cudaStream_t s) {
    static SmemGrants grants;
    const cudaError_t e = grant_smem(reinterpret_cast<const void *>(&scan_tc_kernel<OUT>), Smem::BYTES, grants);
    if (e != cudaSuccess) return e;
    const int units = scan_units<OUT>(p);
    return launch_after(scan_tc_kernel<OUT>, p.classes * p.R * p.H * units, kThreads, Smem::BYTES, s, start_early(p), p, units);
}
template cudaError_t scan_tc_launch<true>(const PrefillParams &p, cudaStream_t s);
template cudaError_t scan_tc_launch<false>(const PrefillParams &p, cudaStream_t s);

}  // namespace prefill

}  // namespace rs
