// What the kernels of the attention over a paged cache share: the plan's
// layout, the launch parameters, the walk over a CTA's pieces, page look-ups
// and the copies of keys and values.
//
// A batch's work is laid end to end, request after request, and cut into one
// equal share for each CTA (one an SM).  A share is a run of pieces: whole
// heads of requests, and parts of one at either end.  A part leaves its
// unnormalised sums, its largest score and its sum of weights in the
// workspace; join_kernel puts the parts of a head together, in order.  So the
// shares are equal whatever the lengths are, few rows on a long cache spread
// over the GPU, and results do not change from run to run.
#pragma once

#include <cuda.h>

#include "rs_common.cuh"
#include "rs_internal.h"

namespace rs {
namespace attn {

constexpr int kKeys = 64;        // keys of a block of the short form
constexpr int kTileKeys = 128;   // keys of a tile of the long form
constexpr int kTileRows = 128;   // query rows (token x head of the group) of a tile
constexpr int kCtas = 152;       // shares of the work: one CTA for each SM of the GPU
// What starting a piece costs, in keys' blocks or tiles: its queries, its epilogue.  About 3 us in the short form, four
// blocks of bf16 and seven of 8 bits: with 1, 4 and 7 blocks 64 requests of four drafts took 97, 88 and 89 us and one
// request on 131,072 keys 56, 56 and 59; 256 requests on an 8-bit cache 216, 204 and 196, 33 of 64 heads on 8 there 89, 87
// and 79.  With 1, 2 and 3 tiles, timed in turns, 16 prompts took 535, 457 and 465 us, a mixed batch of 40 262, 257 and 260.
inline int short_start(bool e4m3) { return e4m3 ? 7 : 4; }
constexpr int kLongStart = 2;

// The head of a plan's buffer.  Lists and starts follow it, see PlanView.
struct PlanHead {
    int n_short, n_long;    // requests of either form
    int short_rows;         // a request of at most this many rows of a key head's group is short
    int ctas, max_len;      // what the plan was made for
    int Hq, Hk, R, cap, type;
    int pad[6];
};
static_assert(sizeof(PlanHead) == 64, "");

// A share's first piece.  Short: part = key block, item unused.  Long: item = the
// request's item of two query tiles, part = key tile.
struct Start {
    int idx, item, head, part;
};

// A head that several shares have parts of, at the first of them that begins within it (n 0 at the
// others): how many parts there are, and its rows.
struct Join {
    int n, head, row, tokens;  // parts, key head, packed row of the first token, tokens
};

struct PlanView {
    PlanHead *head;
    int4 *shorts, *longs;           // [R] request, first row, rows, context
    Start *short_start, *long_start;  // [ctas + 1]
    Join *short_join, *long_join;     // [ctas]
    long long *short_cu, *long_cu;  // [R + 1] work before each listed request
};
inline size_t plan_bytes(int R, int ctas) {
    return sizeof(PlanHead) + 32 * (size_t)R + 2 * sizeof(Start) * (size_t)(ctas + 1) + 2 * sizeof(Join) * (size_t)ctas +
           16 * ((size_t)R + 1);
}
__host__ __device__ inline PlanView plan_view(void *plan, int R, int ctas) {
    unsigned char *p = static_cast<unsigned char *>(plan);
    PlanView v;
    v.head = reinterpret_cast<PlanHead *>(p);
    p += sizeof(PlanHead);
    v.shorts = reinterpret_cast<int4 *>(p);
    v.longs = v.shorts + R;
    v.short_start = reinterpret_cast<Start *>(v.longs + R);
    v.long_start = v.short_start + ctas + 1;
    v.short_join = reinterpret_cast<Join *>(v.long_start + ctas + 1);
    v.long_join = v.short_join + ctas;
    v.short_cu = reinterpret_cast<long long *>(v.long_join + ctas);
    v.long_cu = v.short_cu + R + 1;
    return v;
}

// How a batch is run, decided on the host from what it knows.
struct Form {
    int short_rows;   // 0, 16 or 32
    bool any_long;    // requests longer than that are possible
};
// Up to 32 rows of a group (a token's heads that share a key head, or a few drafts') stay in
// the registers of warps' matrix instructions.  Where longer requests are expected beside them, a bf16
// cache's tokens run as tiles too, which saves a launch: 16 tokens beside 8 prompts of 900 107 us against 109 with
// both forms, a mixed batch of 40 257 against 258.  But a key tile of a single query tile takes 1.7 us, 1.4 at the copy's
// rate: 255 tokens behind 20 to 8,000 keys beside a chunk of 512 rows take 411 us so and 356 with both, which a rule that
// counts the requests could have.  With 8 bits the tiles are bound by the conversion of the codes (2.1 us a key tile
// against 0.7), and the short form is kept.
inline Form form_of(int g, int max_len, bool e4m3) {
    Form f;
    const long long rows = (long long)g * max_len;
    if (rows <= 32)
        f.short_rows = rows <= 16 ? 16 : 32;
    else
        f.short_rows = !e4m3 ? 0 : g <= 16 ? 16 : g <= 32 ? 32 : 0;
    f.any_long = rows > f.short_rows;
    return f;
}

__host__ __device__ inline int tile_tokens(int g) { return kTileRows / g; }  // of one query tile

struct Params {
    int Hq, Hk, g, type, page, page_log, n_pages, max_pages, R, cap, ctas, max_len, short_rows;
    const int32_t *pages;
    const uint16_t *q;
    long long ld_q;
    float c;  // scale * log2(e)
    uint16_t *y;
    void *plan;
    const uint8_t *ks, *vs;
    uint32_t *status;
    float *short_parts, *long_parts;  // the workspace's two halves
};

// Whether a plan is one for this call.
__device__ __forceinline__ bool plan_fits(const PlanHead &h, const Params &p) {
    return h.short_rows == p.short_rows && h.max_len == p.max_len && h.ctas == p.ctas && h.Hq == p.Hq && h.Hk == p.Hk && h.R == p.R &&
           h.cap == p.cap && h.type == p.type;
}

// A part's place in the workspace: two a CTA (the end of a head that the CTA before began,
// and the beginning of one that the next CTA goes on with), rows of D sums, then rows of
// (largest score, sum of weights), scores in units of log2.  The short form with 8 bits has the largest of
// score plus value's exponent there, and the logarithm of the sum relative to it.
__host__ __device__ inline size_t part_floats(int rows, int D) { return (size_t)rows * (D + 2); }

// ---------------------------------------------------------------- waits
// As mbar_wait, but any wait of the CTA that gives up ends the others too.  The time is
// looked at once in a while only.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, unsigned parity, volatile uint32_t *abort, uint32_t *status) {
    unsigned long long t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        const unsigned long long t = global_ns();
        if (!t0) t0 = t;
        if (t - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(status, RS_DEV_TIMEOUT);
            return false;
        }
    }
}
// The same for a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, unsigned parity, volatile uint32_t *abort, uint32_t *status) {
    return __all_sync(~0u, wait_bar(bar, parity, abort, status));
}

// The same where what is waited for is mostly there: one look and a vote.  (The short form from an 8-bit
// cache 272 against 290 us; the long form's 8-bit prompts are a tenth slower with it.)
__device__ __forceinline__ bool wait_long(uint32_t bar, unsigned parity, volatile uint32_t *abort, uint32_t *status) {
    unsigned long long t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i) {
            unsigned ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(bar), "r"(parity)
                : "memory");
            if (__all_sync(~0u, ok)) return true;
        }
        if (__any_sync(~0u, *abort != 0)) return false;
        const unsigned long long t = global_ns();
        if (!t0) t0 = t;
        if (__any_sync(~0u, t - t0 > kWaitLimitNs)) {
            *abort = 1;
            atomicOr(status, RS_DEV_TIMEOUT);
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_ready(uint64_t *bar, unsigned parity, volatile uint32_t *abort, uint32_t *status) {
    if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
    return wait_long(smem_u32(bar), parity, abort, status);
}

// A position in a ring of n barriers, with the parity of its current round.
struct Ring {
    int at = 0;
    unsigned parity = 0;
    __device__ __forceinline__ void step(int n) {
        if (++at == n) at = 0, parity ^= 1;
    }
};

// ---------------------------------------------------------------- copies
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int c0, int c1, int c2, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, unsigned bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
using f2 = unsigned long long;  // two fp32 values, the operand of paired arithmetic
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The power of two of an 8-bit head's scale byte (255, of a head that is not finite, gives infinity).
__device__ __forceinline__ float pow2_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// A request's entries of the page table as a copying warp walks along them: a lane
// holds one of 32, and of the 32 after them, which are loaded long before they are asked for.
struct PageWindow {
    int r = -1, first = 0;  // the request, its first entry held
    int now, next;
    __device__ __forceinline__ int load(const Params &p, int entries, int e) const {
        return e < entries ? __ldg(p.pages + (size_t)r * p.max_pages + e) : -1;
    }
    // Moves to the 32 entries that hold entry e; entries: those that the request uses.  Whole warps.
    __device__ __forceinline__ void at(const Params &p, int request, int entries, int e) {
        const int lane = threadIdx.x & 31, from = e & ~31;
        if (request == r && from == first) return;
        const bool on = request == r && from == first + 32;
        r = request, first = from;
        now = on ? next : load(p, entries, from + lane);
        next = load(p, entries, from + 32 + lane);
    }
    // The page of entry e for each lane's e in the window, -1 (and a status bit) if it is none of the cache's.
    __device__ __forceinline__ int page(const Params &p, int e, bool wanted) const {
        const int got = __shfl_sync(~0u, now, e & 31);
        if (got >= 0 && got < p.n_pages) return wanted ? got : -1;
        if (wanted) atomicOr(p.status, RS_DEV_SLOT);
        return -1;
    }
};

__device__ __forceinline__ void wait_for_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... KArgs, class... Args>
cudaError_t launch(void (*kernel)(KArgs...), int grid, int block, int smem, cudaStream_t s, bool early, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid), cfg.blockDim = dim3(block), cfg.dynamicSmemBytes = smem, cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr, cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- launches
cudaError_t plan_launch(const rs_kv_desc &d, const rs_ragged_desc &rd, const rs_ragged &rg, int max_len, int ctas,
                        const Form &f, void *plan, uint32_t *status, cudaStream_t s);
// early: the launch may begin while the one before it in the stream still runs.
cudaError_t short_launch(const Params &p, int D, bool e4m3, const CUtensorMap &k, const CUtensorMap &v, bool early,
                         cudaStream_t s);
cudaError_t long_launch(const Params &p, int D, bool e4m3, const CUtensorMap &q, const CUtensorMap &k,
                        const CUtensorMap &v, cudaStream_t s);
cudaError_t join_launch(const Params &p, int D, bool e4m3, bool any_long, cudaStream_t s);
cudaError_t kv_write_launch(const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_ragged &rg,
                            const int32_t *pages, const uint16_t *k, const uint16_t *v, long long ld_k, long long ld_v,
                            uint32_t *status, cudaStream_t s);
cudaError_t kv_read_launch(const rs_kv_desc &d, const rs_kv &kv, const rs_ragged_desc &rd, const rs_ragged &rg,
                           const int32_t *pages, uint16_t *k, uint16_t *v, uint32_t *status, cudaStream_t s);

}  // namespace attn
}  // namespace rs
