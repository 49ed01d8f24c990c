// The plan of a ragged batch: offsets, requests and positions of the packed
// rows, the chunk table, and the state-cache blocks that the batch completes.
//
// Integer work of a few exclusive sums over the requests and one look-up per
// row, chunk and block.  A step's plan is a few kilobytes, so its time is
// launch latency; a prompt batch writes 8 bytes a row.  The sums are cheap
// enough for every CTA to redo, which saves a second launch and a grid-wide
// wait: up to kSmallReqs requests each CTA scans all lengths itself (they come
// from L2) and then fills its share of the rows by binary search in shared
// memory.  Larger batches run the scan once in a CTA of its own and fill in a
// second launch.
//
// Measured: 256 requests of one token 6.1 us a call, 1,021 requests with 462,000
// rows 8.2 us; 4,000 requests of one launch 13 us, 4,096 of two 21, 16,384 41 and
// 65,535 113: there the one CTA's passes of 4,096 requests, about 6 us each, are the time.
#include "rs_common.cuh"
#include "rs_internal.h"

namespace rs {
namespace {

constexpr int kItems = 4;         // requests of one thread in one scan pass
constexpr int kSmallReqs = 4000;  // requests of the one-launch form: three offset arrays in 48 KiB
constexpr long long kMaxEnd = 1ll << 30;  // a request's largest position

struct PlanParams {
    int R, cap, ccap, block, max_blocks, n_free;
    const int32_t *lengths, *context, *free_blocks;
    rs_ragged rg;
    uint32_t *status;
};

// Inclusive sum over the CTA of two values per thread; totals to all threads.
template <int NT>
__device__ __forceinline__ void cta_scan2(long long &a, long long &b, long long *warp_a, long long *warp_b,
                                          long long &tot_a, long long &tot_b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) warp_a[warp] = a, warp_b[warp] = b;
    __syncthreads();
    // every warp sums the warps' totals for itself
    long long x = lane < NT / 32 ? warp_a[lane] : 0, y = lane < NT / 32 ? warp_b[lane] : 0;
#pragma unroll
    for (int o = 1; o < NT / 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o);
        if (lane >= o) x += u, y += v;
    }
    tot_a = __shfl_sync(~0u, x, NT / 32 - 1), tot_b = __shfl_sync(~0u, y, NT / 32 - 1);
    const long long pa = __shfl_sync(~0u, x, warp ? warp - 1 : 0), pb = __shfl_sync(~0u, y, warp ? warp - 1 : 0);
    if (warp > 0) a += pa, b += pb;
}

struct Totals {
    long long rows;  // raw rows, those that do not fit among them
    int fit;         // rows that are planned
    int chunks, blocks, active;
};

// Sums NT * kItems requests starting at r0 and writes the offsets of each to
// tok, chk, blk (at [r - r0 + 1] past the base; entry 0 is the caller's).
// t carries the totals from pass to pass.  Rows, chunks and blocks are summed
// together as if every request fitted into the capacity; only where the rows'
// total says otherwise are the latter two summed again without those that do not.
template <int NT>
__device__ __forceinline__ void scan_pass(const PlanParams &p, int r0, Totals &t, int *tok, int *chk, int *blk,
                                          long long *wa, long long *wb, int *red, bool report) {
    int n[kItems], c[kItems];
    bool bad = false;
    const int first = r0 + threadIdx.x * kItems;
    long long rows = 0, packed = 0;
    long long mine[kItems];
    int active = 0;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int r = first + i;
        n[i] = r < p.R ? p.lengths[r] : 0;
        c[i] = r < p.R && p.context ? p.context[r] : 0;
    }
    auto chunks_blocks = [&](int i) {
        const int chunks = n[i] ? (c[i] + n[i] + RS_CHUNK - 1) / RS_CHUNK - c[i] / RS_CHUNK : 0;
        const int blocks = p.block && n[i] ? (c[i] + n[i]) / p.block - c[i] / p.block : 0;
        return (long long)blocks << 32 | chunks;
    };
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (n[i] < 0 || c[i] < 0 || (long long)n[i] + c[i] > kMaxEnd) {
            bad = true;
            n[i] = c[i] = 0;
        }
        rows += n[i];
        packed += chunks_blocks(i);
        mine[i] = packed;
        active += n[i] > 0;
    }
    long long at = rows, pre = packed, tot, tot_p;
    cta_scan2<NT>(at, pre, wa, wb, tot, tot_p);
    at += t.rows - rows;  // raw rows before this thread's requests
    pre -= packed;
    int end[kItems], all;
    bool over = false;
    if (t.rows + tot <= p.cap) {
        all = (int)(t.rows + tot);
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            at += n[i];
            end[i] = (int)at;
        }
    } else {
        // a request fits if its end does; the rest are planned without rows
        int fit = 0;
        packed = 0, active = 0;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            at += n[i];
            if (at > p.cap) {
                over = over || n[i] > 0;
                n[i] = 0;
                end[i] = -1;
            } else {
                end[i] = fit = (int)at;
            }
            active += n[i] > 0;
            packed += chunks_blocks(i);
            mine[i] = packed;
        }
        // rows that fit: the largest fitting end so far
        const int f = __reduce_max_sync(~0u, fit);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = f;
        __syncthreads();
        all = max(t.fit, __reduce_max_sync(~0u, red[threadIdx.x & (NT / 32 - 1)]));
        pre = packed;
        long long zero = 0, none;
        cta_scan2<NT>(pre, zero, wa, wb, tot_p, none);
        pre -= packed;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (first + i >= p.R) continue;
        const long long q = pre + mine[i];
        tok[first + i - r0 + 1] = end[i] < 0 ? all : end[i];
        chk[first + i - r0 + 1] = t.chunks + (int)(q & 0xffffffffll);
        blk[first + i - r0 + 1] = t.blocks + (int)(q >> 32);
    }
    if (report && bad) atomicOr(p.status, RS_DEV_LENGTH);
    if (report && over) atomicOr(p.status, RS_DEV_CAPACITY);
    t.rows += tot;
    t.fit = all;
    t.chunks += (int)(tot_p & 0xffffffffll);
    t.blocks += (int)(tot_p >> 32);
    __syncthreads();  // the scratch is free
    const int warp_active = __reduce_add_sync(~0u, active);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = warp_active;
    __syncthreads();
    t.active += __reduce_add_sync(~0u, (threadIdx.x & 31) < NT / 32 ? red[threadIdx.x & 31] : 0);
    __syncthreads();
}

// Last request r with cu[r] <= x (requests without rows share their successor's offset).
__device__ __forceinline__ int find(const int *cu, int R, int x) {
    int lo = 0, hi = R;  // cu[lo] <= x < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Fills rows, chunks and blocks, CTA `cta` of `ctas`.
template <int NT>
__device__ __forceinline__ void fill(const PlanParams &p, const int *tok, const int *chk, const int *blk, int cta,
                                     int ctas) {
    const int rows = tok[p.R], chunks = chk[p.R], blocks = blk[p.R];
    const long long stride = (long long)ctas * NT, me = (long long)cta * NT + threadIdx.x;
    // four rows a thread: one search, then steps to the next request
    for (long long i = me; i * 4 < p.cap; i += stride) {
        const int x0 = (int)(i * 4);
        int req[4], pos[4];
        int r = x0 < rows ? find(tok, p.R, x0) : 0;
        int next = x0 < rows ? tok[r + 1] : 0, base = 0;
        if (x0 < rows) base = (p.context ? p.context[r] : 0) - tok[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int x = x0 + e;
            if (x < rows) {
                if (x >= next) {
                    do ++r; while (tok[r + 1] <= x);
                    next = tok[r + 1];
                    base = (p.context ? p.context[r] : 0) - tok[r];
                }
                req[e] = r, pos[e] = x + base;
            } else {
                req[e] = pos[e] = -1;
            }
        }
        if (x0 + 4 <= p.cap) {
            *reinterpret_cast<int4 *>(p.rg.token_req + x0) = make_int4(req[0], req[1], req[2], req[3]);
            *reinterpret_cast<int4 *>(p.rg.token_pos + x0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int e = 0; e < p.cap - x0; ++e) p.rg.token_req[x0 + e] = req[e], p.rg.token_pos[x0 + e] = pos[e];
        }
    }
    for (long long i = me; i < p.ccap; i += stride) {
        int4 v = make_int4(-1, 0, 0, 0);
        if (i < chunks) {
            const int r = find(chk, p.R, (int)i);
            const int c = p.context ? p.context[r] : 0, n = tok[r + 1] - tok[r];
            const int at = c / RS_CHUNK + (int)i - chk[r];
            const int lo = max(at * RS_CHUNK, c), hi = min((at + 1) * RS_CHUNK, c + n);
            v = make_int4(r, tok[r] + lo - c, hi - lo, at);
        }
        reinterpret_cast<int4 *>(p.rg.chunks)[i] = v;
    }
    for (long long i = me; i < blocks; i += stride) {
        const int r = find(blk, p.R, (int)i);
        const int c = p.context ? p.context[r] : 0;
        const int j = c / p.block + (int)i - blk[r];
        const bool got = i < p.n_free, place = j < p.max_blocks;
        if (place) p.rg.block_table[(size_t)r * p.max_blocks + j] = got ? p.free_blocks[i] : -1;
        if (!got || !place) atomicOr(p.status, RS_DEV_BLOCKS);
    }
}

__device__ __forceinline__ void write_counts(const PlanParams &p, const Totals &t) {
    p.rg.cu_tokens[0] = p.rg.cu_chunks[0] = p.rg.cu_blocks[0] = 0;
    p.rg.counts[0] = t.fit, p.rg.counts[1] = t.chunks, p.rg.counts[2] = t.blocks, p.rg.counts[3] = t.active;
}

template <int NT>
__global__ void __launch_bounds__(NT) plan_kernel(const __grid_constant__ PlanParams p) {
    constexpr int MAX = NT * kItems < kSmallReqs ? NT * kItems : kSmallReqs;
    __shared__ int tok[MAX + 1], chk[MAX + 1], blk[MAX + 1];
    __shared__ long long wa[32], wb[32];
    __shared__ int red[32];
    if (threadIdx.x == 0) tok[0] = chk[0] = blk[0] = 0;
    Totals t = {};
    scan_pass<NT>(p, 0, t, tok, chk, blk, wa, wb, red, blockIdx.x == 0);
    if (blockIdx.x == 0) {
        for (int r = threadIdx.x; r < p.R; r += NT) {
            p.rg.cu_tokens[r + 1] = tok[r + 1];
            p.rg.cu_chunks[r + 1] = chk[r + 1];
            p.rg.cu_blocks[r + 1] = blk[r + 1];
        }
        if (threadIdx.x == 0) write_counts(p, t);
    }
    fill<NT>(p, tok, chk, blk, blockIdx.x, gridDim.x);
}

constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ long long wa[32], wb[32];
    __shared__ int red[32];
    Totals t = {};
    for (int r0 = 0; r0 < p.R; r0 += kScanThreads * kItems)
        scan_pass<kScanThreads>(p, r0, t, p.rg.cu_tokens + r0, p.rg.cu_chunks + r0, p.rg.cu_blocks + r0, wa, wb, red, true);
    if (threadIdx.x == 0) write_counts(p, t);
}

// Requests planned without rows share the offset of the rows that fit: the pass
// in which the capacity ran out and all later ones write it.
__global__ void __launch_bounds__(kScanThreads) fill_kernel(const __grid_constant__ PlanParams p) {
    fill<kScanThreads>(p, p.rg.cu_tokens, p.rg.cu_chunks, p.rg.cu_blocks, blockIdx.x, gridDim.x);
}

}  // namespace

cudaError_t ragged_plan_launch(const rs_ragged_desc &rd, const int32_t *lengths, const int32_t *context,
                               const int32_t *free_blocks, const rs_ragged &rg, uint32_t *status, cudaStream_t s) {
    PlanParams p = {rd.R, rd.tokens_cap, ragged_chunks_cap(rd), rd.block, rd.max_blocks, rd.n_free,
                    lengths, context, free_blocks, rg, status};
    // a thread for every four rows and every chunk, at most an SM's worth of CTAs an SM;
    // small CTAs where the requests allow, whose barriers are cheaper
    const long long items = ((long long)p.cap + 3) / 4 + p.ccap;
    auto ctas = [&](int nt, int most) {
        const long long n = (items + nt - 1) / nt;
        return (int)(n < most ? n : most);
    };
    if (rd.R <= 256 * kItems) {
        plan_kernel<256><<<ctas(256, 152 * 4), 256, 0, s>>>(p);
        return cudaGetLastError();
    }
    if (rd.R <= kSmallReqs) {
        plan_kernel<1024><<<ctas(1024, 152), 1024, 0, s>>>(p);
        return cudaGetLastError();
    }
    scan_kernel<<<1, kScanThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    fill_kernel<<<ctas(kScanThreads, 152), kScanThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rs
