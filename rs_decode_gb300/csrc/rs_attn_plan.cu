// The plan of a batch's attention: its requests listed by form, the work before
// each of them, and where each CTA's share of the work begins.
//
// Integer work on R requests by one CTA, once for a batch and all its layers:
// sums over the requests, 1,024 at a time, then one thread for each share finds
// its start by binary search.  Its time is the latency of a few dependent loads
// and barriers: 4.5 us for 256 tokens, 7.5 for 16 prompts, 12 for 4,096 requests, 146 for 65,535.
#include "rs_attn.cuh"

namespace rs {
namespace attn {
namespace {

constexpr int kThreads = 1024;

struct PlanParams {
    int Hq, Hk, g, type, R, cap, max_len, short_rows, short_start, ctas;
    long long keys_cap;  // keys that a request's row of the page table has room for
    rs_ragged rg;
    void *plan;
    uint32_t *status;
};

// Work of a long request's first i items on one key head; tq tokens an item of two query
// tiles.  All of them but the request's last are full: they see ceil((ctx + (i + 1) tq) / 128)
// key tiles.  The sum of those is taken from the sum of the numerators, less the remainders
// of 128, which repeat after 128 / gcd(tq, 128) items.
__device__ __forceinline__ long long items_before(int ctx, int tq, int i) {
    const long long first = (long long)ctx + tq + kTileKeys - 1;
    const int low = tq & -tq, period = low >= kTileKeys ? 1 : kTileKeys / low;
    auto remainders = [&](int m) {
        long long s = 0;
        int x = (int)(first & (kTileKeys - 1));
        for (int j = 0; j < m; ++j) {
            s += x;
            x = (x + tq) & (kTileKeys - 1);
        }
        return s;
    };
    long long rest = remainders(i % period);
    if (i >= period) rest += (i / period) * remainders(period);
    const long long sum = i * first + (long long)tq * ((long long)i * (i - 1) / 2);
    return (sum - rest) / kTileKeys + (long long)i * kLongStart;
}

__device__ __forceinline__ void scan3(long long &a, long long &b, long long &c, long long (*part)[32], long long *tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(~0u, a, o), y = __shfl_up_sync(~0u, b, o), z = __shfl_up_sync(~0u, c, o);
        if (lane >= o) a += x, b += y, c += z;
    }
    if (lane == 31) part[0][warp] = a, part[1][warp] = b, part[2][warp] = c;
    __syncthreads();
    long long v[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        long long x = part[k][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        tot[k] = __shfl_sync(~0u, x, 31);
        v[k] = __shfl_sync(~0u, x, warp ? warp - 1 : 0);
        if (!warp) v[k] = 0;
    }
    a += v[0], b += v[1], c += v[2];
    __syncthreads();
}

// Last i with cu[i] <= x, of n + 1 entries, x < cu[n].
__device__ __forceinline__ int find(const long long *cu, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) attn_plan_kernel(const __grid_constant__ PlanParams p) {
    __shared__ long long part[3][32];
    __shared__ Start starts[2 * (kCtas + 1)];
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    const int tq = 2 * tile_tokens(p.g);
    int n_short = 0, n_long = 0;
    long long work_s = 0, work_l = 0;
    if (threadIdx.x == 0) v.short_cu[0] = v.long_cu[0] = 0;
    for (int r0 = 0; r0 < p.R; r0 += kThreads) {
        const int r = r0 + threadIdx.x;
        int row0 = 0, n = 0, ctx = 0;
        if (r < p.R) {
            row0 = p.rg.cu_tokens[r];
            n = p.rg.cu_tokens[r + 1] - row0;
            if (n != 0) {
                const bool rows_ok = row0 >= 0 && n > 0 && n <= p.cap && row0 <= p.cap - n;
                ctx = rows_ok ? p.rg.token_pos[row0] : -1;
                if (ctx < 0 || n > p.max_len || (long long)ctx + n > p.keys_cap) {
                    atomicOr(p.status, RS_DEV_LENGTH);
                    n = 0;
                }
            }
        }
        const bool is_short = n > 0 && (long long)n * p.g <= p.short_rows, is_long = n > 0 && !is_short;
        long long count = (is_short ? 1ll : 0) | (is_long ? 1ll << 32 : 0), ws = 0, wl = 0;
        if (is_short) ws = (long long)p.Hk * ((ctx + n + kKeys - 1) / kKeys + p.short_start);
        if (is_long) {
            const int items = (n + tq - 1) / tq;
            wl = p.Hk * (items_before(ctx, tq, items - 1) + kLongStart + (ctx + n + kTileKeys - 1) / kTileKeys);
        }
        long long tot[3];
        scan3(count, ws, wl, part, tot);
        if (is_short) {
            const int i = n_short + (int)(count & 0xffffffff) - 1;
            v.shorts[i] = make_int4(r, row0, n, ctx);
            v.short_cu[i + 1] = work_s + ws;
        }
        if (is_long) {
            const int i = n_long + (int)(count >> 32) - 1;
            v.longs[i] = make_int4(r, row0, n, ctx);
            v.long_cu[i + 1] = work_l + wl;
        }
        n_short += (int)(tot[0] & 0xffffffff), n_long += (int)(tot[0] >> 32);
        work_s += tot[1], work_l += tot[2];
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        PlanHead h = {};
        h.n_short = n_short, h.n_long = n_long, h.short_rows = p.short_rows, h.ctas = p.ctas, h.max_len = p.max_len;
        h.Hq = p.Hq, h.Hk = p.Hk, h.R = p.R, h.cap = p.cap, h.type = p.type;
        *v.head = h;
    }
    for (int i = threadIdx.x; i < 2 * (p.ctas + 1); i += kThreads) {
        const bool lng = i > p.ctas;
        const int c = lng ? i - p.ctas - 1 : i;
        const long long all = lng ? work_l : work_s, share = (all + p.ctas - 1) / p.ctas, x = c * share;
        Start s = {lng ? n_long : n_short, 0, 0, 0};
        if (x < all && !lng) {
            s.idx = find(v.short_cu, n_short, x);
            const int4 q = v.shorts[s.idx];
            const long long at = x - v.short_cu[s.idx];
            const int one = (q.w + q.z + kKeys - 1) / kKeys + p.short_start;
            s.head = (int)(at / one);
            s.part = max(0, (int)(at % one) - p.short_start);
        } else if (x < all) {
            s.idx = find(v.long_cu, n_long, x);
            const int4 q = v.longs[s.idx];
            const long long at = x - v.long_cu[s.idx];
            const int items = (q.z + tq - 1) / tq;
            int lo = 0, hi = items;  // the last item whose work before it is at most at
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.Hk * items_before(q.w, tq, mid) <= at) lo = mid; else hi = mid;
            }
            s.item = lo;
            const long long in = at - p.Hk * items_before(q.w, tq, lo);
            const int one = kLongStart + (q.w + min(q.z, (lo + 1) * tq) + kTileKeys - 1) / kTileKeys;
            s.head = (int)(in / one);
            s.part = max(0, (int)(in % one) - kLongStart);
        }
        (lng ? v.long_start : v.short_start)[c] = starts[i] = s;
    }
    __syncthreads();
    // Heads that are cut, so that the join does not have to search for them (2 us).  No share that begins
    // within a head is empty: shares are whole units of work, of which each part of a head is one.
    for (int i = threadIdx.x; i < 2 * p.ctas; i += kThreads) {
        const bool lng = i >= p.ctas;
        const int c = lng ? i - p.ctas : i;
        const Start *at = starts + (lng ? p.ctas + 1 : 0);
        const Start s = at[c];
        auto same = [&](const Start &o) { return o.idx == s.idx && o.item == s.item && o.head == s.head && o.part > 0; };
        Join j = {0, 0, 0, 0};
        if (c > 0 && s.idx < (lng ? n_long : n_short) && s.part > 0 && !same(at[c - 1])) {
            int end = c + 1;
            while (end < p.ctas && same(at[end])) ++end;
            const int4 q = (lng ? v.longs : v.shorts)[s.idx];
            const int t0 = s.item * tq;
            j.n = 1 + end - c, j.head = s.head, j.row = q.y + t0, j.tokens = lng ? min(tq, q.z - t0) : q.z;
        }
        (lng ? v.long_join : v.short_join)[c] = j;
    }
}

}  // namespace

cudaError_t plan_launch(const rs_kv_desc &d, const rs_ragged_desc &rd, const rs_ragged &rg, int max_len, int ctas,
                        const Form &f, void *plan, uint32_t *status, cudaStream_t s) {
    PlanParams p = {d.Hq, d.Hk, d.Hq / d.Hk, d.type, rd.R, rd.tokens_cap, max_len, f.short_rows, short_start(d.type == RS_KV_E4M3), ctas,
                    (long long)d.max_pages * d.page, rg, plan, status};
    attn_plan_kernel<<<1, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
}  // namespace rs
