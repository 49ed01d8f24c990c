// Test-only: the attention kernel of many rows with some of its warps left out, as in
// attn_stall_short.cu.  The tensor memory that it holds is freed on every path.
#include "rs_attn_long.cu"

#include "attn_stall.cuh"

namespace rs {
namespace attn {
namespace {

// idle: 1 the copying warps, 2 the warps with a row a thread, 4 the products, 8 (of an 8-bit cache) the conversion and what ends pieces.
template <class C>
__global__ void __launch_bounds__(kThreads, 1)
stalled_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
               const __grid_constant__ CUtensorMap vm, int idle, int *seen) {
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t sm = (smem_u32(raw) + (uint32_t)sizeof(Shared) + 1023) & ~1023u;
    Shared *b = reinterpret_cast<Shared *>(raw);
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    const bool mine = sm + C::TILES <= smem_u32(raw) + C::BYTES && plan_fits(*v.head, p);
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
    if (warp == 8) {
        tmem_alloc(&b->tmem, 512);
        if ((threadIdx.x & 31) == 0) {
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
        if (warp < 8) {
            if (!(idle & 2)) row_role<C>(p, v, warp >> 2, b);
        } else if (warp == 8) {
            if (!(idle & 4)) product_role<C>(p, v, sm, b);
        } else if (warp == 9 || warp == 10) {
            if (!(idle & 1)) copy_role<C>(p, v, &qm, &km, &vm, sm, b, warp - 9);
        } else if (warp >= 12) {
            if (!(idle & 8)) help_role<C>(p, v, sm, b);
        }
    }
    tc_fence_before_sync();
    if (__syncthreads_or(*const_cast<volatile uint32_t *>(&b->abort))) {
        if (warp == 8) {
            commit(&b->end, elect_one());
            mbar_wait(&b->end, 0);
        }
        if (threadIdx.x == 0) {
            drain<C>(b);
            atomicAdd(seen, 1);
            atomicAdd(seen + 1, (int)(b->begun[0] + b->begun[1]));
        }
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 8) tmem_dealloc(b->tmem, 512);
}

template <class C>
cudaError_t stalled(const StallCall &c, int idle, int *seen, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(stalled_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    stalled_kernel<C><<<c.p.ctas, kThreads, C::BYTES, s>>>(c.p, c.q, c.k, c.v, idle, seen);
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace rs

extern "C" int rs_test_long_stall(const rs_kv_desc *d, const rs_kv *kv, const rs_ragged_desc *rd, const rs_attn *in, void *plan, uint16_t *y,
                                  void *work, uint32_t *status, int idle, int *seen, void *stream) {
    using namespace rs::attn;
    StallCall c;
    if (!stall_call(&c, *d, *kv, *rd, *in, plan, y, work, status)) return -1;
    cudaStream_t s = (cudaStream_t)stream;
    return (int)(d->type == RS_KV_E4M3 ? stalled<Cfg<128, true>>(c, idle, seen, s) : stalled<Cfg<128, false>>(c, idle, seen, s));
}
