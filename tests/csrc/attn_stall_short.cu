// Test-only: the attention kernel of few rows with some of its warps left out, so that the
// waits of the others run out (the build shortens their limit).  Every wait is the library's own
// and bounded; nothing faults.
#include "rs_attn_short.cu"

#include "attn_stall.cuh"

namespace rs {
namespace attn {
namespace {

// idle: 1 the copying warps, 2 the computing ones.  seen: CTAs that gave up, and blocks whose copies were begun in them.
template <class C>
__global__ void __launch_bounds__(kThreads, 1)
stalled_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm, int idle, int *seen) {
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BARS), *empty = full + C::STAGES;
    uint64_t *q_full = empty + C::STAGES, *q_empty = q_full + 1;
    uint32_t *abort = reinterpret_cast<uint32_t *>(q_empty + 1);
    const PlanView v = plan_view(p.plan, p.R, p.ctas);
    const bool mine = plan_fits(*v.head, p);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) mbar_init(full + i, 1), mbar_init(empty + i, kWarps / C::GROUPS);
        mbar_init(q_full, 1), mbar_init(q_empty, kWarps);
        for (int i = 0; i < 2 + kCopiers; ++i) abort[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (mine && threadIdx.x >= kWarps * 32 && !(idle & 1)) produce<C>(p, v, &km, &vm, smem_u32(smem), full, empty, abort);
    if (mine && threadIdx.x < kWarps * 32 && !(idle & 2)) consume<C>(p, v, smem, full, empty, abort);
    const bool gave_up = __syncthreads_or(*reinterpret_cast<volatile uint32_t *>(abort));
    // with the computing warps left out nobody else waits for the last copies
    if ((gave_up || idle) && threadIdx.x == 0) drain<C>(full, abort + 1);
    if (gave_up && threadIdx.x == 0) {
        atomicAdd(seen, 1);
        for (int i = 0; i < kCopiers; ++i) atomicAdd(seen + 1, (int)abort[1 + i]);
    }
}

template <class C>
cudaError_t stalled(const StallCall &c, int idle, int *seen, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(stalled_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES);
    if (e != cudaSuccess) return e;
    stalled_kernel<C><<<c.p.ctas, kThreads, C::BYTES, s>>>(c.p, c.k, c.v, idle, seen);
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace rs

// The arguments of rs_attend for heads of 128, then what is left out and the device int[2] of what was seen.
extern "C" int rs_test_short_stall(const rs_kv_desc *d, const rs_kv *kv, const rs_ragged_desc *rd, const rs_attn *in, void *plan, uint16_t *y,
                                   void *work, uint32_t *status, int idle, int *seen, void *stream) {
    using namespace rs::attn;
    StallCall c;
    if (!stall_call(&c, *d, *kv, *rd, *in, plan, y, work, status) || !c.p.short_rows) return -1;
    cudaStream_t s = (cudaStream_t)stream;
    if (d->type == RS_KV_E4M3)
        return (int)(c.p.short_rows == 16 ? stalled<Cfg<128, true, 1>>(c, idle, seen, s) : stalled<Cfg<128, true, 2>>(c, idle, seen, s));
    return (int)(c.p.short_rows == 16 ? stalled<Cfg<128, false, 1>>(c, idle, seen, s) : stalled<Cfg<128, false, 2>>(c, idle, seen, s));
}
