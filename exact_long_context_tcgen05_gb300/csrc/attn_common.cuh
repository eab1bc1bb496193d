// Device helpers shared by the attention kernels over sequences: waits, exponentials, small shared-memory
// operations and the host readers of a translation unit's device error word.
#pragma once
#include "cqsa_internal.h"
#include "sm103_ptx.cuh"

namespace cqsa {

__device__ __forceinline__ void record_dev_error(DevErr* err, int code, int where) {
  if (atomicCAS(&err->code, 0, code) == 0) {
    err->block = blockIdx.x;
    err->where = where;
  }
}

// Wait for a barrier phase, for at most tmo_us, giving up at once when another role of the CTA has (a
// 32-bit flag in shared memory). The thread sleeps in try_wait between looks at the flag and the clock.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint32_t tmo_us, uint32_t abort_addr,
                                              DevErr* err, int code, int where) {
  if (mbar_try_wait_a(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep_a(bar, parity, 1000000u)) return true;
    if (ld_shared_volatile_u32(abort_addr)) return false;
    if (globaltimer_ns() - t0 > static_cast<uint64_t>(tmo_us) * 1000ull) {
      record_dev_error(err, code, where);
      st_shared_volatile_u32(abort_addr, 1u);
      return false;
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Barrier `id` (1..15) over `n` threads (whole warps).
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// Untiled bulk copy into shared memory, counted in bytes on an mbarrier: both addresses 16-byte aligned, a
// size that is a multiple of 16.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Host readers of a device error word, as device_error_word (attn_fwd.cu) is for the forward's.
#define DEV_ERR_READERS(name, word)                                                                                  \
  int name##_error_word(DevErr* out, int clear) {                                                                    \
    int rc = cuda_status(cudaMemcpyFromSymbol(out, word, sizeof(DevErr)), "read " #name " error word");              \
    if (rc != CQSA_OK || !clear || out->code == 0) return rc;                                                        \
    DevErr z = {0, 0, 0, 0};                                                                                         \
    return cuda_status(cudaMemcpyToSymbol(word, &z, sizeof(z)), "clear " #name " error word");                       \
  }

}  // namespace cqsa
