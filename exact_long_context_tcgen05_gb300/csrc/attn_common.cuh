// Device helpers shared by the attention kernels over sequences: waits, exponentials, small shared-memory
// operations and the host readers of a translation unit's device error word.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cqsa_internal.h"
#include "sm103_ptx.cuh"

namespace cqsa {

__device__ __forceinline__ void record_dev_error(DevErr* err, int code, int where) {
  if (atomicCAS(&err->code, 0, code) == 0) {
    err->block = blockIdx.x;
    err->where = where;
  }
}

// A whole warp waits for a barrier phase, for at most tmo_us, giving up at once when another role of the CTA has (a
// 32-bit flag in shared memory). The lanes sleep in try_wait between looks at the flag and the clock, and leave the
// loop together: what follows (tcgen05.ld and .st, ldmatrix, mma.sync) has to be executed by a converged warp.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint32_t tmo_us, uint32_t abort_addr,
                                              DevErr* err, int code, int where) {
  if (__all_sync(0xffffffffu, mbar_try_wait_a(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait_sleep_a(bar, parity, 1000000u))) return true;
    if (__any_sync(0xffffffffu, ld_shared_volatile_u32(abort_addr) != 0)) return false;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > static_cast<uint64_t>(tmo_us) * 1000ull)) {
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

// ---- parts of the tensor-core forward kernels (attn_fwd.cu, attn_seq.cu)
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int bf16) {
  if (bf16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^k for integer-valued k <= 0 (exact; 0 below the normal range).
__device__ __forceinline__ float exp2_int(float k) {
  int e = static_cast<int>(k);
  if (e < -126) return 0.0f;
  return __int_as_float((e + 127) << 23);
}

// 2^k for an integer k, 0 below the normal range and infinity above it.
__device__ __forceinline__ float exp2_int_any(int k) {
  return k < -126 ? 0.0f : __int_as_float((k > 127 ? 255 : k + 127) << 23);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Row maximum of 128 scores: three-input max, four independent chains.
__device__ __forceinline__ float row_max128(const float (&x)[128]) {
  float m0 = fmaxf(x[0], x[1]), m1 = fmaxf(x[2], x[3]), m2 = fmaxf(x[4], x[5]), m3 = fmaxf(x[6], x[7]);
#pragma unroll
  for (int c = 8; c < 128; c += 8) {
    m0 = max3(m0, x[c], x[c + 1]);
    m1 = max3(m1, x[c + 2], x[c + 3]);
    m2 = max3(m2, x[c + 4], x[c + 5]);
    m3 = max3(m3, x[c + 6], x[c + 7]);
  }
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

// p = exp2(fl(x * scale*log2e + 192) - (192 + m_ref)) for the pair (x0, x1), with packed fp32x2
// arithmetic. The first rounding puts the argument on a grid fixed by x alone (2^-16 while the
// sum stays in [128, 256)), so the subtraction of the integer-valued 192 + m_ref is exact.
__device__ __forceinline__ float2 exp_pair(float x0, float x1, float2 sl2v, float2 ncm) {
  const float2 t = __ffma2_rn(make_float2(x0, x1), sl2v, make_float2(192.0f, 192.0f));
  const float2 r = __fadd2_rn(t, ncm);
  return make_float2(fast_exp2(r.x), fast_exp2(r.y));
}

// MMA issue from one elected lane of a converged warp, with descriptors prepared by the whole warp
// and the accumulate flag as an immediate: measured on GB300 to issue at the tensor pipe's own rate
// (a 128x64x16 MMA every 32 cycles), while issuing from a lone thread with register-held flags costs
// ~150 cycles per MMA whatever its size.
template <int ACC>
__device__ __forceinline__ void mma_ss_i(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  if (ACC)
    asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 1;" ::"r"(d), "l"(a), "l"(b), "r"(idesc)
                 : "memory");
  else
    asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, 0;" ::"r"(d), "l"(a), "l"(b), "r"(idesc)
                 : "memory");
}
template <int ACC>
__device__ __forceinline__ void mma_ts_i(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  if (ACC)
    asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, 1;" ::"r"(d), "r"(a), "l"(b), "r"(idesc)
                 : "memory");
  else
    asm volatile("tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, 0;" ::"r"(d), "r"(a), "l"(b), "r"(idesc)
                 : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
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
