// The paged key/value cache: new tokens into their pages, and positions back out of them.
//
// A cache is [n_pages, Hkv, page, d], K and V apart, 16-bit or e4m3 with one exponent byte per vector
// ([n_pages, Hkv, page]). Token i of a sequence's n tokens has position L - n + i of its L positions and
// lives in slot position % page of page table[s][position / page].
//
// One pass, bound by memory: a warp takes one token's K and V, finds its sequence once, and moves the
// token's heads, 16 bytes of 16-bit data a lane (d / 8 lanes a vector, so 2 or 4 heads at a time; four
// steps' loads of K and V are issued together). What a token waits for one after the other (its sequence, its page, its data) costs
// more than its bytes, so up to 32 sequences are looked at in one load a lane. Quantising needs the vector's largest |x|
// first: a shuffle over its d / 8 lanes while the data stays in registers, so the vector is read once. Infinities become NaN
// (e4m3 has no infinity, and a saturated one would read back as an ordinary value) and do not count for the largest.
//
// 24 sequences, 16,384 new tokens, 8 heads of 128 features, bf16 into e4m3 and back: 38 us for both calls (202 MB, 5.3 TB/s;
// 46 with a warp for K and one for V and a search of the counts per warp; 41 without the results' streaming stores, which leave L2 to
// the cache). A step of 24 tokens: 4.1 us for both, two launches' latency.
#include "cqsa_internal.h"
#include "seq_common.cuh"

namespace cqsa {
namespace {

constexpr int kWarps = 4;    // warps (tokens) of a block
constexpr int kAhead = 4;    // steps whose loads, of K and of V, are in flight

// Where token `token` of the packed tensor lives: its vectors' index at head 0 (a head is `page` vectors
// further), -1 for a token of no sequence, -2 for a position below zero or beyond the table, or (writing) a
// page outside the cache.
__device__ __forceinline__ long long cache_row(const CacheArgs& a, int token, int lane, bool writing) {
  int s, first, n, len;
  if (a.n_seqs <= 32) {
    const int k = min(lane, a.n_seqs - 1);
    const int c0 = cu_at(a.cu, k, a.T), c1 = cu_at(a.cu, k + 1, a.T), L = __ldg(a.kv_lens + k);
    const unsigned has = __ballot_sync(0xffffffffu, lane < a.n_seqs && c0 <= token && token < c1);
    if (!has) return -1;
    s = 31 - __clz(has);
    first = __shfl_sync(0xffffffffu, c0, s);
    n = __shfl_sync(0xffffffffu, c1, s) - first;
    len = __shfl_sync(0xffffffffu, L, s);
  } else {
    s = seq_of_token(a.cu, a.n_seqs, a.T, token, lane);
    if (s < 0) return -1;
    len = __ldg(a.kv_lens + s);
    n = seq_tokens(a.cu, s, a.T, &first);
  }
  const long long pos = static_cast<long long>(len) - n + (token - first);
  if (pos < 0 || pos >= static_cast<long long>(a.max_pages) * a.page) return -2;
  const int page_log2 = 31 - __clz(a.page), slot = static_cast<int>(pos) & (a.page - 1);
  const int p = __ldg(a.table + static_cast<long long>(s) * a.max_pages + (static_cast<int>(pos) >> page_log2));
  if (p < 0 || p >= a.n_pages) {
    if (writing) return -2;
    return slot;  // reading: page 0 stands for an entry outside the cache
  }
  return ((static_cast<long long>(p) * a.Hkv) << page_log2) + slot;
}

template <int D, int BF16, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) cache_write_kernel(const CacheArgs a) {
  constexpr int LPV = D / 8;        // lanes of a vector
  constexpr int HPS = 32 / LPV;     // heads of a step
  const int lane = threadIdx.x & 31;
  const long long token = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= a.T) return;
  const uint16_t* src[2] = {static_cast<const uint16_t*>(a.k) + token * a.k_stride, static_cast<const uint16_t*>(a.v) + token * a.v_stride};
  const int hl = lane / LPV, c = lane % LPV;
  uint4 x[2][kAhead];
  auto load = [&](int h0) {  // the token's own data does not wait for the search
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int h = h0 + u * HPS + hl;
        x[kv][u] = h < a.Hkv ? __ldg(reinterpret_cast<const uint4*>(src[kv] + h * D) + c) : make_uint4(0, 0, 0, 0);
      }
  };
  load(0);
  const long long row = cache_row(a, static_cast<int>(token), lane, true);
  if (row < 0) return;
  for (int h0 = 0; h0 < a.Hkv; h0 += kAhead * HPS) {
    if (h0) load(h0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int h = h0 + u * HPS + hl;
        const long long at = row + static_cast<long long>(h) * a.page;
        uint8_t* cache = static_cast<uint8_t*>(kv ? a.v_cache : a.k_cache);
        if (!E4M3) {
          if (h < a.Hkv) reinterpret_cast<uint4*>(cache)[at * LPV + c] = x[kv][u];
          continue;
        }
        const uint32_t w[4] = {x[kv][u].x, x[kv][u].y, x[kv][u].z, x[kv][u].w};
        float f[8], amax = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = unpack16(w[i], BF16);
          f[2 * i] = p.x;
          f[2 * i + 1] = p.y;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float m = fabsf(f[i]);
          const bool finite = m < INFINITY;
          amax = fmaxf(amax, finite ? m : 0.0f);
          if (!finite) f[i] = NAN;
        }
#pragma unroll
        for (int o = LPV / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = e4m3_exponent(amax);
        const float inv = pow2i(-e);
        uint2 codes;
        codes.x = to_e4m3x2(f[0] * inv, f[1] * inv) | (to_e4m3x2(f[2] * inv, f[3] * inv) << 16);
        codes.y = to_e4m3x2(f[4] * inv, f[5] * inv) | (to_e4m3x2(f[6] * inv, f[7] * inv) << 16);
        if (h < a.Hkv) {
          reinterpret_cast<uint2*>(cache)[at * LPV + c] = codes;
          if (c == 0) (kv ? a.v_scale : a.k_scale)[at] = static_cast<uint8_t>(e + 127);
        }
      }
  }
}

template <int D, int BF16, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) cache_read_kernel(const CacheArgs a) {
  constexpr int LPV = D / 8;
  constexpr int HPS = 32 / LPV;
  const int lane = threadIdx.x & 31;
  const long long token = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (token >= a.T) return;
  const long long row = cache_row(a, static_cast<int>(token), lane, false);
  if (row == -1) return;  // behind the last sequence: left as it was
  const int hl = lane / LPV, c = lane % LPV;
  for (int h0 = 0; h0 < a.Hkv; h0 += kAhead * HPS) {
    uint4 x[2][kAhead];
    int e[2][kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int h = h0 + u * HPS + hl;
        const long long at = row + static_cast<long long>(h) * a.page;
        const uint8_t* cache = static_cast<const uint8_t*>(kv ? a.v_cache : a.k_cache);
        x[kv][u] = make_uint4(0, 0, 0, 0);
        e[kv][u] = 0;
        if (h < a.Hkv && row >= 0) {
          if (E4M3) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(cache) + at * LPV + c);
            x[kv][u].x = w.x;
            x[kv][u].y = w.y;
            e[kv][u] = __ldg((kv ? a.v_scale : a.k_scale) + at);
          } else {
            x[kv][u] = __ldg(reinterpret_cast<const uint4*>(cache) + at * LPV + c);
          }
        }
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const int h = h0 + u * HPS + hl;
        uint16_t* dst = static_cast<uint16_t*>(kv ? a.v_out : a.k_out) + token * (static_cast<long long>(a.Hkv) * D);
        uint4 y = x[kv][u];
        if (E4M3) {
          // code * 2^e: exact in fp32 but for its subnormals, then one rounding to 16 bits
          const float s = exp2_byte(static_cast<uint32_t>(e[kv][u]));
          const uint32_t w[4] = {y.x & 0xffffu, y.x >> 16, y.y & 0xffffu, y.y >> 16};
          uint32_t r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 p = unpack16(e4m3x2_to_f16x2(w[i]), 0);
            r[i] = pack16(p.x * s, p.y * s, BF16);
          }
          // From this power on a code may stand for more than the type's largest value (fp16's 65,504 is held as 256 * 2^8): it reads as
          // the largest, as what was written was finite. (Under a branch: 39 us against 41 for 16,384 tokens.)
          if (e[kv][u] >= 127 + (BF16 ? 120 : 8)) {
            constexpr float MOST = BF16 ? 0x1.fep127f : 65504.0f;
            auto held = [](float x) -> float { return x > MOST ? MOST : (x < -MOST ? -MOST : x); };  // (NaN passes on)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 p = unpack16(e4m3x2_to_f16x2(w[i]), 0);
              r[i] = pack16(held(p.x * s), held(p.y * s), BF16);
            }
          }
          y = make_uint4(r[0], r[1], r[2], r[3]);
        }
        if (h < a.Hkv) __stcs(reinterpret_cast<uint4*>(dst + h * D) + c, y);
      }
  }
}

template <int D, int BF16>
int launch_d(const CacheArgs& a, bool write, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) + kWarps - 1) / kWarps));
  if (write) {
    if (a.cache_dtype == CQSA_E4M3) cache_write_kernel<D, BF16, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else cache_write_kernel<D, BF16, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  } else {
    if (a.cache_dtype == CQSA_E4M3) cache_read_kernel<D, BF16, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else cache_read_kernel<D, BF16, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  }
  return cuda_status(cudaGetLastError(), write ? "cache write kernel launch" : "cache read kernel launch");
}

}  // namespace

int launch_kv_cache(const CacheArgs& a, bool write, cudaStream_t stream) {
  if (a.T == 0) return CQSA_OK;
  const bool bf = a.dtype == CQSA_BF16;
  if (a.d == 64) return bf ? launch_d<64, 1>(a, write, stream) : launch_d<64, 0>(a, write, stream);
  return bf ? launch_d<128, 1>(a, write, stream) : launch_d<128, 0>(a, write, stream);
}

}  // namespace cqsa
