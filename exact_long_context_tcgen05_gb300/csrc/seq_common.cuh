// Device helpers shared by the operators over sequences of different lengths (packed prompts, the paged
// cache and the attention over it): where a token's sequence is, and the e4m3 code of a cache vector.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/cqsa.h"

namespace cqsa {

// cu[i] of the cumulative token counts, held inside [0, T] whatever the array says, so that no token
// index derived from it leaves the packed tensors.
__device__ __forceinline__ int cu_at(const int* cu, int i, int T) { return min(max(__ldg(cu + i), 0), T); }

// Tokens of sequence s (0 where the counts fall, which a valid array never does) and its first one.
__device__ __forceinline__ int seq_tokens(const int* cu, int s, int T, int* first) {
  const int a = cu_at(cu, s, T), b = cu_at(cu, s + 1, T);
  *first = a;
  return max(b - a, 0);
}

// Cached positions of sequence s, held inside the positions its row of the page table can name.
__device__ __forceinline__ int seq_positions(const int* kv_lens, int s, long long most) {
  const int n = max(__ldg(kv_lens + s), 0);
  return n > most ? static_cast<int>(most) : n;
}

// The position of the first of a sequence's n new tokens (below zero: those before the first position see nothing). It goes by the
// sequence's own length, also where that passes what its row of the page table can name.
__device__ __forceinline__ int seq_first_position(const int* kv_lens, int s, int n) { return max(__ldg(kv_lens + s), 0) - n; }

// A page index held inside the cache: an entry outside it stands for page 0.
__device__ __forceinline__ int page_at(const int* row, int i, int n_pages) {
  const int p = __ldg(row + i);
  return (p < 0 || p >= n_pages) ? 0 : p;
}

// The sequence a token belongs to (a whole warp asks for one token): the last s with cu[s] <= token, by a
// search in 32 steps at a time; -1 when the token lies behind the last sequence or before the first.
__device__ __forceinline__ int seq_of_token(const int* cu, int n_seqs, int T, int token, int lane) {
  if (token < cu_at(cu, 0, T) || token >= cu_at(cu, n_seqs, T)) return -1;
  int lo = 0, n = n_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < n && cu_at(cu, i, T) <= token;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// A CTA's share of a ragged batch: piece number `place` of sequence `seq` (-1: nothing).
struct Unit {
  int seq, place;
};

// Rank `rank` among the pieces of all sequences (pieces(s) of sequence s), the highest places first; among the pieces of
// one place the sequences' order. One warp: count(L) = pieces at place L or above is a sum over the
// sequences, a binary search finds the place, a walk along the sequences the one of that rank.
template <class F>
__device__ __forceinline__ Unit find_unit(int n_seqs, int rank, int lane, F pieces) {
  const int u0 = lane < n_seqs ? pieces(lane) : 0;  // the first 32 sequences stay in a register
  auto count = [&](int L) -> int {
    int c = max(0, u0 - L);
    for (int s = 32 + lane; s < n_seqs; s += 32) c += max(0, pieces(s) - L);
    return __reduce_add_sync(0xffffffffu, c);
  };
  int most = u0;
  for (int s = 32 + lane; s < n_seqs; s += 32) most = max(most, pieces(s));
  most = __reduce_max_sync(0xffffffffu, most);
  Unit u;
  u.seq = -1;
  u.place = 0;
  if (rank >= count(0)) return u;
  int lo = 0, hi = most;  // count(lo) > rank >= count(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (count(mid) > rank) lo = mid;
    else hi = mid;
  }
  int k = rank - count(lo + 1);
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    const bool has = (s0 == 0 ? u0 : (s0 + lane < n_seqs ? pieces(s0 + lane) : 0)) > lo;
    unsigned b = __ballot_sync(0xffffffffu, has);
    const int n = __popc(b);
    if (k < n) {
      for (int i = 0; i < k; ++i) b &= b - 1;
      u.seq = s0 + __ffs(b) - 1;
      break;
    }
    k -= n;
  }
  u.place = lo;
  return u;
}

// The same pieces in the sequences' order, a sequence's highest place first, for batches of so many sequences that looking
// through them for every rank would take longer than a piece: a walk that goes on from the rank before (ranks
// must not fall), 32 sequences at a time.
struct Walker {
  int s0 = -32, total = 0, mine = 0, before = 0;  // the 32 sequences it stands in; this lane's pieces and those before them
  long long base = 0;                             // pieces before these sequences
  template <class F>
  __device__ __forceinline__ Unit find(int n_seqs, long long rank, int lane, F pieces) {
    while (rank >= base + total) {
      base += total;
      s0 += 32;
      if (s0 >= n_seqs) {
        total = 0;
        s0 = n_seqs;
        Unit none = {-1, 0};
        return none;
      }
      mine = s0 + lane < n_seqs ? pieces(s0 + lane) : 0;
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      before = x - mine;
      total = __shfl_sync(0xffffffffu, x, 31);
    }
    const int r = static_cast<int>(rank - base);
    const int who = __ffs(__ballot_sync(0xffffffffu, r >= before && r < before + mine)) - 1;
    Unit u;
    u.seq = s0 + who;
    u.place = __shfl_sync(0xffffffffu, mine - 1 - (r - before), who);
    return u;
  }
};
// More sequences than this are taken in their order. Ranked, the longest sequence's units do not come last: a hundred prompts of some 50 tokens
// and one of 8,000 behind them take 91 us ranked and 145 in their order (8 query and 2 key heads, d = 64; 390 and 439 with 32 and 8 at
// d = 128). But every unit looks through all sequences: three hundred such prompts alone take 50 us ranked and 34 in order, with
// the long one 122 and 106, a thousand 263 and 81. The backward, with one unit a CTA, is within 10% either way up to 3,000
// sequences but for a thousand with a long one at d = 64 (499 ranked, 634 in order).
constexpr int kRankedSeqs = 256;

// e4m3 with one power of two per vector: the smallest 2^e (e >= -126) under which the largest finite
// |x| is at most 448 = 1.75 * 2^8. A power of two costs e4m3 no precision (the code is a floating-point
// number itself) and makes the value code * 2^e exact in fp32 and, inside its range, in 16 bits; the byte
// kept is e + 127.
__device__ __forceinline__ int e4m3_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}
__device__ __forceinline__ float pow2i(int e) {  // 2^e for e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The byte back as its power of two: 0 stands for 2^-127, 255 for infinity (never written).
__device__ __forceinline__ float exp2_byte(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x400000u);
}

// 4 bits: whole numbers -7 to 7 (kept + 8) times a scale for 32 neighbouring features, (1 + m / 8) 2^(e - 15) for its byte
// 8 e + m (fp16's bits below the sign, but for the lower mantissa): the largest |x| over 7, rounded to nearest even. Four significant
// bits of a scale keep every product with a whole number exact in 16 bits. The byte of a group with a value that is
// not finite is 255, a NaN.
constexpr uint32_t kInt4Least = 0x38800000u, kInt4Most = 0x47700000u;  // 2^-14 and 1.875 * 2^15
__device__ __forceinline__ uint32_t int4_scale_byte(float amax) {
  if (!(amax < INFINITY)) return 255u;
  uint32_t u = __float_as_uint(__fdiv_rn(amax, 7.0f));
  u += 0x7ffffu + ((u >> 20) & 1u);
  return (min(max(u, kInt4Least), kInt4Most) >> 20) - (112u << 3);
}
__device__ __forceinline__ float int4_scale(uint32_t b) { return b >= 248u ? NAN : __uint_as_float((b << 20) + (112u << 23)); }

// Two floats to two e4m3 codes (the first in the low byte), rounded to nearest even.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes to two fp16 numbers (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

__device__ __forceinline__ float2 unpack16(uint32_t w, int bf16) {
  if (bf16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
  if (bf16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace cqsa
