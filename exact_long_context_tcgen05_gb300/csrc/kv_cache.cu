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
constexpr int kAppendWarps = 8;  // warps of an appending block

enum : int { kCacheSame = 0, kCacheE4m3 = 1, kCacheInt4 = 2 };

// The sequence of token `token` of the packed tensor and its position there; false for a token of no sequence.
__device__ __forceinline__ bool find_token(const CacheArgs& a, int token, int lane, int* seq, long long* pos) {
  int s, first, n, len;
  if (a.n_seqs <= 32) {
    const int k = min(lane, a.n_seqs - 1);
    const int c0 = cu_at(a.cu, k, a.T), c1 = cu_at(a.cu, k + 1, a.T), L = __ldg(a.kv_lens + k);
    const unsigned has = __ballot_sync(0xffffffffu, lane < a.n_seqs && c0 <= token && token < c1);
    if (!has) return false;
    s = 31 - __clz(has);
    first = __shfl_sync(0xffffffffu, c0, s);
    n = __shfl_sync(0xffffffffu, c1, s) - first;
    len = __shfl_sync(0xffffffffu, L, s);
  } else {
    s = seq_of_token(a.cu, a.n_seqs, a.T, token, lane);
    if (s < 0) return false;
    len = __ldg(a.kv_lens + s);
    n = seq_tokens(a.cu, s, a.T, &first);
  }
  *seq = s;
  *pos = static_cast<long long>(len) - n + (token - first);
  return true;
}

// Where position `pos` of sequence s lives: its vectors' index at head 0 (a head is `page` vectors further), -2 for a
// position below zero or beyond the table, or (writing) a page outside the cache.
__device__ __forceinline__ long long row_of(const CacheArgs& a, int s, long long pos, bool writing) {
  if (pos < 0 || pos >= static_cast<long long>(a.max_pages) * a.page) return -2;
  const int page_log2 = 31 - __clz(a.page), slot = static_cast<int>(pos) & (a.page - 1);
  const int p = __ldg(a.table + static_cast<long long>(s) * a.max_pages + (static_cast<int>(pos) >> page_log2));
  if (p < 0 || p >= a.n_pages) {
    if (writing) return -2;
    return slot;  // reading: page 0 stands for an entry outside the cache
  }
  return ((static_cast<long long>(p) * a.Hkv) << page_log2) + slot;
}

// The same for token `token` of the packed tensor; -1 for a token of no sequence.
__device__ __forceinline__ long long cache_row(const CacheArgs& a, int token, int lane, bool writing) {
  int s;
  long long pos;
  return find_token(a, token, lane, &s, &pos) ? row_of(a, s, pos, writing) : -1;
}

__device__ __forceinline__ void unpack8(const uint4& x, int bf16, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack16(w[i], bf16);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// A vector into a quantised cache: lane c of its LPV lanes holds features 8 c .. 8 c + 7. The whole warp calls; `on`: this lane's
// vector is to be written, at vector index `at`.
template <int KIND, int LPV>
__device__ __forceinline__ void put_vector(uint8_t* cache, uint8_t* scale, long long at, int c, bool on, float (&f)[8]) {
  float amax = 0.0f;
  if (KIND == kCacheE4m3) {
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
    if (on) {
      reinterpret_cast<uint2*>(cache)[at * LPV + c] = codes;
      if (c == 0) scale[at] = static_cast<uint8_t>(e + 127);
    }
  } else {
    // four lanes hold the 32 features of a scale
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(f[i]);
      amax = fmaxf(amax, m < INFINITY ? m : INFINITY);  // (NaN counts as infinity)
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const uint32_t b = int4_scale_byte(amax);
    const float unit = int4_scale(b), inv = __frcp_rn(unit);
    // The 32-bit quotient f / unit from the reciprocal with one correction by the remainder, which is exact (Markstein's method). The corrected value is within 2^-46 of the
    // quotient before it is rounded, and a quotient by a number of four significant bits is further than 2^-30 from every border between
    // two roundings, so it is the rounded quotient. A sum with 1.5 * 2^23 + 8 then leaves the nearest (even) whole number + 8 in its lowest bits.
    uint32_t word = 0;
    // Under the largest scale magnitudes past 7 of it are held there first (7 * 61,440 is a number): their quotient's remainder could overflow.
    const float most = b == 247u ? 7.0f * 61440.0f : INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = fminf(fmaxf(f[i], -most), most);
      float q = x * inv;
      q = fmaf(fmaf(-q, unit, x), inv, q);
      word += __float_as_uint(__fadd_rn(q, 12582920.0f)) << (4 * i);
    }
    word -= 0x4b400000u * 0x11111111u;  // the sums' exponents and upper bits, shifted together
    if (b == 255u) word = 0x88888888u;
    if (on) {
      reinterpret_cast<uint32_t*>(cache)[at * LPV + c] = word;
      if ((c & 3) == 0) scale[at * (LPV / 4) + (c >> 2)] = static_cast<uint8_t>(b);
    }
  }
}

template <int D, int BF16, int KIND>
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
        if constexpr (KIND == kCacheSame) {
          if (h < a.Hkv) reinterpret_cast<uint4*>(cache)[at * LPV + c] = x[kv][u];
        } else {
          float f[8];
          unpack8(x[kv][u], BF16, f);
          put_vector<KIND, LPV>(cache, kv ? a.v_scale : a.k_scale, at, c, h < a.Hkv, f);
        }
      }
  }
}

template <int D, int BF16, int KIND>
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
        x[kv][u] = make_uint4(KIND == kCacheInt4 ? 0x88888888u : 0u, 0, 0, 0);  // zeros, for a token without a position
        e[kv][u] = 0;
        if (h < a.Hkv && row >= 0) {
          if (KIND == kCacheInt4) {
            x[kv][u].x = __ldg(reinterpret_cast<const uint32_t*>(cache) + at * LPV + c);
            e[kv][u] = __ldg((kv ? a.v_scale : a.k_scale) + at * (LPV / 4) + (c >> 2));
          } else if (KIND == kCacheE4m3) {
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
        if (KIND == kCacheInt4) {
          // whole number * scale: 7 significant bits at most, exact in either 16-bit type
          const float s = int4_scale(static_cast<uint32_t>(e[kv][u]));
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(static_cast<int>((y.x >> (4 * i)) & 15u) - 8) * s;
          if (!BF16) {  // (7 * 61,440: values past fp16's largest read as the largest)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] > 65504.0f ? 65504.0f : (f[i] < -65504.0f ? -65504.0f : f[i]);
          }
          y = make_uint4(pack16(f[0], f[1], BF16), pack16(f[2], f[3], BF16), pack16(f[4], f[5], BF16), pack16(f[6], f[7], BF16));
        } else if (KIND == kCacheE4m3) {
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

// New tokens into their pages with the position rotation applied on the way, and their queries rotated beside them. A pair
// (x, y) of a token's first `rot` features turns by its position's angle: x cos - y sin, y cos + x sin, each product and sum rounded once
// in 32 bits (no fused multiply-add), so that the result is the same as from elementary operations in any program.
//
// wpt warps share a token: its queries, then its keys, then its values. Keys and values lie as in a plain write, 8 features a lane, so that
// quantising is as there; features that are paired across lanes (the first half of the rotated ones with the second) are exchanged as they were
// loaded, four shuffles a vector, whatever `rot` is. Queries, most of the data, need no such thing: where all features turn, a
// lane takes 8 features of the first half and their partners, and turns both (kHalves). The first loads go out before the token's
// sequence and position are looked up, the row of cosines and sines beside the page. Many tokens are bound by memory and issue together, few by that chain.
// Measured: 16,384 bf16 tokens of 32 and 8 heads of 128 into 4 bits and back 85 us in a captured graph (447 MB, 5.2 TB/s; this kernel alone, cold, 68 us at
// 61% of memory's rate and 54% of issue); of 8 and 2 heads of 64 in fp16 into e4m3 and back 26 us; a step of 24 tokens 4.2 us.
enum : int { kHalves = 0, kNeighbours = 1, kPartHalves = 2 };  // all features, paired by halves; pairs of neighbours; fewer features by halves

// (x cos, y cos') + (x' sin, y' sin') of two features, every product and sum rounded. The assembler makes one multiply-add of a packed product and
// a packed sum, also of mul.rn and add.rn, so a product is a multiply-add with a -0 that comes as an
// argument of the kernel (`none`).
__device__ __forceinline__ float2 turned2(float2 f, float2 c, float2 g, float2 s, float2 none) {
  return __fadd2_rn(__ffma2_rn(f, c, none), __ffma2_rn(g, s, none));
}

__device__ __forceinline__ void unpack4x2(const uint4& x, int bf16, float2 (&f)[4]) {
  f[0] = unpack16(x.x, bf16);
  f[1] = unpack16(x.y, bf16);
  f[2] = unpack16(x.z, bf16);
  f[3] = unpack16(x.w, bf16);
}
__device__ __forceinline__ uint4 pack4x2(const float2 (&f)[4], int bf16) {
  return make_uint4(pack16(f[0].x, f[0].y, bf16), pack16(f[1].x, f[1].y, bf16), pack16(f[2].x, f[2].y, bf16), pack16(f[3].x, f[3].y, bf16));
}

template <int D, int BF16, int KIND, int MODE>
__global__ void __launch_bounds__(32 * kAppendWarps, D == 64 ? 4 : 3) cache_append_kernel(const CacheArgs a, const AppendArgs r, int wpt) {
  constexpr int LPV = D / 8, VPS = 32 / LPV;                        // lanes of a vector and vectors of a step
  constexpr int LPQ = MODE == kHalves ? LPV / 2 : LPV, QPS = 32 / LPQ;  // the same of queries
  constexpr int QB = MODE == kHalves ? 2 : 1, QA = MODE == kHalves ? 2 : 3, KA = D == 64 ? 2 : 4;  // 16-byte pieces of a lane; steps that are loaded ahead
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long token = static_cast<long long>(blockIdx.x) * (kAppendWarps / wpt) + warp / wpt;
  if (token >= a.T) return;
  const int part = warp & (wpt - 1), hl = lane / LPV, c = lane % LPV, ql = lane / LPQ, qc = lane % LPQ;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.q) + token * r.q_stride) + qc;
  uint4* q_out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.q_out) + token * r.Hq * D) + qc;
  uint4 x[QA][QB], y[KA];
  auto load_q = [&](int h0) {  // (q_out may be q: not through the read-only path)
#pragma unroll
    for (int u = 0; u < QA; ++u) {
      const int h = h0 + u * wpt * QPS + ql;
#pragma unroll
      for (int b = 0; b < QB; ++b) x[u][b] = h < r.Hq ? q[h * LPV + b * LPQ] : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_kv = [&](const void* from, long long stride, int h0) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(from) + token * stride) + c;
#pragma unroll
    for (int u = 0; u < KA; ++u) {
      const int h = h0 + u * wpt * VPS + hl;
      y[u] = h < a.Hkv ? __ldg(at + h * LPV) : make_uint4(0, 0, 0, 0);
    }
  };
  load_q(part * QPS);
  int s;
  long long pos;
  if (!find_token(a, static_cast<int>(token), lane, &s, &pos)) return;  // behind the last sequence: left as it was
  if (pos < 0 || pos >= r.max_pos) return;
  load_kv(a.k, a.k_stride, part * VPS);
  const long long row = row_of(a, s, pos, true);
  // cosines and sines of this lane's 8 features (of its first 8, for queries by halves); zeros where it turns none
  const int half = r.rot >> 1;
  const bool turns = MODE == kHalves || 8 * c < r.rot, second = MODE != kNeighbours && 8 * c >= half;
  float2 cs[4], sn[4], none;
  none.x = none.y = r.minus_zero;
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = sn[i] = make_float2(0.0f, 0.0f);
  if (turns) {
    const float* at = r.cos_sin + pos * r.rot;
    if (MODE == kNeighbours) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(at + 4 * c)), s4 = __ldg(reinterpret_cast<const float4*>(at + half + 4 * c));
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cs[i] = make_float2(cc[i], cc[i]);
        sn[i] = make_float2(-ss[i], ss[i]);
      }
    } else {
      const int j = MODE == kHalves ? 8 * (c % (LPV / 2)) : (second ? 8 * c - half : 8 * c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(at + j) + i), s4 = __ldg(reinterpret_cast<const float4*>(at + half + j) + i);
        cs[2 * i] = make_float2(c4.x, c4.y);
        cs[2 * i + 1] = make_float2(c4.z, c4.w);
        sn[2 * i] = make_float2(s4.x, s4.y);
        sn[2 * i + 1] = make_float2(s4.z, s4.w);
      }
    }
  }
  const int other = second ? lane - (half >> 3) : (turns ? lane + (half >> 3) : lane);  // the lane of this one's partners
  // this lane's 8 features of a vector turned, by halves with the sines' sign for its place in the pair in sn
  auto turn = [&](const uint4& v, float2 (&f)[4]) {
    unpack4x2(v, BF16, f);
    float2 g[4];
    if (MODE == kNeighbours) {
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = make_float2(f[i].y, f[i].x);
    } else {
      const uint4 w = make_uint4(__shfl_sync(0xffffffffu, v.x, other), __shfl_sync(0xffffffffu, v.y, other),
                                 __shfl_sync(0xffffffffu, v.z, other), __shfl_sync(0xffffffffu, v.w, other));
      unpack4x2(w, BF16, g);
    }
    if (turns) {  // (what does not turn is left alone: 0 times an infinity would not be)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = turned2(f[i], cs[i], g[i], sn[i], none);
    }
  };
  auto sign = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (MODE != kNeighbours && !second) sn[i] = make_float2(-sn[i].x, -sn[i].y);
  };
  if (MODE != kHalves) sign();
  for (int h0 = part * QPS; h0 < r.Hq; h0 += QA * wpt * QPS) {
    if (h0 != part * QPS) load_q(h0);
#pragma unroll
    for (int u = 0; u < QA; ++u) {
      const int h = h0 + u * wpt * QPS + ql;
      if (h0 + u * wpt * QPS >= r.Hq) break;  // (the same for the whole warp)
      float2 f[4];
      if constexpr (MODE == kHalves) {
        float2 g[4], o[4];
        unpack4x2(x[u][0], BF16, f);
        unpack4x2(x[u][QB - 1], BF16, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = turned2(f[i], cs[i], g[i], make_float2(-sn[i].x, -sn[i].y), none);
          g[i] = turned2(g[i], cs[i], f[i], sn[i], none);
        }
        if (h < r.Hq) {
          q_out[h * LPV] = pack4x2(o, BF16);
          q_out[h * LPV + LPQ] = pack4x2(g, BF16);
        }
      } else {
        turn(x[u][0], f);
        if (h < r.Hq) q_out[h * LPV] = turns ? pack4x2(f, BF16) : x[u][0];
      }
    }
  }
  if (MODE == kHalves) sign();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* cache = static_cast<uint8_t*>(kv ? a.v_cache : a.k_cache);
    uint8_t* scale = kv ? a.v_scale : a.k_scale;
    for (int h0 = part * VPS; h0 < a.Hkv; h0 += KA * wpt * VPS) {
      if (kv) load_kv(a.v, a.v_stride, h0);
      else if (h0 != part * VPS) load_kv(a.k, a.k_stride, h0);
#pragma unroll
      for (int u = 0; u < KA; ++u) {
        const int h = h0 + u * wpt * VPS + hl;
        if (h0 + u * wpt * VPS >= a.Hkv) break;  // (the same for the whole warp)
        const bool put = h < a.Hkv && row >= 0;
        const long long at = row + static_cast<long long>(h) * a.page;
        float2 f[4];
        if (!kv) turn(y[u], f);
        else if (KIND != kCacheSame) unpack4x2(y[u], BF16, f);
        if constexpr (KIND == kCacheSame) {
          if (put) reinterpret_cast<uint4*>(cache)[at * LPV + c] = !kv && turns ? pack4x2(f, BF16) : y[u];
        } else {
          float e[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
          put_vector<KIND, LPV>(cache, scale, at, c, put, e);
        }
      }
    }
  }
}

template <int D, int BF16, int KIND>
int launch_append(const CacheArgs& a, const AppendArgs& r, cudaStream_t stream) {
  // A token's chain of loads (counts, position, page and table row) is what a small step takes: its vectors then go to as
  // many warps as there are. With many tokens a warp each (16,384 tokens of 8 and 2 heads of 64, this kernel's first form: 25 us against 32 with two warps each).
  const int wpt = a.T <= 2 * sm_count() ? kAppendWarps : 1, per = kAppendWarps / wpt;
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) + per - 1) / per));
  if (r.interleaved) cache_append_kernel<D, BF16, KIND, kNeighbours><<<grid, 32 * kAppendWarps, 0, stream>>>(a, r, wpt);
  else if (r.rot == D) cache_append_kernel<D, BF16, KIND, kHalves><<<grid, 32 * kAppendWarps, 0, stream>>>(a, r, wpt);
  else cache_append_kernel<D, BF16, KIND, kPartHalves><<<grid, 32 * kAppendWarps, 0, stream>>>(a, r, wpt);
  return cuda_status(cudaGetLastError(), "cache append kernel launch");
}

template <int D, int BF16, int KIND>
int launch_t(const CacheArgs& a, const AppendArgs* r, bool write, cudaStream_t stream) {
  if (r) return launch_append<D, BF16, KIND>(a, *r, stream);
  const dim3 grid(static_cast<unsigned>((static_cast<long long>(a.T) + kWarps - 1) / kWarps));
  if (write) cache_write_kernel<D, BF16, KIND><<<grid, 32 * kWarps, 0, stream>>>(a);
  else cache_read_kernel<D, BF16, KIND><<<grid, 32 * kWarps, 0, stream>>>(a);
  return cuda_status(cudaGetLastError(), write ? "cache write kernel launch" : "cache read kernel launch");
}

template <int D, int BF16>
int launch_d(const CacheArgs& a, const AppendArgs* r, bool write, cudaStream_t stream) {
  if (a.cache_dtype == CQSA_E4M3) return launch_t<D, BF16, kCacheE4m3>(a, r, write, stream);
  if (a.cache_dtype == CQSA_INT4) return launch_t<D, BF16, kCacheInt4>(a, r, write, stream);
  return launch_t<D, BF16, kCacheSame>(a, r, write, stream);
}

int launch(const CacheArgs& a, const AppendArgs* r, bool write, cudaStream_t stream) {
  if (a.T == 0) return CQSA_OK;
  const bool bf = a.dtype == CQSA_BF16;
  if (a.d == 64) return bf ? launch_d<64, 1>(a, r, write, stream) : launch_d<64, 0>(a, r, write, stream);
  return bf ? launch_d<128, 1>(a, r, write, stream) : launch_d<128, 0>(a, r, write, stream);
}

}  // namespace

int launch_kv_cache(const CacheArgs& a, bool write, cudaStream_t stream) { return launch(a, nullptr, write, stream); }

int launch_kv_append(const CacheArgs& a, const AppendArgs& r, cudaStream_t stream) { return launch(a, &r, true, stream); }

}  // namespace cqsa
