// Attention of each new token over a few pages of its sequence, selected by a score that reads a page's bounds instead of its keys.
//
// Bounds: for a page and key head, the largest and the smallest key of each feature as whole multiples (8 bits) of the smallest power of two
// under which all lie within 127: 2 d + 1 bytes, against the page's 512 a slot in 16 bits at d = 128. Queries likewise, a power of two for each
// vector. The score of a page for a token and key head is max over the group's heads of sum_f max(q_f hi_f, q_f lo_f): but for the roundings an
// upper bound of the page's dot products. The sums are whole numbers below 2^21 and are scaled by powers of two, so every order of summation
// gives the same score and every run and program the same choice.
//
// Three kernels before the attention: bounds_kernel (a block per page and head that new tokens came into), score_kernel (the products of pages and
// queries; bound by the reading of bounds for single tokens) and select_few_kernel or select_kernel (a block per token and head: the n-th largest
// score, then the pages from there on up in ascending order, equal scores first come). The attention itself is attn_decode.cu's and attn_decode4.cu's: each
// token is a sequence of its own whose table, one for each key head, lists the pages chosen, its own page last, so that only the end of
// the last page is masked.
//
// Measured in a captured graph, bounds of the new pages included: 48 sequences of 1,000,000 4-bit positions together, 32 and 8 heads of 128, 64 pages
// of 32 each: 72 us (kernel by kernel, cold: bounds 7, scores 22, choice 14, attention 32, joining 5); one token over 131,072 fp16 positions,
// 32 pages of 64: 24 us, five launches; 200 tokens over 65,536: 155 us, of which the attention's reading of 839 MB of pages, each token's own, is most.
// (The torch calls take some 8 us more on the host.) A chunk's time grows with its tokens, 0.54 us each from 1,000 to 8,192 over these positions, 16 pages of
// 64: 0.81 to 0.87 of what attention over all of them takes.
// On half of the first the score kernel has 24% of memory's rate and 49% of issue: loads in flight bound it.
#include <math.h>
#include <string.h>

#include "cqsa_internal.h"
#include "seq_common.cuh"

namespace cqsa {
namespace {

enum : int { kCacheSame = 0, kCacheE4m3 = 1, kCacheInt4 = 2 };

// The exponent of the smallest power of two, 2^-126 or more, under which a finite magnitude is at most 127.
__device__ __forceinline__ int bound_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  return max(static_cast<int>(b >> 23) - 127 - 6 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0), -126);
}

// 8 features of a cached key, lane c of the d / 8 that hold it.
template <int D, int BF16, int KIND>
__device__ __forceinline__ void cached8(const uint8_t* cache, const uint8_t* scale, long long vec, int c, float (&f)[8]) {
  constexpr int LPV = D / 8;
  if constexpr (KIND == kCacheSame) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(cache) + vec * LPV + c);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack16(w[i], BF16);
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else if constexpr (KIND == kCacheE4m3) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(cache) + vec * LPV + c);
    const float s = exp2_byte(__ldg(scale + vec));
    const uint32_t w[4] = {x.x & 0xffffu, x.x >> 16, x.y & 0xffffu, x.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack16(e4m3x2_to_f16x2(w[i]), 0);
      f[2 * i] = p.x * s;
      f[2 * i + 1] = p.y * s;
    }
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(cache) + vec * LPV + c);
    const float s = int4_scale(__ldg(scale + vec * (LPV / 4) + (c >> 2)));
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - 8) * s;
  }
}

// Blocks (x: sequence and head, y: pages of the sequence that hold new tokens, in turn).
constexpr int kBoundThreads = 128;
template <int D, int BF16, int KIND>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const BoundsArgs a) {
  constexpr int LPV = D / 8, RPB = kBoundThreads / LPV, W = kBoundThreads / 32;
  __shared__ float s_hi[W][D], s_lo[W][D];
  const int s = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  int first;
  const int n = seq_tokens(a.cu, s, a.T, &first);
  const int page_log2 = 31 - __clz(a.page);
  const int len = seq_positions(a.kv_lens, s, static_cast<long long>(a.max_pages) << page_log2);
  if (n == 0 || len == 0) return;
  const int p0 = max(seq_first_position(a.kv_lens, s, n), 0) >> page_log2, p1 = (len - 1) >> page_log2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = threadIdx.x % LPV;
  for (int p = p0 + static_cast<int>(blockIdx.y); p <= p1; p += static_cast<int>(gridDim.y)) {
    const int pg = __ldg(a.table + static_cast<long long>(s) * a.max_pages + p);
    if (pg < 0 || pg >= a.n_pages) continue;  // (the same for the whole block)
    const int slots = min(a.page, len - (p << page_log2));
    // Of sequences that share the page and whose new tokens are in it, the one that fills it furthest writes its bounds (equal ones write the same). Every block
    // looks through all sequences: a step of 48 takes 4.0 us in place of 3.4, of 300 8.5 and 7.1, of 3,000 121 and 51.
    if (slots < a.page && a.n_seqs > 1) {
      bool further = false;
      constexpr int AT_ONCE = 4;  // (lengths whose loads are in flight together)
      for (int o0 = threadIdx.x; o0 < a.n_seqs; o0 += AT_ONCE * kBoundThreads) {
        int l[AT_ONCE], c0[AT_ONCE], c1[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          const int o = min(o0 + u * kBoundThreads, a.n_seqs - 1);
          l[u] = __ldg(a.kv_lens + o);
          c0[u] = cu_at(a.cu, o, a.T);
          c1[u] = cu_at(a.cu, o + 1, a.T);
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
          const int o = min(o0 + u * kBoundThreads, a.n_seqs - 1);
          if (l[u] > len && c1[u] > c0[u] && l[u] - (c1[u] - c0[u]) < (p + 1) << page_log2)
            further |= __ldg(a.table + static_cast<long long>(o) * a.max_pages + p) == pg;
        }
      }
      if (__syncthreads_or(further)) continue;
    }
    const long long block = static_cast<long long>(pg) * a.Hkv + h;
    float hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = -INFINITY;
      lo[i] = INFINITY;
    }
    bool odd = false;  // a key that is not finite
#pragma unroll 4
    for (int r = threadIdx.x / LPV; r < slots; r += RPB) {
      float f[8];
      cached8<D, BF16, KIND>(static_cast<const uint8_t*>(a.k_cache), a.k_scale, (block << page_log2) + r, c, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        odd |= !(fabsf(f[i]) < INFINITY);
        hi[i] = fmaxf(hi[i], f[i]);
        lo[i] = fminf(lo[i], f[i]);
      }
    }
#pragma unroll
    for (int o = LPV; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
        lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      }
    if (lane < LPV) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_hi[warp][c * 8 + i] = hi[i];
        s_lo[warp][c * 8 + i] = lo[i];
      }
    }
    const bool any = __syncthreads_or(odd);
    if (warp == 0) {
      // lane l takes D / 32 neighbouring features
      constexpr int F = D / 32;
      float top = 0.0f;
      float x[2][F];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        x[0][i] = -INFINITY;
        x[1][i] = INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          x[0][i] = fmaxf(x[0][i], s_hi[w][lane * F + i]);
          x[1][i] = fminf(x[1][i], s_lo[w][lane * F + i]);
        }
        top = fmaxf(top, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = any ? 0 : bound_exponent(top);
      const float inv = pow2i(-e);
      signed char* to = a.bounds + block * (2 * D) + lane * F;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < F; ++i) to[u * D + i] = any ? 0 : static_cast<signed char>(__float2int_rn(x[u][i] * inv));
      if (lane == 0) a.exps[block] = any ? 255 : static_cast<unsigned char>(e + 127);
    }
    __syncthreads();
  }
}

// Token `token`'s sequence and position (a whole warp); position -1 for a token of no sequence or before the first position, the
// table's last for one behind it.
__device__ __forceinline__ void token_position(const SelectArgs& a, int token, int lane, int* seq, int* pos) {
  const int s = seq_of_token(a.cu, a.n_seqs, a.T, token, lane);
  *seq = s;
  *pos = -1;
  if (s < 0) return;
  int first;
  const int n = seq_tokens(a.cu, s, a.T, &first);
  *pos = max(min(seq_first_position(a.kv_lens, s, n) + (token - first), a.max_pages * a.page - 1), -1);
}

// Scores of pages for some tokens of a sequence and a key head, on the tensor cores (`splits` blocks take kScorePages pages each in turn): 16 pages x (largest | smallest keys), whole
// numbers that fp16 holds exactly, times (positive | negative parts) of 8 rows' queries; sums stay below 2^22, exact in fp32 in any
// order. A token's heads are padded to a power of two `gp` of rows, so that its maximum is one over neighbouring columns. The order of
// the features along the products is the one in which a lane reads 16 bytes of bounds and 32 of queries. Scores are written for
// the pages before a token's own.
constexpr int kScoreThreads = 256, kScorePages = kScoreThreads / 32 * 16, kScoreRows = 64;
__device__ __forceinline__ void product16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two whole numbers of 8 bits (already moved to 0 .. 255) as fp16 numbers.
__device__ __forceinline__ uint32_t whole2(uint32_t w, uint32_t order) {
  const uint32_t x = __byte_perm(w, 0x64646464u, order);  // 1024 + byte
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(-1152.0f, -1152.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ONE: a single tile of 8 rows (single tokens of up to 8 heads), whose fragments need not be kept from one tile of rows to the next.
template <int D, int BF16, bool ONE>
__global__ void __launch_bounds__(kScoreThreads, ONE ? 4 : 2) score_kernel(const SelectArgs a, int token0, int tokens, int at_once, int gp, int splits) {
  constexpr int J = D / 32, LDQ = 2 * D + 8;  // pieces of 16 features that a lane reads of a page, row of the queries
  constexpr int ROWS = ONE ? 8 : kScoreRows;
  __shared__ __align__(16) uint16_t s_q[ROWS * LDQ];
  __shared__ float s_f[ROWS], s_add[ROWS];
  __shared__ int s_e[ROWS];
  const int unit = static_cast<int>(blockIdx.x / splits), base = static_cast<int>(blockIdx.x % splits) * kScorePages;
  const int h = unit % a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int page_log2 = 31 - __clz(a.page), last = min(token0 + (unit / a.Hkv + 1) * at_once, token0 + tokens);
  for (int token = token0 + unit / a.Hkv * at_once; token < last;) {
    // the tokens of one sequence from `token` on (every warp looks for itself: what follows then waits for nobody)
    const int s = seq_of_token(a.cu, a.n_seqs, a.T, token, lane);
    int first = 0, n = 0, pos0 = 0, ns;  // pos0: the first one's position
    if (s >= 0) {
      n = seq_tokens(a.cu, s, a.T, &first);
      pos0 = seq_first_position(a.kv_lens, s, n) + (token - first);
      ns = min(first + n, last) - token;
    } else {
      ns = (token < cu_at(a.cu, 0, a.T) ? min(cu_at(a.cu, 0, a.T), last) : last) - token;
    }
    // pages before the last of them (a token behind the table stands in its last page)
    const int P = s < 0 || pos0 + ns <= 0 ? 0 : min(min(pos0 + ns - 1, a.max_pages * a.page - 1) >> page_log2, a.most_pages);
    if (base >= P) {  // (the same for the whole block)
      token += ns;
      continue;
    }
    const int* row = a.table + static_cast<long long>(s) * a.max_pages;
    const int stride = splits * kScorePages;
    uint4 x[2][J];  // the bounds of pages p0 + g and p0 + 8 + g: fetched a step ahead, the first before the queries are ready
    int ek[2];
    auto fetch = [&](int p0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const long long blk = static_cast<long long>(page_at(row, min(p0 + 8 * u + g, P - 1), a.n_pages)) * a.Hkv + h;
        const uint4* at = reinterpret_cast<const uint4*>(a.bounds + blk * (2 * D)) + t4;
#pragma unroll
        for (int j = 0; j < J; ++j) x[u][j] = __ldg(at + 4 * j);
        ek[u] = __ldg(a.exps + blk);
      }
    };
    if (base + warp * 16 < P) fetch(base + warp * 16);
    // the queries as whole numbers, positive and negative parts apart; rows without a head are zeros whose scores do not count
    const int rows = (ns * gp + 7) & ~7;
    constexpr int F = D / 32, RA = ONE ? 1 : 4, RS = kScoreThreads / 32;  // features of a lane; rows whose loads go out together, and their distance
    for (int r0 = warp; r0 < rows; r0 += RA * RS) {
      float f[RA][F], top[RA];
#pragma unroll
      for (int u = 0; u < RA; ++u) {
        const int r = r0 + u * RS, i = r / gp, head = r - i * gp;
        const uint16_t* q = static_cast<const uint16_t*>(a.q) + static_cast<long long>(token + i) * a.q_stride + static_cast<long long>(h * a.G + head) * D + lane * F;
#pragma unroll
        for (int e = 0; e < F; e += 2) {
          const float2 p = unpack16(r < rows && i < ns && head < a.G ? __ldg(reinterpret_cast<const uint32_t*>(q + e)) : 0u, BF16);
          f[u][e] = p.x;
          f[u][e + 1] = p.y;
        }
      }
#pragma unroll
      for (int u = 0; u < RA; ++u) {
        top[u] = 0.0f;
#pragma unroll
        for (int e = 0; e < F; ++e) {
          if (!(fabsf(f[u][e]) < INFINITY)) f[u][e] = 0.0f;  // (its row is not a number whatever it attends to)
          top[u] = fmaxf(top[u], fabsf(f[u][e]));
        }
        top[u] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top[u])));  // (bits of numbers from 0 on are in order)
      }
#pragma unroll
      for (int u = 0; u < RA; ++u) {
        const int r = r0 + u * RS, i = r / gp, head = r - i * gp;
        if (r >= rows) break;
        const bool real = i < ns && head < a.G;
        const int ex = bound_exponent(top[u]);
        const float inv = pow2i(-ex);
        uint16_t* to = s_q + r * LDQ + lane * F;
#pragma unroll
        for (int e = 0; e < F; e += 2) {
          const float v0 = rintf(f[u][e] * inv), v1 = rintf(f[u][e + 1] * inv);
          *reinterpret_cast<uint32_t*>(to + e) = pack16(fmaxf(v0, 0.0f), fmaxf(v1, 0.0f), 0);
          *reinterpret_cast<uint32_t*>(to + D + e) = pack16(fminf(v0, 0.0f), fminf(v1, 0.0f), 0);
        }
        if (lane == 0) {
          s_e[r] = real ? ex : -100000;
          s_add[r] = real ? 0.0f : -INFINITY;
        }
      }
    }
    __syncthreads();
    // a head's power of two relative to the largest of its token's heads
    for (int r = threadIdx.x; r < rows; r += kScoreThreads) {
      const int r0 = r / gp * gp;
      int top = -100000;
      for (int i = r0; i < min(r0 + gp, rows); ++i) top = max(top, s_e[i]);
      const int k = s_e[r] - top;
      s_f[r] = k < -126 ? 0.0f : pow2i(k);
    }
    __syncthreads();
    for (int p0 = base + warp * 16; p0 < P; p0 += stride) {
      // 16 features of two pages as four products' fragments
      auto fragments = [&](int j, uint32_t (&fr)[4][4]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t w[4] = {x[u][j].x, x[u][j].y, x[u][j].z, x[u][j].w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t y = w[m] ^ 0x80808080u;
            fr[m][u] = whole2(y, 0x4140);
            fr[m][2 + u] = whole2(y, 0x4342);
          }
        }
      };
      auto multiply = [&](float (&c)[4], const uint32_t (&fr)[4][4], int n0, int j) {
        const uint4* b = reinterpret_cast<const uint4*>(s_q + (n0 + g) * LDQ) + 2 * t4 + 8 * j;
        const uint4 lo = b[0], hi = b[1];
        product16816(c, fr[0], lo.x, lo.y);
        product16816(c, fr[1], lo.z, lo.w);
        product16816(c, fr[2], hi.x, hi.y);
        product16816(c, fr[3], hi.z, hi.w);
      };
      uint32_t kept[ONE ? 1 : J][4][4];
      float c1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < J; ++j) {
        fragments(j, kept[ONE ? 0 : j]);
        if (ONE) multiply(c1, kept[0], 0, j);
      }
      const bool odd0 = ek[0] == 255, odd1 = ek[1] == 255;
      const float unit0 = odd0 ? 0.0f : pow2i(ek[0] - 127), unit1 = odd1 ? 0.0f : pow2i(ek[1] - 127);
      if (p0 + stride < P) fetch(p0 + stride);
      float best[2] = {-INFINITY, -INFINITY};
      for (int n0 = 0; n0 < (ONE ? 1 : rows); n0 += 8) {
        float c[4] = {c1[0], c1[1], c1[2], c1[3]};
        if (!ONE) {
#pragma unroll
          for (int j = 0; j < J; ++j) multiply(c, kept[j], n0, j);
        }
        const float2 f = *reinterpret_cast<const float2*>(s_f + n0 + 2 * t4), add = *reinterpret_cast<const float2*>(s_add + n0 + 2 * t4);
        const float v[2][2] = {{c[0] * f.x + add.x, c[1] * f.y + add.y}, {c[2] * f.x + add.x, c[3] * f.y + add.y}};
        auto put = [&](int i, const float (&w)[2]) {  // token i of the segment, pages g and g + 8
          const int own = min((pos0 + i) >> page_log2, P);
          float* out = a.scores + (static_cast<long long>(token - token0 + i) * a.Hkv + h) * a.most_pages;
          if (i < ns && pos0 + i >= 0) {  // (a page that is not finite comes first; + 0: no -0)
            if (p0 + g < own) out[p0 + g] = odd0 ? INFINITY : w[0] * unit0 + 0.0f;
            if (p0 + 8 + g < own) out[p0 + 8 + g] = odd1 ? INFINITY : w[1] * unit1 + 0.0f;
          }
        };
        if (gp == 1) {
          const float w0[2] = {v[0][0], v[1][0]}, w1[2] = {v[0][1], v[1][1]};
          put(n0 + 2 * t4, w0);
          put(n0 + 2 * t4 + 1, w1);
          continue;
        }
        float w[2] = {fmaxf(v[0][0], v[0][1]), fmaxf(v[1][0], v[1][1])};
        for (int o = 1; 2 * o < min(gp, 8); o <<= 1)
#pragma unroll
          for (int u = 0; u < 2; ++u) w[u] = fmaxf(w[u], __shfl_xor_sync(0xffffffffu, w[u], o));
        if (gp <= 8) {
          if ((2 * t4 & (gp - 1)) == 0) put((n0 + 2 * t4) / gp, w);
          continue;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) best[u] = fmaxf(best[u], w[u]);
        if ((n0 + 8) % gp == 0) {
          if (t4 == 0) put(n0 / gp, best);
          best[0] = best[1] = -INFINITY;
        }
      }
    }
    token += ns;
    __syncthreads();
  }
}

// A score as a whole number of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What a block of the selection works on: a token and key head. Writes, for the first key head, the token as a sequence of its own.
struct Choice {
  int seq, pos, page_log2, pages, take;  // pages before the token's own, and how many of them are chosen
};
__device__ __forceinline__ Choice choice_of(const SelectArgs& a, int token, int h, int (&s_at)[2]) {
  if (threadIdx.x < 32) {
    int s, pos;
    token_position(a, token, threadIdx.x, &s, &pos);
    if (threadIdx.x == 0) {
      s_at[0] = s;
      s_at[1] = pos;
    }
  }
  __syncthreads();
  Choice c;
  c.seq = s_at[0];
  c.pos = s_at[1];
  c.page_log2 = 31 - __clz(a.page);
  c.pages = c.pos < 0 ? 0 : min(c.pos >> c.page_log2, a.most_pages);
  c.take = min(a.n_select - 1, c.pages);
  if (h == 0 && threadIdx.x == 0) {
    const int c0 = cu_at(a.cu, 0, a.T), c1 = cu_at(a.cu, a.n_seqs, a.T);
    a.cu_out[token] = min(max(token, c0), c1);
    if (token == a.T - 1) a.cu_out[a.T] = min(max(a.T, c0), c1);
    a.lens_out[token] = c.pos < 0 ? 0 : (c.take << c.page_log2) + (c.pos & (a.page - 1)) + 1;
  }
  return c;
}

// The block's list of chosen pages, indices into the token's row of the table until here, as the user's list and as pages of the cache; behind them
// the token's own page, and nothing.
__device__ __forceinline__ void finish_list(const SelectArgs& a, const Choice& c, const int* row, int* pages, int* list) {
  __syncthreads();
  for (int i = threadIdx.x; i < a.n_select; i += blockDim.x) {
    const int p = i < c.take ? list[i] : (i == c.take && c.pos >= 0 ? c.pos >> c.page_log2 : -1);
    if (pages) pages[i] = p;
    list[i] = p >= 0 ? page_at(row, p, a.n_pages) : 0;
  }
}

// Scores that shared memory holds: the k-th largest is found two bits at a time by counting, which ends as soon as a bound separates just k
// (after some ten rounds mostly). Threads and warps take what pages there are, not as many as the longest sequence has.
constexpr int kFewThreads = 256, kFewPages = 16384;
__global__ void __launch_bounds__(kFewThreads) select_few_kernel(const SelectArgs a, int token0) {
  constexpr int W = kFewThreads / 32;
  extern __shared__ uint32_t s_x[];
  __shared__ int s_at[2], s_count[2][W][2], s_gt[W], s_eq[W];
  const int unit = static_cast<int>(blockIdx.x), token = token0 + unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Choice c = choice_of(a, token, h, s_at);
  if (c.seq < 0) return;  // behind the last sequence: left as it was
  const int P = c.pages, k = c.take;
  int* pages = a.pages ? a.pages + (static_cast<long long>(token) * a.Hkv + h) * a.n_select : nullptr;
  int* list = a.list + (static_cast<long long>(token) * a.Hkv + h) * a.n_select;
  const int* row = a.table + static_cast<long long>(c.seq) * a.max_pages;
  if (k > 0) {
    const float* score = a.scores + static_cast<long long>(unit) * a.most_pages;
    // `least`: more than it are chosen, and of its equals the first `equals`
    uint32_t least = 0, hi = 0, lo = 0xffffffffu;
    int equals = 0;
#pragma unroll 4
    for (int i = tid; i < P; i += kFewThreads) {
      const uint32_t x = ordered(__ldcg(score + i));
      s_x[i] = x;
      hi = max(hi, x);
      lo = min(lo, x);
    }
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo = __reduce_min_sync(0xffffffffu, lo);
    if (lane == 0) {
      s_count[1][warp][0] = static_cast<int>(hi);
      s_count[1][warp][1] = static_cast<int>(lo);
    }
    __syncthreads();
    if (k < P) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        hi = max(hi, static_cast<uint32_t>(s_count[1][w][0]));
        lo = min(lo, static_cast<uint32_t>(s_count[1][w][1]));
      }
      // what the largest and the smallest score have in common all have
      const int first = (31 - __clz(static_cast<int>((hi ^ lo) | 1u))) & ~1;
      uint32_t known = first == 30 ? 0u : hi & ~((4u << first) - 1u);  // the k-th largest is at least this
      bool exact = false;
      int buf = 0;
#pragma unroll 1
      for (int shift = first; shift >= 0; shift -= 2) {
        const uint32_t b1 = known + (1u << shift), b2 = known + (2u << shift), b3 = known + (3u << shift);
        int n1 = 0, n2 = 0, n3 = 0;
#pragma unroll 4
        for (int i = tid; i < P; i += kFewThreads) {
          const uint32_t x = s_x[i];
          n1 += x >= b1;
          n2 += x >= b2;
          n3 += x >= b3;
        }
        const int both = __reduce_add_sync(0xffffffffu, n1 | n2 << 16);  // (below 2^14 each)
        n3 = __reduce_add_sync(0xffffffffu, n3);
        if (lane == 0) {
          s_count[buf][warp][0] = both;
          s_count[buf][warp][1] = n3;
        }
        __syncthreads();
        n1 = n2 = n3 = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int v = s_count[buf][w][0];
          n1 += v & 0xffff;
          n2 += v >> 16;
          n3 += s_count[buf][w][1];
        }
        buf ^= 1;
        const int step = n3 >= k ? 3 : (n2 >= k ? 2 : (n1 >= k ? 1 : 0));
        known += static_cast<uint32_t>(step) << shift;
        if ((step == 3 && n3 == k) || (step == 2 && n2 == k) || (step == 1 && n1 == k)) {
          exact = true;
          break;
        }
      }
      least = exact ? known - 1 : known;  // (a bound that separates k of more is not 0)
      if (!exact) equals = P;             // as many as there is room for
    }
    // chosen pages in ascending order: a warp takes a run of them, counts, and writes from where the runs before it end
    const int run = ((P + W - 1) / W + 31) & ~31, i0 = warp * run;
    int gt = 0, eq = 0;
    for (int i = i0 + lane; i < i0 + run; i += 32) {
      const uint32_t x = i < P ? s_x[i] : 0u;  // (a score is never 0 here)
      gt += __popc(__ballot_sync(0xffffffffu, x > least));
      eq += __popc(__ballot_sync(0xffffffffu, x == least && x != 0u));
    }
    if (lane == 0) {
      s_gt[warp] = gt;
      s_eq[warp] = eq;
    }
    __syncthreads();
    int above = 0, at = 0, eq_before = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) above += s_gt[w];
    if (equals) equals = k - above;
    for (int w = 0; w < warp; ++w) {
      at += s_gt[w] + min(s_eq[w], max(equals - eq_before, 0));
      eq_before += s_eq[w];
    }
    for (int i = i0 + lane; i < i0 + run; i += 32) {
      const uint32_t x = i < P ? s_x[i] : 0u;
      const bool is_eq = x == least && x != 0u;
      const unsigned be = __ballot_sync(0xffffffffu, is_eq), below = (1u << lane) - 1u;
      const bool take = x > least || (is_eq && eq_before + __popc(be & below) < equals);
      const unsigned bt = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int to = at + __popc(bt & below);
        if (to < k) list[to] = i;
      }
      at += __popc(bt);
      eq_before += __popc(be);
    }
  }
  finish_list(a, c, row, pages, list);
}

// Any number of pages: the k-th largest score by counts of its upper, middle and lower bits in shared memory.
constexpr int kSelectThreads = 512, kBins = 2048;
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectArgs a, int token0) {
  constexpr int W = kSelectThreads / 32, BPT = kBins / kSelectThreads;
  __shared__ int s_bins[kBins];
  __shared__ int s_at[2], s_part[W], s_gt[W], s_eq[W];
  __shared__ uint32_t s_found[2];
  const int unit = static_cast<int>(blockIdx.x), token = token0 + unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Choice c = choice_of(a, token, h, s_at);
  const int s = c.seq, P = c.pages, k = c.take;
  if (s < 0) return;  // behind the last sequence: left as it was
  const float* score = a.scores + static_cast<long long>(unit) * a.most_pages;
  uint32_t least = 0;  // the k-th largest score, and how many of its equals are taken
  int equals = P;
  if (k > 0 && k < P) {
    uint32_t known = 0;
    int need = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      for (int i = tid; i < kBins; i += kSelectThreads) s_bins[i] = 0;
      __syncthreads();
      for (int i = tid; i < P; i += kSelectThreads) {
        const uint32_t x = ordered(__ldcg(score + i));
        const bool in = pass == 0 || ((x ^ known) >> (pass == 1 ? 21 : 10)) == 0;
        if (in) atomicAdd(&s_bins[(x >> shift) & (pass == 2 ? 1023u : 2047u)], 1);
      }
      __syncthreads();
      // thread t holds bins from the top: t * BPT and on, counted from the last bin down
      int mine[BPT], sum = 0;
#pragma unroll
      for (int i = 0; i < BPT; ++i) {
        mine[i] = s_bins[kBins - 1 - (tid * BPT + i)];
        sum += mine[i];
      }
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_part[warp] = x;
      __syncthreads();
      int before = x - sum;
      for (int i = 0; i < warp; ++i) before += s_part[i];
#pragma unroll
      for (int i = 0; i < BPT; ++i) {
        if (before < need && need <= before + mine[i]) {
          s_found[0] = static_cast<uint32_t>(kBins - 1 - (tid * BPT + i));
          s_found[1] = static_cast<uint32_t>(need - before);
        }
        before += mine[i];
      }
      __syncthreads();
      known |= s_found[0] << shift;
      need = static_cast<int>(s_found[1]);
      __syncthreads();
    }
    least = known;
    equals = need;
  }
  int* pages = a.pages ? a.pages + (static_cast<long long>(token) * a.Hkv + h) * a.n_select : nullptr;
  int* list = a.list + (static_cast<long long>(token) * a.Hkv + h) * a.n_select;
  const int* row = a.table + static_cast<long long>(s) * a.max_pages;
  // chosen pages in ascending order: a warp takes a run of them, counts, and writes from where the runs before it end
  if (k > 0) {
    const int run = ((P + W - 1) / W + 31) & ~31, i0 = warp * run, i1 = min(i0 + run, P);
    int gt = 0, eq = 0;
    for (int i = i0 + lane; i < i0 + run; i += 32) {
      const uint32_t x = i < i1 ? ordered(__ldcg(score + i)) : 0u;
      gt += __popc(__ballot_sync(0xffffffffu, i < i1 && x > least));
      eq += __popc(__ballot_sync(0xffffffffu, i < i1 && x == least));
    }
    if (lane == 0) {
      s_gt[warp] = gt;
      s_eq[warp] = eq;
    }
    __syncthreads();
    int at = 0, eq_before = 0;
    for (int i = 0; i < warp; ++i) {
      at += s_gt[i] + min(s_eq[i], max(equals - eq_before, 0));
      eq_before += s_eq[i];
    }
    for (int i = i0 + lane; i < i0 + run; i += 32) {
      const uint32_t x = i < i1 ? ordered(__ldcg(score + i)) : 0u;
      const bool is_eq = i < i1 && x == least;
      const unsigned be = __ballot_sync(0xffffffffu, is_eq), below = (1u << lane) - 1u;
      const bool take = (i < i1 && x > least) || (is_eq && eq_before + __popc(be & below) < equals);
      const unsigned bt = __ballot_sync(0xffffffffu, take);
      if (take) {
        const int to = at + __popc(bt & below);
        if (to < k) list[to] = i;
      }
      at += __popc(bt);
      eq_before += __popc(be);
    }
  }
  finish_list(a, c, row, pages, list);
}

template <int D, int BF16>
int launch_bounds_d(const BoundsArgs& a, dim3 grid, cudaStream_t stream) {
  if (a.cache_dtype == CQSA_E4M3) bounds_kernel<D, BF16, kCacheE4m3><<<grid, kBoundThreads, 0, stream>>>(a);
  else if (a.cache_dtype == CQSA_INT4) bounds_kernel<D, BF16, kCacheInt4><<<grid, kBoundThreads, 0, stream>>>(a);
  else bounds_kernel<D, BF16, kCacheSame><<<grid, kBoundThreads, 0, stream>>>(a);
  return cuda_status(cudaGetLastError(), "page bounds kernel launch");
}

template <bool ONE>
int launch_scores(const SelectArgs& a, int token0, int tokens, int at_once, int gp, cudaStream_t stream) {
  // Blocks for so many a SM, whatever the longest sequence is: in a ragged batch most are far shorter. (48 sequences of 1,000,000 positions in pages of
  // 32 together, the whole call: 94 us with 4, 73 with 8, 71 with 12, 77 with 40. Blocks of several tiles of rows begin with more work: 46 us with 4 and 49
  // with 8 for 60 tokens over 400,000 positions, 56 and 63 at 32 and 8 heads of 128. Otherwise 1 to 128 sequences
  // of 1 to 1,000 tokens differ by 3% at most between 2 and 40, 48 ragged ones of d = 128 by 8%: 51 us with 8, 52 with 12, 55 with 24.)
  const long long units = (tokens + at_once - 1LL) / at_once * a.Hkv, most = (a.most_pages + kScorePages - 1) / kScorePages;
  const long long want = static_cast<long long>(ONE ? 12 : 4) * sm_count() / units;
  const int splits = static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
  if (units * splits > 0x7fffffffLL) {
    set_error("selection is too large for one launch (%lld blocks)", units * splits);
    return CQSA_ERR_UNSUPPORTED;
  }
  const unsigned grid = static_cast<unsigned>(units * splits);
  const bool bf = a.dtype == CQSA_BF16;
  if (a.d == 64 && bf) score_kernel<64, 1, ONE><<<grid, kScoreThreads, 0, stream>>>(a, token0, tokens, at_once, gp, splits);
  else if (a.d == 64) score_kernel<64, 0, ONE><<<grid, kScoreThreads, 0, stream>>>(a, token0, tokens, at_once, gp, splits);
  else if (bf) score_kernel<128, 1, ONE><<<grid, kScoreThreads, 0, stream>>>(a, token0, tokens, at_once, gp, splits);
  else score_kernel<128, 0, ONE><<<grid, kScoreThreads, 0, stream>>>(a, token0, tokens, at_once, gp, splits);
  return cuda_status(cudaGetLastError(), "page score kernel launch");
}

// Tokens whose scores are held at a time: 64 MiB of them, one token's at least.
int score_tokens(const SelectArgs& a) {
  const long long per = static_cast<long long>(a.Hkv) * a.most_pages * 4, n = (64LL << 20) / per;
  return static_cast<int>(n < 1 ? 1 : (n < a.T ? n : a.T));
}

}  // namespace

int launch_page_bounds(const BoundsArgs& a, int max_q_len, cudaStream_t stream) {
  const long long x = static_cast<long long>(a.n_seqs) * a.Hkv;
  if (x > 0x7fffffffLL) {
    set_error("n_seqs * Hkv = %lld is too large (2^31 - 1 at most)", x);
    return CQSA_ERR_UNSUPPORTED;
  }
  const long long most = (static_cast<long long>(max_q_len < a.T ? max_q_len : a.T) + a.page - 1) / a.page + 1;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(most < 1 ? 1 : (most < 1024 ? most : 1024)));
  const bool bf = a.dtype == CQSA_BF16;
  if (a.d == 64) return bf ? launch_bounds_d<64, 1>(a, grid, stream) : launch_bounds_d<64, 0>(a, grid, stream);
  return bf ? launch_bounds_d<128, 1>(a, grid, stream) : launch_bounds_d<128, 0>(a, grid, stream);
}

size_t select_workspace(const SelectArgs& a) {
  const size_t scores = static_cast<size_t>(score_tokens(a)) * a.Hkv * a.most_pages * 4;
  const size_t lists = static_cast<size_t>(a.T) * a.Hkv * a.n_select * 4, ints = (2 * static_cast<size_t>(a.T) + 1) * 4;
  return ((scores + 255) & ~size_t(255)) + ((lists + 255) & ~size_t(255)) + ((ints + 255) & ~size_t(255));
}

int launch_select(SelectArgs* args, cudaStream_t stream) {
  SelectArgs& a = *args;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const int at_once = score_tokens(a);
  a.scores = reinterpret_cast<float*>(ws);
  ws += (static_cast<size_t>(at_once) * a.Hkv * a.most_pages * 4 + 255) & ~size_t(255);
  a.list = reinterpret_cast<int*>(ws);
  ws += (static_cast<size_t>(a.T) * a.Hkv * a.n_select * 4 + 255) & ~size_t(255);
  a.cu_out = reinterpret_cast<int*>(ws);
  a.lens_out = a.cu_out + a.T + 1;
  // tokens of a block of scores: as many as a sequence has on average, which share the reading of its bounds, in 64 rows at most
  const bool few = a.most_pages <= kFewPages;
  if (few && a.most_pages > 11 * 1024) {  // beyond the 48 KiB (with the kernel's own) that every kernel may use
    static PerDeviceOnce attr;
    int dev = 0;
    if (!attr.done(&dev)) {
      const cudaError_t e = cudaFuncSetAttribute(select_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewPages * 4);
      if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(page selection smem)");
      attr.mark(dev);
    }
  }
  int gp = 1, block_tokens = 1;
  while (gp < a.G) gp *= 2;
  while (block_tokens <= (a.T - 1) / a.n_seqs && 2 * block_tokens * gp <= kScoreRows) block_tokens *= 2;
  for (int t = 0; t < a.T; t += at_once) {
    const int n = a.T - t < at_once ? a.T - t : at_once;
    if (a.n_select > 1) {
      const int rc = block_tokens * gp <= 8 ? launch_scores<true>(a, t, n, block_tokens, gp, stream)
                                            : launch_scores<false>(a, t, n, block_tokens, gp, stream);
      if (rc != CQSA_OK) return rc;
    }
    const unsigned units = static_cast<unsigned>(static_cast<long long>(n) * a.Hkv);
    if (few) select_few_kernel<<<units, kFewThreads, static_cast<unsigned>(a.most_pages) * 4, stream>>>(a, t);
    else select_kernel<<<units, kSelectThreads, 0, stream>>>(a, t);
    const int rc = cuda_status(cudaGetLastError(), "page selection kernel launch");
    if (rc != CQSA_OK) return rc;
  }
  return CQSA_OK;
}

}  // namespace cqsa
