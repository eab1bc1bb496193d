// Attention of each new token over a few pages of its sequence, selected by a score that reads a page's bounds instead of its keys.
//
// Bounds: for a page and key head, the largest and the smallest key of each feature as whole multiples (8 bits) of the smallest power of two
// under which all lie within 127: 2 d + 1 bytes, against the page's 512 a slot in 16 bits at d = 128. Queries likewise, a power of two for each
// vector. The score of a page for a token and key head is max over the group's heads of sum_f max(q_f hi_f, q_f lo_f): but for the roundings an
// upper bound of the page's dot products. The sums are whole numbers below 2^21 and are scaled by powers of two, so every order of summation
// gives the same score and every run and program the same choice.
//
// Three kernels before the attention: bounds_kernel (a block per page and head that new tokens came into), score_kernel (d / 16 lanes read a page's
// two vectors, 16 bytes each; dp4a against the group's queries in shared memory, positive parts with the largest, negative ones with the
// smallest keys; four pages a lane at a time, so that a query's words are read once for them and their sums are added up across the lanes
// in four exchanges) and select_kernel (a block per token and head: the n-th largest score by a count of its upper, middle and lower bits, then
// the pages from there on up in ascending order, equal scores first come). The attention itself is attn_decode.cu's and attn_decode4.cu's: each
// token is a sequence of its own whose table, one for each key head, lists the pages chosen, its own page last, so that only the end of
// the last page is masked.
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
  const int p0 = max(len - n, 0) >> page_log2, p1 = (len - 1) >> page_log2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = threadIdx.x % LPV;
  for (int p = p0 + static_cast<int>(blockIdx.y); p <= p1; p += static_cast<int>(gridDim.y)) {
    const int pg = __ldg(a.table + static_cast<long long>(s) * a.max_pages + p);
    if (pg < 0 || pg >= a.n_pages) continue;  // (the same for the whole block)
    const int slots = min(a.page, len - (p << page_log2));
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

// Token `token`'s sequence and position (a whole warp); position -1 for a token of no sequence or before the first position.
__device__ __forceinline__ void token_position(const SelectArgs& a, int token, int lane, int* seq, int* pos) {
  const int s = seq_of_token(a.cu, a.n_seqs, a.T, token, lane);
  *seq = s;
  *pos = -1;
  if (s < 0) return;
  int first;
  const int n = seq_tokens(a.cu, s, a.T, &first);
  const int len = seq_positions(a.kv_lens, s, static_cast<long long>(a.max_pages) * a.page);
  *pos = max(len - n + (token - first), -1);
}

// Scores of kScorePages pages for a token and key head. Scores are written for the pages before the token's own.
constexpr int kScoreThreads = 256, kScorePages = 256, kMostHeads = 32;
template <int D, int BF16>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectArgs a, int token0) {
  constexpr int LP = D / 16, GROUPS = 32 / LP, STEP = 4 * GROUPS;  // lanes of a page; pages side by side, and of a warp's step
  __shared__ uint4 s_q[kMostHeads][2][LP];
  __shared__ int s_e[kMostHeads];
  __shared__ int s_at[2];
  const int splits = (a.most_pages + kScorePages - 1) / kScorePages;
  const int unit = static_cast<int>(blockIdx.x / splits), base = static_cast<int>(blockIdx.x % splits) * kScorePages;
  const int token = token0 + unit / a.Hkv, h = unit % a.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    int s, pos;
    token_position(a, token, lane, &s, &pos);
    if (lane == 0) {
      s_at[0] = s;
      s_at[1] = pos;
    }
  }
  __syncthreads();
  const int page_log2 = 31 - __clz(a.page);
  const int P = s_at[1] < 0 ? 0 : min(s_at[1] >> page_log2, a.most_pages);
  if (base >= P) return;
  // the group's queries as whole numbers, positive and negative parts apart
  for (int g = warp; g < a.G; g += kScoreThreads / 32) {
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + static_cast<long long>(token) * a.q_stride + static_cast<long long>(h * a.G + g) * D;
    uint2 x = make_uint2(0, 0);
    if (lane < D / 4) x = __ldg(reinterpret_cast<const uint2*>(q) + lane);
    const float2 lo = unpack16(x.x, BF16), hi = unpack16(x.y, BF16);
    float f[4] = {lo.x, lo.y, hi.x, hi.y}, top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!(fabsf(f[i]) < INFINITY)) f[i] = 0.0f;  // (its row is not a number whatever it attends to)
      top = fmaxf(top, fabsf(f[i]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = bound_exponent(top);
    const float inv = pow2i(-e);
    uint32_t up = 0, down = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = __float2int_rn(f[i] * inv);
      up |= static_cast<uint32_t>(max(v, 0)) << (8 * i);
      down |= (static_cast<uint32_t>(min(v, 0)) & 255u) << (8 * i);
    }
    if (lane < D / 4) {
      reinterpret_cast<uint32_t*>(&s_q[g][0][0])[lane] = up;
      reinterpret_cast<uint32_t*>(&s_q[g][1][0])[lane] = down;
    }
    if (lane == 0) s_e[g] = e;
  }
  __syncthreads();
  int etop = s_e[0];
  for (int g = 1; g < a.G; ++g) etop = max(etop, s_e[g]);
  const int c = lane % LP;
  const int* row = a.table + static_cast<long long>(s_at[0]) * a.max_pages;
  float* out = a.scores + static_cast<long long>(unit) * a.most_pages;
  for (int p0 = base + warp * STEP; p0 < min(base + kScorePages, P); p0 += kScoreThreads / 32 * STEP) {
    uint4 hi[4], lo[4];
    long long blk[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int p = min(p0 + u * GROUPS + lane / LP, P - 1);
      blk[u] = static_cast<long long>(page_at(row, p, a.n_pages)) * a.Hkv + h;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4* at = reinterpret_cast<const uint4*>(a.bounds + blk[u] * (2 * D));
      hi[u] = __ldg(at + c);
      lo[u] = __ldg(at + LP + c);
    }
    // lane c ends up with page c % 4 of its group
    const long long mine = c & 2 ? (c & 1 ? blk[3] : blk[2]) : (c & 1 ? blk[1] : blk[0]);
    const int ek = __ldg(a.exps + mine);
    float best = -INFINITY;
    for (int g = 0; g < a.G; ++g) {
      const uint4 up = s_q[g][0][c], down = s_q[g][1][c];
      int x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        int v = __dp4a(static_cast<int>(up.x), static_cast<int>(hi[u].x), 0);
        v = __dp4a(static_cast<int>(up.y), static_cast<int>(hi[u].y), v);
        v = __dp4a(static_cast<int>(up.z), static_cast<int>(hi[u].z), v);
        v = __dp4a(static_cast<int>(up.w), static_cast<int>(hi[u].w), v);
        v = __dp4a(static_cast<int>(down.x), static_cast<int>(lo[u].x), v);
        v = __dp4a(static_cast<int>(down.y), static_cast<int>(lo[u].y), v);
        v = __dp4a(static_cast<int>(down.z), static_cast<int>(lo[u].z), v);
        x[u] = __dp4a(static_cast<int>(down.w), static_cast<int>(lo[u].w), v);
      }
      const bool b0 = c & 1, b1 = c & 2;
      const int k0 = (b0 ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, b0 ? x[0] : x[1], 1);
      const int k1 = (b0 ? x[3] : x[2]) + __shfl_xor_sync(0xffffffffu, b0 ? x[2] : x[3], 1);
      int k = (b1 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
      if (LP == 8) k += __shfl_xor_sync(0xffffffffu, k, 4);
      best = fmaxf(best, ldexpf(static_cast<float>(k), s_e[g] - etop));
    }
    const int p = p0 + (c & 3) * GROUPS + lane / LP;
    if (c < 4 && p < min(base + kScorePages, P)) out[p] = ek == 255 ? INFINITY : ldexpf(best, ek - 127) + 0.0f;  // (no -0)
  }
}

// A score as a whole number of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 512, kBins = 2048;
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectArgs a, int token0) {
  constexpr int W = kSelectThreads / 32, BPT = kBins / kSelectThreads;
  __shared__ int s_bins[kBins];
  __shared__ int s_at[2], s_part[W], s_gt[W], s_eq[W];
  __shared__ uint32_t s_found[2];
  const int unit = static_cast<int>(blockIdx.x), token = token0 + unit / a.Hkv, h = unit % a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    int s, pos;
    token_position(a, token, lane, &s, &pos);
    if (lane == 0) {
      s_at[0] = s;
      s_at[1] = pos;
    }
  }
  __syncthreads();
  const int s = s_at[0], pos = s_at[1], page_log2 = 31 - __clz(a.page);
  const int P = pos < 0 ? 0 : min(pos >> page_log2, a.most_pages);
  const int k = min(a.n_select - 1, P);  // pages beside the token's own
  if (h == 0 && tid == 0) {  // each token as a sequence of its own
    const int c0 = cu_at(a.cu, 0, a.T), c1 = cu_at(a.cu, a.n_seqs, a.T);
    a.cu_out[token] = min(max(token, c0), c1);
    if (token == a.T - 1) a.cu_out[a.T] = min(max(a.T, c0), c1);
    a.lens_out[token] = pos < 0 ? 0 : (k << page_log2) + (pos & (a.page - 1)) + 1;
  }
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
        if (to < k) {
          if (pages) pages[to] = i;
          list[to] = page_at(row, i, a.n_pages);
        }
      }
      at += __popc(bt);
      eq_before += __popc(be);
    }
  }
  // the token's own page, and nothing behind it
  for (int i = k + tid; i < a.n_select; i += kSelectThreads) {
    const bool own = i == k && pos >= 0;
    if (pages) pages[i] = own ? pos >> page_log2 : -1;
    list[i] = own ? page_at(row, pos >> page_log2, a.n_pages) : 0;
  }
}

template <int D, int BF16>
int launch_bounds_d(const BoundsArgs& a, dim3 grid, cudaStream_t stream) {
  if (a.cache_dtype == CQSA_E4M3) bounds_kernel<D, BF16, kCacheE4m3><<<grid, kBoundThreads, 0, stream>>>(a);
  else if (a.cache_dtype == CQSA_INT4) bounds_kernel<D, BF16, kCacheInt4><<<grid, kBoundThreads, 0, stream>>>(a);
  else bounds_kernel<D, BF16, kCacheSame><<<grid, kBoundThreads, 0, stream>>>(a);
  return cuda_status(cudaGetLastError(), "page bounds kernel launch");
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
  const long long splits = (a.most_pages + kScorePages - 1) / kScorePages;
  for (int t = 0; t < a.T; t += at_once) {
    const int n = a.T - t < at_once ? a.T - t : at_once;
    const long long units = static_cast<long long>(n) * a.Hkv, blocks = units * splits;
    if (blocks > 0x7fffffffLL) {
      set_error("selection is too large for one launch (%lld blocks)", blocks);
      return CQSA_ERR_UNSUPPORTED;
    }
    const unsigned grid = static_cast<unsigned>(blocks);
    if (a.n_select > 1) {
      const bool bf = a.dtype == CQSA_BF16;
      if (a.d == 64 && bf) score_kernel<64, 1><<<grid, kScoreThreads, 0, stream>>>(a, t);
      else if (a.d == 64) score_kernel<64, 0><<<grid, kScoreThreads, 0, stream>>>(a, t);
      else if (bf) score_kernel<128, 1><<<grid, kScoreThreads, 0, stream>>>(a, t);
      else score_kernel<128, 0><<<grid, kScoreThreads, 0, stream>>>(a, t);
      const int rc = cuda_status(cudaGetLastError(), "page score kernel launch");
      if (rc != CQSA_OK) return rc;
    }
    select_kernel<<<static_cast<unsigned>(units), kSelectThreads, 0, stream>>>(a, t);
    const int rc = cuda_status(cudaGetLastError(), "page selection kernel launch");
    if (rc != CQSA_OK) return rc;
  }
  return CQSA_OK;
}

}  // namespace cqsa
