// Parts that the kernels for a few new tokens over pages share (attn_decode.cu: 16-bit and e4m3 pages, attn_decode4.cu: 4-bit
// ones): the equal split of all units' key tiles over the CTAs, warp-level products, and the joining of parts.
#pragma once
#include <math.h>
#include <string.h>

#include "attn_common.cuh"
#include "cqsa_internal.h"
#include "seq_common.cuh"

namespace cqsa {

struct DecParams {
  const void* q;
  void* out;
  float* lse;
  float* part_o;  // [2 * CTAs][16 * NMT][D]
  float* part_l;  // [2 * CTAs][16 * NMT], base 2
  int4* meta;     // [CTAs][2] the unit a CTA's range begins in the middle of: sequence (-1: none), head, first and last
                  // CTA of it; the sequence's first token and tokens
  const int* table;  // the pages of sequence s and key head h: from table + s * row_seq + h * row_head on
  const int* cu;
  const int* kv_lens;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  long long q_stride, row_seq, row_head;
  int n_seqs, T, Hq, Hkv, G, max_pages, n_pages, page_log2, causal;
  float scale_log2;
  unsigned timeout_us;
  int fault;  // test hook: 1 = the first key tile of sequence 0 and head 0 is never loaded
};

namespace {

constexpr int kQuarters = 4;  // warps that share a tile's keys
// Probabilities are kept as 2^14 p (and so are their sums): fp16 holds them without loss of relative precision
// down to p = 2^-28, where plain p would turn subnormal at 2^-14.
constexpr float kPShift = 14.0f;

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
template <int BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A unit counts as its key tiles and kUnit more: what its queries' loads and the joining of its rows cost. Without them
// a CTA that gets many short sequences finishes late (128 ragged sequences of e4m3: the last CTA at 311 us, the mean at 231).
constexpr int kUnit = 2;

// Where a CTA's walk over its range stands: sequence, the length of each of its units, tokens and positions.
struct Walk {
  int s, n, qlen, first, len;
  long long base;  // where the sequence's first unit begins
};

// What a range [w, w1) does in the unit it stands in: head, and key tiles [t0, t1) (none when it only reaches into the
// unit's kUnit). `next`: where the unit (or the range) ends.
struct Piece {
  int h, t0, t1;
  long long next;
};
__device__ __forceinline__ Piece piece_at(const Walk& k, long long w, long long w1) {
  Piece r;
  const long long rel = w - k.base;
  r.h = static_cast<int>(rel / k.n);
  const long long u0 = k.base + static_cast<long long>(r.h) * k.n;
  r.next = min(u0 + k.n, w1);
  r.t0 = max(0, static_cast<int>(w - u0) - kUnit);
  r.t1 = max(0, static_cast<int>(r.next - u0) - kUnit);
  return r;
}

template <int KT>
__device__ __forceinline__ void walk_load(const DecParams& p, Walk& w) {
  w.qlen = seq_tokens(p.cu, w.s, p.T, &w.first);
  w.len = seq_positions(p.kv_lens, w.s, static_cast<long long>(p.max_pages) << p.page_log2);
  // a sequence without new tokens is no work; one without positions is one empty tile (its rows are zero)
  w.n = w.qlen == 0 ? 0 : max(1, (w.len + KT - 1) / KT) + kUnit;
}
template <int KT>
__device__ __forceinline__ void walk_next(const DecParams& p, Walk& w) {
  do {
    w.base += static_cast<long long>(w.n) * p.Hkv;
    ++w.s;
    if (w.s >= p.n_seqs) return;
    walk_load<KT>(p, w);
  } while (w.n == 0);
}

// A CTA's share of all units' key tiles laid end to end: [begin, end) of `all`, one range for each of `ctas` CTAs.
struct Range {
  long long all, ctas, begin, end;
};

// The range of this CTA, by its whole block of NTHR threads. Leaves in shared memory the sequence that the range begins in
// (*s_seq; as it was where the range is empty) and where that sequence's first unit begins (*s_base).
template <int KT, int NTHR>
__device__ __forceinline__ Range find_range(const DecParams& p, long long* s_warp, long long* s_base, int* s_seq) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto tiles_of = [&](int s) -> long long {
    if (s >= p.n_seqs) return 0;
    Walk w;
    w.s = s;
    walk_load<KT>(p, w);
    return static_cast<long long>(w.n) * p.Hkv;
  };
  constexpr int NW = NTHR / 32;
  auto block_scan = [&](long long v, long long* before) -> long long {  // total; *before: sum over lower threads
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long b = 0, t = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if (i < warp) b += s_warp[i];
      t += s_warp[i];
    }
    *before = b + x - v;
    return t;
  };
  long long mine, before;
  {
    Walk w;
    w.s = tid;
    w.n = 0;
    if (tid < p.n_seqs) walk_load<KT>(p, w);
    mine = static_cast<long long>(w.n) * p.Hkv;
  }
  long long W = block_scan(mine, &before);  // the first NTHR sequences
  const long long W_first = W;
  long long unused;
  for (int s0 = NTHR; s0 < p.n_seqs; s0 += NTHR) W += block_scan(tiles_of(s0 + tid), &unused);
  // every range holds a tile: with fewer tiles than CTAs (sequences shorter than the caller said) the last CTAs idle
  const long long nc = min(static_cast<long long>(gridDim.x), W);
  const long long bx = blockIdx.x;
  const long long w0 = bx < nc ? W * bx / nc : 0, w1 = bx < nc ? W * (bx + 1) / nc : 0;
  if (w0 < w1 && before <= w0 && w0 < before + mine) {
    *s_seq = tid;
    *s_base = before;
  }
  for (long long base = W_first, s0 = NTHR; base <= w0 && s0 < p.n_seqs; s0 += NTHR) {
    const long long v = tiles_of(static_cast<int>(s0) + tid);
    const long long t = block_scan(v, &before);
    before += base;
    if (w0 < w1 && before <= w0 && w0 < before + v) {
      *s_seq = static_cast<int>(s0) + tid;
      *s_base = before;
    }
    base += t;
  }
  __syncthreads();
  const Range r = {W, nc, w0, w1};
  return r;
}

// Joins the partials of the units that several ranges share. Block c looks after the unit that range c begins in
// the middle of, if it is the first such range: M = max lse_k, lse = M + log2 sum 2^(lse_k - M),
// out = sum 2^(lse_k - lse) O_k, in the order of the ranges (deterministic).
// A warp takes a row (d = 128: a float4 a lane; d = 64: two rows): its lanes fetch the parts' lse side by side, and the
// parts' values are fetched eight at a time before they are needed, so the chain is two trips to L2 for up to 32 parts.
template <int D, int BF16>
__global__ void __launch_bounds__(128) combine_kernel(const DecParams p, int rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 m = __ldcg(p.meta + 2 * blockIdx.x), q = __ldcg(p.meta + 2 * blockIdx.x + 1);
  if (m.x < 0 || static_cast<int>(blockIdx.x) != m.z + 1) return;
  const int h = m.y, c0 = m.z, parts = m.w - c0 + 1;
  const int first = q.x, n = min(rows, q.y * p.G);  // the sequence's first token and rows
  constexpr int LPR = D / 4;       // lanes of a row
  constexpr int RPW = 32 / LPR;    // rows of a warp
  const int lane = threadIdx.x & 31, c = lane % LPR;
  auto slot_of = [&](int k) -> long long { return 2LL * (c0 + k) + (k == 0 ? 1 : 0); };
  for (int r0 = (threadIdx.x >> 5) * RPW; r0 < n; r0 += 4 * RPW) {
    const int r = min(r0 + lane / LPR, n - 1);  // (a row past the end repeats the last one)
    float M = -INFINITY, L = 0.0f;
    float4 a = make_float4(0, 0, 0, 0);
    for (int k0 = 0; k0 < parts; k0 += LPR) {
      const int kk = min(LPR, parts - k0);
      const float lk = c < kk ? __ldcg(p.part_l + slot_of(k0 + c) * rows + r) : -INFINITY;
      float top = lk;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float Mn = fmaxf(M, top), Mu = Mn == -INFINITY ? 0.0f : Mn;
      const float fix = M == -INFINITY ? 0.0f : exp2f(M - Mu);
      const float w = lk == -INFINITY ? 0.0f : exp2f(lk - Mu);  // NaN passes on
      M = Mn;
      L *= fix;
      a.x *= fix;
      a.y *= fix;
      a.z *= fix;
      a.w *= fix;
      for (int k = 0; k < kk; k += 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (slot_of(k0 + min(k + u, kk - 1)) * rows + r) * LPR + c);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w, (lane & ~(LPR - 1)) + min(k + u, LPR - 1));
          if (k + u < kk) {
            L += wu;
            a.x = fmaf(wu, v[u].x, a.x);
            a.y = fmaf(wu, v[u].y, a.y);
            a.z = fmaf(wu, v[u].z, a.z);
            a.w = fmaf(wu, v[u].w, a.w);
          }
        }
      }
    }
    const float inv = L > 0.0f ? 1.0f / L : (L != L ? NAN : 0.0f);
    const int tok = r / p.G, hq = h * p.G + (r - tok * p.G);
    const long long at = static_cast<long long>(first + tok) * p.Hq + hq;
    reinterpret_cast<uint2*>(p.out)[at * LPR + c] =
        make_uint2(pack16(a.x * inv, a.y * inv, BF16), pack16(a.z * inv, a.w * inv, BF16));
    if (p.lse && c == 0)
      p.lse[static_cast<long long>(hq) * p.T + first + tok] =
          L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : (L != L ? NAN : -INFINITY);
  }
}

// The joining kernel behind a main kernel of `ctas` CTAs and parts of `rows` rows; its start overlaps the main kernel's tail.
template <int D, int BF16>
int launch_combine(const DecParams& p, int rows, int ctas, cudaStream_t stream) {
  if (ctas == 1) return CQSA_OK;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, combine_kernel<D, BF16>, p, rows), "paged attention joining kernel launch");
}

}  // namespace

// attn_decode4.cu: the kernel over 4-bit pages, for `rows` (8, 16 or 32) rows of a unit.
// CTAs of an SM, of 5 warps (9 for 32 rows): three leave a thread 128 registers, which hold the sums of 8 rows at d = 128 and of 16 at d = 64; four leave
// 96, enough for 8 rows at d = 64 (128 sequences of 1,000,000 positions 165 us against 183; at d = 128 they spill, 253 against 235; both
// measured before scales far below the largest had a round of their own).
constexpr int decode4_occ(int rows, int d) { return rows == 8 ? (d == 64 ? 4 : 3) : (rows == 16 ? (d == 64 ? 3 : 2) : 1); }
constexpr int kDecode4Tile = 128;  // keys of its tiles
int launch_decode4(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int d, int bf16, int rows, int ctas, cudaStream_t stream);

}  // namespace cqsa
