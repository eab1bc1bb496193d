// Attention of a few new tokens (one, in a serving step) of each sequence over its pages of a cache.
//
// The G = Hq / Hkv query heads that share a key head, times the sequence's new tokens, are the rows of one
// small product (row r = token r / G, head r % G of the group; 16 or 32 rows), so every cached vector is read
// once. That reading is the whole cost: a 128-feature fp16 vector brings 512 bytes of K and V for 16 * 512
// flops, so the kernel is laid out to keep the memory system busy, and the products run on warp-level
// mma.sync with 16-row tiles. (A tcgen05 product has at least 64 rows and hands its scores
// through tensor memory from one warp role to another; with a handful of rows that latency, and not the
// tensor rate, would set the pace.)
//
// Split: the key tiles of all (sequence, key head) units, laid end to end, are cut into one equal range per
// CTA, one CTA per SM, whatever the sequences' lengths are. A range covers the end of one unit, some whole
// units and the beginning of another; whole units are written out, the (at most two) others leave a normalised
// fp32 partial with its log-sum-exp, which combine_kernel joins exactly as cqsa_merge_partials does. It is
// launched with programmatic stream serialisation, so its start overlaps the main kernel's tail.
//
// A CTA: one producer warp copies key tiles page by page with TMA through a ring of stages (a lane per page
// box); 4 warps (8 for 32 rows), each on a quarter of a tile's keys, take them through S = Q K^T, an online softmax in
// registers, and O += P V, and join their rows in shared memory at the end of a unit's range. The tensor core truncates as it
// accumulates, so a warp adds its O to an fp32 sum (in its part of the joining buffer) every FOLD tiles, as attn_fwd.cu does.
//
// e4m3 pages: codes become fp16 in registers (exact). A key's power of two multiplies its scores in fp32, a
// value's goes onto its probability, relative to the largest exponent met so far (an integer that moves like
// the running maximum). Queries are fp16: bf16 ones are scaled by a power of two per row first, which is
// exact but for elements 2^-14 below the row's largest, whose error stays under 2^-25 of it.
//
// Measured, one token of each sequence, 32 query and 8 key heads, d = 128: 64 sequences of 300,000 bf16 positions together
// 202 us (1.23 GB, 6.1 TB/s); 128 of 500,000 e4m3 positions 204 us (1.03 GB, 5.1 TB/s: conversions and exponents keep the warps
// at 44% of issue, and two CTAs an SM at memory for three quarters of the time); one of 3,001 fp16 positions 12 us on the GPU.
#include <math.h>
#include <string.h>

#include "attn_common.cuh"
#include "cqsa_internal.h"
#include "seq_common.cuh"
#include "sm103_ptx.cuh"

namespace cqsa {
namespace {

__device__ DevErr g_decode_err;

constexpr int kQuarters = 4;  // warps that share a tile's keys
// Probabilities are kept as 2^14 p (and so are their sums): fp16 holds them without loss of relative precision
// down to p = 2^-28, where plain p would turn subnormal at 2^-14.
constexpr float kPShift = 14.0f;

constexpr int decode_occ(bool e4m3, int nmt) { return e4m3 && nmt == 1 ? 2 : 1; }

template <int D, bool E4M3, int NMT>
struct DecCfg {
  static constexpr int KT = E4M3 ? 128 : (D == 64 ? 128 : 64);   // keys of a tile
  static constexpr int KW = KT / kQuarters;                      // keys of a warp
  static constexpr int ROWB = E4M3 ? D : 128;                    // bytes of a shared-memory row
  static constexpr int XB = E4M3 ? 1 : D / 64;                   // boxes along the features
  static constexpr uint32_t TILE = static_cast<uint32_t>(KT) * ROWB * XB;
  static constexpr uint32_t STAGE = 2 * TILE + (E4M3 ? 1024 : 0);
  static constexpr int LDO = D + 8;                              // row of the joining buffer, padded against bank conflicts
  static constexpr uint32_t JOIN = static_cast<uint32_t>(NMT) * kQuarters * 16 * LDO * 4;
  static constexpr uint32_t ML = NMT * kQuarters * 32 * 4;            // m and l of each warp's rows
  // CTAs of an SM
  static constexpr int OCC = decode_occ(E4M3, NMT);
  static constexpr int NST_MAX = static_cast<int>((232448 / OCC - (OCC - 1) * 1024 - 1024 - 512 - JOIN - ML) / STAGE);
  static constexpr int NST = NST_MAX > 6 ? 6 : NST_MAX;
  static constexpr uint32_t SMEM = 1024 + NST * STAGE + JOIN + ML + 512;
  static constexpr int NTHR = 32 + 32 * kQuarters * NMT;
  // Tiles between folds of O: a warp's chain is 4,096 keys, 256 products, as in attn_fwd.cu at d = 128. In one chain a range of
  // 131,072 positions lost 2.2e-4 of sums of one sign, one of 2^21 positions 3.4e-3 (fp16's half step is 4.9e-4).
  static constexpr int FOLD = 16384 / KT;
  static_assert(SMEM <= 232448, "shared memory exceeds 227 KiB");
};

struct DecParams {
  const void* q;
  void* out;
  float* lse;
  float* part_o;  // [2 * CTAs][16 * NMT][D]
  float* part_l;  // [2 * CTAs][16 * NMT], base 2
  int4* meta;     // [CTAs][2] the unit a CTA's range begins in the middle of: sequence (-1: none), head, first and last
                  // CTA of it; the sequence's first token and tokens
  const int* table;
  const int* cu;
  const int* kv_lens;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  long long q_stride;
  int n_seqs, T, Hq, Hkv, G, max_pages, n_pages, page_log2, causal;
  float scale_log2;
  unsigned timeout_us;
  int fault;  // test hook: 1 = the first key tile of sequence 0 and head 0 is never loaded
};

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

// Byte offset of 16-byte chunk c of row r of a tile of ROWB-byte rows as TMA's 128-byte (64-byte for
// 64-byte rows) swizzle lays it down.
template <int ROWB>
__device__ __forceinline__ uint32_t sw_off(int r, int c) {
  if (ROWB == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// The same for a 16-bit tile, [8 rows][half of the features][8][64 features] (make_page_map), 16-byte chunk c of the
// whole vector.
template <int D>
__device__ __forceinline__ uint32_t tile16_off(int r, int c) {
  return static_cast<uint32_t>((r >> 3) * (1024 * (D / 64)) + (c >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
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

template <int D, int BF16, bool E4M3, int NMT>
__global__ void __launch_bounds__(DecCfg<D, E4M3, NMT>::NTHR, DecCfg<D, E4M3, NMT>::OCC)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecParams p) {
  using C = DecCfg<D, E4M3, NMT>;
  constexpr int KT = C::KT, KW = C::KW, NST = C::NST, NTHR = C::NTHR;
  constexpr int MB = E4M3 ? 0 : BF16;  // type of the products: e4m3 pages are fp16 after conversion
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(sm + NST * C::STAGE);
  float* ml = join + C::JOIN / 4;  // [NMT][kQuarters][m 16 | l 16]
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ml) + C::ML);
  uint64_t* empty = full + NST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NST);
  long long* s_base = reinterpret_cast<long long*>(empty + NST + 1);
  long long* s_sum = s_base + 1;  // total tiles
  int* s_seq = reinterpret_cast<int*>(s_sum + 1);
  long long* s_warp = reinterpret_cast<long long*>(s_seq + 2);  // [32]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kQuarters * NMT);
    }
    *abort_flag = 0;
    *s_seq = -1;
    fence_mbar_init();
  }
  // the tiles of all sequences, and the sequence this CTA's range begins in
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
  // the joining kernel may be set up from here on; it waits for this grid's end before it reads anything
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t a_abort = smem_u32(const_cast<int*>(abort_flag));
  Walk wk;
  wk.s = *s_seq;
  wk.base = *s_base;
  wk.n = 0;
  if (wk.s >= 0) walk_load<KT>(p, wk);
  if (wk.s < 0) {
    if (tid == 0) p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  } else if (warp == NW - 1) {
    // ------------------------------------------------------------------ producer warp
    if (lane == 0) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
    const int page = 1 << p.page_log2;
    const int rows = min(page, KT);             // rows of a box
    const int boxes = KT / rows;                // page boxes of a tile
    int it = 0;
    bool ok = true;
    for (long long w = w0; ok && w < w1;) {
      const Piece pc = piece_at(wk, w, w1);
      const int h = pc.h, t0 = pc.t0, t1 = pc.t1;
      const int* row = p.table + static_cast<long long>(wk.s) * p.max_pages;
      for (int t = t0; ok && t < t1; ++t, ++it) {
        const int stage = it % NST;
        if (it >= NST)
          ok = wait_or_abort(smem_u32(&empty[stage]), ((it / NST) - 1) & 1u, p.timeout_us, a_abort, &g_decode_err,
                             kDevTimeoutKV, 40);
        if (!ok) break;
        if (p.fault == 1 && wk.s == 0 && h == 0 && t == 0) {  // (every wait on the tile runs out)
          ok = false;
          break;
        }
        uint8_t* st = sm + stage * C::STAGE;
        const int k0 = t * KT;
        const int nb = min(boxes, max(0, (wk.len - k0 + rows - 1) >> (31 - __clz(rows))));
        if (lane == 0)
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(nb) * rows * (2 * C::ROWB * C::XB + (E4M3 ? 2 : 0)));
        __syncwarp();
        for (int i = lane; i < nb; i += 32) {
          const int pos = k0 + i * rows;
          const int pg = page_at(row, pos >> p.page_log2, p.n_pages), y = pos & (page - 1);
          const uint32_t off = static_cast<uint32_t>(i * rows) * C::ROWB * C::XB;
          const int block = pg * p.Hkv + h;
          if (E4M3) {
            tma_load_3d(st + off, &tmK, &full[stage], 0, y, block);
            tma_load_3d(st + C::TILE + off, &tmV, &full[stage], 0, y, block);
            const long long at = (static_cast<long long>(block) << p.page_log2) + y;
            bulk_load(st + 2 * C::TILE + i * rows, p.k_scale + at, rows, &full[stage]);
            bulk_load(st + 2 * C::TILE + 512 + i * rows, p.v_scale + at, rows, &full[stage]);
          } else {
            tma_load_5d(st + off, &tmK, &full[stage], 0, 0, 0, y >> 3, block);
            tma_load_5d(st + C::TILE + off, &tmV, &full[stage], 0, 0, 0, y >> 3, block);
          }
        }
      }
      w = pc.next;
      if (w < w1 && h == p.Hkv - 1) walk_next<KT>(p, wk);
    }
    __syncwarp();
    // every copy issued has landed before the CTA ends (bounded)
    for (int j = max(0, it - NST); j < it; ++j)
      mbar_wait_bounded(&full[j % NST], (j / NST) & 1u, p.timeout_us * 1000ull);
  } else {
    // ------------------------------------------------------------------ key warps
    const int mt = warp / kQuarters, kg = warp % kQuarters;  // row tile, quarter of the keys
    const int g = lane >> 2, t4 = lane & 3;
    float* jbuf = join + mt * kQuarters * 16 * C::LDO;
    float* mlb = ml + mt * kQuarters * 32;
    bool ok = true;
    int it = 0;
    for (long long w = w0; w < w1;) {
      const Piece pc = piece_at(wk, w, w1);
      const int h = pc.h, t0 = pc.t0, t1 = pc.t1;
      if (w == w0 && tid == 0) {
        // the unit this range begins in the middle of, and the CTAs whose ranges hold its first and last tile
        const long long u0 = wk.base + static_cast<long long>(h) * wk.n, u1 = u0 + wk.n - 1;
        const int c0 = static_cast<int>(((u0 + kUnit + 1) * nc - 1) / W), c1 = static_cast<int>(((u1 + 1) * nc - 1) / W);
        p.meta[2 * blockIdx.x] = t0 == 0 ? make_int4(-1, 0, 0, 0) : make_int4(wk.s, h, c0, c1);
        p.meta[2 * blockIdx.x + 1] = make_int4(wk.first, wk.qlen, 0, 0);
      }
      if (t1 <= t0) {
        w = pc.next;
        if (w < w1 && h == p.Hkv - 1) walk_next<KT>(p, wk);
        continue;
      }
      // ---- the rows' queries as A fragments, and the keys each of this thread's two rows may see
      uint32_t qf[D / 16][4];
      int lim[2];
      float rs[2];  // factor from a raw score to the base-2 exponent
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = mt * 16 + g + 8 * u;
        const int tok = r / p.G;
        const bool valid = tok < wk.qlen;
        lim[u] = !valid ? 0 : (p.causal ? min(wk.len, wk.len - wk.qlen + tok + 1) : wk.len);
        const uint16_t* qr = static_cast<const uint16_t*>(p.q) + static_cast<long long>(wk.first + tok) * p.q_stride +
                             static_cast<long long>(h * p.G + (r - tok * p.G)) * D;
        rs[u] = p.scale_log2;
        if (E4M3) {
          // features 16 ks + 4 t4 .. + 3: the pairs of the fragment's low and high half (the order of the
          // codes that one ldmatrix register holds; the sum over features does not mind)
          float f[D / 16][4];
          float amax = 0.0f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint2 x = make_uint2(0, 0);
            if (valid) x = __ldg(reinterpret_cast<const uint2*>(qr + ks * 16 + 4 * t4));
            const float2 a = unpack16(x.x, BF16), b = unpack16(x.y, BF16);
            f[ks][0] = a.x; f[ks][1] = a.y; f[ks][2] = b.x; f[ks][3] = b.y;
            if (BF16) amax = fmaxf(fmaxf(amax, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
          }
          if (BF16) {
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^-e brings the row's largest value into [1, 2); held to the exponents whose inverse is normal
            const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
            const float inv = pow2i(-e);
            rs[u] = p.scale_log2 * pow2i(e);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
              for (int i = 0; i < 4; ++i) f[ks][i] *= inv;
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[ks][u] = pack16(f[ks][0], f[ks][1], 0);
            qf[ks][2 + u] = pack16(f[ks][2], f[ks][3], 0);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[ks][u] = valid ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t4)) : 0u;
            qf[ks][2 + u] = valid ? __ldg(reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8 + 2 * t4)) : 0u;
          }
        }
      }
      const int lim_all = p.causal ? wk.len - wk.qlen + 1 : wk.len;  // keys that every row sees
      float o[D / 8][4];
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
      int ev = -1;  // e4m3: exponent byte the output sums are relative to
      // The running sum that O is folded into: D / 2 values of this lane, then the references that they are relative to. (The
      // layout of the join below is another, and is written after the next named_sync.)
      float* sum = jbuf + kg * 16 * C::LDO + lane;
      auto sum_factor = [&](int u) -> float {
        const float was = sum[(D / 2 + u) * 32], a = was == -INFINITY ? 0.0f : ex2(was - m[u]);
        return E4M3 ? a * exp2_int_any(__float_as_int(sum[(D / 2 + 2) * 32]) - ev) : a;
      };
      for (int t = t0; t < t1; ++t, ++it) {
        if (t > t0 && (t - t0) % C::FOLD == 0) {
          const bool have = t - t0 > C::FOLD;
          if (!have) named_sync(1 + mt, 32 * kQuarters);  // the unit before has been read out of the buffer
          const float fs[2] = {have ? sum_factor(0) : 0.0f, have ? sum_factor(1) : 0.0f};
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float* at = sum + (j * 4 + i) * 32;
              *at = (have ? *at * fs[i >> 1] : 0.0f) + o[j][i];
              o[j][i] = 0.0f;
            }
          sum[(D / 2) * 32] = m[0];
          sum[(D / 2 + 1) * 32] = m[1];
          sum[(D / 2 + 2) * 32] = __int_as_float(ev);
        }
        const int stage = it % NST;
        if (ok) ok = wait_or_abort(smem_u32(&full[stage]), (it / NST) & 1u, p.timeout_us, a_abort, &g_decode_err,
                                   kDevTimeoutKV, 41);
        uint8_t* st = sm + stage * C::STAGE;
        const uint32_t sk = smem_u32(st), sv = sk + C::TILE;
        const int kw0 = kg * KW;                 // first key of this warp in the tile
        const int k0 = t * KT + kw0;             // its position
        const int left = wk.len - k0;            // positions of the sequence from there
        // ---- e4m3: this thread's keys' exponents (before the products, which hide their way), and the largest of the values'.
        // Slots past the end hold anything: their scores keep a factor of 1, their values' exponents do not count.
        uint32_t kexp[E4M3 ? KW / 8 : 1][2], vexp[E4M3 ? KW / 8 : 1][2];
        if constexpr (E4M3) {
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < KW / 8; ++j) {
            const uint8_t* sc = st + 2 * C::TILE + kw0 + j * 8 + 2 * t4;
            const uint32_t kb = *reinterpret_cast<const uint16_t*>(sc), vb = *reinterpret_cast<const uint16_t*>(sc + 512);
            kexp[j][0] = kb & 255u;
            kexp[j][1] = kb >> 8;
            vexp[j][0] = vb & 255u;
            vexp[j][1] = vb >> 8;
          }
          if (left < KW) {
#pragma unroll
            for (int j = 0; j < KW / 8; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (j * 8 + 2 * t4 + i >= left) {
                  kexp[j][i] = 127u;
                  vexp[j][i] = 0u;
                }
          }
#pragma unroll
          for (int j = 0; j < KW / 8; ++j) top = max(top, max(vexp[j][0], vexp[j][1]));
          top = __reduce_max_sync(0xffffffffu, top);
          if (static_cast<int>(top) > ev) {
            const float a = ev < 0 ? 0.0f : exp2_int_any(ev - static_cast<int>(top));
            ev = static_cast<int>(top);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[j][i] *= a;
          }
        }
        // ---- S = Q K^T
        float s[KW / 8][4];
#pragma unroll
        for (int j = 0; j < KW / 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[j][i] = 0.0f;
        if constexpr (E4M3) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {  // 64 features: four ldmatrix matrices of 16 codes
            uint32_t b[KW / 8][4];
#pragma unroll
            for (int j = 0; j < KW / 8; ++j) ldsm4(sk + sw_off<C::ROWB>(kw0 + j * 8 + (lane & 7), c * 4 + (lane >> 3)), b[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int j = 0; j < KW / 8; ++j)  // neighbouring products are independent
                mma16816<0>(s[j], qf[c * 4 + i], e4m3x2_to_f16x2(b[j][i] & 0xffffu), e4m3x2_to_f16x2(b[j][i] >> 16));
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int j = 0; j < KW / 16; ++j) {
              const int r = kw0 + j * 16 + ((lane >> 4) << 3) + (lane & 7);
              uint32_t b[4];
              ldsm4(sk + tile16_off<D>(r, ks * 2 + ((lane >> 3) & 1)), b);
              mma16816<MB>(s[2 * j], qf[ks], b[0], b[1]);
              mma16816<MB>(s[2 * j + 1], qf[ks], b[2], b[3]);
            }
          }
        }
        // ---- scores in base 2, masks, running maximum
        const bool mask = left < KW || k0 + KW > lim_all || lim[0] == 0 || lim[1] == 0;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < KW / 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // (a byte is an fp32 exponent field; 0, never written, counts as 0)
            float x = s[j][i] * (E4M3 ? rs[i >> 1] * __uint_as_float(kexp[j][i & 1] << 23) : rs[i >> 1]);
            if (mask && k0 + j * 8 + 2 * t4 + (i & 1) >= lim[i >> 1]) x = -INFINITY;
            s[j][i] = x;
            mx[i >> 1] = fmaxf(mx[i >> 1], x);
          }
        float al[2], mu[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
          mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
          const float mn = fmaxf(m[u], mx[u]);
          mu[u] = mn == -INFINITY ? 0.0f : mn;
          al[u] = ex2(m[u] - mu[u]);  // 0 while the row has seen nothing
          mu[u] -= kPShift;
          m[u] = mn;
          l[u] *= al[u];
        }
        if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][0] *= al[0];
            o[j][1] *= al[0];
            o[j][2] *= al[1];
            o[j][3] *= al[1];
          }
        }
        // ---- P, rounded to the products' type (relative 2^-11 for fp16, 2^-8 for bf16, as the output is)
        uint32_t pf[KW / 16][4];
#pragma unroll
        for (int j = 0; j < KW / 8; ++j) {
          float pr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pr[i] = ex2(s[j][i] - mu[i >> 1]);
            l[i >> 1] += pr[i];
          }
          if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] *= exp2_int_any(static_cast<int>(vexp[j][i & 1]) - ev);
          }
          pf[j >> 1][(j & 1) * 2] = pack16(pr[0], pr[1], MB);
          pf[j >> 1][(j & 1) * 2 + 1] = pack16(pr[2], pr[3], MB);
        }
        // ---- values past the sequence's end are zero, whatever the page holds there (0 * NaN is NaN)
        if (left < KW) {
          const int z0 = max(left, 0);
          constexpr int PIECES = C::ROWB * C::XB / 16;  // 16-byte pieces of a vector
          for (int i = lane; i < (KW - z0) * PIECES; i += 32) {
            const int c = i % PIECES, r = kw0 + z0 + i / PIECES;
            st_shared_zero16(sv + (E4M3 ? sw_off<C::ROWB>(r, c) : tile16_off<D>(r, c)));
          }
          fence_async_smem();  // before the next copy into these rows
          __syncwarp();
        }
        // ---- O += P V
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < KW / 16; ++j) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {  // 32 features: two chunks of 16 codes, keys 0-7 and 8-15
              uint32_t b[4];
              const int r = kw0 + j * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
              ldsm4t(sv + sw_off<C::ROWB>(r, c * 2 + (lane >> 4)), b);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t lo = b[2 * x], hi = b[2 * x + 1];  // [key, f0 f1 | key + 1, f0 f1]
                mma16816<0>(o[(c * 2 + x) * 2], pf[j], e4m3x2_to_f16x2(__byte_perm(lo, 0, 0x4420)),
                            e4m3x2_to_f16x2(__byte_perm(hi, 0, 0x4420)));
                mma16816<0>(o[(c * 2 + x) * 2 + 1], pf[j], e4m3x2_to_f16x2(__byte_perm(lo, 0, 0x4431)),
                            e4m3x2_to_f16x2(__byte_perm(hi, 0, 0x4431)));
              }
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < KW / 16; ++j) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t b[4];
              const int r = kw0 + j * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
              ldsm4t(sv + tile16_off<D>(r, c * 2 + (lane >> 4)), b);
              mma16816<MB>(o[2 * c], pf[j], b[0], b[1]);
              mma16816<MB>(o[2 * c + 1], pf[j], b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
      }
      if (t1 - t0 > C::FOLD) {
        const float fs[2] = {sum_factor(0), sum_factor(1)};
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] += sum[(j * 4 + i) * 32] * fs[i >> 1];
      }
      // ---- join the warps' rows: each brings its sums to the common maximum and scale
      // (the exponent reference of e4m3 values is a power of two that is multiplied out here)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (t4 == 0) {
          mlb[kg * 32 + g + 8 * u] = m[u];
          mlb[kg * 32 + 16 + g + 8 * u] = l[u];
        }
      }
      named_sync(1 + mt, 32 * kQuarters);
      float f[2], lse2[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float M = -INFINITY, L = 0.0f;
#pragma unroll
        for (int i = 0; i < kQuarters; ++i) M = fmaxf(M, mlb[i * 32 + g + 8 * u]);
        const float Mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int i = 0; i < kQuarters; ++i) L += mlb[i * 32 + 16 + g + 8 * u] * ex2(mlb[i * 32 + g + 8 * u] - Mu);
        f[u] = L > 0.0f ? ex2(m[u] - Mu) / L : (L != L ? NAN : 0.0f);
        lse2[u] = L > 0.0f ? M - kPShift + log2f(L) : (L != L ? NAN : -INFINITY);
        if (E4M3) f[u] *= ev < 0 ? 0.0f : exp2_byte(static_cast<uint32_t>(ev));
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        float* b0 = jbuf + (kg * 16 + g) * C::LDO;
        float* b1 = b0 + 8 * C::LDO;
        if constexpr (E4M3) {
          // column n of the even (odd) tile of a chunk is feature 16 c + 2 n (+ 1)
          const int ft = (j >> 1) * 16 + 4 * t4 + (j & 1);
          b0[ft] = o[j][0] * f[0];
          b0[ft + 2] = o[j][1] * f[0];
          b1[ft] = o[j][2] * f[1];
          b1[ft + 2] = o[j][3] * f[1];
        } else {
          *reinterpret_cast<float2*>(b0 + j * 8 + 2 * t4) = make_float2(o[j][0] * f[0], o[j][1] * f[0]);
          *reinterpret_cast<float2*>(b1 + j * 8 + 2 * t4) = make_float2(o[j][2] * f[1], o[j][3] * f[1]);
        }
      }
      if (kg == 0 && t4 == 0) {  // a column of the padding carries the rows' lse
        jbuf[g * C::LDO + D] = lse2[0];
        jbuf[(g + 8) * C::LDO + D] = lse2[1];
      }
      named_sync(1 + mt, 32 * kQuarters);
      const bool whole = t0 == 0 && t1 == wk.n - kUnit;
      const long long slot = 2 * static_cast<long long>(blockIdx.x) + (t0 == 0 ? 1 : 0);
      for (int e = kg * 32 + lane; e < 16 * (D / 4); e += 32 * kQuarters) {
        const int row = e / (D / 4), c = e % (D / 4);
        const int r = mt * 16 + row, tok = r / p.G;
        if (tok >= wk.qlen || !ok) continue;
        float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kQuarters; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(jbuf + (i * 16 + row) * C::LDO + c * 4);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        if (whole) {
          const long long at = static_cast<long long>(wk.first + tok) * p.Hq + h * p.G + (r - tok * p.G);
          reinterpret_cast<uint2*>(p.out)[at * (D / 4) + c] = make_uint2(pack16(a.x, a.y, BF16), pack16(a.z, a.w, BF16));
          if (p.lse && c == 0)
            p.lse[static_cast<long long>(h * p.G + (r - tok * p.G)) * p.T + wk.first + tok] = jbuf[row * C::LDO + D] * 0.69314718055994531f;
        } else {
          reinterpret_cast<float4*>(p.part_o)[(slot * (16 * NMT) + r) * (D / 4) + c] = a;
          if (c == 0) p.part_l[slot * (16 * NMT) + r] = jbuf[row * C::LDO + D];
        }
      }
      w = pc.next;
      if (w < w1 && h == p.Hkv - 1) walk_next<KT>(p, wk);
    }
  }
  __syncthreads();
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

template <int D, int BF16, bool E4M3, int NMT>
int launch_t(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int ctas, cudaStream_t stream) {
  using C = DecCfg<D, E4M3, NMT>;
  auto kern = decode_kernel<D, BF16, E4M3, NMT>;
  static PerDeviceOnce attr;
  int dev = 0;
  if (!attr.done(&dev)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(paged attention smem)");
    attr.mark(dev);
  }
  kern<<<ctas, C::NTHR, C::SMEM, stream>>>(mk, mv, p);
  int rc = cuda_status(cudaGetLastError(), "paged attention kernel launch");
  if (rc != CQSA_OK || ctas == 1) return rc;
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
  return cuda_status(cudaLaunchKernelEx(&cfg, combine_kernel<D, BF16>, p, 16 * NMT), "paged attention joining kernel launch");
}

template <int D, int BF16, bool E4M3>
int launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int rows, int ctas, cudaStream_t s) {
  return rows <= 16 ? launch_t<D, BF16, E4M3, 1>(mk, mv, p, ctas, s) : launch_t<D, BF16, E4M3, 2>(mk, mv, p, ctas, s);
}

int tile_keys(const PagedArgs& a) { return a.cache_dtype == CQSA_E4M3 || a.d == 64 ? 128 : 64; }

int decode_rows(const PagedArgs& a) { return static_cast<long long>(a.max_q_len) * (a.Hq / a.Hkv) <= 16 ? 16 : 32; }

// One CTA per SM, fewer when there are fewer key tiles (by the caller's longest sequence; longer ones are
// still computed, with fewer CTAs than they could use).
int decode_ctas(const PagedArgs& a) {
  const long long kt = tile_keys(a);
  const long long tiles = (a.max_kv_len + kt - 1) / kt;
  const long long all = ((tiles < 1 ? 1 : tiles) + kUnit) * a.n_seqs * a.Hkv;
  const int most = sm_count() * decode_occ(a.cache_dtype == CQSA_E4M3, decode_rows(a) / 16);
  return static_cast<int>(all < most ? all : most);
}

}  // namespace

// Up to 32 rows per sequence and key head, by the caller's most new tokens; 32 are this kernel's two row tiles. 32 rows of each sequence here and
// in attn_seq.cu's kernel, us: d = 128, 64 sequences of some 290,000 positions together 251 / 261 over 16-bit pages and 284 / 489 over
// e4m3 ones, 8 sequences of 44,000 16-bit ones 75 / 65, of 112,000 e4m3 ones 122 / 169; d = 64 61 / 67, 59 / 87, 35 / 39, 35 / 44. 16 rows:
// 207 / 253, 157 / 470, 56 / 65, 74 / 169; 54 / 67, 38 / 88, 27 / 41, 30 / 46. (From there on one longer chunk in a batch
// takes its single tokens along; over e4m3 pages that is a step, 284 to 510 us for the first.)
bool decode_applies(const PagedArgs& a) { return static_cast<long long>(a.max_q_len) * (a.Hq / a.Hkv) <= 32; }

size_t decode_workspace(const PagedArgs& a) {
  const size_t rows = static_cast<size_t>(decode_rows(a));
  const size_t n = 2 * static_cast<size_t>(decode_ctas(a));
  return ((n * rows * a.d * 4 + 255) & ~size_t(255)) + ((n * rows * 4 + 255) & ~size_t(255)) + n * sizeof(int4);
}

int launch_decode(const PagedArgs& a, cudaStream_t stream) {
  CUtensorMap mk, mv;
  const int kt = tile_keys(a);
  const int rows_box = a.page < kt ? a.page : kt;
  int rc = make_page_map(&mk, a.k_cache, a, rows_box);
  if (rc == CQSA_OK) rc = make_page_map(&mv, a.v_cache, a, rows_box);
  if (rc != CQSA_OK) return rc;
  const int rr = decode_rows(a);
  const int ctas = decode_ctas(a);
  DecParams p;
  memset(&p, 0, sizeof(p));
  p.q = a.q;
  p.out = a.out;
  p.lse = a.lse;
  const size_t n = 2 * static_cast<size_t>(ctas);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  ws += (n * rr * a.d * 4 + 255) & ~size_t(255);
  p.part_l = reinterpret_cast<float*>(ws);
  ws += (n * rr * 4 + 255) & ~size_t(255);
  p.meta = reinterpret_cast<int4*>(ws);
  p.table = a.table;
  p.cu = a.cu;
  p.kv_lens = a.kv_lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.q_stride = a.q_stride;
  p.n_seqs = a.n_seqs;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_log2 = 31 - __builtin_clz(static_cast<unsigned>(a.page));
  p.causal = a.causal;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.timeout_us = timeout_us();
  p.fault = debug_fault();
  const bool bf = a.dtype == CQSA_BF16;
  if (a.cache_dtype == CQSA_E4M3) {
    if (a.d == 64) return bf ? launch_rows<64, 1, true>(mk, mv, p, rr, ctas, stream) : launch_rows<64, 0, true>(mk, mv, p, rr, ctas, stream);
    return bf ? launch_rows<128, 1, true>(mk, mv, p, rr, ctas, stream) : launch_rows<128, 0, true>(mk, mv, p, rr, ctas, stream);
  }
  if (a.d == 64) return bf ? launch_rows<64, 1, false>(mk, mv, p, rr, ctas, stream) : launch_rows<64, 0, false>(mk, mv, p, rr, ctas, stream);
  return bf ? launch_rows<128, 1, false>(mk, mv, p, rr, ctas, stream) : launch_rows<128, 0, false>(mk, mv, p, rr, ctas, stream);
}

DEV_ERR_READERS(decode, g_decode_err)

}  // namespace cqsa
