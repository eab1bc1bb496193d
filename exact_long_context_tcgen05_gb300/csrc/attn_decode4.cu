// Attention of a few new tokens (one, in a serving step) of each sequence over its pages of a 4-bit cache.
//
// A unit's rows, the split over the CTAs and the joining of parts are attn_decode.cu's. What a quarter of the bytes changes: a cached
// vector of 128 features is 68 bytes, and at the memory's rate an SM has some six cycles, 23 warp instructions, for a key's and a
// value's 256 numbers, so the kernel is laid out to spend few instructions on each.
//
// Products are S^T = K Q^T and O^T = V^T P^T on mma.sync's 16 x 8 x 16 tiles: the cache gives the 16 rows and the queries the 8
// columns, so that up to 8 rows (4 query heads of a key head, say) waste nothing and each 4-bit number is turned into fp16 once for
// them. In both, one ldmatrix of 8 keys x 32 features leaves each lane a word whose four nibbles are four fragments: nibble n of its
// halves is a pair of neighbouring k for K (features 8 t + n and 8 t + n + 4), of neighbouring keys for V (transposed), as
// the products want them; queries and results follow that order of the features. A pair of nibbles becomes a pair of fp16
// numbers by one and-or (1024 + c, or 1024 + 16 c for the odd nibbles) and one add or multiply-add that is exact.
//
// Scales: K's multiplies the sums of its 32 features (fp32), V's goes onto the probabilities (one packed multiplication for 32
// features x 2 keys), relative to the largest power of two met so far, so that P times the scale keeps fp16's precision down to 2^-28 of the
// largest. P^T's fragment is S^T's transposed, one movmatrix for 8 keys. Queries are fp16, as in attn_decode.cu over e4m3.
//
// Measured in a captured graph: one token of each of 128 sequences, 1,000,000 bf16 positions together, 32 query and 8 key heads, d = 128: 238 us
// (1.09 GB, 4.6 TB/s), 167 at d = 64. On half of the positions the warps issue in 63% of the cycles (69% at d = 64), the integer
// pipe in 52%, and 32 keys of a warp are 731 instructions, some 400 of them unpacking and products: that, not memory (55%), sets the
// pace. Four tokens of each of 40 sequences, 400,000 positions, 8 and 2 heads of 64: 38 us; one over 4,001 positions 12 us (the torch
// calls some 2 us more).
#include <math.h>
#include <string.h>

#include "attn_common.cuh"
#include "cqsa_internal.h"
#include "decode_common.cuh"
#include "seq_common.cuh"
#include "sm103_ptx.cuh"

namespace cqsa {
namespace {

__device__ DevErr g_decode4_err;

// NT: column tiles of 8 rows that a warp takes, NMT: groups of warps that take further rows.
template <int D, int NT, int NMT>
struct Dec4Cfg {
  static constexpr int KT = kDecode4Tile, KW = KT / kQuarters;  // keys of a tile, of a warp
  static constexpr int ROWB = D / 2, SPK = D / 32;              // bytes of a vector's codes, its scales
  static constexpr uint32_t TILE = KT * ROWB, SCALES = KT * SPK;
  static constexpr uint32_t STAGE = 2 * (TILE + SCALES);
  static constexpr int ROWS = 8 * NT;
  static constexpr int LDO = D + 4;   // row of the joining buffer, which also holds a warp's running sum, D / 4 values a lane and column tile
  static constexpr uint32_t JOIN = static_cast<uint32_t>(NMT) * kQuarters * ROWS * LDO * 4;
  static constexpr uint32_t ML = NMT * kQuarters * 2 * ROWS * 4;
  // a warp's scales of a tile: K's in fp32 by keys, V's in fp16 by 32 features, in the order of the second product's operand
  static constexpr uint32_t WSC = KW * SPK * 6, WSCALES = NMT * kQuarters * WSC;
  static constexpr int OCC = decode4_occ(ROWS * NMT, D);
  static constexpr int NST_MAX = static_cast<int>((233472 / OCC - 1024 - 1024 - 256 - JOIN - ML - WSCALES) / STAGE);
  static constexpr int NST = NST_MAX > 8 ? 8 : NST_MAX;
  static constexpr uint32_t SMEM = 1024 + NST * STAGE + JOIN + ML + WSCALES + 256;
  static constexpr int NTHR = 32 + 32 * kQuarters * NMT;
  static constexpr int FOLD = 16384 / KT;  // tiles between folds of O into the running sum, as in attn_decode.cu
  static_assert(SMEM <= 232448 && NST >= 2, "shared memory exceeds 227 KiB");
  static_assert(32 * NT * D / 4 <= ROWS * LDO, "the running sum does not fit the joining buffer");
  static_assert(STAGE % 512 == 0, "a stage does not begin where its swizzle does");
};

// Byte offset of 16-byte chunk c of row r under TMA's 64-byte (32-byte for 32-byte rows) swizzle.
template <int ROWB>
__device__ __forceinline__ uint32_t sw4_off(int r, int c) {
  if (ROWB == 64) return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return static_cast<uint32_t>(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

// Constants of the conversion below, in registers that the compiler does not know the values of (it would load them anew for every word).
struct Magic {
  uint32_t base, sub0, mul1, sub1;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(base));  // 1024, 1024
    asm volatile("mov.b32 %0, 0xe408e408;" : "=r"(sub0));  // -1032, -1032
    asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(mul1));  // 1 / 16, 1 / 16
    asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(sub1));  // -72, -72
  }
};

// The four pairs of whole numbers of a word, nibble n of both halves in x[n], as fp16 (exact).
__device__ __forceinline__ void nibbles(const Magic& k, uint32_t w, uint32_t (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(lo) : "r"(w), "r"(k.base));  // (w & mask) | base
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(hi) : "r"(w), "r"(k.base));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(x[2 * i]) : "r"(lo), "r"(k.sub0));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x[2 * i + 1]) : "r"(hi), "r"(k.mul1), "r"(k.sub1));
    w >>= 8;
  }
}

// A product whose sums begin at zero (named so, the zeros take no registers).
__device__ __forceinline__ void mma16816_from0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transposed8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void ld_shared_n(uint32_t a, uint32_t (&r)[N]) {
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  else
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void st_shared_u16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(v)) : "memory");
}
// A key's scale bytes, one for each 32 features.
template <int SPK>
__device__ __forceinline__ uint32_t scales_of(uint32_t base, int key) {
  return SPK == 4 ? ld_shared_u32(base + key * 4) : ld_shared_u16(base + key * 2);
}

// Where a key's value scale for the first 32 features lies in a warp's: key 16 j + 8 x + 2 t + e at [32 features][t][j][x][e].
template <int KW>
__device__ __forceinline__ uint32_t scale_at(uint32_t wv, int key) {
  return wv + ((key >> 1) & 3) * (KW / 2) + (key >> 3) * 4 + (key & 1) * 2;
}

template <int D, int BF16, int NT, int NMT>
__global__ void __launch_bounds__(Dec4Cfg<D, NT, NMT>::NTHR, Dec4Cfg<D, NT, NMT>::OCC)
    decode4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecParams p) {
  using C = Dec4Cfg<D, NT, NMT>;
  constexpr int KT = C::KT, KW = C::KW, NST = C::NST, NTHR = C::NTHR, ROWS = C::ROWS, SPK = C::SPK;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* join = reinterpret_cast<float*>(sm + NST * C::STAGE);
  float* ml = join + C::JOIN / 4;  // [NMT][kQuarters][m ROWS | l ROWS]
  uint8_t* wsc = reinterpret_cast<uint8_t*>(ml) + C::ML;  // [NMT * kQuarters][K's floats | V's halves]
  uint64_t* full = reinterpret_cast<uint64_t*>(wsc + C::WSCALES);
  uint64_t* empty = full + NST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NST);
  long long* s_base = reinterpret_cast<long long*>(empty + NST + 1);
  int* s_seq = reinterpret_cast<int*>(s_base + 1);
  long long* s_warp = reinterpret_cast<long long*>(s_seq + 2);  // [NTHR / 32]

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
  const Range rg = find_range<KT, NTHR>(p, s_warp, s_base, s_seq);
  const long long W = rg.all, nc = rg.ctas, w0 = rg.begin, w1 = rg.end;
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
  } else if (warp == NTHR / 32 - 1) {
    // ------------------------------------------------------------------ producer warp
    if (lane == 0) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
    const int page = 1 << p.page_log2;
    const int rows = min(page, KT);  // rows of a box
    const int boxes = KT / rows;     // page boxes of a tile
    int it = 0;
    bool ok = true;
    for (long long w = w0; ok && w < w1;) {
      const Piece pc = piece_at(wk, w, w1);
      const int h = pc.h, t0 = pc.t0, t1 = pc.t1;
      const int* row = p.table + wk.s * p.row_seq + h * p.row_head;
      for (int t = t0; ok && t < t1; ++t, ++it) {
        const int stage = it % NST;
        if (it >= NST)
          ok = wait_or_abort(smem_u32(&empty[stage]), ((it / NST) - 1) & 1u, p.timeout_us, a_abort, &g_decode4_err,
                             kDevTimeoutKV, 40);
        if (!ok) break;
        if (p.fault == 1 && wk.s == 0 && h == 0 && t == 0) {  // (every wait on the tile runs out)
          ok = false;
          break;
        }
        uint8_t* st = sm + stage * C::STAGE;
        const int k0 = t * KT;
        const int nb = min(boxes, max(0, (wk.len - k0 + rows - 1) >> (31 - __clz(rows))));
        if (lane == 0) mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(nb) * rows * 2 * (C::ROWB + SPK));
        __syncwarp();
        for (int i = lane; i < nb; i += 32) {
          const int pos = k0 + i * rows;
          const int pg = page_at(row, pos >> p.page_log2, p.n_pages), y = pos & (page - 1);
          const uint32_t off = static_cast<uint32_t>(i * rows) * C::ROWB;
          const int block = pg * p.Hkv + h;
          tma_load_3d(st + off, &tmK, &full[stage], 0, y, block);
          tma_load_3d(st + C::TILE + off, &tmV, &full[stage], 0, y, block);
          const long long at = ((static_cast<long long>(block) << p.page_log2) + y) * SPK;
          uint8_t* sc = st + 2 * C::TILE + i * rows * SPK;
          bulk_load(sc, p.k_scale + at, rows * SPK, &full[stage]);
          bulk_load(sc + C::SCALES, p.v_scale + at, rows * SPK, &full[stage]);
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
    const int mt = warp / kQuarters, kg = warp % kQuarters;  // group of rows, quarter of the keys
    const int g = lane >> 2, t4 = lane & 3;
    float* jbuf = join + mt * kQuarters * ROWS * C::LDO;
    float* mlb = ml + mt * kQuarters * 2 * ROWS;
    const Magic magic;
    const uint32_t wk32 = smem_u32(wsc) + warp * C::WSC, wv = wk32 + KW * SPK * 4;
    bool ok = true;
    int stage = 0;
    uint32_t parity = 0;
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
      // ---- this lane's queries (row g of each column tile, 8 features of every 32), and what its two columns (rows 2 t4, 2 t4 + 1) see
      const int pos0 = seq_first_position(p.kv_lens, wk.s, wk.qlen);
      uint32_t qf[NT][D / 32][4];
      int lim[NT][2];
      float rs[NT][2];  // factor from a raw score to the base-2 exponent
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = (mt * NT + nt) * 8 + g, tok = r / p.G;
        const bool valid = tok < wk.qlen;
        const uint16_t* qr = static_cast<const uint16_t*>(p.q) + static_cast<long long>(wk.first + tok) * p.q_stride +
                             static_cast<long long>(h * p.G + (r - tok * p.G)) * D + 8 * t4;
        uint4 x[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) x[c] = valid ? __ldg(reinterpret_cast<const uint4*>(qr + c * 32)) : make_uint4(0, 0, 0, 0);
        int e = 0;
        if (BF16) {
          float amax = 0.0f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t ws[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack16(ws[i], 1);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // 2^-e brings the row's largest value into [1, 2); held to the exponents whose inverse is normal
          e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
          const float inv = pow2i(-e);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ws[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack16(ws[i], 1);
              ws[i] = pack16(f.x * inv, f.y * inv, 0);
            }
            x[c] = make_uint4(ws[0], ws[1], ws[2], ws[3]);
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // features 8 t4 + n and 8 t4 + 4 + n
          qf[nt][c][0] = __byte_perm(x[c].x, x[c].z, 0x5410);
          qf[nt][c][1] = __byte_perm(x[c].x, x[c].z, 0x7632);
          qf[nt][c][2] = __byte_perm(x[c].y, x[c].w, 0x5410);
          qf[nt][c][3] = __byte_perm(x[c].y, x[c].w, 0x7632);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tk = ((mt * NT + nt) * 8 + 2 * t4 + u) / p.G;
          lim[nt][u] = tk >= wk.qlen ? 0 : (p.causal ? min(wk.len, pos0 + tk + 1) : wk.len);
          rs[nt][u] = p.scale_log2;
          if (BF16) rs[nt][u] *= pow2i(__shfl_sync(0xffffffffu, e, (2 * t4 + u) * 4));
        }
      }
      const int lim_all = p.causal ? pos0 + 1 : wk.len;  // keys that every row sees
      float o[NT][D / 32][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) o[nt][c][i >> 2][i & 3] = 0.0f;
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          m[nt][u] = -INFINITY;
          l[nt][u] = 0.0f;
        }
      int ev = -1;  // exponent (biased by 15) of the value scales that the output sums are relative to
      // The running sum that O is folded into: this lane's values, and the references of the rows and of the values' scales that they are
      // relative to. (The layout of the join below is another, and is written after the next named_sync.)
      float* sum = jbuf + kg * ROWS * C::LDO + lane;
      float* refs = mlb + kg * 2 * ROWS;
      auto sum_factor = [&](int nt, int u) -> float {
        const float was = refs[nt * 8 + 2 * t4 + u], a = was == -INFINITY ? 0.0f : ex2(was - m[nt][u]);
        return a * exp2_int_any(__float_as_int(refs[ROWS]) - ev);
      };
      for (int t = t0; t < t1; ++t) {
        if (t > t0 && (t - t0) % C::FOLD == 0) {
          const bool have = t - t0 > C::FOLD;
          if (!have) named_sync(1 + mt, 32 * kQuarters);  // the unit before has been read out of the buffer
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float fs[2] = {have ? sum_factor(nt, 0) : 0.0f, have ? sum_factor(nt, 1) : 0.0f};
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float* at = sum + ((nt * (D / 32) + c) * 8 + i) * 32;
                float& x = o[nt][c][i >> 2][i & 3];
                *at = (have ? *at * fs[i & 1] : 0.0f) + x;
                x = 0.0f;
              }
          }
          __syncwarp();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (g == 0) *reinterpret_cast<float2*>(refs + nt * 8 + 2 * t4) = make_float2(m[nt][0], m[nt][1]);
          if (lane == 0) refs[ROWS] = __int_as_float(ev);
          __syncwarp();
        }
        if (ok) ok = wait_or_abort(smem_u32(&full[stage]), parity, p.timeout_us, a_abort, &g_decode4_err,
                                   kDevTimeoutKV, 41);
        const uint32_t sk = smem_u32(sm) + stage * C::STAGE, sv = sk + C::TILE;
        const int kw0 = kg * KW;                 // first key of this warp in the tile
        const int k0 = t * KT + kw0;             // its position
        const int left = wk.len - k0;            // positions of the sequence from there
        const uint32_t ksc = sk + 2 * C::TILE + kw0 * SPK, vsc = ksc + C::SCALES;
        // ---- each lane turns one key's scales into numbers for its warp.
        // V's are relative to 2^(ev - 15), the largest power of two met so far.
        {
          uint32_t kword = scales_of<SPK>(ksc, lane), vword = scales_of<SPK>(vsc, lane);
          if (lane >= left) kword = vword = 0u;  // slots past the end hold anything
          uint32_t ve = vword & 0x00ff00ffu, vo = (vword >> 8) & 0x00ff00ffu, nan[2] = {0u, 0u};
          auto largest = [&]() -> uint32_t {
            const uint32_t most = __vmaxu2(ve, vo);
            return __reduce_max_sync(0xffffffffu, SPK == 4 ? max(most & 0xffffu, most >> 16) : most);
          };
          uint32_t top = largest();
          if (top > 247u) {  // a NaN is no size that the numbers beside it could be relative to
            nan[0] = __vcmpgtu2(ve, 0x00f700f7u);
            nan[1] = __vcmpgtu2(vo, 0x00f700f7u);
            ve &= ~nan[0];
            vo &= ~nan[1];
            top = largest();
          }
          top >>= 3;
          if (static_cast<int>(top) > ev) {
            const float a = ev < 0 ? 0.0f : exp2_int_any(ev - static_cast<int>(top));
            ev = static_cast<int>(top);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < D / 32; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[nt][c][i >> 2][i & 3] *= a;
          }
          // As fp16 numbers relative to that power their exponents move by 15 - ev. Those 15 powers and more below it would not be normal numbers:
          // they are 0 here, and a round of their own (below).
          const uint32_t up = static_cast<uint32_t>(15 - ev) * 0x04000400u;
          uint32_t h[2] = {ve * 128u + up, vo * 128u + up};
          if (__builtin_expect(ev >= 15, 0)) {
            const uint32_t down = static_cast<uint32_t>(ev - 15) * 0x00080008u;
            h[0] = (__vsub2(ve, down) & __vcmpgeu2(ve, down + 0x00080008u)) * 128u;
            h[1] = (__vsub2(vo, down) & __vcmpgeu2(vo, down + 0x00080008u)) * 128u;
          }
          h[0] |= nan[0];
          h[1] |= nan[1];
          const uint32_t vat = scale_at<KW>(wv, lane);
          st_shared_u16(vat, h[0]);
          st_shared_u16(vat + 2 * KW, h[1]);
          // K's as bf16 numbers, the upper halves of fp32 ones, two bytes at a time. With 112 more as its exponent a byte from 248 on is
          // an infinity or a NaN: times 2^-112, and plus 0 times itself, it is a NaN, and the others are what they stand for. (A test for
          // the former takes 244 us where this takes 242.)
          auto units = [](uint32_t bytes) -> uint32_t {
            uint32_t r;
            asm("{.reg .b32 z;\n\tmul.rn.bf16x2 z, %1, %2;\n\tfma.rn.bf16x2 %0, %1, %3, z;}" : "=r"(r) : "r"(bytes * 16u + 0x70007000u), "r"(0u), "r"(0x07800780u));
            return r;
          };
          const uint32_t ke = units(__byte_perm(kword, 0, 0x4240)), ko = units(__byte_perm(kword, 0, 0x4341));
          float f[4] = {__uint_as_float(ke << 16), __uint_as_float(ko << 16), __uint_as_float(ke & 0xffff0000u), __uint_as_float(ko & 0xffff0000u)};
          if (SPK == 4) {
            st_shared_u16(vat + 4 * KW, h[0] >> 16);
            st_shared_u16(vat + 6 * KW, h[1] >> 16);
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(wk32 + lane * 16), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]) : "memory");
          } else {
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(wk32 + lane * 8), "f"(f[0]), "f"(f[1]) : "memory");
          }
          __syncwarp();
        }
        // ---- S^T = K Q^T, 16 keys and 32 features at a time, each 32 features' sums times their key's scale
        float s[KW / 16][NT][4];
#pragma unroll
        for (int j = 0; j < KW / 16; ++j) {
          uint32_t fa[SPK], fb[SPK];
          ld_shared_n<SPK>(wk32 + (j * 16 + g) * (4 * SPK), fa);
          ld_shared_n<SPK>(wk32 + (j * 16 + 8 + g) * (4 * SPK), fb);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t b[4];
            ldsm4(sk + sw4_off<C::ROWB>(kw0 + j * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), c * 2 + (lane >> 4)), b);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int gr = 2 * c + x;
              uint32_t lo[4], hi[4];  // keys 0-7 and 8-15
              nibbles(magic, b[2 * x], lo);
              nibbles(magic, b[2 * x + 1], hi);
              const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float acc[4];
                mma16816_from0(acc, a0, qf[nt][gr][0], qf[nt][gr][1]);
                mma16816<0>(acc, a1, qf[nt][gr][2], qf[nt][gr][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float f = __uint_as_float(i < 2 ? fa[gr] : fb[gr]);
                  s[j][nt][i] = gr == 0 ? acc[i] * f : fmaf(acc[i], f, s[j][nt][i]);
                }
              }
            }
          }
        }
        // ---- scores in base 2, masks, running maximum, P^T (rounded to fp16) as the second product's operand
        // (rows behind the unit's last have queries of zero, and are not written)
        const bool mask = left < KW || k0 + KW > lim_all;
        uint32_t pf[KW / 16][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < KW / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j][nt][i] *= rs[nt][i & 1];
          if (mask) {
#pragma unroll
            for (int j = 0; j < KW / 16; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k0 + j * 16 + (i >> 1) * 8 + g >= lim[nt][i & 1]) s[j][nt][i] = -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < KW / 16; ++j) {
            mx[0] = max3(mx[0], s[j][nt][0], s[j][nt][2]);
            mx[1] = max3(mx[1], s[j][nt][1], s[j][nt][3]);
          }
          float al[2], mu[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], of));
            // The reference may lie up to 1 below the largest score: 2^15 p times a scale below 2 stays below fp16's largest, and rows in
            // mid-sequence rescale O less often.
            const float was = m[nt][u];
            const bool up = mx[u] > was + 1.0f;
            if (up) m[nt][u] = mx[u];
            al[u] = up ? ex2(was - mx[u]) : 1.0f;  // (0 for a row that has seen nothing yet)
            mu[u] = (m[nt][u] == -INFINITY ? 0.0f : m[nt][u]) - kPShift;
            l[nt][u] *= al[u];
          }
          if (__any_sync(0xffffffffu, al[0] != 1.0f || al[1] != 1.0f)) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
              for (int i = 0; i < 8; ++i) o[nt][c][i >> 2][i & 3] *= al[i & 1];
          }
#pragma unroll
          for (int j = 0; j < KW / 16; ++j) {
            float pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              pr[i] = ex2(s[j][nt][i] - mu[i & 1]);
              l[nt][i & 1] += pr[i];
            }
            pf[j][nt][0] = transposed8x8(pack16(pr[0], pr[1], 0));
            pf[j][nt][1] = transposed8x8(pack16(pr[2], pr[3], 0));
          }
        }
        // ---- O^T += V^T P^T, P (times 2^-15 where `far`) times the values' scales
        auto multiply = [&](bool far) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t sc[2][KW / 8];  // scales of this lane's keys for two times 32 features: [j][x] pairs of 2 t4, 2 t4 + 1
            ld_shared_n<KW / 8>(wv + (2 * c) * (2 * KW) + t4 * (KW / 2), sc[0]);
            ld_shared_n<KW / 8>(wv + (2 * c + 1) * (2 * KW) + t4 * (KW / 2), sc[1]);
#pragma unroll
            for (int j = 0; j < KW / 16; ++j) {
              uint32_t b[4];
              ldsm4t(sv + sw4_off<C::ROWB>(kw0 + j * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), c * 2 + (lane >> 4)), b);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int gr = 2 * c + x;
                uint32_t lo[4], hi[4];
                nibbles(magic, b[2 * x], lo);
                nibbles(magic, b[2 * x + 1], hi);
                const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]}, a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t p0 = mul2(far ? mul2(pf[j][nt][0], 0x02000200u) : pf[j][nt][0], sc[x][2 * j]);
                  const uint32_t p1 = mul2(far ? mul2(pf[j][nt][1], 0x02000200u) : pf[j][nt][1], sc[x][2 * j + 1]);
                  mma16816<0>(o[nt][gr][0], a0, p0, p1);
                  mma16816<0>(o[nt][gr][1], a1, p0, p1);
                }
              }
            }
          }
        };
        // Where the largest scale's power is 1 or more others may lie 15 powers and more below it. A round by themselves takes them
        // times 2^15, with P times 2^-15: P times a scale is the same, and P is exact from 2^-13 on, below which these are under 2^-28 of
        // the largest scale's power. (Before the main round, so that what it needs is not held beside that one's sums: a call for 128
        // sequences of 1,000,000 positions takes 241 us, 244 with this round behind it, 238 without it.)
        if (__builtin_expect(ev >= 15, 0)) {
          int key;  // (the lane, read anew: nothing is kept in registers for this)
          asm volatile("mov.u32 %0, %%laneid;" : "=r"(key));
          const uint32_t vword = scales_of<SPK>(vsc, key), vat = scale_at<KW>(wv, key);
          bool some = false;
          uint32_t x[SPK];
#pragma unroll
          for (int i = 0; i < SPK; ++i) {
            const uint32_t b = (vword >> (8 * i)) & 255u, man = (b & 7u) << 7;
            const int e = static_cast<int>(b >> 3) - ev;
            const bool is = key < left && e <= -15;
            x[i] = is ? (e > -30 ? static_cast<uint32_t>(e + 30) << 10 | man : (0x400u | man) >> 1) : 0u;  // (-30: fp16's numbers there have no leading 1)
            some |= is;
          }
          if (__any_sync(0xffffffffu, some)) {
#pragma unroll
            for (int i = 0; i < SPK; ++i) {
              const uint32_t kept = ld_shared_u16(vat + i * (2 * KW));
              st_shared_u16(vat + i * (2 * KW), x[i]);
              x[i] = kept;
            }
            __syncwarp();
            multiply(true);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < SPK; ++i) st_shared_u16(vat + i * (2 * KW), x[i]);
            __syncwarp();
          }
        }
        multiply(false);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == NST) {
          stage = 0;
          parity ^= 1u;
        }
      }
      if (t1 - t0 > C::FOLD) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float fs[2] = {sum_factor(nt, 0), sum_factor(nt, 1)};
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) o[nt][c][i >> 2][i & 3] += sum[((nt * (D / 32) + c) * 8 + i) * 32] * fs[i & 1];
        }
      }
      // ---- join the warps' rows: each brings its sums to the common maximum and scale (the values' reference is a power of
      // two that is multiplied out here)
      __syncwarp();  // (the sum's references lie where the rows' go)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) l[nt][u] += __shfl_xor_sync(0xffffffffu, l[nt][u], of);
          if (g == 0) {
            mlb[kg * 2 * ROWS + nt * 8 + 2 * t4 + u] = m[nt][u];
            mlb[kg * 2 * ROWS + ROWS + nt * 8 + 2 * t4 + u] = l[nt][u];
          }
        }
      named_sync(1 + mt, 32 * kQuarters);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int row = nt * 8 + 2 * t4 + u;
          float M = -INFINITY, L = 0.0f;
#pragma unroll
          for (int i = 0; i < kQuarters; ++i) M = fmaxf(M, mlb[i * 2 * ROWS + row]);
          const float Mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
          for (int i = 0; i < kQuarters; ++i) L += mlb[i * 2 * ROWS + ROWS + row] * ex2(mlb[i * 2 * ROWS + row] - Mu);
          float f = L > 0.0f ? ex2(m[nt][u] - Mu) / L : (L != L ? NAN : 0.0f);
          f *= ev < 0 ? 0.0f : exp2_int_any(ev - 15);
          float* at = jbuf + (kg * ROWS + row) * C::LDO;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float4 y = make_float4(o[nt][c][0][u] * f, o[nt][c][0][2 + u] * f, o[nt][c][1][u] * f, o[nt][c][1][2 + u] * f);
            if (f == 0.0f) y = make_float4(0, 0, 0, 0);  // (a row that sees nothing, beside values that are not finite)
            *reinterpret_cast<float4*>(at + c * 32 + 4 * g) = y;
          }
          if (kg == 0 && g == 0)  // a column of the padding carries the rows' lse
            at[D] = L > 0.0f ? M - kPShift + log2f(L) : (L != L ? NAN : -INFINITY);
        }
      named_sync(1 + mt, 32 * kQuarters);
      const bool whole = t0 == 0 && t1 == wk.n - kUnit;
      const long long slot = 2 * static_cast<long long>(blockIdx.x) + (t0 == 0 ? 1 : 0);
      for (int e = kg * 32 + lane; e < ROWS * (D / 4); e += 32 * kQuarters) {
        const int row = e / (D / 4), c = e % (D / 4);
        const int r = mt * ROWS + row, tok = r / p.G;
        if (tok >= wk.qlen || !ok) continue;
        float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kQuarters; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(jbuf + (i * ROWS + row) * C::LDO + c * 4);
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
          reinterpret_cast<float4*>(p.part_o)[(slot * (ROWS * NMT) + r) * (D / 4) + c] = a;
          if (c == 0) p.part_l[slot * (ROWS * NMT) + r] = jbuf[row * C::LDO + D];
        }
      }
      w = pc.next;
      if (w < w1 && h == p.Hkv - 1) walk_next<KT>(p, wk);
    }
  }
  __syncthreads();
}

template <int D, int BF16, int NT, int NMT>
int launch4_t(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int ctas, cudaStream_t stream) {
  using C = Dec4Cfg<D, NT, NMT>;
  auto kern = decode4_kernel<D, BF16, NT, NMT>;
  static PerDeviceOnce attr;
  int dev = 0;
  if (!attr.done(&dev)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(4-bit paged attention smem)");
    attr.mark(dev);
  }
  kern<<<ctas, C::NTHR, C::SMEM, stream>>>(mk, mv, p);
  const int rc = cuda_status(cudaGetLastError(), "4-bit paged attention kernel launch");
  return rc == CQSA_OK ? launch_combine<D, BF16>(p, 8 * NT * NMT, ctas, stream) : rc;
}

template <int D, int BF16>
int launch4_d(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int rows, int ctas, cudaStream_t s) {
  if (rows == 8) return launch4_t<D, BF16, 1, 1>(mk, mv, p, ctas, s);
  return rows == 16 ? launch4_t<D, BF16, 2, 1>(mk, mv, p, ctas, s) : launch4_t<D, BF16, 2, 2>(mk, mv, p, ctas, s);
}

}  // namespace

int launch_decode4(const CUtensorMap& mk, const CUtensorMap& mv, const DecParams& p, int d, int bf16, int rows, int ctas,
                   cudaStream_t stream) {
  if (d == 64) return bf16 ? launch4_d<64, 1>(mk, mv, p, rows, ctas, stream) : launch4_d<64, 0>(mk, mv, p, rows, ctas, stream);
  return bf16 ? launch4_d<128, 1>(mk, mv, p, rows, ctas, stream) : launch4_d<128, 0>(mk, mv, p, rows, ctas, stream);
}

DEV_ERR_READERS(decode4, g_decode4_err)

}  // namespace cqsa
