// Attention forward on the tensor cores for sequences of different lengths with grouped heads: whole prompts
// packed end to end (cqsa_attn_packed_fwd), and chunks of new tokens over a paged cache, 16-bit or e4m3
// (cqsa_attn_paged_fwd with more than 32 rows per sequence and key head).
//
// The pipeline is attn_fwd2_kernel's (attn_fwd.cu): TMA producer, one MMA-issuing warp per query tile, one
// softmax warpgroup per query tile, tcgen05 products accumulating in tensor memory, a running reference
// maximum that moves by whole numbers with rare exact rescales. What differs:
//   Rows     a tile's 128 rows are floor(128 / G) tokens times the G query heads of one key head (row
//            r = token r / G, head r % G), loaded by one 3-D TMA box, so that a short sequence or chunk fills tiles G
//            times better and K/V are loaded once for the whole group.
//   Units    two row tiles of one (sequence, key head). One CTA per SM works through several, the next one's loads and
//            first products beside the end of the last. Packed prompts: units are found from cu_seqlens alone, ranked by
//            their place in their sequence, the latest (under the causal mask the heaviest) first.
//   Ranges   chunks over a long cache have few units of very different lengths, so the key tiles of all units, laid end
//            to end, are cut into one equal range per CTA, as attn_decode.cu does: a range's whole units are written out, the
//            two others leave normalised fp32 parts that seq_combine_kernel joins. (Whole units, or every unit in the same
//            number of ranges: 787 us against 712 for 256 units of 266 tiles, 135 against 86 for 12 ragged e4m3 sequences.)
//   P        is rounded once to dtype for P V (2^-8 relative for bf16, as the output is; attn_fwd.cu's
//            hi/lo split, half as many products again, serves fp32 partial results), scaled by 2^6 so that
//            fp16 keeps its relative precision down to p = 2^-19 of the row's largest at least (the reference may lie
//            up to 1 above the row's maximum).
//   Tails    rows of V past a sequence's end (another sequence's tokens, or whatever an unused slot holds) are zeroed in
//            shared memory before the product: p = 0 does not hide an infinity or NaN there.
//   e4m3     the producer copies code vectors as they lie in the pages, and four converter warps turn them into
//            swizzled fp16 tiles, each key relative to the largest power of two met so far (exact but for values 2^-15
//            below it). K's power goes into the scores' scale; V's is a reference that O is rescaled to when it rises.
//            Queries are fp16: bf16 ones are first scaled to [1, 2) by a power of two per row, in place.
//
// Measured, a pass among others whose inputs L2 does not hold: one causal prompt of 32,768 tokens, 8 query and 2 key heads, d = 64, fp16:
// 1,014 us, 1,085 TFLOP/s; 24 ragged prompts of 16,384 tokens together, 32 and 8 heads, d = 128, bf16: 219 us, 1,050 TFLOP/s; 2,048
// tokens over 32,000 positions of 16-bit pages, 32 and 8 heads, d = 128: 765 us, 1,450 TFLOP/s (705 in a loop on one input; over e4m3
// ones 1,195 there); 12 ragged e4m3 sequences (3,000 tokens over 60,000, 8 and 2 heads, d = 64): 81 us. Long rows are bound by the softmax warps' chain of a key tile (tensor-memory loads, row
// maximum, 128 exponentials, P back) beside the products it waits for: the tensor pipe is 69% busy at d = 128 and 46% at
// d = 64; short units add about three key tiles' time each for their start and end. e4m3: the converters take issue slots
// from the softmax warps of their sub-partitions.
#include <math.h>
#include <string.h>

#include "attn_common.cuh"
#include "cqsa_internal.h"
#include "seq_common.cuh"
#include "sm103_ptx.cuh"

namespace cqsa {
namespace {

__device__ DevErr g_seq_err;

constexpr int BN = 128;  // keys per tile
constexpr uint32_t TILE_BYTES = 128 * 64 * 2;  // one 128 x 64 box of 16-bit elements
constexpr uint32_t TMEM_COLS = 512;
// Probabilities (and their sums) are kept as 2^6 p relative to a reference that may lie up to 2^8 below a row's
// largest score before it is raised: rows in mid-sequence then almost never rescale O (each rescale reads and writes
// d columns of tensor memory, and the slowest of a tile's warps sets its pace), and fp16's range holds
// 2^14 above and, with full precision, 2^-14 below.
constexpr float kPShift = 6.0f, kTau = 8.0f;

enum : int { kSrcPacked = 0, kSrcPages = 1, kSrcE4m3 = 2, kSrcInt4 = 3 };

template <int D, int SRC>
struct SeqCfg {
  static constexpr bool INT4 = SRC == kSrcInt4, CONV = SRC == kSrcE4m3 || INT4;
  // P over S where tensor memory (d = 128) or registers (beside the converter warps) leave no room for both
  static constexpr bool ALIAS = D == 128 || CONV;
  static constexpr int KSUB = D / 64;
  // K and V tiles in shared memory, in atoms of 8 keys x 64 features (1 KiB, 128-byte swizzle). A page arrives as one
  // five-dimensional box, [8 keys][half][8][64 features]; packed tokens and converted tiles as [half][128 keys][64].
  static constexpr bool BY8 = SRC == kSrcPages;
  static constexpr uint32_t GROUP = BY8 ? 1024u * (D / 64) : 1024u;   // from 8 keys to the next 8
  static constexpr uint32_t HALF = BY8 ? 1024u : TILE_BYTES;          // from features 0-63 to 64-127
  static constexpr int STAGES = D == 64 ? (CONV ? 3 : 4) : 2;
  static constexpr uint32_t QT_BYTES = KSUB * TILE_BYTES;
  static constexpr uint32_t KV_BYTES = KSUB * TILE_BYTES;
  static constexpr uint32_t COL_S0 = 0, COL_S1 = 128;
  static constexpr uint32_t COL_P0 = ALIAS ? 0u : 256u, COL_P1 = ALIAS ? 128u : 320u;
  static constexpr uint32_t COL_O0 = ALIAS ? 256u : 384u, COL_O1 = COL_O0 + D;
  static constexpr int NBARS = 1 + 4 * STAGES + 2 * 7 + 2 + 2 + 4 + 6;
  // key tiles between folds of O into the fp32 running sum (attn_fwd.cu explains why): in shared memory
  // for d = 64, in the SM's slot of attn_fwd.cu's array for d = 128
  static constexpr int FLUSH = D == 64 ? 128 : 32;
  static constexpr bool OSUM_SMEM = D == 64;
  static constexpr uint32_t OSUM_BYTES = OSUM_SMEM ? 2u * D * 128u * 4u : 0u;
  // Results leave through 4 KiB of shared memory per softmax warp, so that a store covers whole lines: a thread's own row
  // written 16 bytes at a time costs a wavefront per lane. d = 64 takes the running sum's place when it is not in use.
  static constexpr bool STAGED = OSUM_SMEM || !CONV;
  static constexpr uint32_t OUT_BYTES = STAGED && !OSUM_SMEM ? 8u * 4096u : 0u;
  static constexpr uint32_t ROW = INT4 ? D / 2 : D;      // bytes of a vector's codes
  static constexpr uint32_t RAW = CONV ? 128u * ROW : 0u;  // a K or V tile's codes as they lie in the pages
  // running exponents per tile, factors of the queries' rows, the converter warps' largest exponents
  static constexpr uint32_t EXP_BYTES = CONV ? 2u * STAGES * 2u * 4u + 512u + 64u : 0u;
  static constexpr uint32_t SMEM_BYTES = 1024 + 2 * QT_BYTES + 2 * STAGES * KV_BYTES + OSUM_BYTES + OUT_BYTES + 2 * RAW + EXP_BYTES + NBARS * 8 + 112;
  static_assert(SMEM_BYTES <= 232448, "shared memory exceeds 227 KiB");
  static_assert(COL_O1 + D <= TMEM_COLS, "tensor memory layout exceeds 512 columns");
  // setmaxnreg shares of warpgroup 0, the two softmax warpgroups and the converters
  static constexpr int NTHR = CONV ? 512 : 384;
  static constexpr int LAUNCH_REGS = CONV ? 128 : 168;
  // (e4m3: with 192 for the softmax it spills in its loop, 1,720 us against 1,322 on a 2,048-token chunk at d = 128)
  static constexpr int LOW = CONV ? 40 : 72, HIGH = CONV ? (D == 64 ? 208 : 200) : 216, CVT = D == 64 ? 56 : 72;
  static_assert(128 * LOW + 256 * HIGH + (CONV ? 128 * CVT : 0) <= NTHR * LAUNCH_REGS, "register split exceeds the launch allocation");
};

// What a CTA works on next, as its scheduling warp hands it to the others.
struct Work {
  int valid, seq, tok_first, qlen, kvlen, ta, hk;  // two row tiles from token ta of the sequence's
  int jb, je;                                      // key tiles [jb, je) of those the row tiles see
  int slot, pos0, pad;                             // where a part goes (-1: the whole unit, to the output); position of the sequence's first token
};

// A chunk's units weigh as many as the key tiles they see (one at least, for the rows that see nothing) and kUnitWeight
// more, about what a unit costs beside them; a range weighs kLeastRange at least.
constexpr int kUnitWeight = 2, kLeastRange = 6;
constexpr int kPartRows = 256;  // rows of a unit, and of a part

// sum over i in [0, n) of floor((a i + b) / m), a, b >= 0, m > 0, by the reduction that Euclid's algorithm makes of
// (a, m). All values but the sum stay below 2^32.
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long r = 0;
  while (n > 0) {
    r += static_cast<long long>(a / m) * (static_cast<long long>(n) * (n - 1) / 2) + static_cast<long long>(b / m) * n;
    a %= m;
    b %= m;
    const uint32_t top = a * n + b;
    n = top / m;
    b = top % m;
    const uint32_t x = m;
    m = a;
    a = x;
  }
  return r;
}

// The units of a sequence's new tokens over its positions, for one key head: unit i takes tokens [i per, (i + 1) per).
struct ChunkUnits {
  int seq, first, qlen, kvlen, pos0, per, units, causal;
  __device__ __forceinline__ int last(int i) const {  // the last position that unit i sees, -1 or less for none
    return causal ? min(kvlen, pos0 + min((i + 1) * per, qlen)) - 1 : kvlen - 1;
  }
  __device__ __forceinline__ int tiles(int i) const {
    const int p = last(i);
    return p < 0 ? 1 : p / BN + 1;
  }
  // what units [0, i) weigh: their last positions are an arithmetic progression up to the last that there is
  __device__ __forceinline__ long long before(int i) const {
    long long w = static_cast<long long>(i) * (kUnitWeight + 1);
    if (!causal) return w + static_cast<long long>(i) * (max(kvlen - 1, 0) / BN);
    const int rising = max(kvlen - pos0 - 1, 0) / per;  // units that end before it
    if (i > rising) {
      w += static_cast<long long>(i - rising) * (max(kvlen - 1, 0) / BN);
      i = rising;
    }
    if (i == 0) return w;
    const int a = pos0 + per - 1;
    const int skip = a < 0 ? min(i, (-a + per - 1) / per) : 0;
    return w + floor_sum(i - skip, BN, per, max(a + skip * per, 0));
  }
};

struct SeqParams {
  const int* cu;
  const int* kv_lens;  // null: a sequence's positions are its tokens (packed prompts)
  const int* table;
  const uint8_t* k_cache;  // e4m3 and 4 bits only (16-bit pages go through the tensor maps)
  const uint8_t* v_cache;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  void* out;
  float* lse;
  float* part_o;  // [phases * CTAs][2][kPartRows][D]
  float* part_l;  // [phases * CTAs][2][kPartRows], base 2
  int4* meta;     // [phases * CTAs][2] the unit a range begins in the middle of: sequence (-1: none), key head, first and last
                  // range of it; the sequence's first token and tokens, the unit's first token
  float* osum;
  int n_osum;
  int n_seqs, T, Hq, Hkv, G, tpt;  // tpt: tokens of a row tile, floor(128 / G)
  int phases, max_pages, n_pages, page_log2, causal;
  long long most;  // positions that a sequence's pages can hold
  // 4-bit pages: where a sequence's keys and values lie as 16-bit numbers, in pages of kFullPage positions of a scratch cache (-1: nowhere), or null. Kernels
  // of 16-bit pages take the sequences that do, the one of 4-bit pages the others.
  const int* full;
  float scale_log2;
  unsigned timeout_us;
  int fault;  // test hook: 1 = block 0 never loads key tile 1
};
constexpr int kFullPage = 128;

// Feature steps [K0, K1) of S = Q K^T; HALF: bytes from a K tile's first 64 features to the others.
template <int K0, int K1, uint32_t HALF>
__device__ __forceinline__ void issue_s(uint32_t dcol, uint64_t a0, uint64_t b0, uint32_t idesc) {
#pragma unroll
  for (int ks = K0; ks < K1; ++ks) {
    const uint32_t ao = static_cast<uint32_t>((ks >> 2) * (TILE_BYTES >> 4) + (ks & 3) * 2);
    const uint32_t bo = static_cast<uint32_t>((ks >> 2) * (HALF >> 4) + (ks & 3) * 2);
    if (ks == 0) mma_ss_i<0>(dcol, a0 + ao, b0 + bo, idesc);
    else mma_ss_i<1>(dcol, a0 + ao, b0 + bo, idesc);
  }
}
// Keys [16 K0, 16 K1) of O += P V; GROUP: bytes from 8 keys of a V tile to the next 8.
template <bool FIRST, int K0, int K1, uint32_t GROUP>
__device__ __forceinline__ void issue_o(uint32_t ocol, uint32_t pcol, uint64_t v0, uint32_t idesc) {
#pragma unroll
  for (int ks = K0; ks < K1; ++ks) {
    const uint64_t bd = v0 + static_cast<uint32_t>(ks) * (GROUP >> 3);
    if (FIRST && ks == 0) mma_ts_i<0>(ocol, pcol + ks * 8, bd, idesc);
    else mma_ts_i<1>(ocol, pcol + ks * 8, bd, idesc);
  }
}

// 2^k for a difference k <= 0 of two references of a row, a whole number (but for what fp32 rounds off very large ones).
__device__ __forceinline__ float exp2_whole(float k) { return exp2_int(rintf(k)); }

// 2^(x sl2 - m) for a pair of scores.
__device__ __forceinline__ float2 exp2_pair(float x0, float x1, float2 sl2v, float2 nm) {
  const float2 r = __ffma2_rn(make_float2(x0, x1), sl2v, nm);
  return make_float2(fast_exp2(r.x), fast_exp2(r.y));
}

// Zero keys [r0, 128) of a K or V tile (a whole warp): a key's row is 128 bytes of each half, and the swizzle only
// moves 16-byte pieces inside it.
template <class C>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int lane) {
#pragma unroll
  for (int x = 0; x < C::KSUB; ++x)
    for (int i = r0 * 8 + lane; i < 128 * 8; i += 32)
      st_shared_zero16(smem_u32(tile) + x * C::HALF + (i >> 6) * C::GROUP + (i & 63) * 16);
}

template <int D, int BF16, int SRC>
__global__ void __launch_bounds__(SeqCfg<D, SRC>::NTHR, 1)
    attn_seq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const SeqParams p) {
  using C = SeqCfg<D, SRC>;
  constexpr int STAGES = C::STAGES, KSUB = C::KSUB;
  constexpr bool ALIAS = C::ALIAS, CONV = C::CONV;
  constexpr int MB = CONV ? 0 : BF16;  // type of the products
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * C::QT_BYTES;
  uint8_t* sV = sK + STAGES * C::KV_BYTES;
  float* sOsum = reinterpret_cast<float*>(sV + STAGES * C::KV_BYTES);
  uint8_t* sOut = sV + STAGES * C::KV_BYTES;                  // (the running sum's place, or after it)
  uint8_t* sRaw = sV + STAGES * C::KV_BYTES + C::OSUM_BYTES + C::OUT_BYTES;  // e4m3: K and V codes
  int* sExp = reinterpret_cast<int*>(sRaw + 2 * C::RAW);       // [2 * STAGES][K, V] exponents that a tile is relative to
  int8_t* sRow = reinterpret_cast<int8_t*>(sExp + 2 * STAGES * 2);  // [2][256] exponents that the queries' rows are relative to
  int* sTop = reinterpret_cast<int*>(sRow + 512);                   // [2][4 warps][K, V] largest exponents of a tile
  bool osum_ok = true;
  if (!C::OSUM_SMEM) {
    uint32_t smid;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
    osum_ok = smid < static_cast<uint32_t>(p.n_osum);
    sOsum = p.osum + static_cast<size_t>(osum_ok ? smid : 0u) * (2 * 128 * 128);
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + STAGES * C::KV_BYTES + C::OSUM_BYTES + C::OUT_BYTES + 2 * C::RAW + C::EXP_BYTES);
  uint64_t* bar_q = bars;
  uint64_t* bar_k_full = bar_q + 1;
  uint64_t* bar_v_full = bar_k_full + STAGES;
  // P over S (two stages at d = 128): K and V of a stage are released apart, K after S, V after P V; P apart (four
  // stages): together, after P V, on bar_v_empty
  uint64_t* bar_k_empty = bar_v_full + STAGES;
  uint64_t* bar_v_empty = bar_k_empty + STAGES;
  uint64_t* bar_s_full = bar_v_empty + STAGES;   // [2]
  uint64_t* bar_s_free = bar_s_full + 2;         // [2] (P kept apart only)
  uint64_t* bar_p_full = bar_s_free + 2;         // [2]
  uint64_t* bar_p_half = bar_p_full + 2;         // [2] P of the first 64 keys written (P over S only)
  uint64_t* bar_turn = bar_p_half + 2;           // [2] a row tile's turn at the tensor pipe (P over S only)
  uint64_t* bar_pv_done = bar_turn + 2;          // [2]
  uint64_t* bar_o_final = bar_pv_done + 2;       // [2]
  uint64_t* bar_mma_idle = bar_o_final + 2;      // [2]
  uint64_t* bar_fix = bar_mma_idle + 2;          // the last V tile landed (its rows past the end are zeroed then)
  uint64_t* bar_q2 = bar_fix + 1;                // e4m3, bf16 queries: converted in place
  uint64_t* bar_raw = bar_q2 + 1;                // [2] e4m3: codes of K, V landed
  uint64_t* bar_raw_free = bar_raw + 2;          // [2] read by the converters
  uint64_t* bar_top = bar_raw_free + 2;          // e4m3: a tile's exponents exchanged between the converters
  uint64_t* bar_q_free = bar_top + 1;            // every S of the unit issued and done
  uint64_t* bar_unit = bar_q_free + 1;           // [2] next unit written
  uint64_t* bar_unit_free = bar_unit + 2;        // [2] read by every warp that works on it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_unit_free + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Work* sWork = reinterpret_cast<Work*>(tmem_slot + 2);  // [2]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // ---- tensor memory and barriers, side by side
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  } else if (warp == 2 && lane == 0) {
    mbar_init(bar_q, 1);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&bar_k_full[s], CONV ? 4 : 1);  // e4m3: one arrival per converter warp
      mbar_init(&bar_v_full[s], CONV ? 4 : 1);
      mbar_init(&bar_k_empty[s], 2);  // one arrival per MMA warp
      mbar_init(&bar_v_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar_s_full[t], 1);
      // one arrival per thread: with per-warp ones 1,026 us against 1,002 on 32,768 causal tokens at d = 64
      mbar_init(&bar_s_free[t], 128);
      mbar_init(&bar_p_full[t], 128);
      mbar_init(&bar_p_half[t], 128);
      mbar_init(&bar_turn[t], 1);
      mbar_init(&bar_pv_done[t], 1);
      mbar_init(&bar_o_final[t], 1);
      mbar_init(&bar_mma_idle[t], 1);
    }
    mbar_init(bar_fix, 1);
    mbar_init(bar_q2, 4);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar_raw[x], 1);
      mbar_init(&bar_raw_free[x], 4);
      mbar_init(&bar_unit[x], 1);
      mbar_init(&bar_unit_free[x], 1 + 2 + 8 + (CONV ? 4 : 0));
    }
    mbar_init(bar_top, 4);
    mbar_init(bar_q_free, 2);
    *abort_flag = 0;
    fence_mbar_init();
  } else if (warp == 3 && lane == 0) {
    prefetch_tensormap(&tmQ);
    if (!CONV) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x == 0 && !osum_ok) record_dev_error(&g_seq_err, kDevSmSlot, 30);  // exact all the same; only the fold is skipped
  const uint32_t tmo_us = p.timeout_us;
  const uint64_t tmo = static_cast<uint64_t>(tmo_us) * 1000ull;
  const uint32_t a_abort = smem_u32(const_cast<int*>(abort_flag));
  constexpr bool CONVQ = CONV && BF16;

  // A CTA works through units u = blockIdx.x, and then one of every gridDim.x, in an order that turns round every time (the
  // heaviest of one round with the lightest of the next). Warp 3 finds them, two ahead; every other warp takes them from
  // shared memory, so a unit's loads and first products run beside the end of the one before. Barrier phases count
  // on across units: kb key tiles so far, uq units with any.
  struct View {
    Work w;
    int tb, n, kbase, kleft, q_off;  // n: key tiles
  };
  // The unit's two row tiles of tpt tokens each, and its key tiles of the sequence. Both row tiles take all of them, also those
  // that the causal mask hides from the first, and an empty second one too: they stay in step, a tile ahead of each other at
  // most. (With the hidden tiles left out, 3% of a ragged batch's, a second row tile that followed on an empty one ran up to a
  // unit ahead, and its first scores were now and then wrong.)
  auto view_of = [&](const Work& w) -> View {
    View v;
    v.w = w;
    v.tb = w.ta + p.tpt;
    v.q_off = w.pos0;  // position of the sequence's first new token (negative: rows that see nothing)
    // the last position that either row tile sees
    const int t1 = min(w.ta + 2 * p.tpt, w.qlen);
    const int last = p.causal ? min(w.kvlen, v.q_off + t1) - 1 : w.kvlen - 1;
    v.n = max(0, min(w.je, last < 0 ? 0 : last / BN + 1) - w.jb);
    v.kbase = w.jb * BN;             // position of the range's first key
    v.kleft = w.kvlen - v.kbase;     // positions of the sequence from there
    return v;
  };
  // The i-th unit of this CTA; false when there is none, or a role has given up.
  auto take = [&](int i, View* v) -> bool {
    const bool ok = wait_or_abort(smem_u32(&bar_unit[i & 1]), (i >> 1) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutQ, 40);
    if (!ok) return false;
    const int4* at = reinterpret_cast<const int4*>(&sWork[i & 1]);
    const int4 a = at[0], b = at[1], c = at[2];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_unit_free[i & 1]);
    const Work w = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, 0};
    if (!w.valid) return false;
    *v = view_of(w);
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::LOW));
    if (warp == 3) {
      // ------------------------------------------------------------------ units
      const int per = 2 * p.tpt;
      auto give = [&](int i, const Work& w) -> bool {
        if (i >= 2) {
          const bool ok = wait_or_abort(smem_u32(&bar_unit_free[i & 1]), ((i >> 1) - 1) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutQ, 41);
          if (!ok) return false;
        }
        if (lane == 0) {
          int4* at = reinterpret_cast<int4*>(&sWork[i & 1]);
          at[0] = make_int4(w.valid, w.seq, w.tok_first, w.qlen);
          at[1] = make_int4(w.kvlen, w.ta, w.hk, w.jb);
          at[2] = make_int4(w.je, w.slot, w.pos0, 0);
          mbar_arrive(&bar_unit[i & 1]);
        }
        __syncwarp();
        return w.valid != 0;
      };
      const Work none = {0, 0, 0, 0, 0, 0, 0, 0, 0, -1, 0, 0};
      if constexpr (SRC == kSrcPacked) {
        auto pieces = [&](int k) {
          int first;
          return (seq_tokens(p.cu, k, p.T, &first) + per - 1) / per;
        };
        Walker walk;
        for (int i = 0;; ++i) {
          const unsigned u = static_cast<unsigned>(i) * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
          const int rank = static_cast<int>(u / p.Hkv);
          const Unit f = p.n_seqs > kRankedSeqs ? walk.find(p.n_seqs, rank, lane, pieces) : find_unit(p.n_seqs, rank, lane, pieces);
          Work w = none;
          if (f.seq >= 0) {
            w.valid = 1;
            w.seq = f.seq;
            w.qlen = w.kvlen = seq_tokens(p.cu, f.seq, p.T, &w.tok_first);
            w.ta = f.place * per;
            w.hk = static_cast<int>(u % p.Hkv);
            w.je = 0x7fffffff;
          }
          if (!give(i, w)) break;
        }
      } else {
        auto units_of = [&](int k) -> ChunkUnits {
          ChunkUnits c;
          c.seq = k;
          c.qlen = seq_tokens(p.cu, k, p.T, &c.first);
          c.kvlen = seq_positions(p.kv_lens, k, p.most);
          c.pos0 = seq_first_position(p.kv_lens, k, c.qlen);
          if (p.full && (__ldg(p.full + k) >= 0) != (SRC == kSrcPages)) c.qlen = 0;
          c.per = per;
          c.units = (c.qlen + per - 1) / per;
          c.causal = p.causal;
          return c;
        };
        // what 32 sequences from s0 on weigh for one key head, one a lane; *upto: this lane's and those before it
        auto weigh = [&](int s0, long long* upto) -> long long {
          long long x = 0;
          if (s0 + lane < p.n_seqs) {
            const ChunkUnits c = units_of(s0 + lane);
            x = c.before(c.units);
          }
          const long long mine = x;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          *upto = x;
          return mine;
        };
        // (also what the joining kernel finds where a range is empty, or a wait gave up before it)
        for (int ph = lane; ph < p.phases; ph += 32) p.meta[2 * (ph * gridDim.x + blockIdx.x)] = make_int4(-1, 0, 0, 0);
        __syncwarp();
        long long all = 0, upto, mine;
        for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
          mine = weigh(s0, &upto);
          all += __shfl_sync(0xffffffffu, upto, 31);
        }
        int i = 0;
        bool ok = true;
        for (int ph = 0; ok && ph < p.phases; ++ph) {
          // units in the order of sequences, then key heads [h0, h1), then places
          const int h0 = static_cast<int>(static_cast<long long>(p.Hkv) * ph / p.phases);
          const int h1 = static_cast<int>(static_cast<long long>(p.Hkv) * (ph + 1) / p.phases), nh = h1 - h0;
          const long long W = all * nh;
          const long long nc = min(static_cast<long long>(gridDim.x), max(W / kLeastRange, 1LL)), bx = blockIdx.x;
          const long long w0 = W * min(bx, nc) / nc, w1 = W * min(bx + 1, nc) / nc;
          const int range = ph * gridDim.x + blockIdx.x;
          if (w0 >= w1) continue;
          ChunkUnits c;
          int place = 0, hk = 0;
          long long u0 = 0;  // where the unit begins
          for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
            if (p.n_seqs > 32) mine = weigh(s0, &upto);
            const unsigned who = __ballot_sync(0xffffffffu, w0 < u0 + upto * nh);
            if (who) {
              const int k = __ffs(who) - 1;
              c = units_of(s0 + k);
              u0 += __shfl_sync(0xffffffffu, upto - mine, k) * nh;
              break;
            }
            u0 += __shfl_sync(0xffffffffu, upto, 31) * nh;
          }
          const long long head = c.before(c.units);
          hk = static_cast<int>((w0 - u0) / head);
          u0 += hk * head;
          hk += h0;
          for (int n = c.units; n > 1;) {  // the last unit that begins at w0 or before, in 32 steps at a time
            const int step = (n + 31) / 32;
            const bool le = lane * step < n && u0 + c.before(place + lane * step) <= w0;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
            n = min(step, n - k * step);
            place += k * step;
          }
          u0 += c.before(place);
          for (long long w = w0; ok && w < w1;) {
            const int n = c.tiles(place) + kUnitWeight;
            const long long next = min(u0 + n, w1);
            const int t0 = max(static_cast<int>(w - u0) - kUnitWeight, 0), t1 = max(static_cast<int>(next - u0) - kUnitWeight, 0);
            const bool whole = t0 == 0 && t1 == n - kUnitWeight;
            if (w == w0 && lane == 0) {
              // the unit this range begins in the middle of, and the ranges that hold its first and last key tile
              const int c0 = static_cast<int>(((u0 + kUnitWeight + 1) * nc - 1) / W), c1 = static_cast<int>(((u0 + n) * nc - 1) / W);
              const int r0 = ph * gridDim.x;
              p.meta[2 * range] = t0 == 0 ? make_int4(-1, 0, 0, 0) : make_int4(c.seq, hk, r0 + c0, r0 + c1);
              p.meta[2 * range + 1] = make_int4(c.first, c.qlen, place * per, 0);
            }
            if (t0 < t1) {  // (else the range ends before the unit's first key tile)
              const Work g = {1, c.seq, c.first, c.qlen, c.kvlen, place * per, hk, t0, t1, whole ? -1 : 2 * range + (t0 == 0 ? 1 : 0), c.pos0, 0};
              ok = give(i++, g);
            }
            w = next;
            u0 += n;
            if (++place == c.units) {
              place = 0;
              if (++hk == h1) {
                hk = h0;
                for (int k = c.seq + 1; w < w1 && k < p.n_seqs; ++k) {
                  c = units_of(k);
                  if (c.units > 0) break;
                }
              }
            }
          }
        }
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (ok) give(i, none);
      }
    } else if (warp == 0) {
      // ------------------------------------------------------------------ TMA producer
      View v;
      int kb = 0, uq = 0, fixes = 0;          // key tiles, units with any, tails so far
      int k_last[4] = {0, 0, 0, 0}, v_last[4] = {0, 0, 0, 0};  // loads of each stage
      int raw_last[2] = {0, 0};
      bool ok = true;
      for (int unit = 0; ok && take(unit, &v); ++unit) {
        if (v.n == 0) continue;
        const int tok_first = v.w.tok_first, hk = v.w.hk, kbase = v.kbase, kleft = v.kleft, n_max = v.n, seq = v.w.seq;
        if (uq > 0) {
          ok = wait_or_abort(smem_u32(bar_q_free), (uq - 1) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutQ, 42);
          if (!ok) break;
        }
        ++uq;
        const uint32_t q_bytes = static_cast<uint32_t>(p.tpt) * p.G * 128u;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_q, 2 * KSUB * q_bytes);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < KSUB; ++x)
              tma_load_3d(sQ + t * C::QT_BYTES + x * TILE_BYTES, &tmQ, bar_q, x * 64, hk * p.G, tok_first + (t ? v.tb : v.w.ta));
        }
        if constexpr (!CONV) {
          const int page = SRC == kSrcPages ? 1 << p.page_log2 : BN;
          const int rows = min(page, BN);
          const int boxes = BN / rows;
          const int* trow = SRC == kSrcPages ? p.table + static_cast<long long>(seq) * p.max_pages : nullptr;
          const int full = SRC == kSrcPages && p.full ? __ldg(p.full + seq) : -1;
          for (int j = 0; j < n_max; ++j) {
            const int stage = (kb + j) % STAGES;
            const uint32_t round = (kb + j) / STAGES;
            const int left = kleft - j * BN;
            const int nb = min(boxes, (left + rows - 1) / rows);
            int pg = 0, y = 0;
            if (SRC == kSrcPages && lane < nb) {  // page entries are fetched before the wait
              const int pos = kbase + j * BN + lane * rows;
              pg = full >= 0 ? full + (pos >> p.page_log2) : page_at(trow, pos >> p.page_log2, p.n_pages);
              y = pos & (page - 1);
            }
            const uint32_t bytes = static_cast<uint32_t>(nb) * rows * 128u * KSUB;
            ok = wait_or_abort(smem_u32(ALIAS ? &bar_k_empty[stage] : &bar_v_empty[stage]), (round & 1u) ^ 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 10);
            if (!ok) break;
            if (p.fault == 1 && blockIdx.x == 0 && j == 1) {  // (every wait on the tile runs out)
              ok = false;
              break;
            }
            k_last[stage & 3] = round + 1;
            if (lane == 0) mbar_arrive_expect_tx(&bar_k_full[stage], bytes);
            __syncwarp();
            if (lane < nb) {
              uint8_t* dk = sK + stage * C::KV_BYTES + lane * rows * 128 * KSUB;
              if (SRC == kSrcPages) {
                tma_load_5d(dk, &tmK, &bar_k_full[stage], 0, 0, 0, y >> 3, pg * p.Hkv + hk);
              } else {
#pragma unroll
                for (int x = 0; x < KSUB; ++x)
                  tma_load_3d(dk + x * TILE_BYTES, &tmK, &bar_k_full[stage], x * 64, hk, tok_first + kbase + j * BN);
              }
            }
            if (ALIAS) {
              ok = wait_or_abort(smem_u32(&bar_v_empty[stage]), (round & 1u) ^ 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 34);
              if (!ok) break;
            }
            const bool tail = left < BN;
            if (!tail) v_last[stage & 3] = round + 1;
            uint64_t* vbar = tail ? bar_fix : &bar_v_full[stage];
            if (lane == 0) mbar_arrive_expect_tx(vbar, bytes);
            __syncwarp();
            if (lane < nb) {
              uint8_t* dv = sV + stage * C::KV_BYTES + lane * rows * 128 * KSUB;
              if (SRC == kSrcPages) {
                tma_load_5d(dv, &tmV, vbar, 0, 0, 0, y >> 3, pg * p.Hkv + hk);
              } else {
#pragma unroll
                for (int x = 0; x < KSUB; ++x)
                  tma_load_3d(dv + x * TILE_BYTES, &tmV, vbar, x * 64, hk, tok_first + kbase + j * BN);
              }
            }
            __syncwarp();
            if (tail) {  // at most the last key tile of the sequence
              ok = wait_or_abort(smem_u32(bar_fix), fixes & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 31);
              ++fixes;
              if (!ok) break;
              zero_rows<C>(sV + stage * C::KV_BYTES, left, lane);
              fence_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_v_full[stage]);
              v_last[stage & 3] = 0;  // waited for
            }
          }
        }
        if constexpr (CONV) {
          // codes of a tile, page by page (a page's vectors of one head lie together), into the one raw buffer of K and of V
          const int page = 1 << p.page_log2, rows = min(page, BN), boxes = BN / rows;
          const int* trow = p.table + static_cast<long long>(seq) * p.max_pages;
          for (int j = 0; ok && j < n_max; ++j) {
            if (p.fault == 1 && blockIdx.x == 0 && j == 1) ok = false;  // (every wait on the tile runs out)
            if (!ok) break;
            const int nb = min(boxes, (kleft - j * BN + rows - 1) / rows);
            long long at = 0;
            if (lane < nb) {
              const int pos = kbase + j * BN + lane * rows;
              const int pg = page_at(trow, pos >> p.page_log2, p.n_pages);
              at = (((static_cast<long long>(pg) * p.Hkv + hk) << p.page_log2) + (pos & (page - 1))) * C::ROW;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              ok = ok && wait_or_abort(smem_u32(&bar_raw_free[x]), ((kb + j) & 1u) ^ 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 36 + x);
              if (!ok) break;
              if (lane == 0) mbar_arrive_expect_tx(&bar_raw[x], static_cast<uint32_t>(nb) * rows * C::ROW);
              __syncwarp();
              if (lane < nb)
                bulk_load(sRaw + x * C::RAW + lane * rows * C::ROW, (x ? p.v_cache : p.k_cache) + at, rows * C::ROW, &bar_raw[x]);
              raw_last[x] = kb + j + 1;
            }
          }
        }
        kb += n_max;
      }
      // every load issued lands before the CTA exits (bounded waits; already complete on the normal path; a tail that ran
      // out is given one more limit)
#pragma unroll
      for (int i = 0; i < STAGES; ++i) {
        if (k_last[i] > 0) mbar_wait_bounded(&bar_k_full[i], (k_last[i] - 1) & 1u, tmo);
        if (v_last[i] > 0) mbar_wait_bounded(&bar_v_full[i], (v_last[i] - 1) & 1u, tmo);
      }
      for (int x = 0; x < 2; ++x)
        if (raw_last[x] > 0) mbar_wait_bounded(&bar_raw[x], (raw_last[x] - 1) & 1u, tmo);
      if (!ok && fixes > 0) mbar_wait_bounded(bar_fix, (fixes - 1) & 1u, tmo);
      if (uq > 0) mbar_wait_bounded(bar_q, (uq - 1) & 1u, tmo);
    } else {
      // ------------------------------------------------------------------ MMA issuers, one per row tile
      // P apart from S: each on its own schedule. P over S: the tiles take turns, so that a tile's P V and next S run
      // back to back. Without turns the two tiles' groups interleave in the tensor pipe, both finish late, and both softmax
      // warpgroups then compute at the same time (3,640 cycles a key tile at d = 128); one warp issuing for both took
      // 3,300, of which 1,250 went into its own waits and commits.
      const int t = warp - 1;
      const bool leader = elect_one();
      constexpr uint32_t IDESC_S = idesc_f16(MB, 0, 128, 128);
      constexpr uint32_t IDESC_O = idesc_f16(MB, 1, 128, D);
      const uint64_t dQ = smem_desc_sw128(smem_u32(sQ + t * C::QT_BYTES), 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, C::GROUP);
      const uint64_t dV = smem_desc_sw128(smem_u32(sV), D == 128 ? C::HALF : 1024, C::GROUP);
      const uint32_t col_s = tmem + (t ? C::COL_S1 : C::COL_S0);
      const uint32_t col_p = tmem + (t ? C::COL_P1 : C::COL_P0);
      const uint32_t col_o = tmem + (t ? C::COL_O1 : C::COL_O0);
      auto wait_all = [&](uint64_t* bar, uint32_t parity, int code, int where) -> bool {
        return wait_or_abort(smem_u32(bar), parity, tmo_us, a_abort, &g_seq_err, code, where);
      };
      View v;
      int kb = 0, uq = 0;  // key tiles, units with any
      bool ok = true;
      for (int unit = 0; ok && take(unit, &v); ++unit) {
        const int n = v.n;
        if (n == 0) continue;
        auto do_s = [&](int j, bool pass) {
          const int stage = (kb + j) % STAGES;
          const uint64_t b0 = dK + static_cast<uint32_t>(stage) * (C::KV_BYTES >> 4);
          tc_fence_after();
          if (leader) {
            issue_s<0, D / 32, C::HALF>(col_s, dQ, b0, IDESC_S);
            if (pass) mbar_arrive(&bar_turn[t ^ 1]);  // the other tile's issuer wakes up while the rest goes in
            issue_s<D / 32, D / 16, C::HALF>(col_s, dQ, b0, IDESC_S);
            tc_commit(&bar_s_full[t]);
            if (ALIAS) tc_commit(&bar_k_empty[stage]);
            if (j == n - 1) tc_commit(bar_q_free);
          }
          __syncwarp();
        };
        // keys of half `part` (P over S: the first half's product runs while the softmax writes the second), or all (2)
        auto do_pv = [&](int j, int part) {
          const int stage = (kb + j) % STAGES;
          const uint64_t v0 = dV + static_cast<uint32_t>(stage) * (C::KV_BYTES >> 4);
          const bool first = (j == 0) || (osum_ok && j % C::FLUSH == 0);  // O restarts at every segment
          tc_fence_after();
          if (leader) {
            if (part == 2) {
              if (first) issue_o<true, 0, 8, C::GROUP>(col_o, col_p, v0, IDESC_O);
              else issue_o<false, 0, 8, C::GROUP>(col_o, col_p, v0, IDESC_O);
            } else if (part == 0) {
              if (first) issue_o<true, 0, 4, C::GROUP>(col_o, col_p, v0, IDESC_O);
              else issue_o<false, 0, 4, C::GROUP>(col_o, col_p, v0, IDESC_O);
            } else {
              issue_o<false, 4, 8, C::GROUP>(col_o, col_p, v0, IDESC_O);
            }
            if (part != 0) {
              tc_commit(&bar_pv_done[t]);
              if (j == n - 1) tc_commit(&bar_o_final[t]);
              tc_commit(&bar_v_empty[stage]);
            }
          }
          __syncwarp();
        };
        ok = wait_all(CONVQ ? bar_q2 : bar_q, uq & 1u, kDevTimeoutQ, 11);
        ++uq;
        if (ok) ok = wait_all(&bar_k_full[kb % STAGES], (kb / STAGES) & 1u, kDevTimeoutKV, 12);
        // (P apart: the softmax has read the last S of the unit before; P over S: P V before it in this thread's order)
        if (!ALIAS && ok && kb > 0) ok = wait_all(&bar_s_free[t], (kb - 1) & 1u, kDevTimeoutSoftmax, 43);
        if (ok) do_s(0, false);
        for (int j = 0; ok && j < n; ++j) {
          const int stage = (kb + j) % STAGES, n1 = (kb + j + 1) % STAGES;
          const uint32_t par0 = ((kb + j) / STAGES) & 1u, par1 = ((kb + j + 1) / STAGES) & 1u;
          const uint32_t tp = (kb + j) & 1u, turn = tp ^ (t ? 0u : 1u);
          if (!ALIAS) {
            if (j + 1 < n) {
              ok = wait_all(&bar_k_full[n1], par1, kDevTimeoutKV, 13);
              if (ok) ok = wait_all(&bar_s_free[t], tp, kDevTimeoutSoftmax, 14);
              if (ok) do_s(j + 1, false);
            }
            if (ok) ok = wait_all(&bar_v_full[stage], par0, kDevTimeoutKV, 15);
            if (ok) ok = wait_all(&bar_p_full[t], tp, kDevTimeoutSoftmax, 16);
            if (ok) do_pv(j, 2);
          } else {
            ok = wait_all(&bar_v_full[stage], par0, kDevTimeoutKV, 15);
            if (ok && j + 1 < n) ok = wait_all(&bar_k_full[n1], par1, kDevTimeoutKV, 13);
            if (ok) ok = wait_all(&bar_p_half[t], tp, kDevTimeoutSoftmax, 17);
            if (ok) ok = wait_all(&bar_turn[t], turn, kDevTimeoutMMA, 24);
            if (ok) do_pv(j, 0);
            if (ok) ok = wait_all(&bar_p_full[t], tp, kDevTimeoutSoftmax, 16);
            if (ok) do_pv(j, 1);
            // P_t(j) lies over S_t: MMAs of one issuing thread run in order, so S_t(j+1) follows P V's reads
            if (ok && j + 1 < n) do_s(j + 1, true);
            else if (ok && leader) mbar_arrive(&bar_turn[t ^ 1]);
          }
          __syncwarp();
        }
        kb += n;
      }
      if (leader) tc_commit(&bar_mma_idle[warp - 1]);
      __syncwarp();
      mbar_wait_bounded(&bar_mma_idle[warp - 1], 0, tmo);
    }
    tc_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
    if (warp == 1) {
      __syncwarp();
      tc_fence_after();
      tmem_dealloc(tmem, TMEM_COLS);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::HIGH));
    // ------------------------------------------------------------------ softmax warpgroups
    const int wg = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t colS = wg ? C::COL_S1 : C::COL_S0;
    const uint32_t colP = wg ? C::COL_P1 : C::COL_P0;
    const uint32_t colO = wg ? C::COL_O1 : C::COL_O0;
    const uint32_t a_s_full = smem_u32(&bar_s_full[wg]), a_s_free = smem_u32(&bar_s_free[wg]);
    const uint32_t a_p_full = smem_u32(&bar_p_full[wg]), a_pv_done = smem_u32(&bar_pv_done[wg]);
    const int rt = r / p.G;                     // token of this thread's row within the tile
    const int SEG = osum_ok ? C::FLUSH : (1 << 30);
    View v;
    int kb = 0, uq = 0;  // key tiles, units with any
    bool ok = true;
    for (int unit = 0; ok && take(unit, &v); ++unit) {
      const int n = v.n, kleft = v.kleft;
      const int t0 = wg ? v.tb : v.w.ta;
      const int rel = v.q_off + t0 - v.kbase;     // key position (in the range) of the tile's first token
      const int row_lim = p.causal ? rel + rt + 1 : 0x7fffffff;
      const int diag = p.causal ? rel - (BN - 1) : 0x7fffffff;  // tiles from beyond this key on hide keys from some row
      float sl2 = p.scale_log2;
      float m_ref = -INFINITY, l = 0.0f, m_sum = -INFINITY;
      int ev = -100000, ev_sum = 0;  // e4m3: exponent of the values that O (the running sum) is relative to
      for (int j0 = 0; ok && j0 < n; j0 += SEG) {
        if (j0 > 0) {
          // fold O into the running sum, brought from its reference to the current one by an exact power of two
          ok = wait_or_abort(a_pv_done, (kb + j0 - 1) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutMMA, 23);
          if (!ok) break;
          tc_fence_after();
          const bool have = j0 > C::FLUSH;
          float sc = (m_sum == -INFINITY) ? 0.0f : exp2_whole(m_sum - m_ref);
          if (CONV) sc *= exp2_int(static_cast<float>(max(ev_sum - ev, -200)));
          if (C::OSUM_SMEM) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(trow + colO + c * 32, o);
              tmem_wait_ld();
              reg_fence32(o);
              const uint32_t os = smem_u32(sOsum) + static_cast<uint32_t>(((wg * D) * 128 + r) * 4);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t a = os + static_cast<uint32_t>((c * 32 + e) * 128 * 4);
                const float prev = have ? ld_shared_f32(a) * sc : 0.0f;
                st_shared_f32(a, prev + __uint_as_float(o[e]));
              }
            }
          } else {
            float* og = sOsum + (wg * D) * 128 + r;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float prev[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) prev[e] = have ? __ldcg(og + (c * 32 + e) * 128) : 0.0f;
              uint32_t o[32];
              tmem_ld32(trow + colO + c * 32, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) __stcg(og + (c * 32 + e) * 128, prev[e] * sc + __uint_as_float(o[e]));
            }
          }
          m_sum = m_ref;
          ev_sum = ev;
        }
        const int j1 = (n - j0 < SEG) ? n : j0 + SEG;
        for (int j = j0; j < j1; ++j) {
          ok = wait_or_abort(a_s_full, (kb + j) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutMMA, 18);
          if (!ok) break;
          if (CONVQ && j == 0) sl2 = p.scale_log2 * exp2_int_any(sRow[(uq & 1) * 256 + wg * 128 + r]);  // written before the queries were released
          tc_fence_after();
          uint32_t sr[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(trow + colS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sr[c * 32]));
          if (!ALIAS) {
            tc_fence_before();
            mbar_arrive_a(a_s_free);  // S_t may now take S_t(j+1)
          }
          float x[128];
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(sr[c]);
          const int k0 = j * BN;
          if (k0 > kleft - BN || k0 > diag) {
            const int lim = min(kleft, row_lim) - k0;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c >= lim) x[c] = -INFINITY;
          }
          float alpha = 1.0f;
          bool rescale = false;
          float slt = sl2;
          if constexpr (CONV) {  // this tile's K and V are relative to these powers of two, which only rise
            const int2 ex = *reinterpret_cast<const int2*>(sExp + ((kb + j) % (2 * STAGES)) * 2);
            // held above 0, so that a masked score times it stays -inf (scores that small are 0 either way)
            slt = fmaxf(sl2 * exp2_int_any(ex.x), 0x1p-100f);
            if (ex.y > ev) {
              if (j > 0) {
                alpha = exp2_int(static_cast<float>(max(ev - ex.y, -200)));
                rescale = true;
              }
              ev = ex.y;
            }
          }
          const float tmax = row_max128(x) * slt;
          float al_l = 1.0f;  // what the row's sum is multiplied by (the values' exponent does not matter to it)
          if (tmax > m_ref + kTau || (m_ref == -INFINITY && tmax > -INFINITY)) {
            // From the first tile's largest score on by whole numbers, so that rescales are powers of two. That score is taken to fp32's
            // steps beside 768, 2^-14 for most, which leave room for those steps. A row of one key then has P = 2^6 once P is
            // rounded, and gives its value's bits (ragged prompts at d = 128: 217 us against 215 with ceilf(tmax)).
            if (m_ref == -INFINITY) {
              m_ref = (tmax + 768.0f) - 768.0f;
            } else {
              const float up = ceilf(tmax - m_ref);
              m_ref += up;
              al_l = exp2_int(-up);
              alpha *= al_l;
              rescale = true;
            }
          }
          // O takes the new reference (the running sum keeps its own), once PV_t(j-1) has been accumulated
          auto rescale_o = [&]() {
            if (!(__any_sync(0xffffffffu, rescale) && j > 0)) return;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(trow + colO + c * 32, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(trow + colO + c * 32, o);
            }
          };
          const float cm = ((m_ref == -INFINITY) ? 0.0f : m_ref) - kPShift;
          const uint32_t pbuf = trow + colP;
          float sum;
          if constexpr (!ALIAS) {
            const float2 sl2v = make_float2(sl2, sl2), ncm = make_float2(-cm, -cm);
            float2 rs2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            uint32_t pk[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const float2 pp = exp2_pair(x[2 * c], x[2 * c + 1], sl2v, ncm);
              rs2[c & 1] = __fadd2_rn(rs2[c & 1], pp);
              pk[c] = pack2(pp.x, pp.y, MB);
            }
            if (j > 0) {
              ok = wait_or_abort(a_pv_done, (kb + j - 1) & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutMMA, 19);
              if (!ok) break;
              tc_fence_after();
            }
            tmem_st32(pbuf, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
            tmem_st32(pbuf + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
            rescale_o();
            sum = (rs2[0].x + rs2[1].x) + (rs2[0].y + rs2[1].y);
          } else {
            // P over S: S_t(j) is complete, and its commit covers every earlier MMA of the issuing thread, PV_t(j-1)
            // included
            rescale_o();
            sum = 0.0f;
#pragma unroll
            for (int c4 = 0; c4 < 4; ++c4) {
              const float2 sl2v = make_float2(slt, slt), ncm = make_float2(-cm, -cm);
              float2 rs2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
              uint32_t hi[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int c = c4 * 16 + e;
                const float2 pp = exp2_pair(x[2 * c], x[2 * c + 1], sl2v, ncm);
                rs2[e & 1] = __fadd2_rn(rs2[e & 1], pp);
                hi[e] = pack2(pp.x, pp.y, MB);
              }
              tmem_st16(pbuf + c4 * 16, hi);
              if (c4 == 1) {
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_a(smem_u32(&bar_p_half[wg]));
                // keep the second half's work behind this point (it would be interleaved with the first's)
#pragma unroll
                for (int e = 64; e < 128; ++e) asm volatile("" : "+f"(x[e]));
              }
              sum += (rs2[0].x + rs2[1].x) + (rs2[0].y + rs2[1].y);
            }
          }
          l = l * al_l + sum;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_a(a_p_full);
        }
      }

      // ---------------------------------------------------------------- epilogue
      if (ok && n > 0) {
        ok = wait_or_abort(smem_u32(&bar_o_final[wg]), uq & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutMMA, 20);
        tc_fence_after();
      }
      // a row with a NaN score has l = NaN and passes it on; an empty one is 0 / -inf
      const bool has = (n > 0) && !(l <= 0.0f);
      float inv_l = has ? 1.0f / l : 0.0f;
      const float lse2 = has ? m_ref - kPShift + log2f(l) : -INFINITY;
      if (CONV) inv_l *= has ? exp2_int_any(min(max(ev, -126), 127)) : 1.0f;
      const int tok = t0 + rt;
      const bool write = ok && rt < p.tpt && tok < v.w.qlen;
      const int hq = v.w.hk * p.G + (r - rt * p.G);
      const long long row = static_cast<long long>(v.w.tok_first + tok) * p.Hq + hq;
      // (without key tiles nothing says that the tile's other warps have left the unit before, whose running sum may lie here)
      const bool staged = C::STAGED && n > 0 && !(C::OSUM_SMEM && osum_ok && n > C::FLUSH);
      const uint32_t buf = smem_u32(sOut) + (C::OSUM_SMEM ? wg * (D * 128 * 4) + quarter * 4096 : (warp - 4) * 4096);
      const bool part = SRC != kSrcPacked && v.w.slot >= 0;
      // (T * Hq < 2^31)
      const int to_row = part ? v.w.slot * kPartRows + wg * 128 + r : static_cast<int>(row);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        __syncwarp();  // (stores of the rows that count may have parted the lanes)
        if (ok && n > 0) {
          tmem_ld32(trow + colO + c * 32, o);
          tmem_wait_ld();
          reg_fence32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        float y[32];
        if (osum_ok && n > C::FLUSH) {
          const float* os = sOsum + (wg * D + c * 32) * 128 + r;
          float sc = (m_sum == -INFINITY) ? 0.0f : exp2_whole(m_sum - m_ref);
          if (CONV) sc *= exp2_int(static_cast<float>(max(ev_sum - ev, -200)));
          float prev[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) prev[e] = C::OSUM_SMEM ? os[e * 128] : __ldcg(os + e * 128);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = (prev[e] * sc + __uint_as_float(o[e])) * inv_l;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = has ? __uint_as_float(o[e]) * inv_l : 0.0f;
        }
        if (staged) {
          // this warp's 32 rows x 128 bytes, 64 features of the result or 32 of a part; pieces of 16 bytes are swapped by
          // row against bank conflicts
          const uint32_t at = buf + lane * 128;
          auto put = [&](int piece, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((piece ^ (lane & 7)) << 4)), "r"(w0), "r"(w1), "r"(w2), "r"(w3)
                         : "memory");
          };
          if (part) {
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4)
              put(q4, __float_as_uint(y[4 * q4]), __float_as_uint(y[4 * q4 + 1]), __float_as_uint(y[4 * q4 + 2]), __float_as_uint(y[4 * q4 + 3]));
          } else {
#pragma unroll
            for (int q8 = 0; q8 < 4; ++q8)
              put((c & 1) * 4 + q8, pack2(y[8 * q8 + 0], y[8 * q8 + 1], BF16), pack2(y[8 * q8 + 2], y[8 * q8 + 3], BF16),
                  pack2(y[8 * q8 + 4], y[8 * q8 + 5], BF16), pack2(y[8 * q8 + 6], y[8 * q8 + 7], BF16));
          }
          if (part || (c & 1)) {
            uint8_t* base = part ? reinterpret_cast<uint8_t*>(p.part_o + c * 32)
                                 : static_cast<uint8_t*>(p.out) + (c >> 1) * 128;
            const int row_bytes = part ? D * 4 : D * 2;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = i * 4 + (lane >> 3), piece = lane & 7;
              const int to = __shfl_sync(0xffffffffu, write ? to_row : -1, rr);
              uint4 w;
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                           : "r"(buf + rr * 128 + ((piece ^ (rr & 7)) << 4)));
              if (to >= 0) *(reinterpret_cast<uint4*>(base + static_cast<long long>(to) * row_bytes) + piece) = w;
            }
            __syncwarp();
          }
        } else if (write) {
          if (!part) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row * D + c * 32);
#pragma unroll
            for (int q8 = 0; q8 < 4; ++q8) {
              uint4 w;
              w.x = pack2(y[8 * q8 + 0], y[8 * q8 + 1], BF16);
              w.y = pack2(y[8 * q8 + 2], y[8 * q8 + 3], BF16);
              w.z = pack2(y[8 * q8 + 4], y[8 * q8 + 5], BF16);
              w.w = pack2(y[8 * q8 + 6], y[8 * q8 + 7], BF16);
              dst[q8] = w;
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(p.part_o + static_cast<long long>(to_row) * D + c * 32);
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4) dst[q4] = make_float4(y[4 * q4], y[4 * q4 + 1], y[4 * q4 + 2], y[4 * q4 + 3]);
          }
        }
      }
      if (write) {
        if (part) p.part_l[to_row] = lse2;
        else if (p.lse) p.lse[static_cast<long long>(hq) * p.T + v.w.tok_first + tok] = lse2 * 0.69314718055994531f;
      }
      tc_fence_before();  // O has been read: the next unit's P hand-offs release its columns
      kb += n;
      uq += n > 0;
    }
    tc_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
  } else {
    // ------------------------------------------------------------------ converters of e4m3 and 4-bit codes
    if constexpr (CONV) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::CVT));
      const int w = warp - 12;
      View v;
      int kb = 0, uq = 0;
      bool ok = true;
      for (int unit = 0; ok && take(unit, &v); ++unit) {
        const int n_max = v.n, kbase = v.kbase, kleft = v.kleft, hk = v.w.hk;
        if (n_max == 0) continue;
        if (CONVQ) {
          // queries in place: this thread's row of each tile, brought to fp16 relative to its largest power of two
          ok = wait_or_abort(smem_u32(bar_q), uq & 1u, tmo_us, a_abort, &g_seq_err, kDevTimeoutQ, 32);
          const int r = w * 32 + lane;
          for (int t = 0; ok && t < 2; ++t) {
            uint8_t* q = sQ + t * C::QT_BYTES + r * 128;
            float amax = 0.0f;
            for (int i = 0; i < 8 * KSUB; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(q + (i >> 3) * TILE_BYTES + (((i & 7) ^ (r & 7)) << 4));
              const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float2 f = unpack16(ws[u], 1);
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
            const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
            const float inv = pow2i(-e);
            sRow[(uq & 1) * 256 + t * 128 + r] = static_cast<int8_t>(e);
            for (int i = 0; i < 8 * KSUB; ++i) {
              uint4* at = reinterpret_cast<uint4*>(q + (i >> 3) * TILE_BYTES + (((i & 7) ^ (r & 7)) << 4));
              const uint4 x = *at;
              uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float2 f = unpack16(ws[u], 1);
                ws[u] = pack16(f.x * inv, f.y * inv, 0);
              }
              *at = make_uint4(ws[0], ws[1], ws[2], ws[3]);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(bar_q2);
        }
        // K and V tiles: this warp's 32 keys, a 16-byte piece of a code vector per lane and step. The exponents of this
        // lane's key are fetched a tile ahead, its page two.
        constexpr int LPR = C::ROW / 16;   // lanes of a row
        constexpr int RPS = 32 / LPR;      // rows of a step
        const int* trow = p.table + static_cast<long long>(v.w.seq) * p.max_pages;
        const int page_mask = (1 << p.page_log2) - 1;
        constexpr int NONE = -100000;
        // (what a load returns is left alone until a later tile: any arithmetic on it here would wait for it)
        auto page_of = [&](int j) -> int {
          const int k = j * BN + w * 32 + lane;
          return j < n_max && k < kleft ? __ldg(trow + ((kbase + k) >> p.page_log2)) : NONE;
        };
        auto exps_of = [&](int j, int pg) -> int2 {  // this lane's key's bytes in tile j (4 bits: a byte for each 32 features), 0 past the end
          if (j >= n_max || j * BN + w * 32 + lane >= kleft) return make_int2(0, 0);
          if (pg < 0 || pg >= p.n_pages) pg = 0;
          const long long vec = ((static_cast<long long>(pg) * p.Hkv + hk) << p.page_log2) + ((kbase + j * BN + w * 32 + lane) & page_mask);
          if constexpr (C::INT4 && D == 128)
            return make_int2(__ldg(reinterpret_cast<const int*>(p.k_scale) + vec), __ldg(reinterpret_cast<const int*>(p.v_scale) + vec));
          if constexpr (C::INT4 && D == 64)
            return make_int2(__ldg(reinterpret_cast<const uint16_t*>(p.k_scale) + vec), __ldg(reinterpret_cast<const uint16_t*>(p.v_scale) + vec));
          return make_int2(__ldg(p.k_scale + vec), __ldg(p.v_scale + vec));
        };
        // 2^e in both halves of a register, for e <= 0 (0 below fp16's numbers)
        auto pow2h = [&](int e) -> uint32_t { return (e >= -14 ? (e + 15) << 10 : (e < -24 ? 0 : 1 << (e + 24))) * 0x10001u; };
        // row of step i: w * 32 + i * RPS + lane / LPR. 16 features are two 16-byte pieces of the fp16 row; at d = 128 the
        // lanes of the second half store them in the other order, so that a row's eight lanes always meet eight different
        // banks. The swizzle of step i differs from that of step 0 by bit 2 of the row (d = 128) or not at all.
        const int c0 = 2 * (lane % LPR);
        const int flip = D == 128 ? (c0 >> 3) : 0;
        const int r0 = w * 32 + lane / LPR;
        const uint32_t to = (c0 >> 3) * TILE_BYTES + r0 * 128;
        const uint32_t p0 = (((c0 + flip) & 7) ^ (r0 & 7)) << 4, p1 = (((c0 + 1 - flip) & 7) ^ (r0 & 7)) << 4;
        const uint32_t from = smem_u32(sRaw) + r0 * C::ROW + (lane % LPR) * 16;
        auto convert = [&](uint32_t raw, uint32_t tile, uint32_t factor, bool tail) {
#pragma unroll
          for (int i = 0; i < 32 / RPS; ++i) {
            uint32_t c[4], h[8];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(raw + i * RPS * D));
            const uint32_t f = __shfl_sync(0xffffffffu, factor, i * RPS + lane / LPR);
            if (tail && f == 0xffffffffu) c[0] = c[1] = c[2] = c[3] = 0u;  // past the end: whatever the slot holds
            const __half2 f2 = *reinterpret_cast<const __half2*>(&f);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t a = e4m3x2_to_f16x2(c[u] & 0xffffu), b = e4m3x2_to_f16x2(c[u] >> 16);
              __half2 ha = __hmul2(*reinterpret_cast<__half2*>(&a), f2), hb = __hmul2(*reinterpret_cast<__half2*>(&b), f2);
              if (tail && f == 0xffffffffu) ha = hb = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
              h[2 * u] = *reinterpret_cast<uint32_t*>(&ha);
              h[2 * u + 1] = *reinterpret_cast<uint32_t*>(&hb);
            }
            const uint32_t dst = tile + to + i * RPS * 128, x = D == 128 ? (i & 1) * 64u : 0u;
            const bool fl = flip != 0;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (p0 ^ x)), "r"(fl ? h[4] : h[0]), "r"(fl ? h[5] : h[1]),
                         "r"(fl ? h[6] : h[2]), "r"(fl ? h[7] : h[3]) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (p1 ^ x)), "r"(fl ? h[0] : h[4]), "r"(fl ? h[1] : h[5]),
                         "r"(fl ? h[2] : h[6]), "r"(fl ? h[3] : h[7]) : "memory");
          }
        };
        // 4 bits: a lane's 16 bytes are the 32 features of a scale, four pieces of the fp16 row. Lanes of the row's second half
        // (d = 128) take their words in the order 2, 3, 0, 1, so that a row's and its neighbour's lanes meet eight different banks.
        [[maybe_unused]] auto convert4 = [&](uint32_t raw, uint32_t tile, uint32_t word, int ref, int j) {
          const int gr = lane % LPR;
          const bool flip4 = gr >= 2;
          const __half2 mul = __floats2half2_rn(1.0f, 0.0625f), add = __floats2half2_rn(-1032.0f, -72.0f);
          uint32_t base;  // (a register: as a number it would take a second instruction beside the mask)
          asm volatile("mov.b32 %0, 0x64006400;" : "=r"(base));
#pragma unroll
          for (int i = 0; i < 32 / RPS; ++i) {
            const int rw = i * RPS + lane / LPR, row = w * 32 + rw;
            uint32_t c[4];
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]) : "r"(raw + i * RPS * static_cast<int>(C::ROW)));
            const uint32_t b = (__shfl_sync(0xffffffffu, word, rw) >> (8 * gr)) & 255u;
            // relative to 2^ref, at least every scale so far but for its mantissa; zero past the end, where codes are whatever the slot holds
            const float f = j * BN + row < kleft ? int4_scale(b) * exp2_int_any(-ref) : 0.0f;
            const __half2 f2 = __float2half2_rn(f);
            const uint32_t dst = tile + (gr >> 1) * TILE_BYTES + row * 128;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t cw = flip4 ? c[u ^ 2] : c[u];
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // a byte's two numbers from its low and high four bits: 1024 + c and 1024 + 16 c as fp16 numbers, then c - 8 (exact)
                uint32_t x;
                asm("lop3.b32 %0, %1, 0x00f0000f, %2, 0xea;" : "=r"(x) : "r"(__byte_perm(cw, 0, e * 0x1111)), "r"(base));  // (. & mask) | base
                const __half2 y = __hmul2(__hfma2(*reinterpret_cast<__half2*>(&x), mul, add), f2);
                h[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              const int piece = ((gr & 1) << 2) | (flip4 ? u ^ 2 : u);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + ((piece ^ (row & 7)) << 4)), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
            }
          }
        };
        auto exps_in = [&](int j, int2 b) -> int2 {
          if constexpr (C::INT4) {  // the largest exponent of the scales that are numbers
            auto top = [](uint32_t x) -> int {
              uint32_t t = 0;
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                const uint32_t y = (x >> (8 * i)) & 255u;
                t = max(t, y >= 248u ? 0u : y);
              }
              return static_cast<int>(t >> 3) - 15;
            };
            return j * BN + w * 32 + lane < kleft ? make_int2(top(b.x), top(b.y)) : make_int2(NONE, NONE);
          }
          return j * BN + w * 32 + lane < kleft ? make_int2(b.x - 127, b.y - 127) : make_int2(NONE, NONE);
        };
        // the largest exponents of tile j's quarter go to the other warps a tile before they are needed
        auto send_top = [&](int j, int2 b) {
          if (j >= n_max) return;
          const int2 e = exps_in(j, b);
          const int kt = __reduce_max_sync(0xffffffffu, e.x), vt = __reduce_max_sync(0xffffffffu, e.y);
          if (lane == 0) {
            *reinterpret_cast<int2*>(sTop + ((kb + j) & 1) * 8 + w * 2) = make_int2(kt, vt);
            mbar_arrive(bar_top);
          }
        };
        int2 eb = exps_of(0, page_of(0));
        int pg = page_of(1);
        send_top(0, eb);
        int kref = NONE, vref = NONE;  // the largest exponents so far
        for (int j = 0; ok && j < n_max; ++j) {
          const int stage = (kb + j) % STAGES;
          const uint32_t free_par = (((kb + j) / STAGES) & 1u) ^ 1u, raw_par = (kb + j) & 1u;
          const bool tail = kleft - j * BN < BN;
          const bool in = j * BN + w * 32 + lane < kleft;
          const int2 ex = C::INT4 ? eb : exps_in(j, eb);
          eb = exps_of(j + 1, pg);
          pg = page_of(j + 2);
          const int* top = sTop + raw_par * 8;
          ok = wait_or_abort(smem_u32(bar_top), raw_par, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 44);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int2 t = *reinterpret_cast<const int2*>(top + i * 2);
            kref = max(kref, t.x);
            vref = max(vref, t.y);
          }
          if (ok) ok = wait_or_abort(smem_u32(&bar_raw[0]), raw_par, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 38);
          if (ok) ok = wait_or_abort(smem_u32(&bar_k_empty[stage]), free_par, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 33);
          if (ok) {
            // twice as many slots as stages: a K stage is free once S is, before the softmax has read its exponents
            if (w == 0 && lane == 0) *reinterpret_cast<int2*>(sExp + ((kb + j) % (2 * STAGES)) * 2) = make_int2(kref, vref);
            if constexpr (C::INT4) convert4(from, smem_u32(sK) + stage * C::KV_BYTES, static_cast<uint32_t>(ex.x), kref, j);
            else convert(from, smem_u32(sK) + stage * C::KV_BYTES, in ? pow2h(ex.x - kref) : 0xffffffffu, tail);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bar_k_full[stage]);
              mbar_arrive(&bar_raw_free[0]);
            }
            send_top(j + 1, eb);
            ok = wait_or_abort(smem_u32(&bar_raw[1]), raw_par, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 39);
            if (ok) ok = wait_or_abort(smem_u32(&bar_v_empty[stage]), free_par, tmo_us, a_abort, &g_seq_err, kDevTimeoutKV, 35);
          }
          if (ok) {
            if constexpr (C::INT4) convert4(from + C::RAW, smem_u32(sV) + stage * C::KV_BYTES, static_cast<uint32_t>(ex.y), vref, j);
            else convert(from + C::RAW, smem_u32(sV) + stage * C::KV_BYTES, in ? pow2h(ex.y - vref) : 0xffffffffu, tail);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&bar_v_full[stage]);
              mbar_arrive(&bar_raw_free[1]);
            }
          }
        }
        kb += n_max;
        ++uq;
      }
    }
    tc_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
  }
}

// Joins the parts of the units that several ranges share. Blocks (c, .) look after the unit that range c begins in the
// middle of, if it is the first such one: M = max_k lse_k, out = sum_k 2^(lse_k - lse) O_k in the order of the ranges.
constexpr int kJoinBlocks = 8;  // blocks of a unit's rows
template <int D, int BF16>
__global__ void __launch_bounds__(256) seq_combine_kernel(const SeqParams p) {
  constexpr int TPR = D / 4, RPB = 256 / TPR;  // threads of a row, rows of a block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 m = __ldcg(p.meta + 2 * blockIdx.x), q = __ldcg(p.meta + 2 * blockIdx.x + 1);
  if (m.x < 0 || static_cast<int>(blockIdx.x) != m.z + 1) return;
  const int parts = m.w - m.z + 1, c = threadIdx.x % TPR;
  for (int r = blockIdx.y * RPB + threadIdx.x / TPR; r < kPartRows; r += kJoinBlocks * RPB) {
    const int rt = (r & 127) / p.G, tok = q.z + (r >> 7) * p.tpt + rt;
    if (rt >= p.tpt || tok >= q.y) continue;
    // the first part is its range's last piece, the others are their ranges' first
    auto at = [&](int k) -> long long { return (2LL * (m.z + k) + (k == 0 ? 1 : 0)) * kPartRows + r; };
    float M = -INFINITY;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(p.part_l + at(k)));
    float L = 0.0f;
    float4 a = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float lk = __ldcg(p.part_l + at(k));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p.part_o) + at(k) * TPR + c);
      const float w = lk == -INFINITY ? 0.0f : exp2f(lk - M);  // (such a part is zero; NaN passes on)
      L += w;
      a.x = fmaf(w, b.x, a.x);
      a.y = fmaf(w, b.y, a.y);
      a.z = fmaf(w, b.z, a.z);
      a.w = fmaf(w, b.w, a.w);
    }
    const bool has = !(L <= 0.0f);
    const float inv = has ? 1.0f / L : 0.0f;
    const int hq = m.y * p.G + ((r & 127) - rt * p.G);
    const long long row = static_cast<long long>(q.x + tok) * p.Hq + hq;
    reinterpret_cast<uint2*>(p.out)[row * TPR + c] = make_uint2(pack2(a.x * inv, a.y * inv, BF16), pack2(a.z * inv, a.w * inv, BF16));
    if (p.lse && c == 0) p.lse[static_cast<long long>(hq) * p.T + q.x + tok] = has ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

// ---- 4-bit pages as 16-bit numbers, for sequences whose keys many row tiles read
// A tile of 4-bit keys and values costs the converter warps of a CTA some 2,600 cycles beyond what a 16-bit one takes, for every unit of 256 rows that reads
// it; unpacking it once into memory costs the whole GPU 13 ns, two such tiles' worth on one SM. So a sequence of two full units
// or more is unpacked first, as far as the scratch pages go, and read as 16-bit pages: 2,048 tokens over 32,000 positions, 32 and 8 heads of
// 128, 731 us against 1,359. The others go to a second kernel, which short batches do not gain from: 12 ragged sequences, 3,000 tokens over 60,000
// positions, 8 and 2 heads of 64, some 30 key tiles a CTA (72 by the longest sequence), take 84 us packed and 100 in two kernels.
// Where the two forms cross, packed / unpacked (key tiles a CTA by the longest sequence; 8 and 2 heads of 64 in fp16, then 32 and 8 of 128 in bf16):
//   2,048 tokens of one sequence        (13) 42 / 46, (20) 54 / 53, (59) 118 / 96, (112) 204 / 156, (217) 385 / 277
//                                       (54) 195 / 117, (133) 435 / 239, (448) 1,381 / 730
//   8 sequences of 56 to 455 of them    (27) 59 / 84, (53) 87 / 113, (106) 147 / 189, (211) 267 / 286
//                                       (30) 134 / 152, (57) 206 / 197, (109) 316 / 291, (214) 581 / 484, (424) 1,062 / 802
//   rows a sequence, over 8,000 positions each, with work enough (unpacked as far as the scratch pages go): 512 225 / 244 and 848 / 856, 768 220 / 216 and 803 / 716, 1,024 219 / 202 and 813 / 549;
//   of 256 rows, one unit, 242 / 326 and 869 / 978
// kFullTiles lies between the crossings of the two kinds, which the caller's numbers do not tell apart. Below it bf16 rows keep P in fp16.
constexpr int kFullRows = 512;                      // rows of a sequence and key head from which on it is unpacked
constexpr int kFullTiles = 96;                      // key tiles of a CTA, by the caller's longest sequence, from which on any is
constexpr size_t kFullBytes = size_t(512) << 20;    // the most that the scratch pages take

// Where each sequence's scratch pages begin, in the sequences' order while they last. One warp.
__global__ void __launch_bounds__(32) full_pages_kernel(const int* cu, const int* kv_lens, int n_seqs, int T, int G, long long most, int pages, int* full,
                                                        int* total) {
  int used = 0;
  for (int s0 = 0; s0 < n_seqs; s0 += 32) {
    const int s = s0 + threadIdx.x;
    int need = 0;
    if (s < n_seqs) {
      int first;
      const long long rows = static_cast<long long>(seq_tokens(cu, s, T, &first)) * G;
      if (rows >= kFullRows) need = min((seq_positions(kv_lens, s, most) + kFullPage - 1) / kFullPage, pages + 1);
    }
    int upto = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (static_cast<int>(threadIdx.x) >= o) upto = min(upto + y, pages + 1);
    }
    const bool fits = need > 0 && used + upto <= pages;
    if (s < n_seqs) full[s] = fits ? used + upto - need : -1;
    const unsigned in = __ballot_sync(0xffffffffu, fits);
    const int last = in ? 31 - __clz(in) : 0;
    const int now = __shfl_sync(0xffffffffu, upto, last);
    if (__any_sync(0xffffffffu, need > 0 && !fits)) {  // what comes behind one that does not fit stays packed
      if (in) used += now;
      for (int r = s0 + 32 + threadIdx.x; r < n_seqs; r += 32) full[r] = -1;
      break;
    }
    if (in) used += now;
  }
  if (threadIdx.x == 0) *total = used;
}

// One scratch page of one key head a block: 128 positions' keys and values. A lane turns 4 bytes, 8 numbers, into 16, so that a warp's loads and stores cover
// whole lines (with 16 bytes into 64 a lane 42 us for 34,048 positions of 8 heads of 128, 176 MB; so 30).
template <int D, int BF16>
__global__ void __launch_bounds__(256) unpack_kernel(const SeqParams p, const int* total, uint16_t* k_full, uint16_t* v_full) {
  constexpr int WORDS = D / 8, AT_ONCE = 4;
  const int page = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv, lane = threadIdx.x & 31;
  if (page >= __ldg(total)) return;
  // the last sequence whose pages begin at `page` or before (they rise along the sequences that have any)
  int seq = -1;
  for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
    const int b = s0 + lane < p.n_seqs ? __ldg(p.full + s0 + lane) : -1;
    const unsigned in = __ballot_sync(0xffffffffu, b >= 0 && b <= page);
    if (in) seq = s0 + 31 - __clz(in);
  }
  const int pos0 = (page - __ldg(p.full + seq)) * kFullPage, len = seq_positions(p.kv_lens, seq, p.most);
  const int* row = p.table + static_cast<long long>(seq) * p.max_pages;
  const uint32_t* codes[2] = {reinterpret_cast<const uint32_t*>(p.k_cache), reinterpret_cast<const uint32_t*>(p.v_cache)};
  const uint8_t* scales[2] = {p.k_scale, p.v_scale};
  for (int i0 = threadIdx.x; i0 < kFullPage * WORDS; i0 += 256 * AT_ONCE) {
    uint32_t w[AT_ONCE][2], b[AT_ONCE][2];
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int slot = (i0 + u * 256) / WORDS, word = (i0 + u * 256) % WORDS, pos = pos0 + slot;
      w[u][0] = w[u][1] = b[u][0] = b[u][1] = 0u;
      if (pos < len) {
        const long long vec = ((static_cast<long long>(page_at(row, pos >> p.page_log2, p.n_pages)) * p.Hkv + h) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          w[u][kv] = __ldg(codes[kv] + vec * WORDS + word);
          b[u][kv] = __ldg(scales[kv] + vec * (D / 32) + (word >> 2));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int slot = (i0 + u * 256) / WORDS, word = (i0 + u * 256) % WORDS;
      if (pos0 + slot >= len) continue;  // (rows behind a sequence's end are masked, and zeroed where they are read)
      const long long to = ((static_cast<long long>(page) * p.Hkv + h) * kFullPage + slot) * WORDS + word;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float s = int4_scale(b[u][kv]);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = static_cast<float>(static_cast<int>((w[u][kv] >> (4 * e)) & 15u) - 8) * s;
          if (!BF16) f[e] = f[e] > 65504.0f ? 65504.0f : (f[e] < -65504.0f ? -65504.0f : f[e]);  // (as they are read back)
        }
        reinterpret_cast<uint4*>(kv ? v_full : k_full)[to] =
            make_uint4(pack16(f[0], f[1], BF16), pack16(f[2], f[3], BF16), pack16(f[4], f[5], BF16), pack16(f[6], f[7], BF16));
      }
    }
  }
}

template <int D, int BF16, int SRC>
int launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const SeqParams& p, long long grid,
             cudaStream_t stream) {
  using C = SeqCfg<D, SRC>;
  auto kern = attn_seq_kernel<D, BF16, SRC>;
  static PerDeviceOnce attr;
  int dev = 0;
  if (!attr.done(&dev)) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncGetAttributes(sequence attention)");
    // setmaxnreg.inc waits for its registers: refuse to launch unless the launch holds the split
    const int need = 128 * C::LOW + 256 * C::HIGH + (C::CONV ? 128 * C::CVT : 0);
    if (fa.numRegs * C::NTHR < need) {
      set_error("sequence attention kernel built with %d registers/thread; the register split needs %d", fa.numRegs,
                (need + C::NTHR - 1) / C::NTHR);
      return CQSA_ERR_UNSUPPORTED;
    }
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return cuda_status(e, "cudaFuncSetAttribute(sequence attention smem)");
    attr.mark(dev);
  }
  const long long sms = sm_count();
  const unsigned ctas = static_cast<unsigned>(grid < sms ? grid : sms);
  kern<<<ctas, C::NTHR, C::SMEM_BYTES, stream>>>(mq, mk, mv, p);
  int rc = cuda_status(cudaGetLastError(), "sequence attention kernel launch");
  if (rc != CQSA_OK || SRC == kSrcPacked || ctas == 1) return rc;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(ctas * p.phases, kJoinBlocks);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, seq_combine_kernel<D, BF16>, p), "sequence attention joining kernel launch");
}

template <int SRC>
int dispatch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const SeqParams& p, int d, int dtype,
             long long grid, cudaStream_t s) {
  if (grid > 0x7fffffffLL) {
    set_error("problem too large for one launch (%lld units)", grid);
    return CQSA_ERR_UNSUPPORTED;
  }
  const bool bf = dtype == CQSA_BF16;
  if (d == 64) return bf ? launch_t<64, 1, SRC>(mq, mk, mv, p, grid, s) : launch_t<64, 0, SRC>(mq, mk, mv, p, grid, s);
  return bf ? launch_t<128, 1, SRC>(mq, mk, mv, p, grid, s) : launch_t<128, 0, SRC>(mq, mk, mv, p, grid, s);
}

// Packed tokens [T, heads, d] as (feature, head, token) with boxes of 64 features, `heads_box` heads and `rows` tokens.
int make_token_map(CUtensorMap* m, const void* base, int dtype, int d, int heads, int T, long long stride, int heads_box, int rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads_box), static_cast<cuuint32_t>(rows)};
  return encode_tensor_map(m, dtype == CQSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base,
                           dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// An upper bound on the pairs of row tiles of n_seqs sequences that hold T tokens together.
long long pairs_bound(int T, int n_seqs, int tpt) { return T / (2 * tpt) + (T < n_seqs ? T : n_seqs); }

// CTAs of a chunk: one per SM, fewer when the ranges would weigh less than kLeastRange (by the caller's longest sequence; longer
// ones are still computed, with fewer CTAs than they could use).
int chunk_ctas(const PagedArgs& a) {
  const int tpt = 128 / (a.Hq / a.Hkv), sms = sm_count();
  const long long by_tokens = pairs_bound(a.T, a.n_seqs, tpt);
  const long long by_longest = static_cast<long long>(a.n_seqs) * ((a.max_q_len + 2 * tpt - 1) / (2 * tpt));
  const long long units = (by_tokens < by_longest ? by_tokens : by_longest) * a.Hkv;
  const long long tiles = a.max_kv_len / BN + 1;
  const long long n = units * (tiles + kUnitWeight) / kLeastRange;  // (below 2^31 units of less than 2^25 tiles)
  return static_cast<int>(n < 1 ? 1 : (n < sms ? n : sms));
}

// Phases of a chunk's key heads. The CTAs are spread over all units of a phase, so its keys and values are what L2 (129 MB)
// should hold: 2,048 tokens over 34,048 positions with 8 key heads at d = 128, 139 MB, take 768 us in one phase, 733 in two
// and 712 in three; 4 heads (70 MB) 715 in one and 722 in two. Each phase leaves up to two parts per CTA, so a CTA's share
// of it is to be 24 key tiles at least.
int chunk_phases(const PagedArgs& a) {
  const int tpt = 128 / (a.Hq / a.Hkv);
  const double tiles = (a.max_kv_len / BN + 1.0) * a.Hkv * (static_cast<double>(a.T) / (2 * tpt));
  const double vector = a.cache_dtype == CQSA_INT4 ? 1.0625 * a.d : (a.cache_dtype == CQSA_E4M3 ? 2.0 * a.d : 4.0 * a.d);  // bytes of a key and a value
  const double bytes = static_cast<double>(a.n_seqs) * a.max_kv_len * a.Hkv * vector;
  const double most = tiles / (24.0 * chunk_ctas(a)), want = bytes < 96.0 * 1048576.0 ? 1.0 : ceil(bytes / (64.0 * 1048576.0));
  const int n = static_cast<int>(fmin(fmin(want, most), fmin(a.Hkv, 4.0)));
  return n < 1 ? 1 : n;
}

void fill_common(SeqParams* p, int n_seqs, int T, int Hq, int Hkv, int causal, float scale) {
  memset(p, 0, sizeof(*p));
  p->n_seqs = n_seqs;
  p->T = T;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->G = Hq / Hkv;
  p->tpt = 128 / p->G;
  p->causal = causal;
  p->scale_log2 = scale * 1.4426950408889634f;
  p->timeout_us = timeout_us();
  p->fault = debug_fault();
}

}  // namespace

namespace {

size_t parts_workspace(const PagedArgs& a) {
  const size_t parts = 2 * static_cast<size_t>(chunk_ctas(a)) * chunk_phases(a);
  return parts * kPartRows * (static_cast<size_t>(a.d) + 1) * 4 + parts * sizeof(int4);
}

// A 4-bit batch read as 16-bit pages: the same but for the cache's type (which sets the phases).
PagedArgs as_full(const PagedArgs& a) {
  PagedArgs f = a;
  f.cache_dtype = a.dtype;
  f.page = kFullPage;
  return f;
}

// Scratch pages of 4-bit sequences, by the caller's counts and longest sequence: as many as the sequences that are long enough may need, within kFullBytes.
int full_pages(const PagedArgs& a) {
  const long long G = a.Hq / a.Hkv;
  if (a.cache_dtype != CQSA_INT4 || a.max_q_len * G < kFullRows) return 0;
  const long long by_tokens = a.T * G / kFullRows, seqs = by_tokens < a.n_seqs ? by_tokens : a.n_seqs;
  const long long longest = (a.max_kv_len + kFullPage - 1LL) / kFullPage, want = seqs * longest;
  if (static_cast<double>(longest) * a.Hkv * (static_cast<double>(a.T) * G / kPartRows) < static_cast<double>(kFullTiles) * chunk_ctas(a)) return 0;
  const long long most = static_cast<long long>(kFullBytes / (static_cast<size_t>(kFullPage) * a.Hkv * a.d * 4));
  return static_cast<int>(want < most ? want : most);
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t chunk_workspace(const PagedArgs& a) {
  const int pages = full_pages(a);
  if (pages == 0) return parts_workspace(a);
  const size_t one = parts_workspace(a), two = parts_workspace(as_full(a));
  return up256(one > two ? one : two) + up256((static_cast<size_t>(a.n_seqs) + 1) * 4) + 2 * static_cast<size_t>(pages) * a.Hkv * kFullPage * a.d * 2;
}

namespace {

// The parts' place in the workspace, and how a batch is cut.
int set_split(SeqParams* p, const PagedArgs& a) {
  const int ctas = chunk_ctas(a);
  p->phases = chunk_phases(a);
  const size_t parts = 2 * static_cast<size_t>(ctas) * p->phases;
  p->part_o = static_cast<float*>(a.workspace);
  p->part_l = p->part_o + parts * kPartRows * a.d;
  p->meta = reinterpret_cast<int4*>(p->part_l + parts * kPartRows);
  p->page_log2 = 31 - __builtin_clz(static_cast<unsigned>(a.page));
  return ctas;
}

int launch_pages(SeqParams p, const CUtensorMap& mq, const PagedArgs& a, cudaStream_t stream) {
  const int ctas = set_split(&p, a), box = a.page < BN ? a.page : BN;
  CUtensorMap mk, mv;
  int rc = make_page_map(&mk, a.k_cache, a, box);
  if (rc == CQSA_OK) rc = make_page_map(&mv, a.v_cache, a, box);
  return rc == CQSA_OK ? dispatch<kSrcPages>(mq, mk, mv, p, a.d, a.dtype, ctas, stream) : rc;
}

// Unpacks what full_pages allows for and attends to those sequences.
int launch_full(SeqParams* p, const CUtensorMap& mq, const PagedArgs& a, int pages, cudaStream_t stream) {
  const size_t one = parts_workspace(a), two = parts_workspace(as_full(a));
  uint8_t* ws = static_cast<uint8_t*>(a.workspace) + up256(one > two ? one : two);
  int* full = reinterpret_cast<int*>(ws);
  uint16_t* k_full = reinterpret_cast<uint16_t*>(ws + up256((static_cast<size_t>(a.n_seqs) + 1) * 4));
  uint16_t* v_full = k_full + static_cast<size_t>(pages) * a.Hkv * kFullPage * a.d;
  p->full = full;
  full_pages_kernel<<<1, 32, 0, stream>>>(a.cu, a.kv_lens, a.n_seqs, a.T, p->G, p->most, pages, full, full + a.n_seqs);
  int rc = cuda_status(cudaGetLastError(), "scratch page kernel launch");
  if (rc != CQSA_OK) return rc;
  set_split(p, a);
  const unsigned grid = static_cast<unsigned>(pages) * a.Hkv;
  const bool bf = a.dtype == CQSA_BF16;
  if (a.d == 64 && bf) unpack_kernel<64, 1><<<grid, 256, 0, stream>>>(*p, full + a.n_seqs, k_full, v_full);
  else if (a.d == 64) unpack_kernel<64, 0><<<grid, 256, 0, stream>>>(*p, full + a.n_seqs, k_full, v_full);
  else if (bf) unpack_kernel<128, 1><<<grid, 256, 0, stream>>>(*p, full + a.n_seqs, k_full, v_full);
  else unpack_kernel<128, 0><<<grid, 256, 0, stream>>>(*p, full + a.n_seqs, k_full, v_full);
  rc = cuda_status(cudaGetLastError(), "unpacking kernel launch");
  if (rc != CQSA_OK) return rc;
  PagedArgs f = as_full(a);
  f.k_cache = k_full;
  f.v_cache = v_full;
  f.n_pages = pages;
  return launch_pages(*p, mq, f, stream);
}

}  // namespace

int launch_chunk(const PagedArgs& a, cudaStream_t stream) {
  SeqParams p;
  fill_common(&p, a.n_seqs, a.T, a.Hq, a.Hkv, a.causal, a.scale);
  p.cu = a.cu;
  p.kv_lens = a.kv_lens;
  p.table = a.table;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.out = a.out;
  p.lse = a.lse;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.most = static_cast<long long>(a.max_pages) * a.page;
  int rc = osum_slots(&p.osum, &p.n_osum);
  CUtensorMap mq;
  if (rc == CQSA_OK) rc = make_token_map(&mq, a.q, a.dtype, a.d, a.Hq, a.T, a.q_stride, p.G, p.tpt);
  if (rc != CQSA_OK) return rc;
  if (a.cache_dtype != CQSA_E4M3 && a.cache_dtype != CQSA_INT4) return launch_pages(p, mq, a, stream);
  if (const int pages = full_pages(a)) rc = launch_full(&p, mq, a, pages, stream);
  if (rc != CQSA_OK) return rc;
  // (these pages are copied as they lie, without maps: the queries' stands in for theirs)
  const int ctas = set_split(&p, a);
  return a.cache_dtype == CQSA_E4M3 ? dispatch<kSrcE4m3>(mq, mq, mq, p, a.d, a.dtype, ctas, stream)
                                    : dispatch<kSrcInt4>(mq, mq, mq, p, a.d, a.dtype, ctas, stream);
}

int launch_packed(const PackedArgs& a, cudaStream_t stream) {
  SeqParams p;
  fill_common(&p, a.n_seqs, a.T, a.Hq, a.Hkv, a.causal, a.scale);
  p.cu = a.cu;
  p.out = a.out;
  p.lse = a.lse;
  int rc = osum_slots(&p.osum, &p.n_osum);
  CUtensorMap mq, mk, mv;
  if (rc == CQSA_OK) rc = make_token_map(&mq, a.q, a.dtype, a.d, a.Hq, a.T, a.q_stride, p.G, p.tpt);
  if (rc == CQSA_OK) rc = make_token_map(&mk, a.k, a.dtype, a.d, a.Hkv, a.T, a.k_stride, 1, BN);
  if (rc == CQSA_OK) rc = make_token_map(&mv, a.v, a.dtype, a.d, a.Hkv, a.T, a.v_stride, 1, BN);
  if (rc != CQSA_OK) return rc;
  return dispatch<kSrcPacked>(mq, mk, mv, p, a.d, a.dtype, pairs_bound(a.T, a.n_seqs, p.tpt) * a.Hkv, stream);
}

DEV_ERR_READERS(seq, g_seq_err)

}  // namespace cqsa
