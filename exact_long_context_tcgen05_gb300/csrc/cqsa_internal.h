// Internal declarations shared by the library's translation units (not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/cqsa.h"

namespace cqsa {

// Output / partial modes of the attention kernel.
enum AttnMode : int {
  kModeOut = 0,    // normalised output in the input dtype + fp32 LSE (the SDPA-shaped call)
  kModePart = 1,   // normalised fp32 partial output + fp32 LSE of one chunk pair
  kModeAccum = 2,  // merge this chunk pair's result into an fp32 (O_acc, LSE_acc) in place
};

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  int B, H;
  int Nq, Nkv;          // tokens held in the q / kv buffers
  long long q_off;      // absolute position of q-buffer token 0 (causal mask)
  long long kv_off;     // absolute position of kv-buffer token 0
  int d;
  int causal;
  float scale;          // already resolved (0 -> 1/sqrt(d) done by the caller)
  int dtype;            // CQSA_F16 / CQSA_BF16
  int in_layout;        // layout of q/k/v buffers: CQSA_LAYOUT_BHND / CQSA_LAYOUT_BNHD
  int mode;             // AttnMode
  void* out;            // kModeOut: [B,H,Nq,d] (or [B,Nq,H,d] with out_layout) in dtype
  float* lse;           // kModeOut: [B,H,Nq]
  float* o_part;        // kModePart / kModeAccum: fp32 [B,H,Nq,d] (or token-major)
  float* lse_part;      // fp32 [B,H,Nq]
  int out_layout;       // layout of out / o_part
  long long q_tokens_alloc;   // tokens per head in the q buffer when it is a token range of a longer
                              // tensor (its strides follow this count); 0: the buffer holds Nq tokens
  long long kv_tokens_alloc;  // the same for k / v; 0: Nkv
};

// Validates nothing (the ABI layer does); encodes tensor maps and launches on `stream`.
int launch_attention(const AttnArgs& a, cudaStream_t stream);
// Up to kMaxWavePairs (32) chunk pairs in one launch (the wave engine). The pairs share B, H, d, dtype,
// causal, layouts and scale; each has its own buffers, offsets, sizes, mode (kModePart or kModeAccum)
// and accumulator. Pairs writing one accumulator must not share a launch (their epilogues would race).
int launch_attention_multi(const AttnArgs* pairs, int n, cudaStream_t stream);

// Attention backward (attn_bwd.cu), head dimension 64. The monolithic call (launch_attention_bwd) takes
// q, k, v, out, dout [B,H,N,64] with Nq = Nkv = N and offsets 0, writes dq, dk, dv, and uses
// `workspace` (attention_bwd_workspace bytes) for the fp32 dQ accumulator and D. One chunk pair
// (launch_attention_bwd_chunk) takes a query chunk (q, dout, lse, dvec: Nq rows at absolute position
// q_off) and a key chunk (k, v: Nkv rows at kv_off) and adds into dq_acc [B,H,Nq,64], dk_acc and
// dv_acc [B,H,Nkv,64] (fp32, scale applied).
struct BwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* out;
  const void* dout;
  const float* lse;
  const float* dvec;
  void* dq;
  void* dk;
  void* dv;
  float* dq_acc;
  float* dk_acc;
  float* dv_acc;
  void* workspace;
  int B, H, Nq, Nkv, d;
  long long q_off, kv_off;
  int causal;
  float scale;  // resolved
  int dtype;
};
size_t attention_bwd_workspace(int B, int H, int N, int d);
int launch_attention_bwd(const BwdArgs& a, cudaStream_t stream);
int launch_attention_bwd_chunk(const BwdArgs& a, cudaStream_t stream);
// D_i = dout_i . out_i (fp32) for `rows` rows of 64 features; fp32 -> dtype for n elements (n % 4 == 0).
int launch_bwd_dvec(const void* out, const void* dout, float* dvec, long long rows, int d, int dtype,
                    cudaStream_t stream);
// Host-streaming helpers (stream_driver.cu): whether `bytes` of device memory fit the resident budget
// (cqsa_set_stream_kv_resident_bytes), and a copy of tokens [t0, t0 + n) of a (layout, N tokens) tensor
// into the same positions of another of the same shape; *bytes grows by the bytes copied.
bool stream_resident_ok(size_t bytes);
cudaError_t copy_range(void* dst, const void* src, int layout, int B, int H, long long N, int d, long long t0, int n,
                       cudaMemcpyKind kind, cudaStream_t s, long long* bytes);
// D for tokens [t0, t0 + n) of every head of [BH, N, d] out / dout, into dvec [BH, N] at the same rows.
int launch_bwd_dvec_range(const void* out, const void* dout, float* dvec, long long BH, long long n, long long N,
                          long long t0, int d, int dtype, cudaStream_t stream);
int launch_bwd_cast(const float* acc, void* out, long long n, int dtype, cudaStream_t stream);

// The running sums of the d = 128 forward kernels on the current device: `n` slots of 2 x 128 x 128 floats, one
// per SM id (attn_fwd.cu).
int osum_slots(float** slots, int* n);

// LSE merge of n partials (device pointer arrays passed by value).
int launch_merge(const float* const* O_parts, const float* const* LSE_parts, int n, void* out, float* lse,
                 long long rows, int d, int out_dtype, cudaStream_t stream);

// The paged cache (kv_cache.cu) and the attention over it (attn_decode.cu, attn_seq.cu). Sequence s owns
// tokens [cu[s], cu[s+1]) of the packed tensors and positions [0, kv_lens[s]) of its pages.
struct CacheArgs {
  const void* k;        // [T, Hkv, d] new tokens, `*_stride` elements from token to token
  const void* v;
  void* k_out;          // reading: [T, Hkv, d]
  void* v_out;
  void* k_cache;        // [n_pages, Hkv, page, d]
  void* v_cache;
  unsigned char* k_scale;  // e4m3: [n_pages, Hkv, page] exponent bytes; 4 bits: [n_pages, Hkv, page, d / 32] scales
  unsigned char* v_scale;
  const int* table;     // [n_seqs, max_pages]
  const int* cu;
  const int* kv_lens;
  long long k_stride, v_stride;
  int n_seqs, T, Hkv, d, page, n_pages, max_pages, dtype, cache_dtype;
};
int launch_kv_cache(const CacheArgs& a, bool write, cudaStream_t stream);
// What appending adds to writing: the queries, and the rotation.
struct AppendArgs {
  const void* q;        // [T, Hq, d], q_stride elements from token to token (Hq 0: none)
  void* q_out;          // [T, Hq, d]
  const float* cos_sin; // [max_pos, rot]: cosines of rot / 2 pairs, then their sines
  long long q_stride, max_pos;
  int Hq, rot, interleaved;
  float minus_zero;     // -0.0f (kv_cache.cu says what for)
};
int launch_kv_append(const CacheArgs& a, const AppendArgs& r, cudaStream_t stream);

struct PagedArgs {
  const void* q;        // [T, Hq, d]
  void* out;            // [T, Hq, d]
  float* lse;           // [Hq, T] or null
  const void* k_cache;
  const void* v_cache;
  const unsigned char* k_scale;
  const unsigned char* v_scale;
  const int* table;
  const int* cu;
  const int* kv_lens;
  void* workspace;
  long long q_stride;
  long long row_seq, row_head;  // the pages of sequence s and key head h: from table + s * row_seq + h * row_head on
  int n_seqs, T, Hq, Hkv, d, page, n_pages, max_pages, max_q_len, max_kv_len, causal, dtype, cache_dtype;
  float scale;          // resolved
};
// Few rows per sequence: the split kernel of attn_decode.cu.
bool decode_applies(const PagedArgs& a);
size_t decode_workspace(const PagedArgs& a);
int launch_decode(const PagedArgs& a, cudaStream_t stream);
// Chunks of new tokens: the tensor-core kernel of attn_seq.cu.
size_t chunk_workspace(const PagedArgs& a);
int launch_chunk(const PagedArgs& a, cudaStream_t stream);

// Bounds of the keys of pages, and the selection of pages by them (attn_select.cu).
struct BoundsArgs {
  const void* k_cache;
  const unsigned char* k_scale;
  signed char* bounds;   // [n_pages, Hkv, 2, d]
  unsigned char* exps;   // [n_pages, Hkv]
  const int* table;
  const int* cu;
  const int* kv_lens;
  int n_seqs, T, Hkv, d, page, n_pages, max_pages, dtype, cache_dtype;
};
int launch_page_bounds(const BoundsArgs& a, int max_q_len, cudaStream_t stream);
struct SelectArgs {
  const void* q;         // [T, Hq, d], q_stride elements from token to token
  const signed char* bounds;
  const unsigned char* exps;
  const int* table;
  const int* cu;
  const int* kv_lens;
  int* pages;            // [T, Hkv, n_select] of the sequence's table, or null
  void* workspace;
  long long q_stride;
  int n_seqs, T, G, Hkv, d, page, n_pages, max_pages, most_pages, n_select, dtype;
  // what launch_select lays out in the workspace: scores of some tokens, and for the attention each token as a sequence of its own
  float* scores;
  int* list;             // [T, Hkv, n_select] pages of the cache
  int* cu_out;           // [T + 1]
  int* lens_out;         // [T]
};
size_t select_workspace(const SelectArgs& a);
int launch_select(SelectArgs* a, cudaStream_t stream);

// Whole prompts packed end to end (attn_seq.cu; backward: attn_bwd.cu).
struct PackedArgs {
  const void* q;        // [T, Hq, d], `*_stride` elements from token to token
  const void* k;        // [T, Hkv, d]
  const void* v;
  void* out;            // [T, Hq, d]
  float* lse;           // [Hq, T] or null
  const int* cu;
  long long q_stride, k_stride, v_stride;
  int n_seqs, T, Hq, Hkv, d, causal, dtype;
  float scale;          // resolved
};
int launch_packed(const PackedArgs& a, cudaStream_t stream);
// The gradients: a.out and a.lse are the forward's. workspace: packed_bwd_workspace bytes.
size_t packed_bwd_workspace(int n_seqs, int T, int Hq, int Hkv, int d);
int launch_packed_bwd(const PackedArgs& a, const void* dout, void* dq, void* dk, void* dv, void* workspace, cudaStream_t stream);

// Tensor maps (seq_api.cu). `strides` are bytes of dimensions 1 and up.
int encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle);
// A cache by blocks (page * Hkv + head), with boxes of `rows` slots of one block: 16-bit data as (64 features, 8 slots,
// half of the features, 8-slot group, block), which lands as [group][half][8 slots][64 features] under the 128-byte
// swizzle; e4m3 and 4 bits as (byte, slot, block), a whole vector a row (128-, 64- or 32-byte swizzle, the row's size).
int make_page_map(CUtensorMap* m, const void* cache, const PagedArgs& a, int rows);

// Copy tokens [t0, t0+n) of a [B,H,N,d] / [B,N,H,d] tensor (host or device) into a packed chunk buffer.
cudaError_t copy_chunk(void* dst, const void* src, int layout, int B, int H, long long N, int d, long long t0, int n,
                       cudaMemcpyKind kind, cudaStream_t s, long long* bytes);

// Normalised fp32 accumulator (acc [B,H,n,d], lse_acc [B,H,n]) -> out tokens [t0, t0+n) of an N-token
// tensor in `layout` and `dtype`, plus lse_out (may be NULL).
int launch_finalize(const float* acc, const float* lse_acc, void* out, float* lse_out, int B, int H, int n,
                    long long N, long long t0, int d, int layout, int dtype, cudaStream_t stream);

// Reusable device buffers, events and non-blocking streams (per device; csrc/pool.cu). A caller
// returns them only after all work using them has completed.
int pool_alloc(void** p, size_t n);
void pool_free(void* p);
int pool_event(cudaEvent_t* e, bool timing);
void pool_event_free(cudaEvent_t e, bool timing);
int pool_stream(cudaStream_t* s);
void pool_stream_free(cudaStream_t s);

// Set-up that belongs to one device's context (kernel function attributes, cached device attributes)
// runs once per device: bit `dev` records it. Concurrent first calls may both run the set-up, which is
// idempotent; devices numbered 64 and above repeat it on every call.
struct PerDeviceOnce {
  std::atomic<unsigned long long> bits{0};
  // true when the current device's set-up has run; *dev receives the current device (-1 on error)
  bool done(int* dev) const {
    if (cudaGetDevice(dev) != cudaSuccess) {
      *dev = -1;
      return false;
    }
    return seen(*dev);
  }
  // the bookkeeping alone: has device `dev` been marked (ids outside [0, 64) never are)
  bool seen(int dev) const { return dev >= 0 && dev < 64 && ((bits.load(std::memory_order_acquire) >> dev) & 1ull); }
  void mark(int dev) {
    if (dev >= 0 && dev < 64) bits.fetch_or(1ull << dev, std::memory_order_acq_rel);
  }
};

// The device error words (set by a kernel whose bounded wait gave up), read after the caller's own
// streams have drained: each word is copied on `s` and `s` is synchronised, so no other stream of the
// process is waited for. A set word is cleared and reported as CQSA_ERR_TIMEOUT with its code, block
// and site in the error message.
int check_device_error_on(cudaStream_t s);

// Number of SMs of the current device (cached per device; 152 if the query fails).
int sm_count();

// Status helpers
void set_error(const char* fmt, ...);
int cuda_status(cudaError_t e, const char* what);
unsigned long long timeout_ns();
unsigned timeout_us();  // the same limit in microseconds, held in 32 bits
int debug_fault();

}  // namespace cqsa
