// C ABI of the operators over sequences of different lengths: argument checks, workspaces and dispatch.
// Nothing here computes.
#include <math.h>
#include <string.h>

#include "cqsa_internal.h"

namespace cqsa {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

int encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  static std::atomic<EncodeTiledFn> known{nullptr};
  EncodeTiledFn enc = known.load(std::memory_order_acquire);
  if (!enc) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<EncodeTiledFn>(ptr);
    if (!enc) {
      set_error("cuTensorMapEncodeTiled is not available from the driver");
      return CQSA_ERR_CUDA;
    }
    known.store(enc, std::memory_order_release);
  }
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = enc(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
    return CQSA_ERR_CUDA;
  }
  return CQSA_OK;
}

int make_page_map(CUtensorMap* m, const void* cache, const PagedArgs& a, int rows) {
  const cuuint64_t blocks = static_cast<cuuint64_t>(a.n_pages) * a.Hkv;  // (page, head)
  if (a.cache_dtype == CQSA_E4M3) {
    const cuuint64_t vec = static_cast<cuuint64_t>(a.d);
    const cuuint64_t dims[3] = {vec, static_cast<cuuint64_t>(a.page), blocks};
    const cuuint64_t strides[2] = {vec, vec * a.page};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(a.d), static_cast<cuuint32_t>(rows), 1};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, cache, dims, strides, box,
                             a.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  }
  const cuuint64_t vec = static_cast<cuuint64_t>(a.d) * 2, halves = static_cast<cuuint64_t>(a.d / 64);
  const cuuint64_t dims[5] = {64, 8, halves, static_cast<cuuint64_t>(a.page / 8), blocks};
  const cuuint64_t strides[4] = {vec, 128, vec * 8, vec * a.page};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(halves), static_cast<cuuint32_t>(rows / 8), 1};
  return encode_tensor_map(m, a.cache_dtype == CQSA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           5, cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

unsigned timeout_us() {
  const unsigned long long us = timeout_ns() / 1000ull;
  return us >= 0xffffffffull ? 0xffffffffu : static_cast<unsigned>(us) + 1u;
}

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }

int invalid(const char* what) {
  set_error("%s", what);
  return CQSA_ERR_INVALID;
}

// What every call over sequences shares: counts, heads, head dimension and types.
int check_seqs(int n_seqs, int T, int Hq, int Hkv, int d, float scale, int dtype) {
  if (n_seqs < 1 || T < 0 || Hq < 1 || Hkv < 1) {
    set_error("sizes must be positive (n_seqs=%d T=%d Hq=%d Hkv=%d)", n_seqs, T, Hq, Hkv);
    return CQSA_ERR_INVALID;
  }
  if (Hq % Hkv != 0) {
    set_error("Hq = %d is not a multiple of Hkv = %d", Hq, Hkv);
    return CQSA_ERR_INVALID;
  }
  if (Hq / Hkv > 64) {
    set_error("%d query heads for a key head are not supported (64 at most)", Hq / Hkv);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (d != 64 && d != 128) {
    set_error("head dim %d is not supported (64 or 128)", d);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (dtype != CQSA_F16 && dtype != CQSA_BF16) {
    set_error("dtype %d is not supported for Q/K/V (fp16 or bf16)", dtype);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (!isfinite(scale) || scale < 0.0f) return invalid("scale must be finite and >= 0 (0 selects 1/sqrt(d))");
  if (static_cast<long long>(T) * Hq > 0x7fffffffLL) {
    set_error("T * Hq = %lld is too large (2^31 - 1 at most)", static_cast<long long>(T) * Hq);
    return CQSA_ERR_UNSUPPORTED;
  }
  return CQSA_OK;
}

// Token stride in elements: 0 selects heads * d; otherwise at least that, in whole 16 bytes.
int resolve_stride(long long* stride, int heads, int d, const char* name) {
  const long long dense = static_cast<long long>(heads) * d;
  if (*stride == 0) *stride = dense;
  if (*stride < dense || (*stride & 7) || *stride > (1LL << 38)) {
    set_error("%s token stride %lld: it must be 0 or a multiple of 8 elements of at least heads * d = %lld", name, *stride, dense);
    return CQSA_ERR_INVALID;
  }
  return CQSA_OK;
}

int check_cache(int Hkv, const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale, const int* table,
                int max_pages, int page, int n_pages, int dtype, int cache_dtype) {
  if (!k_cache || !v_cache || !table) return invalid("k_cache, v_cache and block_table must be non-null device pointers");
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(table, 4))
    return invalid("k_cache and v_cache must be 16-byte aligned (block_table 4-byte)");
  if (page < 16 || page > 256 || (page & (page - 1))) {
    set_error("page size %d is not supported (16, 32, 64, 128 or 256)", page);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (n_pages < 1 || max_pages < 1) return invalid("n_pages and max_pages must be positive");
  if (static_cast<long long>(max_pages) * page > 0x7fffffffLL - 512) {
    set_error("max_pages * page_size = %lld positions are too many", static_cast<long long>(max_pages) * page);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (static_cast<long long>(n_pages) * Hkv > 0x7fffffffLL) {
    set_error("n_pages * Hkv = %lld is too large (2^31 - 1 at most)", static_cast<long long>(n_pages) * Hkv);
    return CQSA_ERR_UNSUPPORTED;
  }
  if (cache_dtype == CQSA_E4M3) {
    if (!k_scale || !v_scale) return invalid("an e4m3 cache needs k_scale and v_scale");
    if (!aligned(k_scale, 16) || !aligned(v_scale, 16)) return invalid("k_scale and v_scale must be 16-byte aligned");
  } else if (cache_dtype != dtype) {
    set_error("cache_dtype %d must be the tokens' dtype or CQSA_E4M3", cache_dtype);
    return CQSA_ERR_UNSUPPORTED;
  }
  return CQSA_OK;
}

float resolve_scale(float scale, int d) { return scale == 0.0f ? 1.0f / sqrtf(static_cast<float>(d)) : scale; }

// The checks and arguments that reading and writing the cache share.
int cache_args(CacheArgs* a, void* k_cache, void* v_cache, unsigned char* k_scale, unsigned char* v_scale,
               const int* block_table, int max_pages, const int* cu, const int* kv_lens, int n_seqs, int T, int Hkv, int d,
               int page, int n_pages, int dtype, int cache_dtype) {
  int rc = check_seqs(n_seqs, T, Hkv, Hkv, d, 0.0f, dtype);
  if (rc == CQSA_OK) rc = check_cache(Hkv, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, page, n_pages, dtype, cache_dtype);
  if (rc != CQSA_OK) return rc;
  if (!cu || !kv_lens || !aligned(cu, 4) || !aligned(kv_lens, 4))
    return invalid("cu_seqlens and kv_lens must be non-null 4-byte aligned device pointers");
  memset(a, 0, sizeof(*a));
  a->k_cache = k_cache;
  a->v_cache = v_cache;
  a->k_scale = k_scale;
  a->v_scale = v_scale;
  a->table = block_table;
  a->cu = cu;
  a->kv_lens = kv_lens;
  a->n_seqs = n_seqs;
  a->T = T;
  a->Hkv = Hkv;
  a->d = d;
  a->page = page;
  a->n_pages = n_pages;
  a->max_pages = max_pages;
  a->dtype = dtype;
  a->cache_dtype = cache_dtype;
  return CQSA_OK;
}

// The checks and arguments that the packed forward and backward share.
int packed_args(PackedArgs* a, const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                long long v_stride, void* out, float* lse, const int* cu, int n_seqs, int T, int Hq, int Hkv, int d, int causal,
                float scale, int dtype) {
  set_error("%s", "");
  int rc = check_seqs(n_seqs, T, Hq, Hkv, d, scale, dtype);
  if (rc == CQSA_OK) rc = resolve_stride(&q_stride, Hq, d, "q");
  if (rc == CQSA_OK) rc = resolve_stride(&k_stride, Hkv, d, "k");
  if (rc == CQSA_OK) rc = resolve_stride(&v_stride, Hkv, d, "v");
  if (rc != CQSA_OK) return rc;
  if (!cu || !aligned(cu, 4)) return invalid("cu_seqlens must be a non-null 4-byte aligned device pointer");
  if (T > 0 && (!q || !k || !v || !out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(lse, 4)))
    return invalid("q, k, v and out must be non-null 16-byte aligned device pointers (lse 4-byte)");
  memset(a, 0, sizeof(*a));
  a->q = q;
  a->k = k;
  a->v = v;
  a->out = out;
  a->lse = lse;
  a->cu = cu;
  a->q_stride = q_stride;
  a->k_stride = k_stride;
  a->v_stride = v_stride;
  a->n_seqs = n_seqs;
  a->T = T;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->d = d;
  a->causal = causal != 0;
  a->dtype = dtype;
  a->scale = resolve_scale(scale, d);
  return CQSA_OK;
}

int paged_sizes(PagedArgs* a, int n_seqs, int T, int Hq, int Hkv, int d, int page, int max_q_len, int max_kv_len,
                int dtype, int cache_dtype) {
  memset(a, 0, sizeof(*a));
  a->n_seqs = n_seqs;
  a->T = T;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->d = d;
  a->page = page;
  a->max_q_len = max_q_len < T ? max_q_len : T;
  a->max_kv_len = max_kv_len;
  a->dtype = dtype;
  a->cache_dtype = cache_dtype;
  if (max_q_len < 0 || max_kv_len < 0) return invalid("max_q_len and max_kv_len must be >= 0");
  return CQSA_OK;
}

size_t paged_workspace(const PagedArgs& a) {
  if (a.T == 0) return 0;
  return decode_applies(a) ? decode_workspace(a) : chunk_workspace(a);
}

}  // namespace
}  // namespace cqsa

using namespace cqsa;

extern "C" {

int cqsa_attn_packed_fwd(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                         long long v_stride, void* out, float* lse, const int* cu_seqlens, int n_seqs, int T, int Hq, int Hkv,
                         int d, int causal, float scale, int dtype, cudaStream_t stream) {
  PackedArgs a;
  const int rc = packed_args(&a, q, k, v, q_stride, k_stride, v_stride, out, lse, cu_seqlens, n_seqs, T, Hq, Hkv, d, causal,
                             scale, dtype);
  if (rc != CQSA_OK || T == 0) return rc;
  return launch_packed(a, stream);
}

size_t cqsa_attn_packed_bwd_workspace_size(int n_seqs, int T, int Hq, int Hkv, int d) {
  if (T < 1 || check_seqs(n_seqs, T, Hq, Hkv, d, 0.0f, CQSA_F16) != CQSA_OK) return 0;
  return packed_bwd_workspace(n_seqs, T, Hq, Hkv, d);
}

int cqsa_attn_packed_bwd(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                         long long v_stride, const void* out, const void* dout, const float* lse, void* dq, void* dk, void* dv,
                         void* workspace, size_t workspace_bytes, const int* cu_seqlens, int n_seqs, int T, int Hq, int Hkv,
                         int d, int causal, float scale, int dtype, cudaStream_t stream) {
  PackedArgs a;
  const int rc = packed_args(&a, q, k, v, q_stride, k_stride, v_stride, const_cast<void*>(out), const_cast<float*>(lse),
                             cu_seqlens, n_seqs, T, Hq, Hkv, d, causal, scale, dtype);
  if (rc != CQSA_OK || T == 0) return rc;
  if (!dout || !lse || !dq || !dk || !dv || !aligned(dout, 16) || !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return invalid("dout, dq, dk, dv (16-byte aligned) and lse must be non-null device pointers");
  const size_t need = packed_bwd_workspace(n_seqs, T, Hq, Hkv, d);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) {
    set_error("a 16-byte aligned workspace of the %zu bytes that cqsa_attn_packed_bwd_workspace_size reports is needed (got %zu)",
              need, workspace ? workspace_bytes : static_cast<size_t>(0));
    return CQSA_ERR_INVALID;
  }
  return launch_packed_bwd(a, dout, dq, dk, dv, workspace, stream);
}

int cqsa_kv_cache_write(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache, void* v_cache,
                        unsigned char* k_scale, unsigned char* v_scale, const int* block_table, int max_pages,
                        const int* cu_seqlens, const int* kv_lens, int n_seqs, int T, int Hkv, int d, int page_size,
                        int n_pages, int dtype, int cache_dtype, cudaStream_t stream) {
  set_error("%s", "");
  CacheArgs a;
  int rc = cache_args(&a, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, cu_seqlens, kv_lens, n_seqs, T, Hkv,
                      d, page_size, n_pages, dtype, cache_dtype);
  if (rc == CQSA_OK) rc = resolve_stride(&k_stride, Hkv, d, "k");
  if (rc == CQSA_OK) rc = resolve_stride(&v_stride, Hkv, d, "v");
  if (rc != CQSA_OK) return rc;
  if (T > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16)))
    return invalid("k and v must be non-null 16-byte aligned device pointers");
  a.k = k;
  a.v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  return launch_kv_cache(a, true, stream);
}

int cqsa_kv_cache_read(void* k, void* v, const void* k_cache, const void* v_cache, const unsigned char* k_scale,
                       const unsigned char* v_scale, const int* block_table, int max_pages, const int* cu_seqlens,
                       const int* kv_lens, int n_seqs, int T, int Hkv, int d, int page_size, int n_pages, int dtype,
                       int cache_dtype, cudaStream_t stream) {
  set_error("%s", "");
  CacheArgs a;
  int rc = cache_args(&a, const_cast<void*>(k_cache), const_cast<void*>(v_cache), const_cast<unsigned char*>(k_scale),
                      const_cast<unsigned char*>(v_scale), block_table, max_pages, cu_seqlens, kv_lens, n_seqs, T, Hkv, d,
                      page_size, n_pages, dtype, cache_dtype);
  if (rc != CQSA_OK) return rc;
  if (T > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16)))
    return invalid("k and v must be non-null 16-byte aligned device pointers");
  a.k_out = k;
  a.v_out = v;
  return launch_kv_cache(a, false, stream);
}

size_t cqsa_attn_paged_workspace_size(int n_seqs, int T, int Hq, int Hkv, int d, int page_size, int max_q_len, int max_kv_len,
                                      int dtype, int cache_dtype) {
  if (check_seqs(n_seqs, T, Hq, Hkv, d, 0.0f, dtype) != CQSA_OK || page_size < 1) return 0;
  PagedArgs a;
  if (paged_sizes(&a, n_seqs, T, Hq, Hkv, d, page_size, max_q_len, max_kv_len, dtype, cache_dtype) != CQSA_OK) return 0;
  return paged_workspace(a);
}

int cqsa_attn_paged_fwd(const void* q, long long q_stride, void* out, float* lse, const void* k_cache, const void* v_cache,
                        const unsigned char* k_scale, const unsigned char* v_scale, const int* block_table, int max_pages,
                        const int* cu_seqlens, const int* kv_lens, int n_seqs, int T, int max_q_len, int max_kv_len, int Hq,
                        int Hkv, int d, int page_size, int n_pages, int causal, float scale, int dtype, int cache_dtype,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  set_error("%s", "");
  int rc = check_seqs(n_seqs, T, Hq, Hkv, d, scale, dtype);
  if (rc == CQSA_OK) rc = check_cache(Hkv, k_cache, v_cache, k_scale, v_scale, block_table, max_pages, page_size, n_pages, dtype, cache_dtype);
  if (rc == CQSA_OK) rc = resolve_stride(&q_stride, Hq, d, "q");
  if (rc != CQSA_OK) return rc;
  if (!cu_seqlens || !kv_lens || !aligned(cu_seqlens, 4) || !aligned(kv_lens, 4))
    return invalid("cu_seqlens and kv_lens must be non-null 4-byte aligned device pointers");
  PagedArgs a;
  rc = paged_sizes(&a, n_seqs, T, Hq, Hkv, d, page_size, max_q_len, max_kv_len, dtype, cache_dtype);
  if (rc != CQSA_OK || T == 0 || max_q_len == 0) return rc;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)))
    return invalid("q and out must be non-null 16-byte aligned device pointers (lse 4-byte)");
  const size_t need = paged_workspace(a);
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) {
    set_error("a 16-byte aligned workspace of the %zu bytes that cqsa_attn_paged_workspace_size reports is needed (got %zu)",
              need, workspace ? workspace_bytes : static_cast<size_t>(0));
    return CQSA_ERR_INVALID;
  }
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.kv_lens = kv_lens;
  a.workspace = workspace;
  a.q_stride = q_stride;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.causal = causal != 0;
  a.scale = resolve_scale(scale, d);
  return decode_applies(a) ? launch_decode(a, stream) : launch_chunk(a, stream);
}

}  // extern "C"
