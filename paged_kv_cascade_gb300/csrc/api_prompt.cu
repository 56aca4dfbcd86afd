// C ABI entry points of a prompt's way into the cache: pages and slots for new
// tokens, rotary positions on the way into the pool, chunk attention.
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "pkc.h"
#include "pkc_internal.h"

using namespace pkc;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A pool of pages and its table, whatever the rows hold.
int check_table(const char* call, int batch, int page_size, int block_table_stride, int64_t num_pages) {
  if (batch < 0 || page_size < 1 || block_table_stride < 1 || num_pages < 0)
    return set_error(PKC_ERR_INVALID_ARG,
                     "%s: batch and num_pages must be >= 0, page_size and block_table_stride >= 1", call);
  if ((int64_t)block_table_stride * page_size > INT32_MAX - 65536)  // token positions are 32-bit
    return set_error(PKC_ERR_UNSUPPORTED, "%s: a block table of more than 2^31 - 65537 tokens", call);
  return PKC_OK;
}

int check_free(const char* call, int batch, int64_t num_pages) {
  if (batch > PKC_PAGES_MAX_BATCH)
    return set_error(PKC_ERR_UNSUPPORTED, "%s: more than %d requests (got %d)", call, PKC_PAGES_MAX_BATCH, batch);
  if (num_pages > PKC_PAGES_MAX_PAGES)
    return set_error(PKC_ERR_UNSUPPORTED, "%s: a pool of more than 2^26 pages", call);
  return PKC_OK;
}

bool power_of_two(float x) {
  int e;
  return std::frexp(x, &e) == 0.5f;
}

// Whether n dense rows of o_row 16-bit elements from o on meet n rows of x_row elements,
// `stride` apart, from x on.  (In elements: addresses are even, and sums stay below 2^64.)
bool rows_meet(const void* o, const void* x, uint64_t o_row, uint64_t x_row, uint64_t stride, uint64_t n) {
  const uint64_t o0 = reinterpret_cast<uintptr_t>(o) / 2, x0 = reinterpret_cast<uintptr_t>(x) / 2;
  const uint64_t first = o0 < x0 + x_row ? 0 : (o0 - x0 - x_row) / stride + 1;  // the first row that ends behind o
  return first < n && x0 + first * stride < o0 + n * o_row;
}

}  // namespace

extern "C" {

int pkc_release_pages(int32_t* block_table, int block_table_stride, const int32_t* cache_seqlens, int batch,
                      int page_size, int64_t num_pages, uint32_t* free_pages, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (int rc = check_table("release_pages", batch, page_size, block_table_stride, num_pages)) return rc;
  if (int rc = check_free("release_pages", batch, num_pages)) return rc;
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (batch == 0) return PKC_OK;
  if (!block_table || !cache_seqlens || !free_pages)
    return set_error(PKC_ERR_INVALID_ARG, "release_pages: NULL pointer");
  if (!aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(free_pages, 4))
    return set_error(PKC_ERR_INVALID_ARG, "release_pages: arrays must be 4-byte aligned");
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.block_table = block_table; p.cache_seqlens = cache_seqlens; p.free_pages = free_pages;
  p.bt_stride = block_table_stride; p.num_pages = num_pages; p.batch = batch; p.page_size = page_size;
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_release_pages(p, stream);
  return e ? cuda_error(e, "release_pages launch") : PKC_OK;
}

int pkc_assign_pages(int32_t* block_table, int block_table_stride, const int32_t* cache_seqlens,
                     const int32_t* new_indptr, int total_new, int batch, int page_size, int64_t num_pages,
                     uint32_t* free_pages, int64_t* slots, int32_t* positions, int32_t* seqlens_out, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (int rc = check_table("assign_pages", batch, page_size, block_table_stride, num_pages)) return rc;
  if (int rc = check_free("assign_pages", batch, num_pages)) return rc;
  if (total_new < 0)
    return set_error(PKC_ERR_INVALID_ARG, "assign_pages: total_new must be >= 0 (got %d)", total_new);
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (batch == 0 && total_new == 0) return PKC_OK;
  if (total_new > 0 && (!slots || !positions)) return set_error(PKC_ERR_INVALID_ARG, "assign_pages: NULL pointer");
  if (batch > 0 && (!block_table || !cache_seqlens || !new_indptr || !free_pages))
    return set_error(PKC_ERR_INVALID_ARG, "assign_pages: NULL pointer");
  if (!aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(new_indptr, 4) || !aligned(free_pages, 4) ||
      !aligned(slots, 8) || !aligned(positions, 4) || !aligned(seqlens_out, 4))
    return set_error(PKC_ERR_INVALID_ARG, "assign_pages: slots must be 8-byte aligned, other arrays 4-byte");
  PagesParams p;
  std::memset(&p, 0, sizeof(p));
  p.block_table = block_table; p.cache_seqlens = cache_seqlens; p.indptr = new_indptr; p.free_pages = free_pages;
  p.slots = slots; p.positions = positions; p.seqlens_out = seqlens_out;
  p.bt_stride = block_table_stride; p.num_pages = num_pages; p.batch = batch; p.page_size = page_size;
  p.total = total_new;
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_assign_pages(p, stream);
  return e ? cuda_error(e, "assign_pages launch") : PKC_OK;
}

int pkc_rope_append_kv(const void* q, int64_t q_stride, const void* k_new, const void* v_new, int64_t kv_stride,
                       const int32_t* positions, const int64_t* slots, const double* inv_freq, int rotary_dim,
                       int interleaved, float amplitude, int total, int num_qo_heads, int num_kv_heads, int head_dim,
                       void* q_out, void* k_cache, void* v_cache, int page_size, int64_t num_pages, float k_scale,
                       float v_scale, int dtype, int kv_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (total < 0 || num_qo_heads <= 0 || num_kv_heads <= 0 || page_size < 1 || num_pages < 0)
    return set_error(PKC_ERR_INVALID_ARG,
                     "rope_append_kv: total and num_pages must be >= 0, head counts and page_size >= 1");
  if (head_dim != PKC_HEAD_DIM)
    return set_error(PKC_ERR_UNSUPPORTED, "rope_append_kv: head_dim must be %d (got %d)", PKC_HEAD_DIM, head_dim);
  if (num_qo_heads > 1 << 16 || num_kv_heads > 1 << 16)  // a token's rows are addressed with 32 bits
    return set_error(PKC_ERR_UNSUPPORTED, "rope_append_kv: more than 2^16 heads");
  if (num_pages > INT32_MAX)  // page ids are 32-bit
    return set_error(PKC_ERR_UNSUPPORTED, "rope_append_kv: a pool of more than 2^31 - 1 pages");
  if (rotary_dim < 2 || rotary_dim > PKC_HEAD_DIM || rotary_dim % 2 != 0)
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: rotary_dim must be even, in 2 .. %d (got %d)", PKC_HEAD_DIM,
                     rotary_dim);
  if (rotary_dim % 16 != 0)
    return set_error(PKC_ERR_UNSUPPORTED, "rope_append_kv: rotary_dim must be a multiple of 16 (got %d)", rotary_dim);
  if (interleaved != 0 && interleaved != 1)
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: interleaved must be 0 or 1 (got %d)", interleaved);
  if (dtype != PKC_F16 && dtype != PKC_BF16)
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: dtype must be PKC_F16 or PKC_BF16 (got %d)", dtype);
  if (kv_dtype != dtype && kv_dtype != PKC_E4M3)
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: kv_dtype must be dtype or PKC_E4M3 (got %d)", kv_dtype);
  if (!std::isfinite(amplitude)) return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: amplitude must be finite");
  // (the reciprocal of a power of two has to be a normal number)
  if (!(k_scale >= 0x1p-100f && k_scale <= 0x1p100f && v_scale >= 0x1p-100f && v_scale <= 0x1p100f) ||
      (kv_dtype != PKC_E4M3 && (k_scale != 1.f || v_scale != 1.f)))
    return set_error(PKC_ERR_INVALID_ARG,
                     "rope_append_kv: k_scale and v_scale must be in 2^-100 .. 2^100, and 1 but for an e4m3 cache");
  if (q_stride < (int64_t)num_qo_heads * PKC_HEAD_DIM || kv_stride < (int64_t)num_kv_heads * PKC_HEAD_DIM ||
      q_stride % 8 != 0 || kv_stride % 8 != 0)
    return set_error(PKC_ERR_INVALID_ARG,
                     "rope_append_kv: strides must be multiples of 8 elements and at least a token's rows");
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (total == 0) return PKC_OK;
  if (!q || !k_new || !v_new || !positions || !slots || !inv_freq || !q_out || !k_cache || !v_cache)
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: NULL pointer");
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) || !aligned16(k_cache) ||
      !aligned16(v_cache) || !aligned(slots, 8) || !aligned(inv_freq, 8) || !aligned(positions, 4))
    return set_error(PKC_ERR_INVALID_ARG,
                     "rope_append_kv: rows and pools must be 16-byte aligned, slots and inv_freq 8-byte");
  // a row of q, k_new or v_new may be read after the rows of other tokens are written
  const uint64_t q_row = (uint64_t)num_qo_heads * PKC_HEAD_DIM;
  const bool in_place = q_out == q && (total == 1 || (uint64_t)q_stride == q_row);
  if (!in_place && rows_meet(q_out, q, q_row, q_row, q_stride, total))
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: q_out must not overlap q, but may be q if q is dense");
  const uint64_t kv_row = (uint64_t)num_kv_heads * PKC_HEAD_DIM;
  if (rows_meet(q_out, k_new, q_row, kv_row, kv_stride, total) || rows_meet(q_out, v_new, q_row, kv_row, kv_stride, total))
    return set_error(PKC_ERR_INVALID_ARG, "rope_append_kv: q_out must not overlap k_new or v_new");
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q; p.k_new = k_new; p.v_new = v_new; p.q_stride = q_stride; p.kv_stride = kv_stride;
  p.positions = positions; p.slots = slots; p.inv_freq = inv_freq;
  p.q_out = q_out; p.k_cache = k_cache; p.v_cache = v_cache; p.pool_tokens = num_pages * page_size;
  p.rotary_dim = rotary_dim; p.interleaved = interleaved; p.total = total; p.hq = num_qo_heads; p.hkv = num_kv_heads;
  p.amplitude = amplitude; p.k_scale = k_scale; p.v_scale = v_scale;
  p.k_inv_scale = 1.f / k_scale; p.v_inv_scale = 1.f / v_scale;
  p.divide = !(power_of_two(k_scale) && power_of_two(v_scale));
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_rope_append(p, dtype, kv_dtype, stream);
  return e ? cuda_error(e, "rope_append_kv launch") : PKC_OK;
}

int pkc_chunk_workspace_size(size_t* bytes) {
  if (!bytes) return set_error(PKC_ERR_INVALID_ARG, "chunk_workspace_size: NULL pointer");
  *bytes = PKC_STATUS_BYTES + chunk_partial_bytes();
  return PKC_OK;
}

int pkc_paged_chunk_state(const void* q, const int32_t* q_indptr, int total_q, const void* k_cache,
                          const void* v_cache, const int32_t* block_table, int block_table_stride,
                          const int32_t* cache_seqlens, int batch, int num_qo_heads, int num_kv_heads, int head_dim,
                          int page_size, int64_t num_pages, float sm_scale, int causal, int window, void* workspace,
                          size_t workspace_bytes, void* o, float* lse, int dtype, int out_dtype, void* stream) {
  if (int rc = check_attn_dims(batch, num_qo_heads, num_kv_heads, head_dim, dtype)) return rc;
  if (int rc = check_table("paged_chunk_state", batch, page_size, block_table_stride, num_pages)) return rc;
  if (num_kv_heads > 1 << 16)
    return set_error(PKC_ERR_UNSUPPORTED, "paged_chunk_state: more than 2^16 KV heads (got %d)", num_kv_heads);
  if (num_pages > INT32_MAX - 1)  // page ids are 32-bit; num_pages itself stands for "no page"
    return set_error(PKC_ERR_UNSUPPORTED, "paged_chunk_state: a pool of more than 2^31 - 2 pages");
  if (total_q < 0) return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: total_q must be >= 0 (got %d)", total_q);
  if (!std::isfinite(sm_scale * 1.4426950408889634f) || sm_scale < 0.f)
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: sm_scale must be finite and >= 0");
  if (causal != 0 && causal != 1)
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: causal must be 0 or 1 (got %d)", causal);
  if (window < 0) return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: window must be >= 0 (got %d)", window);
  if (out_dtype != dtype && out_dtype != PKC_F32)
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: out_dtype must be dtype or PKC_F32 (got %d)", out_dtype);
  const size_t partial = chunk_partial_bytes();
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES + partial)) return rc;
  if (batch == 0 || total_q == 0) return PKC_OK;
  if (!q || !q_indptr || !k_cache || !v_cache || !block_table || !cache_seqlens || !o || !lse)
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: NULL pointer");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned(lse, 4) ||
      !aligned(q_indptr, 4) || !aligned(block_table, 4) || !aligned(cache_seqlens, 4))
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: q, o and the caches must be 16-byte aligned");
  // a row of q may be read after the rows next to it are written
  const uintptr_t rows = (uintptr_t)total_q * num_qo_heads * PKC_HEAD_DIM;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
  if (q0 < o0 + rows * (out_dtype == PKC_F32 ? 4 : 2) && o0 < q0 + rows * 2)
    return set_error(PKC_ERR_INVALID_ARG, "paged_chunk_state: o must not overlap q");
  ChunkParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q; p.q_indptr = q_indptr; p.total_q = total_q; p.k_cache = k_cache; p.v_cache = v_cache;
  p.block_table = block_table; p.cache_seqlens = cache_seqlens; p.bt_stride = block_table_stride;
  p.num_pages = num_pages; p.batch = batch; p.hq = num_qo_heads; p.hkv = num_kv_heads;
  p.g = num_qo_heads / num_kv_heads; p.page_size = page_size;
  p.causal = causal; p.window = window;
  p.scale_log2 = sm_scale * 1.4426950408889634f;
  p.o = o; p.lse = lse; p.out_dtype = out_dtype;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t at = (workspace_bytes - partial) & ~size_t(255);  // >= PKC_STATUS_BYTES, a multiple of 256 like partial
  p.part_o = reinterpret_cast<float*>(ws + at);
  p.part_ml = nullptr;  // set by the launcher, behind part_o
  p.status = reinterpret_cast<int32_t*>(ws);
  const int e = launch_paged_chunk(p, dtype, stream);
  return e ? cuda_error(e, "paged_chunk_state launch") : PKC_OK;
}

}  // extern "C"
