// C ABI entry points of the compressed, bounded cache: the mx4 paged cache
// (append, read-back, decode) and eviction (accumulated attention weights,
// select, compact).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "pkc.h"
#include "pkc_internal.h"

using namespace pkc;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

int page_shift_of(int page_size) {
  for (int s = 0; s < 31; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// Sizes of a paged pool and its table.
int check_pool(const char* call, int batch, int hkv, int head_dim, int page_size, int block_table_stride,
               int64_t num_pages) {
  if (batch < 0 || hkv <= 0 || page_size < 1 || block_table_stride < 1 || num_pages < 0)
    return set_error(PKC_ERR_INVALID_ARG,
                     "%s: batch and num_pages must be >= 0, num_kv_heads, page_size and block_table_stride >= 1", call);
  if (head_dim != PKC_HEAD_DIM)
    return set_error(PKC_ERR_UNSUPPORTED, "%s: head_dim must be %d (got %d)", call, PKC_HEAD_DIM, head_dim);
  if (hkv > 1 << 16)  // a token's rows are addressed with 32 bits
    return set_error(PKC_ERR_UNSUPPORTED, "%s: more than 2^16 KV heads (got %d)", call, hkv);
  if ((int64_t)block_table_stride * page_size > INT32_MAX - 65536)  // token positions are 32-bit
    return set_error(PKC_ERR_UNSUPPORTED, "%s: a block table of more than 2^31 - 65537 tokens", call);
  if (num_pages > (int64_t)(UINT32_MAX - 1) / page_size)  // and slots of the pool
    return set_error(PKC_ERR_UNSUPPORTED, "%s: a pool of more than 2^32 - 2 tokens", call);
  return PKC_OK;
}

int check_mx4_pools(const char* call, const void* k_codes, const void* k_scales, const void* v_codes,
                    const void* v_scales) {
  if (!k_codes || !k_scales || !v_codes || !v_scales) return set_error(PKC_ERR_INVALID_ARG, "%s: NULL cache pointer", call);
  if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned4(k_scales) || !aligned4(v_scales))
    return set_error(PKC_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned, scales 4-byte aligned", call);
  return PKC_OK;
}

// The common part of append and gather: every field but the 16-bit rows.
int fill_rows(Mx4RowsParams& p, const char* call, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
              const int32_t* block_table, int block_table_stride, const int32_t* indptr, const int32_t* base,
              int total, int batch, int hkv, int head_dim, int page_size, int64_t num_pages, int dtype,
              void* workspace, size_t workspace_bytes) {
  if (int rc = check_pool(call, batch, hkv, head_dim, page_size, block_table_stride, num_pages)) return rc;
  if (total < 0) return set_error(PKC_ERR_INVALID_ARG, "%s: the number of rows must be >= 0 (got %d)", call, total);
  if (dtype != PKC_F16 && dtype != PKC_BF16)
    return set_error(PKC_ERR_INVALID_ARG, "%s: dtype must be PKC_F16 or PKC_BF16 (got %d)", call, dtype);
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  std::memset(&p, 0, sizeof(p));
  if (batch == 0 || total == 0) return PKC_OK;
  if (int rc = check_mx4_pools(call, k_codes, k_scales, v_codes, v_scales)) return rc;
  if (!block_table || !indptr || !base) return set_error(PKC_ERR_INVALID_ARG, "%s: NULL pointer", call);
  p.k_codes = k_codes; p.k_scales = k_scales; p.v_codes = v_codes; p.v_scales = v_scales;
  p.block_table = block_table; p.indptr = indptr; p.base = base;
  p.bt_stride = block_table_stride; p.num_pages = num_pages;
  p.total = total; p.batch = batch; p.hkv = hkv; p.page_size = page_size; p.page_shift = page_shift_of(page_size);
  p.status = static_cast<int32_t*>(workspace);
  return PKC_OK;
}

}  // namespace

extern "C" {

int pkc_append_kv_mx4(const void* k_new, const void* v_new, const int32_t* new_indptr, int total_new, void* k_codes,
                      void* k_scales, void* v_codes, void* v_scales, const int32_t* block_table,
                      int block_table_stride, int32_t* cache_seqlens, int batch, int num_kv_heads, int head_dim,
                      int page_size, int64_t num_pages, int dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  Mx4RowsParams p;
  if (int rc = fill_rows(p, "append_kv_mx4", k_codes, k_scales, v_codes, v_scales, block_table, block_table_stride,
                         new_indptr, cache_seqlens, total_new, batch, num_kv_heads, head_dim, page_size, num_pages,
                         dtype, workspace, workspace_bytes))
    return rc;
  if (batch == 0 || total_new == 0) return PKC_OK;
  if (!k_new || !v_new) return set_error(PKC_ERR_INVALID_ARG, "append_kv_mx4: NULL pointer");
  if (!aligned16(k_new) || !aligned16(v_new))
    return set_error(PKC_ERR_INVALID_ARG, "append_kv_mx4: k_new and v_new must be 16-byte aligned");
  p.k_rows = k_new; p.v_rows = v_new; p.lengths = cache_seqlens;
  const int e = launch_append_mx4(p, dtype, stream);
  return e ? cuda_error(e, "append_kv_mx4 launch") : PKC_OK;
}

int pkc_gather_kv_mx4(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                      const int32_t* block_table, int block_table_stride, const int32_t* first,
                      const int32_t* out_indptr, int total, int batch, int num_kv_heads, int head_dim, int page_size,
                      int64_t num_pages, void* k_out, void* v_out, int dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  Mx4RowsParams p;
  if (int rc = fill_rows(p, "gather_kv_mx4", const_cast<void*>(k_codes), const_cast<void*>(k_scales),
                         const_cast<void*>(v_codes), const_cast<void*>(v_scales), block_table, block_table_stride,
                         out_indptr, first, total, batch, num_kv_heads, head_dim, page_size, num_pages, dtype,
                         workspace, workspace_bytes))
    return rc;
  if (batch == 0 || total == 0) return PKC_OK;
  if (!k_out || !v_out) return set_error(PKC_ERR_INVALID_ARG, "gather_kv_mx4: NULL pointer");
  if (!aligned16(k_out) || !aligned16(v_out))
    return set_error(PKC_ERR_INVALID_ARG, "gather_kv_mx4: k_out and v_out must be 16-byte aligned");
  p.k_out = k_out; p.v_out = v_out;
  const int e = launch_gather_mx4(p, dtype, stream);
  return e ? cuda_error(e, "gather_kv_mx4 launch") : PKC_OK;
}

int pkc_paged_decode_state_mx4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                               const void* v_scales, const int32_t* block_table, int block_table_stride,
                               const int32_t* cache_seqlens, int batch, int num_qo_heads, int num_kv_heads,
                               int head_dim, int page_size, int64_t num_pages, float sm_scale,
                               const int32_t* plan_host, void* workspace, size_t workspace_bytes, void* o, float* lse,
                               int dtype, void* stream) {
  if (int rc = check_attn_dims(batch, num_qo_heads, num_kv_heads, head_dim, dtype)) return rc;
  if (int rc = check_plan(plan_host, batch)) return rc;
  if (int rc = check_pool("paged_decode_state_mx4", batch, num_kv_heads, head_dim, page_size, block_table_stride,
                          num_pages))
    return rc;
  const int num_ctas = plan_host ? plan_host[PKC_PLAN_NUM_CTAS] : 0;
  const WsLayout L = ws_layout(batch, num_qo_heads, head_dim, num_ctas);
  if (int rc = check_ws(workspace, workspace_bytes, L.fixed_end)) return rc;
  if (batch == 0) return PKC_OK;
  if (int rc = check_mx4_pools("paged_decode_state_mx4", k_codes, k_scales, v_codes, v_scales)) return rc;
  if (!q || !block_table || !cache_seqlens || !o || !lse)
    return set_error(PKC_ERR_INVALID_ARG, "paged_decode_state_mx4: NULL pointer");
  if (!aligned16(q) || !aligned16(o))
    return set_error(PKC_ERR_INVALID_ARG, "paged_decode_state_mx4: q and o must be 16-byte aligned");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Mx4DecodeParams mp;
  std::memset(&mp, 0, sizeof(mp));
  DecodeParams& dp = mp.d;
  dp.q = q; dp.k_cache = k_codes; dp.v_cache = v_codes;
  mp.k_scales = k_scales; mp.v_scales = v_scales; mp.num_ctas = num_ctas; mp.page_shift = page_shift_of(page_size);
  dp.block_table = block_table; dp.cache_seqlens = cache_seqlens;
  dp.bt_stride = block_table_stride; dp.num_pages = num_pages;
  dp.batch = batch; dp.hq = num_qo_heads; dp.hkv = num_kv_heads; dp.page_size = page_size;
  dp.scale_log2 = sm_scale * 1.4426950408889634f;
  dp.plan = plan_host ? reinterpret_cast<const int32_t*>(ws + L.plan) : nullptr;
  dp.plan_words = plan_host ? plan_host[PKC_PLAN_TOTAL_WORDS] : 0;
  dp.o_direct = o; dp.lse_direct = lse;
  dp.part_o = reinterpret_cast<float*>(ws + L.part_o);
  dp.part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  dp.status = reinterpret_cast<int32_t*>(ws);
  int e = launch_paged_decode_mx4(mp, plan_host ? plan_host[PKC_PLAN_N_WORK] : 0, dtype, stream);
  if (e) return cuda_error(e, "paged_decode_state_mx4 launch");
  if (plan_host) {  // split requests' partial states (+) into the output
    Mx4JoinParams jp;
    std::memset(&jp, 0, sizeof(jp));
    jp.plan = dp.plan; jp.plan_words = dp.plan_words;
    jp.batch = batch; jp.hq = num_qo_heads;
    jp.part_o = dp.part_o; jp.part_lse = dp.part_lse;
    jp.o = o; jp.lse = lse;
    e = launch_join_mx4(jp, plan_host[PKC_PLAN_N_SPLIT] + plan_host[PKC_PLAN_N_EMPTY],
                        plan_host[PKC_PLAN_N_PARTIALS], dtype, stream);
    if (e) return cuda_error(e, "paged_decode_state_mx4 join launch");
  }
  return PKC_OK;
}

int pkc_accumulate_weights(const void* q, const float* lse, const void* k_cache, const void* k_scales,
                           const int32_t* block_table, int block_table_stride, const int32_t* cache_seqlens,
                           int batch, int num_qo_heads, int num_kv_heads, int head_dim, int page_size,
                           int64_t num_pages, float sm_scale, float k_scale, float decay, float* weights,
                           int64_t weights_stride, int dtype, int kv_dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (int rc = check_attn_dims(batch, num_qo_heads, num_kv_heads, head_dim, dtype)) return rc;
  if (int rc = check_pool("accumulate_weights", batch, num_kv_heads, head_dim, page_size, block_table_stride,
                          num_pages))
    return rc;
  const bool pair = kv_dtype == PKC_MX4 || (kv_dtype == PKC_E4M3 && dtype == PKC_F16) ||
                    ((kv_dtype == PKC_F16 || kv_dtype == PKC_BF16) && dtype == kv_dtype);
  if (!pair)
    return set_error(PKC_ERR_INVALID_ARG,
                     "accumulate_weights: no queries of dtype %d with a cache of kv_dtype %d (16-bit caches take "
                     "their own type, e4m3 fp16, mx4 fp16 or bf16)",
                     dtype, kv_dtype);
  if (!(k_scale > 0.f) || !std::isfinite(k_scale) || (kv_dtype != PKC_E4M3 && k_scale != 1.f))
    return set_error(PKC_ERR_INVALID_ARG, "accumulate_weights: k_scale must be finite and > 0, and 1 but for an e4m3 cache");
  if (!(decay >= 0.f && decay <= 1.f))
    return set_error(PKC_ERR_INVALID_ARG, "accumulate_weights: decay must be in [0, 1]");
  if (weights_stride < 1) return set_error(PKC_ERR_INVALID_ARG, "accumulate_weights: weights_stride must be >= 1");
  if ((int64_t)batch * num_kv_heads > INT32_MAX / 32)
    return set_error(PKC_ERR_UNSUPPORTED, "accumulate_weights: more than 2^26 (request, head) rows");
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (batch == 0) return PKC_OK;
  if (!q || !lse || !k_cache || !block_table || !cache_seqlens || !weights || (kv_dtype == PKC_MX4 && !k_scales))
    return set_error(PKC_ERR_INVALID_ARG, "accumulate_weights: NULL pointer");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned4(k_scales))
    return set_error(PKC_ERR_INVALID_ARG, "accumulate_weights: q and k_cache must be 16-byte aligned, k_scales 4-byte");
  WeightsParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q; p.lse = lse; p.k_cache = k_cache; p.k_scales = k_scales;
  p.block_table = block_table; p.cache_seqlens = cache_seqlens; p.weights = weights;
  p.bt_stride = block_table_stride; p.num_pages = num_pages; p.w_stride = weights_stride;
  p.batch = batch; p.hkv = num_kv_heads; p.g = num_qo_heads / num_kv_heads;
  p.page_size = page_size; p.page_shift = page_shift_of(page_size);
  p.scale_log2 = sm_scale * k_scale * 1.4426950408889634f;
  p.decay = decay;
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_weights(p, dtype, kv_dtype, stream);
  return e ? cuda_error(e, "accumulate_weights launch") : PKC_OK;
}

int pkc_evict_select(const float* weights, int64_t weights_stride, const int32_t* cache_seqlens, int batch,
                     int num_kv_heads, int budget, int sinks, int recent, int32_t* keep, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (batch < 0 || num_kv_heads <= 0 || weights_stride < 1)
    return set_error(PKC_ERR_INVALID_ARG, "evict_select: batch must be >= 0, num_kv_heads and weights_stride >= 1");
  if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
    return set_error(PKC_ERR_INVALID_ARG,
                     "evict_select: budget must be >= 1, sinks and recent >= 0 and together at most the budget "
                     "(got %d, %d, %d)",
                     budget, sinks, recent);
  if (budget > 1 << 30) return set_error(PKC_ERR_UNSUPPORTED, "evict_select: a budget of more than 2^30");
  if (weights_stride > (int64_t)1 << 22)
    return set_error(PKC_ERR_UNSUPPORTED, "evict_select: rows of more than 2^22 weights");
  if ((int64_t)batch * num_kv_heads > INT32_MAX / 8)
    return set_error(PKC_ERR_UNSUPPORTED, "evict_select: more than 2^28 rows");
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (batch == 0) return PKC_OK;
  if (!weights || !cache_seqlens || !keep) return set_error(PKC_ERR_INVALID_ARG, "evict_select: NULL pointer");
  SelectParams p;
  std::memset(&p, 0, sizeof(p));
  p.weights = weights; p.cache_seqlens = cache_seqlens; p.keep = keep; p.w_stride = weights_stride;
  p.batch = batch; p.hkv = num_kv_heads; p.budget = budget; p.sinks = sinks; p.recent = recent;
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_evict_select(p, stream);
  return e ? cuda_error(e, "evict_select launch") : PKC_OK;
}

int pkc_evict_compact(const int32_t* keep, int budget, void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                      const int32_t* block_table, int block_table_stride, int32_t* cache_seqlens, float* weights,
                      int64_t weights_stride, int batch, int num_kv_heads, int head_dim, int page_size,
                      int64_t num_pages, int kv_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_pool("evict_compact", batch, num_kv_heads, head_dim, page_size, block_table_stride, num_pages))
    return rc;
  if (budget < 1) return set_error(PKC_ERR_INVALID_ARG, "evict_compact: budget must be >= 1 (got %d)", budget);
  if (budget > 1 << 30) return set_error(PKC_ERR_UNSUPPORTED, "evict_compact: a budget of more than 2^30");
  if (kv_dtype != PKC_F16 && kv_dtype != PKC_BF16 && kv_dtype != PKC_E4M3 && kv_dtype != PKC_MX4)
    return set_error(PKC_ERR_INVALID_ARG, "evict_compact: kv_dtype must be PKC_F16, PKC_BF16, PKC_E4M3 or PKC_MX4 (got %d)",
                     kv_dtype);
  if (weights && weights_stride < 1) return set_error(PKC_ERR_INVALID_ARG, "evict_compact: weights_stride must be >= 1");
  if ((int64_t)batch * num_kv_heads > INT32_MAX / 32)
    return set_error(PKC_ERR_UNSUPPORTED, "evict_compact: more than 2^26 (request, head) rows");
  if (int rc = check_ws(workspace, workspace_bytes, PKC_STATUS_BYTES)) return rc;
  if (batch == 0) return PKC_OK;
  const bool mx4 = kv_dtype == PKC_MX4;
  if (!keep || !k_cache || !v_cache || !block_table || !cache_seqlens || (mx4 && (!k_scales || !v_scales)))
    return set_error(PKC_ERR_INVALID_ARG, "evict_compact: NULL pointer");
  if (!aligned16(k_cache) || !aligned16(v_cache) || (mx4 && (!aligned4(k_scales) || !aligned4(v_scales))))
    return set_error(PKC_ERR_INVALID_ARG, "evict_compact: caches must be 16-byte aligned, scales 4-byte");
  CompactParams p;
  std::memset(&p, 0, sizeof(p));
  p.keep = keep; p.budget = budget; p.k_cache = k_cache; p.v_cache = v_cache;
  p.k_scales = mx4 ? k_scales : nullptr; p.v_scales = mx4 ? v_scales : nullptr;
  p.weights = weights; p.w_stride = weights_stride;
  p.block_table = block_table; p.cache_seqlens = cache_seqlens;
  p.bt_stride = block_table_stride; p.num_pages = num_pages;
  p.batch = batch; p.hkv = num_kv_heads; p.page_size = page_size; p.page_shift = page_shift_of(page_size);
  p.row_bytes = mx4 ? 64 : kv_dtype == PKC_E4M3 ? 128 : 256;
  p.status = static_cast<int32_t*>(workspace);
  const int e = launch_evict_compact(p, stream);
  return e ? cuda_error(e, "evict_compact launch") : PKC_OK;
}

}  // extern "C"
