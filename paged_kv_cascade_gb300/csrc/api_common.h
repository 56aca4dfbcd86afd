// Argument checks and plan look-ups shared by the C entry points.
#pragma once
#include <cstddef>
#include <cstdint>

#include "pkc.h"
#include "pkc_internal.h"

namespace pkc {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int check_attn_dims(int batch, int hq, int hkv, int head_dim, int dtype) {
  if (batch < 0) return set_error(PKC_ERR_INVALID_ARG, "batch must be >= 0 (got %d)", batch);
  if (head_dim != PKC_HEAD_DIM)
    return set_error(PKC_ERR_UNSUPPORTED, "head_dim %d is not supported (only 128)", head_dim);
  if (hkv <= 0 || hq <= 0 || hq % hkv != 0)
    return set_error(PKC_ERR_INVALID_ARG, "num_qo_heads (%d) must be a positive multiple of num_kv_heads (%d)",
                     hq, hkv);
  const int g = hq / hkv;
  if (g != 1 && g != 2 && g != 4 && g != 8)
    return set_error(PKC_ERR_UNSUPPORTED, "query heads per KV head must be 1, 2, 4 or 8 (got %d)", g);
  if (dtype != PKC_F16 && dtype != PKC_BF16)
    return set_error(PKC_ERR_INVALID_ARG, "dtype must be PKC_F16 or PKC_BF16 (got %d)", dtype);
  return PKC_OK;
}

inline int check_plan(const int32_t* plan, int batch) {
  if (!plan) return PKC_OK;
  if (plan[PKC_PLAN_MAGIC] != PKC_PLAN_MAGIC_VALUE) return set_error(PKC_ERR_PLAN, "plan: bad magic word");
  if (plan[PKC_PLAN_N_REQ] != batch)
    return set_error(PKC_ERR_PLAN, "plan was made for %d requests, call has batch %d", plan[PKC_PLAN_N_REQ], batch);
  if (plan[PKC_PLAN_TILE_Q] != 1 || plan[PKC_PLAN_N_UNITS] != batch)
    return set_error(PKC_ERR_PLAN, "decode needs a plan with tile_q 1 and one query row per request");
  if (plan[PKC_PLAN_NUM_CTAS] < 1) return set_error(PKC_ERR_PLAN, "plan: num_ctas < 1");
  return PKC_OK;
}

inline int check_ws(const void* ws, size_t bytes, size_t need) {
  if (!ws) return set_error(PKC_ERR_WORKSPACE, "workspace is NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return set_error(PKC_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < need) return set_error(PKC_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  return PKC_OK;
}

// Copy the plan-array offsets the contraction kernel needs.
inline void contract_plan_offsets(ContractParams& c, const int32_t* plan_host) {
  if (!plan_host) return;
  c.plan_words = plan_host[PKC_PLAN_TOTAL_WORDS];
  c.off_unit_list = plan_host[PKC_PLAN_OFF_UNIT_LIST];
  c.off_unit_req = plan_host[PKC_PLAN_OFF_UNIT_REQ];
  c.off_unit_n_chunks = plan_host[PKC_PLAN_OFF_UNIT_N_CHUNKS];
  c.off_unit_partial_begin = plan_host[PKC_PLAN_OFF_UNIT_PARTIAL_BEGIN];
}

}  // namespace pkc
