// paged.cuh -- what the paged K/V cache's kernels share: element access and the host-side
// checks of rq_paged_kv (include/rq.h).
#pragma once

#include <limits.h>

#include "../../include/rq.h"
#include "common.cuh"

namespace rqk {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The cache's own description: sizes, types, alignment.
inline rq_status paged_kv_check(const rq_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return RQ_ERR_ARG;
  if (kv->dtype != RQ_F32 && kv->dtype != RQ_BF16) return RQ_ERR_ARG;
  if (kv->heads < 1 || kv->block_size < 1 || kv->n_blocks < 1) return RQ_ERR_ARG;
  if (kv->head_dim != 32 && kv->head_dim != 64 && kv->head_dim != 128) return RQ_ERR_UNSUPPORTED;
  const int64_t unit = kv->dtype == RQ_BF16 ? 8 : 4;  // elements of 16 bytes
  for (int64_t s : {kv->block_stride, kv->row_stride, kv->head_stride})
    if (s < 0 || s % unit != 0) return RQ_ERR_ARG;
  return RQ_OK;
}

}  // namespace rqk
