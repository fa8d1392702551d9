// What the calls over a paged key/value cache share (include/asffn.h, "Tree
// attention"): the checks of its descriptor and of the requests, and the place
// of a token in it.
#pragma once

#include "asffn.h"
#include "common.cuh"
#include "host.cuh"

namespace asf {

inline asf_status check_cache(const asf_kv_cache *c) {
  if (!c || !c->k || !c->v) return ASF_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->page <= 0 || c->heads <= 0 || c->head_dim <= 0) return ASF_ERR_INVALID_ARG;
  if (c->head_dim > 128 || c->heads > ASF_MAX_KV_HEADS) return ASF_ERR_UNSUPPORTED;
  if (c->head_dim % 8 || c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8) return ASF_ERR_MISALIGNED;
  if (!al16(c->k) || !al16(c->v)) return ASF_ERR_MISALIGNED;
  if (c->page_stride < 0 || c->token_stride < c->head_dim || c->head_stride < 0 ||
      (c->heads > 1 && c->head_stride < c->head_dim) || (c->pages > 1 && c->page_stride < c->head_dim))
    return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
// whether bytes lie between the first and the last of the cache's keys, or of its values
inline bool in_cache(const asf_kv_cache *c, const void *p, size_t bytes) {
  const size_t span = 2 * ((size_t)(c->pages - 1) * c->page_stride + (size_t)(c->page - 1) * c->token_stride +
                           (size_t)(c->heads - 1) * c->head_stride + c->head_dim);
  return overlap(p, bytes, c->k, span) || overlap(p, bytes, c->v, span);
}
inline asf_status check_requests(const int32_t *table, int max_pages, int R, const int32_t *lens, const int32_t *begin, int T) {
  if (!table || !lens || !begin) return ASF_ERR_INVALID_ARG;
  if (max_pages < 1 || R < 1 || R > ASF_MAX_BATCH || T < 1 || T > ASF_MAX_BATCH) return ASF_ERR_INVALID_ARG;
  return ASF_OK;
}
inline asf_status check_tables(const int32_t *table, int max_pages, int page, const int32_t *lens, const int32_t *begin) {
  if ((int64_t)max_pages * page > ASF_MAX_KEYS) return ASF_ERR_UNSUPPORTED;
  if (!al4(table) || !al4(lens) || !al4(begin)) return ASF_ERR_MISALIGNED;
  return ASF_OK;
}

// The request whose range holds a token, and the token's position in it; r is
// negative behind the last range and between ranges.  A lane of every warp reads
// one request's range and length, all at once: the chain to the first store is
// two loads (these, then the table) instead of four.  Whole warps call it.
struct Place {
  int r;
  int64_t pos;                         // negative: the request's own numbers are bad
};
__device__ __forceinline__ Place place_of(const int32_t *lens, const int32_t *begin, int R, int T, int tok, int32_t *err,
                                          bool flags) {
  const int lane = threadIdx.x & 31;
  int b0 = 0, b1 = T, n = 0;
  if (lane < R) {
    b0 = ld_cg_i32(begin + lane);
    b1 = ld_cg_i32(begin + lane + 1);
    n = ld_cg_i32(lens + lane);
  }
  const bool bad = __any_sync(0xffffffffu, b0 < 0 || b1 < b0 || b1 > T);
  if (bad && flags) flag_error(err, kErrIndex);
  int r = 0;
  for (int q = 0; q < R; ++q) r += tok >= __shfl_sync(0xffffffffu, b1, q);
  const int t0 = __shfl_sync(0xffffffffu, b0, r & 31), len = __shfl_sync(0xffffffffu, n, r & 31);
  if (r >= R || tok < t0) return {-1, -1};
  return {r, t0 >= 0 && len >= 0 ? (int64_t)len + (tok - t0) : -1};
}

}  // namespace asf
