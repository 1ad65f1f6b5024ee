// The paged cache's checks, shared by its writer, its reader and attention over it.
#pragma once

#include "device_block.h"

namespace svdq {
namespace {

// sizes and strides
inline svdq_status cache_sizes(const svdq_kv_cache& c) {
  if (c.format < SVDQ_KV_VALUES || c.format > SVDQ_KV_FP8) return SVDQ_ERR_UNSUPPORTED;
  const bool scaled = c.format != SVDQ_KV_VALUES;
  if (c.pages < 1 || c.pages > (1 << 28) || c.page < 16 || c.page > 256 || (c.page & (c.page - 1)) != 0 ||
      c.heads < 1 || c.heads > 65536 || c.D < 16 || c.D > SVDQ_KV_MAX_HEAD_DIM || c.D % 16 != 0)
    return SVDQ_ERR_SHAPE;
  const int64_t rows = (int64_t)c.heads * c.page, most = (int64_t)1 << 34;
  if (c.k_page < rows * c.D || c.v_page < rows * c.D || c.k_page > most || c.v_page > most ||
      (scaled && (c.scale_page < rows || c.scale_page > most)))
    return SVDQ_ERR_SHAPE;
  const int64_t unit = scaled ? 16 : 8;
  if (c.k_page % unit != 0 || c.v_page % unit != 0 || (scaled && c.scale_page % 4 != 0)) return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

inline svdq_status cache_check(const svdq_kv_cache& c) {
  if (!c.k || !c.v) return SVDQ_ERR_ARG;
  const svdq_status s = cache_sizes(c);
  if (s != SVDQ_OK) return s;
  if (c.format != SVDQ_KV_VALUES && (!c.k_scale || !c.v_scale)) return SVDQ_ERR_ARG;
  if (!on16(c.k) || !on16(c.v) || !on16(c.k_scale) || !on16(c.v_scale)) return SVDQ_ERR_ALIGN;
  return SVDQ_OK;
}

[[maybe_unused]] inline bool table_fits(const svdq_kv_cache& c, int32_t B, int32_t T, int64_t row) {
  return B >= 1 && T >= 1 && (int64_t)T * c.page <= (1 << 24) && (B == 1 || row >= T);
}

}  // namespace
}  // namespace svdq
