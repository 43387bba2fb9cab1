// attn_cache_host.h -- host-side checks of pointers and caches that the entry points of the generation path share.
#pragma once

#include <cstdint>

#include "attn_gb300.h"

namespace attn {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Checks of a cache that every entry point that takes one makes.
inline int check_cache(const attn_kv_cache& c, int H_kv, int d) {
  if (c.dtype != ATTN_CACHE_BF16 && c.dtype != ATTN_CACHE_E4M3) return ATTN_ERR_UNSUPPORTED;
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)))
    return ATTN_ERR_UNSUPPORTED;
  if (c.num_pages <= 0) return ATTN_ERR_SHAPE;
  const bool e4m3 = c.dtype == ATTN_CACHE_E4M3;
  const int64_t size = e4m3 ? 1 : 2;
  // (the tensor map's strides are below 2^40 bytes)
  if (c.page_stride < static_cast<int64_t>(H_kv) * c.page_size * d ||
      c.page_stride * size % 16 != 0 || c.page_stride >= (1ll << 39))
    return ATTN_ERR_SHAPE;
  if (!c.k || !c.v || (e4m3 && (!c.k_scale || !c.v_scale))) return ATTN_ERR_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) ||
      (e4m3 && (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))))
    return ATTN_ERR_ALIGN;
  return ATTN_OK;
}

inline int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

}  // namespace attn
