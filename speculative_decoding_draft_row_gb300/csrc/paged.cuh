// paged.cuh - what the calls on a paged key-value cache share: the checks of its description.
#pragma once

#include <algorithm>

#include "launch.cuh"
#include "rope.cuh"

namespace tfd_paged {

inline int elem_bytes(const tfd_kv_pages& c) { return c.fmt == TFD_KV_E4M3 ? 1 : 2; }

// Bytes from the first to the last element of k (and of v); -1 where that passes 2^48, or where the
// strides let two vectors share an element.
inline int64_t cache_bytes(const tfd_kv_pages& c) {
  int64_t n[3] = {c.pages, c.page_size, c.heads};
  int64_t s[3] = {c.page_stride, c.token_stride, c.head_stride};
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return s[a] < s[b]; });
  unsigned __int128 reach = (unsigned)c.dim;  // elements that the smaller strides span
  for (int i : order) {
    if (n[i] == 1) continue;
    if ((unsigned __int128)s[i] < reach) return -1;
    reach += (unsigned __int128)s[i] * (uint64_t)(n[i] - 1);
  }
  reach *= (unsigned)elem_bytes(c);
  return reach >> 48 ? -1 : (int64_t)reach;
}

inline tfd_status check_cache(const tfd_kv_pages* p) {
  using tfd_host::aligned;
  if (!p || !p->k || !p->v) return TFD_ERR_INVALID;
  const tfd_kv_pages& c = *p;
  if (c.fmt != TFD_KV_BF16 && c.fmt != TFD_KV_E4M3) return TFD_ERR_INVALID;
  if (c.pages < 1 || c.page_size < 1 || c.page_size > TFD_MAX_PAGE || c.heads < 1 ||
      c.heads > 1024 || (int64_t)c.pages * c.page_size > 2147483647)
    return TFD_ERR_INVALID;
  if (c.dim != 64 && c.dim != 128) return TFD_ERR_UNSUPPORTED;
  const int64_t step = 16 / elem_bytes(c);
  if (c.page_stride < 1 || c.token_stride < 1 || c.head_stride < 1 || c.page_stride % step ||
      c.token_stride % step || c.head_stride % step)
    return TFD_ERR_INVALID;
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return TFD_ERR_INVALID;
  if (c.fmt == TFD_KV_E4M3 &&
      (!c.k_scales || !c.v_scales || !aligned(c.k_scales, 4) || !aligned(c.v_scales, 4)))
    return TFD_ERR_INVALID;
  return cache_bytes(c) < 0 ? TFD_ERR_INVALID : TFD_OK;
}

// Whether a range shares a byte with the cache (its scales included).
inline bool overlaps_cache(const tfd_kv_pages& c, const void* p, int64_t bytes) {
  using tfd_host::overlap;
  const int64_t kv = cache_bytes(c);
  if (overlap(p, bytes, c.k, kv) || overlap(p, bytes, c.v, kv)) return true;
  if (c.fmt != TFD_KV_E4M3) return false;
  const int64_t sb = (int64_t)c.pages * c.page_size * c.heads * 4;
  return overlap(p, bytes, c.k_scales, sb) || overlap(p, bytes, c.v_scales, sb);
}

inline bool check_qk(int qk, float eps, float rope_base) {
  if (qk & ~(TFD_QK_NORM | TFD_QK_ROPE)) return false;
  if ((qk & TFD_QK_NORM) && !(eps >= 0.0f)) return false;
  return !(qk & TFD_QK_ROPE) || rope_base > 0.0f;
}

}  // namespace tfd_paged
