// Host checks that the entry points of the key/value cache and of a serving
// step's other operators share.
#pragma once

#include "kv_device.hpp"

namespace w4k {

inline bool kv_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline w4a16_status_t kv_launched(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

inline bool page_supported(int page) { return page == 16 || page == 32 || page == 64 || page == 128 || page == 256; }

// sizes of a cache, without its pointers
inline w4a16_status_t check_cache(const w4a16_kv_cache_t* c) {
  if (!c) return W4A16_ERR_NULL;
  if (c->type != W4A16_KV_INT8 && c->type != W4A16_KV_FP8) return W4A16_ERR_UNSUPPORTED;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return W4A16_ERR_UNSUPPORTED;
  if (!page_supported(c->page)) return W4A16_ERR_UNSUPPORTED;
  if (c->heads < 1 || c->heads > W4A16_KV_MAX_HEADS || c->pages < 0) return W4A16_ERR_SHAPE;
  if ((int64_t)c->pages * c->page > 0x7FFFFFFFLL || (int64_t)c->pages * c->heads > 0x7FFFFFFFLL)
    return W4A16_ERR_SHAPE;
  return W4A16_OK;
}

inline w4a16_status_t check_cache_pointers(const w4a16_kv_cache_t* c) {
  if (!c->k || !c->v || !c->k_scales || !c->v_scales) return W4A16_ERR_NULL;
  if (!kv_aligned(c->k, 16) || !kv_aligned(c->v, 16) || !kv_aligned(c->k_scales, 2) || !kv_aligned(c->v_scales, 2))
    return W4A16_ERR_ALIGN;
  return W4A16_OK;
}

inline KvCache device_cache(const w4a16_kv_cache_t* c) {
  return KvCache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scales, c->v_scales, c->pages,
                 c->heads, __builtin_ctz((unsigned)c->page)};
}

}  // namespace w4k
