// kv_cache.cuh — checks and addresses of a paged KV cache shared by its kernels.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

static inline int dspark_kv_bytes(int type) { return type == DSPARK_KV_E4M3 ? 1 : 2; }

// The stated limits of dspark_kv_cache: what the kernels' index arithmetic and
// the copies' alignment rest on.
static inline bool dspark_kv_cache_ok(const dspark_kv_cache *c) {
  if (!c || !c->k || !c->v || c->n_pages < 1 || c->heads < 1) return false;
  if (c->dim != 64 && c->dim != 128) return false;
  if (c->type != DSPARK_KV_BF16 && c->type != DSPARK_KV_E4M3) return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return false;
  if (((uintptr_t)c->k | (uintptr_t)c->v) & 15) return false;
  const int64_t size = dspark_kv_bytes(c->type);
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s <= 0 || s >= (int64_t)1 << 40 || s * size % 16 || s * size >= (int64_t)1 << 40) return false;
  return true;
}

// A cache as kernels take it, strides in bytes.
struct CacheView {
  uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t page_bytes, token_bytes, head_bytes;
  int n_pages, page_shift, heads, dim;
};

static inline CacheView view_of(const dspark_kv_cache *c) {
  const int64_t size = dspark_kv_bytes(c->type);
  CacheView v;
  v.k = (uint8_t *)c->k;
  v.v = (uint8_t *)c->v;
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.page_bytes = c->page_stride * size;
  v.token_bytes = c->token_stride * size;
  v.head_bytes = c->head_stride * size;
  v.n_pages = c->n_pages;
  v.page_shift = 31 - __builtin_clz((unsigned)c->page_size);
  v.heads = c->heads;
  v.dim = c->dim;
  return v;
}

// Two f32 values as e4m3, saturating at +-448 (the conversion's finite form).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
