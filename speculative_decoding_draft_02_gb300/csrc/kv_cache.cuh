// kv_cache.cuh — checks of a paged KV cache shared by its kernels.
#pragma once
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
