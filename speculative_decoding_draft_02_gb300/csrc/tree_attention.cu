// tree_attention.cu — attention of every request's drafted tree (or chain, or
// single token) over its paged KV cache.
//
//   s_p = scale * q . K_p,  out = sum_p e^{s_p} V_p / sum_p e^{s_p}
// over p < ctx, and p = ctx + j for the nodes j in the row's ancestor mask.
#include <cuda_fp8.h>

#include "kv_cache.cuh"

DSPARK_DECLARE_STATUS(s_status_attention)

namespace {

struct AttnArgs {
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  int64_t page_stride, token_stride, head_stride;
  int n_pages, page_shift, heads, dim;
  int R, heads_q, max_nodes, n_rows, max_pages;
  const bf16 *q;
  int64_t q_row, q_head;
  const int *ctx, *row_start;
  const uint64_t *anc;
  const int *block_table;
  float scale;
  bf16 *out;
  int64_t out_row, out_head;
  float *lse;
};

template <int TYPE>
__device__ __forceinline__ float element(const uint8_t *base, int64_t i) {
  if constexpr (TYPE == DSPARK_KV_E4M3) {
    __nv_fp8_e4m3 x;
    x.__x = base[i];
    return (float)x;
  } else {
    return __bfloat162float(reinterpret_cast<const bf16 *>(base)[i]);
  }
}

// Block (row, head): four warps stride over the tokens, a lane holding dim / 32
// elements, each warp with its own running maximum and sum; joined at the end.
template <int TYPE, int D>
__global__ void __launch_bounds__(128) tree_attention_rows(const AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int row = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (row >= a.row_start[a.R] || row < a.row_start[0]) return;
  int lo = 0, hi = a.R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.row_start[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const int r = lo, row0 = a.row_start[r], node = row - row0;
  int n = a.row_start[r + 1] - row0;
  if (n > a.max_nodes) {
    if (threadIdx.x == 0) dspark_set_status(DSPARK_ERR_LENGTH);
    n = a.max_nodes;
  }
  if (node >= n) return;
  int64_t ctx = max(a.ctx[r], 0), total = ctx + n;
  const int64_t most = (int64_t)a.max_pages << a.page_shift;
  if (total > most) {
    if (threadIdx.x == 0) dspark_set_status(DSPARK_ERR_LENGTH);
    total = most;
    ctx = min(ctx, total);
  }
  const uint64_t mask = a.anc ? a.anc[row] : (2ull << node) - 1;
  const int kv = h / (a.heads_q / a.heads);
  const float ks = a.k_scale ? a.k_scale[kv] : 1.0f, vs = a.v_scale ? a.v_scale[kv] : 1.0f;
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e)
    q[e] = __bfloat162float(a.q[row * a.q_row + h * a.q_head + lane + 32 * e]) * a.scale * ks;
  float m = -INFINITY, l = 0.0f;
  bool any = false;
  for (int64_t p = warp; p < total; p += 4) {
    if (p >= ctx && !((mask >> (p - ctx)) & 1)) continue;
    any = true;
    const int page = a.block_table[(size_t)r * a.max_pages + (p >> a.page_shift)];
    const bool in = page >= 0 && page < a.n_pages;
    if (!in) dspark_set_status(DSPARK_ERR_PAGES);
    const int64_t at = in ? page * a.page_stride + (p & ((1 << a.page_shift) - 1)) * a.token_stride +
                                kv * a.head_stride
                          : 0;
    float s = 0.0f;
    for (int e = 0; e < E; ++e)
      s += in ? q[e] * element<TYPE>(a.k, at + lane + 32 * e) : 0.0f;
    s = warp_sum(s);
    const float top = fmaxf(m, s), keep = m == top ? 1.0f : __expf(m - top);
    const float w = __expf(s - top);
    l = l * keep + w;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * keep + (in ? w * element<TYPE>(a.v, at + lane + 32 * e) : 0.0f);
    m = top;
  }
  const int seen = __syncthreads_or(any);
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float total_l = 0.0f;
  for (int w = 0; w < 4; ++w) total_l += sl[w] == 0.0f ? 0.0f : sl[w] * __expf(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.0f;
    for (int w = 0; w < 4; ++w) x += sl[w] == 0.0f ? 0.0f : so[w][d] * __expf(sm[w] - top);
    a.out[row * a.out_row + h * a.out_head + d] =
        __float2bfloat16_rn(seen ? x / total_l * vs : 0.0f);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(size_t)row * a.heads_q + h] = seen ? top + logf(total_l) : -INFINITY;
}

}  // namespace

extern "C" size_t dspark_tree_attention_workspace_bytes(const dspark_kv_cache *cache, int32_t R,
                                                        int32_t heads_q, int32_t max_nodes) {
  if (!dspark_kv_cache_ok(cache) || R < 1 || heads_q < 1 || heads_q % cache->heads ||
      heads_q / cache->heads > 64 || max_nodes < 1 || max_nodes > DSPARK_MAX_NODES)
    return 0;
  return 256;
}

extern "C" int dspark_tree_attention(const dspark_kv_cache *cache, int32_t R, int32_t heads_q,
                                     int32_t max_nodes, int32_t n_rows, int32_t max_pages,
                                     const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                     const int32_t *ctx, const int32_t *row_start,
                                     const uint64_t *anc, const int32_t *block_table, float scale,
                                     void *out, int64_t out_row_stride, int64_t out_head_stride,
                                     float *lse, void *workspace, size_t workspace_bytes,
                                     dspark_stream_t stream) {
  const size_t need = dspark_tree_attention_workspace_bytes(cache, R, heads_q, max_nodes);
  if (need == 0 || n_rows < 0 || max_pages < 1) return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  if (!q || !ctx || !row_start || !block_table ||
      !out || ((uintptr_t)q & 15) || ((uintptr_t)out & 1) || q_row_stride <= 0 ||
      q_head_stride <= 0 || q_row_stride % 8 || q_head_stride % 8 || out_row_stride <= 0 ||
      out_head_stride <= 0)
    return DSPARK_ERR_ARG;
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)
    return DSPARK_ERR_WORKSPACE;
  AttnArgs a;
  a.k = (const uint8_t *)cache->k;
  a.v = (const uint8_t *)cache->v;
  a.k_scale = cache->type == DSPARK_KV_E4M3 ? cache->k_scale : nullptr;
  a.v_scale = cache->type == DSPARK_KV_E4M3 ? cache->v_scale : nullptr;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
  a.heads = cache->heads;
  a.dim = cache->dim;
  a.R = R;
  a.heads_q = heads_q;
  a.max_nodes = max_nodes;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.q = (const bf16 *)q;
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.ctx = ctx;
  a.row_start = row_start;
  a.anc = anc;
  a.block_table = block_table;
  a.scale = scale;
  a.out = (bf16 *)out;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.lse = lse;
  const dim3 grid(n_rows, heads_q);
  if (cache->type == DSPARK_KV_E4M3) {
    if (cache->dim == 64) tree_attention_rows<DSPARK_KV_E4M3, 64><<<grid, 128, 0, stream>>>(a);
    else tree_attention_rows<DSPARK_KV_E4M3, 128><<<grid, 128, 0, stream>>>(a);
  } else {
    if (cache->dim == 64) tree_attention_rows<DSPARK_KV_BF16, 64><<<grid, 128, 0, stream>>>(a);
    else tree_attention_rows<DSPARK_KV_BF16, 128><<<grid, 128, 0, stream>>>(a);
  }
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(1);
  return DSPARK_OK;
}

int dspark_status_attention(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_attention, sizeof(int)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_attention, &zero, sizeof(int));
  }
  return v;
}
