// chunk_attention.cu — dspark_chunk_attention: checks, and the launches of
// chunk_attention.cuh.
#include "kv_cache.cuh"
#include "tcgen05_attn.cuh"
#include "tensor_map.cuh"

DSPARK_DECLARE_STATUS(s_status_chunk)

#include "chunk_attention.cuh"

namespace {

using chunk::Args;

struct Layout {
  size_t ml, desc, bytes;
};
Layout layout_of(int ctas, int dim) {
  Layout l;
  l.ml = dspark_align_up((size_t)ctas * 2 * 2 * chunk::BM * dim * sizeof(float), 256);
  l.desc = l.ml + dspark_align_up((size_t)ctas * 2 * 4 * chunk::BM * sizeof(float), 256);
  l.bytes = l.desc + dspark_align_up((size_t)ctas * 8 * sizeof(int), 256);
  return l;
}

// Few rows leave the 128-row tiles empty: up to 32 of them (nodes x query heads of a KV
// head) the tree attention, which has the tokens there, is the faster one.  64 requests over
// 512 to 4096 tokens, 8 KV heads, tree and chunks: 32 rows 82 and 90 us, 64 rows 119 and 91;
// 8 bits: 91 and 114, 186 and 114.  One request over 4000: 32 rows 22 and 23, 64 rows 26 and 22.
bool as_tree(int max_rows, int group) {
  return max_rows <= DSPARK_MAX_NODES && max_rows * group <= 32;
}

struct Launch {
  const dspark_kv_cache *cache;
  Args a;
  const void *q;
  int64_t q_row, q_head;
  int ctas;
  cudaStream_t stream;
};

template <int TYPE, int D>
int launch(const Launch &l) {
  using G = chunk::Geo<TYPE, D>;
  const dspark_kv_cache *c = l.cache;
  const Args &a = l.a;
  const uint64_t size = G::FP8 ? 1 : 2;
  const uint64_t dims[4] = {(uint64_t)D, (uint64_t)c->page_size, (uint64_t)c->heads,
                            (uint64_t)c->n_pages};
  const uint64_t strides[3] = {c->token_stride * size, c->head_stride * size,
                               c->page_stride * size};
  const uint32_t rows = c->page_size < chunk::BT ? c->page_size : chunk::BT;
  const uint32_t box[4] = {G::FP8 ? (uint32_t)D : 64u, rows, 1, 1};
  const CUtensorMapDataType type =
      G::FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle swizzle =
      G::FP8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t q_dims[3] = {(uint64_t)D, (uint64_t)(a.heads * a.group), (uint64_t)a.n_rows};
  const uint64_t q_strides[2] = {(uint64_t)l.q_head * 2, (uint64_t)l.q_row * 2};
  const uint32_t q_box[3] = {64, (uint32_t)a.group, (uint32_t)a.nodes_tile};
  CUtensorMap tk, tv, tq;
  if (!make_map(&tk, type, c->k, dims, strides, box, swizzle) ||
      !make_map(&tv, type, c->v, dims, strides, box, swizzle) ||
      !make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.q, q_dims, q_strides, q_box,
                CU_TENSOR_MAP_SWIZZLE_128B))
    return DSPARK_ERR_CUDA;
  auto kernel = chunk::chunk_attention_kernel<TYPE, D>;
  static DsparkPerDevice attr;
  if (dspark_per_device(attr, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    G::SMEM_BYTES) == cudaSuccess
                   ? 1
                   : -1;
      }) < 0)
    return DSPARK_ERR_CUDA;
  if (dspark_launch_pdl(kernel, dim3(l.ctas), dim3(G::THREADS), G::SMEM_BYTES, l.stream, tk, tv,
                        tq, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  // Requests too short to be cut (a table has no place for two pieces) leave nothing to join.
  if (((int64_t)a.max_pages << a.page_shift) <= (2 * chunk::MIN_PIECE - 1) * chunk::BT) {
    DSPARK_CHECK_LAUNCH();
    dspark_count_launches(1);
    return DSPARK_OK;
  }
  if (dspark_launch_pdl(chunk::chunk_attention_join<D>, dim3(l.ctas, 2, D / 16), dim3(chunk::BM),
                        0, l.stream, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  DSPARK_CHECK_LAUNCH();
  dspark_count_launches(2);
  return DSPARK_OK;
}

}  // namespace

extern "C" size_t dspark_chunk_attention_workspace_bytes(const dspark_kv_cache *cache, int32_t R,
                                                         int32_t heads_q, int32_t max_rows) {
  if (!dspark_kv_cache_ok(cache) || R < 1 || heads_q < 1 || heads_q % cache->heads ||
      heads_q / cache->heads > 64 || max_rows < 1)
    return 0;
  const size_t own = layout_of(dspark_sm_count(), cache->dim).bytes;
  if (!as_tree(max_rows, heads_q / cache->heads)) return own;
  const size_t tree = dspark_tree_attention_workspace_bytes(cache, R, heads_q, max_rows);
  return own > tree ? own : tree;
}

extern "C" int dspark_chunk_attention(const dspark_kv_cache *cache, int32_t R, int32_t heads_q,
                                      int32_t max_rows, int32_t n_rows, int32_t max_pages,
                                      const void *q, int64_t q_row_stride, int64_t q_head_stride,
                                      const int32_t *ctx, const int32_t *row_start,
                                      const int32_t *block_table, float scale, void *out,
                                      int64_t out_row_stride, int64_t out_head_stride, float *lse,
                                      void *workspace, size_t workspace_bytes,
                                      dspark_stream_t stream) {
  const size_t need = dspark_chunk_attention_workspace_bytes(cache, R, heads_q, max_rows);
  if (need == 0 || n_rows < 0 || max_pages < 1) return DSPARK_ERR_ARG;
  if (n_rows == 0) return DSPARK_OK;
  const int64_t most = (int64_t)1 << 39;  // elements: a tensor map's strides are below 2^40 bytes
  if (!q || !ctx || !row_start || !block_table || !out ||
      (((uintptr_t)q | (uintptr_t)out) & 15) || q_row_stride <= 0 || q_head_stride <= 0 ||
      q_row_stride >= most || q_head_stride >= most || q_row_stride % 8 || q_head_stride % 8 ||
      out_row_stride <= 0 || out_head_stride <= 0 || out_row_stride >= most ||
      out_head_stride >= most || out_row_stride % 8 || out_head_stride % 8)
    return DSPARK_ERR_ARG;
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)
    return DSPARK_ERR_WORKSPACE;
  const int64_t tree_out = (int64_t)1 << 24;  // the tree attention's limit
  if (as_tree(max_rows, heads_q / cache->heads) && out_row_stride <= tree_out &&
      out_head_stride <= tree_out)
    return dspark_tree_attention(cache, R, heads_q, max_rows, n_rows, max_pages, q, q_row_stride,
                                 q_head_stride, ctx, row_start, nullptr, block_table, scale, out,
                                 out_row_stride, out_head_stride, lse, workspace, workspace_bytes,
                                 stream);
  Launch l;
  l.cache = cache;
  l.q = q;
  l.q_row = q_row_stride;
  l.q_head = q_head_stride;
  l.ctas = dspark_sm_count();
  l.stream = stream;
  const bool fp8 = cache->type == DSPARK_KV_E4M3;
  const Layout at = layout_of(l.ctas, cache->dim);
  const int64_t size = dspark_kv_bytes(cache->type);
  Args &a = l.a;
  a.R = R;
  a.heads = cache->heads;
  a.group = heads_q / cache->heads;
  a.nodes_tile = chunk::BM / a.group;
  a.max_rows = max_rows;
  a.n_rows = n_rows;
  a.max_pages = max_pages;
  a.page_shift = 31 - __builtin_clz((unsigned)cache->page_size);
  a.n_pages = cache->n_pages;
  a.ctx = ctx;
  a.row_start = row_start;
  a.block_table = block_table;
  a.k_scale = fp8 ? cache->k_scale : nullptr;
  a.v_scale = fp8 ? cache->v_scale : nullptr;
  a.v = (const uint8_t *)cache->v;
  a.page_bytes = cache->page_stride * size;
  a.token_bytes = cache->token_stride * size;
  a.head_bytes = cache->head_stride * size;
  a.scale = scale;
  a.out = (bf16 *)out;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.wide = ((uintptr_t)out & 31) == 0 && out_row_stride % 16 == 0 && out_head_stride % 16 == 0;
  a.lse = lse;
  a.part_o = (float4 *)workspace;
  a.part_ml = (float *)((uint8_t *)workspace + at.ml);
  a.desc = (int *)((uint8_t *)workspace + at.desc);
  if (fp8)
    return cache->dim == 64 ? launch<DSPARK_KV_E4M3, 64>(l) : launch<DSPARK_KV_E4M3, 128>(l);
  return cache->dim == 64 ? launch<DSPARK_KV_BF16, 64>(l) : launch<DSPARK_KV_BF16, 128>(l);
}

int dspark_status_chunk(int clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, s_status_chunk, sizeof(int)) != cudaSuccess) return DSPARK_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    cudaMemcpyToSymbol(s_status_chunk, &zero, sizeof(int));
  }
  return v;
}
